// Routing of tokens to experts and its gradient.
//
// One warp serves a token.  Lane l holds EPL consecutive experts (EPL * 32 >=
// E), so that the lowest lane of those that tie is also the lowest expert.
// The choice goes by 32-bit keys that compare as the numbers do; 0 is "never":
// the k best are found one after another by a warp-wide maximum of the lanes'
// own best keys and a ballot.  Scores are computed where they are compared; of
// the chosen experts each is computed again by a lane of its own, which then
// also holds the slot's index and weight.

#include "ddp_reducer.h"

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "ddp_device.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxExperts = 512;
constexpr unsigned kAll = 0xffffffffu;

struct RouteParams {
    const void* logits;
    const float* bias;
    const uint8_t* mask;
    int32_t* indices;
    float* weights;
    int32_t* counts;
    const float* grad_weights;   // backward
    void* grad_logits;
    long long tokens, stride, grad_stride;
    int E, k, groups, top_groups;
    int softmax, renorm;
    float scale;
};

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(uint16_t x) { return ddpk::dev::widen1(x); }
template <typename T> __device__ __forceinline__ T narrow(float x);
template <> __device__ __forceinline__ float narrow<float>(float x) { return x; }
template <> __device__ __forceinline__ uint16_t narrow<uint16_t>(float x) {
    return static_cast<uint16_t>(__float_as_uint(ddpk::dev::round_bf16(x)) >> 16);
}

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }

// A key that orders like the number (-0 equal to +0); 0 for -inf and NaN.
__device__ __forceinline__ uint32_t key_of(float x) {
    if (!(x > neg_inf())) return 0;
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b ^ (static_cast<int>(b) < 0 ? 0xffffffffu : 0x80000000u);
}

__device__ __forceinline__ float number_of(uint32_t key) {
    return key == 0 ? neg_inf() : __uint_as_float(key ^ (key & 0x80000000u ? 0x80000000u : 0xffffffffu));
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(kAll, x, o);
    return x;
}

__device__ __forceinline__ float sigmoid(float x) { return __fdiv_rn(1.0f, __fadd_rn(1.0f, expf(-x))); }

// Largest number and sum of exponentials of a row (its NaN and -inf left out).
template <int EPL>
__device__ __forceinline__ void softmax_stats(const float (&x)[EPL], float& top, float& sum) {
    uint32_t best = 0;
#pragma unroll
    for (int j = 0; j < EPL; ++j) best = max(best, key_of(x[j]));
    top = number_of(__reduce_max_sync(kAll, best));
    float part = 0.0f;
#pragma unroll
    for (int j = 0; j < EPL; ++j) part += x[j] > neg_inf() ? expf(x[j] - top) : 0.0f;
    sum = warp_sum(part);
}

template <int EPL, typename T>
__device__ __forceinline__ void load_row(const T* row, int E, float (&x)[EPL]) {
    const int e0 = (threadIdx.x & 31) * EPL;
#pragma unroll
    for (int j = 0; j < EPL; ++j) x[j] = e0 + j < E ? widen(row[e0 + j]) : neg_inf();
}

template <int EPL, typename T>
__global__ void __launch_bounds__(kThreads)
route_kernel(const __grid_constant__ RouteParams a) {
    __shared__ int hist[kMaxExperts];
    __shared__ float rows[kWarps][EPL * 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int E = a.E, k = a.k;
    if (a.counts)
        for (int i = threadIdx.x; i < E; i += kThreads) hist[i] = 0;
    ddpk::dev::pdl_wait();
    ddpk::dev::pdl_trigger();
    __syncthreads();

    float bias[EPL];
#pragma unroll
    for (int j = 0; j < EPL; ++j) bias[j] = a.bias && lane * EPL + j < E ? a.bias[lane * EPL + j] : 0.0f;
    const bool by_logit = !a.bias && a.groups == 1;

    for (long long t = static_cast<long long>(blockIdx.x) * kWarps + warp; t < a.tokens;
         t += static_cast<long long>(gridDim.x) * kWarps) {
        int index = -1;               // lane r: slot r
        float score = 0.0f;
        bool bad = false;
        if (!a.mask || a.mask[t]) {
            const T* row = static_cast<const T*>(a.logits) + t * a.stride;
            float x[EPL];
            uint32_t key[EPL];
            load_row<EPL>(row, E, x);
            float top = 0.0f, sum = 1.0f;
#pragma unroll
            for (int j = 0; j < EPL; ++j)
                bad |= !(x[j] == x[j]) || (a.softmax && x[j] == -neg_inf());
            bad = __any_sync(kAll, bad);
            if (a.softmax) softmax_stats<EPL>(x, top, sum);
#pragma unroll
            for (int j = 0; j < EPL; ++j) {
                float c = x[j];
                if (!by_logit) {
                    const float s = a.softmax ? __fdiv_rn(expf(x[j] - top), sum) : sigmoid(x[j]);
                    c = __fadd_rn(s, bias[j]);
                }
                key[j] = x[j] > neg_inf() ? key_of(c) : 0u;
            }

            if (a.groups > 1) {
                // lane g: the worth of group g, then whether it stays
                const int size = E / a.groups;
                float* c = rows[warp];
#pragma unroll
                for (int j = 0; j < EPL; ++j) c[lane * EPL + j] = number_of(key[j]);
                __syncwarp();
                uint32_t worth = 0;
                if (lane < a.groups) {
                    float a1 = neg_inf(), a2 = neg_inf();
                    for (int i = 0; i < size; ++i) {
                        const float y = c[lane * size + i];
                        a2 = fmaxf(a2, fminf(a1, y));
                        a1 = fmaxf(a1, y);
                    }
                    worth = max(key_of(size > 1 ? __fadd_rn(a1, a2) : a1), 1u);
                }
                __syncwarp();
                unsigned stay = 0;
                for (int r = 0; r < a.top_groups; ++r) {
                    const uint32_t best = __reduce_max_sync(kAll, worth);
                    const int g = __ffs(__ballot_sync(kAll, worth == best)) - 1;
                    stay |= 1u << g;
                    if (lane == g) worth = 0;
                }
#pragma unroll
                for (int j = 0; j < EPL; ++j) {
                    const int e = lane * EPL + j;
                    if (e < E && !(stay >> (e / size) & 1)) key[j] = 0;
                }
            }

            for (int r = 0; r < k; ++r) {
                uint32_t mine = 0;
                int at = 0;
#pragma unroll
                for (int j = EPL - 1; j >= 0; --j)
                    if (key[j] >= mine) { mine = key[j]; at = j; }
                const uint32_t best = __reduce_max_sync(kAll, mine);
                if (best == 0) break;
                const int from = __ffs(__ballot_sync(kAll, mine == best)) - 1;
                const int chosen = __shfl_sync(kAll, lane * EPL + at, from);
                if (lane == r) index = chosen;
#pragma unroll
                for (int j = 0; j < EPL; ++j)
                    if (lane * EPL + j == chosen) key[j] = 0;
            }
            if (index >= 0) {
                const float y = widen(row[index]);
                score = a.softmax ? __fdiv_rn(expf(y - top), sum) : sigmoid(y);
            }
        }
        float w = score;
        if (a.renorm) {
            const float total = warp_sum(score);
            w = total > 0.0f ? __fdiv_rn(score, total) : 0.0f;
        }
        w = __fmul_rn(w, a.scale);
        if (bad) w = __int_as_float(0x7fffffff);
        if (lane < k) {
            a.indices[t * k + lane] = index;
            a.weights[t * k + lane] = w;
            if (a.counts && index >= 0) atomicAdd(hist + index, 1);
        }
    }
    if (a.counts) {
        __syncthreads();
        for (int i = threadIdx.x; i < E; i += kThreads)
            if (hist[i]) atomicAdd(a.counts + i, hist[i]);
    }
}

// The gradient.  With D = sum over the slots of part_r, in the slots r
//   part_r = g_r w_r                          (weights as they are)
//   part_r = w_r (g_r - sum_l g_l w_l / scale)  (renormalised)
// sigmoid:  dx = part_r (1 - s_r) at the chosen, 0 elsewhere
// softmax:  dx = [chosen] part_r - s_i D; renormalised D is zero, and only the
//           chosen get a gradient
template <int EPL, typename T>
__global__ void __launch_bounds__(kThreads)
route_backward_kernel(const __grid_constant__ RouteParams a) {
    __shared__ float rows[kWarps][EPL * 32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int E = a.E, k = a.k;
    float* out = rows[warp];
    ddpk::dev::pdl_wait();
    ddpk::dev::pdl_trigger();
    for (long long t = static_cast<long long>(blockIdx.x) * kWarps + warp; t < a.tokens;
         t += static_cast<long long>(gridDim.x) * kWarps) {
        const T* row = static_cast<const T*>(a.logits) + t * a.stride;
        int index = -1;
        float part = 0.0f;
        if (lane < k) index = a.indices[t * k + lane];
        if (index < 0 || index >= E) index = -1;      // never an address past the row
        float w = 0.0f, g = 0.0f;
        if (index >= 0) {
            w = a.weights[t * k + lane];
            g = a.grad_weights[t * k + lane];
        }
        part = g * w;
        const float total = warp_sum(part);
        if (a.renorm) part = index >= 0 ? w * (g - total / a.scale) : 0.0f;
        if (!a.softmax && index >= 0) part *= 1.0f - sigmoid(widen(row[index]));
#pragma unroll
        for (int j = 0; j < EPL; ++j) out[j * 32 + lane] = 0.0f;
        __syncwarp();
        if (index >= 0) out[index] = part;
        __syncwarp();
        const bool whole = a.softmax && !a.renorm && __any_sync(kAll, index >= 0);
        float x[EPL], top = 0.0f, sum = 1.0f;
        if (whole) {
            load_row<EPL>(row, E, x);
            softmax_stats<EPL>(x, top, sum);
        }
        T* to = static_cast<T*>(a.grad_logits) + t * a.grad_stride;
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            const int e = lane * EPL + j;
            float d = out[e];
            if (whole && x[j] != neg_inf()) d -= expf(x[j] - top) / sum * total;
            if (e < E) to[e] = narrow<T>(d);
        }
        __syncwarp();
    }
}

template <typename T, int EPL>
cudaError_t launch_epl(bool backward, int grid, const RouteParams& a, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return backward ? cudaLaunchKernelEx(&cfg, route_backward_kernel<EPL, T>, a)
                    : cudaLaunchKernelEx(&cfg, route_kernel<EPL, T>, a);
}

template <typename T>
cudaError_t launch(bool backward, const RouteParams& a, cudaStream_t stream) {
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    const long long want = (a.tokens + kWarps - 1) / kWarps, most = 8LL * sms;
    const int grid = static_cast<int>(want < most ? want : most);
    if (a.E <= 32) return launch_epl<T, 1>(backward, grid, a, stream);
    if (a.E <= 64) return launch_epl<T, 2>(backward, grid, a, stream);
    if (a.E <= 128) return launch_epl<T, 4>(backward, grid, a, stream);
    if (a.E <= 256) return launch_epl<T, 8>(backward, grid, a, stream);
    return launch_epl<T, 16>(backward, grid, a, stream);
}

bool valid(const ddp_route_args* x) {
    return x && x->tokens >= 0 && x->experts >= 1 && x->experts <= kMaxExperts && x->row_stride >= x->experts &&
           (x->score == DDP_SCORE_SOFTMAX || x->score == DDP_SCORE_SIGMOID) && x->groups >= 1 && x->groups <= 32 &&
           x->experts % x->groups == 0 && x->top_groups >= 1 && x->top_groups <= x->groups && x->k >= 1 && x->k <= 32 &&
           x->k <= x->top_groups * (x->experts / x->groups) && std::isfinite(x->scale) && x->scale != 0.0f &&
           (x->dtype == DDP_F32 || x->dtype == DDP_BF16);
}

RouteParams params_of(const ddp_route_args* x) {
    RouteParams a = {};
    a.tokens = x->tokens;
    a.stride = x->row_stride;
    a.E = x->experts;
    a.k = x->k;
    a.groups = x->groups;
    a.top_groups = x->top_groups;
    a.softmax = x->score == DDP_SCORE_SOFTMAX;
    a.renorm = x->renorm != 0;
    a.scale = x->scale;
    return a;
}

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

}  // namespace

extern "C" {

int ddp_route(const ddp_route_args* x, const void* logits, const float* bias, const uint8_t* mask, int32_t* indices,
              float* weights, int32_t* counts, void* stream) {
    if (!valid(x)) return DDP_ERR_INVALID_ARG;
    if (x->tokens == 0) return DDP_OK;
    if (!logits || !indices || !weights) return DDP_ERR_INVALID_ARG;
    if (!aligned(logits, x->dtype == DDP_F32 ? 4 : 2) || !aligned(bias, 4) || !aligned(indices, 4) ||
        !aligned(weights, 4) || !aligned(counts, 4))
        return DDP_ERR_INVALID_ARG;
    RouteParams a = params_of(x);
    a.logits = logits;
    a.bias = bias;
    a.mask = mask;
    a.indices = indices;
    a.weights = weights;
    a.counts = counts;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = x->dtype == DDP_F32 ? launch<float>(false, a, st) : launch<uint16_t>(false, a, st);
    return e == cudaSuccess ? DDP_OK : DDP_ERR_CUDA;
}

int ddp_route_backward(const ddp_route_args* x, const void* logits, const int32_t* indices, const float* weights,
                       const float* grad_weights, void* grad_logits, int64_t grad_stride, void* stream) {
    if (!valid(x) || grad_stride < x->experts) return DDP_ERR_INVALID_ARG;
    if (x->tokens == 0) return DDP_OK;
    const uintptr_t size = x->dtype == DDP_F32 ? 4 : 2;
    if (!logits || !indices || !weights || !grad_weights || !grad_logits) return DDP_ERR_INVALID_ARG;
    if (!aligned(logits, size) || !aligned(grad_logits, size) || !aligned(indices, 4) || !aligned(weights, 4) ||
        !aligned(grad_weights, 4))
        return DDP_ERR_INVALID_ARG;
    RouteParams a = params_of(x);
    a.logits = logits;
    a.indices = const_cast<int32_t*>(indices);
    a.weights = const_cast<float*>(weights);
    a.grad_weights = grad_weights;
    a.grad_logits = grad_logits;
    a.grad_stride = grad_stride;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = x->dtype == DDP_F32 ? launch<float>(true, a, st) : launch<uint16_t>(true, a, st);
    return e == cudaSuccess ? DDP_OK : DDP_ERR_CUDA;
}

}  // extern "C"
