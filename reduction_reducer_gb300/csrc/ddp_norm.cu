// Layer norm over rows, and its gradient with the reduction of the weight's
// and the bias's over all rows.
//
// A row lies in the registers of a group of threads: a lane or more of a warp, or
// a whole CTA, eight elements a thread and chunk; mean and variance are two sums
// over the group, of the values and then of the squares of their distances from
// the mean (never a difference of large sums).  Rows longer than a CTA holds
// are read again for each sum.

#include "ddp_reducer.h"

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "ddp_rows.cuh"

namespace {

using namespace ddpk::rows;

constexpr int kThreads = 256;          // of a CTA that holds several rows
constexpr int kMaxWarps = 32;
constexpr int kRows = 4;               // backward: rows of a group at once
constexpr int kJoinLanes = 32;         // join_kernel: threads of a column
constexpr int kMaxParts = kSms * 5;    // backward: CTAs that sum the weight's gradient over rows of their own
constexpr int kMinRows = 8;            // and rows of each, at least

struct NormParams {
    const void* x;
    const void* weight;
    const void* bias;
    const void* grad;          // backward
    void* out;                 // y, or the gradient of x
    float* stats;              // mean and 1 / deviation of each row
    float* parts;              // backward: of each CTA, the weight's gradient and the bias's
    void* grad_weight;
    void* grad_bias;
    long long rows, x_stride, out_stride, grad_stride;
    int dim;
    float eps;
    int param_bf16;
    int accumulate;
    int nparts;
};

// Thread t's element j of chunk c in a group of G threads.
template <bool VEC>
__device__ __forceinline__ int place(int c, int j, int t, int G) {
    return VEC ? (c * G + t) * 8 + j : (c * 8 + j) * G + t;
}

// A thread's elements of a row; zeros past its end.
template <int CH, bool VEC, typename T>
__device__ __forceinline__ void load_row(const T* row, bool on, int t, int G, int dim, float (&x)[CH * 8]) {
    if constexpr (VEC) {
        Eight<T> raw[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int at = place<true>(c, 0, t, G);
            if (on && at < dim) raw[c].load_once(row + at);
            else raw[c].zero();
        }
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            float f[8];
            raw[c].get(f);
#pragma unroll
            for (int j = 0; j < 8; ++j) x[c * 8 + j] = f[j];
        }
    } else {
#pragma unroll
        for (int i = 0; i < CH * 8; ++i) {
            const int at = place<false>(i / 8, i % 8, t, G);
            x[i] = on && at < dim ? widen(row[at]) : 0.0f;
        }
    }
}

template <int CH, bool VEC, typename T>
__device__ __forceinline__ void store_row(T* row, int t, int G, int dim, const float (&x)[CH * 8]) {
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        if constexpr (VEC) {
            const int at = place<true>(c, 0, t, G);
            float f[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = x[c * 8 + j];
            Eight<T> raw;
            raw.put(f);
            if (at < dim) raw.store_once(row + at);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int at = place<false>(c, j, t, G);
                if (at < dim) row[at] = narrow<T>(x[c * 8 + j]);
            }
        }
    }
}

// Eight of a parameter vector, from an element of the thread's on.
template <bool VEC>
__device__ __forceinline__ void load_param(const void* p, int bf16, int c, int t, int G, int dim, float (&f)[8]) {
    if constexpr (VEC) {
        const int at = place<true>(c, 0, t, G);
        if (at >= dim) {
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = 0.0f;
        } else if (bf16) {
            Eight<uint16_t> raw;
            raw.load(static_cast<const uint16_t*>(p) + at);
            raw.get(f);
        } else {
            Eight<float> raw;
            raw.load(static_cast<const float*>(p) + at);
            raw.get(f);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int at = place<false>(c, j, t, G);
            f[j] = at >= dim ? 0.0f : bf16 ? widen(static_cast<const uint16_t*>(p)[at]) : static_cast<const float*>(p)[at];
        }
    }
}

// Over a group of LANES lanes, or (LANES = 0) over the CTA through `shared`
// [kMaxWarps], which no thread may still be reading.
template <int LANES>
__device__ __forceinline__ float group_sum(float x, float* shared) {
    if constexpr (LANES > 0) {
        return lanes_sum<LANES>(x);
    } else {
        const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
        x = lanes_sum<32>(x);
        if (lane == 0) shared[threadIdx.x >> 5] = x;
        __syncthreads();
        return lanes_sum<32>(lane < warps ? shared[lane] : 0.0f);
    }
}

__device__ __forceinline__ float param_at(const void* p, int bf16, int at) {
    return bf16 ? widen(static_cast<const uint16_t*>(p)[at]) : static_cast<const float*>(p)[at];
}

// ---------------------------------------------------------------- forward

template <typename T, int LANES, int CH, bool VEC>
__global__ void __launch_bounds__(LANES ? kThreads : 1024) norm_kernel(const __grid_constant__ NormParams p) {
    __shared__ float shared[2][kMaxWarps];
    const int G = LANES ? LANES : blockDim.x, t = threadIdx.x % G;
    const int groups = LANES ? kThreads / LANES : 1, group = LANES ? threadIdx.x / LANES : 0;
    ddpk::dev::pdl_wait();
    ddpk::dev::pdl_trigger();
    const long long stride = static_cast<long long>(gridDim.x) * groups;
    // all groups of a warp take as many rounds, for their sums' shuffles
    for (long long r0 = static_cast<long long>(blockIdx.x) * groups; r0 < p.rows; r0 += stride) {
        const long long row = r0 + group;
        const bool on = row < p.rows;
        float x[CH * 8];
        load_row<CH, VEC>(static_cast<const T*>(p.x) + row * p.x_stride, on, t, G, p.dim, x);
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < CH * 8; ++i) sum += x[i];
        const float mean = __fdiv_rn(group_sum<LANES>(sum, shared[0]), static_cast<float>(p.dim));
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < CH * 8; ++i) {
            x[i] -= mean;
            if (place<VEC>(i / 8, i % 8, t, G) < p.dim) sum = fmaf(x[i], x[i], sum);
        }
        const float variance = __fdiv_rn(group_sum<LANES>(sum, shared[1]), static_cast<float>(p.dim));
        const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(variance + p.eps));
        if (on && t == 0) *reinterpret_cast<float2*>(p.stats + 2 * row) = make_float2(mean, rstd);
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            float w[8], b[8];
            if (p.weight) load_param<VEC>(p.weight, p.param_bf16, c, t, G, p.dim, w);
            if (p.bias) load_param<VEC>(p.bias, p.param_bf16, c, t, G, p.dim, b);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                float y = x[c * 8 + j] * rstd;
                if (p.weight) y *= w[j];
                if (p.bias) y += b[j];
                x[c * 8 + j] = y;
            }
        }
        if (on) store_row<CH, VEC>(static_cast<T*>(p.out) + row * p.out_stride, t, G, p.dim, x);
    }
}

// Rows of any length, a CTA each, read three times.
template <typename T>
__global__ void __launch_bounds__(1024) norm_long_kernel(const __grid_constant__ NormParams p) {
    __shared__ float shared[2][kMaxWarps];
    ddpk::dev::pdl_wait();
    ddpk::dev::pdl_trigger();
    for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const T* const x = static_cast<const T*>(p.x) + row * p.x_stride;
        T* const y = static_cast<T*>(p.out) + row * p.out_stride;
        float sum = 0.0f;
        for (int i = threadIdx.x; i < p.dim; i += blockDim.x) sum += widen(x[i]);
        const float mean = __fdiv_rn(group_sum<0>(sum, shared[0]), static_cast<float>(p.dim));
        sum = 0.0f;
        for (int i = threadIdx.x; i < p.dim; i += blockDim.x) {
            const float d = widen(x[i]) - mean;
            sum = fmaf(d, d, sum);
        }
        const float variance = __fdiv_rn(group_sum<0>(sum, shared[1]), static_cast<float>(p.dim));
        const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(variance + p.eps));
        if (threadIdx.x == 0) *reinterpret_cast<float2*>(p.stats + 2 * row) = make_float2(mean, rstd);
        for (int i = threadIdx.x; i < p.dim; i += blockDim.x) {
            float v = (widen(x[i]) - mean) * rstd;
            if (p.weight) v *= param_at(p.weight, p.param_bf16, i);
            if (p.bias) v += param_at(p.bias, p.param_bf16, i);
            y[i] = narrow<T>(v);
        }
    }
}

// ---------------------------------------------------------------- backward

// Sums of eight values over a warp, for nine shuffles: each step halves the
// values that a lane keeps.  The sum of value i is in the lanes whose bits 4, 3
// and 2 spell i.
__device__ __forceinline__ float sum_eight(float (&v)[8]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int n = 4, o = 16; n; n /= 2, o /= 2) {
        const bool upper = lane & o;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float mine = upper ? v[i + n] : v[i], other = upper ? v[i] : v[i + n];
            v[i] = mine + __shfl_xor_sync(kAll, other, o);
        }
    }
    v[0] += __shfl_xor_sync(kAll, v[0], 2);
    return v[0] + __shfl_xor_sync(kAll, v[0], 1);
}

__device__ __forceinline__ int lane_of_eight(int i) { return (i & 4) << 2 | (i & 2) << 2 | (i & 1) << 2; }

// dx = r (g - mean(g) - xh mean(g xh)), g = dy w, xh = (x - mean) r; dw = sum dy xh
// and db = sum dy over the CTA's rows, a thread its columns.
template <typename T, int LANES, int CH, bool VEC>
__global__ void __launch_bounds__(LANES ? kThreads : 512) norm_backward_kernel(const __grid_constant__ NormParams p) {
    __shared__ float shared[2][kMaxWarps][8];
    __shared__ float columns[LANES ? 16 * kThreads : 1];
    const int G = LANES ? LANES : blockDim.x, t = threadIdx.x % G;
    const int groups = LANES ? kThreads / LANES : 1, group = LANES ? threadIdx.x / LANES : 0;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    ddpk::dev::pdl_wait();
    ddpk::dev::pdl_trigger();
    float dw[CH * 8], db[CH * 8], w[CH * 8];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
        float f[8];
        if (p.weight) load_param<VEC>(p.weight, p.param_bf16, c, t, G, p.dim, f);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            w[c * 8 + j] = p.weight ? f[j] : 1.0f;
            dw[c * 8 + j] = db[c * 8 + j] = 0.0f;
        }
    }
    const float over = __fdiv_rn(1.0f, static_cast<float>(p.dim));
    const int tile = groups * kRows;
    int phase = 0;
    for (long long r0 = static_cast<long long>(blockIdx.x) * tile; r0 < p.rows; r0 += static_cast<long long>(gridDim.x) * tile) {
        float x[kRows][CH * 8], dy[kRows][CH * 8], sums[2 * kRows];
        float2 stat[kRows];
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const long long row = r0 + r * groups + group;
            const bool on = row < p.rows;
            stat[r] = on ? *reinterpret_cast<const float2*>(p.stats + 2 * row) : make_float2(0.0f, 0.0f);
            load_row<CH, VEC>(static_cast<const T*>(p.x) + row * p.x_stride, on, t, G, p.dim, x[r]);
            load_row<CH, VEC>(static_cast<const T*>(p.grad) + row * p.grad_stride, on, t, G, p.dim, dy[r]);
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            float a = 0.0f, b = 0.0f;
#pragma unroll
            for (int i = 0; i < CH * 8; ++i) {
                x[r][i] = (x[r][i] - stat[r].x) * stat[r].y;
                db[i] += dy[r][i];
                dw[i] = fmaf(dy[r][i], x[r][i], dw[i]);          // zeros past the row's end: dy is zero there
                dy[r][i] *= w[i];
                a += dy[r][i];
                b = fmaf(dy[r][i], x[r][i], b);
            }
            sums[2 * r] = a;
            sums[2 * r + 1] = b;
        }
        if constexpr (LANES > 0) {
#pragma unroll
            for (int i = 0; i < 2 * kRows; ++i) sums[i] = lanes_sum<LANES>(sums[i]);
        } else {
            static_assert(kRows == 4, "eight sums");
            float s = sum_eight(sums);
            if ((lane & 3) == 0) shared[phase][warp][lane >> 2] = s;     // value lane / 4: its bits are the lane's 4, 3, 2
            __syncthreads();
#pragma unroll
            for (int i = 0; i < 8; ++i) sums[i] = lane < warps ? shared[phase][lane][i] : 0.0f;
            s = sum_eight(sums);
#pragma unroll
            for (int i = 0; i < 8; ++i) sums[i] = __shfl_sync(kAll, s, lane_of_eight(i));
            phase ^= 1;                                          // the other half is free: everyone is past this round's barrier
        }
#pragma unroll
        for (int r = 0; r < kRows; ++r) {
            const long long row = r0 + r * groups + group;
            const float a = sums[2 * r] * over, b = sums[2 * r + 1] * over;
#pragma unroll
            for (int i = 0; i < CH * 8; ++i) x[r][i] = stat[r].y * (dy[r][i] - a - x[r][i] * b);
            if (p.out && row < p.rows) store_row<CH, VEC>(static_cast<T*>(p.out) + row * p.out_stride, t, G, p.dim, x[r]);
        }
    }
    if (!p.parts) return;
    float* const part = p.parts + static_cast<long long>(blockIdx.x) * 2 * p.dim;
    if constexpr (LANES > 0) {
        // the groups' sums, in order
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            columns[(2 * i) * kThreads + threadIdx.x] = dw[i];
            columns[(2 * i + 1) * kThreads + threadIdx.x] = db[i];
        }
        __syncthreads();
        for (int i = threadIdx.x; i < 16 * LANES; i += kThreads) {
            const int which = i / LANES, from = i % LANES, at = place<VEC>(0, which / 2, from, LANES);
            float sum = 0.0f;
            for (int g = 0; g < groups; ++g) sum += columns[which * kThreads + g * LANES + from];
            if (at < p.dim) part[(which & 1) * p.dim + at] = sum;
        }
    } else {
#pragma unroll
        for (int i = 0; i < CH * 8; ++i) {
            const int at = place<VEC>(i / 8, i % 8, t, G);
            if (at < p.dim) {
                part[at] = dw[i];
                part[p.dim + at] = db[i];
            }
        }
    }
}

// Rows of any length, a CTA each, read twice: the gradient of x alone.
template <typename T>
__global__ void __launch_bounds__(1024) norm_backward_long_kernel(const __grid_constant__ NormParams p) {
    __shared__ float shared[2][kMaxWarps];
    ddpk::dev::pdl_wait();
    ddpk::dev::pdl_trigger();
    for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const T* const x = static_cast<const T*>(p.x) + row * p.x_stride;
        const T* const dy = static_cast<const T*>(p.grad) + row * p.grad_stride;
        T* const dx = static_cast<T*>(p.out) + row * p.out_stride;
        const float2 stat = *reinterpret_cast<const float2*>(p.stats + 2 * row);
        float a = 0.0f, b = 0.0f;
        for (int i = threadIdx.x; i < p.dim; i += blockDim.x) {
            const float g = widen(dy[i]) * (p.weight ? param_at(p.weight, p.param_bf16, i) : 1.0f);
            a += g;
            b = fmaf(g, (widen(x[i]) - stat.x) * stat.y, b);
        }
        a = __fdiv_rn(group_sum<0>(a, shared[0]), static_cast<float>(p.dim));
        b = __fdiv_rn(group_sum<0>(b, shared[1]), static_cast<float>(p.dim));
        for (int i = threadIdx.x; i < p.dim; i += blockDim.x) {
            const float g = widen(dy[i]) * (p.weight ? param_at(p.weight, p.param_bf16, i) : 1.0f);
            dx[i] = narrow<T>(stat.y * (g - a - (widen(x[i]) - stat.x) * stat.y * b));
        }
        __syncthreads();                   // shared is written again by the next row
    }
}

// And the weight's and the bias's: a thread a column, a CTA 256 of them over every nparts-th row.
template <typename T>
__global__ void __launch_bounds__(kThreads) norm_columns_kernel(const __grid_constant__ NormParams p) {
    ddpk::dev::pdl_wait();
    ddpk::dev::pdl_trigger();
    const int part = blockIdx.x % p.nparts, at = blockIdx.x / p.nparts * kThreads + threadIdx.x;
    if (at >= p.dim) return;
    float dw = 0.0f, db = 0.0f;
    for (long long row = part; row < p.rows; row += p.nparts) {
        const float2 stat = *reinterpret_cast<const float2*>(p.stats + 2 * row);
        const float g = widen(static_cast<const T*>(p.grad)[row * p.grad_stride + at]);
        dw = fmaf(g, (widen(static_cast<const T*>(p.x)[row * p.x_stride + at]) - stat.x) * stat.y, dw);
        db += g;
    }
    p.parts[static_cast<long long>(part) * 2 * p.dim + at] = dw;
    p.parts[static_cast<long long>(part) * 2 * p.dim + p.dim + at] = db;
}

// The parts' sums in a fixed order: 32 columns of a CTA, a warp every 32nd part.
__global__ void __launch_bounds__(32 * kJoinLanes) join_kernel(const __grid_constant__ NormParams p) {
    __shared__ float sums[kJoinLanes][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    ddpk::dev::pdl_wait();
    ddpk::dev::pdl_trigger();
    const int at = blockIdx.x * 32 + lane;
    float sum = 0.0f;
    if (at < 2 * p.dim)
#pragma unroll 8
        for (int i = warp; i < p.nparts; i += kJoinLanes) sum += p.parts[static_cast<long long>(i) * 2 * p.dim + at];
    sums[warp][lane] = sum;
    __syncthreads();
    sum = lanes_sum<32>(sums[lane][warp]);               // column `warp` of this CTA's
    const int column = blockIdx.x * 32 + warp;
    if (lane == 0 && column < 2 * p.dim) {
        void* const to = column < p.dim ? p.grad_weight : p.grad_bias;
        const int i = column < p.dim ? column : column - p.dim;
        if (!to) return;
        if (p.param_bf16) static_cast<uint16_t*>(to)[i] = narrow<uint16_t>(sum);
        else static_cast<float*>(to)[i] = p.accumulate ? static_cast<float*>(to)[i] + sum : sum;
    }
}

// ---------------------------------------------------------------- host

int round_up(int x, int to) { return (x + to - 1) / to * to; }

// How a row lies in threads.
struct Split {
    int lanes;       // of a row; 0: a CTA's threads
    int chunks;      // of eight elements, of a thread; 0: the row is read again and again
    int threads;     // of a CTA
};

Split forward_split(int dim) {
    const int eights = (dim + 7) / 8;
    if (eights <= 8) return {8, 1, kThreads};
    if (eights <= 32) return {32, 1, kThreads};
    if (eights <= 64) return {32, 2, kThreads};
    if (eights <= 128) return {32, 4, kThreads};
    if (eights <= 4 * 1024) return {0, 4, round_up((eights + 3) / 4, 32)};
    return {0, 0, 1024};
}

Split backward_split(int dim) {
    const int eights = (dim + 7) / 8;
    if (eights <= 8) return {8, 1, kThreads};
    if (eights <= 32) return {32, 1, kThreads};
    if (eights <= 512) return {0, 1, round_up(eights, 32)};
    return {0, 0, 1024};
}

// CTAs of the gradient, each with a part of the weight's.
int backward_parts(int dim, long long rows) {
    const Split s = backward_split(dim);
    const long long tile = s.chunks ? (s.lanes ? kThreads / s.lanes : 1) * kRows : kMinRows;
    const long long most = s.chunks ? kMaxParts : 64, need = (rows + tile - 1) / tile;
    return static_cast<int>(need < most ? need : most);
}

template <typename T, int LANES, int CH>
cudaError_t forward_as(const Split& s, bool vec, const NormParams& p, cudaStream_t stream) {
    const int groups = LANES ? kThreads / LANES : 1;
    const long long need = (p.rows + groups - 1) / groups, most = static_cast<long long>(kSms) * 64;
    return launch(vec ? norm_kernel<T, LANES, CH, true> : norm_kernel<T, LANES, CH, false>, need < most ? need : most,
                  s.threads, 0, stream, p);
}

template <typename T>
cudaError_t forward(bool vec, const NormParams& p, cudaStream_t stream) {
    const Split s = forward_split(p.dim);
    if (!s.chunks) return launch(norm_long_kernel<T>, p.rows < kSms * 2 ? p.rows : kSms * 2, s.threads, 0, stream, p);
    if (s.lanes == 8) return forward_as<T, 8, 1>(s, vec, p, stream);
    if (s.lanes == 0) return forward_as<T, 0, 4>(s, vec, p, stream);
    if (s.chunks == 1) return forward_as<T, 32, 1>(s, vec, p, stream);
    if (s.chunks == 2) return forward_as<T, 32, 2>(s, vec, p, stream);
    return forward_as<T, 32, 4>(s, vec, p, stream);
}

template <typename T, int LANES>
cudaError_t backward_as(const Split& s, bool vec, const NormParams& p, cudaStream_t stream) {
    return launch(vec ? norm_backward_kernel<T, LANES, 1, true> : norm_backward_kernel<T, LANES, 1, false>, p.nparts,
                  s.threads, 0, stream, p);
}

template <typename T>
cudaError_t backward(bool vec, const NormParams& p, cudaStream_t stream) {
    const Split s = backward_split(p.dim);
    if (s.chunks) {
        const cudaError_t e = s.lanes == 8 ? backward_as<T, 8>(s, vec, p, stream)
                                           : s.lanes ? backward_as<T, 32>(s, vec, p, stream) : backward_as<T, 0>(s, vec, p, stream);
        if (e != cudaSuccess || !p.parts) return e;
    } else {
        if (p.out) {
            const cudaError_t e = launch(norm_backward_long_kernel<T>, p.rows < kSms * 2 ? p.rows : kSms * 2, s.threads, 0, stream, p);
            if (e != cudaSuccess) return e;
        }
        if (!p.parts) return cudaSuccess;
        const cudaError_t e = launch(norm_columns_kernel<T>, static_cast<long long>(p.nparts) * ((p.dim + kThreads - 1) / kThreads),
                                     kThreads, 0, stream, p);
        if (e != cudaSuccess) return e;
    }
    return launch(join_kernel, (2LL * p.dim + 31) / 32, 32 * kJoinLanes, 0, stream, p);
}

bool valid(const ddp_layer_norm_args* a) {
    return a && a->rows >= 0 && a->dim >= 1 && a->dim <= 1 << 24 && a->x_stride >= a->dim && a->out_stride >= a->dim &&
           std::isfinite(a->eps) && a->eps >= 0.0f && (a->dtype == DDP_F32 || a->dtype == DDP_BF16) &&
           (a->param_dtype == DDP_F32 || a->param_dtype == DDP_BF16);
}

NormParams params_of(const ddp_layer_norm_args* a) {
    NormParams p = {};
    p.rows = a->rows;
    p.dim = static_cast<int>(a->dim);
    p.x_stride = a->x_stride;
    p.out_stride = a->out_stride;
    p.eps = a->eps;
    p.param_bf16 = a->param_dtype == DDP_BF16;
    return p;
}

}  // namespace

extern "C" {

int ddp_layer_norm(const ddp_layer_norm_args* a, const void* x, const void* weight, const void* bias, void* y, float* stats,
                   void* stream) {
    if (!valid(a)) return DDP_ERR_INVALID_ARG;
    if (a->rows == 0) return DDP_OK;
    const int size = a->dtype == DDP_F32 ? 4 : 2, param_size = a->param_dtype == DDP_F32 ? 4 : 2;
    if (!x || !y || !stats || !aligned(x, size) || !aligned(y, size) || !aligned(stats, 8) || !aligned(weight, param_size) ||
        !aligned(bias, param_size))
        return DDP_ERR_INVALID_ARG;
    NormParams p = params_of(a);
    p.x = x;
    p.weight = weight;
    p.bias = bias;
    p.out = y;
    p.stats = stats;
    const bool vec = a->dim % 8 == 0 && aligned(x, 16) && aligned(y, 16) && aligned(weight, 16) && aligned(bias, 16) &&
                     (a->rows == 1 || (a->x_stride * size % 16 == 0 && a->out_stride * size % 16 == 0));
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = a->dtype == DDP_F32 ? forward<float>(vec, p, st) : forward<uint16_t>(vec, p, st);
    return e == cudaSuccess ? DDP_OK : DDP_ERR_CUDA;
}

int64_t ddp_layer_norm_workspace(const ddp_layer_norm_args* a) {
    if (!valid(a)) return DDP_ERR_INVALID_ARG;
    return a->rows == 0 ? 0 : 8LL * a->dim * backward_parts(static_cast<int>(a->dim), a->rows);
}

int ddp_layer_norm_backward(const ddp_layer_norm_args* a, const void* grad_y, int64_t grad_stride, const void* x,
                            const float* stats, const void* weight, void* grad_x, void* grad_weight, void* grad_bias,
                            int32_t accumulate, void* workspace, void* stream) {
    if (!valid(a) || grad_stride < a->dim || (accumulate && a->param_dtype != DDP_F32)) return DDP_ERR_INVALID_ARG;
    const int size = a->dtype == DDP_F32 ? 4 : 2, param_size = a->param_dtype == DDP_F32 ? 4 : 2;
    const bool params = grad_weight || grad_bias;
    if (!aligned(grad_weight, param_size) || !aligned(grad_bias, param_size)) return DDP_ERR_INVALID_ARG;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (a->rows == 0) {                                          // sums over nothing
        cudaError_t e = cudaSuccess;
        if (grad_weight && !accumulate) e = cudaMemsetAsync(grad_weight, 0, a->dim * param_size, st);
        if (grad_bias && !accumulate && e == cudaSuccess) e = cudaMemsetAsync(grad_bias, 0, a->dim * param_size, st);
        return e == cudaSuccess ? DDP_OK : DDP_ERR_CUDA;
    }
    if (!grad_y || !x || !stats || (!grad_x && !params) || (params && !workspace) || !aligned(grad_y, size) ||
        !aligned(x, size) || !aligned(stats, 8) || !aligned(weight, param_size) || !aligned(grad_x, size) || !aligned(workspace, 16))
        return DDP_ERR_INVALID_ARG;
    NormParams p = params_of(a);
    p.x = x;
    p.grad = grad_y;
    p.grad_stride = grad_stride;
    p.stats = const_cast<float*>(stats);
    p.weight = weight;
    p.out = grad_x;
    p.grad_weight = grad_weight;
    p.grad_bias = grad_bias;
    p.accumulate = accumulate != 0;
    p.parts = params ? static_cast<float*>(workspace) : nullptr;
    p.nparts = backward_parts(p.dim, p.rows);
    const bool vec = a->dim % 8 == 0 && aligned(x, 16) && aligned(grad_y, 16) && aligned(grad_x, 16) && aligned(weight, 16) &&
                     (a->rows == 1 || (a->x_stride * size % 16 == 0 && a->out_stride * size % 16 == 0 && grad_stride * size % 16 == 0));
    const cudaError_t e = a->dtype == DDP_F32 ? backward<float>(vec, p, st) : backward<uint16_t>(vec, p, st);
    return e == cudaSuccess ? DDP_OK : DDP_ERR_CUDA;
}

}  // extern "C"
