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

#include <algorithm>
#include <cmath>
#include <cstdint>

#include "ddp_rows.cuh"

namespace {

using namespace ddpk::rows;

constexpr int kForwardThreads = 128;   // of a CTA that holds several rows
constexpr int kBackwardThreads = 256;
constexpr int kMaxWarps = 16;          // of a CTA that holds a row, in registers
constexpr int kLongThreads = 1024;     // of one that reads it again and again
constexpr int kLongWarps = kLongThreads / 32;
constexpr int kLongParts = 64;         // of rows of any length, over which the columns are summed
constexpr int kColumns = 256;          // of a CTA of norm_columns_kernel
constexpr int kJoinLanes = 32;         // join_kernel: threads of a column
constexpr int kForwardWaves = 3;       // 65,536 x 1024 in bf16: one 50.1 us, two 46.3, three 44.7, four 45.8, six 52.7
constexpr int kWarpsPerSm = 16;        // resident, at 128 registers (odd bf16 rows of 32 columns a lane take 155: 12)
// Rows of a group on their way, with the one under work (of 512 threads' fp32
// rows more would not fit); and rounds of rows of the gradient.
template <typename T> constexpr int kForwardStages = sizeof(T) == 2 ? 4 : 3;
constexpr int kBackwardStages = 3;

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

// Thread t's i-th element of a row in a group of G threads: 16 bytes next to one
// another at a time, or (rows that do not lie in vectors) every G-th element.
template <typename T, bool VEC>
__device__ __forceinline__ int place(int i, int t, int G) {
    constexpr int kUnit = 16 / static_cast<int>(sizeof(T));
    return VEC ? (i / kUnit * G + t) * kUnit + i % kUnit : i * G + t;
}

__device__ __forceinline__ float param_at(const void* p, int bf16, int at) {
    return bf16 ? widen(static_cast<const uint16_t*>(p)[at]) : static_cast<const float*>(p)[at];
}

// A thread's elements of a parameter vector, in pairs; `none` where there is no
// vector, and past its end.
template <typename T, int CH, bool VEC>
__device__ __forceinline__ void load_param(const void* p, int bf16, float none, int t, int G, int dim, float2 (&f)[CH * 4]) {
#pragma unroll
    for (int i = 0; i < CH * 4; ++i) {
        f[i] = both(none);
        if (!p) continue;
        const int at = place<T, VEC>(2 * i, t, G), next = place<T, VEC>(2 * i + 1, t, G);
        if (at < dim) f[i].x = param_at(p, bf16, at);
        if (next < dim) f[i].y = param_at(p, bf16, next);
    }
}

// Rows on their way to the shared memory of a CTA.  Rows that lie in vectors: each
// thread copies, and reads, 16-byte pieces of its own.  Others: the group copies
// the 16-byte words that its row touches (none without an element of it), and all
// of the group read from them.
template <typename T, int CH, bool VEC>
struct Lines {
    static constexpr int kUnit = 16 / static_cast<int>(sizeof(T)), kPieces = CH * 8 / kUnit;

    uint4* at;

    // words of one row of each group
    static __device__ __host__ __forceinline__ int size(int threads, int groups) { return kPieces * threads + (VEC ? 0 : groups); }

    __device__ __forceinline__ Lines(uint4* row, int group, int G) : at(row + (VEC ? threadIdx.x : group * (kPieces * G + 1))) {}

    __device__ __forceinline__ void request(const T* row, int t, int G, int dim) const {
        if constexpr (VEC) {
#pragma unroll
            for (int k = 0; k < kPieces; ++k)
                if ((k * G + t) * kUnit < dim) copy_async(at + k * blockDim.x, row + (k * G + t) * kUnit);
        } else {
            const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(row) & 15);
            const uint4* const words = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(row) - shift);
            const int count = (shift + dim * static_cast<int>(sizeof(T)) + 15) / 16;
            for (int k = t; k < count; k += G) copy_async(at + k, words + k);
        }
    }
    // zeros past the row's end
    __device__ __forceinline__ void take(const T* row, int t, int G, int dim, float2 (&x)[CH * 4]) const {
        if constexpr (!VEC) {
            const T* const from = reinterpret_cast<const T*>(reinterpret_cast<const char*>(at) + (reinterpret_cast<uintptr_t>(row) & 15));
#pragma unroll
            for (int i = 0; i < CH * 4; ++i) {
                const int a = place<T, false>(2 * i, t, G), b = place<T, false>(2 * i + 1, t, G);
                x[i].x = a < dim ? widen(from[a]) : 0.0f;
                x[i].y = b < dim ? widen(from[b]) : 0.0f;
            }
        } else {
#pragma unroll
            for (int k = 0; k < kPieces; ++k) {
                const uint4 raw = (k * G + t) * kUnit < dim ? at[k * blockDim.x] : make_uint4(0, 0, 0, 0);
                const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
                if constexpr (sizeof(T) == 2) {
#pragma unroll
                    for (int j = 0; j < 4; ++j) x[k * 4 + j] = make_float2(__uint_as_float(w[j] << 16), __uint_as_float(w[j] & 0xffff0000u));
                } else {
                    x[k * 2] = make_float2(__uint_as_float(w[0]), __uint_as_float(w[1]));
                    x[k * 2 + 1] = make_float2(__uint_as_float(w[2]), __uint_as_float(w[3]));
                }
            }
        }
    }
};

template <int CH, bool VEC, typename T>
__device__ __forceinline__ void store_row(T* row, int t, int G, int dim, const float2 (&x)[CH * 4]) {
    if constexpr (VEC) {
        using L = Lines<T, CH, true>;
#pragma unroll
        for (int k = 0; k < L::kPieces; ++k) {
            uint4 w;
            if constexpr (sizeof(T) == 2)
                w = make_uint4(pack_bf16(x[k * 4].x, x[k * 4].y), pack_bf16(x[k * 4 + 1].x, x[k * 4 + 1].y),
                               pack_bf16(x[k * 4 + 2].x, x[k * 4 + 2].y), pack_bf16(x[k * 4 + 3].x, x[k * 4 + 3].y));
            else
                w = make_uint4(__float_as_uint(x[k * 2].x), __float_as_uint(x[k * 2].y), __float_as_uint(x[k * 2 + 1].x),
                               __float_as_uint(x[k * 2 + 1].y));
            if ((k * G + t) * L::kUnit < dim) __stcs(reinterpret_cast<uint4*>(row + (k * G + t) * L::kUnit), w);
        }
    } else {
#pragma unroll
        for (int i = 0; i < CH * 8; ++i) {
            const int at = place<T, false>(i, t, G);
            if (at < dim) row[at] = narrow<T>(i & 1 ? x[i / 2].y : x[i / 2].x);
        }
    }
}

// Until the copies of a round have landed, for all of those who read them.
template <int LANES, bool VEC, int LEFT>
__device__ __forceinline__ void landed() {
    copy_wait<LEFT>();
    if constexpr (!VEC) {
        if constexpr (LANES > 0) __syncwarp();
        else __syncthreads();
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

// ---------------------------------------------------------------- forward

// y = (x - mean) / sqrt(var + eps) w + b.  A group takes every so many rows, which
// are copied to shared memory ahead, and keeps its columns' weight and bias in
// registers.  65,536 rows of 1,024 in bf16: 44.6 us, 6.0 TB/s of the bytes that it
// has to move, at a plain copy's 6.7 40 us; each row loaded when
// it was due took 81, addresses computed for each 50.  A warp holds a row in 32
// elements a lane, so that the two sums are ten shuffles and no barrier.
template <typename T, int LANES, int CH, bool VEC>
__global__ void __launch_bounds__(LANES ? kForwardThreads : 32 * kMaxWarps) norm_kernel(const __grid_constant__ NormParams p) {
    extern __shared__ uint4 ahead[];
    __shared__ float shared[2][kMaxWarps];
    constexpr int kStages = kForwardStages<T>;
    using L = Lines<T, CH, VEC>;
    const int G = LANES ? LANES : blockDim.x, t = threadIdx.x % G;
    const int groups = LANES ? kForwardThreads / LANES : 1, group = LANES ? threadIdx.x / LANES : 0;
    ddpk::dev::pdl_wait();
    ddpk::dev::pdl_trigger();
    const long long stride = static_cast<long long>(gridDim.x) * groups, first = static_cast<long long>(blockIdx.x) * groups + group;
    const auto lines = [&](int stage) { return L(ahead + stage * L::size(blockDim.x, groups), group, G); };
    const T* x_next = static_cast<const T*>(p.x) + first * p.x_stride;
    const T* x_now = x_next;
    T* out_next = static_cast<T*>(p.out) + first * p.out_stride;
    long long asked = first;                                     // the row that is asked for next
    const auto request = [&](int stage) {
        if (asked < p.rows) lines(stage).request(x_next, t, G, p.dim);
        copy_commit();
        asked += stride;
        x_next += stride * p.x_stride;
    };
#pragma unroll
    for (int s = 0; s + 1 < kStages; ++s) request(s);
    float2 w[CH * 4], b[CH * 4];
    load_param<T, CH, VEC>(p.weight, p.param_bf16, 1.0f, t, G, p.dim, w);
    load_param<T, CH, VEC>(p.bias, p.param_bf16, 0.0f, t, G, p.dim, b);
    int stage = 0;
    // all groups of a warp take as many rounds, for their sums' shuffles
    for (long long row = first; row - group < p.rows; row += stride) {
        const bool on = row < p.rows;
        float2 x[CH * 4];
        landed<LANES, VEC, kStages - 2>();
        lines(stage).take(x_now, t, G, p.dim, x);
        x_now += stride * p.x_stride;
        // into the stage before this one, whose row everyone has taken
        request(stage ? stage - 1 : kStages - 1);
        stage = stage + 1 < kStages ? stage + 1 : 0;
        float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < CH * 4; ++i) sum = add2(sum, x[i]);
        const float mean = __fdiv_rn(group_sum<LANES>(sum.x + sum.y, shared[0]), static_cast<float>(p.dim));
        sum = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int i = 0; i < CH * 4; ++i) {
            x[i] = add2(x[i], both(-mean));
            // elements past the row's end count for nothing
            if constexpr (VEC) {
                if (place<T, true>(2 * i, t, G) < p.dim) sum = fma2(x[i], x[i], sum);
            } else {
                if (place<T, false>(2 * i, t, G) < p.dim) sum.x = fmaf(x[i].x, x[i].x, sum.x);
                if (place<T, false>(2 * i + 1, t, G) < p.dim) sum.y = fmaf(x[i].y, x[i].y, sum.y);
            }
        }
        const float variance = __fdiv_rn(group_sum<LANES>(sum.x + sum.y, shared[1]), static_cast<float>(p.dim));
        const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(variance + p.eps));
        if (on && t == 0) *reinterpret_cast<float2*>(p.stats + 2 * row) = make_float2(mean, rstd);
#pragma unroll
        for (int i = 0; i < CH * 4; ++i) x[i] = fma2(mul2(x[i], both(rstd)), w[i], b[i]);
        if (on) store_row<CH, VEC>(out_next, t, G, p.dim, x);
        out_next += stride * p.out_stride;
    }
}

// Rows of any length, a CTA each, read three times.
template <typename T>
__global__ void __launch_bounds__(kLongThreads) norm_long_kernel(const __grid_constant__ NormParams p) {
    __shared__ float shared[2][kLongWarps];
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

// Sums of N values over a warp: each of the first steps halves the values that a
// lane keeps (eight take nine shuffles instead of 40).  The sum of value i is in
// lane_of<N>(i), and in the lanes whose bits above those of the last steps are
// the same.
template <int N>
__device__ __forceinline__ float sum_many(float (&v)[N]) {
    const int lane = threadIdx.x & 31;
    int o = 16;
#pragma unroll
    for (int n = N / 2; n; n /= 2, o /= 2) {
        const bool upper = lane & o;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float mine = upper ? v[i + n] : v[i], other = upper ? v[i] : v[i + n];
            v[i] = mine + __shfl_xor_sync(kAll, other, o);
        }
    }
    float sum = v[0];
#pragma unroll
    for (int q = 16 / N; q; q /= 2) sum += __shfl_xor_sync(kAll, sum, q);
    return sum;
}

template <int N>
__device__ __forceinline__ int lane_of(int i) { return i * (32 / N); }

// dx = r (g - mean(g) - xh mean(g xh)), g = dy w, xh = (x - mean) r; dw = sum dy xh
// and db = sum dy over the CTA's rows, a thread its columns.  A round is ROWS rows
// of each group, so that a barrier serves as many.  65,536 rows of 1,024 in bf16:
// 68 us with the parts' sums, 5.9 TB/s (floor 60); without copies ahead 113.  A CTA
// of 128 threads holds the row, since the columns' sums dw and db live in
// registers and a warp of 32 columns a lane has no room for them.
template <typename T, int LANES, int CH, int ROWS, bool VEC, int MAXT>
__global__ void __launch_bounds__(MAXT, 32 * kWarpsPerSm / MAXT) norm_backward_kernel(const __grid_constant__ NormParams p) {
    constexpr int N = 2 * ROWS;
    extern __shared__ uint4 ahead[];
    __shared__ float shared[2][kMaxWarps][N];
    const int G = LANES ? LANES : blockDim.x, t = threadIdx.x % G;
    const int groups = LANES ? kBackwardThreads / LANES : 1, group = LANES ? threadIdx.x / LANES : 0;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    ddpk::dev::pdl_wait();
    ddpk::dev::pdl_trigger();
    using L = Lines<T, CH, VEC>;
    const int tile = groups * ROWS;
    const long long first = static_cast<long long>(blockIdx.x) * tile, stride = static_cast<long long>(gridDim.x) * tile;
    const auto lines = [&](int stage, int r, int which) {
        return L(ahead + ((stage * ROWS + r) * 2 + which) * L::size(blockDim.x, groups), group, G);
    };
    // of this thread's first row of a round: how many rows are left from it on, and where it is
    const auto left_of = [&](long long r0) { return static_cast<int>(min(p.rows - r0 - group, 1LL << 30)); };
    const long long x_step = groups * p.x_stride, dy_step = groups * p.grad_stride, out_step = groups * p.out_stride;
    const T* x_next = static_cast<const T*>(p.x) + (first + group) * p.x_stride;
    const T* dy_next = static_cast<const T*>(p.grad) + (first + group) * p.grad_stride;
    const T* x_now = x_next;                                     // (for their places among 16 bytes)
    const T* dy_now = dy_next;
    T* out_next = static_cast<T*>(p.out) + (first + group) * p.out_stride;
    const float2* stat_next = reinterpret_cast<const float2*>(p.stats) + first + group;
    long long asked = first;                                     // of the round that is asked for next
    const auto request = [&](int stage) {
        const int left = left_of(asked);
#pragma unroll
        for (int r = 0; r < ROWS; ++r)
            if (r * groups < left) {
                lines(stage, r, 0).request(x_next + r * x_step, t, G, p.dim);
                lines(stage, r, 1).request(dy_next + r * dy_step, t, G, p.dim);
            }
        copy_commit();
        asked += stride;
        x_next += stride * p.x_stride;
        dy_next += stride * p.grad_stride;
    };
#pragma unroll
    for (int s = 0; s + 1 < kBackwardStages; ++s) request(s);
    float2 dw[CH * 4], db[CH * 4], w[CH * 4];
    load_param<T, CH, VEC>(p.weight, p.param_bf16, 1.0f, t, G, p.dim, w);
#pragma unroll
    for (int i = 0; i < CH * 4; ++i) dw[i] = db[i] = make_float2(0.0f, 0.0f);
    const float over = __fdiv_rn(1.0f, static_cast<float>(p.dim));
    int phase = 0, stage = 0;
    for (long long r0 = first; r0 < p.rows; r0 += stride) {
        float2 x[ROWS][CH * 4], dy[ROWS][CH * 4], stat[ROWS];
        float sums[N];
        const int left = left_of(r0);
#pragma unroll
        for (int r = 0; r < ROWS; ++r) stat[r] = r * groups < left ? stat_next[r * groups] : make_float2(0.0f, 0.0f);
        landed<LANES, VEC, kBackwardStages - 2>();
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            const int dim = r * groups < left ? p.dim : 0;       // (zeros)
            lines(stage, r, 0).take(x_now + r * x_step, t, G, dim, x[r]);
            lines(stage, r, 1).take(dy_now + r * dy_step, t, G, dim, dy[r]);
        }
        x_now += stride * p.x_stride;
        dy_now += stride * p.grad_stride;
        request(stage ? stage - 1 : kBackwardStages - 1);        // used up a round ago
        stage = stage + 1 < kBackwardStages ? stage + 1 : 0;
        stat_next += stride;
        if (t < ROWS && t * groups < left_of(r0 + stride))       // near by the time that they are loaded
            asm volatile("prefetch.global.L1 [%0];" ::"l"(stat_next + t * groups));
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            float2 a = make_float2(0.0f, 0.0f), b = a;
#pragma unroll
            for (int i = 0; i < CH * 4; ++i) {
                x[r][i] = mul2(add2(x[r][i], both(-stat[r].x)), both(stat[r].y));
                db[i] = add2(db[i], dy[r][i]);
                dw[i] = fma2(dy[r][i], x[r][i], dw[i]);          // nothing past the row's end: dy is zero there
                dy[r][i] = mul2(dy[r][i], w[i]);
                a = add2(a, dy[r][i]);
                b = fma2(dy[r][i], x[r][i], b);
            }
            sums[2 * r] = a.x + a.y;
            sums[2 * r + 1] = b.x + b.y;
        }
        if constexpr (LANES > 0) {
#pragma unroll
            for (int i = 0; i < N; ++i) sums[i] = lanes_sum<LANES>(sums[i]);
        } else {
            float s = sum_many<N>(sums);
            if (lane % (32 / N) == 0) shared[phase][warp][lane / (32 / N)] = s;
            __syncthreads();
#pragma unroll
            for (int i = 0; i < N; ++i) sums[i] = lane < warps ? shared[phase][lane][i] : 0.0f;
            s = sum_many<N>(sums);
#pragma unroll
            for (int i = 0; i < N; ++i) sums[i] = __shfl_sync(kAll, s, lane_of<N>(i));
            phase ^= 1;                                          // the other half is free: everyone is past this round's barrier
        }
        if (!p.out) continue;
#pragma unroll
        for (int r = 0; r < ROWS; ++r) {
            const float2 a = both(-sums[2 * r] * over), b = both(-sums[2 * r + 1] * over);
#pragma unroll
            for (int i = 0; i < CH * 4; ++i) x[r][i] = mul2(both(stat[r].y), fma2(x[r][i], b, add2(dy[r][i], a)));
            if (r * groups < left) store_row<CH, VEC>(out_next + r * out_step, t, G, p.dim, x[r]);
        }
        out_next += stride * p.out_stride;
    }
    if (!p.parts) return;
    float* const part = p.parts + static_cast<long long>(blockIdx.x) * 2 * p.dim;
    if constexpr (LANES > 0) {
        // the groups' sums, in order, through the memory of the rows, which are used up
        float* const columns = reinterpret_cast<float*>(ahead);
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            columns[(2 * i) * kBackwardThreads + threadIdx.x] = i & 1 ? dw[i / 2].y : dw[i / 2].x;
            columns[(2 * i + 1) * kBackwardThreads + threadIdx.x] = i & 1 ? db[i / 2].y : db[i / 2].x;
        }
        __syncthreads();
        for (int i = threadIdx.x; i < 16 * LANES; i += kBackwardThreads) {
            const int which = i / LANES, of = i % LANES, at = place<T, VEC>(which / 2, of, LANES);
            float sum = 0.0f;
            for (int g = 0; g < groups; ++g) sum += columns[which * kBackwardThreads + g * LANES + of];
            if (at < p.dim) part[(which & 1) * p.dim + at] = sum;
        }
    } else {
#pragma unroll
        for (int i = 0; i < CH * 8; ++i) {
            const int at = place<T, VEC>(i, t, G);
            if (at < p.dim) {
                part[at] = i & 1 ? dw[i / 2].y : dw[i / 2].x;
                part[p.dim + at] = i & 1 ? db[i / 2].y : db[i / 2].x;
            }
        }
    }
}

// Rows of any length, a CTA each, read twice: the gradient of x alone.
template <typename T>
__global__ void __launch_bounds__(kLongThreads) norm_backward_long_kernel(const __grid_constant__ NormParams p) {
    __shared__ float shared[2][kLongWarps];
    ddpk::dev::pdl_wait();
    ddpk::dev::pdl_trigger();
    for (long long row = blockIdx.x; row < p.rows; row += gridDim.x) {
        const T* const x = static_cast<const T*>(p.x) + row * p.x_stride;
        const T* const dy = static_cast<const T*>(p.grad) + row * p.grad_stride;
        T* const dx = static_cast<T*>(p.out) + row * p.out_stride;
        const float2 stat = *reinterpret_cast<const float2*>(p.stats + 2 * row);
        const auto weight = [&](int i) { return p.weight ? param_at(p.weight, p.param_bf16, i) : 1.0f; };
        float a = 0.0f, b = 0.0f;
#pragma unroll 4
        for (int i = threadIdx.x; i < p.dim; i += kLongThreads) {
            const float g = widen(dy[i]) * weight(i);
            a += g;
            b = fmaf(g, (widen(x[i]) - stat.x) * stat.y, b);
        }
        a = __fdiv_rn(group_sum<0>(a, shared[0]), static_cast<float>(p.dim));
        b = __fdiv_rn(group_sum<0>(b, shared[1]), static_cast<float>(p.dim));
        for (int i0 = threadIdx.x; i0 < p.dim; i0 += 4 * kLongThreads) {
            float g[4], xh[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const int i = i0 + u * kLongThreads;
                g[u] = i < p.dim ? widen(dy[i]) * weight(i) : 0.0f;
                xh[u] = i < p.dim ? (widen(x[i]) - stat.x) * stat.y : 0.0f;
            }
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (i0 + u * kLongThreads < p.dim) dx[i0 + u * kLongThreads] = narrow<T>(stat.y * (g[u] - a - xh[u] * b));
        }
        __syncthreads();                   // shared is written again by the next row
    }
}

// And the weight's and the bias's: a thread a column, a CTA 256 of them over every nparts-th row.
template <typename T>
__global__ void __launch_bounds__(kColumns) norm_columns_kernel(const __grid_constant__ NormParams p) {
    ddpk::dev::pdl_wait();
    ddpk::dev::pdl_trigger();
    const int part = blockIdx.x % p.nparts, at = blockIdx.x / p.nparts * kColumns + threadIdx.x;
    if (at >= p.dim) return;
    float dw = 0.0f, db = 0.0f;
#pragma unroll 8
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

// Lanes of a warp while they hold a row in 32 elements each, which needs no
// barriers; then a CTA of up to 512 threads.
Split forward_split(int dim) {
    const int eights = (dim + 7) / 8;
    if (eights <= 8) return {8, 1, kForwardThreads};
    if (eights <= 16) return {16, 1, kForwardThreads};
    if (eights <= 32) return {32, 1, kForwardThreads};
    if (eights <= 64) return {32, 2, kForwardThreads};
    if (eights <= 128) return {32, 4, kForwardThreads};
    if (eights <= 4 * 32 * kMaxWarps) return {0, 4, round_up((eights + 3) / 4, 32)};
    return {0, 0, kLongThreads};
}

// The gradient holds 32 values of a round's rows and gradients each in bf16 and
// 16 in fp32, so that a round takes as many bytes: chunks x rows is 4 or 2.  32
// columns of a thread do not fit its registers with their sums, but read in
// vectors they are still faster than the rows of any length (4,089 bf16 rows of
// 16,384: 152 us and 269; of 11,101, one by one: 536 and 310).
Split backward_split(int dim, int size, bool vec) {
    const int eights = (dim + 7) / 8, most = 32 * kMaxWarps;
    if (eights <= 8) return {8, 1, kBackwardThreads};
    if (eights <= 16) return {16, 1, kBackwardThreads};
    if (eights <= 32) return {32, 1, kBackwardThreads};
    if (eights <= most) return {0, 1, round_up(eights, 32)};
    if (eights <= 2 * most) return {0, 2, round_up((eights + 1) / 2, 32)};
    if (eights <= 4 * most && size == 2 && vec) return {0, 4, round_up((eights + 3) / 4, 32)};
    return {0, 0, kLongThreads};
}

int resident(int threads) { return kSms * (32 * kWarpsPerSm / threads > 1 ? 32 * kWarpsPerSm / threads : 1); }

// CTAs of the gradient, each with a part of the weight's.
int backward_parts(int dim, int size, bool vec, long long rows) {
    const Split s = backward_split(dim, size, vec);
    const long long tile = s.chunks ? (s.lanes ? kBackwardThreads / s.lanes : 1) * (size == 2 ? 4 : 2) / s.chunks : 8;
    const long long most = s.chunks ? resident(s.threads) : kLongParts, need = (rows + tile - 1) / tile;
    return static_cast<int>(need < most ? need : most);
}

template <typename T, int LANES, int CH>
cudaError_t forward_as(const Split& s, bool vec, const NormParams& p, cudaStream_t stream) {
    static std::atomic<uint64_t> allowed[2];                     // of the kernel for vectors, and of the other
    const int groups = LANES ? kForwardThreads / LANES : 1;
    const long long need = (p.rows + groups - 1) / groups, most = kForwardWaves * resident(s.threads);
    const size_t shared = 16ull * kForwardStages<T> *
                          (vec ? Lines<T, CH, true>::size(s.threads, groups) : Lines<T, CH, false>::size(s.threads, groups));
    void (*const kernel)(NormParams) = vec ? norm_kernel<T, LANES, CH, true> : norm_kernel<T, LANES, CH, false>;
    const cudaError_t e = allow_shared(reinterpret_cast<const void*>(kernel), shared, allowed[vec]);
    return e != cudaSuccess ? e : launch(kernel, need < most ? need : most, s.threads, shared, stream, p);
}

template <typename T>
cudaError_t forward(bool vec, const NormParams& p, cudaStream_t stream) {
    const Split s = forward_split(p.dim);
    if (!s.chunks) return launch(norm_long_kernel<T>, p.rows < kSms * 2 ? p.rows : kSms * 2, s.threads, 0, stream, p);
    if (s.lanes == 8) return forward_as<T, 8, 1>(s, vec, p, stream);
    if (s.lanes == 16) return forward_as<T, 16, 1>(s, vec, p, stream);
    if (s.lanes == 0) return forward_as<T, 0, 4>(s, vec, p, stream);
    if (s.chunks == 1) return forward_as<T, 32, 1>(s, vec, p, stream);
    if (s.chunks == 2) return forward_as<T, 32, 2>(s, vec, p, stream);
    return forward_as<T, 32, 4>(s, vec, p, stream);
}

template <typename T, int LANES, int CH, int ROWS, int MAXT>
cudaError_t backward_as(const Split& s, bool vec, const NormParams& p, cudaStream_t stream) {
    static std::atomic<uint64_t> allowed[2];                     // of the kernel for vectors, and of the other
    static_assert(kBackwardStages * ROWS * 2 * Lines<T, CH, true>::kPieces >= 4, "16 columns of a thread");
    const int groups = LANES ? kBackwardThreads / LANES : 1;
    const size_t shared = 16ull * kBackwardStages * ROWS * 2 *
                          (vec ? Lines<T, CH, true>::size(s.threads, groups) : Lines<T, CH, false>::size(s.threads, groups));
    void (*kernel)(NormParams) = norm_backward_kernel<T, LANES, CH, ROWS, true, MAXT>;
    if constexpr (CH < 4)
        if (!vec) kernel = norm_backward_kernel<T, LANES, CH, ROWS, false, MAXT>;
    const cudaError_t e = allow_shared(reinterpret_cast<const void*>(kernel), shared, allowed[vec]);
    return e != cudaSuccess ? e : launch(kernel, p.nparts, s.threads, shared, stream, p);
}

template <typename T>
cudaError_t backward(bool vec, const NormParams& p, cudaStream_t stream) {
    constexpr int R = sizeof(T) == 2 ? 4 : 2;                // rows x chunks
    const Split s = backward_split(p.dim, sizeof(T), vec);
    cudaError_t e = cudaSuccess;
    if (s.chunks == 1)
        e = s.lanes == 8    ? backward_as<T, 8, 1, R, 256>(s, vec, p, stream)
            : s.lanes == 16 ? backward_as<T, 16, 1, R, 256>(s, vec, p, stream)
            : s.lanes == 32 ? backward_as<T, 32, 1, R, 256>(s, vec, p, stream)
            : s.threads <= 128 ? backward_as<T, 0, 1, R, 128>(s, vec, p, stream) : backward_as<T, 0, 1, R, 512>(s, vec, p, stream);
    else if (s.chunks == 2) {
        e = backward_as<T, 0, 2, R / 2, 512>(s, vec, p, stream);
    } else if (s.chunks == 4) {
        if constexpr (R == 4) e = backward_as<T, 0, 4, 1, 512>(s, vec, p, stream);
    } else {
        if (p.out) e = launch(norm_backward_long_kernel<T>, p.rows < kSms * 2 ? p.rows : kSms * 2, s.threads, 0, stream, p);
        if (e == cudaSuccess && p.parts)
            e = launch(norm_columns_kernel<T>, static_cast<long long>(p.nparts) * ((p.dim + kColumns - 1) / kColumns), kColumns, 0,
                       stream, p);
    }
    if (e != cudaSuccess || !p.parts) return e;
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
    const bool vec = a->dim * size % 16 == 0 && aligned(x, 16) && aligned(y, 16) &&
                     (a->rows == 1 || (a->x_stride * size % 16 == 0 && a->out_stride * size % 16 == 0));
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = a->dtype == DDP_F32 ? forward<float>(vec, p, st) : forward<uint16_t>(vec, p, st);
    return e == cudaSuccess ? DDP_OK : DDP_ERR_CUDA;
}

int64_t ddp_layer_norm_workspace(const ddp_layer_norm_args* a) {
    if (!valid(a)) return DDP_ERR_INVALID_ARG;
    if (a->rows == 0) return 0;
    const int dim = static_cast<int>(a->dim), size = a->dtype == DDP_F32 ? 4 : 2;
    return 8LL * dim * std::max(backward_parts(dim, size, false, a->rows), backward_parts(dim, size, true, a->rows));
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
    const bool vec = a->dim * size % 16 == 0 && aligned(x, 16) && aligned(grad_y, 16) && aligned(grad_x, 16) &&
                     (a->rows == 1 || (a->x_stride * size % 16 == 0 && a->out_stride * size % 16 == 0 && grad_stride * size % 16 == 0));
    p.nparts = backward_parts(p.dim, size, vec, p.rows);
    const cudaError_t e = a->dtype == DDP_F32 ? backward<float>(vec, p, st) : backward<uint16_t>(vec, p, st);
    return e == cudaSuccess ? DDP_OK : DDP_ERR_CUDA;
}

}  // extern "C"
