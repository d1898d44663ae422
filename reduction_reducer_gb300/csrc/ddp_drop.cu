// Dropout from a counter: which elements stay follows from the seed and each
// element's place, and is never stored; the backward pass is the same call.
//
// The random bits are Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel
// random numbers: as easy as 1, 2, 3", 2011): the counter is (place / 8, offset),
// the key the seed.  An element is dropped where its 32 bits lie below p 2^32.
// One block of four words gives eight elements the upper 16 bits of theirs; where
// these alone do not tell (one in 65,536), a second block gives the lower 16.  A
// probability thus counts in 32 bits, for about half the instructions of a word
// an element.

#include "ddp_reducer.h"

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "ddp_rows.cuh"

namespace {

using namespace ddpk::rows;

constexpr int kThreads = 256;
constexpr int kGroups = 2;        // of eight elements, of a thread

struct DropParams {
    const void* x;
    const void* residual;
    void* out;
    long long n, cols, x_stride, residual_stride, out_stride;
    const uint64_t* device_seed;
    uint64_t seed;
    uint32_t offset_lo, offset_hi;
    uint32_t least;          // an element stays where its bits are no less
    int none;                // nothing stays (and least is 2^32 - 1)
    float scale;
};

struct Words { uint32_t w[4]; };

__device__ __forceinline__ Words philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, uint32_t k0, uint32_t k1) {
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t a = static_cast<uint64_t>(c0) * 0xD2511F53u, b = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
        c0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ (k0 + r * 0x9E3779B9u);
        c1 = static_cast<uint32_t>(b);
        c2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ (k1 + r * 0xBB67AE85u);
        c3 = static_cast<uint32_t>(a);
    }
    return Words{{c0, c1, c2, c3}};
}

// Which of the eight elements of a group stay.
__device__ __forceinline__ void staying(const DropParams& p, long long group, uint32_t k0, uint32_t k1, bool (&stays)[8]) {
    const uint32_t lo = static_cast<uint32_t>(group), hi = static_cast<uint32_t>(group >> 32);
    const Words u = philox(lo, hi, p.offset_lo, p.offset_hi, k0, k1);
    const uint32_t border = p.least & 0xffff0000u;
    uint32_t closest = 0xffffffffu;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        // the 16 bits at the top, and something below them that does not matter
        const uint32_t bits = j & 1 ? u.w[j / 2] : u.w[j / 2] << 16;
        stays[j] = bits >= border;
        closest = min(closest, bits - border);
    }
    if (closest < 0x10000u && (p.least & 0xffffu)) {      // some have the border's upper half: the lower decides
        const Words v = philox(lo, hi, p.offset_lo, p.offset_hi | 0x80000000u, k0, k1);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t upper = j & 1 ? u.w[j / 2] & 0xffff0000u : u.w[j / 2] << 16;
            const uint32_t lower = j & 1 ? v.w[j / 2] >> 16 : v.w[j / 2] & 0xffffu;
            if (upper == border && (lower < (p.least & 0xffffu) || p.none)) stays[j] = false;
        }
    }
}

// The kernel reads 16 bf16 or fp32 elements a thread and has their bits computed
// while these are on their way.  65,536 x 1,024 in bf16 onto a residual: 61 us (403
// MB, 6.6 TB/s, the copy's rate); without a residual 55 for 268 MB (floor 40): 48.7 M
// warp instructions, 71 % of the integer pipe.  These are 185 for eight elements of a
// lane, of which a block's wide products and exclusive-ors are 40; the others are
// comparisons, the closest to the border, the products with the scale, widening,
// packing and addresses.  A mask of eight bits instead of eight flags took 57 and 64.

// Whole: one run of n elements from boundaries of eight.  Rows: rows of a multiple
// of eight elements, each from one.  Single: anything else, element by element.  us
// for 65,536 rows, without a residual / with one: 1,024 bf16 in one run 56 / 61, in
// rows of 1,032 67 / 74, in rows of 1,028 176 / 181; fp32 78 / 113, 78 / 114, 257 / 273.
enum Layout { kWhole, kRows, kSingle };

template <typename T, bool RESIDUAL, Layout LAYOUT, bool SEED>
__global__ void __launch_bounds__(kThreads) drop_kernel(const __grid_constant__ DropParams p) {
    ddpk::dev::pdl_wait();
    ddpk::dev::pdl_trigger();
    const uint64_t seed = SEED ? *p.device_seed : p.seed;
    const uint32_t k0 = static_cast<uint32_t>(seed), k1 = static_cast<uint32_t>(seed >> 32);
    const T* const x = static_cast<const T*>(p.x);
    const T* const residual = static_cast<const T*>(p.residual);
    T* const out = static_cast<T*>(p.out);
    const long long first = static_cast<long long>(blockIdx.x) * (kThreads * kGroups) + threadIdx.x;
    if constexpr (LAYOUT == kSingle) {
        for (int i = 0; i < kGroups; ++i) {
            const long long group = first + i * kThreads, from = group * 8;
            if (from >= p.n) return;
            bool stays[8];
            staying(p, group, k0, k1, stays);
            long long row = from / p.cols, col = from % p.cols;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (from + j >= p.n) break;
                float y = stays[j] ? widen(x[row * p.x_stride + col]) * p.scale : 0.0f;
                if constexpr (RESIDUAL) y += widen(residual[row * p.residual_stride + col]);
                out[row * p.out_stride + col] = narrow<T>(y);
                if (++col == p.cols) { col = 0; ++row; }
            }
        }
    } else {
        Eight<T> a[kGroups], r[kGroups];
        long long at[kGroups];
        int count[kGroups];
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            const long long from = (first + i * kThreads) * 8;
            const long long left = p.n - from;
            count[i] = left >= 8 ? 8 : left > 0 ? static_cast<int>(left) : 0;
            long long rx = from, rr = from;
            at[i] = from;
            if constexpr (LAYOUT == kRows) {
                const long long row = from / p.cols, col = from % p.cols;
                rx = row * p.x_stride + col;
                rr = row * p.residual_stride + col;
                at[i] = row * p.out_stride + col;
            }
            if (count[i] == 8) {
                a[i].load_wide(x + rx);
                if constexpr (RESIDUAL) r[i].load_wide(residual + rr);
            }
        }
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            bool stays[8];
            staying(p, first + i * kThreads, k0, k1, stays);
            if (count[i] == 8) {
                float y[8], z[8];
                a[i].get(y);
                if constexpr (RESIDUAL) r[i].get(z);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    y[j] = stays[j] ? y[j] * p.scale : 0.0f;
                    if constexpr (RESIDUAL) y[j] += z[j];
                }
                a[i].put(y);
                a[i].store_wide(out + at[i]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) {                 // the last few of a whole run
                    if (j >= count[i]) break;
                    float y = stays[j] ? widen(x[at[i] + j]) * p.scale : 0.0f;
                    if constexpr (RESIDUAL) y += widen(residual[at[i] + j]);
                    out[at[i] + j] = narrow<T>(y);
                }
            }
        }
    }
}

template <typename T, bool RESIDUAL, bool SEED>
void (*kernel_of(Layout layout))(DropParams) {
    return layout == kWhole ? drop_kernel<T, RESIDUAL, kWhole, SEED>
                            : layout == kRows ? drop_kernel<T, RESIDUAL, kRows, SEED> : drop_kernel<T, RESIDUAL, kSingle, SEED>;
}

template <typename T>
cudaError_t launch_drop(Layout layout, long long ctas, const DropParams& p, cudaStream_t stream) {
    void (*const kernel)(DropParams) = p.residual ? (p.device_seed ? kernel_of<T, true, true>(layout) : kernel_of<T, true, false>(layout))
                                                  : (p.device_seed ? kernel_of<T, false, true>(layout) : kernel_of<T, false, false>(layout));
    return launch(kernel, ctas, kThreads, 0, stream, p);
}

}  // namespace

extern "C" int ddp_drop(const ddp_drop_args* a, const void* x, const void* residual, void* out, void* stream) {
    if (!a || a->rows < 0 || a->cols < 0 || a->x_stride < a->cols || a->out_stride < a->cols ||
        (residual && a->residual_stride < a->cols) || !(a->p >= 0.0 && a->p <= 1.0) || a->offset >> 63 ||
        (a->dtype != DDP_F32 && a->dtype != DDP_BF16))
        return DDP_ERR_INVALID_ARG;
    if (a->rows == 0 || a->cols == 0) return DDP_OK;
    const int size = a->dtype == DDP_F32 ? 4 : 2;
    if (a->rows > INT64_MAX / 8 / a->cols || !x || !out || !aligned(x, size) || !aligned(residual, size) ||
        !aligned(out, size) || !aligned(a->device_seed, 8))
        return DDP_ERR_INVALID_ARG;
    DropParams p = {};
    p.x = x;
    p.residual = residual;
    p.out = out;
    p.n = a->rows * a->cols;
    p.cols = a->cols;
    p.x_stride = a->x_stride;
    p.residual_stride = residual ? a->residual_stride : a->x_stride;
    p.out_stride = a->out_stride;
    p.device_seed = a->device_seed;
    p.seed = a->seed;
    p.offset_lo = static_cast<uint32_t>(a->offset);
    p.offset_hi = static_cast<uint32_t>(a->offset >> 32);
    const long long least = std::llrint(a->p * 4294967296.0);
    p.none = least >> 32 != 0;
    p.least = p.none ? 0xffffffffu : static_cast<uint32_t>(least);
    p.scale = p.none ? 0.0f : static_cast<float>(1.0 / (1.0 - a->p));
    const int eight = 8 * size;                             // bytes, and where eights have to start
    const bool vectors = aligned(x, eight) && aligned(residual, eight) && aligned(out, eight);
    const auto strided = [&](int64_t stride) { return stride % 8 != 0; };
    Layout layout = kSingle;
    if (a->rows == 1 || (p.x_stride == p.cols && p.residual_stride == p.cols && p.out_stride == p.cols)) {
        p.cols = p.n;                                       // one run
        if (vectors) layout = kWhole;
    } else if (vectors && p.cols % 8 == 0 && !strided(p.x_stride) && !strided(p.residual_stride) && !strided(p.out_stride)) {
        layout = kRows;
    }
    const long long groups = (p.n + 7) / 8, ctas = (groups + kThreads * kGroups - 1) / (kThreads * kGroups);
    if (ctas > INT32_MAX) return DDP_ERR_INVALID_ARG;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = a->dtype == DDP_F32 ? launch_drop<float>(layout, ctas, p, st) : launch_drop<uint16_t>(layout, ctas, p, st);
    return e == cudaSuccess ? DDP_OK : DDP_ERR_CUDA;
}
