// Rows of a table for tokens, and the table's gradient: the rows' gradients
// summed for each token.
//
// The gradient sorts the tokens first (a stable radix sort, so that equal tokens
// keep their order), and each row of the table then sums its tokens' gradients
// one after another: equal inputs give equal bits, and a row's sum does not depend
// on the other tokens'.  Tokens that fall often are summed in parts of kLong (or
// more) rows by a CTA each, and whoever ends last adds the parts in their order.

#include "ddp_reducer.h"

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "ddp_rows.cuh"

namespace {

using namespace ddpk::rows;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kAhead = 4;              // forward: rows of a thread at once
constexpr int kMaxBits = 8;            // of a digit of the sort
constexpr int kMaxBins = 1 << kMaxBits;
constexpr int kItems = 8;              // of a thread in a tile of the sort
constexpr int kTile = kThreads * kItems;
constexpr int kMaxSortCtas = 128;
constexpr int kLong = 64;              // tokens of a part, at least
constexpr int kMaxParts = 512;         // of one row, at most
constexpr int kUnroll = 8;             // rows on their way at once

struct EmbedParams {
    const void* table;
    const void* tokens;
    void* out;
    long long n, vocab, table_stride, out_stride;
    int dim;
    int wide;                // tokens of 64 bits
    int row_threads;         // of a row, a power of two
    float scale;
};

struct SortParams {
    const void* tokens;      // first pass
    const int* keys_in;      // later ones
    const int* places_in;
    int* keys;
    int* places;
    int* counts;             // [ctas][bins]
    int* tickets;            // zeroed by the first pass
    long long ntickets;
    long long n, vocab, share;     // share: tokens of a CTA, a multiple of kTile
    int wide, ctas, shift, bits;
};

struct SumParams {
    const void* grad;
    const int* keys;
    const int* places;
    void* out;
    float* parts;
    int* tickets;
    long long n, vocab, grad_stride, out_stride, windows;
    int dim, long_row, rows, row_threads;      // long_row: tokens of a part; rows: of the table, of a CTA
    int accumulate;
    float scale;
};

// The row of the table, or -1.
__device__ __forceinline__ long long token_at(const void* tokens, int wide, long long i, long long vocab) {
    const long long t = wide ? static_cast<const long long*>(tokens)[i] : static_cast<const int*>(tokens)[i];
    return t >= 0 && t < vocab ? t : -1;
}

// ---------------------------------------------------------------- forward

template <typename Tin, typename Tout, bool VEC>
__global__ void __launch_bounds__(kThreads) embed_kernel(const __grid_constant__ EmbedParams p) {
    ddpk::dev::pdl_wait();
    ddpk::dev::pdl_trigger();
    constexpr int N = VEC ? 8 : 1;
    const int t = threadIdx.x % p.row_threads, slot = threadIdx.x / p.row_threads, slots = kThreads / p.row_threads;
    const Tin* const table = static_cast<const Tin*>(p.table);
    Tout* const out = static_cast<Tout*>(p.out);
    const long long tile = static_cast<long long>(slots) * kAhead;
    for (long long r0 = blockIdx.x * tile + slot; r0 < p.n; r0 += gridDim.x * tile) {
        long long from[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const long long r = r0 + u * slots;
            from[u] = r < p.n ? token_at(p.tokens, p.wide, r, p.vocab) : -1;
        }
        for (int at = t * N; at < p.dim; at += p.row_threads * N) {
            if constexpr (VEC) {
                Eight<Tin> raw[kAhead];
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    if (from[u] >= 0) raw[u].load(table + from[u] * p.table_stride + at);
                    else raw[u].zero();
                }
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    float f[8];
                    raw[u].get(f);
#pragma unroll
                    for (int j = 0; j < 8; ++j) f[j] *= p.scale;
                    if (from[u] < 0) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) f[j] = 0.0f;       // (and not -0)
                    }
                    Eight<Tout> y;
                    y.put(f);
                    if (r0 + u * slots < p.n) y.store_once(out + (r0 + u * slots) * p.out_stride + at);
                }
            } else {
                float f[kAhead];
#pragma unroll
                for (int u = 0; u < kAhead; ++u)
                    f[u] = from[u] >= 0 ? widen(table[from[u] * p.table_stride + at]) * p.scale : 0.0f;
#pragma unroll
                for (int u = 0; u < kAhead; ++u)
                    if (r0 + u * slots < p.n) out[(r0 + u * slots) * p.out_stride + at] = narrow<Tout>(f[u]);
            }
        }
    }
}

// ---------------------------------------------------------------- sort

// Token i as a key; those outside of the table come last.
__device__ __forceinline__ int key_at(const SortParams& p, long long i) {
    if (p.keys_in) return p.keys_in[i];
    const long long t = token_at(p.tokens, p.wide, i, p.vocab);
    return static_cast<int>(t < 0 ? p.vocab : t);
}

// How often each digit falls in each CTA's share.
__global__ void __launch_bounds__(kThreads) sort_count_kernel(const __grid_constant__ SortParams p) {
    __shared__ int bins[kMaxBins];
    const int nbins = 1 << p.bits;
    for (int b = threadIdx.x; b < nbins; b += kThreads) bins[b] = 0;
    ddpk::dev::pdl_wait();
    ddpk::dev::pdl_trigger();
    for (long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; i < p.ntickets;
         i += static_cast<long long>(gridDim.x) * kThreads)
        p.tickets[i] = 0;
    __syncthreads();
    const long long from = blockIdx.x * p.share, to = min(p.n, from + p.share);
#pragma unroll 4
    for (long long i = from + threadIdx.x; i < to; i += kThreads) atomicAdd(&bins[key_at(p, i) >> p.shift & (nbins - 1)], 1);
    __syncthreads();
    for (int b = threadIdx.x; b < nbins; b += kThreads) p.counts[blockIdx.x * nbins + b] = bins[b];
}

// Each token to its place by the digit, behind the earlier ones of the same.
__global__ void __launch_bounds__(kThreads) sort_move_kernel(const __grid_constant__ SortParams p) {
    __shared__ int next[kMaxBins];                 // place of the next token of a digit
    __shared__ int of_warp[kWarps][kMaxBins];      // in a tile, of each warp: how many, and then where they begin
    __shared__ int totals[kWarps];
    const int nbins = 1 << p.bits, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    ddpk::dev::pdl_wait();
    ddpk::dev::pdl_trigger();
    // a thread a digit: what smaller digits have, and the same in earlier shares
    const int b = threadIdx.x;
    int all = 0, earlier = 0;
    if (b < nbins) {
#pragma unroll 8
        for (int c = 0; c < p.ctas; ++c) {
            const int n = p.counts[c * nbins + b];
            all += n;
            if (c < static_cast<int>(blockIdx.x)) earlier += n;
        }
    }
    int before = all;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
        const int x = __shfl_up_sync(kAll, before, o);
        if (lane >= o) before += x;
    }
    if (lane == 31) totals[warp] = before;
    __syncthreads();
    for (int w = 0; w < warp; ++w) before += totals[w];
    if (b < nbins) next[b] = before - all + earlier;

    const long long from = blockIdx.x * p.share, to = min(p.n, from + p.share);
    for (long long t0 = from; t0 < to; t0 += kTile) {
        for (int i = lane; i < nbins; i += 32) of_warp[warp][i] = 0;
        __syncwarp();
        int key[kItems], place[kItems], rank[kItems];
        const long long mine = t0 + warp * (32 * kItems) + lane;
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const long long at = mine + i * 32;
            key[i] = at < to ? key_at(p, at) : -1;
            place[i] = at < to ? (p.keys_in ? p.places_in[at] : static_cast<int>(at)) : 0;
        }
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const int digit = key[i] < 0 ? nbins : key[i] >> p.shift & (nbins - 1);
            const unsigned same = __match_any_sync(kAll, digit);
            const int first = __ffs(same) - 1;
            int had = 0;
            if (lane == first && key[i] >= 0) {
                had = of_warp[warp][digit];
                of_warp[warp][digit] = had + __popc(same);
            }
            __syncwarp();
            rank[i] = __shfl_sync(kAll, had, first) + __popc(same & ((1u << lane) - 1));
        }
        __syncthreads();
        if (b < nbins) {
            int at = next[b];
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const int n = of_warp[w][b];
                of_warp[w][b] = at;
                at += n;
            }
            next[b] = at;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            if (key[i] < 0) continue;
            const int at = of_warp[warp][key[i] >> p.shift & (nbins - 1)] + rank[i];
            p.keys[at] = key[i];
            p.places[at] = place[i];
        }
        __syncwarp();                              // a warp's own counts alone are cleared next
    }
}

// ---------------------------------------------------------------- sums

// How many of the n sorted keys are below `key`, of which those before lo are
// and those from hi on are not; by a whole warp.
__device__ __forceinline__ long long warp_lower_bound(const int* keys, long long lo, long long hi, long long key) {
    const int lane = threadIdx.x & 31;
    while (hi > lo) {
        const long long step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step - 1;
        const bool below = at < hi && keys[at] < key;
        const int n = __popc(__ballot_sync(kAll, below));       // steps that lie below: the keys are sorted
        lo += n * step;
        hi = min(hi, lo + step - 1);
        if (step == 1) break;
    }
    return lo;
}

__device__ __forceinline__ long long lower_bound(const int* keys, long long lo, long long hi, long long key) {
    while (hi > lo) {
        const long long mid = (lo + hi) / 2;
        if (keys[mid] < key) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

// The gradients at sorted places [lo, hi), columns from `at` on.
template <typename T, bool VEC>
__device__ __forceinline__ void sum_rows(const SumParams& p, long long lo, long long hi, int at, float (&sum)[VEC ? 8 : 1]) {
    constexpr int N = VEC ? 8 : 1;
    const T* const grad = static_cast<const T*>(p.grad);
#pragma unroll
    for (int j = 0; j < N; ++j) sum[j] = 0.0f;
    for (long long i = lo; i < hi; i += kUnroll) {
        if constexpr (VEC) {
            Eight<T> raw[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
                if (i + u < hi) raw[u].load_once(grad + static_cast<long long>(p.places[i + u]) * p.grad_stride + at);
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                if (i + u < hi) {
                    float f[8];
                    raw[u].get(f);
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum[j] += f[j];
                }
            }
        } else {
            float f[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
                f[u] = i + u < hi ? widen(grad[static_cast<long long>(p.places[i + u]) * p.grad_stride + at]) : 0.0f;
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) sum[0] += f[u];
        }
    }
}

// A row of the table's gradient, columns from `at` on.
template <typename Tout, bool VEC>
__device__ __forceinline__ void put_row(const SumParams& p, long long row, int at, const float (&sum)[VEC ? 8 : 1]) {
    Tout* const to = static_cast<Tout*>(p.out) + row * p.out_stride + at;
    if constexpr (VEC) {
        float f[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = sum[j] * p.scale;
        Eight<Tout> raw;
        if (p.accumulate) {
            float old[8];
            raw.load_once(to);
            raw.get(old);
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] += old[j];
        }
        raw.put(f);
        raw.store_once(to);
    } else {
        *to = narrow<Tout>(p.accumulate ? widen(*to) + sum[0] * p.scale : sum[0] * p.scale);
    }
}

// The first `windows` CTAs look for long rows: each takes the parts that begin in
// its window of long_row sorted places (at most one that is its row's first, and
// one that is not: a part's slot is 2 window + (first)).  The others take `rows`
// rows of the table each, but the long ones.
template <typename T, typename Tout, bool VEC>
__global__ void __launch_bounds__(kThreads) embed_sum_kernel(const __grid_constant__ SumParams p) {
    constexpr int N = VEC ? 8 : 1;
    __shared__ long long bounds[4];
    __shared__ long long starts[kThreads + 1];
    __shared__ int last;
    const int warp = threadIdx.x >> 5;
    ddpk::dev::pdl_wait();
    ddpk::dev::pdl_trigger();
    if (blockIdx.x < p.windows) {
        // a long row that begins behind the window's start reaches past its end, so the
        // rows at both ends are all that can have a part here
        const long long w0 = static_cast<long long>(blockIdx.x) * p.long_row, w1 = w0 + p.long_row;
        const int key0 = p.keys[w0], key1 = w1 < p.n ? p.keys[w1] : key0;
        if (warp < 4) {
            const long long at = warp < 2 ? w0 : min(w1, p.n - 1), key = warp < 2 ? key0 : key1;
            const long long x = warp_lower_bound(p.keys, warp & 1 ? at : 0, warp & 1 ? p.n : at, key + (warp & 1));
            if ((threadIdx.x & 31) == 0) bounds[warp] = x;
        }
        __syncthreads();
        for (int which = 0; which < 2; ++which) {
            const int key = which ? key1 : key0;
            if (key >= p.vocab || (which && key1 == key0)) break;
            const long long start = bounds[2 * which], end = bounds[2 * which + 1], count = end - start;
            const long long part = start > w0 ? 0 : (w0 - start + p.long_row - 1) / p.long_row, from = start + part * p.long_row;
            if (count <= p.long_row || from >= min(w1, end)) continue;
            const long long to = min(end, from + p.long_row), nparts = (count + p.long_row - 1) / p.long_row;
            float* const mine = p.parts + (2LL * blockIdx.x + (part == 0)) * p.dim;
            for (int at = threadIdx.x * N; at < p.dim; at += kThreads * N) {
                float sum[N];
                sum_rows<T, VEC>(p, from, to, at, sum);
#pragma unroll
                for (int j = 0; j < N; ++j) __stcg(mine + at + j, sum[j]);
            }
            __threadfence();
            __syncthreads();
            if (threadIdx.x == 0) last = atomicAdd(p.tickets + start / p.long_row, 1) == nparts - 1;
            __syncthreads();
            if (last) {
                __threadfence();
                for (int at = threadIdx.x * N; at < p.dim; at += kThreads * N) {
                    float sum[N] = {};
                    for (long long q = 0; q < nparts; ++q) {
                        const long long window = (start + q * p.long_row) / p.long_row;
                        const float* const from_part = p.parts + (2 * window + (q == 0)) * p.dim + at;
#pragma unroll
                        for (int j = 0; j < N; ++j) sum[j] += __ldcg(from_part + j);
                    }
                    put_row<Tout, VEC>(p, key, at, sum);
                }
            }
            __syncthreads();
        }
        return;
    }
    const long long v0 = static_cast<long long>(blockIdx.x - p.windows) * p.rows, v1 = min(p.vocab, v0 + p.rows);
    if (warp < 2) {
        const long long x = warp_lower_bound(p.keys, 0, p.n, warp ? v1 : v0);
        if ((threadIdx.x & 31) == 0) bounds[warp] = x;
    }
    __syncthreads();
    for (int r = threadIdx.x; r <= v1 - v0; r += kThreads) starts[r] = lower_bound(p.keys, bounds[0], bounds[1], v0 + r);
    __syncthreads();
    const int t = threadIdx.x % p.row_threads, slot = threadIdx.x / p.row_threads, slots = kThreads / p.row_threads;
    for (int r = slot; r < v1 - v0; r += slots) {
        const long long lo = starts[r], hi = starts[r + 1];
        if (hi - lo > p.long_row || (lo == hi && p.accumulate)) continue;
        for (int at = t * N; at < p.dim; at += p.row_threads * N) {
            float sum[N];
            sum_rows<T, VEC>(p, lo, hi, at, sum);
            put_row<Tout, VEC>(p, v0 + r, at, sum);
        }
    }
}

// ---------------------------------------------------------------- host

struct Plan {
    int sort_ctas, passes, bits, long_row;
    long long share, windows;
    int64_t keys, places, counts, parts, tickets, bytes;      // offsets into the workspace; two of the first two
};

int64_t up(int64_t x) { return (x + 255) / 256 * 256; }

Plan plan_of(const ddp_embed_args* a) {
    Plan q = {};
    const int64_t n = a->tokens;
    int bits = 1;
    while (a->vocab >> bits) ++bits;                            // keys reach vocab itself
    q.passes = (bits + kMaxBits - 1) / kMaxBits;
    q.bits = (bits + q.passes - 1) / q.passes;
    const int64_t tiles = (n + kTile - 1) / kTile, each = (tiles + kMaxSortCtas - 1) / kMaxSortCtas;
    q.share = each * kTile;
    q.sort_ctas = static_cast<int>((n + q.share - 1) / q.share);
    q.long_row = kLong;
    while (static_cast<int64_t>(q.long_row) * kMaxParts < n) q.long_row *= 2;
    q.windows = (n + q.long_row - 1) / q.long_row;
    int64_t at = 0;
    q.keys = at;
    at += 2 * up(4 * n);
    q.places = at;
    at += 2 * up(4 * n);
    q.counts = at;
    at += up(4LL * kMaxBins * q.sort_ctas);
    q.tickets = at;
    at += up(4 * q.windows);
    q.parts = at;
    at += up(8 * q.windows * a->dim);
    q.bytes = at;
    return q;
}

bool valid(const ddp_embed_args* a) {
    return a && a->tokens >= 0 && a->tokens <= INT32_MAX && a->vocab >= 1 && a->vocab < INT32_MAX && a->dim >= 1 &&
           a->dim <= 1 << 24 && a->table_stride >= a->dim && a->row_stride >= a->dim && std::isfinite(a->scale) &&
           (a->table_dtype == DDP_F32 || a->table_dtype == DDP_BF16) && (a->dtype == DDP_F32 || a->dtype == DDP_BF16) &&
           (a->index_bits == 32 || a->index_bits == 64);
}

int size_of(int dtype) { return dtype == DDP_F32 ? 4 : 2; }

bool vectors(const ddp_embed_args* a, const void* table, const void* rows) {
    return a->dim % 8 == 0 && aligned(table, 16) && aligned(rows, 16) &&
           (a->vocab == 1 || a->table_stride * size_of(a->table_dtype) % 16 == 0) &&
           (a->tokens == 1 || a->row_stride * size_of(a->dtype) % 16 == 0);
}

int row_threads(int64_t dim, bool vec) {
    const int64_t pieces = vec ? dim / 8 : dim;
    return pieces >= kThreads ? kThreads : power_of_two(pieces);
}

template <typename Tin, typename Tout>
cudaError_t embed_as(bool vec, long long ctas, const EmbedParams& p, cudaStream_t stream) {
    return launch(vec ? embed_kernel<Tin, Tout, true> : embed_kernel<Tin, Tout, false>, ctas, kThreads, 0, stream, p);
}

template <typename T, typename Tout>
cudaError_t sum_as(bool vec, long long ctas, const SumParams& p, cudaStream_t stream) {
    return launch(vec ? embed_sum_kernel<T, Tout, true> : embed_sum_kernel<T, Tout, false>, ctas, kThreads, 0, stream, p);
}

}  // namespace

extern "C" {

int ddp_embed(const ddp_embed_args* a, const void* table, const void* tokens, void* out, void* stream) {
    if (!valid(a)) return DDP_ERR_INVALID_ARG;
    if (a->tokens == 0) return DDP_OK;
    if (!table || !tokens || !out || !aligned(table, size_of(a->table_dtype)) || !aligned(out, size_of(a->dtype)) ||
        !aligned(tokens, a->index_bits / 8))
        return DDP_ERR_INVALID_ARG;
    EmbedParams p = {};
    p.table = table;
    p.tokens = tokens;
    p.out = out;
    p.n = a->tokens;
    p.vocab = a->vocab;
    p.dim = static_cast<int>(a->dim);
    p.table_stride = a->table_stride;
    p.out_stride = a->row_stride;
    p.wide = a->index_bits == 64;
    p.scale = a->scale;
    const bool vec = vectors(a, table, out);
    p.row_threads = row_threads(a->dim, vec);
    const long long tile = static_cast<long long>(kThreads / p.row_threads) * kAhead;
    const long long ctas = (p.n + tile - 1) / tile;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool in32 = a->table_dtype == DDP_F32, out32 = a->dtype == DDP_F32;
    const cudaError_t e = in32 ? (out32 ? embed_as<float, float>(vec, ctas, p, st) : embed_as<float, uint16_t>(vec, ctas, p, st))
                               : (out32 ? embed_as<uint16_t, float>(vec, ctas, p, st) : embed_as<uint16_t, uint16_t>(vec, ctas, p, st));
    return e == cudaSuccess ? DDP_OK : DDP_ERR_CUDA;
}

int64_t ddp_embed_workspace(const ddp_embed_args* a) {
    if (!valid(a)) return DDP_ERR_INVALID_ARG;
    return a->tokens ? plan_of(a).bytes : 0;
}

int ddp_embed_backward(const ddp_embed_args* a, const void* grad, const void* tokens, void* grad_table, int32_t accumulate,
                       void* workspace, void* stream) {
    if (!valid(a) || (accumulate && a->table_dtype != DDP_F32)) return DDP_ERR_INVALID_ARG;
    if (!grad_table || !aligned(grad_table, size_of(a->table_dtype))) return DDP_ERR_INVALID_ARG;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (a->tokens == 0) {
        if (accumulate) return DDP_OK;
        const size_t size = size_of(a->table_dtype);
        return cudaMemset2DAsync(grad_table, a->table_stride * size, 0, a->dim * size, a->vocab, st) == cudaSuccess
                   ? DDP_OK : DDP_ERR_CUDA;
    }
    if (!grad || !tokens || !workspace || !aligned(grad, size_of(a->dtype)) || !aligned(tokens, a->index_bits / 8) ||
        !aligned(workspace, 16))
        return DDP_ERR_INVALID_ARG;
    const Plan q = plan_of(a);
    uint8_t* const ws = static_cast<uint8_t*>(workspace);
    int* const keys[2] = {reinterpret_cast<int*>(ws + q.keys), reinterpret_cast<int*>(ws + q.keys + up(4 * a->tokens))};
    int* const places[2] = {reinterpret_cast<int*>(ws + q.places), reinterpret_cast<int*>(ws + q.places + up(4 * a->tokens))};
    SortParams s = {};
    s.tokens = tokens;
    s.counts = reinterpret_cast<int*>(ws + q.counts);
    s.tickets = reinterpret_cast<int*>(ws + q.tickets);
    s.n = a->tokens;
    s.vocab = a->vocab;
    s.share = q.share;
    s.wide = a->index_bits == 64;
    s.ctas = q.sort_ctas;
    s.bits = q.bits;
    cudaError_t e = cudaSuccess;
    for (int pass = 0; pass < q.passes && e == cudaSuccess; ++pass) {
        s.shift = pass * q.bits;
        s.keys_in = pass ? keys[(pass - 1) & 1] : nullptr;
        s.places_in = pass ? places[(pass - 1) & 1] : nullptr;
        s.keys = keys[pass & 1];
        s.places = places[pass & 1];
        s.ntickets = pass ? 0 : q.windows;
        e = launch(sort_count_kernel, s.ctas, kThreads, 0, st, s);
        if (e == cudaSuccess) e = launch(sort_move_kernel, s.ctas, kThreads, 0, st, s);
    }
    if (e != cudaSuccess) return DDP_ERR_CUDA;
    SumParams p = {};
    p.grad = grad;
    p.keys = s.keys;
    p.places = s.places;
    p.out = grad_table;
    p.parts = reinterpret_cast<float*>(ws + q.parts);
    p.tickets = s.tickets;
    p.n = a->tokens;
    p.vocab = a->vocab;
    p.dim = static_cast<int>(a->dim);
    p.grad_stride = a->row_stride;
    p.out_stride = a->table_stride;
    p.windows = q.windows;
    p.long_row = q.long_row;
    p.accumulate = accumulate != 0;
    p.scale = a->scale;
    const bool vec = vectors(a, grad_table, grad);
    p.row_threads = row_threads(a->dim, vec);
    const int slots = kThreads / p.row_threads;
    p.rows = slots * 4 < 16 ? 16 : slots * 4 < kThreads ? slots * 4 : kThreads;
    const long long ctas = p.windows + (p.vocab + p.rows - 1) / p.rows;
    const bool in32 = a->dtype == DDP_F32, out32 = a->table_dtype == DDP_F32;
    e = in32 ? (out32 ? sum_as<float, float>(vec, ctas, p, st) : sum_as<float, uint16_t>(vec, ctas, p, st))
             : (out32 ? sum_as<uint16_t, float>(vec, ctas, p, st) : sum_as<uint16_t, uint16_t>(vec, ctas, p, st));
    return e == cudaSuccess ? DDP_OK : DDP_ERR_CUDA;
}

}  // extern "C"
