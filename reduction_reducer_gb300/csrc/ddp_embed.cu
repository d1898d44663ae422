// Rows of a table for tokens, and the table's gradient: the rows' gradients
// summed for each token.
//
// The gradient sorts the tokens first (a stable radix sort, so that equal tokens
// keep their order), and each row of the table then sums its tokens' gradients
// one after another: equal inputs give equal bits, and a row's sum does not depend
// on the other tokens'.  A word that falls often is summed in parts of kPart
// tokens, and whoever ends last adds the parts (groups of them) in their order.
// Atomic additions in the tokens' stead would need no sort, but leave the order
// open, and a common word's additions would queue at one address.

#include "ddp_reducer.h"

#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "ddp_rows.cuh"

namespace {

using namespace ddpk::rows;

constexpr int kThreads = 256;
constexpr int kAhead = 4;              // forward: rows of a thread at once
constexpr int kColumns = 4;            // and, where they do not lie in vectors, columns of each,
constexpr int kShiftColumns = 96;      // while these are fewer (65,536 rows of 45 bf16: by columns 7.2 us, shifted 16.9; 133: 22.0, 16.9)
constexpr int kMaxBits = 8;            // of a digit of the sort
constexpr int kMaxBins = 1 << kMaxBits;
constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kItems = 4;              // of a thread in a tile of the sort
constexpr int kTile = kSortThreads * kItems;
constexpr int kMaxSortCtas = 128;
constexpr int kSmall = 8192;           // tokens that are sorted by counting
constexpr int kRankLanes = 16;
constexpr int kPart = 32;              // sorted places of a window, and tokens that are summed in one go
constexpr int kGroup = 32;             // parts of a row that are added up in one go
constexpr int kChunk = 256;            // columns of a warp
// Rows of a warp on their way, with the one under work.
template <typename T> constexpr int kRing = sizeof(T) == 2 ? 8 : 4;
// Words of one.
template <typename T, bool VEC> constexpr int slot_of = kChunk * static_cast<int>(sizeof(T)) / 16 + (VEC ? 0 : 1);
// Shares of a window, while there are fewer warps: one place each where the GPU
// would not be full (111 tokens of 14 columns: four shares 9.2 us, eight 7.3, 32 6.1), and two
// where warps would not be many (65,536 tokens onto 50,257 rows of 1,024: one 76.7, two 73.7, four
// 76.1; of 64: one 41.4, two 41.3, four 45.1, eight 50.4).
constexpr int kMaxSplits = 32, kFewWarps = kSms * 24;
constexpr int kMoreSplits = 2, kMoreWarps = kSms * 96;
constexpr int64_t kMaxTokens = 1 << 24;      // of a gradient: groups of a row's parts are counted in 15 bits
constexpr int kFillBytes = 64 * 1024;  // of the rows that a CTA looks at for empty ones

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
    int* counts;             // [ctas][bins] of this pass
    int* next_counts;        // and of the next one, zeros before (NULL: there is none)
    long long nzeros;        // first pass: counts to be zeroed, a multiple of four
    int* tickets;            // zeroed by the first pass
    long long ntickets;      // a multiple of four
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
    long long n, vocab, grad_stride, out_stride, windows, tickets_each;
    int dim, rows, row_threads;                // rows: of the table, of a CTA
    int splits, chunks;                        // shares of a window; kChunk columns of a row
    unsigned sum_ctas;
    int accumulate;
    float scale;
};

// The row of the table, or -1.
__device__ __forceinline__ long long token_at(const void* tokens, int wide, long long i, long long vocab) {
    const long long t = wide ? static_cast<const long long*>(tokens)[i] : static_cast<const int*>(tokens)[i];
    return t >= 0 && t < vocab ? t : -1;
}

// ---------------------------------------------------------------- forward

// out[i] = scale table[tokens[i]].  A thread has kAhead rows' eight columns on their
// way at once; a row is as many threads as it has eights.  65,536 rows of 1,024
// from fp32 to bf16: 38.3 us, 189 MB from and to HBM (4.9 TB/s, floor 28 us).  What
// bounds it is latency: a CTA has one tile, and waits for its tokens and then for
// their rows; HBM is at 44 % of its rate and L2, from which common words' rows come
// again and again, at 39 %, with 41 % of the warps resident.  So occupancy is what
// it lives on: three CTAs an SM 45.2 us, four 38.9; of bf16 tables, which leave more
// registers, four 35.0 and five 31.2.  Rows that do not lie in vectors and are short
// go element by element.
template <typename Tin, typename Tout, bool VEC>
__global__ void __launch_bounds__(kThreads, VEC && sizeof(Tin) == 2 ? 5 : 4) embed_kernel(const __grid_constant__ EmbedParams p) {
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
        for (int at = t * N; at < p.dim; at += p.row_threads * (VEC ? N : kColumns)) {
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
                    const float2 s = both(from[u] >= 0 ? p.scale : 0.0f);      // (no -0 where there is no row)
#pragma unroll
                    for (int j = 0; j < 8; j += 2) {
                        const float2 d = mul2(make_float2(f[j], f[j + 1]), s);
                        f[j] = d.x;
                        f[j + 1] = d.y;
                    }
                    Eight<Tout> y;
                    y.put(f);
                    if (r0 + u * slots < p.n) y.store_wide(out + (r0 + u * slots) * p.out_stride + at);
                }
            } else {
                float f[kAhead][kColumns];
#pragma unroll
                for (int u = 0; u < kAhead; ++u)
#pragma unroll
                    for (int k = 0; k < kColumns; ++k) {
                        const int col = at + k * p.row_threads;
                        f[u][k] = from[u] >= 0 && col < p.dim ? widen(table[from[u] * p.table_stride + col]) : 0.0f;
                    }
#pragma unroll
                for (int u = 0; u < kAhead; ++u)
#pragma unroll
                    for (int k = 0; k < kColumns; ++k) {
                        const int col = at + k * p.row_threads;
                        if (r0 + u * slots < p.n && col < p.dim)
                            out[(r0 + u * slots) * p.out_stride + col] = narrow<Tout>(from[u] >= 0 ? f[u][k] * p.scale : 0.0f);
                    }
            }
        }
    }
}

// Rows that do not lie in vectors, a warp each: eights that start on 16 bytes of the
// result, shifted out of the aligned words that the table's row lies in; a lane
// loads those that its eights begin in, and has the next lane's for their ends.  No
// word is loaded that does not hold an element of the row.  65,493 rows of 1,023
// from fp32 to bf16 54 us, from bf16 37 (floor 29 and 25; 92 and 110 by columns).
template <typename Tin, typename Tout>
__global__ void __launch_bounds__(kThreads, 4) embed_shift_kernel(const __grid_constant__ EmbedParams p) {
    constexpr int kEights = sizeof(Tin) == 2 ? 4 : 2;
    ddpk::dev::pdl_wait();
    ddpk::dev::pdl_trigger();
    const int lane = threadIdx.x & 31;
    const long long r = static_cast<long long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    if (r >= p.n) return;
    const long long token = token_at(p.tokens, p.wide, r, p.vocab);
    const bool zero = token < 0;
    Tout* const out = static_cast<Tout*>(p.out) + r * p.out_stride;
    const int head = min(p.dim, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(out) & 15)) % 16 / sizeof(Tout)));
    const int units = (p.dim - head) / 8, ends = p.dim - 8 * units;
    const Tin* const from = static_cast<const Tin*>(p.table) + (zero ? 0 : token) * p.table_stride;
    const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(from + head) & 15);
    const Tin* const words = reinterpret_cast<const Tin*>(reinterpret_cast<const char*>(from + head) - shift);
    if (lane < ends) {                                     // at most seven elements of each end
        const int i = lane < head ? lane : lane + 8 * units;
        out[i] = narrow<Tout>(zero ? 0.0f : widen(from[i]) * p.scale);
    }
    for (int i0 = 0; i0 < units; i0 += 32 * kEights) {
        Eight<Tin> raw[kEights];
        uint4 last = make_uint4(0, 0, 0, 0);                // lane 0: what follows the warp's eights
#pragma unroll
        for (int u = 0; u < kEights; ++u) {
            const int i = i0 + u * 32 + lane;
            raw[u].zero();
            if (!zero && i < units) raw[u].load(words + 8 * i);
            else if (!zero && i == units && shift) *reinterpret_cast<uint4*>(&raw[u]) = *reinterpret_cast<const uint4*>(words + 8 * i);
        }
        if (!zero && shift && lane == 0 && i0 + 32 * kEights <= units)
            last = *reinterpret_cast<const uint4*>(words + 8 * (i0 + 32 * kEights));
#pragma unroll
        for (int u = 0; u < kEights; ++u) {
            const int i = i0 + u * 32 + lane;
            if (i - lane >= units) break;                  // the whole warp's
            if (shift && !zero) {
                const uint4 mine = *reinterpret_cast<const uint4*>(&raw[u]);
                const uint4 ahead = u + 1 < kEights ? *reinterpret_cast<const uint4*>(&raw[u + 1 < kEights ? u + 1 : 0]) : last;
                const uint4 give = lane == 0 ? ahead : mine;        // lane 0 to lane 31
                const int next = (lane + 1) & 31;
                const uint4 behind = make_uint4(__shfl_sync(kAll, give.x, next), __shfl_sync(kAll, give.y, next),
                                                __shfl_sync(kAll, give.z, next), __shfl_sync(kAll, give.w, next));
                raw[u] = shifted(raw[u], behind, shift);
            }
            if (i >= units) continue;
            float f[8];
            raw[u].get(f);
            const float2 s = both(zero ? 0.0f : p.scale);
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const float2 d = mul2(make_float2(f[j], f[j + 1]), s);
                f[j] = d.x;
                f[j + 1] = d.y;
            }
            Eight<Tout> y;
            y.put(f);
            y.store_once(out + head + 8 * i);
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

// A stable counting sort of 32-bit keys, digit by digit, a share of the tokens a
// CTA.  It is latency (a few trips to L2 a launch): 65,536 tokens onto 50,257 rows
// are two digits of eight bits in three launches, 4 + 9 + 7 us.

// How often each value of the first digit falls in each CTA's share.
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const __grid_constant__ SortParams p) {
    __shared__ int bins[kMaxBins];
    const int nbins = 1 << p.bits;
    for (int b = threadIdx.x; b < nbins; b += kSortThreads) bins[b] = 0;
    ddpk::dev::pdl_wait();
    ddpk::dev::pdl_trigger();
    for (long long i = static_cast<long long>(blockIdx.x) * kSortThreads + threadIdx.x; i < p.ntickets / 4;
         i += static_cast<long long>(gridDim.x) * kSortThreads)
        reinterpret_cast<int4*>(p.tickets)[i] = make_int4(0, 0, 0, 0);
    for (long long i = static_cast<long long>(blockIdx.x) * kSortThreads + threadIdx.x; i < p.nzeros / 4;
         i += static_cast<long long>(gridDim.x) * kSortThreads)
        reinterpret_cast<int4*>(p.next_counts)[i] = make_int4(0, 0, 0, 0);
    __syncthreads();
    const long long from = blockIdx.x * p.share, to = min(p.n, from + p.share);
#pragma unroll 4
    for (long long i = from + threadIdx.x; i < to; i += kSortThreads) atomicAdd(&bins[key_at(p, i) >> p.shift & (nbins - 1)], 1);
    __syncthreads();
    for (int b = threadIdx.x; b < nbins; b += kSortThreads) p.counts[blockIdx.x * nbins + b] = bins[b];
}

// Each token to its place by the digit, behind the earlier ones of the same; and
// how often the next digit falls in each share that tokens are moved to.
__global__ void __launch_bounds__(kSortThreads) sort_move_kernel(const __grid_constant__ SortParams p) {
    constexpr int kHalves = kSortThreads / kMaxBins;
    __shared__ int next[kMaxBins];                 // place of the next token of a digit
    __shared__ int of_warp[kSortWarps][kMaxBins];  // in a tile, of each warp: how many, and then where they begin
    __shared__ int2 halves[kHalves][kMaxBins];
    __shared__ int totals[kMaxBins / 32];
    const int nbins = 1 << p.bits, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, b = threadIdx.x % kMaxBins;
    const long long from = blockIdx.x * p.share, to = min(p.n, from + p.share);
    int key[kItems], place[kItems], rank[kItems];
    const auto load = [&](long long t0) {
#pragma unroll
        for (int i = 0; i < kItems; ++i) {
            const long long at = t0 + warp * (32 * kItems) + lane + i * 32;
            key[i] = at < to ? key_at(p, at) : -1;
            place[i] = at < to ? (p.keys_in ? p.places_in[at] : static_cast<int>(at)) : 0;
        }
    };
    ddpk::dev::pdl_wait();
    ddpk::dev::pdl_trigger();
    load(from);
    // what smaller digits have, and the same in earlier shares: a digit's counts by kHalves threads
    int2 sum = make_int2(0, 0);
    if (b < nbins) {
#pragma unroll 16
        for (int c = threadIdx.x / kMaxBins; c < p.ctas; c += kHalves) {
            const int n = p.counts[c * nbins + b];
            sum.x += n;
            if (c < static_cast<int>(blockIdx.x)) sum.y += n;
        }
    }
    halves[threadIdx.x / kMaxBins][b] = sum;
    __syncthreads();
    int all = 0, before = 0, earlier = 0;
    if (threadIdx.x < kMaxBins) {
#pragma unroll
        for (int h = 0; h < kHalves; ++h) { all += halves[h][b].x; earlier += halves[h][b].y; }
        before = all;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int x = __shfl_up_sync(kAll, before, o);
            if (lane >= o) before += x;
        }
        if (lane == 31) totals[warp] = before;
    }
    __syncthreads();
    if (threadIdx.x < kMaxBins) {
        for (int w = 0; w < warp; ++w) before += totals[w];
        next[b] = before - all + earlier;
    }
    for (long long t0 = from; t0 < to; t0 += kTile) {
        if (t0 > from) load(t0);
        for (int i = lane; i < nbins; i += 32) of_warp[warp][i] = 0;
        __syncwarp();
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
        if (threadIdx.x < nbins) {
            int at = next[b];
#pragma unroll
            for (int w = 0; w < kSortWarps; ++w) {
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
            if (p.next_counts)
                atomicAdd(p.next_counts + static_cast<unsigned>(at) / static_cast<unsigned>(p.share) * nbins +
                              (key[i] >> p.shift >> p.bits & (nbins - 1)), 1);
        }
        __syncwarp();                              // a warp's own counts alone are cleared next
    }
}

// Few tokens: each one's place is the number of smaller ones and of equal ones
// before it, counted against all of them by kRankLanes lanes, each with every
// kRankLanes-th four.  4,096 tokens are a million warp instructions, spread over
// all SMs in one launch.
__global__ void __launch_bounds__(kThreads) sort_small_kernel(const __grid_constant__ SortParams p) {
    extern __shared__ int4 all[];
    const int n = static_cast<int>(p.n), fours = (n + 3) / 4;
    ddpk::dev::pdl_wait();
    ddpk::dev::pdl_trigger();
    for (long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; i < p.ntickets / 4;
         i += static_cast<long long>(gridDim.x) * kThreads)
        reinterpret_cast<int4*>(p.tickets)[i] = make_int4(0, 0, 0, 0);
#pragma unroll 8
    for (int i = threadIdx.x; i < 4 * fours; i += kThreads) reinterpret_cast<int*>(all)[i] = i < n ? key_at(p, i) : INT32_MAX;
    __syncthreads();
    const int i = blockIdx.x * (kThreads / kRankLanes) + threadIdx.x / kRankLanes, lane = threadIdx.x % kRankLanes;
    const int key = i < n ? reinterpret_cast<const int*>(all)[i] : 0, mine = i / 4;
    int rank = 0;
#pragma unroll 4
    for (int c = lane; c < fours; c += kRankLanes) {
        const int4 x = all[c];
        const int least = key + (c < mine);                  // equal ones count before this token's four
        rank += (x.x < least) + (x.y < least) + (x.z < least) + (x.w < least);
    }
    if (lane == mine % kRankLanes && i < n)                  // and within it
        for (int j = 4 * mine; j < i; ++j) rank += reinterpret_cast<const int*>(all)[j] == key;
#pragma unroll
    for (int o = kRankLanes / 2; o; o /= 2) rank += __shfl_xor_sync(kAll, rank, o);
    if (lane == 0 && i < n) {
        p.keys[rank] = key;
        p.places[rank] = i;
    }
}

// ---------------------------------------------------------------- sums

// How many of the n sorted keys are below `key`, of which those before lo are
// and those from hi on are not; by a whole warp.
__device__ __forceinline__ long long warp_lower_bound(const int* keys, long long lo, long long hi, long long key) {
    const int lane = threadIdx.x & 31;
    while (hi > lo) {
        const long long step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step - 1;
        const bool below = at < hi && __ldcg(keys + at) < key;
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
        if (__ldcg(keys + mid) < key) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

// The eight columns of a lane among the kChunk of its warp: next to one another,
// or (rows that do not lie in vectors) every 32nd.
template <bool VEC>
struct Columns {
    int first, dim;

    __device__ __forceinline__ Columns(int chunk, int dim)
        : first(chunk * kChunk + (threadIdx.x & 31) * (VEC ? 8 : 1)), dim(dim) {}
    __device__ __forceinline__ int at(int j) const { return first + j * (VEC ? 1 : 32); }
    __device__ __forceinline__ bool on(int j) const { return (VEC ? first : at(j)) < dim; }
};

struct Sum {
    float v[8];
    bool whole;              // a row's, not a part's
};

// Additions that are not waited for (red) take numbers below 2^-126 for zeros.  Where
// what is added is kLeast or more that changes nothing: beside it such a number is
// less than half a step, and what is left of two numbers of that size is a multiple
// of 2^-125.  Less than that, zeros too, is added to what is loaded: 65,536 rows of
// 1,024 in bf16 onto 50,257, a tenth of the elements zeros, 76 us, without zeros 74.
constexpr float kLeast = 0x1p-101f;

__device__ __forceinline__ void add_later(float* to, float x) {
    asm volatile("red.relaxed.gpu.global.add.f32 [%0], %1;" ::"l"(to), "f"(x) : "memory");
}

// Rows that do not lie in vectors, where some of what is added is that small; adding
// zero is left out.
__device__ __noinline__ void add_small(float* to, Columns<false> c, Sum f) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        if (!c.on(j) || f.v[j] == 0.0f) continue;
        if (fabsf(f.v[j]) < kLeast) to[c.at(j)] += f.v[j];
        else add_later(to + c.at(j), f.v[j]);
    }
}

// A row of the table's gradient: one addition for each element, so no order is left
// open.
template <typename Tout, bool VEC>
__device__ __forceinline__ void put_row(const SumParams& p, long long row, const Columns<VEC>& c, const Sum& sum) {
    Tout* const to = static_cast<Tout*>(p.out) + row * p.out_stride;
    Sum f = sum;
#pragma unroll
    for (int j = 0; j < 8; ++j) f.v[j] *= p.scale;
    if constexpr (sizeof(Tout) == 4) {
        if (p.accumulate) {
            bool small = false;
            if constexpr (VEC) {
                if (!c.on(0)) return;
#pragma unroll
                for (int j = 0; j < 8; ++j) small |= fabsf(f.v[j]) < kLeast;
                if (small) {
                    Eight<Tout> there;
                    there.load_wide(to + c.first);
                    there.add_to(f.v);
                    there.put(f.v);
                    there.store_wide(to + c.first);
                    return;
                }
#pragma unroll
                for (int j = 0; j < 8; j += 4)
                    asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(to + c.first + j), "f"(f.v[j]),
                                 "f"(f.v[j + 1]), "f"(f.v[j + 2]), "f"(f.v[j + 3]) : "memory");
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) small |= c.on(j) && fabsf(f.v[j]) < kLeast && f.v[j] != 0.0f;
                if (small) return add_small(to, c, f);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (c.on(j) && f.v[j] != 0.0f) add_later(to + c.at(j), f.v[j]);
            }
            return;
        }
    }
    if constexpr (VEC) {
        Eight<Tout> raw;
        raw.put(f.v);
        if (c.on(0)) raw.store_wide(to + c.first);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (c.on(j)) to[c.at(j)] = narrow<Tout>(f.v[j]);
    }
}

// A warp's columns of part m of a row of more than kPart tokens, whose first is at
// sorted place `start`, are summed: keeps them, and, where this warp is the last
// of a group of kGroup parts (and its group the row's last), adds up the group's
// (and the groups') in their order and gives the whole.  A window of kPart places
// holds at most two beginnings of parts, of which one is its row's first: each
// has a slot of its own.  Tickets count arrivals; that of the row's end, which
// alone knows how many there are, adds their number above kArrivals.
template <bool VEC>
__device__ __noinline__ Sum join_parts(const SumParams& p, long long start, int m, bool ends, int chunk, Sum sum) {
    constexpr int kArrivals = 1 << 16, kMask = kArrivals - 1;
    const Columns<VEC> c(chunk, p.dim);
    const int lane = threadIdx.x & 31, group = m / kGroup * kGroup;
    const auto slot = [&](int part) { return (start + static_cast<long long>(part) * kPart) / kPart * 2 + (part == 0); };
    const auto put = [&](int part) {
        float* const to = p.parts + slot(part) * p.dim;
        if constexpr (VEC) {
            if (c.on(0)) {
                __stcg(reinterpret_cast<float4*>(to + c.first), make_float4(sum.v[0], sum.v[1], sum.v[2], sum.v[3]));
                __stcg(reinterpret_cast<float4*>(to + c.first) + 1, make_float4(sum.v[4], sum.v[5], sum.v[6], sum.v[7]));
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c.on(j)) __stcg(to + c.at(j), sum.v[j]);
        }
        __threadfence();
        __syncwarp();
    };
    const auto arrive = [&](int* tickets, int part, int count) {
        int now = 0;
        if (lane == 0) {
            const int add = 1 + count * kArrivals;
            now = atomicAdd(tickets + slot(part) * p.chunks + chunk, add) + add;
        }
        return __shfl_sync(kAll, now, 0);
    };
    const auto add = [&](int from, int to, int step) {
        __threadfence();
#pragma unroll
        for (int j = 0; j < 8; ++j) sum.v[j] = 0.0f;
#pragma unroll 8
        for (int q = from; q < to; q += step) {
            const float* const x = p.parts + slot(q) * p.dim;
            float f[8] = {};
            if constexpr (VEC) {
                if (c.on(0)) {
                    const float4 a = __ldcg(reinterpret_cast<const float4*>(x + c.first)), b = __ldcg(reinterpret_cast<const float4*>(x + c.first) + 1);
                    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w; f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
                }
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) f[j] = c.on(j) ? __ldcg(x + c.at(j)) : 0.0f;
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) sum.v[j] += f[j];
        }
    };
    sum.whole = false;
    put(m);
    const int here = arrive(p.tickets, group, ends ? m - group + 1 : 0), arrived = here & kMask, due = here / kArrivals;
    if (arrived != (due ? due : kGroup)) return sum;
    add(group, group + arrived, 1);
    if (group || !due) {                                         // (else the row's only group)
        put(group);
        const int all = arrive(p.tickets + p.tickets_each, 0, due ? group / kGroup + 1 : 0);
        if ((all & kMask) != all / kArrivals) return sum;
        add(0, all / kArrivals * kGroup, kGroup);
    }
    sum.whole = true;
    return sum;
}

// A warp sums kChunk columns of the rows, and parts of rows, that begin among some
// of the kPart sorted places of a window (all of them, or, with `splits`, a share),
// one after another, with the next ones' gradients on their way to shared memory.
// It needs no other warp: the window's keys and places lie in its lanes.  The
// loop over rows is short code on purpose: a warp that sums a few rows would wait
// longer for instructions than for the rows.
// 65,536 rows of 1,024 in bf16, added to fp32 rows: 134 MB read, and 130 MB of the
// table's rows read and written, in 57 us cold (74 with the sort, floor 39); without
// the copies ahead 114 with the sort.  2.43 instructions a cycle while an SM has warps
// (62 % of what a scheduler can issue), 1.86 over all: 2,048 CTAs are 3.4 waves, whose
// warps have one to many rows, and SMs run dry at the end.  Most instructions are
// what a row costs whatever its length: its place from another lane, its address,
// whether it ends here.  4,093 rows onto 30,522, 125 MB of zeros beside them: 33 us.
template <typename T, typename Tout, bool VEC>
__device__ __forceinline__ void sum_window(const SumParams& p, long long window, int split, int chunk, uint4* memory) {
    const int lane = threadIdx.x & 31;
    const long long w0 = window * kPart, at0 = w0 + lane, at1 = at0 + kPart;
    // the window's, those behind it that its last rows reach, and those before it
    const int key0 = at0 < p.n ? p.keys[at0] : INT32_MAX, key1 = at1 < p.n ? p.keys[at1] : INT32_MAX;
    const int before = at0 >= kPart ? p.keys[at0 - kPart] : -1;
    const int place0 = at0 < p.n ? p.places[at0] : 0, place1 = at1 < p.n ? p.places[at1] : 0;
    // the first ones of the 32 windows before it, for a row that began there
    const long long back = w0 - (lane + 1) * kPart;
    const int far = back >= 0 ? p.keys[back] : -1;
    const int first = __shfl_sync(kAll, key0, 0);
    const int up0 = __shfl_up_sync(kAll, key0, 1), up1 = __shfl_up_sync(kAll, key1, 1);
    const int end_before = __shfl_sync(kAll, before, 31), end0 = __shfl_sync(kAll, key0, 31);
    // bit q: a row begins at the window's place q
    const uint32_t rows0 = __ballot_sync(kAll, key0 != (lane ? up0 : end_before));
    const uint32_t rows1 = __ballot_sync(kAll, key1 != (lane ? up1 : end0));
    const int valid = __popc(__ballot_sync(kAll, key0 < p.vocab)) + __popc(__ballot_sync(kAll, key1 < p.vocab));
    long long start = w0;                                        // where the window's first row begins
    if (!(rows0 & 1)) {
        const uint32_t others = __ballot_sync(kAll, before != first);
        if (others) start = w0 - __clz(others);
        else if (first < p.vocab) {
            const int same = __popc(__ballot_sync(kAll, far == first));      // the nearest of them: the keys are sorted
            start = w0 - static_cast<long long>(same) * kPart;
            if (same == 32) {
                start = warp_lower_bound(p.keys, 0, start, first);
            } else {
                const long long at = start - kPart + lane;
                start -= __clz(__ballot_sync(kAll, (at >= 0 ? p.keys[at] : -1) != first));
            }
        }
    }
    // and bit q: a part of a row does
    const auto begin_of = [&](uint32_t rows, long long other) {  // of the row that this lane's place is in
        const uint32_t up_to = rows & (0xffffffffu >> (31 - lane));
        return up_to ? 31 - __clz(up_to) : other;
    };
    const uint32_t parts0 = __ballot_sync(kAll, (lane - begin_of(rows0, start - w0)) % kPart == 0);
    const long long open = rows0 ? 31 - __clz(rows0) : start - w0;           // where the row that goes on behind begins
    const uint32_t parts1 = __ballot_sync(kAll, (kPart + lane - (rows1 & (0xffffffffu >> (31 - lane)) ? kPart + begin_of(rows1, 0) : open)) % kPart == 0);
    const int each = kPart / p.splits, a = split * each, b = a + each;
    const auto next_begin = [&](int q) {                         // the first beginning at q or behind it
        const uint32_t bits = q < 32 ? parts0 & (0xffffffffu << q) : 0u;
        return bits ? __ffs(bits) - 1 : parts1 ? 31 + __ffs(parts1) : 2 * kPart;
    };
    const int i0 = next_begin(a), i1 = min(next_begin(b), valid);
    if (i0 >= min(b, valid)) return;
    const Columns<VEC> c(chunk, p.dim);
    const T* const grad = static_cast<const T*>(p.grad);
    // A row's columns of this chunk on their way to shared memory: a lane's own
    // eight, or, where rows do not lie in vectors, the 16-byte words that the
    // chunk touches, of which a lane reads every 32nd element.
    constexpr int kSlot = slot_of<T, VEC>, kEach = 16 / static_cast<int>(sizeof(T)), kPieces = 8 / kEach;
    uint4* const ring = memory + (threadIdx.x >> 5) * (kRing<T> * kSlot);
    const int columns = min(kChunk, p.dim - chunk * kChunk);
    const auto row_of = [&](int q) {
        const int place = __shfl_sync(kAll, q < kPart ? place0 : place1, q & 31);
        return grad + static_cast<long long>(place) * p.grad_stride + chunk * kChunk;
    };
    const auto head_of = [&](const T* from) { return static_cast<int>((reinterpret_cast<uintptr_t>(from) & 15) / sizeof(T)); };
    const auto request = [&](int q) {
        const T* const from = row_of(q);
        uint4* const to = ring + q % kRing<T> * kSlot + lane;
        if constexpr (VEC) {
            if (q < i1 && c.on(0))
#pragma unroll
                for (int u = 0; u < kPieces; ++u) copy_async(to + 32 * u, reinterpret_cast<const uint4*>(from + 8 * lane) + u);
        } else if (q < i1) {
            const int words = (head_of(from) + columns + kEach - 1) / kEach;
            const uint4* const first_word = reinterpret_cast<const uint4*>(from - head_of(from)) + lane;
#pragma unroll
            for (int u = 0; u <= kPieces; ++u)
                if (lane + 32 * u < words) copy_async(to + 32 * u, first_word + 32 * u);
        }
        copy_commit();
    };
    for (int k = 0; k + 1 < kRing<T>; ++k) request(i0 + k);
    Sum sum = {};
    int begin = i0;
#pragma unroll 1
    for (int i = i0; i < i1; ++i) {
        copy_wait<kRing<T> - 2>();
        const uint4* const row = ring + i % kRing<T> * kSlot;
        if constexpr (VEC) {
            Eight<T> raw;
            uint4* const words = reinterpret_cast<uint4*>(&raw);
#pragma unroll
            for (int u = 0; u < kPieces; ++u) words[u] = row[lane + 32 * u];
            raw.add_to(sum.v);
        } else {
            __syncwarp();
            const T* const x = reinterpret_cast<const T*>(row) + head_of(row_of(i)) + lane;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c.on(j)) sum.v[j] += widen(x[32 * j]);
        }
        request(i + kRing<T> - 1);                               // into the place of the row before, which is used up
        const int q = i + 1;
        if (q < i1 && !((q < kPart ? parts0 >> q : parts1 >> (q - kPart)) & 1)) continue;
        // a row ends here, or a part of one that is long
        const int key = __shfl_sync(kAll, q <= kPart ? key0 : key1, i & 31);
        sum.whole = true;
        const bool ends = (q < kPart ? rows0 >> q : rows1 >> (q - kPart)) & 1;
        if (!ends || !(rows0 >> begin & 1)) {
            const uint32_t up_to = rows0 & (0xffffffffu >> (31 - begin));
            const long long row = up_to ? w0 + 31 - __clz(up_to) : start;
            sum = join_parts<VEC>(p, row, static_cast<int>((w0 + begin - row) / kPart), ends, chunk, sum);
        }
        if (sum.whole) put_row<Tout, VEC>(p, key, c, sum);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum.v[j] = 0.0f;
        begin = q;
    }
}

// Zeros into those of a CTA's `rows` rows of the table that have no token.
template <typename Tout>
__device__ __forceinline__ void fill_rows(const SumParams& p, long long v0) {
    __shared__ long long bounds[2];
    __shared__ int starts[kThreads + 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long v1 = min(p.vocab, v0 + p.rows);
    if (warp < 2) {
        const long long x = warp_lower_bound(p.keys, 0, p.n, warp ? v1 : v0);
        if (lane == 0) bounds[warp] = x;
    }
    __syncthreads();
    for (int r = threadIdx.x; r <= v1 - v0; r += kThreads)
        starts[r] = static_cast<int>(lower_bound(p.keys, bounds[0], bounds[1], v0 + r));
    __syncthreads();
    const int t = threadIdx.x % p.row_threads, slot = threadIdx.x / p.row_threads, slots = kThreads / p.row_threads;
    for (int r = slot; r < v1 - v0; r += slots) {
        if (starts[r] != starts[r + 1]) continue;
        Tout* const to = static_cast<Tout*>(p.out) + (v0 + r) * p.out_stride;
        // a few elements up to a 16-byte boundary, 16 bytes at a time, the rest
        const int head = min(p.dim, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(to) & 15)) % 16 / sizeof(Tout)));
        constexpr int kEach = 16 / sizeof(Tout);
        const int pieces = (p.dim - head) / kEach;
        for (int i = t; i < pieces; i += p.row_threads) __stcs(reinterpret_cast<uint4*>(to + head) + i, make_uint4(0, 0, 0, 0));
        for (int i = t; i < p.dim - pieces * kEach; i += p.row_threads)
            to[i < head ? i : i + pieces * kEach] = narrow<Tout>(0.0f);
    }
}

// The first sum_ctas CTAs sum, a warp an item of window, split and chunk of
// columns; the others write the rows without a token, meanwhile.
template <typename T, typename Tout, bool VEC>
__global__ void __launch_bounds__(kThreads, 4) embed_sum_kernel(const __grid_constant__ SumParams p) {
    extern __shared__ uint4 memory[];
    ddpk::dev::pdl_wait();
    ddpk::dev::pdl_trigger();
    if (blockIdx.x >= p.sum_ctas) return fill_rows<Tout>(p, static_cast<long long>(blockIdx.x - p.sum_ctas) * p.rows);
    const long long item = static_cast<long long>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    const int chunk = static_cast<int>(item % p.chunks), split = static_cast<int>(item / p.chunks % p.splits);
    const long long window = item / p.chunks / p.splits;
    if (window < p.windows) sum_window<T, Tout, VEC>(p, window, split, chunk, memory);
}

// ---------------------------------------------------------------- host

struct Plan {
    int sort_ctas, passes, bits;
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
    if (q.bits < 2) q.bits = 2;                                 // a pass's counts fill 16 bytes
    const int64_t tiles = (n + kTile - 1) / kTile, each = (tiles + kMaxSortCtas - 1) / kMaxSortCtas;
    q.share = each * kTile;
    q.sort_ctas = static_cast<int>((n + q.share - 1) / q.share);
    q.windows = (n + kPart - 1) / kPart;
    int64_t at = 0;
    q.keys = at;
    at += 2 * up(4 * n);
    q.places = at;
    at += 2 * up(4 * n);
    q.counts = at;
    at += up(4LL * kMaxBins * q.sort_ctas * q.passes);
    q.tickets = at;
    at += 2 * up(4 * (2 * q.windows * ((a->dim + kChunk - 1) / kChunk) + 4));
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
    return a->dim % 8 == 0 && aligned(table, 8 * size_of(a->table_dtype)) && aligned(rows, 8 * size_of(a->dtype)) &&
           (a->vocab == 1 || a->table_stride % 8 == 0) && (a->tokens == 1 || a->row_stride % 8 == 0);
}

int row_threads(int64_t pieces) { return pieces >= kThreads ? kThreads : power_of_two(pieces); }

template <typename Tin, typename Tout>
cudaError_t embed_as(bool vec, EmbedParams& p, cudaStream_t stream) {
    if (!vec && p.dim >= kShiftColumns)
        return launch(embed_shift_kernel<Tin, Tout>, (p.n + kThreads / 32 - 1) / (kThreads / 32), kThreads, 0, stream, p);
    p.row_threads = row_threads(vec ? p.dim / 8 : (p.dim + kColumns - 1) / kColumns);
    const long long tile = static_cast<long long>(kThreads / p.row_threads) * kAhead;
    return launch(vec ? embed_kernel<Tin, Tout, true> : embed_kernel<Tin, Tout, false>, (p.n + tile - 1) / tile, kThreads, 0, stream, p);
}

template <typename T, typename Tout>
cudaError_t sum_as(bool vec, long long ctas, const SumParams& p, cudaStream_t stream) {
    return launch(vec ? embed_sum_kernel<T, Tout, true> : embed_sum_kernel<T, Tout, false>, ctas, kThreads,
                  kThreads / 32 * kRing<T> * (vec ? slot_of<T, true> : slot_of<T, false>) * sizeof(uint4), stream, p);
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
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool in32 = a->table_dtype == DDP_F32, out32 = a->dtype == DDP_F32;
    const cudaError_t e = in32 ? (out32 ? embed_as<float, float>(vec, p, st) : embed_as<float, uint16_t>(vec, p, st))
                               : (out32 ? embed_as<uint16_t, float>(vec, p, st) : embed_as<uint16_t, uint16_t>(vec, p, st));
    return e == cudaSuccess ? DDP_OK : DDP_ERR_CUDA;
}

int64_t ddp_embed_workspace(const ddp_embed_args* a) {
    if (!valid(a) || a->tokens > kMaxTokens) return DDP_ERR_INVALID_ARG;
    return a->tokens ? plan_of(a).bytes : 0;
}

int ddp_embed_backward(const ddp_embed_args* a, const void* grad, const void* tokens, void* grad_table, int32_t accumulate,
                       void* workspace, void* stream) {
    if (!valid(a) || a->tokens > kMaxTokens || (accumulate && a->table_dtype != DDP_F32)) return DDP_ERR_INVALID_ARG;
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
    const bool vec = vectors(a, grad_table, grad);
    SortParams s = {};
    s.tokens = tokens;
    int* const counts = reinterpret_cast<int*>(ws + q.counts);
    s.tickets = reinterpret_cast<int*>(ws + q.tickets);
    s.n = a->tokens;
    s.vocab = a->vocab;
    s.share = q.share;
    s.wide = a->index_bits == 64;
    s.ctas = q.sort_ctas;
    s.bits = q.bits;
    SumParams p = {};
    p.windows = q.windows;
    p.chunks = static_cast<int>((a->dim + kChunk - 1) / kChunk);
    p.tickets_each = (2 * q.windows * p.chunks + 3) / 4 * 4;
    // the second level of them is for rows of more parts than a group's
    s.ntickets = p.tickets_each * (a->tokens > kPart * kGroup ? 2 : 1);
    cudaError_t e = cudaSuccess;
    if (a->tokens <= kSmall) {
        s.keys = keys[0];
        s.places = places[0];
        const long long each = kThreads / kRankLanes;
        e = launch(sort_small_kernel, (a->tokens + each - 1) / each, kThreads, (a->tokens + 3) / 4 * 16, st, s);
    } else {
        const int64_t each = static_cast<int64_t>(s.ctas) << q.bits;         // counts of a pass
        for (int pass = 0; pass < q.passes && e == cudaSuccess; ++pass) {
            s.shift = pass * q.bits;
            s.keys_in = pass ? keys[(pass - 1) & 1] : nullptr;
            s.places_in = pass ? places[(pass - 1) & 1] : nullptr;
            s.keys = keys[pass & 1];
            s.places = places[pass & 1];
            s.counts = counts + pass * each;
            s.next_counts = pass + 1 < q.passes ? s.counts + each : nullptr;
            if (pass == 0) {
                s.nzeros = each * (q.passes - 1);
                e = launch(sort_count_kernel, s.ctas, kSortThreads, 0, st, s);
            }
            if (e == cudaSuccess) e = launch(sort_move_kernel, s.ctas, kSortThreads, 0, st, s);
        }
    }
    if (e != cudaSuccess) return DDP_ERR_CUDA;
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
    p.accumulate = accumulate != 0;
    p.scale = a->scale;
    p.splits = 1;
    while (p.splits < kMaxSplits && q.windows * p.chunks * p.splits < kFewWarps) p.splits *= 2;
    while (p.splits < kMoreSplits && q.windows * p.chunks * p.splits < kMoreWarps) p.splits *= 2;
    const int64_t warps = q.windows * p.chunks * p.splits, sums = (warps + kThreads / 32 - 1) / (kThreads / 32);
    if (sums > INT32_MAX) return DDP_ERR_INVALID_ARG;
    p.sum_ctas = static_cast<unsigned>(sums);
    const int64_t row_bytes = a->dim * size_of(a->table_dtype), fit = kFillBytes / row_bytes;
    const int64_t each = (a->vocab + 8 * kSms - 1) / (8 * kSms), rows = fit < each ? fit : each;
    p.rows = static_cast<int>(rows < 8 ? 8 : rows < kThreads ? rows : kThreads);
    p.row_threads = row_threads(row_bytes / 16);
    const long long ctas = sums + (accumulate ? 0 : (p.vocab + p.rows - 1) / p.rows);
    const bool in32 = a->dtype == DDP_F32, out32 = a->table_dtype == DDP_F32;
    e = in32 ? (out32 ? sum_as<float, float>(vec, ctas, p, st) : sum_as<float, uint16_t>(vec, ctas, p, st))
             : (out32 ? sum_as<uint16_t, float>(vec, ctas, p, st) : sum_as<uint16_t, uint16_t>(vec, ctas, p, st));
    return e == cudaSuccess ? DDP_OK : DDP_ERR_CUDA;
}

}  // extern "C"
