// Rows of a table for tokens, and the table's gradient: the rows' gradients
// summed for each token.
//
// The gradient sorts the tokens first (a stable radix sort, so that equal tokens
// keep their order), and each row of the table then sums its tokens' gradients
// one after another: equal inputs give equal bits, and a row's sum does not depend
// on the other tokens'.  A word that falls often is summed in parts of kPart
// tokens, and whoever ends last adds the parts (groups of them) in their order.

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
constexpr int kSmall = 8192;           // tokens that are sorted by counting
constexpr int kRankLanes = 8;
constexpr int kPart = 64;              // sorted places of a CTA, and tokens that are summed in one go
constexpr int kGroup = 64;             // parts of a row that are added up in one go
constexpr int kUnroll = 8;             // rows on their way at once
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
    int* counts;             // [ctas][bins]
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
    for (long long i = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x; i < p.ntickets / 4;
         i += static_cast<long long>(gridDim.x) * kThreads)
        reinterpret_cast<int4*>(p.tickets)[i] = make_int4(0, 0, 0, 0);
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
#pragma unroll 4
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

// A row of the table's gradient, columns from `at` on.  What is added to is not
// waited for: one addition for each element, so no order is left open.
template <typename Tout, bool VEC>
__device__ __forceinline__ void put_row(const SumParams& p, long long row, int at, const float (&sum)[VEC ? 8 : 1]) {
    Tout* const to = static_cast<Tout*>(p.out) + row * p.out_stride + at;
    float f[VEC ? 8 : 1];
#pragma unroll
    for (int j = 0; j < (VEC ? 8 : 1); ++j) f[j] = sum[j] * p.scale;
    if constexpr (sizeof(Tout) == 4) {
        if (p.accumulate) {
            if constexpr (VEC) {
#pragma unroll
                for (int j = 0; j < 8; j += 4)
                    asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(to + j), "f"(f[j]), "f"(f[j + 1]),
                                 "f"(f[j + 2]), "f"(f[j + 3]) : "memory");
            } else {
                asm volatile("red.relaxed.gpu.global.add.f32 [%0], %1;" ::"l"(to), "f"(f[0]) : "memory");
            }
            return;
        }
    }
    if constexpr (VEC) {
        Eight<Tout> raw;
        raw.put(f);
        raw.store_once(to);
    } else {
        *to = narrow<Tout>(f[0]);
    }
}

// A part of a row of more than kPart tokens: part m of those that begin at sorted
// place `start` and end before `end`.  A CTA's window of kPart places holds at most
// two beginnings of parts, of which one is its row's first.
struct Parts {
    long long start, end;

    __device__ __forceinline__ int count() const { return static_cast<int>((end - start + kPart - 1) / kPart); }
    __device__ __forceinline__ long long slot(int m) const { return (start + static_cast<long long>(m) * kPart) / kPart * 2 + (m == 0); }
};

// One thread's columns of part m are summed: keeps them, and, where this thread
// is the last of a group of parts (and its group the row's last), adds up the
// group's (and the groups') in their order and gives the whole in `sum`.
template <int N>
__device__ __forceinline__ bool join_parts(const SumParams& p, const Parts& of, int m, int at, float (&sum)[N]) {
    const auto put = [&](int part) {
        float* const to = p.parts + of.slot(part) * p.dim + at;
#pragma unroll
        for (int j = 0; j < N; ++j) __stcg(to + j, sum[j]);
        __threadfence();
    };
    const auto add = [&](int from, int to, int step) {
        __threadfence();
#pragma unroll
        for (int j = 0; j < N; ++j) sum[j] = 0.0f;
#pragma unroll 8
        for (int q = from; q < to; q += step) {
            const float* const x = p.parts + of.slot(q) * p.dim + at;
#pragma unroll
            for (int j = 0; j < N; ++j) sum[j] += __ldcg(x + j);
        }
    };
    const int count = of.count(), group = m / kGroup * kGroup, end = min(count, group + kGroup);
    const long long columns = (p.dim + N - 1) / N, column = at / N;
    put(m);
    if (atomicAdd(p.tickets + of.slot(group) * columns + column, 1) != end - group - 1) return false;
    add(group, end, 1);
    if (count <= kGroup) return true;
    put(group);
    if (atomicAdd(p.tickets + p.tickets_each + of.slot(0) * columns + column, 1) != (count + kGroup - 1) / kGroup - 1) return false;
    add(0, count, kGroup);
    return true;
}

// A CTA sums the tokens of a window of kPart sorted places: a run of rows and
// parts of rows that begin in the window, one after another, with the next ones'
// gradients on their way.
template <typename T, typename Tout, bool VEC>
__global__ void __launch_bounds__(kThreads) embed_sum_kernel(const __grid_constant__ SumParams p) {
    constexpr int N = VEC ? 8 : 1;
    __shared__ int keys[2 * kPart + 1];            // from the place before the window's first on
    __shared__ int places[2 * kPart];
    __shared__ uint32_t begins[2 * kPart / 32];    // bit q: a row, or a part of one, begins at the window's place q
    __shared__ int valid;                          // places that hold a token of the table
    __shared__ long long of_first[2], of_last[2];           // the rows at the window's ends, where they are long
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t = threadIdx.x % p.row_threads, slot = threadIdx.x / p.row_threads, slots = blockDim.x / p.row_threads;
    ddpk::dev::pdl_wait();
    ddpk::dev::pdl_trigger();
    const long long w0 = static_cast<long long>(blockIdx.x) * kPart;
    for (int i = threadIdx.x; i <= 2 * kPart; i += blockDim.x) {
        const long long at = w0 - 1 + i;
        keys[i] = at < 0 ? -1 : at < p.n ? p.keys[at] : INT32_MAX;
        if (i) places[i - 1] = at < p.n ? p.places[at] : 0;
    }
    __syncthreads();
    const int first = keys[1], last = keys[kPart];
    if (warp == 0) {
        const bool goes_on = keys[0] == first, is_long = goes_on || keys[kPart + 1] == first;
        if (is_long && first < p.vocab) {
            const long long start = goes_on ? warp_lower_bound(p.keys, 0, w0, first) : w0;
            const long long end = warp_lower_bound(p.keys, w0, p.n, first + 1LL);
            if (lane == 0) { of_first[0] = start; of_first[1] = end; }
            __syncwarp();
        }
        const long long start = goes_on && first < p.vocab ? of_first[0] : w0;
        uint32_t rows[2 * kPart / 32];
        int count = 0;
#pragma unroll
        for (int w = 0; w < 2 * kPart / 32; ++w) {
            const int q = 32 * w + lane;
            rows[w] = __ballot_sync(kAll, keys[q + 1] != keys[q]);
            count += __popc(__ballot_sync(kAll, keys[q + 1] < p.vocab));
            long long from = start;                      // where this place's row begins
#pragma unroll
            for (int v = 0; v <= w; ++v) {
                const uint32_t up_to = v < w ? rows[v] : rows[v] & (0xffffffffu >> (31 - lane));
                if (up_to) from = w0 + 32 * v + 31 - __clz(up_to);
            }
            const uint32_t b = __ballot_sync(kAll, (w0 + q - from) % kPart == 0);
            if (lane == 0) begins[w] = b;
        }
        if (lane == 0) valid = count;
    } else if (warp == 1 && last != first && keys[kPart + 1] == last && last < p.vocab) {
        int from = kPart;                                // of a row that begins in the window and goes on behind it
        while (keys[from - 1] == last) --from;
        const long long end = warp_lower_bound(p.keys, w0 + kPart, p.n, last + 1LL);
        if (lane == 0) { of_last[0] = w0 + from - 1; of_last[1] = end; }
    }
    __syncthreads();
    const int each = kPart / slots, a = slot * each, b = a + each;
    const auto next_begin = [&](int q) {                 // the first beginning at q or behind it
        for (int w = q / 32; w < 2 * kPart / 32; ++w) {
            const uint32_t bits = begins[w] & (w == q / 32 ? 0xffffffffu << (q % 32) : 0xffffffffu);
            if (bits) return 32 * w + __ffs(bits) - 1;
        }
        return 2 * kPart;
    };
    const int i0 = next_begin(a), i1 = min(next_begin(b), valid);
    if (i0 >= min(b, valid)) return;
    const T* const grad = static_cast<const T*>(p.grad);
    for (int at = t * N; at < p.dim; at += p.row_threads * N) {
        float sum[N];
#pragma unroll
        for (int j = 0; j < N; ++j) sum[j] = 0.0f;
        int begin = i0;
        for (int i = i0; i < i1; i += kUnroll) {
            Eight<T> raw[VEC ? kUnroll : 1];
            float single[VEC ? 1 : kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const T* const from = grad + static_cast<long long>(i + u < i1 ? places[i + u] : 0) * p.grad_stride + at;
                if constexpr (VEC) {
                    if (i + u < i1) raw[u].load_once(from);
                } else {
                    single[u] = i + u < i1 ? widen(*from) : 0.0f;
                }
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                const int q = i + u + 1;
                if (q > i1) break;
                if constexpr (VEC) {
                    float f[8];
                    raw[u].get(f);
#pragma unroll
                    for (int j = 0; j < 8; ++j) sum[j] += f[j];
                } else {
                    sum[0] += single[u];
                }
                if (q < i1 && !(begins[q / 32] >> (q % 32) & 1)) continue;
                // a row ends here, or a part of one that is long
                const int key = keys[q];
                bool whole = true;
                if (keys[q + 1] == key || keys[begin] == key) {
                    const Parts of = key == first ? Parts{of_first[0], of_first[1]} : Parts{of_last[0], of_last[1]};
                    whole = join_parts<N>(p, of, static_cast<int>((w0 + begin - of.start) / kPart), at, sum);
                }
                if (whole) put_row<Tout, VEC>(p, key, at, sum);
#pragma unroll
                for (int j = 0; j < N; ++j) sum[j] = 0.0f;
                begin = q;
            }
        }
    }
}

// Zeros into the rows of the table that have no token, `rows` of them a CTA.  It
// needs the sorted keys alone, which were there before the sums' kernel let it
// start, so it runs beside that one and waits for it only before it ends.
template <typename Tout>
__global__ void __launch_bounds__(kThreads) embed_fill_kernel(const __grid_constant__ SumParams p) {
    __shared__ long long bounds[2];
    __shared__ int starts[kThreads + 1];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long v0 = static_cast<long long>(blockIdx.x) * p.rows, v1 = min(p.vocab, v0 + p.rows);
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
    ddpk::dev::pdl_wait();
    ddpk::dev::pdl_trigger();
}

// ---------------------------------------------------------------- host

struct Plan {
    int sort_ctas, passes, bits;
    long long share, windows;
    int64_t keys, places, counts, parts, tickets, bytes;      // offsets into the workspace; two of the first two
};

int64_t up(int64_t x) { return (x + 255) / 256 * 256; }

// The same whatever the alignment: tickets for columns one by one.
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
    q.windows = (n + kPart - 1) / kPart;
    int64_t at = 0;
    q.keys = at;
    at += 2 * up(4 * n);
    q.places = at;
    at += 2 * up(4 * n);
    q.counts = at;
    at += up(4LL * kMaxBins * q.sort_ctas);
    q.tickets = at;
    at += 2 * up(4 * (2 * q.windows * a->dim + 4));
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
cudaError_t sum_as(bool vec, int threads, const SumParams& p, cudaStream_t stream) {
    return launch(vec ? embed_sum_kernel<T, Tout, true> : embed_sum_kernel<T, Tout, false>, p.windows, threads, 0, stream, p);
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
    const bool vec = vectors(a, grad_table, grad);
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
    SumParams p = {};
    p.windows = q.windows;
    p.tickets_each = (2 * q.windows * (vec ? a->dim / 8 : a->dim) + 3) / 4 * 4;
    // the second level of them is for rows of more parts than a group's
    s.ntickets = p.tickets_each * (a->tokens > kPart * kGroup ? 2 : 1);
    cudaError_t e = cudaSuccess;
    if (a->tokens <= kSmall) {
        s.keys = keys[0];
        s.places = places[0];
        const long long each = kThreads / kRankLanes;
        e = launch(sort_small_kernel, (a->tokens + each - 1) / each, kThreads, (a->tokens + 3) / 4 * 16, st, s);
    } else {
        for (int pass = 0; pass < q.passes && e == cudaSuccess; ++pass) {
            s.shift = pass * q.bits;
            s.keys_in = pass ? keys[(pass - 1) & 1] : nullptr;
            s.places_in = pass ? places[(pass - 1) & 1] : nullptr;
            s.keys = keys[pass & 1];
            s.places = places[pass & 1];
            e = launch(sort_count_kernel, s.ctas, kThreads, 0, st, s);
            if (e == cudaSuccess) e = launch(sort_move_kernel, s.ctas, kThreads, 0, st, s);
            s.ntickets = 0;
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
    p.row_threads = row_threads(a->dim, vec);
    const int threads = kPart * p.row_threads < kThreads ? kPart * p.row_threads : kThreads;
    const bool in32 = a->dtype == DDP_F32, out32 = a->table_dtype == DDP_F32;
    e = in32 ? (out32 ? sum_as<float, float>(vec, threads, p, st) : sum_as<float, uint16_t>(vec, threads, p, st))
             : (out32 ? sum_as<uint16_t, float>(vec, threads, p, st) : sum_as<uint16_t, uint16_t>(vec, threads, p, st));
    if (e == cudaSuccess && !accumulate) {
        const int64_t row_bytes = a->dim * size_of(a->table_dtype), fit = kFillBytes / row_bytes;
        p.rows = static_cast<int>(fit < 8 ? 8 : fit < kThreads ? fit : kThreads);
        p.row_threads = row_bytes / 16 >= kThreads ? kThreads : power_of_two(row_bytes / 16);
        e = launch(out32 ? embed_fill_kernel<float> : embed_fill_kernel<uint16_t>, (p.vocab + p.rows - 1) / p.rows, kThreads, 0, st, p);
    }
    return e == cudaSuccess ? DDP_OK : DDP_ERR_CUDA;
}

}  // extern "C"
