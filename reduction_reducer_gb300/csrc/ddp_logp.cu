// Log probabilities of given tokens, with the entropy and the best alternatives
// of each place, and the gradient of its logits.
//
// The forward pass reads a row once: every thread keeps its elements' largest m,
// the sum S of e^(x - m) and the sum A of e^(x - m) (x - m), and rescales the sums
// when m grows; log p_t = x_t - m - log S and the entropy is log S - A / S, two
// terms of one sign.  A row is a warp's, a CTA's, or, where rows are too few to
// fill the GPU, a cluster's, whose first CTA joins the parts.
//
// The alternatives: the k-th largest of the threads' own best is a bound that at
// least k elements reach, and only the k threads whose best reaches it can hold
// any.  These threads' elements are read again (from L2), and the few that reach
// the bound sorted.  Keys are the value's order above the lowest index, so no two
// are equal and ties go to the lowest index.

#include "ddp_reducer.h"

#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <type_traits>

#include "ddp_rows.cuh"

namespace {

using namespace ddpk::rows;
namespace cg = cooperative_groups;

constexpr int kWarps = 8;              // of a CTA: with a row to itself, or a row a warp
constexpr int kWarpVocab = 2048;       // up to which a row is a warp's
// Bytes of a row up to which it is a warp's, of some rows and of many.
constexpr int64_t kSomeRows = 6 * kSms, kSomeBytes = 16 << 10, kManyRows = 16 * kSms, kManyBytes = 32 << 10;
constexpr int kStages = 4;             // pieces of a thread on their way, with the one under work
constexpr int kUnits = 2;              // of 16 bytes, of a piece
constexpr int kMaxTop = 32;
constexpr int kMaxSplit = 8;           // CTAs of a row
constexpr int kBackThreads = 128;
constexpr int kBackCtas = 12;          // on an SM: loads on their way (8,192 x 50,257 in bf16: eight 267 us, ten 247, twelve 234)
template <typename T> constexpr int kBackEights = sizeof(T) == 2 ? 4 : 2;      // of a thread
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kFloor = -1000.0f;     // 2^-1000 is zero; stands in for -inf where it meets a zero
constexpr float kFar = 64.0f;          // from where on the rounding of m scale (half a step: 1.9e-6) is more than log S's

struct LogpParams {
    const void* logits;
    const void* targets;
    float* logp;
    float* entropy;
    float* stats;
    int* top_index;
    float* top_logp;
    const float* grad_logp;        // backward
    const float* grad_entropy;
    void* out;
    long long rows, stride, out_stride;
    long long segment;             // elements of a CTA of a row
    int vocab, top, wide, split;
    float scale, scale2;           // scale2: scale log2(e)
    int rounds;                    // m scale is rounded: scale is no power of two
};

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The target of a row; -1: none (the row is left out), -2: no targets at all.
__device__ __forceinline__ int target_of(const LogpParams& p, long long row) {
    if (!p.targets) return -2;
    const long long t = p.wide ? static_cast<const long long*>(p.targets)[row] : static_cast<const int*>(p.targets)[row];
    return t >= 0 && t < p.vocab ? static_cast<int>(t) : -1;
}

// m: largest; s: sum of 2^((x - m) c); a: sum of 2^((x - m) c) (x - m) c.
struct Sums {
    float m, s, a;
};

__device__ __forceinline__ Sums join(const Sums& x, const Sums& y, float c) {
    const float m = fmaxf(x.m, y.m);
    // (-inf) - (-inf) is NaN, which the maximum takes for the floor
    const float dx = fmaxf((x.m - m) * c, kFloor), dy = fmaxf((y.m - m) * c, kFloor);
    const float fx = exp2_fast(dx), fy = exp2_fast(dy);
    return Sums{m, x.s * fx + y.s * fy, fx * fmaf(dx, x.s, x.a) + fy * fmaf(dy, y.s, y.a)};
}

template <int LANES>
__device__ __forceinline__ Sums join_lanes(Sums x, float c) {
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) {
        const Sums y = {__shfl_xor_sync(kAll, x.m, o), __shfl_xor_sync(kAll, x.s, o), __shfl_xor_sync(kAll, x.a, o)};
        x = join(x, y, c);
    }
    return x;
}

// The largest so far is `top` or what it was.  Whether it grew.
template <bool ENTROPY>
__device__ __forceinline__ bool grow(float top, float c, Sums& t) {
    const bool grew = top > t.m;
    if (grew) {
        const float d = fmaxf((t.m - top) * c, kFloor), f = exp2_fast(d);
        if constexpr (ENTROPY) t.a = f * fmaf(d, t.s, t.a);
        t.s *= f;
        t.m = top;
    }
    return grew;
}

// 2 N more elements.  Whether the largest grew.
template <int N, bool ENTROPY>
__device__ __forceinline__ bool take(const float2 (&x)[N], float c, Sums& t) {
    float top = fmaxf(x[0].x, x[0].y);
#pragma unroll
    for (int i = 1; i < N; ++i) top = fmaxf(top, fmaxf(x[i].x, x[i].y));
    const bool grew = grow<ENTROPY>(top, c, t);
    const float m = t.m == neg_inf() ? 0.0f : t.m;
    float2 s = make_float2(0.0f, 0.0f), a = s;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float2 d = mul2(add2(x[i], both(-m)), both(c)), e = make_float2(exp2_fast(d.x), exp2_fast(d.y));
        s = add2(s, e);
        if constexpr (ENTROPY) a = fma2(e, make_float2(fmaxf(d.x, kFloor), fmaxf(d.y, kFloor)), a);
    }
    t.s += s.x + s.y;
    if constexpr (ENTROPY) t.a += a.x + a.y;
    return grew;
}

// The same of pairs of bf16 as they lie in memory: the largest is found for both
// of a pair at once, and the differences take the pairs as they are.  8,192 rows of
// 50,257 with the entropy 119 us, with the elements widened 130; a floor taken in
// pairs too, below m, 124.
template <int N, bool ENTROPY>
__device__ __forceinline__ bool take(const uint32_t (&x)[N], float c, Sums& t) {
    uint32_t tops = x[0];
#pragma unroll
    for (int i = 1; i < N; ++i) asm("max.bf16x2 %0, %0, %1;" : "+r"(tops) : "r"(x[i]));
    const bool grew = grow<ENTROPY>(fmaxf(__uint_as_float(tops << 16), __uint_as_float(tops & 0xffff0000u)), c, t);
    const float m = t.m == neg_inf() ? 0.0f : t.m;
    float2 s = make_float2(0.0f, 0.0f), a = s;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float2 d = mul2(add_pair(x[i], both(-m)), both(c)), e = make_float2(exp2_fast(d.x), exp2_fast(d.y));
        s = add2(s, e);
        if constexpr (ENTROPY) a = fma2(e, make_float2(fmaxf(d.x, kFloor), fmaxf(d.y, kFloor)), a);
    }
    t.s += s.x + s.y;
    if constexpr (ENTROPY) t.a += a.x + a.y;
    return grew;
}

template <bool ENTROPY>
__device__ __forceinline__ bool take_one(float x, float c, Sums& t) {
    const float2 pair[1] = {make_float2(x, neg_inf())};
    return take<1, ENTROPY>(pair, c, t);
}

// A run of n elements of a row: `head` elements, `units` of N each from a 16-byte
// boundary on, and a rest.
template <typename T, int N>
struct Run {
    const T* from;
    int n, head, units;

    __device__ __forceinline__ Run(const T* row, long long lo, long long hi) {
        from = row + lo;
        n = hi > lo ? static_cast<int>(hi - lo) : 0;
        head = min(n, static_cast<int>((16 - (reinterpret_cast<uintptr_t>(from) & 15)) % 16 / sizeof(T)));
        units = (n - head) / N;
    }
    __device__ __forceinline__ const T* unit(int i) const { return from + head + N * i; }
    __device__ __forceinline__ int rest() const { return head + N * units; }
};

// A 16-byte unit as fp32 numbers.
__device__ __forceinline__ void numbers(uint4 v, float (&f)[8]) { ddpk::dev::Vec<uint16_t>::unpack(v, f); }
__device__ __forceinline__ void numbers(uint4 v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x); f[1] = __uint_as_float(v.y); f[2] = __uint_as_float(v.z); f[3] = __uint_as_float(v.w);
}

// The largest of one, NaN aside.
template <typename T>
__device__ __forceinline__ float largest(uint4 v) {
    if constexpr (sizeof(T) == 4)
        return fmaxf(fmaxf(__uint_as_float(v.x), __uint_as_float(v.y)), fmaxf(__uint_as_float(v.z), __uint_as_float(v.w)));
    uint32_t x = v.x;
    asm("max.bf16x2 %0, %0, %1;\n\tmax.bf16x2 %0, %0, %2;\n\tmax.bf16x2 %0, %0, %3;" : "+r"(x) : "r"(v.y), "r"(v.z), "r"(v.w));
    return fmaxf(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}

// ---------------------------------------------------------------- the best alternatives

using Key = unsigned long long;

// 0 for what is never chosen (-inf, NaN); the larger value, then the lower index first.
__device__ __forceinline__ Key key_of(float x, int index) {
    if (!(x > neg_inf())) return 0;
    const uint32_t b = __float_as_uint(x + 0.0f);                       // -0 as +0
    const uint32_t order = b ^ (static_cast<uint32_t>(static_cast<int>(b) >> 31) | 0x80000000u);
    return static_cast<Key>(order) << 32 | (0xffffffffu - static_cast<uint32_t>(index));
}

__device__ __forceinline__ int index_of(Key k) { return static_cast<int>(0xffffffffu - static_cast<uint32_t>(k)); }

__device__ __forceinline__ float value_of(Key k) {
    const uint32_t order = static_cast<uint32_t>(k >> 32);
    return __uint_as_float(order ^ (order & 0x80000000u ? 0x80000000u : 0xffffffffu));
}

__device__ __forceinline__ Key exchange(Key k, int o, bool larger) {
    const Key other = __shfl_xor_sync(kAll, k, o);
    return (other > k) == larger ? other : k;
}

// A warp's 32 keys in descending order (bitonic).
__device__ __forceinline__ Key sort_keys(Key k) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int size = 2; size <= 32; size *= 2)
#pragma unroll
        for (int o = size / 2; o; o /= 2) k = exchange(k, o, ((lane & o) == 0) == ((lane & size) == 0));
    return k;
}

// The 32 largest of two lists in descending order.
__device__ __forceinline__ Key merge_keys(Key x, Key y) {
    const int lane = threadIdx.x & 31;
    y = __shfl_sync(kAll, y, 31 - lane);
    Key k = x > y ? x : y;
#pragma unroll
    for (int o = 16; o; o /= 2) k = exchange(k, o, (lane & o) == 0);
    return k;
}

// The largest keys that a warp was given, up to 32: in order in its lanes, and
// more that wait in its part of the memory of the pieces, which are used up: kRow
// keys of each of the rows.
struct Best {
    static constexpr int kRow = 64, kStride = 64 * kWarps;
    Key list, least;       // least: what a key has to reach
    int waiting, k;
    Key* buffer;

    __device__ __forceinline__ Key& place(int i) const { return buffer[i / kRow * kStride + i % kRow]; }

    // the last 32 that wait into the list
    __device__ __forceinline__ void flush() {
        const int lane = threadIdx.x & 31, n = min(waiting, 32);
        waiting -= n;
        list = merge_keys(list, sort_keys(lane < n ? place(waiting + lane) : 0));
        const Key kth = __shfl_sync(kAll, list, k - 1);
        if (kth > least) least = kth;
    }
    // by the whole warp; a unit's elements, at most, before the next settle
    __device__ __forceinline__ void push(Key x) {
        const bool on = x >= least && x != 0;
        const unsigned b = __ballot_sync(kAll, on);
        if (on) place(waiting + __popc(b & ((1u << (threadIdx.x & 31)) - 1))) = x;
        waiting += __popc(b);
    }
    __device__ __forceinline__ void settle(int left) {
        __syncwarp();
#pragma unroll 1
        while (waiting > left) flush();
        __syncwarp();
    }
    // The run's units first, first + step, ..., a lane each, by the whole warp, with
    // three on their way.  Units without an element that reaches the bound are
    // passed over.  The code is short on purpose, since it runs few times for its
    // instructions' way: with every element pushed by itself 8,192 rows of 2,500 in
    // bf16 with five of the best took 38 us instead of 30, units passed over but four
    // at a time unrolled 47.
    template <typename T, int N>
    __device__ __forceinline__ void scan(const Run<T, N>& run, int first, int step, int base) {
        static_assert(31 + 32 * N <= kStages * kUnits * kRow, "a unit of every lane has to fit behind 31 keys");
        const auto load = [&](int at) { return at < run.units ? *reinterpret_cast<const uint4*>(run.unit(at)) : make_uint4(0, 0, 0, 0); };
        const int hop = 32 * step;
        int at = first + static_cast<int>(threadIdx.x & 31) * step;
        uint4 next[3] = {load(at), load(at + hop), load(at + 2 * hop)};
#pragma unroll 1
        for (int i = first; i < run.units; i += hop, at += hop) {
            const uint4 raw = next[0];
            next[0] = next[1];
            next[1] = next[2];
            next[2] = load(at + 3 * hop);
            const float bound = least ? value_of(least) : neg_inf(), top = at < run.units ? largest<T>(raw) : neg_inf();
            const bool on = top >= bound && top > neg_inf();
            if (!__ballot_sync(kAll, on)) continue;
            float x[N];
            numbers(raw, x);
#pragma unroll
            for (int j = 0; j < N; ++j) push(on ? key_of(x[j], base + run.head + N * at + j) : 0);
            settle(31);
        }
    }
};

// ---------------------------------------------------------------- statistics

// What a row's statistics keep of its largest logit m is m scale, and the gradient
// is formed from (x - m) scale as the log probabilities are: with m scale in its
// stead the rounding of m scale would be an error of log p, 3e-4 at 10,000 and 57 in
// a row that is masked with -1e9.  So m has to follow from m scale and log S.
// Two fp32 numbers at most, neighbours, have the same product with scale (their
// products lie more than half a step apart): from kFar on the last bit of log S,
// a step of its own, is m's.  A product past the fp32 range says nothing of m:
// there the statistics are m itself and -log S (-0 for 0), which they are in no
// other row.
template <typename T>
__device__ __forceinline__ float2 stats_of(const LogpParams& p, float m, float log_sum) {
    const float z = __fmul_rn(m, p.scale);
    if (isinf(z) && !isinf(m)) return make_float2(m, -log_sum);
    if (sizeof(T) == 4 && p.rounds && fabsf(z) > kFar)
        log_sum = __int_as_float((__float_as_int(log_sum) & ~1) | (__float_as_int(m) & 1));
    return make_float2(z, log_sum);
}

// (x - m) scale, also where the difference alone is past the fp32 range.
__device__ __forceinline__ float below(float x, float m, float scale) {
    const float d = x - m;
    return isinf(d) && !isinf(x) && !isinf(m) ? x * scale - m * scale : d * scale;
}

// log p = (x times + plus) unit - log S, in base two: (x - m) scale, or, where the
// product's rounding is none or does not matter, x scale - m scale.
struct Origin {
    float times, plus, unit, log_sum;
};

// Of a row whose m scale is far from zero: a call, as few rows take it (inlined the
// gradient of the others took 235.2 us instead of 234.6).
template <typename T>
__device__ __noinline__ Origin far_origin_of(float2 stat, float scale, float scale2, int rounds) {
    float m = stat.x;
    bool known = __float_as_int(stat.y) < 0 && isinf(__fmul_rn(m, scale));
    if (known) {
        stat.y = -stat.y;
    } else if (rounds) {
        const float near = __fdiv_rn(stat.x, scale);               // within a step of m
        if constexpr (sizeof(T) == 2) {
            m = widen(narrow<T>(near));
            known = __fmul_rn(m, scale) == stat.x;
        } else {
#pragma unroll
            for (int i = -1; i <= 1; ++i) {
                const float c = __int_as_float(__float_as_int(near) + i);
                if (__fmul_rn(c, scale) == stat.x && ((__float_as_int(c) ^ __float_as_int(stat.y)) & 1) == 0) {
                    m = c;
                    known = true;
                }
            }
        }
    }
    if (known) return Origin{1.0f, -m, scale2, stat.y};
    return Origin{scale, -stat.x, kLog2e, stat.y};             // exact as it is, or not this library's statistics
}

template <typename T>
__device__ __forceinline__ Origin origin_of(const LogpParams& p, float2 stat) {
    if (fabsf(stat.x) > kFar) return far_origin_of<T>(stat, p.scale, p.scale2, p.rounds);
    return Origin{p.scale, -stat.x, kLog2e, stat.y};
}

// ---------------------------------------------------------------- forward

template <bool TOP>
struct Shared {
    Sums sums[kWarps];
    Sums whole;                    // of this CTA's part of the row
    Key lists[TOP ? kWarps : 1][32];
};

// The lists of all warps of a CTA as one, in the first warp's lanes.
__device__ __forceinline__ Key join_lists(Key mine, Key (*lists)[32]) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    lists[warp][lane] = mine;
#pragma unroll
    for (int n = kWarps / 2; n; n /= 2) {
        __syncthreads();
        if (warp < n) {
            mine = merge_keys(mine, lists[warp + n][lane]);
            lists[warp][lane] = mine;
        }
    }
    return mine;
}

// A thread's 16-byte units lie a row's threads apart (neighbours' next to one another:
// fp32 logits two units a lane took 1.55 times as long, for sectors fetched twice),
// kStages - 1 pieces of them on their way to shared memory while it adds up another.
// 8,192 rows of 50,257 in bf16, a tenth of them left out, with the entropy: 119 us,
// 6.2 TB/s (floor 111); a warp issues in 78 % of the cycles (10 warp instructions
// for 32 elements).  Loaded when they were due, and added up one by one, 172.  Four rows with eight alternatives:
// 9.6 us, most of it the alternatives' second pass and the two waits for the cluster.
template <typename T, int WARPS, bool ENTROPY, bool TOP>
__global__ void __launch_bounds__(32 * kWarps, TOP ? 4 : 5) logp_kernel(const __grid_constant__ LogpParams p) {
    constexpr int kThreads = 32 * WARPS;                    // of a row, in this CTA
    constexpr int N = 16 / static_cast<int>(sizeof(T));     // of 16 bytes
    __shared__ uint4 ahead[kStages][kUnits][32 * kWarps];
    __shared__ Shared<TOP> shared;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t = WARPS == 1 ? lane : threadIdx.x;
    ddpk::dev::pdl_wait();
    ddpk::dev::pdl_trigger();
    const long long row = WARPS == 1 ? static_cast<long long>(blockIdx.x) * kWarps + warp : blockIdx.x / p.split;
    const int part = WARPS == 1 ? 0 : blockIdx.x % p.split;
    if (WARPS == 1 && row >= p.rows) return;
    const bool writer = part == 0 && (WARPS == 1 || warp == 0);     // this warp writes what the row gives
    const int target = target_of(p, row);
    if (target == -1) {                                     // the same in all CTAs of a cluster
        if (writer) {
            if (lane == 0) {
                if (p.logp) p.logp[row] = 0.0f;
                if (p.entropy) p.entropy[row] = 0.0f;
                *reinterpret_cast<float2*>(p.stats + 2 * row) = make_float2(0.0f, 0.0f);
            }
            if (lane < p.top) {
                p.top_index[row * p.top + lane] = -1;
                p.top_logp[row * p.top + lane] = 0.0f;
            }
        }
        return;
    }
    const T* const logits = static_cast<const T*>(p.logits) + row * p.stride;
    const long long lo = part * p.segment, hi = min(static_cast<long long>(p.vocab), lo + p.segment);
    const Run<T, N> run(logits, lo, hi);
    const float c = p.scale2;
    Sums sums = {neg_inf(), 0.0f, 0.0f};
    // where this thread's largest lies: in the units of a piece from this one on; -2: head, -3: rest
    int best = -1;
    const auto request = [&](int piece) {
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            const int i = t + (piece * kUnits + u) * kThreads;
            if (i < run.units) copy_async(&ahead[piece % kStages][u][threadIdx.x], run.unit(i));
        }
        copy_commit();
    };
#pragma unroll
    for (int s = 0; s + 1 < kStages; ++s) request(s);
    if (t < run.head && take_one<ENTROPY>(widen(run.from[t]), c, sums)) best = -2;
    for (int piece = 0; t + piece * kUnits * kThreads < run.units; ++piece) {
        copy_wait<kStages - 2>();
        using Pair = typename std::conditional<sizeof(T) == 2, uint32_t, float2>::type;
        Pair x[N / 2 * kUnits];
#pragma unroll
        for (int u = 0; u < kUnits; ++u) {
            const bool on = u == 0 || t + (piece * kUnits + u) * kThreads < run.units;
            const uint4 v = ahead[piece % kStages][u][threadIdx.x];
            uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (!on) w[j] = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;      // -inf
#pragma unroll
            for (int j = 0; j < N / 2; ++j) {
                if constexpr (sizeof(T) == 2) x[u * (N / 2) + j] = w[j];
                else x[u * (N / 2) + j] = make_float2(__uint_as_float(w[2 * j]), __uint_as_float(w[2 * j + 1]));
            }
        }
        request(piece + kStages - 1);                       // into the place of the piece before, which is used up
        if (take<N / 2 * kUnits, ENTROPY>(x, c, sums)) best = t + piece * kUnits * kThreads;
    }
    if (t < run.n - run.rest() && take_one<ENTROPY>(widen(run.from[run.rest() + t]), c, sums)) best = -3;

    Key list = 0;
    if constexpr (TOP) {
        const int base = static_cast<int>(lo);
        // this thread's best: the first of its batch that is as large
        Key mine = 0;
        if (best == -2) mine = key_of(sums.m, base + t);
        if (best == -3) mine = key_of(sums.m, base + run.rest() + t);
        if (best >= 0) {
            for (int u = 0; u < kUnits && !mine; ++u) {
                const int at = best + u * kThreads;
                if (at >= run.units) break;
                float x[N];
                numbers(*reinterpret_cast<const uint4*>(run.unit(at)), x);
#pragma unroll
                for (int j = N - 1; j >= 0; --j)
                    if (x[j] == sums.m) mine = key_of(x[j], base + run.head + N * at + j);
            }
        }
        __syncwarp();                                       // the pieces' memory is free from here on
        list = sort_keys(mine);
        if constexpr (WARPS > 1) {
            list = join_lists(list, shared.lists);
            __syncthreads();
            list = shared.lists[0][lane];                   // the threads' best 32, in every warp
            __syncthreads();
        }
        Best found = {0, __shfl_sync(kAll, list, p.top - 1), 0, p.top, reinterpret_cast<Key*>(ahead) + warp * Best::kRow};
        if constexpr (WARPS == 1) {
            found.scan(run, 0, 1, base);
            found.push(lane < run.head ? key_of(widen(run.from[lane]), base + lane) : 0);
            const int at = run.rest() + lane;
            found.push(at < run.n ? key_of(widen(run.from[at]), base + at) : 0);
        } else {
            for (int w = warp; w < p.top; w += WARPS) {
                const Key winner = __shfl_sync(kAll, list, w);
                if (!winner) break;
                int of = index_of(winner) - base;           // whose it is
                of = of < run.head ? of : of >= run.rest() ? of - run.rest() : (of - run.head) / N % kThreads;
                found.scan(run, of, kThreads, base);
                const int at = lane == 0 && of < run.head ? of : lane == 1 && run.rest() + of < run.n ? run.rest() + of : -1;
                found.push(at >= 0 ? key_of(widen(run.from[at]), base + at) : 0);
                found.settle(31);
            }
        }
        found.settle(0);
        list = found.list;
        if constexpr (WARPS > 1) list = join_lists(list, shared.lists);
    }

    sums = join_lanes<32>(sums, c);
    if constexpr (WARPS > 1) {
        if (lane == 0) shared.sums[warp] = sums;
        __syncthreads();
        if (warp == 0) sums = join_lanes<WARPS>(shared.sums[lane % WARPS], c);
        if (p.split > 1) {
            cg::cluster_group cluster = cg::this_cluster();
            if (threadIdx.x == 0) shared.whole = sums;
            cluster.sync();
            if (writer) {
                const int r = lane % kMaxSplit;             // in every eight lanes
                sums = r < p.split ? *cluster.map_shared_rank(&shared.whole, r) : Sums{neg_inf(), 0.0f, 0.0f};
                sums = join_lanes<kMaxSplit>(sums, c);
                if constexpr (TOP)
                    for (int q = 1; q < p.split; ++q) list = merge_keys(list, *cluster.map_shared_rank(&shared.lists[0][lane], q));
            }
            cluster.sync();                                 // their shared memory stays until it is read
        }
    }
    if (!writer) return;
    const bool nothing = sums.m == neg_inf() && sums.s == 0.0f;      // no logit above -inf
    const float log_sum = nothing ? 0.0f : logf(sums.s);
    if (lane == 0) {
        if (p.logp && target >= 0)
            p.logp[row] = nothing ? neg_inf() : below(widen(logits[target]), sums.m, p.scale) - log_sum;
        if (ENTROPY) p.entropy[row] = nothing ? 0.0f : log_sum - kLn2 * __fdiv_rn(sums.a, sums.s);
        *reinterpret_cast<float2*>(p.stats + 2 * row) = stats_of<T>(p, sums.m, log_sum);
    }
    if constexpr (TOP) {
        if (lane < p.top) {
            p.top_index[row * p.top + lane] = list ? index_of(list) : -1;
            p.top_logp[row * p.top + lane] =
                list ? below(value_of(list), sums.m, p.scale) - log_sum : sums.s == sums.s ? neg_inf() : nan_value();
        }
    }
}

// ---------------------------------------------------------------- backward

// d log p_t / d z_i = [i = t] - p_i and d H / d z_i = -p_i (log p_i + H): a thread's
// elements of a row take p (alpha + beta log2 p).
struct Slope {
    float times, plus, unit, log_sum2, alpha, beta;

    template <bool ENTROPY>
    __device__ __forceinline__ float2 at(float2 x) const {
        const float2 d = fma2(fma2(x, both(times), both(plus)), both(unit), both(-log_sum2));      // log2 p
        float2 y = both(alpha);
        if constexpr (ENTROPY) y = fma2(both(beta), make_float2(fmaxf(d.x, kFloor), fmaxf(d.y, kFloor)), y);
        return mul2(make_float2(exp2_fast(d.x), exp2_fast(d.y)), y);
    }
};

// Eights that start on 16 bytes of the gradient; the logits' eights lie `shift`
// bytes off, the same all along a row.  A lane loads the aligned words that its
// eights begin in, and has the next lane's for their ends; none is loaded that
// does not hold a logit of the row.  A CTA takes 4,096 (fp32: 2,048) elements and
// has nothing to wait for but its loads, and twelve are resident.  8,192 rows of
// 50,257 in bf16, entropy too: 234.6 us, 6.7 TB/s, the copy's rate (floor 233); logits
// element by element 415, shifted out of two loads each 271.  4,096 rows in fp32 231,
// and 3 % more where m is far from zero and is looked for.
template <typename T, bool ENTROPY>
__global__ void __launch_bounds__(kBackThreads, kBackCtas) logp_backward_kernel(const __grid_constant__ LogpParams p) {
    constexpr int kEights = kBackEights<T>;
    ddpk::dev::pdl_wait();
    ddpk::dev::pdl_trigger();
    const long long row = blockIdx.x / p.split;
    const long long lo = blockIdx.x % p.split * p.segment, hi = min(static_cast<long long>(p.vocab), lo + p.segment);
    const T* const from = static_cast<const T*>(p.logits) + row * p.stride + lo;
    const Run<T, 8> run(static_cast<const T*>(p.out) + row * p.out_stride, lo, hi);
    T* const to = static_cast<T*>(p.out) + row * p.out_stride + lo;
    const int target = target_of(p, row);
    const float2 stat = *reinterpret_cast<const float2*>(p.stats + 2 * row);
    const bool zero = target == -1 || (stat.x == neg_inf() && stat.y == 0.0f);     // (a row of NaN has a NaN sum)
    const int shift = static_cast<int>(reinterpret_cast<uintptr_t>(from + run.head) & 15);
    const int lane = threadIdx.x & 31, first = (threadIdx.x >> 5) * (32 * kEights) + lane;
    const T* const words = reinterpret_cast<const T*>(reinterpret_cast<const char*>(from + run.head) - shift);
    Eight<T> raw[kEights];
    uint4 last = make_uint4(0, 0, 0, 0);                    // lane 0: what follows the warp's eights
#pragma unroll
    for (int u = 0; u < kEights; ++u) {
        const int i = first + u * 32;
        if (!zero && i < run.units) raw[u].load(words + 8 * i);
        else if (!zero && i == run.units && shift) *reinterpret_cast<uint4*>(&raw[u]) = *reinterpret_cast<const uint4*>(words + 8 * i);
    }
    if (!zero && shift && lane == 0 && first + 32 * kEights <= run.units)
        last = *reinterpret_cast<const uint4*>(words + 8 * (first + 32 * kEights));
    const float g = p.grad_logp && target >= 0 ? p.grad_logp[row] : 0.0f;
    const float h = ENTROPY ? p.grad_entropy[row] : 0.0f;
    const Origin origin = origin_of<T>(p, stat);
    const Slope slope = {origin.times, origin.plus, origin.unit, origin.log_sum * kLog2e,
                         -p.scale * (ENTROPY ? fmaf(h, p.entropy[row], g) : g), -p.scale * h * kLn2};
    const float extra = p.scale * g;
    const int aim = target - static_cast<int>(lo);
    // the ends, at most seven elements each
    const int ends = run.n - 8 * run.units;
    if (threadIdx.x < ends) {
        const int i = threadIdx.x < run.head ? threadIdx.x : threadIdx.x + 8 * run.units;
        float y = zero ? 0.0f : slope.at<ENTROPY>(both(widen(from[i]))).x;
        if (i == aim && !zero) y += extra;
        to[i] = narrow<T>(y);
    }
#pragma unroll
    for (int u = 0; u < kEights; ++u) {
        const int i = first + u * 32;
        if (i - lane >= run.units) break;                  // the whole warp's
        if (shift && !zero) {
            const uint4 mine = *reinterpret_cast<const uint4*>(&raw[u]);
            const uint4 ahead = u + 1 < kEights ? *reinterpret_cast<const uint4*>(&raw[u + 1 < kEights ? u + 1 : 0]) : last;
            const uint4 give = lane == 0 ? ahead : mine;    // lane 0 to lane 31
            const int next = (lane + 1) & 31;
            const uint4 behind = make_uint4(__shfl_sync(kAll, give.x, next), __shfl_sync(kAll, give.y, next),
                                            __shfl_sync(kAll, give.z, next), __shfl_sync(kAll, give.w, next));
            raw[u] = shifted(raw[u], behind, shift);
        }
        if (i >= run.units) continue;
        Eight<T> out;
        out.zero();
        if (!zero) {
            float x[8];
            raw[u].get(x);
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const float2 y = slope.at<ENTROPY>(make_float2(x[j], x[j + 1]));
                x[j] = y.x;
                x[j + 1] = y.y;
            }
            const unsigned place = static_cast<unsigned>(aim - run.head - 8 * i);
            if (place < 8) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (place == j) x[j] += extra;
            }
            out.put(x);
        }
        out.store_once(to + run.head + 8 * i);
    }
}

// ---------------------------------------------------------------- host

template <typename T, int WARPS>
cudaError_t forward_as(const LogpParams& p, cudaStream_t stream) {
    void (*kernel)(LogpParams);
    if (p.entropy) kernel = p.top ? logp_kernel<T, WARPS, true, true> : logp_kernel<T, WARPS, true, false>;
    else kernel = p.top ? logp_kernel<T, WARPS, false, true> : logp_kernel<T, WARPS, false, false>;
    if (WARPS == 1) return launch(kernel, (p.rows + kWarps - 1) / kWarps, 32 * kWarps, 0, stream, p);
    return launch(kernel, p.rows * p.split, 32 * kWarps, 0, stream, p, p.split);
}

template <typename T>
cudaError_t forward(LogpParams& p, cudaStream_t stream) {
    p.split = 1;
    p.segment = p.vocab;
    // Rows of a middling length, where there are many: what a CTA does at a row's
    // ends (its warps' sums and lists joined, few CTAs at a time) costs more than a
    // warp's longer row.  us with a CTA / a warp each, 8,192 rows: 2,500 bf16 32 /
    // 12, with 5 of the best 104 / 30; 8,192 bf16 37 / 28, with 5 111 / 53, fp32 49 /
    // 49, with 5 111 / 110; 16,384 bf16 50 / 50, with 5 127 / 116, fp32 79 / 86, with
    // 5 136 / 213.  1,024 rows: 8,192 bf16 6.0 / 4.4, with 5 16.0 / 15.0; 12,000 bf16
    // with 5 17.4 / 19.5.
    const int64_t bytes = p.vocab * static_cast<int64_t>(sizeof(T));
    const bool many = (p.rows >= kSomeRows && bytes <= kSomeBytes) || (p.rows >= kManyRows && bytes <= kManyBytes);
    if (p.vocab <= kWarpVocab || many) return forward_as<T, 1>(p, stream);
    // few rows: as many CTAs a row as keep every thread eight elements or more
    while (p.split < kMaxSplit && p.rows * p.split < 2 * kSms && p.vocab / (2 * p.split) >= 8 * 32 * kWarps) p.split *= 2;
    p.segment = ((p.vocab + p.split - 1) / p.split + 7) / 8 * 8;
    return forward_as<T, kWarps>(p, stream);
}

template <typename T>
cudaError_t backward(LogpParams& p, cudaStream_t stream) {
    p.segment = 8LL * kBackThreads * kBackEights<T>;
    p.split = static_cast<int>((p.vocab + p.segment - 1) / p.segment);
    return launch(p.grad_entropy ? logp_backward_kernel<T, true> : logp_backward_kernel<T, false>, p.rows * p.split, kBackThreads, 0,
                  stream, p);
}

bool valid(const ddp_logprobs_args* a) {
    return a && a->rows >= 0 && a->rows <= INT32_MAX / 8 && a->vocab >= 1 && a->vocab <= 1 << 24 && a->row_stride >= a->vocab &&
           a->top >= 0 && a->top <= kMaxTop && a->top <= a->vocab && a->scale >= 0x1p-64f && a->scale <= 0x1p64f &&
           (a->dtype == DDP_F32 || a->dtype == DDP_BF16) && (a->index_bits == 32 || a->index_bits == 64);
}

LogpParams params_of(const ddp_logprobs_args* a) {
    LogpParams p = {};
    p.rows = a->rows;
    p.vocab = static_cast<int>(a->vocab);
    p.stride = a->row_stride;
    p.top = a->top;
    p.wide = a->index_bits == 64;
    p.scale = a->scale;
    p.scale2 = static_cast<float>(a->scale * 1.4426950408889634);
    int exponent;
    p.rounds = std::frexp(a->scale, &exponent) != 0.5f;
    return p;
}

}  // namespace

extern "C" {

int ddp_logprobs(const ddp_logprobs_args* a, const void* logits, const void* targets, float* logp, float* entropy, float* stats,
                 int32_t* top_index, float* top_logp, void* stream) {
    if (!valid(a)) return DDP_ERR_INVALID_ARG;
    if (a->rows == 0) return DDP_OK;
    if (!logits || !stats || !targets != !logp || (a->top > 0 && (!top_index || !top_logp)) ||
        !aligned(logits, a->dtype == DDP_F32 ? 4 : 2) || !aligned(targets, a->index_bits / 8) || !aligned(logp, 4) ||
        !aligned(entropy, 4) || !aligned(stats, 8) || !aligned(top_index, 4) || !aligned(top_logp, 4))
        return DDP_ERR_INVALID_ARG;
    LogpParams p = params_of(a);
    p.logits = logits;
    p.targets = targets;
    p.logp = logp;
    p.entropy = entropy;
    p.stats = stats;
    p.top_index = top_index;
    p.top_logp = top_logp;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = a->dtype == DDP_F32 ? forward<float>(p, st) : forward<uint16_t>(p, st);
    return e == cudaSuccess ? DDP_OK : DDP_ERR_CUDA;
}

int ddp_logprobs_backward(const ddp_logprobs_args* a, const void* logits, const void* targets, const float* stats,
                          const float* entropy, const float* grad_logp, const float* grad_entropy, void* grad_logits,
                          int64_t grad_stride, void* stream) {
    ddp_logprobs_args without_top = a ? *a : ddp_logprobs_args{};
    without_top.top = 0;
    if (!a || !valid(&without_top) || grad_stride < a->vocab) return DDP_ERR_INVALID_ARG;
    if (a->rows == 0) return DDP_OK;
    const int size = a->dtype == DDP_F32 ? 4 : 2;
    if (!logits || !stats || !grad_logits || (grad_logp && !targets) || !entropy != !grad_entropy || (!grad_logp && !grad_entropy) ||
        !aligned(logits, size) || !aligned(grad_logits, size) || !aligned(targets, a->index_bits / 8) || !aligned(stats, 8) ||
        !aligned(entropy, 4) || !aligned(grad_logp, 4) || !aligned(grad_entropy, 4))
        return DDP_ERR_INVALID_ARG;
    LogpParams p = params_of(a);
    p.logits = logits;
    p.targets = targets;
    p.stats = const_cast<float*>(stats);
    p.entropy = const_cast<float*>(entropy);
    p.grad_logp = grad_logp;
    p.grad_entropy = grad_entropy;
    p.out = grad_logits;
    p.out_stride = grad_stride;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = a->dtype == DDP_F32 ? backward<float>(p, st) : backward<uint16_t>(p, st);
    return e == cudaSuccess ? DDP_OK : DDP_ERR_CUDA;
}

}  // extern "C"
