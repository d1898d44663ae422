// Routing of tokens to experts and its gradient.
//
// A token's experts lie in runs of 8 `chunks` to a lane over LPT lanes, so a
// warp holds 32 / LPT tokens; a group's experts start on a lane of their own
// (its last lanes may be partly empty) and take a power of two of lanes.  The
// choice goes by 32-bit keys: 23 bits of the compared value above 9 bits of 511
// - expert, so no two are equal, the larger key is the better expert, and ties
// of the value go to the lowest expert.  Each lane keeps the eight largest of
// its chunks sorted; the k best of a token are the largest of its lanes' first,
// k times over.
//
// The fp32 definition of a score is expf and IEEE division; the sum of a
// softmax adds eight experts of a group in turn, then pairs of eights of the
// group and pairs of groups (each counted up to a power of two, with zeros),
// which is the order of every layout of experts over lanes: a token's scores do
// not depend on the batch that it is routed in.
//
// 23 bits, and scores from the hardware's approximate exponential and
// reciprocal, do not always tell which of two experts the fp32 definition puts
// first.  Where values that the choice told apart are nearer than the errors
// of both, the k chosen and the next best are put into order by the definition
// (order_exact); where that may not be enough, or a logit or bias is not an
// ordinary number, the token is chosen by it alone (choose_exact).  The scores
// of the chosen experts are always computed by the definition.
//
// The forward kernel is bound by instructions, not by HBM: over 256 experts it
// reads 1 KiB a token and executes about 390 warp instructions (scores, keys
// and sorting of 256 values; k rounds; the k slots' exact scores), half of them
// on the integer and compare pipe, which takes one every other cycle.  GB300,
// 65,536 tokens, logits in HBM: 256 experts in 8 groups with a bias 32.8 us (2.1
// TB/s; the logits alone at the copy peak 10 us), ungrouped softmax over 64 / 128
// / 256 experts in bf16 13.2 / 18.3 / 27.9 us renormalised, and 16.6 / 24.6 / 40.0
// as it is, for the sum over the row.  A few tokens take 3.3 us.

#include "ddp_reducer.h"

#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdint>

#include "ddp_device.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxExperts = 512;
constexpr int kMaxSlots = 256;           // slots of a warp's tokens at once
constexpr unsigned kAll = 0xffffffffu;
constexpr int kForwardCtas = 3;          // route_kernel's on an SM: 80 registers; at 64 it spills (65,536 tokens 37.7 -> 49.5 us)
constexpr int kChosenCtas = 8, kWholeCtas = 16;      // the backward kernels' on an SM at most

// Least distance, in units of 2^-21 (the keys' step), of two values whose
// order is certain.  A sigmoid score plus bias is within 0.9e-6 of the fp32
// definition's (approximate exponential 2^-22, reciprocal 2^-23, each weighed
// by the sigmoid's slope; the definition's own roundings; the key's), so two
// are certain 3.8 units apart, and sums of two 8.6.  A softmax score is a quotient
// by the definition's own sum: approximate exponential 2^-22, its argument's
// rounding (0.37 2^-24 of a score at most), quotient and product 2^-21, expf and
// division 2^-22: 1.1e-6 with the key's, 4.6 units for two and 9.2 for sums of two.
constexpr uint32_t kMarginSoftmax = 24, kMarginSigmoid = 6;

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
    int chunks;                  // forward: of 8 experts, of a lane
    int group_slots;             // forward: slots of a group: a multiple of a lane's, over it a power of two
    int reps;                    // forward: rounds of 32 / LPT tokens before their slots are weighed
    int fits;                    // forward: the groups fit the lanes' slots (else every token is chosen exactly)
    int vec;                     // rows start 16-byte aligned (chosen-only backward: the gradient's, next to one another)
    int row_tokens;              // chosen-only backward: tokens of a warp at once
    int slot_lanes;              // chosen-only backward: lanes of a token, a power of two >= k
};

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(uint16_t x) { return ddpk::dev::widen1(x); }
template <typename T> __device__ __forceinline__ T narrow(float x);
template <> __device__ __forceinline__ float narrow<float>(float x) { return x; }
template <> __device__ __forceinline__ uint16_t narrow<uint16_t>(float x) {
    return static_cast<uint16_t>(__float_as_uint(ddpk::dev::round_bf16(x)) >> 16);
}

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }
__device__ __forceinline__ float nan_value() { return __int_as_float(0x7fffffff); }

// A key that orders like the number (-0 equal to +0); 0 for -inf and NaN.
__device__ __forceinline__ uint32_t order_bits(float x) {
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b ^ (static_cast<uint32_t>(static_cast<int>(b) >> 31) | 0x80000000u);
}

__device__ __forceinline__ uint32_t key_of(float x) { return x > neg_inf() ? order_bits(x) : 0u; }

__device__ __forceinline__ float number_of(uint32_t key) {
    return key == 0 ? neg_inf() : __uint_as_float(key ^ (key & 0x80000000u ? 0x80000000u : 0xffffffffu));
}

// Over a token's LPT lanes.
template <int LPT>
__device__ __forceinline__ uint32_t token_max(uint32_t x) {
    if constexpr (LPT == 32) {
        return __reduce_max_sync(kAll, x);
    } else {
#pragma unroll
        for (int o = LPT / 2; o; o >>= 1) x = max(x, __shfl_xor_sync(kAll, x, o));
        return x;
    }
}

// Neighbours first, as the definition of a softmax's sum has it.
template <int LPT>
__device__ __forceinline__ float token_sum(float x) {
#pragma unroll
    for (int o = 1; o < LPT; o *= 2) x = __fadd_rn(x, __shfl_xor_sync(kAll, x, o));
    return x;
}

__device__ __forceinline__ float sigmoid(float x) { return __fdiv_rn(1.0f, __fadd_rn(1.0f, expf(-x))); }

__device__ __forceinline__ float fast_exp(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
    return y;
}

__device__ __forceinline__ float fast_reciprocal(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float fast_sigmoid(float x) { return fast_reciprocal(1.0f + fast_exp(-x)); }

// A lane's experts of a row: n consecutive ones from `from` (n <= EPL); the
// rest are `fill`.
template <int EPL, typename T>
__device__ __forceinline__ void load_lane(const T* from, int n, bool vec, float fill, float (&x)[EPL]) {
    if (vec && n == EPL) {
        constexpr int V = 16 / sizeof(T);
        using Raw = typename ddpk::dev::Vec<T>::Raw;
#pragma unroll
        for (int c = 0; c < EPL / V; ++c) {
            float f[V];
            ddpk::dev::Vec<T>::unpack(__ldg(reinterpret_cast<const Raw*>(from) + c), f);
#pragma unroll
            for (int i = 0; i < V; ++i) x[c * V + i] = f[i];
        }
    } else {
#pragma unroll
        for (int j = 0; j < EPL; ++j) x[j] = j < n ? widen(from[j]) : fill;
    }
}

template <int EPL>
__device__ __forceinline__ void store_lane(float* to, int n, bool vec, const float (&d)[EPL]) {
    if (vec && n == EPL) {
#pragma unroll
        for (int c = 0; c < EPL; c += 4) ddpk::dev::st_stream(to + c, make_float4(d[c], d[c + 1], d[c + 2], d[c + 3]));
    } else {
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            if (j < n) to[j] = d[j];
    }
}

template <int EPL>
__device__ __forceinline__ void store_lane(uint16_t* to, int n, bool vec, const float (&d)[EPL]) {
    uint32_t x[EPL / 2];
#pragma unroll
    for (int j = 0; j < EPL; j += 2)
        x[j / 2] = narrow<uint16_t>(d[j]) | static_cast<uint32_t>(narrow<uint16_t>(d[j + 1])) << 16;
    if (vec && n == EPL) {
#pragma unroll
        for (int c = 0; c < EPL / 2; c += 4)
            __stcs(reinterpret_cast<uint4*>(to) + c / 4, make_uint4(x[c], x[c + 1], x[c + 2], x[c + 3]));
    } else {
#pragma unroll
        for (int j = 0; j < EPL; ++j)
            if (j < n) to[j] = static_cast<uint16_t>(x[j / 2] >> (16 * (j % 2)));
    }
}

// Larger first.
__device__ __forceinline__ void order(uint32_t& a, uint32_t& b) {
    const uint32_t x = max(a, b), y = min(a, b);
    a = x;
    b = y;
}

// Eight in descending order (19 comparisons, Batcher's odd-even merge sort).
__device__ __forceinline__ void sort8(uint32_t (&x)[8]) {
    order(x[0], x[1]); order(x[2], x[3]); order(x[4], x[5]); order(x[6], x[7]);
    order(x[0], x[2]); order(x[1], x[3]); order(x[4], x[6]); order(x[5], x[7]);
    order(x[1], x[2]); order(x[5], x[6]);
    order(x[0], x[4]); order(x[1], x[5]); order(x[2], x[6]); order(x[3], x[7]);
    order(x[2], x[4]); order(x[3], x[5]);
    order(x[1], x[2]); order(x[3], x[4]); order(x[5], x[6]);
}

// The eight largest of two sorted eights, in descending order: the larger of
// x[i] and y[7 - i] are a bitonic sequence, which three steps sort.
__device__ __forceinline__ void merge8(uint32_t (&x)[8], const uint32_t (&y)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = max(x[i], y[7 - i]);
#pragma unroll
    for (int d = 4; d; d /= 2)
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (!(i & d)) order(x[i], x[i + d]);
}

// What the scores of a token's slots are computed from.
struct Stat {
    float top, sum;    // softmax
    int bad;           // every weight is NaN
};

struct WarpRows {
    float c[kMaxExperts];        // choose_exact: what the choice goes by
    int32_t sel[kMaxSlots];
    int32_t next[32];            // a token's best that was not chosen
    float score[kMaxSlots];
    Stat stat[32];
};

// One token's choice by the fp32 definition, by a whole warp.  sel: as the
// keys give it, 511 - expert in the low 9 bits below something not zero; 0 for
// none.
template <typename T>
__device__ __noinline__ void choose_exact(const RouteParams& a, const T* row, float* c, int32_t* sel, Stat* stat) {
    const int lane = threadIdx.x & 31;
    const int E = a.E;
    const bool by_logit = !a.bias && a.groups == 1;
    bool bad = false;
    uint32_t most = 0;
    for (int e = lane; e < E; e += 32) {
        const float x = widen(row[e]);
        bad |= !(x == x) || (a.softmax && x == -neg_inf());
        most = max(most, key_of(x));
    }
    bad = __any_sync(kAll, bad);
    float top = 0.0f, sum = 1.0f;
    if (a.softmax && !(a.renorm && by_logit)) {          // (weights over their sum need none)
        top = number_of(__reduce_max_sync(kAll, most));
        // the eights of a group up to a power of two, 120 of all groups at most: one a lane at a time
        const int size = E / a.groups;
        int shift = 0;
        while (8 << shift < size) ++shift;
        float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (32 * i >= a.groups << shift) break;
            const int at = 32 * i + lane, g = at >> shift, first = 8 * (at & ((1 << shift) - 1));
            const int n = g < a.groups ? min(size - first, 8) : 0;
            float eight = 0.0f;
            for (int j = 0; j < n; ++j) {
                const float x = widen(row[g * size + first + j]);
                if (x > neg_inf()) eight = __fadd_rn(eight, expf(x - top));
            }
            part[i] = token_sum<32>(eight);
        }
        sum = __fadd_rn(__fadd_rn(part[0], part[1]), __fadd_rn(part[2], part[3]));
    }
    for (int e = lane; e < E; e += 32) {
        const float x = widen(row[e]);
        float y = x;
        if (!by_logit) {
            y = a.softmax ? __fdiv_rn(expf(x - top), sum) : sigmoid(x);
            if (a.bias) y = __fadd_rn(y, a.bias[e]);
        }
        c[e] = x > neg_inf() && y > neg_inf() ? y + 0.0f : neg_inf();
    }
    __syncwarp();
    if (a.groups > 1) {
        const int size = E / a.groups;
        uint32_t worth = 0;
        if (lane < a.groups) {           // lane g: group g
            float a1 = neg_inf(), a2 = neg_inf();
            for (int i = 0; i < size; ++i) {
                const float y = c[lane * size + i];
                a2 = fmaxf(a2, fminf(a1, y));
                a1 = fmaxf(a1, y);
            }
            worth = max(key_of(size > 1 ? __fadd_rn(a1, a2) : a1), 1u);
        }
        unsigned stay = 0;
        for (int r = 0; r < a.top_groups; ++r) {
            const uint32_t best = __reduce_max_sync(kAll, worth);
            const int g = __ffs(__ballot_sync(kAll, worth == best)) - 1;
            stay |= 1u << g;
            if (lane == g) worth = 0;
        }
        __syncwarp();
        for (int e = lane; e < E; e += 32)
            if (!(stay >> (e / size) & 1)) c[e] = neg_inf();
        __syncwarp();
    }
    for (int r = 0; r < a.k; ++r) {
        uint32_t mine = 0;
        int at = E;
        for (int e = lane; e < E; e += 32) {
            const uint32_t key = key_of(c[e]);
            if (key > mine) { mine = key; at = e; }
        }
        const uint32_t best = __reduce_max_sync(kAll, mine);
        const int chosen = __reduce_min_sync(kAll, best && mine == best ? at : E);
        if (lane == 0) sel[r] = chosen < E ? kMaxExperts | (kMaxExperts - 1 - chosen) : 0;
        if (lane == (chosen & 31) && chosen < E) c[chosen] = neg_inf();
        __syncwarp();
    }
    if (lane == 0) *stat = Stat{top, sum, bad};
    __syncwarp();
}

// The order of a token's k chosen and the next best, by the fp32 definition,
// by a whole warp: for tokens where these are known to be the k + 1 best, but
// not in which order.  sel, next: as the keys give them; k < 32.
template <typename T>
__device__ __forceinline__ void order_exact(const RouteParams& a, const T* row, int32_t* sel, int32_t next, const Stat& stat) {
    const int lane = threadIdx.x & 31;
    const int32_t word = lane < a.k ? sel[lane] : lane == a.k ? next : 0;
    const int e = kMaxExperts - 1 - (word & (kMaxExperts - 1));
    uint32_t key = 0;
    if (word) {
        const float x = widen(row[e]);
        float y = x;
        if (a.bias || a.groups > 1) {
            y = a.softmax ? __fdiv_rn(expf(x - stat.top), stat.sum) : sigmoid(x);
            if (a.bias) y = __fadd_rn(y, a.bias[e]);
        }
        key = key_of(y);
    }
    int rank = 0;
    for (int r = 0; r <= a.k; ++r) {
        const uint32_t other = __shfl_sync(kAll, key, r);
        const int place = __shfl_sync(kAll, e, r);
        rank += other > key || (other == key && place < e);
    }
    __syncwarp();
    if (word && rank < a.k) sel[rank] = kMaxExperts | (kMaxExperts - 1 - e);
    __syncwarp();
}

// Whether this lane's group stays, by the fp32 definition; for all tokens of a
// warp.  The lane's experts are n from e0 on; k1, k2, k3: its largest keys.
// Its two largest values are those of k1 and k2, unless k3 is less than `near`
// below.
template <int LPT, typename T>
__device__ __noinline__ bool groups_exact(const RouteParams& a, const T* row, int e0, int n, uint32_t k1, uint32_t k2,
                                          uint32_t k3, uint32_t near, float top, float sum, int g, int group_lanes,
                                          int size) {
    const auto value = [&](int e) {
        const float x = widen(row[e]);
        const float s = a.softmax ? __fdiv_rn(expf(x - top), sum) : sigmoid(x);
        return a.bias ? __fadd_rn(s, a.bias[e]) : s;
    };
    float a1 = neg_inf(), a2 = neg_inf();
    const bool two = k2 - k3 >= near;
    for (int j = 0; j < (two ? min(n, 2) : n); ++j) {
        const float c = value(two ? kMaxExperts - 1 - static_cast<int>((j ? k2 : k1) & (kMaxExperts - 1)) : e0 + j);
        a2 = fmaxf(a2, fminf(a1, c));
        a1 = fmaxf(a1, c);
    }
    for (int o = 1; o < group_lanes; o *= 2) {
        const float b1 = __shfl_xor_sync(kAll, a1, o), b2 = __shfl_xor_sync(kAll, a2, o);
        a2 = fmaxf(fminf(a1, b1), fmaxf(a2, b2));
        a1 = fmaxf(a1, b1);
    }
    uint32_t worth = g < a.groups ? max(key_of(size > 1 ? __fadd_rn(a1, a2) : a1), 1u) : 0u;
    bool stays = false;
    for (int r = 0; r < a.top_groups; ++r) {
        const uint32_t best = token_max<LPT>(worth);
        const uint32_t first = token_max<LPT>(worth == best ? static_cast<uint32_t>(32 - g) : 0u);   // the lowest of those that tie
        if (worth == best && g == 32 - static_cast<int>(first)) { worth = 0; stays = true; }
    }
    return stays;
}

// A token's largest logit and the sum of its exponentials by the definition:
// eights, pairs of eights within the lane and then over the lanes.  The lane's
// experts are n (none where negative) from `from` on.  65,536 tokens over 64 / 128
// / 256 experts in bf16 16.6 / 24.6 / 40.0 us; with a sum of approximate
// exponentials, which the weights and near ties then rest on, 15.0 / 22.8 / 37.0.
template <int LPT, typename T>
__device__ __forceinline__ float2 softmax_stat(const T* from, int n, int chunks, bool vec) {
    uint32_t most = 0;
    for (int c = 0; c < chunks; ++c) {
        float y[8];
        load_lane<8>(from + 8 * c, min(n - 8 * c, 8), vec, neg_inf(), y);
#pragma unroll
        for (int j = 0; j < 8; ++j) most = max(most, key_of(y[j]));
    }
    const float top = number_of(token_max<LPT>(most));
    float sum = 0.0f, pair = 0.0f;
    for (int c = 0; c < chunks; ++c) {
        float y[8];
        load_lane<8>(from + 8 * c, min(n - 8 * c, 8), vec, neg_inf(), y);
        float eight = expf(y[0] - top);
#pragma unroll
        for (int j = 1; j < 8; ++j) eight = __fadd_rn(eight, expf(y[j] - top));
        if (c & 1) { sum = __fadd_rn(sum, __fadd_rn(pair, eight)); pair = 0.0f; }
        else pair = eight;
    }
    return make_float2(top, token_sum<LPT>(__fadd_rn(sum, pair)));    // one chunk: its eight alone
}

template <int LPT, typename T>
__global__ void __launch_bounds__(kThreads, kForwardCtas)
route_kernel(const __grid_constant__ RouteParams a) {
    constexpr int kTokens = 32 / LPT;     // of a warp
    __shared__ int hist[kMaxExperts];
    __shared__ float4 biases[kMaxExperts / 4];     // piece h of chunk c of lane l at (2 c + h) LPT + l
    __shared__ uint32_t widest_bits;               // largest magnitude of a bias
    __shared__ WarpRows rows[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int l = lane % LPT, tl = lane / LPT;
    const int E = a.E, k = a.k, chunks = a.chunks, lane_slots = 8 * chunks;
    WarpRows& mem = rows[warp];
    if (a.counts)
        for (int i = threadIdx.x; i < E; i += kThreads) hist[i] = 0;
    if (threadIdx.x == 0) widest_bits = 0;
    __syncthreads();
    ddpk::dev::pdl_wait();
    ddpk::dev::pdl_trigger();

    // this lane's experts: n from e0 on, of group g
    const int size = E / a.groups, group_lanes = a.group_slots / lane_slots;
    const int g = l * lane_slots / a.group_slots, off = l * lane_slots % a.group_slots;
    const int e0 = g * size + off;
    const int n = g < a.groups ? max(0, min(size - off, lane_slots)) : 0;
    const bool by_logit = !a.bias && a.groups == 1;
    const bool vec = a.vec && (e0 * sizeof(T)) % 16 == 0;
    if (a.bias && a.fits)                          // else a group's slots may lie past the biases'
        for (int e = threadIdx.x; e < E; e += kThreads) {
            const float b = a.bias[e];
            const int at = e / size * a.group_slots + e % size, j = at % lane_slots;
            reinterpret_cast<float*>(&biases[j / 4 * LPT + at / lane_slots])[j % 4] = b;
            atomicMax(&widest_bits, __float_as_uint(b) & 0x7fffffffu);    // of a NaN above infinity's
        }
    __syncthreads();
    // scores + bias lie in [-range, range), a power of two and not within a
    // part in 2^20 of its upper end: keys hold them times 2 / range, rounded
    const float widest = __uint_as_float(widest_bits);
    const bool fast = a.fits && widest < 0x1p20f;
    const float over_range = 2.0f / __uint_as_float((__float_as_uint((1.0f + widest) * 1.000001f) & 0x7f800000u) + 0x00800000u);
    const uint32_t by_score = a.softmax ? kMarginSoftmax : kMarginSigmoid;
    const uint32_t near = !by_logit ? (by_score + 1) << 9 : sizeof(T) == 2 ? 0u : 2u << 9;   // a key holds all of a bf16 logit
    const uint32_t over_k = (65536u + k - 1) / k;                 // i / k for i < 256
    // renormalised softmax weights of a choice by logits need no sum over the
    // row, and their largest logit is that of the first chosen
    const bool need_sum = a.softmax && (!a.renorm || !by_logit);

    const int tile = kTokens * a.reps;
    const long long stride = static_cast<long long>(gridDim.x) * kWarps * tile;
    long long t0 = (static_cast<long long>(blockIdx.x) * kWarps + warp) * tile;
    // this lane's next eight logits
    float x[8];
    const auto load = [&](long long t, int c) {
        const int left = t < a.tokens ? n - 8 * c : 0;
        if (fast) load_lane<8>(static_cast<const T*>(a.logits) + t * a.stride + e0 + 8 * c, min(left, 8), vec, 0.0f, x);
    };
    const auto routed = [&](long long t) { return t < a.tokens && (!a.mask || a.mask[t]); };
    bool next_on = routed(t0 + tl);
    load(t0 + tl, 0);
    for (; t0 < a.tokens; t0 += stride) {
        for (int rep = 0; rep < a.reps; ++rep) {
            const int slot = rep * kTokens + tl;                  // the token's place in the tile
            const long long next = rep + 1 < a.reps ? t0 + slot + kTokens : t0 + stride + tl;
            const bool on = next_on;
            next_on = routed(next);
            int32_t* sel = mem.sel + slot * k;
            bool again = on, reorder = false;                     // choose exactly; put into order exactly
            if (fast) {
                float top = 0.0f, sum = 1.0f, over = 1.0f;
                if (need_sum) {
                    const float2 stat = softmax_stat<LPT>(
                        static_cast<const T*>(a.logits) + (t0 + slot) * a.stride + e0, on ? n : 0, chunks, vec);
                    top = stat.x;
                    sum = stat.y;
                    over = __fdividef(1.0f, sum);
                }
                uint32_t head[8];                                 // this lane's best
                float zero = 0.0f;                                // NaN where a logit is not finite
#pragma unroll 1
                for (int c = 0; c < chunks; ++c) {
                    uint32_t key[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) zero = fmaf(x[j], 0.0f, zero);
                    const uint32_t place = kMaxExperts - 1 - e0 - 8 * c;
                    if (by_logit) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) key[j] = (order_bits(x[j]) & ~0x1ffu) | (place - j);
                    } else {
                        if (a.softmax) {
#pragma unroll
                            for (int j = 0; j < 8; ++j) x[j] = fast_exp(x[j] - top) * over;
                        } else {
#pragma unroll
                            for (int j = 0; j < 8; ++j) x[j] = fast_sigmoid(x[j]);
                        }
                        if (a.bias) {
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                const float4 b = biases[(2 * c + h) * LPT + l];
                                x[4 * h] += b.x; x[4 * h + 1] += b.y; x[4 * h + 2] += b.z; x[4 * h + 3] += b.w;
                            }
                        }
                        // [4, 8) is where fp32 has steps of 2^-21; the exponent is shifted out
#pragma unroll
                        for (int j = 0; j < 8; ++j) key[j] = __float_as_uint(fmaf(x[j], over_range, 6.0f)) * 512u + (place - j);
                    }
                    const int left = on ? n - 8 * c : 0;
                    if (left < 8) {
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            if (j >= left) key[j] = 0;
                    }
                    // the next eight are on their way while these are sorted
                    load(c + 1 < chunks ? t0 + slot : next, c + 1 < chunks ? c + 1 : 0);
                    sort8(key);
                    if (c == 0) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) head[j] = key[j];
                    } else {
                        merge8(head, key);
                    }
                }
                again = !(zero == 0.0f);

                if (a.top_groups < a.groups) {
                    uint32_t a1 = head[0] >> 9, a2 = head[1] >> 9;
                    for (int o = 1; o < group_lanes; o *= 2) {
                        const uint32_t b1 = __shfl_xor_sync(kAll, a1, o), b2 = __shfl_xor_sync(kAll, a2, o);
                        a2 = max(min(a1, b1), max(a2, b2));
                        a1 = max(a1, b1);
                    }
                    // lanes past the last group have none
                    uint32_t worth = g < a.groups ? (a1 + a2) << 5 | static_cast<uint32_t>(31 - g) : 0u;
                    // no two groups' worth is equal.  Over at most eight lanes each counts
                    // the better ones, whose shuffles need not wait for one another; over
                    // more the best are taken out in turn (65,536 tokens, 256 experts in
                    // 8 groups 33.6 / 34.9 us, 64 in 8 17.3 / 18.3)
                    bool stays = false, tie;
                    if constexpr (LPT <= 8) {
                        // a lane's rank: lanes of better groups; the last group that stays knows the next
                        int rank = 0;
                        uint32_t below = 0;
#pragma unroll
                        for (int o = 1; o < LPT; ++o) {
                            const uint32_t other = __shfl_xor_sync(kAll, worth, o);
                            if (other > worth) ++rank;
                            else if (other != worth) below = max(below, other);
                        }
                        const int staying = a.top_groups * group_lanes;
                        stays = rank < staying;
                        tie = rank + group_lanes == staying && (worth >> 5) - (below >> 5) < 2 * by_score;
                    } else {
                        uint32_t worst = 0;
                        for (int r = 0; r < a.top_groups; ++r) {
                            worst = token_max<LPT>(worth);
                            if (worth == worst) { worth = 0; stays = true; }
                        }
                        tie = (worst >> 5) - (token_max<LPT>(worth) >> 5) < 2 * by_score;
                    }
                    if (__any_sync(kAll, on && tie))
                        stays = groups_exact<LPT>(a, static_cast<const T*>(a.logits) + (t0 + slot) * a.stride, e0, on ? n : 0,
                                                  head[0], head[1], head[2], near, top, sum, g, group_lanes, size);
                    if (!stays) head[0] = 0;
                }

                // keys less than `near` apart may be of values less than the margin apart
                uint32_t last = 0xffffffffu, least = 0xffffffffu;
                const bool had = head[0] != 0;
                const auto pop = [&](uint32_t best) {
                    least = min(least, last - best);
                    last = best;
                    if (head[0] == best) {
#pragma unroll
                        for (int i = 0; i < 7; ++i) head[i] = head[i + 1];
                        head[7] = 0;
                    }
                };
#pragma unroll 2
                for (int r = 0; r < k; ++r) {
                    const uint32_t best = token_max<LPT>(head[0]);
                    if (l == 0) sel[r] = static_cast<int32_t>(best);
                    pop(best);
                }
                const uint32_t after = token_max<LPT>(head[0]);
                if (l == 0) mem.next[slot] = static_cast<int32_t>(after);
                least = min(least, last - after);
                if (on && !again && least < near) {
                    // which of the k + 1 best comes where is not certain; that they are it, mostly is
                    pop(after);
                    reorder = true;
                }
                if (__any_sync(kAll, reorder)) {
                    const uint32_t beyond = token_max<LPT>(head[0]);
                    if (reorder && (k == 32 || after - beyond < near)) again = true;
                }
                // a lane of more than eight experts may have had a ninth among the best
                again |= on && n > 8 && had && head[0] == 0;
                if (l == 0) mem.stat[slot] = Stat{top, sum, 0};
                again = again && on;
            } else if (!on) {
                for (int r = l; r < k; r += LPT) sel[r] = 0;
                if (l == 0) mem.stat[slot] = Stat{0.0f, 1.0f, 0};
            }
            const unsigned exactly = __ballot_sync(kAll, again);
            unsigned left = exactly | __ballot_sync(kAll, reorder);
            __syncwarp();
            while (left) {
                const int which = (__ffs(left) - 1) / LPT;
                const unsigned lanes = static_cast<unsigned>(((1ull << LPT) - 1) << (which * LPT));
                const int place = rep * kTokens + which;
                const T* row = static_cast<const T*>(a.logits) + (t0 + place) * a.stride;
                if (exactly & lanes) choose_exact(a, row, mem.c, mem.sel + place * k, mem.stat + place);
                else order_exact(a, row, mem.sel + place * k, mem.next[place], mem.stat[place]);
                left &= ~lanes;
            }
        }
        __syncwarp();
        // the slots' scores, and then the weights, a lane a slot
        const long long tokens = min(a.tokens - t0, static_cast<long long>(tile));
        const int slots = static_cast<int>(tokens) * k;
        for (int i = lane; i < slots; i += 32) {
            const int token = static_cast<int>(i * over_k >> 16), chosen = mem.sel[i];
            float score = 0.0f;
            int e = -1;
            if (chosen) {
                e = kMaxExperts - 1 - (chosen & (kMaxExperts - 1));
                const T* row = static_cast<const T*>(a.logits) + (t0 + token) * a.stride;
                const float x = widen(row[e]);
                Stat st = mem.stat[token];
                if (a.softmax && !need_sum) {
                    st.top = widen(row[kMaxExperts - 1 - (mem.sel[token * k] & (kMaxExperts - 1))]);
                    st.sum = 1.0f;
                }
                score = a.softmax ? __fdiv_rn(expf(x - st.top), st.sum) : sigmoid(x);
                if (a.counts) atomicAdd(hist + e, 1);
            }
            mem.score[i] = score;
            a.indices[t0 * k + i] = e;
        }
        __syncwarp();
        for (int i = lane; i < slots; i += 32) {
            const int token = static_cast<int>(i * over_k >> 16);
            float w = mem.score[i];
            if (a.renorm) {
                float total = 0.0f;
#pragma unroll 4
                for (int r = 0; r < k; ++r) total += mem.score[token * k + r];
                w = total > 0.0f ? __fdiv_rn(w, total) : 0.0f;
            }
            a.weights[t0 * k + i] = mem.stat[token].bad ? nan_value() : __fmul_rn(w, a.scale);
        }
        __syncwarp();
    }
    if (a.counts) {
        __syncthreads();
        for (int i = threadIdx.x; i < E; i += kThreads)
            if (hist[i]) atomicAdd(a.counts + i, hist[i]);
    }
}

// The gradient.  In the slots r, and with D their sum,
//   part_r = g_r w_r                            (weights as they are)
//   part_r = w_r (g_r - sum_l g_l w_l / scale)  (renormalised)
// sigmoid:  dx = part_r (1 - s_r) at the chosen, 0 elsewhere
// softmax:  dx = [chosen] part_r - s_i D; renormalised D is zero, and only the
//           chosen get a gradient
// GB300, 65,536 tokens over 256 experts, buffers in HBM: sigmoid in bf16 13.4 us,
// where 34 MB of gradient are written, 6 of slots read, and 26 as a sector or two
// for each slot's logit; softmax renormalised, which needs none, 7.6 us.  (Scores
// taken from the weights' ratios and one logit a token gave 11.3 us and gradients
// of confident experts that were off by percents at logits of 10 and could have
// the wrong sign at 15.)  Softmax not
// renormalised, 131,072 tokens over 128 experts in fp32, 28.4 us (5.2 TB/s): HBM,
// and the latency of a round's loads, sums and shared memory in turn.

constexpr int kRowBytes = 4096;          // of a warp's rows under construction

// Gradients that only the chosen get: the slots of row_tokens tokens at once,
// slot_lanes lanes a token; their values go into rows of zeros in shared
// memory, which leave in 16-byte stores and are cleared where they were set.
template <typename T>
__global__ void __launch_bounds__(kThreads)
route_backward_chosen_kernel(const __grid_constant__ RouteParams a) {
    __shared__ __align__(16) uint8_t buffer[kWarps][kRowBytes];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int E = a.E, k = a.k, lanes = a.slot_lanes;
    const int tl = lane / lanes, r = lane % lanes;
    T* const rows = reinterpret_cast<T*>(buffer[warp]);
    for (int i = lane; i < kRowBytes / 16; i += 32) reinterpret_cast<uint4*>(buffer[warp])[i] = make_uint4(0, 0, 0, 0);
    ddpk::dev::pdl_wait();
    ddpk::dev::pdl_trigger();
    __syncwarp();
    const int tile = a.row_tokens;
    for (long long t0 = (static_cast<long long>(blockIdx.x) * kWarps + warp) * tile; t0 < a.tokens;
         t0 += static_cast<long long>(gridDim.x) * kWarps * tile) {
        const long long t = t0 + tl;
        const int tokens = static_cast<int>(min(a.tokens - t0, static_cast<long long>(tile)));
        int index = -1;
        float w = 0.0f, g = 0.0f;
        if (tl < tokens && r < k) {
            index = a.indices[t * k + r];
            w = a.weights[t * k + r];
            g = a.grad_weights[t * k + r];
        }
        if (index < 0 || index >= E) { index = -1; w = g = 0.0f; }    // never an address past the row
        float part = g * w;
        if (a.renorm) {
            float total = part;
            for (int o = lanes / 2; o; o >>= 1) total += __shfl_xor_sync(kAll, total, o);
            part = w * (g - __fdiv_rn(total, a.scale));      // (1 / scale may be infinite)
        }
        // 1 - s = sigmoid(-x) from the slot's own logit: a difference would leave nothing of it where s is near 1
        if (!a.softmax && index >= 0) part *= sigmoid(-widen(static_cast<const T*>(a.logits)[t * a.stride + index]));
        if (index >= 0) rows[tl * E + index] = narrow<T>(part);
        __syncwarp();
        T* const to = static_cast<T*>(a.grad_logits) + t0 * a.grad_stride;
        if (a.vec) {
            const int pieces = tokens * E * static_cast<int>(sizeof(T)) / 16;
            for (int i = lane; i < pieces; i += 32)
                __stcs(reinterpret_cast<uint4*>(to) + i, reinterpret_cast<const uint4*>(rows)[i]);
        } else {
            for (int token = 0; token < tokens; ++token)
                for (int e = lane; e < E; e += 32) to[token * a.grad_stride + e] = rows[token * E + e];
        }
        __syncwarp();
        if (index >= 0) rows[tl * E + index] = narrow<T>(0.0f);
        __syncwarp();
    }
}

// Softmax weights as they are: every expert of a token gets a gradient.  The
// chosen experts' parts meet the lanes' experts in shared memory, laid out so
// that a lane's 16-byte accesses meet no other's banks (131,072 tokens over 128
// experts 28.4 us; a lane's experts next to one another 36.2).
template <int LPT, int EPL, typename T>
__global__ void __launch_bounds__(kThreads)
route_backward_whole_kernel(const __grid_constant__ RouteParams a) {
    constexpr int kTokens = 32 / LPT;
    // the chosen experts' parts, zeros elsewhere: a lane's c-th four at 32 c + lane
    __shared__ float4 rows[kWarps][8 * EPL];
    __shared__ float parts[kWarps][kMaxSlots];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int l = lane % LPT, tl = lane / LPT;
    const int E = a.E, k = a.k;
    float4* const row_part = rows[warp];
    float* const part = parts[warp];
    const int e0 = l * EPL, n = max(0, min(E - e0, EPL));
    const bool vec = a.vec && (e0 * sizeof(T)) % 16 == 0;
    const uint32_t over_k = (65536u + k - 1) / k;                 // i / k for i < 256
    for (int c = 0; c < EPL / 4; ++c) row_part[c * 32 + lane] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    ddpk::dev::pdl_wait();
    ddpk::dev::pdl_trigger();
    __syncwarp();
    for (long long t0 = (static_cast<long long>(blockIdx.x) * kWarps + warp) * kTokens; t0 < a.tokens;
         t0 += static_cast<long long>(gridDim.x) * kWarps * kTokens) {
        const long long t = t0 + tl;
        const bool on = t < a.tokens;
        const int slots = static_cast<int>(min(a.tokens - t0, static_cast<long long>(kTokens))) * k;
        float x[EPL];
        load_lane<EPL>(static_cast<const T*>(a.logits) + t * a.stride + e0, on ? n : 0, vec, neg_inf(), x);
        for (int i = lane; i < slots; i += 32) {
            const int index = a.indices[t0 * k + i];
            float p = 0.0f;
            if (index >= 0 && index < E) {
                p = a.grad_weights[t0 * k + i] * a.weights[t0 * k + i];
                const int at = static_cast<int>(i * over_k >> 16) * (LPT * EPL) + index;
                reinterpret_cast<float*>(row_part)[(at % EPL / 4 * 32 + at / EPL) * 4 + at % 4] = p;
            }
            part[i] = p;
        }
        float top = x[0], sum = 0.0f;
#pragma unroll
        for (int j = 1; j < EPL; ++j) top = fmaxf(top, x[j]);
#pragma unroll
        for (int o = LPT / 2; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, o));
        // the approximate exponential errs by 2^-22 and 2^-24 |x - top| of a score
#pragma unroll
        for (int j = 0; j < EPL; ++j) {
            x[j] = fast_exp(x[j] - top);
            sum += x[j];
        }
        sum = token_sum<LPT>(sum);
        __syncwarp();
        float total = 0.0f;
        if (on)
#pragma unroll 4
            for (int r = 0; r < k; ++r) total += part[tl * k + r];
        const float f = __fdividef(total, sum);
        T* const to = static_cast<T*>(a.grad_logits) + t * a.grad_stride + e0;
        float d[EPL];
#pragma unroll
        for (int c = 0; c < EPL / 4; ++c) {
            const float4 q = row_part[c * 32 + lane];
            row_part[c * 32 + lane] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            d[4 * c] = q.x; d[4 * c + 1] = q.y; d[4 * c + 2] = q.z; d[4 * c + 3] = q.w;
        }
        if (total != 0.0f) {                                      // a masked token's logits may be anything
#pragma unroll
            for (int j = 0; j < EPL; ++j) d[j] = fmaf(-x[j], f, d[j]);
        }
        if (on) store_lane<EPL>(to, n, vec, d);
        __syncwarp();
    }
}

template <typename K>
cudaError_t launch(K kernel, long long warps, int sms, int ctas_per_sm, const RouteParams& a, cudaStream_t stream) {
    const long long want = (warps + kWarps - 1) / kWarps, most = static_cast<long long>(ctas_per_sm) * sms;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(want < most ? want : most));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

// Of the current device, asked for once.
cudaError_t multiprocessors(int* sms) {
    static std::atomic<int> known[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    *sms = dev < 64 ? known[dev].load(std::memory_order_relaxed) : 0;
    if (*sms) return cudaSuccess;
    e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess && dev < 64) known[dev].store(*sms, std::memory_order_relaxed);
    return e;
}

int power_of_two(int x) {
    int p = 1;
    while (p < x) p *= 2;
    return p;
}

template <int LPT, typename T>
cudaError_t launch_forward(int sms, RouteParams& a, cudaStream_t stream) {
    constexpr int kTokens = 32 / LPT;
    const long long groups = (a.tokens + kTokens - 1) / kTokens;
    // with tokens enough for every warp, those of four rounds are weighed
    // together: their slots then fill the warp's lanes
    a.reps = kTokens < 4 && groups >= 4LL * kForwardCtas * sms * kWarps ? 4 / kTokens : 1;
    return launch(route_kernel<LPT, T>, (groups + a.reps - 1) / a.reps, sms, kForwardCtas, a, stream);
}

template <int LPT, int EPL, typename T>
cudaError_t launch_whole(int sms, const RouteParams& a, cudaStream_t stream) {
    constexpr int kTokens = 32 / LPT;
    return launch(route_backward_whole_kernel<LPT, EPL, T>, (a.tokens + kTokens - 1) / kTokens, sms, kWholeCtas, a, stream);
}

template <typename T>
cudaError_t launch_any(bool backward, RouteParams& a, cudaStream_t stream) {
    int sms = 0;
    const cudaError_t e = multiprocessors(&sms);
    if (e != cudaSuccess) return e;
    if (backward && !(a.softmax && !a.renorm)) {
        a.slot_lanes = power_of_two(a.k);
        const int room = kRowBytes / static_cast<int>(sizeof(T)) / a.E, tokens = 32 / a.slot_lanes;
        a.row_tokens = room < tokens ? room : tokens;
        return launch(route_backward_chosen_kernel<T>, (a.tokens + a.row_tokens - 1) / a.row_tokens, sms, kChosenCtas,
                      a, stream);
    }
    if (backward) {
        if (a.E > 256) return launch_whole<32, 16, T>(sms, a, stream);
        switch (power_of_two((a.E + 7) / 8)) {
            case 1: return launch_whole<1, 8, T>(sms, a, stream);
            case 2: return launch_whole<2, 8, T>(sms, a, stream);
            case 4: return launch_whole<4, 8, T>(sms, a, stream);
            case 8: return launch_whole<8, 8, T>(sms, a, stream);
            case 16: return launch_whole<16, 8, T>(sms, a, stream);
            default: return launch_whole<32, 8, T>(sms, a, stream);
        }
    }
    // slots of a group, each group from a lane of its own on
    const int size = a.E / a.groups;
    int lanes = 0;
    a.fits = 0;
    // Four chunks a lane put several tokens into a warp, which share its rounds
    // and its bookkeeping, for a longer chain of instructions: from about 2^20
    // logits on.  Against one, 65,536 tokens over 64 experts 10.3 / 15.6 us, 128
    // 17.2 / 27.8, 256 27.4 / 39.2, 512 49.3 / 54.0, over 256 in 8 groups 37.7 /
    // 47.1 (before the near ties of groups and their ranks took less); 2,048
    // tokens over 128 5.3 / 4.2, 256 over 256 in groups 6.4 / 4.5.
    for (a.chunks = a.tokens * a.E >= 1 << 20 ? 4 : 1; a.chunks; a.chunks /= 2) {
        const int mine = 8 * a.chunks;
        a.group_slots = power_of_two((size + mine - 1) / mine) * mine;
        lanes = power_of_two(a.groups * a.group_slots / mine);
        const int staying = a.top_groups * a.group_slots / mine;
        a.fits = lanes <= 32 && lanes * mine <= kMaxExperts;
        // more chunks while they waste no lanes, the slots fit, and more than
        // eight of a token's best in one lane stay rare
        if (a.chunks == 1 || (a.fits && a.groups * a.group_slots <= a.E + a.E / 2 && 32 / lanes * a.k <= kMaxSlots &&
                              (a.k < 8 || a.k <= 2 * staying)))
            break;
    }
    if (!a.fits) {
        // 256 slots are not enough for one chunk a lane: two
        a.chunks = 2;
        a.group_slots = power_of_two((size + 15) / 16) * 16;
        lanes = 32;
        a.fits = a.groups * a.group_slots <= kMaxExperts;
        if (!a.fits) a.group_slots = kMaxExperts;    // every token is chosen exactly: one a warp
    }
    switch (lanes) {
        case 1: return launch_forward<1, T>(sms, a, stream);
        case 2: return launch_forward<2, T>(sms, a, stream);
        case 4: return launch_forward<4, T>(sms, a, stream);
        case 8: return launch_forward<8, T>(sms, a, stream);
        case 16: return launch_forward<16, T>(sms, a, stream);
        default: return launch_forward<32, T>(sms, a, stream);
    }
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
    const int64_t size = x->dtype == DDP_F32 ? 4 : 2;
    a.vec = aligned(logits, 16) && x->row_stride * size % 16 == 0;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = x->dtype == DDP_F32 ? launch_any<float>(false, a, st) : launch_any<uint16_t>(false, a, st);
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
    const int64_t bytes = static_cast<int64_t>(size);
    if (a.softmax && !a.renorm)
        a.vec = aligned(logits, 16) && x->row_stride * bytes % 16 == 0 && aligned(grad_logits, 16) &&
                grad_stride * bytes % 16 == 0;
    else
        a.vec = aligned(grad_logits, 16) && grad_stride == x->experts && x->experts * bytes % 16 == 0;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = x->dtype == DDP_F32 ? launch_any<float>(true, a, st) : launch_any<uint16_t>(true, a, st);
    return e == cudaSuccess ? DDP_OK : DDP_ERR_CUDA;
}

}  // extern "C"
