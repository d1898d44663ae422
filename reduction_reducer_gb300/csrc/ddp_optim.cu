// The optimizer step behind the gradient path: AdamW over every parameter in
// one launch (moments in 32 or in 8 bits), and the global gradient norm it
// clips by.
//
// Both kernels see the tensors as blocks of 256 elements (a tensor's last may
// be short), and up to kMaxRun consecutive blocks of a tensor as a run, numbered
// through all non-empty tensors in registration order.  A CTA owns an equal
// share of the runs, its warps take them in turn, and a warp finds its first
// run's tensor with the warp-ballot search over the tensors' first runs; so one
// launch serves any mix of large matrices and small vectors.  Runs of eight
// blocks let a warp read and write an 8-bit moment's scales as whole 32-byte
// sectors.  Within a block lane l holds elements
// 4 l .. 4 l + 3 and 128 + 4 l .. 128 + 4 l + 3: every 128-bit access of a
// warp covers 512 consecutive bytes, and an 8-bit moment's block, whose scale
// needs the largest magnitude of all 256 values, is one warp's registers.

#include "ddp_reducer.h"

#include <cuda_runtime.h>

#include <cfloat>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>
#include <string>
#include <type_traits>
#include <vector>

#include "ddp_device.cuh"

namespace {

constexpr int kBlock = DDP_ADAMW_BLOCK;
constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kNormThreads = 512;
constexpr int kMaxRun = 8;                // blocks
static_assert(kBlock == 256, "a warp holds a block as 8 values a lane");

// One non-empty tensor, as the kernels read it.
struct __align__(16) Tensor {
    const float* g;
    void* p;            // parameter: fp32, or bf16
    float* master;      // fp32 master copy of a bf16 parameter
    void* m;            // moments: fp32, or e4m3 / e5m2 codes
    void* v;
    float* ms;          // scales of 8-bit moments, one per block
    float* vs;
    long long n;
    long long block0;   // number of its first block among all tensors'
    float wd;
    int var;            // its index among all tensors
    int vec_g;          // gradients: 16-byte aligned
    int vec;            // all others: 16-byte aligned (bf16 parameters 8)
};

struct Scalars {
    float beta1, beta1c, beta2, beta2c;   // betas and 1 - beta
    float lr, step;                       // step = lr / (1 - beta1^t)
    float rbc2;                           // 1 / sqrt(1 - beta2^t)
    float eps, max_norm;
    uint32_t seed_lo, seed_hi;
    int clip, skip_nonfinite;
    float one;
};

struct StepParams {
    const Tensor* tensors;
    const long long* first;    // [S + 1] first run of each tensor
    const float* norm;
    const uint8_t* used;
    long long runs, piece;     // all runs; runs per CTA
    int S;
    int run;                   // blocks of a run
    Scalars c;
};

// ------------------------------------------------------------------ four values

// Whole: four values by one access.  Else value i where i < left (left may be
// negative), past it nothing is read and zeros are given.
__device__ __forceinline__ void load4(const float* p, bool whole, int left, float (&f)[4]) {
    if (whole) {
        const float4 x = __ldcs(reinterpret_cast<const float4*>(p));
        f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = i < left ? p[i] : 0.0f;
    }
}

__device__ __forceinline__ void store4(float* p, bool whole, int left, const float (&f)[4]) {
    if (whole) {
        __stcs(reinterpret_cast<float4*>(p), make_float4(f[0], f[1], f[2], f[3]));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < left) p[i] = f[i];
    }
}

__device__ __forceinline__ uint32_t load4(const uint8_t* p, bool whole, int left) {
    if (whole) return __ldcs(reinterpret_cast<const uint32_t*>(p));
    uint32_t x = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (i < left) x |= static_cast<uint32_t>(p[i]) << (8 * i);
    return x;
}

__device__ __forceinline__ void store4(uint8_t* p, bool whole, int left, uint32_t x) {
    if (whole) {
        __stcs(reinterpret_cast<uint32_t*>(p), x);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < left) p[i] = static_cast<uint8_t>(x >> (8 * i));
    }
}

// Two fp32 -> two bf16, round to nearest even, the first in the low half.
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    uint32_t x;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(x) : "f"(hi), "f"(lo));
    return x;
}

__device__ __forceinline__ void store4(uint16_t* p, bool whole, int left, const float (&f)[4]) {
    const uint32_t x[2] = {bf16_pair(f[0], f[1]), bf16_pair(f[2], f[3])};
    if (whole) {
        __stcs(reinterpret_cast<uint2*>(p), make_uint2(x[0], x[1]));
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < left) p[i] = static_cast<uint16_t>(x[i / 2] >> (16 * (i % 2)));
    }
}

// ------------------------------------------------------------------ two values

// Packed fp32 instructions.
__device__ __forceinline__ uint64_t bits2(float2 x) { return *reinterpret_cast<uint64_t*>(&x); }
__device__ __forceinline__ float2 from2(uint64_t x) { return *reinterpret_cast<float2*>(&x); }
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    uint64_t x;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(x) : "l"(bits2(a)), "l"(bits2(b)));
    return from2(x);
}

__device__ __forceinline__ float2 mul2_down(float2 a, float2 b) {      // toward zero
    uint64_t x;
    asm("mul.rz.f32x2 %0, %1, %2;" : "=l"(x) : "l"(bits2(a)), "l"(bits2(b)));
    return from2(x);
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    uint64_t x;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(x) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
    return from2(x);
}

// ------------------------------------------------------------------ 8-bit moments

// Four e4m3 codes -> their values, by way of fp16, which holds them exactly.
__device__ __forceinline__ void e4m3_values(uint32_t c, float (&f)[4]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        asm("{\n\t.reg .b16 c, a, b;\n\t.reg .b32 p;\n\t"
            "cvt.u16.u32 c, %2;\n\tcvt.rn.f16x2.e4m3x2 p, c;\n\tmov.b32 {a, b}, p;\n\t"
            "cvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
            : "=f"(f[2 * h]), "=f"(f[2 * h + 1]) : "r"(c >> (16 * h)));
    }
}

// Four e5m2 codes -> their values: a code is the upper byte of an fp16.
__device__ __forceinline__ void e5m2_values(uint32_t c, float (&f)[4]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.f32.f16 %0, a;\n\tcvt.f32.f16 %1, b;\n\t}"
            : "=f"(f[2 * h]), "=f"(f[2 * h + 1]) : "r"(__byte_perm(c, 0, h ? 0x3424 : 0x1404)));
    }
}

// Two codes' upper bits from y = x / scale and two hashes: an fp32 number
// times 2^-120 (2^-112) has the sign, the exponent field and, below 2^-126,
// the subnormal spacing of e4m3 (e5m2); cutting that product down instead of
// rounding it leaves the digits as they are.  Random bits added to the dropped
// digits, all below the kept ones, carry with the probability of the rest.
// The code is then in bits 20 (21) and up, the sign in bit 31.
__device__ __forceinline__ void e4m3_round(float2 y, uint32_t r0, uint32_t r1, uint32_t& x0, uint32_t& x1) {
    const float2 z = mul2_down(y, make_float2(0x1p-120f, 0x1p-120f));
    x0 = __float_as_uint(z.x) + (r0 >> 16 << 4);
    x1 = __float_as_uint(z.y) + (r1 >> 16 << 4);
}

__device__ __forceinline__ void e5m2_round(float2 y, uint32_t r0, uint32_t r1, uint32_t& x0, uint32_t& x1) {
    const float2 z = mul2_down(y, make_float2(0x1p-112f, 0x1p-112f));
    x0 = __float_as_uint(z.x) + ((r0 & 0xffffu) << 5);
    x1 = __float_as_uint(z.y) + ((r1 & 0xffffu) << 5);
}

// The low bytes of four words.
__device__ __forceinline__ uint32_t low_bytes(const uint32_t (&x)[4]) {
    return __byte_perm(__byte_perm(x[0], x[1], 0x0040), __byte_perm(x[2], x[3], 0x0040), 0x5410);
}

// Four e4m3 codes with their signs.  The block's largest value can come out an
// ulp above 448 and then carry into the NaN code, one up.
__device__ __forceinline__ uint32_t e4m3_pack(const uint32_t (&x)[4]) {
    const uint32_t k[4] = {x[0] >> 20, x[1] >> 20, x[2] >> 20, x[3] >> 20};
    uint32_t c = low_bytes(k) & 0x7f7f7f7fu;
    c -= (c + 0x01010101u & 0x80808080u) >> 7;
    const uint32_t sign = __byte_perm(__byte_perm(x[0], x[1], 0x0073), __byte_perm(x[2], x[3], 0x0073), 0x5410);
    return c | (sign & 0x80808080u);
}

// Four e5m2 codes of numbers that are not negative.  `any`: the numbers' bits;
// one that is not zero gets no zero code (m / (sqrt(v) + eps) must not meet a
// v rounded to zero).
__device__ __forceinline__ uint32_t e5m2_pack(const uint32_t (&x)[4], const uint32_t (&any)[4]) {
    uint32_t k[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) k[q] = max(x[q] >> 21, min(any[q], 1u));
    uint32_t c = low_bytes(k);
    return c - ((c + 0x04040404u & 0x80808080u) >> 7);
}

// Largest magnitude, NaN above all.
__device__ __forceinline__ float peak(float a, float b) {
    float x;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(x) : "f"(a), "f"(fabsf(b)));
    return x;
}

// The scale of a block from a lane's largest magnitude: magnitudes compare as
// their bits, NaN above infinity.  A normal number, so that its reciprocal is
// one: blocks of less than 2^-126 times the format's top lie on the codes below it.
__device__ __forceinline__ float block_scale(float mine, float over_top) {
    const uint32_t most = __reduce_max_sync(0xffffffffu, __float_as_uint(mine));
    const float s = __fmul_rn(__uint_as_float(most), over_top);
    if (!(s < __int_as_float(0x7f800000))) return __int_as_float(0x7fffffff);
    return most ? fmaxf(s, 0x1p-126f) : 0.0f;
}

// 32 random bits of (seed, block, place): odd multipliers from the fractional
// bits of sqrt(2) and sqrt(3), places spread by the golden ratio's.
__device__ __forceinline__ uint32_t mix(uint32_t x) {
    x ^= x >> 16;
    x *= 0x6A09E667u;
    x ^= x >> 15;
    x *= 0xBB67AE85u;
    return x ^ (x >> 16);
}

__device__ __forceinline__ uint32_t block_key(const Scalars& c, long long block) {
    return mix(mix(static_cast<uint32_t>(block) ^ c.seed_lo) + c.seed_hi);
}

__device__ __forceinline__ uint32_t random_bits(uint32_t key, uint32_t place) { return mix(key + place * 0x9E3779B9u); }

// ------------------------------------------------------------------ the step

// Products and sums are rounded one by one: the stored moments, and with them
// the 8-bit codes, are then those of the formula's own order of fp32
// operations.  A packed product and a packed sum are contracted by the
// assembler whatever their rounding modes say, a sum as a multiple of `one`,
// which only the host knows to be 1, is not.
__device__ __forceinline__ void moments(const Scalars& c, float2 g, float2& m, float2& v) {
    m = fma2(mul2(m, both(c.beta1)), both(c.one), mul2(g, both(c.beta1c)));
    v = fma2(mul2(v, both(c.beta2)), both(c.one), mul2(mul2(g, g), both(c.beta2c)));
}

// The hardware's root and reciprocal (1 ulp each): w' is rounded to far less
// than the 2^-24 of w that an update of lr w can show.  A v below 2^-126, which
// gradients below 3e-18 give, is taken for what it is: with SMALL, where no v is
// above 2^100, the flushing root of 2^24 v (rbc2 is then over 2^12), else the
// root that does not flush, of three more instructions (8-bit moments, 100 M
// elements 236.5 / 239.2 us; 32-bit ones wait for HBM: 399 with either).  A
// denominator is at least eps, a normal number, and past 2^126, where the
// reciprocal would be subnormal, only with such an eps: no update then.
template <bool SMALL>
__device__ __forceinline__ float2 weight(const Scalars& c, float keep, float2 w, float2 m, float2 v) {
    float2 root, over, denom;
    if constexpr (SMALL) {
        v = mul2(v, both(0x1p24f));
        asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(root.x) : "f"(v.x));
        asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(root.y) : "f"(v.y));
        denom = fma2(root, both(c.rbc2 * 0x1p-12f), both(c.eps));
    } else {
        asm("sqrt.approx.f32 %0, %1;" : "=f"(root.x) : "f"(v.x));
        asm("sqrt.approx.f32 %0, %1;" : "=f"(root.y) : "f"(v.y));
        denom = fma2(root, both(c.rbc2), both(c.eps));
    }
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(over.x) : "f"(denom.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(over.y) : "f"(denom.y));
    return fma2(mul2(m, both(-c.step)), over, mul2(w, both(keep)));
}

// 16 bytes from global to shared memory, asynchronously.
__device__ __forceinline__ void copy16(void* to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                 :: "r"(static_cast<uint32_t>(__cvta_generic_to_shared(to))), "l"(from) : "memory");
}

__device__ __forceinline__ void copy4(void* to, const void* from) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;"
                 :: "r"(static_cast<uint32_t>(__cvta_generic_to_shared(to))), "l"(from) : "memory");
}

// A block's inputs on their way to a warp.
struct __align__(16) Stage {
    float g[kBlock], w[kBlock];
    uint8_t m[kBlock], v[kBlock];
};

// Bound by HBM: an element moves 28 bytes with 32-bit moments (weight and both
// moments read and written, gradient read), 30 with bf16 weights beside their
// master copies, 16 and 18 with 8-bit ones.  GB300, copy peak 6,780 GB/s:
// BERT-large (335 M elements) 1,342 us, 6,990 GB/s; GPT-2-medium with bf16
// weights 1,528 us, 6,970 GB/s, and with 8-bit moments 962 us, 6,660 GB/s;
// ResNet-50 103 us, 6,930 GB/s.
//
// 32-bit moments: eight 128-bit loads a lane in flight on 24 or 28 warps an SM
// carry it; single blocks to a warp, its neighbours on the next ones.  8-bit moments
// take about 77 instructions an element, so a warp's loads must run while it
// computes: its next whole block is copied to shared memory meanwhile (without
// the copy, and with a scale a block read and written by itself, GPT-2-medium
// took 1,217 us; the scales as whole sectors were most of the difference).
template <bool BF16, bool Q8>
__global__ void __launch_bounds__(kThreads)
adamw_kernel(const __grid_constant__ StepParams a) {
    __shared__ Stage stages[Q8 ? kWarps : 1][2];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long begin = static_cast<long long>(blockIdx.x) * a.piece;
    const long long end = min(begin + a.piece, a.runs);
    long long u = begin + warp;
    int s = u < end ? ddpk::dev::find_segment(a.first, 0, a.S, u) : 0;   // the library's own table: before the wait
    ddpk::dev::pdl_wait();
    ddpk::dev::pdl_trigger();

    // the next run from u on of a tensor that has a gradient
    const auto settle = [&](long long& u, int& s) {
        for (; u < end; u += kWarps) {
            while (u >= __ldg(a.first + s + 1)) ++s;
            if (!a.used || a.used[a.tensors[s].var]) break;
        }
    };
    // block j of tensor s on its way, where it is whole
    const auto fetch = [&](const Tensor& t, long long j, Stage& to) {
        const long long at = j * kBlock;
        if (t.vec && t.n - at >= kBlock) {
            const float* w = (BF16 ? t.master : static_cast<float*>(t.p)) + at + 4 * lane;
            copy16(to.w + 4 * lane, w);
            copy16(to.w + 4 * lane + 128, w + 128);
            if (t.vec_g) {
                copy16(to.g + 4 * lane, t.g + at + 4 * lane);
                copy16(to.g + 4 * lane + 128, t.g + at + 4 * lane + 128);
            } else {        // bucket views start anywhere
#pragma unroll
                for (int i = 0; i < kBlock; i += 32) copy4(to.g + i + lane, t.g + at + i + lane);
            }
            const int c = 16 * (lane & 15);
            if (lane < 16) copy16(to.m + c, static_cast<const uint8_t*>(t.m) + at + c);
            else copy16(to.v + c, static_cast<const uint8_t*>(t.v) + at + c);
        }
    };
    // lanes r and 8 + r: the scales of block r of a run of `blocks`
    const auto scale_at = [&](const Tensor& t, long long j0, int blocks) -> float* {
        const int r = lane % kMaxRun;
        return lane < 2 * kMaxRun && r < blocks ? (lane < kMaxRun ? t.ms : t.vs) + j0 + r : nullptr;
    };
    const auto blocks_of = [&](const Tensor& t, long long j0) {
        return static_cast<int>(min((t.n + kBlock - 1) / kBlock - j0, static_cast<long long>(a.run)));
    };

    settle(u, s);
    int stage = 0;
    float next_scale = 0.0f;
    if (Q8 && u < end) {
        const Tensor& t = a.tensors[s];
        const long long j0 = (u - __ldg(a.first + s)) * a.run;
        fetch(t, j0, stages[warp][0]);
        if (const float* x = scale_at(t, j0, blocks_of(t, j0))) next_scale = *x;
        asm volatile("cp.async.commit_group;" ::: "memory");
    }

    // (after the first inputs are on their way, which do not wait for it)
    float clip = 1.0f;
    if (a.norm) {
        const float norm = *a.norm;
        if (a.c.skip_nonfinite && !(norm < __int_as_float(0x7f800000))) {
            if constexpr (Q8) asm volatile("cp.async.wait_all;" ::: "memory");
            return;
        }
        if (a.c.clip) {
            const float x = __fdiv_rn(a.c.max_norm, __fadd_rn(norm, 1e-6f));
            clip = x > 1.0f ? 1.0f : x;        // a NaN stays one
        }
    }

    while (u < end) {
        // an entry in registers is not read again after every store; with 8-bit
        // moments there are none left for it (GPT-2-medium, by value / by
        // reference: 1,529 / 1,543 us, 8-bit 973 / 958)
        typename std::conditional<Q8, const Tensor&, const Tensor>::type t = a.tensors[s];
        const long long j0 = (u - __ldg(a.first + s)) * a.run;
        const int blocks = blocks_of(t, j0);
        long long next_u = u + kWarps;
        int next_s = s;
        settle(next_u, next_s);
        float scale = next_scale;
        for (int r = 0; r < blocks; ++r) {
            const long long j = j0 + r;
            if constexpr (Q8) {
                if (r + 1 < blocks) {
                    fetch(t, j + 1, stages[warp][stage ^ 1]);
                } else if (next_u < end) {
                    const Tensor& to = a.tensors[next_s];
                    const long long to_j = (next_u - __ldg(a.first + next_s)) * a.run;
                    fetch(to, to_j, stages[warp][stage ^ 1]);
                    if (const float* x = scale_at(to, to_j, blocks_of(to, to_j))) next_scale = *x;
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
            }
            const int left = static_cast<int>(min(t.n - j * kBlock, static_cast<long long>(kBlock)));
            const bool whole = t.vec && left == kBlock, whole_g = t.vec_g && left == kBlock;
            const float keep = __fsub_rn(1.0f, __fmul_rn(a.c.lr, t.wd));
            const long long i = j * kBlock + 4 * lane;       // this lane's first element, and how many are left from it
            const int more = left - 4 * lane;
            const float* const g_ptr = t.g + i;
            float* const w_ptr = (BF16 ? t.master : static_cast<float*>(t.p)) + i;
            using State = typename std::conditional<Q8, uint8_t, float>::type;
            State* const m_ptr = static_cast<State*>(t.m) + i;
            State* const v_ptr = static_cast<State*>(t.v) + i;
            float g[2][4], w[2][4], m[2][4], v[2][4];
            uint32_t mc[2], vc[2];
            float ms = 0.0f, vs = 0.0f;
            if constexpr (Q8) {
                ms = __shfl_sync(0xffffffffu, scale, r);
                vs = __shfl_sync(0xffffffffu, scale, kMaxRun + r);
                asm volatile("cp.async.wait_group 1;" ::: "memory");
                __syncwarp();
                const Stage& in = stages[warp][stage];
                stage ^= 1;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int e = 4 * lane + 128 * h;
                    if (whole) {
                        const float4 x = *reinterpret_cast<const float4*>(in.w + e);
                        w[h][0] = x.x; w[h][1] = x.y; w[h][2] = x.z; w[h][3] = x.w;
                        mc[h] = *reinterpret_cast<const uint32_t*>(in.m + e);
                        vc[h] = *reinterpret_cast<const uint32_t*>(in.v + e);
                    } else {
                        load4(w_ptr + 128 * h, false, more - 128 * h, w[h]);
                        mc[h] = load4(m_ptr + 128 * h, false, more - 128 * h);
                        vc[h] = load4(v_ptr + 128 * h, false, more - 128 * h);
                    }
                    if (whole) {
                        const float4 x = *reinterpret_cast<const float4*>(in.g + e);
                        g[h][0] = x.x; g[h][1] = x.y; g[h][2] = x.z; g[h][3] = x.w;
                    } else {
                        load4(g_ptr + 128 * h, whole_g, more - 128 * h, g[h]);
                    }
                    e4m3_values(mc[h], m[h]);
                    e5m2_values(vc[h], v[h]);
                }
                __syncwarp();
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    load4(g_ptr + 128 * h, whole_g, more - 128 * h, g[h]);
                    load4(w_ptr + 128 * h, whole, more - 128 * h, w[h]);
                    load4(m_ptr + 128 * h, whole, more - 128 * h, m[h]);
                    load4(v_ptr + 128 * h, whole, more - 128 * h, v[h]);
                }
            }
            float peak_m = 0.0f, peak_v = 0.0f;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int q = 0; q < 4; q += 2) {
                    float2 mm = make_float2(m[h][q], m[h][q + 1]), vv = make_float2(v[h][q], v[h][q + 1]);
                    if constexpr (Q8) {
                        mm = mul2(mm, both(ms));
                        vv = mul2(vv, both(vs));
                    }
                    moments(a.c, mul2(make_float2(g[h][q], g[h][q + 1]), both(clip)), mm, vv);
                    m[h][q] = mm.x; m[h][q + 1] = mm.y;
                    v[h][q] = vv.x; v[h][q + 1] = vv.y;
                    if constexpr (Q8) {     // past the tensor's end both moments are zero
                        peak_m = peak(peak(peak_m, mm.x), mm.y);
                        peak_v = peak(peak(peak_v, vv.x), vv.y);
                    }
                }
            const auto weights = [&](auto small) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int q = 0; q < 4; q += 2) {
                        const float2 x = weight<decltype(small)::value>(
                            a.c, keep, make_float2(w[h][q], w[h][q + 1]), make_float2(m[h][q], m[h][q + 1]),
                            make_float2(v[h][q], v[h][q + 1]));
                        w[h][q] = x.x; w[h][q + 1] = x.y;
                    }
            };
            if (Q8 && peak_v <= 0x1p100f) weights(std::true_type());
            else weights(std::false_type());
            if constexpr (Q8) {
                ms = block_scale(peak_m, 1.0f / 448.0f);
                vs = block_scale(peak_v, 1.0f / 57344.0f);
                const float mi = ms > 0.0f ? __fdiv_rn(1.0f, ms) : 0.0f;
                const float vi = vs > 0.0f ? __fdiv_rn(1.0f, vs) : 0.0f;
                const uint32_t key = block_key(a.c, t.block0 + j) + static_cast<uint32_t>(4 * lane) * 0x9E3779B9u;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t x[4], y[4], any[4];
#pragma unroll
                    for (int q = 0; q < 4; q += 2) {
                        const uint32_t r0 = random_bits(key, 128 * h + q), r1 = random_bits(key, 128 * h + q + 1);
                        const float2 vy = mul2(make_float2(v[h][q], v[h][q + 1]), both(vi));
                        e4m3_round(mul2(make_float2(m[h][q], m[h][q + 1]), both(mi)), r0, r1, x[q], x[q + 1]);
                        e5m2_round(vy, r0, r1, y[q], y[q + 1]);
                        any[q] = __float_as_uint(v[h][q]);            // vy can be zero beside a huge v
                        any[q + 1] = __float_as_uint(v[h][q + 1]);
                    }
                    mc[h] = ms >= 0.0f ? e4m3_pack(x) : 0u;      // a block of NaN holds zeros and a NaN scale
                    vc[h] = vs >= 0.0f ? e5m2_pack(y, any) : 0u;
                }
                if (lane == r) scale = ms;
                if (lane == kMaxRun + r) scale = vs;
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                store4(w_ptr + 128 * h, whole, more - 128 * h, w[h]);
                if constexpr (BF16) store4(static_cast<uint16_t*>(t.p) + i + 128 * h, whole, more - 128 * h, w[h]);
                if constexpr (Q8) {
                    store4(m_ptr + 128 * h, whole, more - 128 * h, mc[h]);
                    store4(v_ptr + 128 * h, whole, more - 128 * h, vc[h]);
                } else {
                    store4(m_ptr + 128 * h, whole, more - 128 * h, m[h]);
                    store4(v_ptr + 128 * h, whole, more - 128 * h, v[h]);
                }
            }
        }
        if constexpr (Q8)
            if (float* x = scale_at(t, j0, blocks)) *x = scale;
        u = next_u;
        s = next_s;
    }
}

// ------------------------------------------------------------------ the norm

// A sum in two fp32 numbers: hi the rounded sum, lo what the roundings left out
// (exactly, per addition), about 46 bits together.  GB300 has two double lanes
// an SM: with doubles the warps' and CTAs' sums alone took 2 us of a norm.
struct Sum {
    float hi, lo;
};

struct NormParams {
    const Tensor* tensors;
    const long long* first;
    const uint8_t* used;
    Sum* partial;              // [grid]
    unsigned* done;            // CTAs finished; wraps to 0
    float* norm;
    long long runs, piece;
    int S;
    int run;
};

__device__ __forceinline__ Sum plus(const Sum& a, const Sum& b) {
    const float s = __fadd_rn(a.hi, b.hi), t = __fsub_rn(s, a.hi);
    const float rest = __fadd_rn(__fsub_rn(a.hi, __fsub_rn(s, t)), __fsub_rn(b.hi, t));
    return Sum{s, __fadd_rn(__fadd_rn(a.lo, b.lo), rest)};
}

__device__ __forceinline__ Sum warp_sum(Sum x) {
#pragma unroll
    for (int o = 16; o; o >>= 1)
        x = plus(x, Sum{__shfl_xor_sync(0xffffffffu, x.hi, o), __shfl_xor_sync(0xffffffffu, x.lo, o)});
    return x;
}

// All threads' sum, in every thread of the first warp.
__device__ __forceinline__ Sum cta_sum(Sum x, Sum* smem) {
    x = warp_sum(x);
    const int lane = threadIdx.x & 31;
    if (lane == 0) smem[threadIdx.x >> 5] = x;
    __syncthreads();
    return threadIdx.x < 32 ? warp_sum(lane < kNormThreads / 32 ? smem[lane] : Sum{0.0f, 0.0f}) : Sum{0.0f, 0.0f};
}

// An infinite hi has a lo that is no number.
__device__ __forceinline__ float root(const Sum& x) {
    return isfinite(x.hi) ? static_cast<float>(sqrt(static_cast<double>(x.hi) + static_cast<double>(x.lo))) : sqrtf(x.hi);
}

// Reads 4 bytes an element and nothing else of size.  Eight 128-bit loads a
// lane in flight; a lane's squares of a run (at most 68) are fp32 sums, runs
// and CTAs are added in two fp32 numbers, partial sums in an order that does not
// depend on which CTA comes last.  GB300: BERT-large 192 us, 6,970 GB/s (a
// read-only torch sum streams at 6,435 to 6,570); ResNet-50 20 us and 1 M
// elements 5.4 us, of which 2 are an empty launch's.  CTAs of 512 threads: as
// many as fit finish together and count at one address (BERT-large, 128 / 256 /
// 512 threads 202 / 195 / 192 us).
__global__ void __launch_bounds__(kNormThreads)
norm_kernel(const __grid_constant__ NormParams a) {
    __shared__ Sum smem[kNormThreads / 32];
    __shared__ bool last;
    const int lane = threadIdx.x & 31;
    const long long begin = static_cast<long long>(blockIdx.x) * a.piece;
    const long long end = min(begin + a.piece, a.runs);
    long long u = begin + (threadIdx.x >> 5);
    int s = u < end ? ddpk::dev::find_segment(a.first, 0, a.S, u) : 0;
    ddpk::dev::pdl_wait();
    ddpk::dev::pdl_trigger();

    Sum sum{0.0f, 0.0f};
    for (; u < end; u += kNormThreads / 32) {
        while (u >= __ldg(a.first + s + 1)) ++s;
        const Tensor& t = a.tensors[s];
        if (a.used && !a.used[t.var]) continue;
        const long long at = (u - __ldg(a.first + s)) * a.run * kBlock;
        const int n = static_cast<int>(min(t.n - at, static_cast<long long>(a.run) * kBlock));
        const float* const g = t.g + at;
        // up to three elements on either side of the 16-byte aligned ones
        const int head = min(n, static_cast<int>(-(reinterpret_cast<uintptr_t>(g) >> 2) & 3));
        const int vectors = (n - head) / 4, tail = n - head - 4 * vectors;
        const float4* const v = reinterpret_cast<const float4*>(g + head);
        // a lane's squares of a run: at most 68, in four fp32 sums
        float part[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        const auto add = [&](const float4& x) {
            part[0] = __fmaf_rn(x.x, x.x, part[0]);
            part[1] = __fmaf_rn(x.y, x.y, part[1]);
            part[2] = __fmaf_rn(x.z, x.z, part[2]);
            part[3] = __fmaf_rn(x.w, x.w, part[3]);
        };
        int i = lane;
        for (; i + 7 * 32 < vectors; i += 8 * 32) {
            float4 x[8];
#pragma unroll
            for (int h = 0; h < 8; ++h) x[h] = ddpk::dev::ld_stream(v + i + 32 * h);
#pragma unroll
            for (int h = 0; h < 8; ++h) add(x[h]);
        }
#pragma unroll 4
        for (; i < vectors; i += 32) add(ddpk::dev::ld_stream(v + i));
        if (lane < head + tail) {
            const float x = lane < head ? g[lane] : g[n - tail + lane - head];
            part[0] = __fmaf_rn(x, x, part[0]);
        }
        sum = plus(sum, Sum{(part[0] + part[1]) + (part[2] + part[3]), 0.0f});
    }
    const Sum total = cta_sum(sum, smem);
    if (gridDim.x == 1) {
        if (threadIdx.x == 0) *a.norm = root(total);
        return;
    }
    if (threadIdx.x == 0) {
        a.partial[blockIdx.x] = total;
        __threadfence();
        last = atomicInc(a.done, gridDim.x - 1) == gridDim.x - 1;
        __threadfence();
    }
    __syncthreads();
    if (!last) return;
    // the CTA that finishes last adds the partial sums, in an order of their own
    Sum x{0.0f, 0.0f};
    for (unsigned i = threadIdx.x; i < gridDim.x; i += kNormThreads) {
        const float2 y = __ldcg(reinterpret_cast<const float2*>(a.partial + i));
        x = plus(x, Sum{y.x, y.y});
    }
    __syncthreads();
    const Sum all = cta_sum(x, smem);
    if (threadIdx.x == 0) *a.norm = root(all);
}

template <typename K, typename P>
cudaError_t launch(K kernel, int threads, int grid, const P& params, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, params);
}

// How a kernel cuts the tensors into runs of at most `run` blocks.
struct Runs {
    int run = 1;
    int64_t count = 0;
    const long long* first = nullptr;    // device [S + 1]
};

thread_local std::string g_create_error;

}  // namespace

struct ddp_adamw {
    std::vector<int64_t> numel;
    bool bf16 = false;
    bool q8 = false;
    // binding
    int device = -1;
    int sms = 0;
    bool has_params = false;
    bool bound = false;
    int S = 0;
    Runs step, norm;
    void* table = nullptr;       // device: Tensor[S], first[S + 1], partial[], done
    const Tensor* tensors = nullptr;
    Sum* partial = nullptr;
    unsigned* done = nullptr;
    std::string error;

    int fail(int status, const char* what) {
        try { error = what; } catch (...) {}
        return status;
    }
    int cuda(cudaError_t e) { return fail(DDP_ERR_CUDA, cudaGetErrorString(e)); }
};

namespace {

// CTAs per SM at most.  The step takes many short shares, which keep the SMs'
// streams near one another and end together (BERT-large, 32 / 64 / 128 a SM:
// 1,397 / 1,373 / 1,355 us, 256: 1,345; GPT-2-medium with 8-bit moments, 128 /
// 256: 959 / 981); the norm takes one resident wave, of which the last adds all
// partial sums (BERT-large, 2 / 3 / 4: 201 / 192 / 216 us).
constexpr int kNormCtasPerSm = 3;
constexpr int kStepCtasPerSm[2] = {256, 128};    // 32-bit and 8-bit moments
constexpr int kStep8WarpsPerSm = 28;             // resident: seven CTAs of 69 registers

bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

// CTAs for `runs`, at most `most`: as few runs a warp as fills the grid.
void split(int64_t runs, int warps, int64_t most, int* grid, long long* piece) {
    const int64_t ctas = (runs + warps - 1) / warps;
    const int64_t n = ctas < most ? ctas : most;
    *piece = (runs + n - 1) / n;
    *grid = static_cast<int>((runs + *piece - 1) / *piece);
}

int check_device(ddp_adamw* o) {
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return o->cuda(e);
    if (dev != o->device) return o->fail(DDP_ERR_INVALID_ARG, "the current device is not the one of ddp_adamw_bind");
    return DDP_OK;
}

}  // namespace

extern "C" {

int ddp_adamw_create(const int64_t* numel, int32_t P, ddp_dtype param_dtype, int32_t state_bits, ddp_adamw** out) {
    const auto fail = [](const char* what) {
        try { g_create_error = what; } catch (...) {}
        return DDP_ERR_INVALID_ARG;
    };
    if (!out) return fail("out is NULL");
    *out = nullptr;
    if (P < 0 || (P > 0 && !numel)) return fail("P < 0, or numel is NULL");
    if (param_dtype != DDP_F32 && param_dtype != DDP_BF16) return fail("param_dtype is neither DDP_F32 nor DDP_BF16");
    if (state_bits != 32 && state_bits != 8) return fail("state_bits is neither 32 nor 8");
    for (int32_t v = 0; v < P; ++v)
        if (numel[v] < 0) return fail("negative numel");
    ddp_adamw* o = new (std::nothrow) ddp_adamw;
    if (!o) return DDP_ERR_NO_MEMORY;
    try {
        o->numel.assign(numel, numel + P);
    } catch (...) {
        delete o;
        return DDP_ERR_NO_MEMORY;
    }
    o->bf16 = param_dtype == DDP_BF16;
    o->q8 = state_bits == 8;
    *out = o;
    return DDP_OK;
}

int ddp_adamw_bind(ddp_adamw* o, const float* const* grads, void* const* params, float* const* master,
                   void* const* exp_avg, void* const* exp_avg_sq, float* const* exp_avg_scale,
                   float* const* exp_avg_sq_scale, const float* weight_decay) {
    if (!o) return DDP_ERR_INVALID_ARG;
    const int P = static_cast<int>(o->numel.size());
    if (P > 0 && !grads) return o->fail(DDP_ERR_INVALID_ARG, "grads is NULL");
    const bool step = params != nullptr;
    if (step && P > 0) {
        if (!exp_avg || !exp_avg_sq) return o->fail(DDP_ERR_INVALID_ARG, "exp_avg or exp_avg_sq is NULL");
        if (o->bf16 != (master != nullptr))
            return o->fail(DDP_ERR_INVALID_ARG, "master copies belong to bf16 parameters, and to them alone");
        if (o->q8 != (exp_avg_scale != nullptr) || o->q8 != (exp_avg_sq_scale != nullptr))
            return o->fail(DDP_ERR_INVALID_ARG, "scales belong to 8-bit moments, and to them alone");
    }
    try {
        std::vector<Tensor> tensors;
        long long blocks = 0;
        for (int v = 0; v < P; ++v) {
            const int64_t n = o->numel[v];
            if (n == 0) continue;
            Tensor t = {};
            t.g = grads[v];
            t.n = n;
            t.var = v;
            if (!t.g || !aligned(t.g, 4)) return o->fail(DDP_ERR_INVALID_ARG, "a gradient is NULL or misaligned");
            t.vec_g = aligned(t.g, 16);
            if (step) {
                const uintptr_t psize = o->bf16 ? 2 : 4, ssize = o->q8 ? 1 : 4;
                t.p = params[v];
                t.m = exp_avg[v];
                t.v = exp_avg_sq[v];
                t.master = o->bf16 ? master[v] : nullptr;
                t.ms = o->q8 ? exp_avg_scale[v] : nullptr;
                t.vs = o->q8 ? exp_avg_sq_scale[v] : nullptr;
                t.wd = weight_decay ? weight_decay[v] : 0.0f;
                if (!t.p || !t.m || !t.v || (o->bf16 && !t.master) || (o->q8 && (!t.ms || !t.vs)))
                    return o->fail(DDP_ERR_INVALID_ARG, "a tensor that is not empty has a NULL address");
                if (!aligned(t.p, psize) || !aligned(t.m, ssize) || !aligned(t.v, ssize) || !aligned(t.master, 4) ||
                    !aligned(t.ms, 4) || !aligned(t.vs, 4))
                    return o->fail(DDP_ERR_INVALID_ARG, "an address is not aligned to its element");
                if (!(t.wd >= 0.0f) || std::isinf(t.wd))
                    return o->fail(DDP_ERR_INVALID_ARG, "weight_decay is negative or not finite");
                t.vec = aligned(t.p, 4 * psize) && aligned(t.m, 16) && aligned(t.v, 16) && aligned(t.master, 16);
            }
            t.block0 = blocks;
            tensors.push_back(t);
            blocks += (n + kBlock - 1) / kBlock;
        }

        int dev = 0, sms = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
        if (e != cudaSuccess) return o->cuda(e);
        // first runs for the norm, then for the step.  The norm's are of eight
        // blocks where they still give an SM 32 warps theirs (10 M elements,
        // eight / four: 11.4 / 12.8 us).  32-bit moments have no scales and take
        // single blocks: a warp's neighbours then work on the same pages
        // (GPT-2-medium, bf16 weights: 1,579 us against 1,595).  With 8-bit
        // moments the runs fill whole waves of the warps that fit an SM: one of
        // runs of at most two blocks, else two or more of up to eight (runs halved
        // from eight on until an SM has 64 / this: 3 M elements 13.1 / 11.4 us, 4 M
        // 16.2 / 14.2, 3 M of which a third is unused 11.1 / 9.5, 10 M 28.5 / 27.7;
        // one wave of longer runs loses where tensors are unused: 11.3)
        const size_t S = tensors.size();
        std::vector<long long> first;
        Runs runs[2];
        for (int k = 0; k < 2; ++k) {
            if (k == 0) {
                runs[k].run = kMaxRun;
                while (runs[k].run > 1 && blocks < static_cast<int64_t>(runs[k].run) * sms * 32) runs[k].run /= 2;
            } else if (o->q8) {
                int64_t run = 0, warps = 0;
                do {
                    warps += static_cast<int64_t>(sms) * kStep8WarpsPerSm;
                    run = (blocks + warps - 1) / warps;
                } while (run > (warps == static_cast<int64_t>(sms) * kStep8WarpsPerSm ? 2 : kMaxRun));
                if (run > 1) runs[k].run = static_cast<int>(run);
            }
            for (const Tensor& t : tensors) {
                first.push_back(runs[k].count);
                runs[k].count += ((t.n + kBlock - 1) / kBlock + runs[k].run - 1) / runs[k].run;
            }
            first.push_back(runs[k].count);
        }
        const size_t at_first = S * sizeof(Tensor);
        const size_t at_partial = at_first + (first.size() * sizeof(long long) + 15) / 16 * 16;
        const size_t at_done = at_partial + static_cast<size_t>(sms) * kNormCtasPerSm * sizeof(Sum);
        std::vector<unsigned char> image(at_done + 16, 0);
        if (S) std::memcpy(image.data(), tensors.data(), at_first);
        std::memcpy(image.data() + at_first, first.data(), first.size() * sizeof(long long));
        void* table = nullptr;
        e = cudaMalloc(&table, image.size());
        if (e != cudaSuccess) {
            cudaGetLastError();
            return e == cudaErrorMemoryAllocation ? o->fail(DDP_ERR_NO_MEMORY, cudaGetErrorString(e)) : o->cuda(e);
        }
        // a copy from pageable memory returns before it has landed, and streams
        // that do not block on the legacy one would not wait for it
        e = cudaMemcpy(table, image.data(), image.size(), cudaMemcpyHostToDevice);
        if (e == cudaSuccess) e = cudaStreamSynchronize(cudaStreamLegacy);
        if (e != cudaSuccess) {
            cudaFree(table);
            return o->cuda(e);
        }
        if (o->table) cudaFree(o->table);      // waits for the kernels that read it
        unsigned char* base = static_cast<unsigned char*>(table);
        o->table = table;
        o->tensors = reinterpret_cast<const Tensor*>(base);
        runs[0].first = reinterpret_cast<const long long*>(base + at_first);
        runs[1].first = runs[0].first + S + 1;
        o->norm = runs[0];
        o->step = runs[1];
        o->partial = reinterpret_cast<Sum*>(base + at_partial);
        o->done = reinterpret_cast<unsigned*>(base + at_done);
        o->S = static_cast<int>(S);
        o->device = dev;
        o->sms = sms;
        o->has_params = step;
        o->bound = true;
    } catch (...) {
        return o->fail(DDP_ERR_NO_MEMORY, "out of host memory");
    }
    return DDP_OK;
}

int ddp_adamw_step(ddp_adamw* o, const ddp_adamw_args* x, void* stream) {
    if (!o) return DDP_ERR_INVALID_ARG;
    if (!x) return o->fail(DDP_ERR_INVALID_ARG, "args is NULL");
    if (x->t < 1) return o->fail(DDP_ERR_INVALID_ARG, "t < 1");
    const auto number = [](double y) { return std::isfinite(static_cast<float>(y)); };   // as the kernel has it
    if (!(x->lr >= 0.0) || !number(x->lr)) return o->fail(DDP_ERR_INVALID_ARG, "lr is negative or not finite");
    if (!(x->beta1 >= 0.0 && x->beta1 < 1.0) || !(x->beta2 >= 0.0 && x->beta2 < 1.0))
        return o->fail(DDP_ERR_INVALID_ARG, "a beta is not in [0, 1)");
    if (!(static_cast<float>(x->eps) >= FLT_MIN) || !number(x->eps))
        return o->fail(DDP_ERR_INVALID_ARG, "eps is not a positive (normal fp32) number");
    if (!(x->max_norm >= 0.0) || !number(x->max_norm))
        return o->fail(DDP_ERR_INVALID_ARG, "max_norm is negative or not finite");
    if ((x->max_norm > 0.0 || x->skip_nonfinite) && !x->norm)
        return o->fail(DDP_ERR_INVALID_ARG, "max_norm and skip_nonfinite need a norm");
    if (!aligned(x->norm, 4)) return o->fail(DDP_ERR_INVALID_ARG, "norm is not aligned to its element");
    if (!o->bound || !o->has_params) return o->fail(DDP_ERR_NOT_BOUND, "no parameters are bound");
    if (const int st = check_device(o)) return st;
    if (o->step.count == 0) return DDP_OK;

    StepParams a = {};
    a.tensors = o->tensors;
    a.first = o->step.first;
    a.norm = x->norm;
    a.used = x->used;
    a.runs = o->step.count;
    a.run = o->step.run;
    a.S = o->S;
    a.c.beta1 = static_cast<float>(x->beta1);
    a.c.beta1c = static_cast<float>(1.0 - x->beta1);
    a.c.beta2 = static_cast<float>(x->beta2);
    a.c.beta2c = static_cast<float>(1.0 - x->beta2);
    a.c.lr = static_cast<float>(x->lr);
    a.c.step = static_cast<float>(x->lr / (1.0 - std::pow(x->beta1, static_cast<double>(x->t))));
    a.c.rbc2 = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(x->beta2, static_cast<double>(x->t))));
    a.c.eps = static_cast<float>(x->eps);
    a.c.max_norm = static_cast<float>(x->max_norm);
    a.c.one = 1.0f;
    a.c.clip = x->max_norm > 0.0;
    a.c.skip_nonfinite = x->skip_nonfinite != 0;
    a.c.seed_lo = static_cast<uint32_t>(x->seed);
    a.c.seed_hi = static_cast<uint32_t>(x->seed >> 32);
    int grid = 0;
    split(o->step.count, kWarps, static_cast<int64_t>(o->sms) * kStepCtasPerSm[o->q8], &grid, &a.piece);
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e = o->bf16 ? (o->q8 ? launch(adamw_kernel<true, true>, kThreads, grid, a, st)
                                           : launch(adamw_kernel<true, false>, kThreads, grid, a, st))
                                  : (o->q8 ? launch(adamw_kernel<false, true>, kThreads, grid, a, st)
                                           : launch(adamw_kernel<false, false>, kThreads, grid, a, st));
    return e == cudaSuccess ? DDP_OK : o->cuda(e);
}

int ddp_adamw_grad_norm(ddp_adamw* o, const uint8_t* used, float* norm, void* stream) {
    if (!o) return DDP_ERR_INVALID_ARG;
    if (!norm || !aligned(norm, 4)) return o->fail(DDP_ERR_INVALID_ARG, "norm is NULL or not aligned to its element");
    if (!o->bound) return o->fail(DDP_ERR_NOT_BOUND, "no gradients are bound");
    if (const int st = check_device(o)) return st;
    NormParams a = {};
    a.tensors = o->tensors;
    a.first = o->norm.first;
    a.used = used;
    a.partial = o->partial;
    a.done = o->done;
    a.norm = norm;
    a.runs = o->norm.count;
    a.run = o->norm.run;
    a.S = o->S;
    int grid = 1;                    // without elements one CTA writes the zero
    if (o->norm.count) split(o->norm.count, kNormThreads / 32, static_cast<int64_t>(o->sms) * kNormCtasPerSm, &grid, &a.piece);
    const cudaError_t e = launch(norm_kernel, kNormThreads, grid, a, static_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? DDP_OK : o->cuda(e);
}

const char* ddp_adamw_last_error(const ddp_adamw* o) { return o ? o->error.c_str() : g_create_error.c_str(); }

void ddp_adamw_destroy(ddp_adamw* o) {
    if (!o) return;
    if (o->table) cudaFree(o->table);
    delete o;
}

}  // extern "C"
