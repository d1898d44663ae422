// Helpers of the operators that work on rows of activations (embedding, layer
// norm, dropout, log probabilities): eight neighbouring elements at a time,
// sums over a warp, launches.
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda_runtime.h>

#include "ddp_device.cuh"

namespace ddpk {
namespace rows {

constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(uint16_t x) { return dev::widen1(x); }

template <typename T> __device__ __forceinline__ T narrow(float x);
template <> __device__ __forceinline__ float narrow<float>(float x) { return x; }
template <> __device__ __forceinline__ uint16_t narrow<uint16_t>(float x) {
    uint16_t h;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(x));
    return h;
}

// Two fp32 numbers rounded to bf16 (to nearest even), the first in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float neg_inf() { return __int_as_float(0xff800000); }
__device__ __forceinline__ float nan_value() { return __int_as_float(0x7fffffff); }

// A pair of bf16 as they lie in memory plus fp32 numbers, without widening them first.
__device__ __forceinline__ float2 add_pair(uint32_t x, float2 y) {
    float2 d;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tadd.f32.bf16 %0, l, %3;\n\tadd.f32.bf16 %1, h, %4;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "r"(x), "f"(y.x), "f"(y.y));
    return d;
}

// 16 bytes that this kernel reads once, past L1; not through the read-only
// path, so that the same thread may store to them afterwards.
__device__ __forceinline__ uint4 ld_once(const void* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// Eight neighbouring elements as they lie in memory: one or two accesses of 16
// bytes, from a 16-byte boundary, or (wide) one, from a boundary of their size.
template <typename T> struct Eight;

template <> struct Eight<uint16_t> {
    uint4 v;
    __device__ __forceinline__ void load(const uint16_t* p) { v = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&f)[8]) const { dev::Vec<uint16_t>::unpack(v, f); }
    __device__ __forceinline__ void add_to(float (&f)[8]) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 d = add_pair(w[i], make_float2(f[2 * i], f[2 * i + 1]));
            f[2 * i] = d.x;
            f[2 * i + 1] = d.y;
        }
    }
    __device__ __forceinline__ void put(const float (&f)[8]) {
        v = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
    }
    __device__ __forceinline__ void load_wide(const uint16_t* p) { v = ld_once(p); }
    __device__ __forceinline__ void store_wide(uint16_t* p) const { __stcs(reinterpret_cast<uint4*>(p), v); }
    __device__ __forceinline__ void store_once(uint16_t* p) const { __stcs(reinterpret_cast<uint4*>(p), v); }
};

template <> struct Eight<float> {
    uint4 v[2];
    __device__ __forceinline__ void load(const float* p) {
        v[0] = reinterpret_cast<const uint4*>(p)[0];
        v[1] = reinterpret_cast<const uint4*>(p)[1];
    }
    __device__ __forceinline__ void zero() { v[0] = v[1] = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float (&f)[8]) const {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            f[4 * i] = __uint_as_float(v[i].x); f[4 * i + 1] = __uint_as_float(v[i].y);
            f[4 * i + 2] = __uint_as_float(v[i].z); f[4 * i + 3] = __uint_as_float(v[i].w);
        }
    }
    __device__ __forceinline__ void add_to(float (&f)[8]) const {
        float x[8];
        get(x);
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] += x[i];
    }
    __device__ __forceinline__ void put(const float (&f)[8]) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            v[i] = make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]), __float_as_uint(f[4 * i + 2]),
                              __float_as_uint(f[4 * i + 3]));
    }
    // whole sectors at once, from a 32-byte boundary: halves of one that two
    // accesses past L1 ask for are fetched twice
    __device__ __forceinline__ void load_wide(const float* p) {
        asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(v[0].x), "=r"(v[0].y), "=r"(v[0].z), "=r"(v[0].w), "=r"(v[1].x), "=r"(v[1].y), "=r"(v[1].z), "=r"(v[1].w)
                     : "l"(p));
    }
    __device__ __forceinline__ void store_wide(float* p) const {
        asm volatile("st.global.cs.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0].x), "r"(v[0].y), "r"(v[0].z),
                     "r"(v[0].w), "r"(v[1].x), "r"(v[1].y), "r"(v[1].z), "r"(v[1].w) : "memory");
    }
    __device__ __forceinline__ void store_once(float* p) const {
        __stcs(reinterpret_cast<uint4*>(p), v[0]);
        __stcs(reinterpret_cast<uint4*>(p) + 1, v[1]);
    }
};

template <int N> struct Constant { static constexpr int value = N; };

// Eight elements that begin `shift` bytes, whole elements, behind the start of
// 16-byte words: of those words and of the one behind them.
template <typename T>
__device__ __forceinline__ Eight<T> shifted(const Eight<T>& here, uint4 behind, int shift) {
    constexpr int kWords = static_cast<int>(sizeof(Eight<T>)) / 4;
    uint32_t w[kWords + 4], out[kWords];
    const uint4* const words = reinterpret_cast<const uint4*>(&here);
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i) { w[4 * i] = words[i].x; w[4 * i + 1] = words[i].y; w[4 * i + 2] = words[i].z; w[4 * i + 3] = words[i].w; }
    w[kWords] = behind.x; w[kWords + 1] = behind.y; w[kWords + 2] = behind.z; w[kWords + 3] = behind.w;
    const int bits = shift % 4 * 8;
    // the shift is the row's: one of four constant selections
    const auto select = [&](auto first) {
#pragma unroll
        for (int k = 0; k < kWords; ++k) {
            constexpr int from = decltype(first)::value;
            out[k] = sizeof(T) == 4 ? w[from + k] : __funnelshift_r(w[from + k], w[from + k + 1], bits);
        }
    };
    switch (shift / 4) {
        case 0: select(Constant<0>()); break;
        case 1: select(Constant<1>()); break;
        case 2: select(Constant<2>()); break;
        default: select(Constant<3>()); break;
    }
    Eight<T> x;
    uint4* const to = reinterpret_cast<uint4*>(&x);
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i) to[i] = make_uint4(out[4 * i], out[4 * i + 1], out[4 * i + 2], out[4 * i + 3]);
    return x;
}

// Over LANES neighbouring lanes (a power of two), the result in all of them.
template <int LANES>
__device__ __forceinline__ float lanes_sum(float x) {
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) x += __shfl_xor_sync(kAll, x, o);
    return x;
}

// Two fp32 numbers at a time, each rounded as by itself.
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tadd.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 d;
    asm("{\n\t.reg .b64 x, y;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmul.rn.f32x2 x, x, y;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return d;
}

__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 d;
    asm("{\n\t.reg .b64 x, y, z;\n\tmov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
        "fma.rn.f32x2 x, x, y, z;\n\tmov.b64 {%0, %1}, x;\n\t}"
        : "=f"(d.x), "=f"(d.y) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return d;
}

__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }

// Copies of 16 bytes to shared memory that the thread waits for by groups of
// its own; what a thread copied it may read after the wait without a barrier.
__device__ __forceinline__ void copy_async(void* to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(__cvta_generic_to_shared(to))), "l"(from)
                 : "memory");
}

__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// Until at most LEFT of the thread's groups are on their way.
template <int LEFT>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(LEFT) : "memory"); }

// ------------------------------------------------------------------ host

inline bool aligned(const void* p, uintptr_t to) { return (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0; }

inline int power_of_two(long long x) {
    int p = 1;
    while (p < x) p *= 2;
    return p;
}

// A launch that may begin while the one before it ends; the kernel waits for
// that one's end (dev::pdl_wait) before it touches memory.
template <typename P>
cudaError_t launch(void (*kernel)(P), long long ctas, int threads, size_t shared, cudaStream_t stream, const P& params,
                   int cluster = 1) {
    if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas));
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = shared;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, params);
}

// Lets a kernel have more than 48 KB of shared memory (of which up to 3 KB are
// its static variables), once on each device: `done` is the kernel's own.
inline cudaError_t allow_shared(const void* kernel, size_t shared, std::atomic<uint64_t>& done) {
    if (shared <= 45 * 1024) return cudaSuccess;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 224 * 1024);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// The multiprocessors that grids are sized for, and shares of work counted by:
// a constant, so that sums are split alike wherever the library runs.
constexpr int kSms = 152;

}  // namespace rows
}  // namespace ddpk
