// attn_common.cuh -- device pieces shared by the kernels around the linear layers: the two
// 16-bit element types and the keys a query sees.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ck_device.cuh"

namespace ck {

// Further bits of the device error word (see ck_device_error in the C ABI).
enum : uint32_t {
    kErrIndex = 1u << 7,       // a position, length, slot, page or sequence bound was out of range
    kErrWaitAttention = 1u << 8,  // a role of the prompt attention kernel gave up waiting
};

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// the larger of two, NaN where either is one (fmaxf drops it)
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// 16-bit element types: conversions to and from fp32 (round to nearest even)
struct Bf16 {
    using T = __nv_bfloat16;
    using T2 = __nv_bfloat162;
    static __device__ __forceinline__ float2 to2(uint32_t w)
    {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
    }
    static __device__ __forceinline__ uint32_t pack2(float lo, float hi)
    {
        const T2 v = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
    static __device__ __forceinline__ float to(T v) { return __bfloat162float(v); }
    static __device__ __forceinline__ T from(float v) { return __float2bfloat16_rn(v); }
};
struct Fp16 {
    using T = __half;
    using T2 = __half2;
    static __device__ __forceinline__ float2 to2(uint32_t w)
    {
        return __half22float2(*reinterpret_cast<const __half2*>(&w));
    }
    static __device__ __forceinline__ uint32_t pack2(float lo, float hi)
    {
        const T2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&v);
    }
    static __device__ __forceinline__ float to(T v) { return __half2float(v); }
    static __device__ __forceinline__ T from(float v) { return __float2half_rn(v); }
};

// The keys that one query sees, as two runs: [0, head) and [tail, end).  Numbered through,
// key number v of `count()` is v (v < head) or v - head + tail.
struct VisibleKeys {
    int head, tail, end;
    __host__ __device__ int count() const { return head + (end - tail); }
    __host__ __device__ int key(int v) const { return v < head ? v : v - head + tail; }
};

// end = keys up to and including the query's own position (0: none visible); window <= 0: all
__host__ __device__ inline VisibleKeys visible_keys(int end, int64_t window, int64_t sinks)
{
    VisibleKeys r;
    r.end = end < 0 ? 0 : end;
    const int64_t tail = window > 0 && window < r.end ? r.end - window : 0;
    r.tail = (int)tail;
    r.head = (int)(sinks < tail ? sinks : tail);
    return r;
}

}  // namespace ck
