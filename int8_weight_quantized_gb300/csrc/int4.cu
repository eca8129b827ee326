// int4.cu -- the linear layer with 4-bit weights and group scales, for few rows, and its
// weight preparation.
//
//   y[m,n] = out( sum_g scale[n,g] * (sum_{k in g} x[m,k] * c[n,k]) + bias[n] + residual[m,n] )
//   c = code - 8 in [-8, 7], eight codes to a 32-bit word: the code of k = 8 j + 2 i in bits
//   4 i .. 4 i + 3 of word j, that of k = 8 j + 2 i + 1 in bits 16 + 4 i .. (a pair of
//   neighbouring k is then one shift and one mask away from two 16-bit halves).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_common.cuh"
#include "transformer.h"

namespace ck {
namespace {

__device__ __forceinline__ int code_shift(int e)
{
    return 4 * (e >> 1) + 16 * (e & 1);
}

template <class E>
__global__ void __launch_bounds__(128) int4_row_kernel(const Int4Linear p)
{
    griddep_wait();
    using T = typename E::T;
    const int lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
    const int64_t m = unit / p.N, n = unit - m * p.N;
    if (m >= p.M)
        return;
    const uint32_t* w = p.w4 + n * (p.K / 8);
    const __nv_bfloat16* sc = static_cast<const __nv_bfloat16*>(p.w_scale) + n * (p.K / p.group);
    const T* x = static_cast<const T*>(p.x) + m * p.K;
    float sum = 0.0f;
    for (int64_t j = lane; j < p.K / 8; j += 32) {
        const uint32_t word = __ldg(w + j);
        float part = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            part = fmaf(E::to(x[8 * j + e]), (float)((int)((word >> code_shift(e)) & 15u) - 8), part);
        sum = fmaf(part, __bfloat162float(sc[8 * j / p.group]), sum);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1)
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane != 0)
        return;
    if (p.bias != nullptr)
        sum += E::to(static_cast<const T*>(p.bias)[n]);
    const int64_t at = m * p.N + n;
    if (p.out_dtype == CK_OUT_F32)
        static_cast<float*>(p.y)[at] = sum + (p.residual ? static_cast<const float*>(p.residual)[at] : 0.0f);
    else if (p.out_dtype == CK_OUT_F16)
        static_cast<__half*>(p.y)[at] =
            __float2half_rn(sum + (p.residual ? __half2float(static_cast<const __half*>(p.residual)[at]) : 0.0f));
    else
        static_cast<__nv_bfloat16*>(p.y)[at] = __float2bfloat16_rn(
            sum + (p.residual ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.residual)[at]) : 0.0f));
}

// Weight preparation: one thread per word for the codes; the group's scale is found by the
// group / 8 threads that share it (group <= 256: within a warp).
__global__ void __launch_bounds__(256) int4_weight_kernel(const float* W, int64_t words, int group, uint32_t* w4,
                                                          __nv_bfloat16* w_scale)
{
    griddep_wait();
    const int lanes = group / 8;  // a power of two up to 32
    const int64_t j = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const bool in = j < words;  // words is a multiple of lanes: a group is all in or all out
    float v[8];
    float top = 0.0f;
    if (in) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(W + 8 * j));
        const float4 b = __ldg(reinterpret_cast<const float4*>(W + 8 * j + 4));
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            top = fmaxf(top, fabsf(v[e]));
    }
    for (int o = lanes >> 1; o; o >>= 1)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (!in)
        return;
    const __nv_bfloat16 s16 = __float2bfloat16_rn(__fdiv_rn(top, 7.0f));
    const float s = __bfloat162float(s16);
    uint32_t word = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int c = s > 0.0f ? (int)fminf(fmaxf(rintf(__fdiv_rn(v[e], s)), -7.0f), 7.0f) : 0;
        word |= (uint32_t)(c + 8) << code_shift(e);
    }
    w4[j] = word;
    if (threadIdx.x % lanes == 0)
        w_scale[j / lanes] = s16;
}

__global__ void __launch_bounds__(256) int4_pack_kernel(const int8_t* codes, int64_t words, uint32_t* w4)
{
    griddep_wait();
    const int64_t j = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (j >= words)
        return;
    const uint2 r = __ldg(reinterpret_cast<const uint2*>(codes + 8 * j));
    uint32_t word = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int c = (int)(int8_t)(((e < 4 ? r.x : r.y) >> (8 * (e & 3))) & 255u);
        word |= (uint32_t)(min(max(c, -8), 7) + 8) << code_shift(e);
    }
    w4[j] = word;
}

}  // namespace

size_t int4_linear_workspace(int64_t M, int64_t N, int64_t K)
{
    (void)M, (void)N, (void)K;
    return 16;
}

cudaError_t launch_int4_linear(const Int4Linear& p, const DeviceInfo& dev, cudaStream_t s)
{
    (void)dev;
    const unsigned blocks = (unsigned)((p.M * p.N + 3) / 4);
    return p.f16 ? launch_pdl(int4_row_kernel<Fp16>, dim3(blocks), dim3(128), 0, s, p)
                 : launch_pdl(int4_row_kernel<Bf16>, dim3(blocks), dim3(128), 0, s, p);
}

cudaError_t launch_int4_weight(const float* W, int64_t N, int64_t K, int group, uint32_t* w4, void* w_scale,
                               const DeviceInfo& dev, cudaStream_t s)
{
    (void)dev;
    const int64_t words = N * (K / 8);
    return launch_pdl(int4_weight_kernel, dim3((unsigned)((words + 255) / 256)), dim3(256), 0, s, W, words, group, w4,
                      static_cast<__nv_bfloat16*>(w_scale));
}

cudaError_t launch_int4_pack(const int8_t* codes, int64_t N, int64_t K, uint32_t* w4, const DeviceInfo& dev,
                             cudaStream_t s)
{
    (void)dev;
    const int64_t words = N * (K / 8);
    return launch_pdl(int4_pack_kernel, dim3((unsigned)((words + 255) / 256)), dim3(256), 0, s, codes, words, w4);
}

}  // namespace ck
