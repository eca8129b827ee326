// adapter.cu -- low-rank adapters of many requests at once, beside a projection that they share.
//
//   y[m] = residual[m] + scaling[i] (x[m] A_i^T) B_i^T,  i = index[m];  y[m] = residual[m] where i < 0
#include <cmath>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_common.cuh"
#include "transformer.h"

namespace ck {
namespace {

// The low-rank row of x: one warp per (row, rank).
template <class E>
__global__ void __launch_bounds__(256) shrink_kernel(const AdapterLinear p, unsigned int* err)
{
    using T = typename E::T;
    griddep_wait();
    const int lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int64_t m = unit / p.rank;
    const int r = (int)(unit - m * p.rank);
    if (m < p.M) {
        const int i = __ldg(p.index + m);
        if (i >= p.adapters) {
            if (lane == 0 && r == 0)
                atomicOr(err, kErrIndex);
        } else if (i >= 0) {
            const T* x = static_cast<const T*>(p.x) + m * p.K;
            const T* a = static_cast<const T*>(p.a) + ((int64_t)i * p.rank + r) * p.K;
            float sum = 0.0f;
            for (int64_t k = lane; k < p.K; k += 32)
                sum = fmaf(E::to(x[k]), E::to(a[k]), sum);
#pragma unroll
            for (int o = 16; o; o >>= 1)
                sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (lane == 0)
                static_cast<float*>(p.workspace)[m * p.rank + r] = sum;
        }
    }
    griddep_launch_dependents();
}

template <int OUT>
__device__ __forceinline__ float load_out(const void* base, int64_t i)
{
    if (OUT == CK_OUT_F32)
        return static_cast<const float*>(base)[i];
    return OUT == CK_OUT_F16 ? Fp16::to(static_cast<const __half*>(base)[i]) : Bf16::to(static_cast<const __nv_bfloat16*>(base)[i]);
}

template <int OUT>
__device__ __forceinline__ void store_out(void* base, int64_t i, float v)
{
    if (OUT == CK_OUT_F32)
        static_cast<float*>(base)[i] = v;
    else if (OUT == CK_OUT_F16)
        static_cast<__half*>(base)[i] = Fp16::from(v);
    else
        static_cast<__nv_bfloat16*>(base)[i] = Bf16::from(v);
}

// One thread per output.
template <class E, int OUT>
__global__ void __launch_bounds__(256) expand_kernel(const AdapterLinear p)
{
    using T = typename E::T;
    griddep_wait();
    const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
    const int64_t m = at / p.N, n = at - m * p.N;
    if (m < p.M) {
        const int i = __ldg(p.index + m);
        float v = p.residual ? load_out<OUT>(p.residual, at) : 0.0f;
        if (i >= p.adapters) {
            v = NAN;
        } else if (i >= 0) {
            const T* b = static_cast<const T*>(p.b) + ((int64_t)i * p.N + n) * p.rank;
            const float* h = static_cast<const float*>(p.workspace) + m * p.rank;
            float sum = 0.0f;
            for (int r = 0; r < p.rank; ++r)
                sum = fmaf(h[r], E::to(b[r]), sum);
            v += sum * (p.scaling ? __ldg(p.scaling + i) : 1.0f);
        }
        store_out<OUT>(p.y, at, v);
    }
    griddep_launch_dependents();
}

}  // namespace

size_t adapter_workspace(int64_t M, int64_t, int64_t, int rank)
{
    return (size_t)M * rank * sizeof(float);
}

cudaError_t launch_adapter_linear(const AdapterLinear& p, const DeviceInfo& dev, cudaStream_t s)
{
    (void)dev;
    unsigned int* err = nullptr;
    cudaError_t e = device_error_ptr(&err);
    if (e != cudaSuccess)
        return e;
    const dim3 shrink((unsigned)((p.M * p.rank + 7) / 8)), expand((unsigned)((p.M * p.N + 255) / 256));
    auto run = [&](auto type) {
        using E = decltype(type);
        const cudaError_t r = launch_pdl(shrink_kernel<E>, shrink, dim3(256), 0, s, p, err);
        if (r != cudaSuccess)
            return r;
        if (p.out_dtype == CK_OUT_F32)
            return launch_pdl(expand_kernel<E, CK_OUT_F32>, expand, dim3(256), 0, s, p);
        if (p.out_dtype == CK_OUT_F16)
            return launch_pdl(expand_kernel<E, CK_OUT_F16>, expand, dim3(256), 0, s, p);
        return launch_pdl(expand_kernel<E, CK_OUT_BF16>, expand, dim3(256), 0, s, p);
    };
    return p.f16 ? run(Fp16()) : run(Bf16());
}

}  // namespace ck
