// logprobs.cu -- log probabilities of given tokens, the entropy and the top alternatives of rows of
// logits.
//
//   t_j = scale * (x_j - max x),  s = sum_j exp(t_j)
//   logprob = t_token - log s,  lse = scale * max x + log s,  entropy = log s - sum_j t_j exp(t_j) / s
//   top: the largest logits in order (NaN above all; of equal ones the lowest index first)
#include <cmath>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_common.cuh"
#include "transformer.h"

namespace ck {
namespace {

constexpr int THREADS = 1024;

template <int TYPE>
__device__ __forceinline__ float logit_at(const void* row, int64_t j)
{
    if (TYPE == CK_OUT_F32)
        return __ldg(static_cast<const float*>(row) + j);
    return TYPE == CK_OUT_F16 ? Fp16::to(__ldg(static_cast<const __half*>(row) + j))
                              : Bf16::to(__ldg(static_cast<const __nv_bfloat16*>(row) + j));
}

// Logits as integers in their order: NaN above +inf, -0 and +0 equal.
__device__ __forceinline__ uint32_t order_of(float x)
{
    if (x != x)
        return 0xffffffffu;
    const uint32_t u = x == 0.0f ? 0u : __float_as_uint(x);
    return (int32_t)u < 0 ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ double block_sum(double v, double* scratch)
{
#pragma unroll
    for (int o = 16; o; o >>= 1)
        v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0)
        scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0.0;
    for (int w = 0; w < THREADS / 32; ++w)
        v += scratch[w];
    return v;
}

__device__ __forceinline__ uint64_t block_max(uint64_t v, uint64_t* scratch)
{
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        const uint64_t u = __shfl_xor_sync(0xffffffffu, v, o);
        v = u > v ? u : v;
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0)
        scratch[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0;
    for (int w = 0; w < THREADS / 32; ++w)
        v = scratch[w] > v ? scratch[w] : v;
    return v;
}

// One block per row; the row is read once for the sums and once for each alternative.
template <int TYPE>
__global__ void __launch_bounds__(THREADS) row_kernel(const TokenLogprobs p, unsigned int* err)
{
    griddep_wait();
    __shared__ uint64_t scratch[THREADS / 32];
    const int64_t m = blockIdx.x;
    constexpr int SIZE = TYPE == CK_OUT_F32 ? 4 : 2;
    const void* row = static_cast<const char*>(p.logits) + m * p.stride * SIZE;
    // (order, index) as one number, the lowest index above the others
    auto key_of = [&](int64_t j) { return (uint64_t)order_of(logit_at<TYPE>(row, j)) << 32 | (0xffffffffu - (uint32_t)j); };
    uint64_t best = 0;
    for (int64_t j = threadIdx.x; j < p.vocab; j += THREADS) {
        const uint64_t k = key_of(j);
        best = k > best ? k : best;
    }
    best = block_max(best, scratch);
    const float high = logit_at<TYPE>(row, (int64_t)(0xffffffffu - (uint32_t)best));
    double sum = 0.0, weighted = 0.0;  // without the largest's own 1
    for (int64_t j = threadIdx.x; j < p.vocab; j += THREADS) {
        if (j == (int64_t)(0xffffffffu - (uint32_t)best) && high - high == 0.0f)
            continue;
        const float t = p.scale * (logit_at<TYPE>(row, j) - high);
        const float e = expf(t);
        sum += e;
        weighted += e == 0.0f ? 0.0f : e * t;
    }
    sum = block_sum(sum, reinterpret_cast<double*>(scratch));
    weighted = block_sum(weighted, reinterpret_cast<double*>(scratch));
    const double log_sum = high - high == 0.0f ? log1p(sum) : NAN;
    if (threadIdx.x == 0) {
        if (p.logprob) {
            const int token = __ldg(p.tokens + m);
            float r = 0.0f;
            if (token >= p.vocab) {
                r = NAN;
                atomicOr(err, kErrIndex);
            } else if (token >= 0) {
                r = (float)((double)p.scale * (logit_at<TYPE>(row, token) - high) - log_sum);
            }
            p.logprob[m] = r;
        }
        if (p.entropy)
            p.entropy[m] = (float)(log_sum - weighted / (1.0 + sum));
        if (p.lse)
            p.lse[m] = high == -INFINITY ? -INFINITY : high == INFINITY ? INFINITY : (float)((double)p.scale * high + log_sum);
    }
    for (int i = 0; i < p.top; ++i) {
        const int64_t j = (int64_t)(0xffffffffu - (uint32_t)best);
        if (threadIdx.x == 0) {
            p.top_index[m * p.top + i] = (int32_t)j;
            p.top_logprob[m * p.top + i] = (float)((double)p.scale * (logit_at<TYPE>(row, j) - high) - log_sum);
        }
        if (i + 1 == p.top)
            break;
        uint64_t next = 0;
        for (int64_t n = threadIdx.x; n < p.vocab; n += THREADS) {
            const uint64_t k = key_of(n);
            next = k < best && k > next ? k : next;
        }
        best = block_max(next, scratch);
    }
    griddep_launch_dependents();
}

}  // namespace

size_t logprobs_workspace(int64_t, int64_t, int)
{
    return 0;
}

int logprobs_launches(const TokenLogprobs&, const DeviceInfo&)
{
    return 1;
}

cudaError_t launch_token_logprobs(const TokenLogprobs& p, const DeviceInfo& dev, cudaStream_t s)
{
    (void)dev;
    unsigned int* err = nullptr;
    const cudaError_t e = device_error_ptr(&err);
    if (e != cudaSuccess)
        return e;
    auto run = [&](auto kernel) { return launch_pdl(kernel, dim3((unsigned)p.rows), dim3(THREADS), 0, s, p, err); };
    return p.dtype == CK_OUT_F32 ? run(row_kernel<CK_OUT_F32>)
                                 : p.dtype == CK_OUT_F16 ? run(row_kernel<CK_OUT_F16>) : run(row_kernel<CK_OUT_BF16>);
}

}  // namespace ck
