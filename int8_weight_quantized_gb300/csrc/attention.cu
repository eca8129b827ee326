// attention.cu -- attention over whole prompts, ragged batches of them, causal or not, with a
// sliding window and first tokens that stay visible.
//
//   out[i,h] = sum_j w_j v_j / sum_j w_j,  w_j = exp(scale * q_i . k_j - max), j over the keys
//   of query i's sequence that it sees; zeros where it sees none.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_common.cuh"
#include "transformer.h"

namespace ck {
namespace {

// The sequence whose queries hold row `row`: the last b with cu[b] <= row (-1: none).
__device__ __forceinline__ int64_t sequence_of(const int32_t* cu, int64_t batch, int64_t row)
{
    int64_t lo = 0, hi = batch;  // cu[lo] <= row < cu[hi], once checked
    if (__ldg(cu) > row || __ldg(cu + batch) <= row)
        return -1;
    while (hi - lo > 1) {
        const int64_t mid = (lo + hi) >> 1;
        if (__ldg(cu + mid) <= row)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

template <class E, int DIM>
__global__ void __launch_bounds__(128) prompt_row_kernel(const PromptAttention p, unsigned int* err)
{
    griddep_wait();
    __shared__ float qs_all[4][DIM];
    using T = typename E::T;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t unit = (int64_t)blockIdx.x * 4 + warp;
    const int64_t i = unit / p.q_heads;
    const int h = (int)(unit - i * p.q_heads);
    if (i >= p.total_q)
        return;
    const int64_t b = sequence_of(p.cu_q, p.batch, i);
    if (b < 0)
        return;
    const int64_t q0 = __ldg(p.cu_q + b), q1 = __ldg(p.cu_q + b + 1);
    const int64_t k0 = __ldg(p.cu_k + b), k1 = __ldg(p.cu_k + b + 1);
    const bool bad = q0 < 0 || q1 > p.total_q || q1 < q0 || k0 < 0 || k1 < k0 || k1 > p.total_k;
    float* qs = qs_all[warp];
    const T* q = static_cast<const T*>(p.q) + i * p.q_stride + (int64_t)h * DIM;
    for (int d = lane; d < DIM; d += 32)
        qs[d] = E::to(q[d]) * (p.scale * kLog2e);
    __syncwarp();
    const int hk = h / (p.q_heads / p.kv_heads);
    const int nk = bad ? 0 : (int)(k1 - k0);
    const VisibleKeys keys = p.causal ? visible_keys((int)(nk - (q1 - 1 - i)), p.window, p.sinks)
                                      : visible_keys(nk, 0, 0);
    float acc[(DIM + 31) / 32], m, l;
    attend_row<E, false, DIM>(qs, bad ? 0 : keys.count(), [&](int v) {
        const int64_t j = k0 + keys.key(v);
        KvRow r;
        r.k = static_cast<const T*>(p.k) + j * p.k_stride + (int64_t)hk * DIM;
        r.v = static_cast<const T*>(p.v) + j * p.v_stride + (int64_t)hk * DIM;
        r.ks = r.vs = 1.0f;
        return r;
    }, acc, m, l);
    if (bad && lane == 0)
        atomicOr(err, kErrIndex);
#pragma unroll
    for (int c = 0; c < (DIM + 31) / 32; ++c)
        static_cast<T*>(p.out)[(i * p.q_heads + h) * DIM + lane + 32 * c] =
            E::from(bad ? NAN : keys.count() == 0 ? 0.0f : acc[c] / l);
    if (p.lse != nullptr && lane == 0)
        p.lse[(int64_t)h * p.total_q + i] = bad ? NAN : (m + log2f(l)) * kLn2;
}

template <class E, int DIM>
cudaError_t launch(const PromptAttention& p, unsigned int* err, cudaStream_t s)
{
    const int64_t units = p.total_q * p.q_heads;
    return launch_pdl(prompt_row_kernel<E, DIM>, dim3((unsigned)((units + 3) / 4)), dim3(128), 0, s, p, err);
}

}  // namespace

cudaError_t launch_attention(const PromptAttention& p, const DeviceInfo& dev, cudaStream_t s, std::string* why)
{
    (void)dev, (void)why;
    unsigned int* err = nullptr;
    cudaError_t e = device_error_ptr(&err);
    if (e != cudaSuccess)
        return e;
    if (p.dim == 64)
        return p.f16 ? launch<Fp16, 64>(p, err, s) : launch<Bf16, 64>(p, err, s);
    return p.f16 ? launch<Fp16, 128>(p, err, s) : launch<Bf16, 128>(p, err, s);
}

}  // namespace ck
