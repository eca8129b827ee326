// paged_attention.cu -- attention of one new token per sequence over the paged cache.
//
//   out[b,h] = sum_j w_j v_j / sum_j w_j,  w_j = exp(scale * q[b,h] . k_j - max),  j over the
//   keys of sequence b that its last token sees (all, or the first `sinks` and the last
//   `window`); zeros where the sequence is empty.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_common.cuh"
#include "transformer.h"

namespace ck {
namespace {

template <class E, bool INT8, int DIM>
__global__ void __launch_bounds__(32) paged_row_kernel(const PagedAttention p, unsigned int* err)
{
    griddep_wait();
    __shared__ float qs[DIM];
    using T = typename E::T;
    const int lane = threadIdx.x;
    const int64_t b = blockIdx.x / p.q_heads;
    const int h = (int)(blockIdx.x - b * p.q_heads);
    const int hk = h / (p.q_heads / p.cache.heads);
    const T* q = static_cast<const T*>(p.q) + b * p.q_stride + (int64_t)h * DIM;
    for (int d = lane; d < DIM; d += 32)
        qs[d] = E::to(q[d]) * (p.scale * kLog2e);
    __syncwarp();
    const int64_t len = __ldg(p.seq_lens + b);
    bool bad = len < 0 || len > p.max_blocks * p.cache.page_size;
    const VisibleKeys keys = visible_keys(bad ? 0 : (int)len, p.window, p.sinks);
    const int32_t* table = p.block_table + b * p.max_blocks;
    const size_t row_bytes = (size_t)DIM * (INT8 ? 1 : 2);
    bool off_table = false;
    float acc[(DIM + 31) / 32], m, l;
    attend_row<E, INT8, DIM>(qs, keys.count(), [&](int v) {
        const int j = keys.key(v);
        int64_t page = __ldg(table + j / p.cache.page_size);
        if (page < 0 || page >= p.cache.num_pages) {
            off_table = true;
            page = 0;
        }
        const int64_t row = (page * p.cache.heads + hk) * p.cache.page_size + j % p.cache.page_size;
        KvRow r;
        r.k = static_cast<const uint8_t*>(p.cache.k) + row * row_bytes;
        r.v = static_cast<const uint8_t*>(p.cache.v) + row * row_bytes;
        r.ks = INT8 ? __ldg(p.cache.k_scale + row) : 1.0f;
        r.vs = INT8 ? __ldg(p.cache.v_scale + row) : 1.0f;
        return r;
    }, acc, m, l);
    bad = __any_sync(0xffffffffu, bad || off_table);
    if (bad && lane == 0)
        atomicOr(err, kErrIndex);
    const int64_t at = b * p.q_heads + h;
#pragma unroll
    for (int i = 0; i < (DIM + 31) / 32; ++i)
        static_cast<T*>(p.out)[at * DIM + lane + 32 * i] =
            E::from(bad ? NAN : keys.count() == 0 ? 0.0f : acc[i] / l);
    if (p.lse != nullptr && lane == 0)
        p.lse[at] = bad ? NAN : (m + log2f(l)) * kLn2;
}

template <class E, bool INT8, int DIM>
cudaError_t launch(const PagedAttention& p, unsigned int* err, cudaStream_t s)
{
    return launch_pdl(paged_row_kernel<E, INT8, DIM>, dim3((unsigned)(p.batch * p.q_heads)), dim3(32), 0, s, p, err);
}

template <int DIM>
cudaError_t by_type(const PagedAttention& p, unsigned int* err, cudaStream_t s)
{
    if (p.cache.dtype == CK_KV_INT8)
        return p.f16 ? launch<Fp16, true, DIM>(p, err, s) : launch<Bf16, true, DIM>(p, err, s);
    return p.f16 ? launch<Fp16, false, DIM>(p, err, s) : launch<Bf16, false, DIM>(p, err, s);
}

}  // namespace

size_t paged_attention_workspace(int64_t batch, int q_heads, int kv_heads, int dim)
{
    (void)batch, (void)q_heads, (void)kv_heads, (void)dim;
    return 16;
}

cudaError_t launch_paged_attention(const PagedAttention& p, const DeviceInfo& dev, cudaStream_t s)
{
    (void)dev;
    unsigned int* err = nullptr;
    cudaError_t e = device_error_ptr(&err);
    if (e != cudaSuccess)
        return e;
    return p.cache.dim == 64 ? by_type<64>(p, err, s) : by_type<128>(p, err, s);
}

}  // namespace ck
