// transformer.h -- host-side interface between the C ABI (api_transformer.cu) and the kernels
// of the operators around the linear layers: norm_rope.cu, paged_attention.cu, attention.cu,
// int4.cu.  The public contract is include/ck_int8.h.
#pragma once

#include <cstddef>
#include <cstdint>
#include <string>

#include <cuda_runtime.h>

#include "ck_int8.h"
#include "ck_internal.h"

namespace ck {

// A paged cache as the kernels see it (ck_kv_cache_t after its checks).
struct KvCache {
    void* k = nullptr;
    void* v = nullptr;
    float* k_scale = nullptr;  // int8 caches only
    float* v_scale = nullptr;
    int64_t num_pages = 0;
    int page_size = 0;
    int heads = 0;
    int dim = 0;
    int dtype = 0;  // ck_kv_dtype_t
};

struct NormRope {
    const void* qkv;
    int64_t qkv_stride;  // elements between tokens
    int64_t tokens;
    int q_heads, kv_heads, dim, rot;
    bool f16, norm, interleaved;
    const void* q_weight;  // [dim] or nullptr
    const void* k_weight;
    float eps;
    const int32_t* positions;
    const float* cos_sin;  // [max_pos, rot]
    int64_t max_pos;
    void* q_out;
    void* k_out;  // or nullptr
    KvCache cache;  // k == nullptr: none
    const int64_t* slots;
};
cudaError_t launch_norm_rope(const NormRope& p, const DeviceInfo& dev, cudaStream_t s);

struct PagedAttention {
    const void* q;
    int64_t q_stride;  // elements between sequences
    KvCache cache;
    const int32_t* block_table;
    int64_t max_blocks;
    const int32_t* seq_lens;
    int64_t batch;
    int q_heads;
    bool f16;
    float scale;
    int64_t window, sinks;
    int page_shift;  // log2 of the page size, -1 if it is no power of two
    void* out;
    float* lse;  // or nullptr
    void* workspace;
};
// by query heads per kv head and the most keys a sequence can have
size_t paged_attention_workspace(int group, int dim, int64_t max_len);
int paged_attention_launches(const PagedAttention& p);  // kernels that the call enqueues
cudaError_t launch_paged_attention(const PagedAttention& p, const DeviceInfo& dev, cudaStream_t s);

struct PromptAttention {
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;  // elements between tokens
    const int32_t *cu_q, *cu_k;
    int64_t batch, total_q, total_k;
    int q_heads, kv_heads, dim;
    bool f16, causal;
    float scale;
    int64_t window, sinks;
    void* out;
    float* lse;  // or nullptr
};
cudaError_t launch_attention(const PromptAttention& p, const DeviceInfo& dev, cudaStream_t s, std::string* why);

struct Int4Linear {
    const void* x;
    const uint32_t* w4;
    const void* w_scale;  // bf16 [N, K / group]
    const void* bias;     // x's type or nullptr
    const void* residual; // out type or nullptr
    void* y;
    int64_t M, N, K;
    int group;
    bool f16;
    int out_dtype;
};
cudaError_t launch_int4_linear(const Int4Linear& p, const DeviceInfo& dev, cudaStream_t s);
cudaError_t launch_int4_weight(const float* W, int64_t N, int64_t K, int group, uint32_t* w4, void* w_scale,
                               const DeviceInfo& dev, cudaStream_t s);
cudaError_t launch_int4_pack(const int8_t* codes, int64_t N, int64_t K, uint32_t* w4, const DeviceInfo& dev,
                             cudaStream_t s);

}  // namespace ck
