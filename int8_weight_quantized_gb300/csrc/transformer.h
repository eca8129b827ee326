// transformer.h -- host-side interface between the C ABI (api_transformer.cu) and the kernels
// of the operators around the linear layers: norm_rope.cu, paged_attention.cu, prefix_attention.cu,
// cache_read.cu, attention.cu, adapter.cu, logprobs.cu, int4.cu.  The public contract is include/ck_int8.h.
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

// Groups of sequences that share the keys of a prefix (count == 0: there are none): sequences
// cu[i] .. cu[i + 1] - 1 stand behind prefix i.
struct SharedPrefixes {
    const int32_t* table;  // [count, max_blocks] pages
    int64_t max_blocks;
    const int32_t* lens;   // [count]
    const int32_t* cu;     // [count + 1]
    int64_t count;
    int64_t max_len;       // max_blocks * page_size
#ifdef __CUDACC__
    // the prefix of sequence b, -1: none (bounds ascending)
    __device__ __forceinline__ int of(int64_t b) const
    {
        int64_t lo = -1, hi = count;  // the last bound <= b
        while (lo < hi) {
            const int64_t mid = (lo + hi + 1) >> 1;
            if (__ldg(cu + mid) <= b)
                lo = mid;
            else
                hi = mid - 1;
        }
        return lo == count ? -1 : (int)lo;
    }
    // by a whole warp: whether bounds descend or leave 0 .. batch
    __device__ __forceinline__ bool bad_groups(int64_t batch) const
    {
        bool bad = false;
        for (int64_t i = threadIdx.x & 31; i <= count; i += 32) {
            const int64_t c = __ldg(cu + i);
            bad |= c < 0 || c > batch || (i > 0 && c < __ldg(cu + i - 1));
        }
        return __any_sync(0xffffffffu, bad);
    }
#endif
};

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
    SharedPrefixes shared;
    // behind prefixes, the shared part in pieces: theirs (nullptr: not so), the blocks that compute them,
    // room for the sums over own keys, whether blocks share segments of these
    float* pieces;
    int piece_blocks;
    float* own_sums;
    bool own_split;
};
// by query heads per kv head and the most keys a sequence can have
size_t paged_attention_workspace(int group, int dim, int64_t max_len);
int paged_attention_launches(const PagedAttention& p);  // kernels that the call enqueues
cudaError_t launch_paged_attention(const PagedAttention& p, const DeviceInfo& dev, cudaStream_t s);

// Attention behind shared prefixes (p.shared.count >= 1).
size_t prefix_attention_workspace(int64_t batch, int group, int kv_heads, int dim, int64_t prefixes, int64_t max_prefix_len,
                                  int64_t max_len);
int prefix_attention_launches(const PagedAttention& p);
cudaError_t launch_prefix_attention(PagedAttention p, const DeviceInfo& dev, cudaStream_t s, std::string* why);
cudaError_t launch_prefix_pieces(const PagedAttention& p, float* parts, const DeviceInfo& dev, cudaStream_t s,
                                 std::string* why);

// Rows of the cache back as contiguous 16-bit keys and values.
struct CacheRead {
    KvCache cache;
    const int32_t* block_table;
    int64_t max_blocks;
    const int32_t* cu;  // [batch + 1] bounds of the sequences' rows
    int64_t batch, total;
    bool f16;
    void *k_out, *v_out;  // [total, heads, dim]
};
cudaError_t launch_cache_read(const CacheRead& p, const DeviceInfo& dev, cudaStream_t s);

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

struct AdapterLinear {
    const void *x, *a, *b;   // [M, K], [adapters, rank, K], [adapters, N, rank]
    const int32_t* index;    // [M], negative: none
    const float* scaling;    // [adapters] or nullptr
    const void* residual;    // out type [M, N] or nullptr
    void* y;
    int64_t M, N, K, adapters;
    int rank;
    bool f16;
    int out_dtype;
    void* workspace;
};
size_t adapter_workspace(int64_t M, int64_t N, int64_t K, int rank);
cudaError_t launch_adapter_linear(const AdapterLinear& p, const DeviceInfo& dev, cudaStream_t s, std::string* why);

struct TokenLogprobs {
    const void* logits;
    int64_t stride;         // elements between rows
    const int32_t* tokens;  // [rows] or nullptr
    int64_t rows, vocab;
    int dtype;              // ck_dtype_t
    float scale;
    int top;
    float *logprob, *entropy, *lse;  // [rows], each or nullptr
    float* top_logprob;              // [rows, top]
    int32_t* top_index;
    void* workspace;
};
size_t logprobs_workspace(int64_t rows, int64_t vocab, int top);
int logprobs_launches(const TokenLogprobs& p);  // kernels that the call enqueues
cudaError_t launch_token_logprobs(const TokenLogprobs& p, const DeviceInfo& dev, cudaStream_t s);

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
