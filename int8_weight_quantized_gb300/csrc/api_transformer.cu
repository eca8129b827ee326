// api_transformer.cu -- the extern "C" boundary of the operators around the linear layers:
// argument checks, device check and launch of each.
#include <algorithm>
#include <cmath>
#include <string>

#include "api_common.h"
#include "transformer.h"

namespace ck {
namespace {

constexpr int64_t kMaxCount = 0x7FFFFFFF;  // grids, lengths and row counts are 32-bit

bool valid_16bit(int dtype)
{
    return dtype == CK_OUT_BF16 || dtype == CK_OUT_F16;
}

int check_heads(int64_t q_heads, int64_t kv_heads)
{
    if (q_heads < 1 || kv_heads < 1 || q_heads > 65536 || kv_heads > 65536 || q_heads % kv_heads != 0)
        return fail(CK_ERR_INVALID_ARG,
                    "q_heads must be a multiple of kv_heads, both in 1..65536 (got q_heads=%lld kv_heads=%lld)",
                    (long long)q_heads, (long long)kv_heads);
    return CK_OK;
}

int check_attention_dim(int64_t head_dim)
{
    if (head_dim != 64 && head_dim != 128)
        return fail(CK_ERR_INVALID_ARG, "head_dim must be 64 or 128 (got %lld)", (long long)head_dim);
    return CK_OK;
}

int check_dtype(int dtype)
{
    if (!valid_16bit(dtype))
        return fail(CK_ERR_INVALID_ARG, "dtype must be 0 (bf16) or 1 (fp16), got %d", dtype);
    return CK_OK;
}

int check_mask(int64_t window, int64_t sinks)
{
    if (window < 0 || sinks < 0)
        return fail(CK_ERR_INVALID_ARG, "window and sinks must be >= 0 (got window=%lld sinks=%lld)",
                    (long long)window, (long long)sinks);
    return CK_OK;
}

int check_stride(const char* name, int64_t stride, int64_t least)
{
    if (stride < least || stride % 8 != 0)
        return fail(CK_ERR_INVALID_ARG, "%s must be a multiple of 8 and at least %lld (got %lld)", name,
                    (long long)least, (long long)stride);
    return CK_OK;
}

// Check a cache description against the heads and element type that read or fill it.
int check_cache(const ck_kv_cache_t* c, int64_t kv_heads, int64_t head_dim, int dtype, KvCache* out)
{
    if (c->kv_heads != kv_heads || c->head_dim != head_dim)
        return fail(CK_ERR_INVALID_ARG, "cache holds %lld heads of %lld values, expected %lld of %lld",
                    (long long)c->kv_heads, (long long)c->head_dim, (long long)kv_heads, (long long)head_dim);
    if (c->num_pages < 1 || c->page_size < 1 || c->page_size > kMaxCount || c->num_pages > kMaxCount)
        return fail(CK_ERR_INVALID_ARG, "cache num_pages and page_size must be in 1..2^31-1 (got %lld and %lld)",
                    (long long)c->num_pages, (long long)c->page_size);
    if (c->num_pages * c->page_size > 0xFFFFFFFFll / kv_heads)
        return fail(CK_ERR_INVALID_ARG, "cache rows (pages * page_size * heads) must be below 2^32");
    if (c->dtype != CK_KV_INT8 && c->dtype != (dtype == CK_OUT_F16 ? CK_KV_F16 : CK_KV_BF16))
        return fail(CK_ERR_INVALID_ARG, "cache dtype %d is neither int8 (2) nor the activations' type (%d)", c->dtype,
                    dtype);
    CK_REQUIRE_PTR(c->k);
    CK_REQUIRE_PTR(c->v);
    if (c->dtype == CK_KV_INT8) {
        CK_REQUIRE_PTR(c->k_scale);
        CK_REQUIRE_PTR(c->v_scale);
    }
    out->k = c->k;
    out->v = c->v;
    out->k_scale = c->k_scale;
    out->v_scale = c->v_scale;
    out->num_pages = c->num_pages;
    out->page_size = (int)c->page_size;
    out->heads = (int)kv_heads;
    out->dim = (int)head_dim;
    out->dtype = c->dtype;
    return CK_OK;
}

#define CK_CHECK(call)            \
    do {                          \
        const int st_ = (call);   \
        if (st_ != CK_OK)         \
            return st_;           \
    } while (0)

// index arrays: aligned like their elements, so that slices of them qualify
#define CK_REQUIRE_INDEX(p)                                                                     \
    do {                                                                                        \
        if ((p) == nullptr)                                                                     \
            return fail(CK_ERR_INVALID_ARG, "%s must not be NULL", #p);                         \
        if (reinterpret_cast<uintptr_t>(p) % sizeof(*(p)) != 0)                                 \
            return fail(CK_ERR_INVALID_ARG, "%s must be aligned like its elements", #p);        \
    } while (0)

#define CK_OPTIONAL_PTR(p)                                                      \
    do {                                                                        \
        if ((p) != nullptr && !aligned16(p))                                    \
            return fail(CK_ERR_INVALID_ARG, "%s must be 16-byte aligned", #p);  \
    } while (0)

}  // namespace
}  // namespace ck

using namespace ck;

extern "C" {

int ck_qk_norm_rope(const void* qkv, int64_t qkv_stride, int64_t tokens, int64_t q_heads, int64_t kv_heads,
                    int64_t head_dim, int dtype, int norm, const void* q_weight, const void* k_weight, float eps,
                    int64_t rot_dim, int interleaved, const int32_t* positions, const float* cos_sin, int64_t max_pos,
                    void* q_out, void* k_out, const ck_kv_cache_t* cache, const int64_t* slots, void* stream)
{
    CK_CHECK(check_dtype(dtype));
    CK_CHECK(check_heads(q_heads, kv_heads));
    if (head_dim < 8 || head_dim > 256 || head_dim % 8 != 0)
        return fail(CK_ERR_INVALID_ARG, "head_dim must be a multiple of 8 in 8..256 (got %lld)", (long long)head_dim);
    if (rot_dim < 0 || rot_dim > head_dim || rot_dim % 16 != 0)
        return fail(CK_ERR_INVALID_ARG, "rot_dim must be a multiple of 16 in 0..head_dim (got %lld)",
                    (long long)rot_dim);
    if ((norm != 0 && norm != 1) || (interleaved != 0 && interleaved != 1))
        return fail(CK_ERR_INVALID_ARG, "norm and interleaved must be 0 or 1 (got %d and %d)", norm, interleaved);
    if (norm && !(eps >= 0.0f && std::isfinite(eps)))
        return fail(CK_ERR_INVALID_ARG, "eps must be finite and >= 0");
    const int64_t heads = q_heads + 2 * kv_heads;
    CK_CHECK(check_stride("qkv_stride", qkv_stride, heads * head_dim));
    if (tokens < 0 || tokens > kMaxCount / heads)
        return fail(CK_ERR_INVALID_ARG, "tokens must be >= 0 and tokens * heads below 2^31 (got tokens=%lld)",
                    (long long)tokens);
    if (rot_dim > 0 && (max_pos < 1 || max_pos > kMaxCount))
        return fail(CK_ERR_INVALID_ARG, "max_pos must be in 1..2^31-1 (got %lld)", (long long)max_pos);
    if (tokens == 0)
        return CK_OK;
    NormRope p{};
    CK_REQUIRE_PTR(qkv);
    CK_REQUIRE_PTR(q_out);
    if (rot_dim > 0) {
        CK_REQUIRE_INDEX(positions);
        CK_REQUIRE_PTR(cos_sin);
    }
    CK_OPTIONAL_PTR(q_weight);
    CK_OPTIONAL_PTR(k_weight);
    CK_OPTIONAL_PTR(k_out);
    if (cache != nullptr) {
        CK_CHECK(check_cache(cache, kv_heads, head_dim, dtype, &p.cache));
        CK_REQUIRE_INDEX(slots);
    }
    DeviceInfo dev;
    CK_CHECK(check_device(&dev));
    p.qkv = qkv;
    p.qkv_stride = qkv_stride;
    p.tokens = tokens;
    p.q_heads = (int)q_heads;
    p.kv_heads = (int)kv_heads;
    p.dim = (int)head_dim;
    p.rot = (int)rot_dim;
    p.f16 = dtype == CK_OUT_F16;
    p.norm = norm != 0;
    p.interleaved = interleaved != 0;
    p.q_weight = q_weight;
    p.k_weight = k_weight;
    p.eps = eps;
    p.positions = positions;
    p.cos_sin = cos_sin;
    p.max_pos = max_pos;
    p.q_out = q_out;
    p.k_out = k_out;
    p.slots = slots;
    log_shape("qk_norm_rope", tokens, heads, head_dim, p.cache.k ? 1 + p.cache.dtype : 0, "one pass");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    ProfScope ps(kProfNormRope, 1, s);
    const cudaError_t e = launch_norm_rope(p, dev, s);
    return e == cudaSuccess ? CK_OK : cuda_fail(e, "ck_qk_norm_rope launch");
}

size_t ck_paged_attention_workspace_size(int64_t batch, int64_t q_heads, int64_t kv_heads, int64_t head_dim,
                                         int64_t max_len)
{
    if (batch < 0 || max_len < 0 || q_heads < 1 || kv_heads < 1 || head_dim < 1 || q_heads > 65536 || kv_heads > 65536 ||
        head_dim > 256)
        return 0;
    return paged_attention_workspace((int)(q_heads / kv_heads), (int)head_dim, max_len);
}

int ck_paged_attention(const void* q, int64_t q_stride, const ck_kv_cache_t* cache, const int32_t* block_table,
                       int64_t max_blocks, const int32_t* seq_lens, int64_t batch, int64_t q_heads, int dtype,
                       float scale, int64_t window, int64_t sinks, void* out, float* lse, void* workspace,
                       size_t workspace_bytes, void* stream)
{
    CK_CHECK(check_dtype(dtype));
    if (cache == nullptr)
        return fail(CK_ERR_INVALID_ARG, "cache must not be NULL");
    CK_CHECK(check_heads(q_heads, cache->kv_heads));
    CK_CHECK(check_attention_dim(cache->head_dim));
    CK_CHECK(check_mask(window, sinks));
    CK_CHECK(check_stride("q_stride", q_stride, q_heads * cache->head_dim));
    if (!std::isfinite(scale))
        return fail(CK_ERR_INVALID_ARG, "scale must be finite");
    if (batch < 0 || batch > kMaxCount / q_heads)
        return fail(CK_ERR_INVALID_ARG, "batch must be >= 0 and batch * q_heads below 2^31 (got batch=%lld)",
                    (long long)batch);
    if (max_blocks < 1 || cache->page_size < 1 || cache->page_size > kMaxCount ||
        max_blocks > kMaxCount / cache->page_size)
        return fail(CK_ERR_INVALID_ARG, "max_blocks and page_size must be >= 1, their product below 2^31 (got %lld, %lld)",
                    (long long)max_blocks, (long long)cache->page_size);
    PagedAttention p{};
    if (batch == 0)
        return CK_OK;
    CK_CHECK(check_cache(cache, cache->kv_heads, cache->head_dim, dtype, &p.cache));
    CK_REQUIRE_PTR(q);
    CK_REQUIRE_INDEX(block_table);
    CK_REQUIRE_INDEX(seq_lens);
    CK_REQUIRE_PTR(out);
    CK_OPTIONAL_PTR(lse);
    const size_t need =
        paged_attention_workspace((int)q_heads / p.cache.heads, p.cache.dim, max_blocks * p.cache.page_size);
    if (need > 0) {
        CK_REQUIRE_PTR(workspace);
        if (workspace_bytes < need)
            return fail(CK_ERR_INVALID_ARG, "workspace too small: %zu bytes given, %zu needed", workspace_bytes, need);
    }
    DeviceInfo dev;
    CK_CHECK(check_device(&dev));
    p.q = q;
    p.q_stride = q_stride;
    p.block_table = block_table;
    p.max_blocks = max_blocks;
    p.seq_lens = seq_lens;
    p.batch = batch;
    p.q_heads = (int)q_heads;
    p.f16 = dtype == CK_OUT_F16;
    p.scale = scale;
    p.window = window;
    p.sinks = sinks;
    p.page_shift = -1;
    if ((p.cache.page_size & (p.cache.page_size - 1)) == 0)
        for (p.page_shift = 0; (1 << p.page_shift) < p.cache.page_size;)
            ++p.page_shift;
    p.out = out;
    p.lse = lse;
    p.workspace = workspace;
    log_shape("paged_attention", batch, q_heads, p.cache.dim, p.cache.dtype, "split over the length, joined");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    ProfScope ps(kProfAttention, paged_attention_launches(p), s);
    const cudaError_t e = launch_paged_attention(p, dev, s);
    return e == cudaSuccess ? CK_OK : cuda_fail(e, "ck_paged_attention launch");
}

int ck_attention(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                 const int32_t* cu_q, const int32_t* cu_k, int64_t batch, int64_t total_q, int64_t total_k,
                 int64_t q_heads, int64_t kv_heads, int64_t head_dim, int dtype, float scale, int causal,
                 int64_t window, int64_t sinks, void* out, float* lse, void* stream)
{
    CK_CHECK(check_dtype(dtype));
    CK_CHECK(check_heads(q_heads, kv_heads));
    CK_CHECK(check_attention_dim(head_dim));
    CK_CHECK(check_mask(window, sinks));
    if (causal != 0 && causal != 1)
        return fail(CK_ERR_INVALID_ARG, "causal must be 0 or 1 (got %d)", causal);
    if (!causal && window != 0)
        return fail(CK_ERR_INVALID_ARG, "a window needs causal = 1");
    CK_CHECK(check_stride("q_stride", q_stride, q_heads * head_dim));
    CK_CHECK(check_stride("k_stride", k_stride, kv_heads * head_dim));
    CK_CHECK(check_stride("v_stride", v_stride, kv_heads * head_dim));
    if (!std::isfinite(scale))
        return fail(CK_ERR_INVALID_ARG, "scale must be finite");
    if (batch < 0 || total_q < 0 || total_k < 0 || batch > kMaxCount / q_heads || total_q > kMaxCount / q_heads ||
        total_k > kMaxCount)
        return fail(CK_ERR_INVALID_ARG,
                    "batch, total_q and total_k must be >= 0, and with the heads below 2^31 (got %lld, %lld, %lld)",
                    (long long)batch, (long long)total_q, (long long)total_k);
    if (batch == 0 || total_q == 0)
        return CK_OK;
    CK_REQUIRE_PTR(q);
    if (total_k > 0) {  // without keys every query gets zeros; k and v may be NULL
        CK_REQUIRE_PTR(k);
        CK_REQUIRE_PTR(v);
    }
    CK_REQUIRE_INDEX(cu_q);
    CK_REQUIRE_INDEX(cu_k);
    CK_REQUIRE_PTR(out);
    CK_OPTIONAL_PTR(lse);
    DeviceInfo dev;
    CK_CHECK(check_device(&dev));
    PromptAttention p{};
    p.q = q;
    p.k = k;
    p.v = v;
    p.q_stride = q_stride;
    p.k_stride = k_stride;
    p.v_stride = v_stride;
    p.cu_q = cu_q;
    p.cu_k = cu_k;
    p.batch = batch;
    p.total_q = total_q;
    p.total_k = total_k;
    p.q_heads = (int)q_heads;
    p.kv_heads = (int)kv_heads;
    p.dim = (int)head_dim;
    p.f16 = dtype == CK_OUT_F16;
    p.causal = causal != 0;
    p.scale = scale;
    p.window = window;
    p.sinks = sinks;
    p.out = out;
    p.lse = lse;
    log_shape("attention", total_q, q_heads, head_dim, causal, "whole prompts");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    std::string why;
    cudaError_t e;
    {
        ProfScope ps(kProfAttention, 1, s);
        e = launch_attention(p, dev, s, &why);
    }
    if (e != cudaSuccess)
        return why.empty() ? cuda_fail(e, "ck_attention launch") : fail(CK_ERR_CUDA, "%s", why.c_str());
    return CK_OK;
}

static int check_int4_shape(int64_t N, int64_t K)
{
    if (N < 1 || K < 1 || N > kMaxCount || K > kMaxCount)
        return fail(CK_ERR_INVALID_ARG, "N and K must be in 1..2^31-1 (got N=%lld K=%lld)", (long long)N, (long long)K);
    if (N % 8 != 0)
        return fail(CK_ERR_INVALID_ARG, "N must be a multiple of 8 (got %lld)", (long long)N);
    if (K % 128 != 0)
        return fail(CK_ERR_INVALID_ARG, "K must be a multiple of 128 (got %lld)", (long long)K);
    if (N > (int64_t)kMaxCount * 256 / K)
        return fail(CK_ERR_INVALID_ARG, "N * K must be below 2^39 (got N=%lld K=%lld)", (long long)N, (long long)K);
    return CK_OK;
}

static int check_group(int64_t group, int64_t K)
{
    if (group != 32 && group != 64 && group != 128 && group != 256)
        return fail(CK_ERR_INVALID_ARG, "group must be 32, 64, 128 or 256 (got %lld)", (long long)group);
    if (K % group != 0)
        return fail(CK_ERR_INVALID_ARG, "K must be a multiple of group (got K=%lld group=%lld)", (long long)K,
                    (long long)group);
    return CK_OK;
}

int ck_int4_prepare_weight(const float* W, int64_t N, int64_t K, int64_t group, uint32_t* w4, void* w_scale,
                           void* stream)
{
    CK_CHECK(check_int4_shape(N, K));
    CK_CHECK(check_group(group, K));
    CK_REQUIRE_PTR(W);
    CK_REQUIRE_PTR(w4);
    CK_REQUIRE_PTR(w_scale);
    DeviceInfo dev;
    CK_CHECK(check_device(&dev));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    ProfScope ps(kProfInt4, 1, s);
    const cudaError_t e = launch_int4_weight(W, N, K, (int)group, w4, w_scale, dev, s);
    return e == cudaSuccess ? CK_OK : cuda_fail(e, "ck_int4_prepare_weight launch");
}

int ck_int4_pack(const int8_t* codes, int64_t N, int64_t K, uint32_t* w4, void* stream)
{
    CK_CHECK(check_int4_shape(N, K));
    CK_REQUIRE_PTR(codes);
    CK_REQUIRE_PTR(w4);
    DeviceInfo dev;
    CK_CHECK(check_device(&dev));
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    ProfScope ps(kProfInt4, 1, s);
    const cudaError_t e = launch_int4_pack(codes, N, K, w4, dev, s);
    return e == cudaSuccess ? CK_OK : cuda_fail(e, "ck_int4_pack launch");
}

int ck_int4_linear(const void* x, const uint32_t* w4, const void* w_scale, const void* bias, const void* residual,
                   void* y, int64_t M, int64_t N, int64_t K, int64_t group, int dtype, int out_dtype, void* stream)
{
    CK_CHECK(check_dtype(dtype));
    if (out_dtype != CK_OUT_BF16 && out_dtype != CK_OUT_F16 && out_dtype != CK_OUT_F32)
        return fail(CK_ERR_INVALID_ARG, "out_dtype must be 0 (bf16), 1 (fp16) or 2 (fp32), got %d", out_dtype);
    CK_CHECK(check_int4_shape(N, K));
    CK_CHECK(check_group(group, K));
    if (M < 0 || M > (1 << 19))
        return fail(CK_ERR_INVALID_ARG, "M must be in 0..524288 (got %lld)", (long long)M);
    if (M == 0)
        return CK_OK;
    CK_REQUIRE_PTR(x);
    CK_REQUIRE_PTR(w4);
    CK_REQUIRE_PTR(w_scale);
    CK_REQUIRE_PTR(y);
    CK_OPTIONAL_PTR(bias);
    CK_OPTIONAL_PTR(residual);
    DeviceInfo dev;
    CK_CHECK(check_device(&dev));
    Int4Linear p{};
    p.x = x;
    p.w4 = w4;
    p.w_scale = w_scale;
    p.bias = bias;
    p.residual = residual;
    p.y = y;
    p.M = M;
    p.N = N;
    p.K = K;
    p.group = (int)group;
    p.f16 = dtype == CK_OUT_F16;
    p.out_dtype = out_dtype;
    log_shape("int4_linear", M, N, K, (int)group, "4-bit weights, group scales");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    ProfScope ps(kProfInt4, 1, s);
    const cudaError_t e = launch_int4_linear(p, dev, s);
    return e == cudaSuccess ? CK_OK : cuda_fail(e, "ck_int4_linear launch");
}

}  // extern "C"
