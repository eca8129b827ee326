// norm_rope.cu -- what stands between the QKV projection and attention, in one pass over the
// projection's output: the RMS norm of every query and key head, the rotation by position,
// and the keys' and values' way into the paged cache (16-bit, or int8 in the library's own
// quantize rule).
//
//   n    = x * rsqrt(mean(x^2) + eps) * w          fp32, over the head's `dim` values
//   y_a  = n_a cos - n_b sin,  y_b = n_b cos + n_a sin   for each pair (a, b) of the first
//          `rot` values: (i, i + rot/2), or (2i, 2i + 1) when interleaved; the rest pass
//   int8 cache rows: scale = max|y| / 127, code = clamp(rint(y / scale), -127, 127), from the
//          fp32 y, which is never rounded to 16 bits on the way
//
// Bound: HBM, each value read once and written once (twice where the keys are also kept
// contiguous).  A head is shared by LANES = 8, 16 or 32 lanes of 8 values (one 16-byte load
// and store each).  A group of lanes takes up to HEADS_PER heads of ONE token, one after the
// other, so the token's cosines and sines are read once and kept in registers: read again
// for each head they would be four times the head's own bytes in L1 traffic.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_common.cuh"
#include "transformer.h"

namespace ck {
namespace {

constexpr int WARPS = 4;
constexpr int HEADS_PER = 4;  // heads a lane group takes, one after the other

template <class E>
__device__ __forceinline__ void unpack8(const uint4& r, float (&v)[8])
{
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = E::to2(w[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
    }
}

template <class E>
__device__ __forceinline__ uint4 pack8(const float (&v)[8])
{
    return make_uint4(E::pack2(v[0], v[1]), E::pack2(v[2], v[3]), E::pack2(v[4], v[5]), E::pack2(v[6], v[7]));
}

template <class E, int LANES>
__global__ void __launch_bounds__(WARPS * 32) norm_rope_kernel(const NormRope p, unsigned int* err)
{
    griddep_wait();
    using T = typename E::T;
    constexpr int GROUPS = WARPS * 32 / LANES;
    const int lane = threadIdx.x % LANES;
    const int group = threadIdx.x / LANES;
    const int heads = p.q_heads + 2 * p.kv_heads;
    const int chunks = (heads + HEADS_PER - 1) / HEADS_PER;
    const uint32_t unit = blockIdx.x * GROUPS + group;  // tokens * heads is below 2^31
    const int64_t token = unit / (uint32_t)chunks;
    if (token >= p.tokens)
        return;  // whole lane groups leave together; shuffles below name only their group
    const uint32_t mask = LANES == 32 ? 0xffffffffu : ((1u << LANES) - 1u) << ((threadIdx.x & 31) / LANES * LANES);
    const int h0 = (int)(unit - token * chunks) * HEADS_PER;
    const int d0 = lane * 8;
    const bool in = d0 < p.dim;       // dim % 8 == 0: a lane is all in or all out
    const bool rotated = d0 < p.rot;  // rot % 16 == 0, likewise
    const int half = p.rot / 2;

    // the heads' loads first: they are in flight while the position and its angles arrive
    const T* src = static_cast<const T*>(p.qkv) + token * p.qkv_stride;
    uint4 raw[HEADS_PER];
#pragma unroll
    for (int j = 0; j < HEADS_PER; ++j)
        if (in && h0 + j < heads)
            raw[j] = __ldcs(reinterpret_cast<const uint4*>(src + (int64_t)(h0 + j) * p.dim + d0));
        else
            raw[j] = make_uint4(0, 0, 0, 0);

    // the token's angles for this lane's 8 values, and where it goes in the cache
    float cs[8], sn[8];
    bool bad = false;
    if (p.rot > 0 && h0 < p.q_heads + p.kv_heads) {
        const int64_t pos = __ldg(p.positions + token);
        bad = pos < 0 || pos >= p.max_pos;
        if (rotated && !bad) {
            const float* row = p.cos_sin + pos * p.rot;
            if (p.interleaved) {
                const float4 c = __ldg(reinterpret_cast<const float4*>(row + d0 / 2));
                const float4 s = __ldg(reinterpret_cast<const float4*>(row + half + d0 / 2));
                cs[0] = cs[1] = c.x, cs[2] = cs[3] = c.y, cs[4] = cs[5] = c.z, cs[6] = cs[7] = c.w;
                sn[0] = sn[1] = s.x, sn[2] = sn[3] = s.y, sn[4] = sn[5] = s.z, sn[6] = sn[7] = s.w;
            } else {
                const int i0 = d0 < half ? d0 : d0 - half;
#pragma unroll
                for (int i = 0; i < 8; i += 4) {
                    const float4 c = __ldg(reinterpret_cast<const float4*>(row + i0 + i));
                    const float4 s = __ldg(reinterpret_cast<const float4*>(row + half + i0 + i));
                    cs[i] = c.x, cs[i + 1] = c.y, cs[i + 2] = c.z, cs[i + 3] = c.w;
                    sn[i] = s.x, sn[i + 1] = s.y, sn[i + 2] = s.z, sn[i + 3] = s.w;
                }
            }
        }
    }
    int64_t page = -1, off = 0;
    if (p.cache.k != nullptr && h0 + HEADS_PER > p.q_heads) {
        const int64_t slot = __ldg(p.slots + token);
        const bool outside = slot >= p.cache.num_pages * p.cache.page_size;
        if (slot >= 0 && !outside) {  // below 2^32 then: the cache's rows are
            const uint32_t pg = (uint32_t)slot / (uint32_t)p.cache.page_size;
            page = pg;
            off = slot - (int64_t)pg * p.cache.page_size;
        }
        if (outside && lane == 0)
            atomicOr(err, kErrIndex);
    }
    if (bad && lane == 0)
        atomicOr(err, kErrIndex);

#pragma unroll
    for (int j = 0; j < HEADS_PER; ++j) {
        const int h = h0 + j;
        if (h >= heads)
            break;
        const bool is_v = h >= p.q_heads + p.kv_heads;
        const bool is_q = h < p.q_heads;
        float v[8];
        unpack8<E>(raw[j], v);
        if (!is_v) {
            if (p.norm) {
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    sum = fmaf(v[i], v[i], sum);
#pragma unroll
                for (int o = LANES / 2; o; o >>= 1)
                    sum += __shfl_xor_sync(mask, sum, o);
                const float inv = 1.0f / sqrtf(sum / (float)p.dim + p.eps);
                float w[8];
                const void* weight = is_q ? p.q_weight : p.k_weight;
                if (weight != nullptr && in)
                    unpack8<E>(__ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(weight) + d0)), w);
                else
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        w[i] = 1.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[i] = v[i] * inv * w[i];
            }
            if (p.rot > 0) {
                float other[8];
                if (p.interleaved) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        other[i] = v[i ^ 1];
                } else {
                    // the pair's other half lives rot / 16 lanes away (rot % 16 == 0)
                    const int step = p.rot / 16;
                    const int from = rotated ? (d0 < half ? lane + step : lane - step) : lane;
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        other[i] = __shfl_sync(mask, v[i], from, LANES);
                }
                if (rotated && !bad) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const bool first = p.interleaved ? (i & 1) == 0 : d0 < half;
                        v[i] = first ? v[i] * cs[i] - other[i] * sn[i] : v[i] * cs[i] + other[i] * sn[i];
                    }
                }
            }
            if (bad)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[i] = NAN;
        }
        if (is_q) {
            if (in)
                *reinterpret_cast<uint4*>(static_cast<T*>(p.q_out) + (token * p.q_heads + h) * p.dim + d0) = pack8<E>(v);
            continue;
        }
        const int hk = h - p.q_heads - (is_v ? p.kv_heads : 0);
        if (!is_v && p.k_out != nullptr && in)
            *reinterpret_cast<uint4*>(static_cast<T*>(p.k_out) + (token * p.kv_heads + hk) * p.dim + d0) = pack8<E>(v);
        if (page < 0)
            continue;
        const int64_t row = (page * p.cache.heads + hk) * p.cache.page_size + off;
        void* dst = is_v ? p.cache.v : p.cache.k;
        if (p.cache.dtype == CK_KV_INT8) {
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                top = fmaxf(top, fabsf(v[i]));
#pragma unroll
            for (int o = LANES / 2; o; o >>= 1)
                top = fmaxf(top, __shfl_xor_sync(mask, top, o));
            const float scale = __fdiv_rn(top, 127.0f);
            uint32_t c[2] = {0, 0};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // v / scale is at most 127 (1 + 2^-23) unless the scale is subnormal: clamp
                const float t = scale > 0.0f ? fminf(fmaxf(rintf(__fdiv_rn(v[i], scale)), -127.0f), 127.0f) : 0.0f;
                c[i >> 2] |= (uint32_t)((int)t & 255) << (8 * (i & 3));
            }
            if (in)
                *reinterpret_cast<uint2*>(static_cast<int8_t*>(dst) + row * p.dim + d0) = make_uint2(c[0], c[1]);
            if (lane == 0)
                (is_v ? p.cache.v_scale : p.cache.k_scale)[row] = scale;
        } else if (in) {
            *reinterpret_cast<uint4*>(static_cast<T*>(dst) + row * p.dim + d0) = pack8<E>(v);
        }
    }
}

template <class E, int LANES>
cudaError_t launch(const NormRope& p, unsigned int* err, cudaStream_t s)
{
    const int64_t chunks = (p.q_heads + 2 * p.kv_heads + HEADS_PER - 1) / HEADS_PER;
    const int64_t per_block = WARPS * 32 / LANES;
    const int64_t blocks = (p.tokens * chunks + per_block - 1) / per_block;
    return launch_pdl(norm_rope_kernel<E, LANES>, dim3((unsigned)blocks), dim3(WARPS * 32), 0, s, p, err);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRope& p, const DeviceInfo& dev, cudaStream_t s)
{
    (void)dev;
    unsigned int* err = nullptr;
    cudaError_t e = device_error_ptr(&err);
    if (e != cudaSuccess)
        return e;
    if (p.dim <= 64)
        return p.f16 ? launch<Fp16, 8>(p, err, s) : launch<Bf16, 8>(p, err, s);
    if (p.dim <= 128)
        return p.f16 ? launch<Fp16, 16>(p, err, s) : launch<Bf16, 16>(p, err, s);
    return p.f16 ? launch<Fp16, 32>(p, err, s) : launch<Bf16, 32>(p, err, s);
}

}  // namespace ck
