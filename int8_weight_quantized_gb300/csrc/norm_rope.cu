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
// contiguous).  A head is shared by dim / 8 of LANES = 8, 16 or 32 lanes, 8 values each, as two
// runs of 4 (8-byte loads and stores): for rotation by halves the runs are the two halves of 4
// pairs, so that no value has to cross lanes (as one run of 8 they took 8 shuffles a head).  A
// group of lanes takes up to HEADS_PER heads of ONE token, one after the other, so the token's
// angles and the weights are read once and kept in registers.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_common.cuh"
#include "transformer.h"

namespace ck {
namespace {

constexpr int WARPS = 4;
constexpr int HEADS_PER = 4;  // heads a lane group takes, one after the other

template <class E>
__device__ __forceinline__ void unpack4(const uint2& r, float* v)
{
    const float2 a = E::to2(r.x), b = E::to2(r.y);
    v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
}

template <class E>
__device__ __forceinline__ uint2 pack4(const float* v)
{
    return make_uint2(E::pack2(v[0], v[1]), E::pack2(v[2], v[3]));
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
    const bool in = lane * 8 < p.dim;       // dim % 8 == 0: a lane is all in or all out
    const bool rotated = lane * 8 < p.rot;  // rot % 16 == 0, likewise
    const int half = p.rot / 2;
    // the lane's two runs of 4 values
    const bool halves = rotated && !p.interleaved;
    const int d0 = halves ? lane * 4 : lane * 8;
    const int d1 = halves ? half + lane * 4 : d0 + 4;

    // the heads' loads first: they are in flight while the position and its angles arrive
    const T* src = static_cast<const T*>(p.qkv) + token * p.qkv_stride + (int64_t)h0 * p.dim;
    uint2 raw[HEADS_PER][2];
#pragma unroll
    for (int j = 0; j < HEADS_PER; ++j) {
        const bool load = in && h0 + j < heads;
        raw[j][0] = load ? __ldcs(reinterpret_cast<const uint2*>(src + j * p.dim + d0)) : make_uint2(0, 0);
        raw[j][1] = load ? __ldcs(reinterpret_cast<const uint2*>(src + j * p.dim + d1)) : make_uint2(0, 0);
    }

    // the token's angles for the lane's 4 pairs, and where it goes in the cache
    float cs[4], sn[4];
    bool bad = false;
    if (p.rot > 0 && h0 < p.q_heads + p.kv_heads) {
        const int64_t pos = __ldg(p.positions + token);
        bad = pos < 0 || pos >= p.max_pos;
        if (rotated && !bad) {
            const float* row = p.cos_sin + pos * p.rot + lane * 4;
            const float4 c = __ldg(reinterpret_cast<const float4*>(row));
            const float4 s = __ldg(reinterpret_cast<const float4*>(row + half));
            cs[0] = c.x, cs[1] = c.y, cs[2] = c.z, cs[3] = c.w;
            sn[0] = s.x, sn[1] = s.y, sn[2] = s.z, sn[3] = s.w;
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

    float w[8];           // the weights of queries or keys, whichever the last head was
    int w_of = -1;
    const float per_dim = 1.0f / (float)p.dim;
#pragma unroll
    for (int j = 0; j < HEADS_PER; ++j) {
        const int h = h0 + j;
        if (h >= heads)
            break;
        const bool is_v = h >= p.q_heads + p.kv_heads;
        const bool is_q = h < p.q_heads;
        float v[8];
        unpack4<E>(raw[j][0], v);
        unpack4<E>(raw[j][1], v + 4);
        if (!is_v) {
            if (p.norm) {
                if (w_of != (int)is_q) {
                    w_of = is_q;
                    const T* weight = static_cast<const T*>(is_q ? p.q_weight : p.k_weight);
                    if (weight != nullptr && in) {
                        unpack4<E>(__ldg(reinterpret_cast<const uint2*>(weight + d0)), w);
                        unpack4<E>(__ldg(reinterpret_cast<const uint2*>(weight + d1)), w + 4);
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            w[i] = 1.0f;
                    }
                }
                float sum = 0.0f;
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    sum = fmaf(v[i], v[i], sum);
#pragma unroll
                for (int o = LANES / 2; o; o >>= 1)
                    sum += __shfl_xor_sync(mask, sum, o);
                const float inv = rsqrtf(fmaf(sum, per_dim, p.eps));  // within 2 units of 2^-24
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[i] = v[i] * inv * w[i];
            }
            if (rotated && !bad) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float& a = p.interleaved ? v[2 * i] : v[i];
                    float& b = p.interleaved ? v[2 * i + 1] : v[4 + i];
                    const float x = a * cs[i] - b * sn[i];
                    b = b * cs[i] + a * sn[i];
                    a = x;
                }
            }
            if (bad)
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    v[i] = NAN;
        }
        // two runs of four values of a row
        auto store16 = [&](void* base, int64_t row) {
            T* dst = static_cast<T*>(base) + row * p.dim;
            *reinterpret_cast<uint2*>(dst + d0) = pack4<E>(v);
            *reinterpret_cast<uint2*>(dst + d1) = pack4<E>(v + 4);
        };
        if (is_q) {
            if (in)
                store16(p.q_out, token * p.q_heads + h);
            continue;
        }
        const int hk = h - p.q_heads - (is_v ? p.kv_heads : 0);
        if (!is_v && p.k_out != nullptr && in)
            store16(p.k_out, token * p.kv_heads + hk);
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
            if (in) {
                int8_t* at = static_cast<int8_t*>(dst) + row * p.dim;
                *reinterpret_cast<uint32_t*>(at + d0) = c[0];
                *reinterpret_cast<uint32_t*>(at + d1) = c[1];
            }
            if (lane == 0)
                (is_v ? p.cache.v_scale : p.cache.k_scale)[row] = scale;
        } else if (in) {
            store16(dst, row);
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
