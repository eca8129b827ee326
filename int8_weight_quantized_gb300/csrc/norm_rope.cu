// norm_rope.cu -- what stands between the QKV projection and attention, in one pass over the
// projection's output: the RMS norm of every query and key head, the rotation by position,
// and the keys' and values' way into the paged cache (16-bit, or int8 in the library's own
// quantize rule).
//
//   n    = x * rsqrt(mean(x^2) + eps) * w          fp32, over the head's `dim` values
//   y_a  = n_a cos - n_b sin,  y_b = n_b cos + n_a sin   for each pair (a, b) of the first
//          `rot` values: (i, i + rot/2), or (2i, 2i + 1) when interleaved; the rest pass
//   int8 cache rows: scale = max|y| / 127, code = clamp(rint(y / scale), -127, 127), from the
//          fp32 y, which is never rounded to 16 bits on the way; a row that holds a NaN or an
//          infinity, which codes cannot, gets the scale NaN, so that what reads it is NaN
//
// Bound: HBM, each value read once and written once (twice where the keys are also kept
// contiguous).  A head is shared by dim / 8 of LANES = 8, 16 or 32 lanes, 8 values each, as two
// runs of 4 (8-byte loads and stores): for rotation by halves the runs are the two halves of 4
// pairs, so that no value has to cross lanes (as one run of 8 they took 8 shuffles a head).  A
// group of lanes takes up to HEADS_PER heads of one kind (queries, keys or values) of ONE token,
// so that the token's angles and the weights are read once and what depends on the kind is
// settled once, outside the loop over heads: with the kind tested per head the kernel spent
// three quarters of its 237 instructions per two heads on tests and addresses.
//
// Measured (GB300): 8192 tokens of 32 query and 8 key heads of 128, bf16, keys also kept
// contiguous: 45.3 to 45.9 us, 4.9 TB/s, 73% of a copy's bandwidth, interleaved 45.7, into int8 rows
// 62; 4096 tokens of 16 and 4 heads of 256: 23.6 us, 4.4 TB/s; one token 3.0 us (launch).  The
// arithmetic issues in 73% of the cycles, accesses are of 8 bytes, and at the 64 registers that 8
// blocks per SM leave the kernels that rotate spill 24 to 48 bytes a thread (the quantization to
// int8 is a branch of each); which of these sets the time is not settled.  More warps at 48
// registers (10 blocks per SM, 50.8 us) or resident blocks that fetch the next heads while they
// work on these (49 to 56 us at 4 to 6 blocks per SM) were slower.
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

// ROT: 0 no rotation, 1 by halves, 2 interleaved
template <class E, int LANES, int ROT>
__global__ void __launch_bounds__(WARPS * 32, 8) norm_rope_kernel(const NormRope p, unsigned int* err)
{
    griddep_wait();
    using T = typename E::T;
    constexpr int GROUPS = WARPS * 32 / LANES;
    const int lane = threadIdx.x % LANES;
    const uint32_t unit = blockIdx.x * GROUPS + threadIdx.x / LANES;  // tokens * heads is below 2^31
    const uint32_t q_chunks = (p.q_heads + HEADS_PER - 1) / HEADS_PER, kv_chunks = (p.kv_heads + HEADS_PER - 1) / HEADS_PER;
    const uint32_t chunks = q_chunks + 2 * kv_chunks;
    const uint32_t tok = unit / chunks;
    if (tok >= p.tokens)
        return;  // whole lane groups leave together; shuffles below name only their group
    const uint32_t mask = LANES == 32 ? 0xffffffffu : ((1u << LANES) - 1u) << ((threadIdx.x & 31) / LANES * LANES);
    const int64_t token = tok;
    int chunk = (int)(unit - tok * chunks);
    const bool is_q = chunk < (int)q_chunks;
    chunk -= is_q ? 0 : (int)q_chunks;
    const bool is_v = !is_q && chunk >= (int)kv_chunks;
    chunk -= is_v ? (int)kv_chunks : 0;
    const int first = chunk * HEADS_PER;  // head among its kind
    const int count = min(HEADS_PER, (is_q ? p.q_heads : p.kv_heads) - first);

    const bool in = lane * 8 < p.dim;                    // dim % 8 == 0: a lane is all in or all out
    const bool rotated = ROT != 0 && lane * 8 < p.rot;  // rot % 16 == 0, likewise
    const int half = p.rot / 2;
    // the lane's two runs of 4 values
    const int d0 = ROT == 1 && rotated ? lane * 4 : lane * 8;
    const int d1 = ROT == 1 && rotated ? half + lane * 4 : d0 + 4;

    // the heads' loads first: they are in flight while the position and its angles arrive
    const T* src = static_cast<const T*>(p.qkv) + token * p.qkv_stride +
                   (first + (is_q ? 0 : p.q_heads) + (is_v ? p.kv_heads : 0)) * p.dim;
    uint2 raw[HEADS_PER][2];
#pragma unroll
    for (int j = 0; j < HEADS_PER; ++j) {
        const bool load = in && j < count;
        raw[j][0] = load ? __ldcs(reinterpret_cast<const uint2*>(src + j * p.dim + d0)) : make_uint2(0, 0);
        raw[j][1] = load ? __ldcs(reinterpret_cast<const uint2*>(src + j * p.dim + d1)) : make_uint2(0, 0);
    }

    // where keys and values go in the cache: the row of head `first`, heads page_size rows apart
    int64_t row = -1;
    if (!is_q && p.cache.k != nullptr) {
        const int64_t slot = __ldg(p.slots + token);
        const bool outside = slot >= p.cache.num_pages * p.cache.page_size;
        if (slot >= 0 && !outside) {  // below 2^32 then: the cache's rows are
            const uint32_t pg = (uint32_t)slot / (uint32_t)p.cache.page_size;
            const uint32_t off = (uint32_t)slot - pg * (uint32_t)p.cache.page_size;
            row = ((int64_t)pg * p.cache.heads + first) * p.cache.page_size + off;
        } else if (outside && lane == 0) {
            atomicOr(err, kErrIndex);
        }
    }
    void* const cache = is_v ? p.cache.v : p.cache.k;
    const int64_t row_step = (int64_t)p.cache.page_size;
    const bool int8 = p.cache.dtype == CK_KV_INT8;

    if (is_v && !int8) {  // copied as they are
        if (row < 0 || !in)
            return;
        T* dst = static_cast<T*>(cache) + row * p.dim;
#pragma unroll
        for (int j = 0; j < HEADS_PER; ++j) {
            if (j < count) {
                *reinterpret_cast<uint2*>(dst + d0) = raw[j][0];
                *reinterpret_cast<uint2*>(dst + d1) = raw[j][1];
                dst += row_step * p.dim;
            }
        }
        return;
    }

    // the token's angles for the lane's 4 pairs, and the weights
    float cs[4], sn[4], w[8];
    bool bad = false;
    if (ROT != 0 && !is_v) {
        const int64_t pos = __ldg(p.positions + token);
        bad = pos < 0 || pos >= p.max_pos;
        if (bad && lane == 0)
            atomicOr(err, kErrIndex);
        if (rotated && !bad) {
            const float* angles = p.cos_sin + pos * p.rot + lane * 4;
            const float4 c = __ldg(reinterpret_cast<const float4*>(angles));
            const float4 s = __ldg(reinterpret_cast<const float4*>(angles + half));
            cs[0] = c.x, cs[1] = c.y, cs[2] = c.z, cs[3] = c.w;
            sn[0] = s.x, sn[1] = s.y, sn[2] = s.z, sn[3] = s.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                cs[i] = 1.0f, sn[i] = 0.0f;
        }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        w[i] = 1.0f;
    const bool norm = p.norm && !is_v;
    const T* weight = static_cast<const T*>(is_q ? p.q_weight : p.k_weight);
    if (norm && weight != nullptr && in) {
        unpack4<E>(__ldg(reinterpret_cast<const uint2*>(weight + d0)), w);
        unpack4<E>(__ldg(reinterpret_cast<const uint2*>(weight + d1)), w + 4);
    }
    const float per_dim = 1.0f / (float)p.dim;
    // 16-bit rows: queries, or keys kept contiguous, then keys in the cache
    T* out = static_cast<T*>(is_q ? p.q_out : is_v ? nullptr : p.k_out);
    if (out != nullptr)
        out += (token * (is_q ? p.q_heads : p.kv_heads) + first) * p.dim;
    T* cache16 = row >= 0 && !int8 ? static_cast<T*>(cache) + row * p.dim : nullptr;

#pragma unroll
    for (int j = 0; j < HEADS_PER; ++j) {
        if (j >= count)
            break;
        float v[8];
        unpack4<E>(raw[j][0], v);
        unpack4<E>(raw[j][1], v + 4);
        if (norm) {
            float2 sum2 = make_float2(0.0f, 0.0f);
#pragma unroll
            for (int i = 0; i < 8; i += 2)
                sum2 = f2_fma_rn(make_float2(v[i], v[i + 1]), make_float2(v[i], v[i + 1]), sum2);
            float sum = sum2.x + sum2.y;
#pragma unroll
            for (int o = LANES / 2; o; o >>= 1)
                sum += __shfl_xor_sync(mask, sum, o);
            const float inv = rsqrtf(fmaf(sum, per_dim, p.eps));  // within 2 units of 2^-24
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                const float2 n = f2_mul_rn(make_float2(v[i], v[i + 1]), make_float2(inv, inv));
                const float2 y = f2_mul_rn(n, make_float2(w[i], w[i + 1]));
                v[i] = y.x, v[i + 1] = y.y;
            }
        }
        if (ROT == 1 && rotated && !is_v) {
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                const float2 a = make_float2(v[i], v[i + 1]), b = make_float2(v[4 + i], v[5 + i]);
                const float2 c = make_float2(cs[i], cs[i + 1]), s = make_float2(sn[i], sn[i + 1]);
                const float2 x = f2_fma_rn(a, c, f2_mul_rn(b, make_float2(-s.x, -s.y)));
                const float2 y = f2_fma_rn(b, c, f2_mul_rn(a, s));
                v[i] = x.x, v[i + 1] = x.y, v[4 + i] = y.x, v[5 + i] = y.y;
            }
        }
        if (ROT == 2 && rotated && !is_v) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float &a = v[2 * i], &b = v[2 * i + 1];
                const float x = a * cs[i] - b * sn[i];
                b = b * cs[i] + a * sn[i];
                a = x;
            }
        }
        if (ROT != 0 && bad)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                v[i] = NAN;
        if (in) {
            const uint2 a = pack4<E>(v), b = pack4<E>(v + 4);
            if (out != nullptr) {
                *reinterpret_cast<uint2*>(out + d0) = a;
                *reinterpret_cast<uint2*>(out + d1) = b;
                out += p.dim;
            }
            if (cache16 != nullptr) {
                *reinterpret_cast<uint2*>(cache16 + d0) = a;
                *reinterpret_cast<uint2*>(cache16 + d1) = b;
                cache16 += row_step * p.dim;
            }
        }
        if (int8 && row >= 0) {  // the same for a whole lane group
            float top = 0.0f;
#pragma unroll
            for (int i = 0; i < 8; ++i)
                top = max_nan(top, fabsf(v[i]));
#pragma unroll
            for (int o = LANES / 2; o; o >>= 1)
                top = max_nan(top, __shfl_xor_sync(mask, top, o));
            // no numbers in the row (a position out of range, a NaN or infinity of the input): no scale
            const float scale = top < INFINITY ? __fdiv_rn(top, 127.0f) : NAN;
            uint32_t c[2] = {0, 0};
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                // v / scale is at most 127 (1 + 2^-23) unless the scale is subnormal: clamp (codes are 0
                // where there is no scale)
                const float q = scale > 0.0f ? fminf(fmaxf(rintf(__fdiv_rn(v[i], scale)), -127.0f), 127.0f) : 0.0f;
                c[i >> 2] |= (uint32_t)((int)q & 255) << (8 * (i & 3));
            }
            const int64_t at = row + j * row_step;
            if (in) {
                int8_t* dst = static_cast<int8_t*>(cache) + at * p.dim;
                *reinterpret_cast<uint32_t*>(dst + d0) = c[0];
                *reinterpret_cast<uint32_t*>(dst + d1) = c[1];
            }
            if (lane == 0)
                (is_v ? p.cache.v_scale : p.cache.k_scale)[at] = scale;
        }
    }
}

template <class E, int LANES, int ROT>
cudaError_t launch(const NormRope& p, unsigned int* err, cudaStream_t s)
{
    const int64_t chunks =
        (p.q_heads + HEADS_PER - 1) / HEADS_PER + 2 * (int64_t)((p.kv_heads + HEADS_PER - 1) / HEADS_PER);
    const int64_t per_block = WARPS * 32 / LANES;
    const int64_t blocks = (p.tokens * chunks + per_block - 1) / per_block;
    return launch_pdl(norm_rope_kernel<E, LANES, ROT>, dim3((unsigned)blocks), dim3(WARPS * 32), 0, s, p, err);
}

template <class E, int LANES>
cudaError_t by_rotation(const NormRope& p, unsigned int* err, cudaStream_t s)
{
    return p.rot == 0 ? launch<E, LANES, 0>(p, err, s)
           : p.interleaved ? launch<E, LANES, 2>(p, err, s) : launch<E, LANES, 1>(p, err, s);
}

template <class E>
cudaError_t by_dim(const NormRope& p, unsigned int* err, cudaStream_t s)
{
    return p.dim <= 64 ? by_rotation<E, 8>(p, err, s)
           : p.dim <= 128 ? by_rotation<E, 16>(p, err, s) : by_rotation<E, 32>(p, err, s);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRope& p, const DeviceInfo& dev, cudaStream_t s)
{
    (void)dev;
    unsigned int* err = nullptr;
    cudaError_t e = device_error_ptr(&err);
    if (e != cudaSuccess)
        return e;
    return p.f16 ? by_dim<Fp16>(p, err, s) : by_dim<Bf16>(p, err, s);
}

}  // namespace ck
