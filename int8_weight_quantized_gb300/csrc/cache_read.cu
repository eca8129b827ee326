// cache_read.cu -- rows of the paged cache back as contiguous 16-bit keys and values: what
// attention over whole prompts needs where a prompt's first tokens are in the cache already (its
// second chunk, a request behind a cached prefix).
//
//   k_out[cu[b] + t, h] = cache row (T_b[t / page_size], h, t % page_size) (times its scale, int8)
//
// Bound: HBM, each row read once and written once.
#include <algorithm>
#include <cmath>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_common.cuh"
#include "transformer.h"

namespace ck {
namespace {

constexpr int THREADS = 256;
constexpr int MOST_TOKENS = 32;  // of a block

// The last sequence that begins at or before row t, -1: none.
__device__ __forceinline__ int64_t sequence_of(const int32_t* cu, int64_t batch, int64_t t)
{
    int64_t lo = -1, hi = batch;
    while (lo < hi) {
        const int64_t mid = (lo + hi + 1) >> 1;
        if (__ldg(cu + mid) <= t)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// 8 codes times their row's scale, rounded once to 16 bits
template <class E>
__device__ __forceinline__ uint4 widen8(uint2 codes, float scale)
{
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t pair = (i < 2 ? codes.x : codes.y) >> (16 * (i & 1));
        r[i] = E::pack2((float)(int8_t)(pair & 0xFFu) * scale, (float)(int8_t)((pair >> 8) & 0xFFu) * scale);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

template <class E, bool INT8>
__global__ void __launch_bounds__(THREADS) read_kernel(const CacheRead p, int per, unsigned int* err)
{
    griddep_wait();
    // where each of the block's tokens lies: its row of head 0, -1: no such row (NaN), -2: no output
    __shared__ int64_t rows[MOST_TOKENS];
    const int64_t first = (int64_t)blockIdx.x * per;
    const int page_size = p.cache.page_size;
    bool bad = false;
    if (threadIdx.x < per) {
        const int64_t t = first + threadIdx.x;
        int64_t row = -2;
        if (t < p.total) {
            const int64_t b = sequence_of(p.cu, p.batch, t);
            if (b >= 0 && b < p.batch) {
                const int64_t at = t - __ldg(p.cu + b);
                const int64_t blk = at / page_size;
                row = -1;
                if (blk < p.max_blocks) {
                    const int64_t page = __ldg(p.block_table + b * p.max_blocks + blk);
                    if (page >= 0 && page < p.cache.num_pages)
                        row = page * p.cache.heads * page_size + (at - blk * page_size);
                }
                bad = row == -1;
            }
        }
        rows[threadIdx.x] = row;
    }
    // every bound, by some block
    for (int64_t b = (int64_t)blockIdx.x * THREADS + threadIdx.x; b < p.batch; b += (int64_t)gridDim.x * THREADS) {
        const int32_t lo = __ldg(p.cu + b), hi = __ldg(p.cu + b + 1);
        bad |= lo < 0 || hi < lo || hi > p.total;
    }
    if (bad)
        atomicOr(err, kErrIndex);
    __syncthreads();
    const int lanes = p.cache.dim / 8;  // 8 values each
    const int pieces = p.cache.heads * lanes;
    for (int i = threadIdx.x; i < per * pieces; i += THREADS) {
        const int tok = i / pieces, rest = i - tok * pieces, h = rest / lanes, c = rest - h * lanes;
        const int64_t row = rows[tok];
        if (row == -2)
            continue;
        const int64_t out = ((first + tok) * p.cache.heads + h) * lanes + c;
        uint4 k, v;
        if (row >= 0) {
            const int64_t at = row + (int64_t)h * page_size;
            const int64_t in = at * lanes + c;
            if (INT8) {
                k = widen8<E>(__ldg(static_cast<const uint2*>(p.cache.k) + in), __ldg(p.cache.k_scale + at));
                v = widen8<E>(__ldg(static_cast<const uint2*>(p.cache.v) + in), __ldg(p.cache.v_scale + at));
            } else {
                k = __ldg(static_cast<const uint4*>(p.cache.k) + in);
                v = __ldg(static_cast<const uint4*>(p.cache.v) + in);
            }
        } else {
            const uint32_t nan = E::pack2(NAN, NAN);
            k = v = make_uint4(nan, nan, nan, nan);
        }
        static_cast<uint4*>(p.k_out)[out] = k;
        static_cast<uint4*>(p.v_out)[out] = v;
    }
    griddep_launch_dependents();
}

}  // namespace

cudaError_t launch_cache_read(const CacheRead& p, const DeviceInfo& dev, cudaStream_t s)
{
    unsigned int* err = nullptr;
    const cudaError_t e = device_error_ptr(&err);
    if (e != cudaSuccess)
        return e;
    int per = 1;
    while (per < MOST_TOKENS && p.total / (2 * per) >= 4 * dev.sm_count)
        per *= 2;
    auto run = [&](auto kernel) {
        return launch_pdl(kernel, dim3((unsigned)((p.total + per - 1) / per)), dim3(THREADS), 0, s, p, per, err);
    };
    if (p.cache.dtype == CK_KV_INT8)
        return p.f16 ? run(read_kernel<Fp16, true>) : run(read_kernel<Bf16, true>);
    return p.f16 ? run(read_kernel<Fp16, false>) : run(read_kernel<Bf16, false>);
}

}  // namespace ck
