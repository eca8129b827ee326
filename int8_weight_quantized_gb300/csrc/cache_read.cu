// cache_read.cu -- rows of the paged cache back as contiguous 16-bit keys and values: what
// attention over whole prompts needs where a prompt's first tokens are in the cache already (its
// second chunk, a request behind a cached prefix).
//
//   k_out[cu[b] + t, h] = cache row (T_b[t / page_size], h, t % page_size) (times its scale, int8)
//
// Bound: HBM, each row read once and written once.  A block looks up its tokens' rows once, 8 values to a
// lane (a store of 16 bytes), four rows of keys and of values of a thread on their way at once.
//
// Measured (GB300): 65536 tokens of 8 heads of 128 in int8 rows 65 us, 6.26 TB/s, 92% of a copy's bandwidth,
// in 16-bit rows 82 us, 97%; heads of 64, int8 rows, 37; 300 tokens 5 to 6 us (launch and two look-ups one after
// the other).  With 16 codes to a lane, whose two stores leave every second 16 bytes to the other: 76; two
// rows at once 66; 32 tokens to a block 67.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_common.cuh"
#include "transformer.h"

namespace ck {
namespace {

constexpr int THREADS = 256;
constexpr int MOST_TOKENS = 64;  // of a block

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

// codes times their row's scale, rounded once to 16 bits
template <class E>
__device__ __forceinline__ uint4 widen8(uint32_t lo, uint32_t hi, float scale)
{
    uint32_t r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t pair = (i < 2 ? lo : hi) >> (16 * (i & 1));
        r[i] = E::pack2((float)(int8_t)(pair & 0xFFu) * scale, (float)(int8_t)((pair >> 8) & 0xFFu) * scale);
    }
    return make_uint4(r[0], r[1], r[2], r[3]);
}

// A lane's part of a row: 8 values.
template <class E, bool INT8>
struct Part {
    using Raw = typename std::conditional<INT8, uint2, uint4>::type;
    Raw raw;
    float scale = 1.0f;
    __device__ __forceinline__ void load(const void* base, const float* scales, int64_t row, int lanes, int c)
    {
        raw = __ldg(static_cast<const Raw*>(base) + row * lanes + c);
        if (INT8)
            scale = __ldg(scales + row);
    }
    __device__ __forceinline__ void store(void* base, int64_t row, int lanes, int c, bool nan) const
    {
        uint4 x;
        if constexpr (INT8)
            x = widen8<E>(raw.x, raw.y, scale);
        else
            x = raw;
        const uint32_t bad = E::pack2(NAN, NAN);
        static_cast<uint4*>(base)[row * lanes + c] = nan ? make_uint4(bad, bad, bad, bad) : x;
    }
};

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
    // Row r of the block's is head r % heads of token r / heads, and its outputs come after those of row r - 1.  A row
    // to as many lanes as it takes, rounded up to a power of two; a thread takes every `step`-th row, AHEAD of
    // them at once.
    constexpr int AHEAD = 4;
    const int lanes = p.cache.dim / 8, heads = p.cache.heads;
    int wide = 1;
    while (wide < lanes)
        wide *= 2;
    const int c = threadIdx.x % wide, step = THREADS / wide;
    const int step_tok = step / heads, step_h = step - step_tok * heads;
    int r = threadIdx.x / wide, tok = r / heads, h = r - tok * heads;
    if (c < lanes)
        while (tok < per) {
            Part<E, INT8> k[AHEAD], v[AHEAD];
            int64_t row[AHEAD];
#pragma unroll
            for (int n = 0; n < AHEAD; ++n) {
                row[n] = tok < per ? rows[tok] : -2;
                if (row[n] >= 0) {
                    const int64_t at = row[n] + (int64_t)h * page_size;
                    k[n].load(p.cache.k, p.cache.k_scale, at, lanes, c);
                    v[n].load(p.cache.v, p.cache.v_scale, at, lanes, c);
                }
                tok += step_tok, h += step_h;
                if (h >= heads)
                    h -= heads, ++tok;
            }
#pragma unroll
            for (int n = 0; n < AHEAD; ++n, r += step)
                if (row[n] != -2) {
                    k[n].store(p.k_out, first * heads + r, lanes, c, row[n] < 0);
                    v[n].store(p.v_out, first * heads + r, lanes, c, row[n] < 0);
                }
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
    // tokens of a block: some 128 rows, fewer where that leaves less than four blocks to an SM
    int per = 1;
    while (per < MOST_TOKENS && 2 * per * p.cache.heads <= 128 && p.total / (2 * per) >= 4 * dev.sm_count)
        per *= 2;
    auto run = [&](auto kernel) {
        return launch_pdl(kernel, dim3((unsigned)((p.total + per - 1) / per)), dim3(THREADS), 0, s, p, per, err);
    };
    if (p.cache.dtype == CK_KV_INT8)
        return p.f16 ? run(read_kernel<Fp16, true>) : run(read_kernel<Bf16, true>);
    return p.f16 ? run(read_kernel<Fp16, false>) : run(read_kernel<Bf16, false>);
}

}  // namespace ck
