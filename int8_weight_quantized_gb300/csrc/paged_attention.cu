// paged_attention.cu -- attention of one new token per sequence over the paged cache.
//
//   out[b,h] = sum_j w_j v_j / sum_j w_j,  w_j = exp(scale * q[b,h] . k_j - max),  j over the
//   keys of sequence b that its last token sees (all, or the first `sinks` and the last
//   `window`); zeros where the sequence is empty.
//
// Bound: HBM.  Every visible key and value row is read once per kv head, for the up to 16
// query heads that share it; nothing else is read more than once.
//
// Work.  A segment is one (sequence, kv head, 8 NT query heads); its visible keys, numbered
// through without the hidden ones, are cut into tiles of 64 (int8: 128).  All segments' tiles in a row are
// shared out evenly: block c of C takes tiles [c T / C, (c + 1) T / C), whatever the lengths
// (each block sums the lengths up itself, so nothing depends on the host knowing them and a
// captured graph may be replayed with new lengths).  A block leaves a segment that it holds
// whole as the final output, and the at most two that it shares with a neighbour as partial
// sums (maximum, sum of weights, weighted values); join_kernel adds those up, always in the
// same order.  Where no segment can hold more than kWholeKeys keys, one block takes each
// whole segment and there is no second launch.
//
// Inside a block each of the 4 warps takes 16 (int8: 32) keys of a tile on its own: its own ring of
// asynchronous copies (no block-wide barrier while tiles stream), its own running maximum and
// sum; the four are joined once per segment.  Both products run on the 16x8x16 matrix
// instruction with keys (then value columns) as its 16 rows and the query heads as its 8
// columns -- S^T = K Q^T, O^T = V^T P^T --, so that the usual 1 to 8 heads of a group waste
// little of the softmax arithmetic (heads as rows, 16 of them: 646 instead of about 400
// instructions per 16 keys on int8 rows, which were bound by that).  Between the two products
// the weights stay in registers: two 8x8 transposes.
//
// int8 rows: a code is exact in fp16, so both products run in fp16: the query scaled by the
// power of two that brings its largest value into [1, 2) (undone in the fp32 score), and the
// row scales folded in as fp32: k's into the score, v's, as its base-2 logarithm, into the
// exponent of the weight.  What is rounded to fp16 is the product of weight and value scale,
// relative to the largest such product so far (or 2^kLag below it), whatever key that belongs
// to: relative to the largest scale, a key with nearly all the weight and a small value row lost
// its bits, or all of it, to a large row that has no weight.  The sum of the weights keeps its
// own reference, the largest score.
//
// Measured (GB300; 32 query heads on 8 of 128 values): 64 sequences of 0 to 8192 tokens in 16-bit
// rows 170 to 174 us, 6.3 TB/s, 94% of a copy's bandwidth; one of 131071 tokens 89 us, 91%; 32
// sequences of 1025 to 16384 tokens in int8 rows 99 to 101 us, 88%, heads of 64 65.5, 69%; one of 274
// tokens 6.4 to 6.8 us, of 64 tokens 4 to 5 (two products, a few tiles per warp: latency).  int8 rows are
// bound by instructions: each code is widened for the matrix instruction, which has no int8 by 16-bit
// form.
//
// Rounding to fewer bits: each weight once (on int8 rows its product with the value scale), to the
// type of the values' product (bf16 or fp16), which is what the matrix instruction takes; on int8
// rows also the query, to fp16 after its scaling, which is exact but for values below 2^-17 (of bf16)
// or 2^-14 (of fp16) of the head's largest, and those are off by 2^-25 of it at most.  Sums, maxima
// and scores are fp32.
#include <algorithm>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_common.cuh"
#include "transformer.h"
#include "warp_mma.cuh"

namespace ck {
namespace {

constexpr int WARPS = 4;
// Segments of at most this many keys are not split: 64 sequences of 1 to 500 tokens 19.4 us, split
// 31.5 (a block pays about 1 us for each segment that it takes up, and the sums have to be joined).
constexpr int kWholeKeys = 512;
// int8 rows: how far (log2) the products of weight and value scale may exceed what they are kept
// relative to (fp16 holds 2^15, its least normal value is 2^-14), before that follows them.
constexpr float kLag = 8.0f;

// NT: tiles of 8 query heads that a segment holds (1, or 2 where a group has more than 8)
template <bool INT8, int DIM, int NT>
struct Shape {
    static constexpr int HEADS = 8 * NT;
    // Keys of a warp's unit.  int8 rows take twice as many: a unit's fixed cost (look-up, copy
    // addresses, maximum and sum) is spread over the same bytes as with 16-bit rows.
    static constexpr int KEYS = INT8 ? 32 : 16;
    static constexpr int KT = KEYS / 16;                     // tiles of 16 keys
    static constexpr int TILE = WARPS * KEYS;                // keys of a block's tile
    static constexpr int ROW = DIM * (INT8 ? 1 : 2);        // bytes of a row
    static constexpr int SCALES = INT8 ? 2 * KEYS * 4 : 0;   // k scales, v scales
    static constexpr int UNIT = 2 * KEYS * ROW + SCALES;
    // About 200 KB of rings an SM.  16-bit rows: two blocks; int8 rows, whose arithmetic per
    // byte is twice that, three (two with 16 heads, which hold twice the sums).
    static constexpr int BLOCKS = INT8 && NT == 1 ? 3 : 2;
    static constexpr int STAGES = (BLOCKS == 3 ? 16384 : 24576) / (UNIT - SCALES);
    static constexpr int LD = DIM + 4;                       // joined sums: floats per head
    static constexpr size_t RING = (size_t)WARPS * STAGES * UNIT;
    // Sums that the warps join theirs in: two, where that leaves room for BLOCKS blocks on an SM.
    // (One segment of 274 tokens 7.5 us with one and 7.0 with two, 32 of 1025 to 16384 tokens in int8
    // rows 106.6 and 102.3; 16 heads to an int8 head, whose second block went: 16.5 and 18.6.)
    static constexpr size_t sums_bytes(int slabs) { return slabs * HEADS * LD * 4 + WARPS * HEADS * 8; }
    static constexpr int SLABS = RING + sums_bytes(2) <= 233472 / BLOCKS - 1024 ? 2 : 1;
    static constexpr size_t SMEM = RING + sums_bytes(SLABS);
    static constexpr size_t PART = (size_t)HEADS * (DIM + 2);  // floats of one partial
};

// ---- the division of work, the same in both kernels
struct Lengths {
    const int32_t* seq_lens;
    int64_t max_len, window, sinks;
    int subs;  // segments of a sequence
    int tile;  // keys of a tile
    __device__ int length(int64_t b, bool* bad) const
    {
        const int64_t n = __ldg(seq_lens + b);
        *bad = n < 0 || n > max_len;
        return *bad ? 0 : (int)n;
    }
    __device__ int tiles(int64_t b) const
    {
        bool bad;
        return (visible_keys(length(b, &bad), window, sinks).count() + tile - 1) / tile;
    }
};

// By a whole warp: tiles of all segments before sequence `upto`.
__device__ __forceinline__ int64_t tiles_before(const Lengths& L, int64_t upto)
{
    const int lane = threadIdx.x & 31;
    int64_t sum = 0;
    for (int64_t b = lane; b < upto; b += 32)
        sum += (int64_t)L.tiles(b) * L.subs;
#pragma unroll
    for (int o = 16; o; o >>= 1)
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return sum;
}

__device__ __forceinline__ int64_t first_tile(int64_t c, int64_t C, int64_t T)
{
    return c * T / C;
}

// By a whole warp: the sequence that holds tile `t` of all tiles, and the tiles before it.
__device__ __forceinline__ int64_t sequence_at(const Lengths& L, int64_t batch, int64_t t, int64_t* before)
{
    const int lane = threadIdx.x & 31;
    int64_t base = 0;
    for (int64_t b0 = 0; b0 < batch; b0 += 32) {
        int64_t mine = b0 + lane < batch ? (int64_t)L.tiles(b0 + lane) * L.subs : 0;
        int64_t upto = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, upto, o);
            if (lane >= o)
                upto += v;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, base + upto > t);
        if (past) {
            const int l = __ffs(past) - 1;
            *before = base + __shfl_sync(0xffffffffu, upto - mine, l);
            return b0 + l;
        }
        base += __shfl_sync(0xffffffffu, upto, 31);
    }
    *before = base;
    return batch;
}

// Walks the tiles of a block's range.
struct Cursor {
    int64_t b;
    int sub, tile, tiles;
    int64_t left;  // tiles of the range from here on
    VisibleKeys keys;
    __device__ void open(const Lengths& L)
    {
        bool bad;
        keys = visible_keys(L.length(b, &bad), L.window, L.sinks);
        tiles = (keys.count() + L.tile - 1) / L.tile;
    }
    __device__ void next(const Lengths& L)
    {
        if (--left <= 0 || ++tile < tiles)
            return;
        tile = 0;
        if (++sub < L.subs)
            return;
        sub = 0;
        do {
            ++b;
            open(L);
        } while (tiles == 0);  // left > 0: a later sequence has tiles
    }
};

// ---- int8 codes to pairs of fp16, exact: byte ^ 0x80 in the mantissa of 1024, minus 1152
__device__ __forceinline__ uint32_t half2_of(uint32_t biased_pair_bytes, uint32_t sel)
{
    const uint32_t w = __byte_perm(biased_pair_bytes, 0x64646464u, sel);
    const __half2 v = __hsub2(*reinterpret_cast<const __half2*>(&w), __half2half2(__ushort_as_half(0x6480)));
    return *reinterpret_cast<const uint32_t*>(&v);
}

// Byte address of 16-byte chunk c of row r of a ring unit's K or V part, so that the reads
// below spread over all banks.
template <bool INT8, int DIM, bool V>
__device__ __forceinline__ uint32_t chunk_at(int r, int c)
{
    constexpr int CHUNKS = Shape<INT8, DIM, 1>::ROW / 16;
    int p;
    if (!INT8)
        p = c ^ (r & 7);  // ldmatrix: one chunk of 8 neighbouring rows
    else if (CHUNKS == 8)
        p = V ? c ^ (((r >> 1) & 3) << 1) : c ^ ((r & 1) << 2);
    else
        p = V ? c ^ ((r >> 1) & 3) : c;
    return (uint32_t)(r * Shape<INT8, DIM, 1>::ROW + p * 16);
}

template <class E, bool INT8, int DIM, int NT>
__global__ void __launch_bounds__(WARPS * 32, Shape<INT8, DIM, NT>::BLOCKS)
    paged_kernel(const PagedAttention p, int64_t C, bool split, unsigned int* err)
{
    using S = Shape<INT8, DIM, NT>;
    using T = typename E::T;
    using M = typename std::conditional<INT8, Fp16, E>::type;  // the products' type
    constexpr int HEADS = S::HEADS, KEYS = S::KEYS, KT = S::KT, TILE = S::TILE;
    extern __shared__ __align__(128) uint8_t smem[];
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int group = p.q_heads / p.cache.heads;  // query heads per kv head
    const int qtiles = (group + HEADS - 1) / HEADS;
    const int page_size = p.cache.page_size;
    Lengths L{p.seq_lens, p.max_blocks * page_size, p.window, p.sinks, p.cache.heads * qtiles, TILE};

    // sequences without visible keys have no tiles: zeros, or NaN where the length is out of range
    for (int64_t b = blockIdx.x; b < p.batch; b += gridDim.x) {
        bool bad;
        const int n = L.length(b, &bad);
        if (n > 0)
            continue;
        if (bad && threadIdx.x == 0)
            atomicOr(err, kErrIndex);
        for (int i = threadIdx.x; i < p.q_heads * DIM; i += WARPS * 32)
            static_cast<T*>(p.out)[b * p.q_heads * DIM + i] = E::from(bad ? NAN : 0.0f);
        if (p.lse != nullptr)
            for (int i = threadIdx.x; i < p.q_heads; i += WARPS * 32)
                p.lse[b * p.q_heads + i] = bad ? NAN : -INFINITY;
    }

    // this block's range of tiles
    Cursor at;
    if (split) {
        const int64_t total = tiles_before(L, p.batch);
        C = min(C, total);  // no block of those that take part is without tiles
        if (blockIdx.x >= C)
            return;
        const int64_t t0 = first_tile(blockIdx.x, C, total), t1 = first_tile(blockIdx.x + 1, C, total);
        at.left = t1 - t0;
        int64_t before;
        at.b = sequence_at(L, p.batch, t0, &before);
        at.open(L);
        at.sub = (int)((t0 - before) / at.tiles);
        at.tile = (int)((t0 - before) % at.tiles);
    } else {
        at.b = blockIdx.x / L.subs;
        at.sub = (int)(blockIdx.x - at.b * L.subs);
        at.tile = 0;
        at.open(L);
        at.left = at.tiles;
        if (at.left <= 0)
            return;
    }

    const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * S::STAGES * S::UNIT);
    float* joined = reinterpret_cast<float*>(smem + S::RING);             // [SLABS][HEADS][LD]
    float2* maxsum = reinterpret_cast<float2*>(joined + S::SLABS * HEADS * S::LD);  // [WARPS][HEADS]

    // ---- copies: lane l looks up the row of key l % KEYS of the warp's unit one unit ahead
    constexpr int CH = S::ROW / 16;       // 16-byte chunks of a row
    constexpr int RPI = 32 / CH;          // rows of one copy instruction
    const uint8_t* const k_lane = static_cast<const uint8_t*>(p.cache.k) + lane % CH * 16;
    const uint8_t* const v_lane = static_cast<const uint8_t*>(p.cache.v) + lane % CH * 16;
    Cursor ahead = at;
    int32_t page = 0;
    int in_page = 0;
    bool have = false;
    auto look_up = [&]() {
        const int v = ahead.tile * TILE + warp * KEYS + lane % KEYS;
        have = ahead.left > 0 && v < ahead.keys.count();
        if (have) {
            const int j = ahead.keys.key(v);
            // page_shift: the page size is that power of two; -1: it is none
            const int blk = p.page_shift >= 0 ? j >> p.page_shift : j / page_size;
            in_page = j - blk * page_size;
            page = __ldg(p.block_table + ahead.b * p.max_blocks + blk);
        }
    };
    uint32_t bad_units = 0;  // bit s: the unit in stage s has a page number out of range
    auto issue = [&](int stage) {
        if (ahead.left > 0) {
            const bool in_pool = page >= 0 && page < p.cache.num_pages;
            const uint32_t bad = __ballot_sync(0xffffffffu, have && !in_pool);
            bad_units = (bad_units & ~(1u << stage)) | ((bad ? 1u : 0u) << stage);
            const bool ok = have && in_pool;
            const int hk = qtiles == 1 ? ahead.sub : ahead.sub / qtiles;
            // (the cache's rows are below 2^32)
            const uint32_t row = ok ? ((uint32_t)page * p.cache.heads + hk) * page_size + in_page : 0u;
            const uint32_t oks = __ballot_sync(0xffffffffu, ok);
            const uint32_t dst = ring + stage * S::UNIT;
#pragma unroll
            for (int i = 0; i < KEYS / RPI; ++i) {
                const int r = i * RPI + lane / CH;
                const uint64_t off = (uint64_t)__shfl_sync(0xffffffffu, row, r) * S::ROW;
                const bool r_ok = (oks >> r) & 1u;
                cp_async16(dst + chunk_at<INT8, DIM, false>(r, lane % CH), k_lane + off, r_ok);
                cp_async16(dst + KEYS * S::ROW + chunk_at<INT8, DIM, true>(r, lane % CH), v_lane + off, r_ok);
            }
            if (INT8) {
                static_assert(!INT8 || KEYS == 32, "a scale of each kind per lane");
                const uint32_t sc = dst + 2 * KEYS * S::ROW + lane * 4;
                cp_async_small<4>(sc, p.cache.k_scale + row, ok);
                cp_async_small<4>(sc + KEYS * 4, p.cache.v_scale + row, ok);
            }
            ahead.next(L);
            look_up();
        }
        cp_async_commit();
    };
    look_up();
#pragma unroll
    for (int s = 0; s < S::STAGES - 1; ++s)
        issue(s);

    uint32_t qb[NT][DIM / 16][2];  // queries of head 8 nt + g
    float o[NT][DIM / 16][4];      // sums of heads 8 nt + 2t, + 1 (columns), two value rows
    float m[NT][2], l[NT][2];      // of those heads: maximum, sum of weights
    float mv[NT][2];               // int8: what the sums o are relative to instead of m, see kLag
    float c_head[NT][2];           // score factor of those heads, in units of log2
    bool bad = false;
    bool fresh = true;
    int first_of_segment = 0;  // the block's first tile of the segment
    int stage = 0;
    int piece = 0;             // partial slots used

    for (;;) {
        if (fresh) {  // a new segment: its queries
            const int hk = at.sub / qtiles, qt = at.sub - hk * qtiles;
            const int h0 = hk * group + qt * HEADS;
            const int heads = min(HEADS, group - qt * HEADS);
            const T* q = static_cast<const T*>(p.q) + at.b * p.q_stride + (int64_t)h0 * DIM;
            const float c = p.scale * kLog2e;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int head = 8 * nt + g;
                const T* qh = q + (int64_t)head * DIM;
                if (!INT8) {
#pragma unroll
                    for (int kk = 0; kk < DIM / 16; ++kk) {
                        const uint32_t* src = reinterpret_cast<const uint32_t*>(qh + 16 * kk + 2 * t);
                        qb[nt][kk][0] = head < heads ? __ldg(src) : 0u;
                        qb[nt][kk][1] = head < heads ? __ldg(src + 4) : 0u;
                    }
                    c_head[nt][0] = c_head[nt][1] = c;
                } else {
                    // the int8 products' order: k-step kk, lane t <- d = 64 (kk / 4) + 16 t + 4 (kk % 4) ..
                    float v[DIM / 4];
                    float top = 0.0f;
#pragma unroll
                    for (int kk = 0; kk < DIM / 16; ++kk) {
                        const uint2 w = head < heads
                                            ? __ldg(reinterpret_cast<const uint2*>(qh + 64 * (kk / 4) + 16 * t + 4 * (kk % 4)))
                                            : make_uint2(0u, 0u);
                        const float2 a = E::to2(w.x), b = E::to2(w.y);
                        v[4 * kk] = a.x, v[4 * kk + 1] = a.y, v[4 * kk + 2] = b.x, v[4 * kk + 3] = b.y;
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            top = fmaxf(top, fabsf(v[4 * kk + i]));
                    }
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    const int e = top > 0.0f && top < INFINITY ? ilogbf(top) : 0;
#pragma unroll
                    for (int kk = 0; kk < DIM / 16; ++kk) {
                        qb[nt][kk][0] = Fp16::pack2(ldexpf(v[4 * kk], -e), ldexpf(v[4 * kk + 1], -e));
                        qb[nt][kk][1] = Fp16::pack2(ldexpf(v[4 * kk + 2], -e), ldexpf(v[4 * kk + 3], -e));
                    }
                    const float ch = ldexpf(c, e);  // of head g: pass it to the lanes of its column
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        c_head[nt][j] = __shfl_sync(0xffffffffu, ch, (2 * t + j) * 4);
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    m[nt][j] = mv[nt][j] = -INFINITY;
                    l[nt][j] = 0.0f;
                }
#pragma unroll
                for (int e = 0; e < DIM / 16; ++e)
                    o[nt][e][0] = o[nt][e][1] = o[nt][e][2] = o[nt][e][3] = 0.0f;
            }
            bad = false;
            fresh = false;
            first_of_segment = at.tile;
        }

        issue(stage == 0 ? S::STAGES - 1 : stage - 1);
        cp_async_wait<S::STAGES - 1>();
        __syncwarp();

        const int v0 = at.tile * TILE + warp * KEYS;  // the unit's first key number
        const int n = at.keys.count();
        if (v0 < n) {  // warp-uniform
            bad |= (bad_units >> stage) & 1u;
            const uint32_t ks = ring + stage * S::UNIT;
            const uint32_t vs = ks + KEYS * S::ROW;
            // S^T: rows keys 16 kt + g, + 8; columns heads 2t, 2t + 1 of each nt
            float s[NT][KT][4], s_odd[NT][4] = {};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int kt = 0; kt < KT; ++kt)
                    s[nt][kt][0] = s[nt][kt][1] = s[nt][kt][2] = s[nt][kt][3] = 0.0f;
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
                if (!INT8) {
                    // two sums: half the wait of a chain of products
#pragma unroll
                    for (int kk = 0; kk < DIM / 16; ++kk) {
                        uint32_t ka[4];
                        ldmatrix_x4(ka, ks + chunk_at<INT8, DIM, false>(16 * kt + (lane & 15), 2 * kk + (lane >> 4)));
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma_16816<M>(kk & 1 ? s_odd[nt] : s[nt][kt], ka, qb[nt][kk][0], qb[nt][kk][1]);
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            s[nt][kt][i] += s_odd[nt][i], s_odd[nt][i] = 0.0f;
                } else {
#pragma unroll
                    for (int hf = 0; hf < DIM / 64; ++hf) {
                        const uint4 r0 = lds128(ks + chunk_at<INT8, DIM, false>(16 * kt + g, 4 * hf + t));
                        const uint4 r1 = lds128(ks + chunk_at<INT8, DIM, false>(16 * kt + g + 8, 4 * hf + t));
                        const uint32_t w0[4] = {r0.x, r0.y, r0.z, r0.w}, w1[4] = {r1.x, r1.y, r1.z, r1.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t u0 = w0[i] ^ 0x80808080u, u1 = w1[i] ^ 0x80808080u;
                            const uint32_t ka[4] = {half2_of(u0, 0x4140), half2_of(u1, 0x4140), half2_of(u0, 0x4342),
                                                    half2_of(u1, 0x4342)};
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma_16816<M>(s[nt][kt], ka, qb[nt][4 * hf + i][0], qb[nt][4 * hf + i][1]);
                        }
                    }
                }
            }
            // int8: of keys 16 kt + g, + 8 the key scales, and the value scales in units of log2
            float kscale[KT][2], vlog[KT][2];
            if (INT8) {
                const uint32_t sc = vs + KEYS * S::ROW;
#pragma unroll
                for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        kscale[kt][h] = __uint_as_float(lds32(sc + (16 * kt + g + 8 * h) * 4));
                        vlog[kt][h] = fast_log2(__uint_as_float(lds32(sc + (KEYS + 16 * kt + g + 8 * h) * 4)));
                    }
            }
            uint32_t pb[NT][KT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float w[KT][4];  // weights for the values' product
                float a[2][KT][2], top[2], keep[2];  // a: scores in units of log2; keys past the end out
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    top[j] = -INFINITY;
#pragma unroll
                    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float x = s[nt][kt][2 * h + j] * c_head[nt][j];
                            a[j][kt][h] = v0 + 16 * kt + g + 8 * h < n ? (INT8 ? x * kscale[kt][h] : x) : -INFINITY;
                            top[j] = fmaxf(top[j], a[j][kt][h]);
                        }
                }
#pragma unroll
                for (int x = 4; x <= 16; x <<= 1) {
                    const float t0 = __shfl_xor_sync(0xffffffffu, top[0], x), t1 = __shfl_xor_sync(0xffffffffu, top[1], x);
                    top[0] = fmaxf(top[0], t0), top[1] = fmaxf(top[1], t1);
                }
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const float m2 = fmaxf(m[nt][j], top[j]);
                    const float ref = m2 == -INFINITY ? 0.0f : m2;
                    keep[j] = fast_exp2(m[nt][j] - ref);
                    m[nt][j] = m2;
                    l[nt][j] *= keep[j];
#pragma unroll
                    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const float x = fast_exp2(a[j][kt][h] - ref);
                            l[nt][j] += x;
                            w[kt][2 * h + j] = x;
                        }
                }
                if (INT8) {
                    // the products of weight and value scale, relative to a reference of their own
                    float over[2];  // the lane's largest
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        over[j] = -INFINITY;
#pragma unroll
                        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                a[j][kt][h] += vlog[kt][h];
                                over[j] = fmaxf(over[j], a[j][kt][h]);
                            }
                        keep[j] = 1.0f;
                    }
                    if (__any_sync(0xffffffffu, over[0] > mv[nt][0] + kLag || over[1] > mv[nt][1] + kLag))
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
#pragma unroll
                            for (int x = 4; x <= 16; x <<= 1)
                                over[j] = fmaxf(over[j], __shfl_xor_sync(0xffffffffu, over[j], x));
                            if (over[j] > mv[nt][j]) {
                                keep[j] = fast_exp2(mv[nt][j] - over[j]);
                                mv[nt][j] = over[j];
                            }
                        }
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float ref = mv[nt][j] == -INFINITY ? 0.0f : mv[nt][j];
#pragma unroll
                        for (int kt = 0; kt < KT; ++kt)
#pragma unroll
                            for (int h = 0; h < 2; ++h)
                                w[kt][2 * h + j] = fast_exp2(a[j][kt][h] - ref);
                    }
                }
                if (__any_sync(0xffffffffu, keep[0] != 1.0f || keep[1] != 1.0f))
#pragma unroll
                    for (int e = 0; e < DIM / 16; ++e)
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            o[nt][e][i] *= keep[i & 1];
#pragma unroll
                for (int kt = 0; kt < KT; ++kt) {
                    pb[nt][kt][0] = transpose_8x8(M::pack2(w[kt][0], w[kt][1]));
                    pb[nt][kt][1] = transpose_8x8(M::pack2(w[kt][2], w[kt][3]));
                }
            }
#pragma unroll
            for (int kt = 0; kt < KT; ++kt) {
                if (!INT8) {
#pragma unroll
                    for (int e = 0; e < DIM / 16; ++e) {
                        uint32_t va[4];
                        ldmatrix_x4_trans(va, vs + chunk_at<INT8, DIM, true>(16 * kt + (lane & 7) + ((lane >> 4) << 3),
                                                                            2 * e + ((lane >> 3) & 1)));
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma_16816<M>(o[nt][e], va, pb[nt][kt][0], pb[nt][kt][1]);
                    }
                } else {
                    // this lane's 4 keys (16 kt + 2t, 2t+1, 2t+8, 2t+9), values (DIM/8) g .. (DIM/8) (g+1) - 1:
                    // value 2 e of those is row g of tile e, value 2 e + 1 its row g + 8
                    constexpr int WORDS = DIM / 32;
                    uint32_t w[4][WORDS];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int r = 16 * kt + 2 * t + (i & 1) + 8 * (i >> 1);
                        if (DIM == 128) {
                            const uint4 x = lds128(vs + chunk_at<INT8, DIM, true>(r, g));
                            w[i][0] = x.x, w[i][1] = x.y, w[i][WORDS - 2] = x.z, w[i][WORDS - 1] = x.w;
                        } else {
                            const uint2 x = lds64(vs + chunk_at<INT8, DIM, true>(r, g >> 1) + 8 * (g & 1));
                            w[i][0] = x.x, w[i][1] = x.y;
                        }
                    }
#pragma unroll
                    for (int k = 0; k < WORDS; ++k) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {  // values 4 k + 2 h, + 1: tile 2 k + h
                            const uint32_t sel = h ? 0x7362 : 0x5140;
                            const uint32_t k01 = __byte_perm(w[0][k], w[1][k], sel) ^ 0x80808080u;
                            const uint32_t k23 = __byte_perm(w[2][k], w[3][k], sel) ^ 0x80808080u;
                            const uint32_t va[4] = {half2_of(k01, 0x4140), half2_of(k01, 0x4342), half2_of(k23, 0x4140),
                                                    half2_of(k23, 0x4342)};
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                mma_16816<M>(o[nt][2 * k + h], va, pb[nt][kt][0], pb[nt][kt][1]);
                        }
                    }
                }
            }
        }
        __syncwarp();
        stage = stage + 1 == S::STAGES ? 0 : stage + 1;

        const bool range_end = at.left == 1;
        const bool segment_end = at.tile + 1 == at.tiles;
        if (segment_end || range_end) {
            // ---- join the four warps, then leave the segment's output or this block's part of it
            const int hk = at.sub / qtiles, qt = at.sub - hk * qtiles;
            const int h0 = hk * group + qt * HEADS;
            const int heads = min(HEADS, group - qt * HEADS);
            if (bad && lane == 0)
                atomicOr(err, kErrIndex);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
#pragma unroll
                    for (int x = 4; x <= 16; x <<= 1)
                        l[nt][j] += __shfl_xor_sync(0xffffffffu, l[nt][j], x);
                    if (g == 0)
                        maxsum[warp * HEADS + 8 * nt + 2 * t + j] = make_float2(m[nt][j], bad ? NAN : l[nt][j]);
                }
            __syncthreads();
            float f[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    float top = -INFINITY;
#pragma unroll
                    for (int w = 0; w < WARPS; ++w)
                        top = fmaxf(top, maxsum[w * HEADS + 8 * nt + 2 * t + j].x);
                    // (int8: the square root, twice, since 2^(mv - top) is subnormal for tiny value scales)
                    f[nt][j] = m[nt][j] == -INFINITY ? 0.0f : fast_exp2(INT8 ? 0.5f * (mv[nt][j] - top) : m[nt][j] - top);
                }
            // SLABS warps at a time, each in sums of its own
            for (int w = 0; w < WARPS; w += S::SLABS) {
                if (warp / S::SLABS * S::SLABS == w)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < DIM / 16; ++e)
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int d = INT8 ? DIM / 8 * g + 2 * e + (i >> 1) : 16 * e + g + 8 * (i >> 1);
                                float* dst = joined + (warp % S::SLABS * HEADS + 8 * nt + 2 * t + (i & 1)) * S::LD + d;
                                float x = o[nt][e][i] * f[nt][i & 1];
                                if (INT8)
                                    x *= f[nt][i & 1];
                                *dst = w == 0 ? x : *dst + x;
                            }
                __syncthreads();
            }
            const bool whole = segment_end && first_of_segment == 0;
            float* part = static_cast<float*>(p.workspace) + (2 * (int64_t)blockIdx.x + piece) * S::PART;
            for (int i = threadIdx.x; i < heads * (DIM / 4); i += WARPS * 32) {
                const int row = i / (DIM / 4), d = i % (DIM / 4) * 4;
                float4 x = *reinterpret_cast<const float4*>(joined + row * S::LD + d);
                if (S::SLABS == 2) {
                    const float4 y = *reinterpret_cast<const float4*>(joined + (HEADS + row) * S::LD + d);
                    x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
                }
                if (!whole) {
                    *reinterpret_cast<float4*>(part + row * DIM + d) = x;
                    continue;
                }
                float top = -INFINITY, sum = 0.0f;
#pragma unroll
                for (int w = 0; w < WARPS; ++w)
                    top = fmaxf(top, maxsum[w * HEADS + row].x);
#pragma unroll
                for (int w = 0; w < WARPS; ++w) {
                    const float2 ms = maxsum[w * HEADS + row];
                    sum += ms.x == -INFINITY ? (ms.y != ms.y ? ms.y : 0.0f) : ms.y * fast_exp2(ms.x - top);
                }
                const int64_t at_row = at.b * p.q_heads + h0 + row;
                *reinterpret_cast<uint2*>(static_cast<T*>(p.out) + at_row * DIM + d) =
                    make_uint2(E::pack2(x.x / sum, x.y / sum), E::pack2(x.z / sum, x.w / sum));
                if (d == 0 && p.lse != nullptr)
                    p.lse[at_row] = (top + log2f(sum)) * kLn2;
            }
            if (!whole) {
                for (int row = threadIdx.x; row < heads; row += WARPS * 32) {
                    float top = -INFINITY, sum = 0.0f;
#pragma unroll
                    for (int w = 0; w < WARPS; ++w)
                        top = fmaxf(top, maxsum[w * HEADS + row].x);
#pragma unroll
                    for (int w = 0; w < WARPS; ++w) {
                        const float2 ms = maxsum[w * HEADS + row];
                        sum += ms.x == -INFINITY ? (ms.y != ms.y ? ms.y : 0.0f) : ms.y * fast_exp2(ms.x - top);
                    }
                    reinterpret_cast<float2*>(part + HEADS * DIM)[row] = make_float2(top, sum);
                }
                ++piece;
            }
            if (range_end)
                break;
            __syncthreads();  // the join's buffers are free again
            fresh = true;
        }
        at.next(L);
    }
    cp_async_wait<0>();
    griddep_launch_dependents();
}

// Adds up the partial sums of the segments that blocks share: one block per (sequence, query
// head), its 4 warps every fourth part each, then the four together.
template <class E, int DIM, int NT>
__global__ void __launch_bounds__(128) join_kernel(const PagedAttention p, int64_t C, int tile)
{
    using T = typename E::T;
    griddep_wait();
    constexpr int HEADS = 8 * NT;
    constexpr size_t PART = (size_t)HEADS * (DIM + 2);
    __shared__ float4 sums[4][32];
    __shared__ float2 maxsum[4];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t b = blockIdx.x / p.q_heads;
    const int h = (int)(blockIdx.x - b * p.q_heads);
    const int group = p.q_heads / p.cache.heads;
    const int qtiles = (group + HEADS - 1) / HEADS;
    Lengths L{p.seq_lens, p.max_blocks * p.cache.page_size, p.window, p.sinks, p.cache.heads * qtiles, tile};
    const int tiles = L.tiles(b);
    if (tiles == 0)
        return;  // the first kernel wrote it
    const int64_t total = tiles_before(L, p.batch);
    C = min(C, total);
    const int in_group = h % group;
    const int64_t sub = h / group * qtiles + in_group / HEADS;
    const int row = in_group % HEADS;
    const int64_t t0 = tiles_before(L, b) + sub * tiles, t1 = t0 + tiles;
    // block c holds tile t: c = floor(((t + 1) C - 1) / T)
    const int64_t c0 = ((t0 + 1) * C - 1) / total, c1 = (t1 * C - 1) / total;
    if (c0 == c1)
        return;  // one block held the whole segment and wrote the output
    const float* ws = static_cast<const float*>(p.workspace);
    float m = -INFINITY, l = 0.0f;
    float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    for (int64_t c = c0 + warp; c <= c1; c += 4) {
        // Slot 0 holds the first partial that block c left.  That is this segment, unless c = c0
        // began inside an earlier segment and had to leave that one first.
        int slot = 0;
        if (c == c0) {
            const int64_t begin = first_tile(c, C, total);
            if (begin < t0) {
                // an earlier piece was partial exactly if the block began inside its segment
                int64_t before;
                const int64_t bb = sequence_at(L, p.batch, begin, &before);
                const int bt = L.tiles(bb);
                slot = (begin - before) % bt != 0 ? 1 : 0;
            }
        }
        const float* part = ws + (2 * c + slot) * PART;
        const float2 ms = __ldcg(reinterpret_cast<const float2*>(part + HEADS * DIM) + row);
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (lane < DIM / 4)
            x = __ldcg(reinterpret_cast<const float4*>(part + row * DIM) + lane);
        const float m2 = fmaxf(m, ms.x);
        const float ref = m2 == -INFINITY ? 0.0f : m2;
        const float a = fast_exp2(m - ref), f = fast_exp2(ms.x - ref);
        l = l * a + ms.y * f;
        acc.x = acc.x * a + x.x * f, acc.y = acc.y * a + x.y * f;
        acc.z = acc.z * a + x.z * f, acc.w = acc.w * a + x.w * f;
        m = m2;
    }
    sums[warp][lane] = acc;
    if (lane == 0)
        maxsum[warp] = make_float2(m, l);
    __syncthreads();
    if (warp != 0)
        return;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < 4; ++w)
        top = fmaxf(top, maxsum[w].x);
    const float ref = top == -INFINITY ? 0.0f : top;
    float sum = 0.0f;
    acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        const float f = fast_exp2(maxsum[w].x - ref);
        const float4 x = sums[w][lane];
        sum += maxsum[w].y * f;
        acc.x += x.x * f, acc.y += x.y * f, acc.z += x.z * f, acc.w += x.w * f;
    }
    const int64_t at_row = b * p.q_heads + h;
    if (lane < DIM / 4)
        *reinterpret_cast<uint2*>(static_cast<T*>(p.out) + at_row * DIM + lane * 4) =
            make_uint2(E::pack2(acc.x / sum, acc.y / sum), E::pack2(acc.z / sum, acc.w / sum));
    if (lane == 0 && p.lse != nullptr)
        p.lse[at_row] = (top + log2f(sum)) * kLn2;
}

constexpr int kMostBlocks = 152 * 3;  // of any device this library runs on

// The most keys that a sequence can see.  (The workspace goes by the table alone; a window only
// shortens.)
int64_t longest_of(const PagedAttention& p)
{
    const int64_t longest = p.max_blocks * p.cache.page_size;
    // (by a difference: the sum of a window and first tokens of any size could overflow)
    return p.window > 0 && p.sinks < longest && p.window < longest - p.sinks ? p.window + p.sinks : longest;
}

template <class E, bool INT8, int DIM, int NT>
cudaError_t launch(const PagedAttention& p, const DeviceInfo& dev, unsigned int* err, cudaStream_t s)
{
    using S = Shape<INT8, DIM, NT>;
    // a kernel attribute belongs to the context it was set in: set once per context
    static ContextCache<int> cache;
    int done = 0;
    cudaError_t e = cache.get(&done, [](int* d) {
        *d = 1;
        return cudaFuncSetAttribute(paged_kernel<E, INT8, DIM, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)S::SMEM);
    });
    if (e != cudaSuccess)
        return e;
    const int group = p.q_heads / p.cache.heads;
    const int64_t segments = p.batch * p.cache.heads * ((group + S::HEADS - 1) / S::HEADS);
    const int64_t longest = longest_of(p);
    const int64_t tiles = (longest + S::TILE - 1) / S::TILE;
    const bool split = longest > kWholeKeys;
    const int64_t most = std::min<int64_t>(kMostBlocks, (int64_t)dev.sm_count * S::BLOCKS);
    const int64_t blocks = split ? std::min(most, segments * tiles) : segments;
    e = launch_pdl(paged_kernel<E, INT8, DIM, NT>, dim3((unsigned)blocks), dim3(WARPS * 32), S::SMEM, s, p, blocks, split,
                   err);
    if (e == cudaSuccess && split)
        e = launch_pdl(join_kernel<E, DIM, NT>, dim3((unsigned)(p.batch * p.q_heads)), dim3(128), 0, s, p, blocks, S::TILE);
    return e;
}

template <class E, int DIM, int NT>
cudaError_t by_cache(const PagedAttention& p, const DeviceInfo& dev, unsigned int* err, cudaStream_t s)
{
    return p.cache.dtype == CK_KV_INT8 ? launch<E, true, DIM, NT>(p, dev, err, s)
                                       : launch<E, false, DIM, NT>(p, dev, err, s);
}

template <int DIM>
cudaError_t by_type(const PagedAttention& p, const DeviceInfo& dev, unsigned int* err, cudaStream_t s)
{
    if (p.q_heads / p.cache.heads <= 8)
        return p.f16 ? by_cache<Fp16, DIM, 1>(p, dev, err, s) : by_cache<Bf16, DIM, 1>(p, dev, err, s);
    return p.f16 ? by_cache<Fp16, DIM, 2>(p, dev, err, s) : by_cache<Bf16, DIM, 2>(p, dev, err, s);
}

}  // namespace

size_t paged_attention_workspace(int group, int dim, int64_t max_len)
{
    return max_len <= kWholeKeys ? 0 : (size_t)kMostBlocks * 2 * (group <= 8 ? 8 : 16) * (dim + 2) * sizeof(float);
}

int paged_attention_launches(const PagedAttention& p)
{
    return longest_of(p) > kWholeKeys ? 2 : 1;
}

cudaError_t launch_paged_attention(const PagedAttention& p, const DeviceInfo& dev, cudaStream_t s)
{
    unsigned int* err = nullptr;
    cudaError_t e = device_error_ptr(&err);
    if (e != cudaSuccess)
        return e;
    return p.cache.dim == 64 ? by_type<64>(p, dev, err, s) : by_type<128>(p, dev, err, s);
}

}  // namespace ck
