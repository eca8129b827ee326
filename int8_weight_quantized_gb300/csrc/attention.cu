// attention.cu -- attention over whole prompts, ragged batches of them, causal or not, with a
// sliding window and first tokens that stay visible.
//
//   out[i,h] = sum_j w_j v_j / sum_j w_j,  w_j = exp(scale * q_i . k_j - max), j over the keys
//   of query i's sequence that it sees; zeros where it sees none (NaN, 0 / 0, where all scores that
//   it sees are -inf).
//
// Bound: the tensor cores, 4 dim flops per visible pair and head (and next to them the
// exponentials, one per pair and head).
//
// An item is two tiles of 128 queries: the same queries of two heads that share their keys, or,
// where a group's heads are odd in number, 256 queries of one head; or one tile alone, where there
// are few.  It walks the key tiles (128
// keys) that any of them sees, a query tile skipping those that it sees nothing of.  One block per
// SM takes items by turns (the longest first, every second round backwards), and its roles run on
// from item to item: the first scores of the next are computed while the last sums of one are
// stored.
//   warp 0      copies by TMA: the two Q tiles, then K and V tiles through one ring;
//   warp 1      issues the products, one lane: S_t = Q_t K^T (both operands in shared
//               memory) and O_t += P_t V (P from tensor memory, V as it lies, keys by columns),
//               all accumulators in tensor memory;
//   warp 2      works out the items ahead of the others, which find them in shared memory (a
//               search and divisions: 2000 to 3000 cycles between two items while every role did
//               its own);
//   warp 3      checks the sequences' bounds, then idles (it completes the warpgroup for the register
//               re-balancing);
//   warps 4-11  softmax, a warpgroup for each query tile, one thread per query row: reads its
//               row of S with its maximum, writes the weights back over S as the 16-bit
//               operand P of the second product, with heads of 128 in two parts.
// While the softmax of one tile runs, the products of the other keep the tensor cores busy:
// the issue order is O_0 += P_0 V_j, S_0 = Q_0 K_{j+1}, O_1 += P_1 V_j, S_1 = Q_1 K_{j+1}.
//
// A few first tokens (up to 32 of them, before the windows) are a narrow key tile: 32 scores a row,
// a quarter of the value product (before the loads brought the maximum: window of 1024 with 4 first
// tokens over 16000 148 us with a whole tile, 140 so; six short prompts 18.7 and 16.8).
//
// Measured (GB300; 16 query heads on 4 of 128 values, bf16): 16384 causal tokens 672 to 690 us, 1590
// to 1640 TFLOP/s, 81 to 84% of cuBLAS's measured rate; 8192 not causal 358 to 389 us, 1410 to 1540;
// window of 1024 with 4 first tokens over 16000 (2 key heads) 123 to 132 us; heads of 64, 8192 causal
// 131 us, 1050.
// A step (a key tile against both query tiles) takes 1.56 us, some 2900 cycles, of which the 32
// products of the two tiles take 2250: what it lasts is the chain of one tile, its score product, its softmax,
// the rest of its value product, and hand-overs of 300 to 400 cycles between them.  Between two
// items some 5000 cycles pass in the output and the next tile's first, masked softmax: a sixth of
// an item with that window.
//
// Online softmax: the load of the scores from tensor memory brings their maximum along
// (tcgen05.ld.red; found by the row's thread it took a fifth of the softmax: 703 instead of 685 us
// for 16384 tokens, 153 instead of 133 with heads of 64).  A row's sums stay relative to a reference
// m that may trail its maximum by up to 2^8; beyond that the thread brings m, the sum and O (in
// tensor memory) up to it first, which is seldom.  m only scales sums in floating point, so how far
// it trails costs no precision.  S_{j+1} being complete means that O += P_j V_j is, since it was
// issued before.
//
// What a mask hides has no part in a row: hidden scores are replaced, not multiplied.  A V row
// that some of a tile's queries see and others do not, or that lies beyond the sequence's end,
// is multiplied by a weight of zero for those: harmless unless it holds an infinity or NaN, and
// then the sums of the rows it does not belong to become NaN, never a wrong number.  So a warp that
// has met a sum that is not finite goes through its items once more when all are done, and where a
// masked tile's V rows hold such a value, it computes those rows again from visible keys
// (repair_rows): after all items, since no other role then waits for it, with a limit on its wait.
// Measured, one channel of infinities in every V row, fp16, heads of 128: 4096 causal tokens of 4
// heads 2.4 ms (0.05 without; 52 as rows one at a time between the items, which at some 100000 tokens
// would have outlasted the other roles' limits), 16384 of 16 heads 56 ms; a NaN in the last of 4096
// rows alone 0.5 ms.
//
// Rounding to fewer bits: each weight once, to the 16-bit type of V, as the tensor core takes
// it; scores, sums, maxima and O are fp32.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_common.cuh"
#include "tensor_core.cuh"
#include "transformer.h"
#include "warp_mma.cuh"

namespace ck {
namespace {

constexpr int BM = 128;              // query rows of a tile, keys of a key tile
constexpr int THREADS = 384;
// registers after the warpgroups re-balance; 384 threads start with 168 each
constexpr uint32_t REGS_LOAD = 88, REGS_SOFTMAX = 208;
constexpr uint32_t REGS_NEEDED_PER_BLOCK = 128 * REGS_LOAD + 256 * REGS_SOFTMAX;
constexpr uint32_t TMEM_COLS = 512;
constexpr int NARROW = 32;           // keys of a key tile of a few first tokens
// Weights of a tile that are handed over first, so that their value product starts while the others
// are worked out: 16384 causal tokens 672 us, 693 with all at once, 693 with 32, 673 with 96 (window
// of 1024 over 16000: 125, 128, 126, 129).  With heads of 64 it changes nothing (8192 causal tokens
// 135 us) or adds a wait (six short prompts 15.7 us, 15.4 with all at once).
template <int DIM>
constexpr int FIRST_KEYS = DIM == 128 ? 64 : 0;
constexpr int ITEMS = 2;              // items worked out ahead
constexpr int ITEM_READERS = 10;      // warps 0, 1 and 4-11
constexpr uint64_t TIMEOUT_NS = 2000000000ull;
constexpr float kLag = 8.0f;         // how far (log2) a row's reference may trail its maximum

template <int DIM>
struct Cfg {
    static constexpr int BOXES = DIM / 64;                     // 128-byte wide boxes of a tile
    static constexpr uint32_t BOX_BYTES = BM * 128;
    static constexpr uint32_t TILE_BYTES = BOXES * BOX_BYTES;  // a Q, K or V tile
    static constexpr int STAGES = DIM == 128 ? 2 : 4;          // ring of {V_j, K_{j+1}}; K_0 apart
    static constexpr uint32_t Q_BYTES = 2 * TILE_BYTES;
    static constexpr size_t STATE = 512;                       // barriers, items
    static constexpr size_t SMEM = 1024 + Q_BYTES + (1 + 2 * STAGES) * TILE_BYTES + STATE;
    static_assert(SMEM <= 232448, "shared memory budget");
};

struct PromptArgs {
    const void *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;
    const int32_t *cu_q, *cu_k;
    int64_t batch, total_q, total_k;
    int q_heads, kv_heads;
    bool causal, negate;
    float scale, c;  // c = |scale| log2 e
    int64_t window, sinks;
    void* out;
    float* lse;
    bool pair;       // an item's two tiles are the same queries of two heads
    int rows_log2;   // query rows of an item
    int64_t slots;   // items along the queries
    int64_t items;   // slots * (heads, or pairs of heads)
};

// Which keys an item's rows see, and the key tiles to walk.  WINDOW: whether the call has one.
template <bool WINDOW>
struct Item {
    int64_t q_row, k_row;  // first query row of the item, first key row of the sequence
    int head;              // of tile 0
    int step;              // query rows between the item's tiles: BM, or 0 where they differ by head
    bool done;             // there is no such item: the block's work is done
    bool bad;              // its sequence's bounds are out of range
    int rows;              // queries of the item
    int keys;              // keys of the sequence
    int offset;            // query r of the item stands at key position r + offset
    bool causal;
    int window, sinks;
    int prefix, first, count;  // key tiles: 0 .. prefix - 1, then first ..; count in all

    __device__ __forceinline__ int key0(int j) const { return BM * (!WINDOW || j < prefix ? j : first + (j - prefix)); }
    __device__ __forceinline__ int hi(int r) const { return causal ? min(r + offset, keys - 1) : keys - 1; }  // last key row r sees
    __device__ __forceinline__ int lo(int r) const { return WINDOW ? max(r + offset - window + 1, 0) : 0; }
    __device__ __forceinline__ int last_row(int t) const { return min(step * t + BM, rows) - 1; }
    __device__ __forceinline__ bool any(int t) const { return step * t < rows && hi(last_row(t)) >= 0; }
    // key tiles that query tile t has a part in: j < heads() (first tokens) or begin(t) <= j, up
    // to last(t) (-1: none)
    __device__ __forceinline__ int heads() const { return WINDOW ? prefix + (max(sinks - BM * first, 0) + BM - 1) / BM : 0; }
    __device__ __forceinline__ int last(int t) const { return any(t) ? (WINDOW ? prefix - first : 0) + hi(last_row(t)) / BM : -1; }
    __device__ __forceinline__ int begin(int t) const { return WINDOW ? prefix + max(lo(step * t) / BM - first, 0) : 0; }
    // whether of key tile 0 only the first NARROW keys are seen: first tokens before the windows
    __device__ __forceinline__ bool narrow() const { return WINDOW && prefix == 1 && sinks <= NARROW; }
    // whether some row does not see all of it
    __device__ __forceinline__ bool partial(int t, int k0) const
    {
        return k0 + BM - 1 > hi(step * t) || (WINDOW && lo(last_row(t)) > k0 && k0 + BM > sinks);
    }
};

// The sequence with slot `s` (slot_of(b) = max(cu[b], 0) / rows + b leaves room for every ragged
// end, needs no sums over lengths and ascends): the last b with slot_of(b) <= s.
__device__ __forceinline__ int64_t sequence_of_slot(const int32_t* cu, int64_t batch, int rows_log2, int64_t s)
{
    int64_t lo = 0, hi = batch;
    while (hi - lo > 1) {
        const int64_t mid = (lo + hi) >> 1;
        if ((int64_t)(max(__ldg(cu + mid), 0) >> rows_log2) + mid <= s)
            lo = mid;
        else
            hi = mid;
    }
    return lo;
}

// The key tiles of one query tile, as the roles test them.
template <bool WINDOW>
struct Active {
    int heads, begin, last;
    __device__ __forceinline__ bool operator()(int j) const { return j <= last && (!WINDOW || j < heads || j >= begin); }
};

// Bits of a pair of 16-bit values whose exponents are all ones: infinity or NaN.
template <class E>
__device__ __forceinline__ uint32_t not_finite(uint32_t pair)
{
    constexpr uint32_t EXP = std::is_same<E, Bf16>::value ? 0x7F80u : 0x7C00u;
    return ((pair & EXP) == EXP ? 0x0000FFFFu : 0u) | ((pair >> 16 & EXP) == EXP ? 0xFFFF0000u : 0u);
}

// Rows r0 .. r0 + 15 of an item, of which those in `rows` are wanted, by one warp, from visible keys
// only: the outputs alone (hidden values do not reach a row's maximum and sum).  Both products on
// the 16x8x16 matrix instruction, 16 keys at a time, query rows as its rows, online softmax; weights
// rounded once to the type of V, as above.  Infinities and NaN of V take no part in the product,
// which they would reach through hidden keys' weights of zero: each is added to the rows that see it.
template <class E, int DIM, bool WINDOW>
__device__ __forceinline__ void attend_rows(const PromptArgs& p, const Item<WINDOW>& w, int r0, uint32_t rows, int head,
                                            int kv_head)
{
    using T = typename E::T;
    constexpr int W = DIM / 8;  // columns of V that a lane loads of a key; tiles of 8 output columns
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    const T* k = static_cast<const T*>(p.k) + w.k_row * p.k_stride + (int64_t)kv_head * DIM;
    const T* v = static_cast<const T*>(p.v) + w.k_row * p.v_stride + (int64_t)kv_head * DIM;
    const float factor = p.scale * kLog2e;

    // this lane's two rows: what they see, their queries (k-step pair i, lane t: values 32 i + 8 t ..)
    int hi[2], lo[2];
    uint32_t qa[DIM / 16][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int r = r0 + g + 8 * h;
        const bool wanted = (rows >> (g + 8 * h)) & 1u;
        hi[h] = wanted ? w.hi(r) : -1;
        lo[h] = wanted ? w.lo(r) : 0x7FFFFFFF;
        const T* q = static_cast<const T*>(p.q) + (w.q_row + (wanted ? r : 0)) * p.q_stride + (int64_t)head * DIM + 8 * t;
#pragma unroll
        for (int i = 0; i < DIM / 32; ++i) {
            const uint4 x = __ldg(reinterpret_cast<const uint4*>(q + 32 * i));
            qa[2 * i][h] = x.x, qa[2 * i][2 + h] = x.y;
            qa[2 * i + 1][h] = x.z, qa[2 * i + 1][2 + h] = x.w;
        }
    }
    const int last = __reduce_max_sync(0xffffffffu, max(hi[0], hi[1]));
    const int first = WINDOW ? min(__reduce_min_sync(0xffffffffu, min(lo[0], lo[1])), last + 1) : 0;

    float acc[W][4] = {};  // tile e: rows g, g + 8 of columns W (2t) + e, W (2t + 1) + e
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
    // the first tokens before the windows, then the windows' union
#pragma unroll 1
    for (int run = WINDOW ? 0 : 1; run < 2; ++run) {
        const int end = run == 0 ? min(w.sinks, first) : last + 1;
#pragma unroll 1
        for (int k0 = run == 0 ? 0 : first; k0 < end; k0 += 16) {
            auto row_of = [&](int i) { return (int64_t)min(k0 + i, end - 1); };  // keys past the run: its last, hidden
            auto sees = [&](int h, int i) {
                const int key = k0 + i;
                return key < end && key <= hi[h] && (!WINDOW || key >= lo[h] || (key < w.sinks && hi[h] >= 0));
            };
            float x[2][4] = {};  // [h]: rows; keys 8 u + 2t, + 1 in 2 u, + 1
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                float s[4] = {};
                const T* src = k + row_of(8 * u + g) * p.k_stride + 8 * t;
#pragma unroll
                for (int i = 0; i < DIM / 32; ++i) {
                    const uint4 b = __ldg(reinterpret_cast<const uint4*>(src + 32 * i));
                    mma_16816<E>(s, qa[2 * i], b.x, b.y);
                    mma_16816<E>(s, qa[2 * i + 1], b.z, b.w);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    x[i >> 1][2 * u + (i & 1)] = sees(i >> 1, 8 * u + 2 * t + (i & 1)) ? s[i] * factor : -INFINITY;
            }
            float keep[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float top = fmaxf(fmaxf(x[h][0], x[h][1]), fmaxf(x[h][2], x[h][3]));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2)), m[h]);
                const float ref = top == -INFINITY ? 0.0f : top;
                keep[h] = fast_exp2(m[h] - ref);
                m[h] = top;
                l[h] *= keep[h];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[h][i] = fast_exp2(x[h][i] - ref);
                    l[h] += x[h][i];
                }
            }
            const uint32_t pa[4] = {E::pack2(x[0][0], x[0][1]), E::pack2(x[1][0], x[1][1]), E::pack2(x[0][2], x[0][3]),
                                    E::pack2(x[1][2], x[1][3])};
            if (__any_sync(0xffffffffu, keep[0] != 1.0f || keep[1] != 1.0f))
#pragma unroll
                for (int e = 0; e < W; ++e)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        acc[e][i] *= keep[i >> 1];
            // values: this lane's keys 2t, 2t + 1, 2t + 8, 2t + 9, columns W g .. W g + W - 1
            uint32_t bad = 0;  // keys that hold an infinity or NaN
#pragma unroll
            for (int c = 0; c < W / 8; ++c) {
                uint32_t vw[4][4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int key = 2 * t + (i & 1) + 8 * (i >> 1);
                    const uint4 b = __ldg(reinterpret_cast<const uint4*>(v + row_of(key) * p.v_stride + W * g + 8 * c));
                    vw[i][0] = b.x, vw[i][1] = b.y, vw[i][2] = b.z, vw[i][3] = b.w;
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const uint32_t drop = not_finite<E>(vw[i][n]);
                        vw[i][n] &= ~drop;
                        bad |= drop ? 1u << key : 0u;
                    }
                }
#pragma unroll
                for (int n = 0; n < 8; ++n)
                    mma_16816<E>(acc[8 * c + n], pa, __byte_perm(vw[0][n / 2], vw[1][n / 2], n & 1 ? 0x7632 : 0x5410),
                                 __byte_perm(vw[2][n / 2], vw[3][n / 2], n & 1 ? 0x7632 : 0x5410));
            }
            bad = __reduce_or_sync(0xffffffffu, bad);
#pragma unroll 1
            for (; bad; bad &= bad - 1) {
                const int key = __ffs(bad) - 1;
                const bool seen[2] = {sees(0, key), sees(1, key)};
                const T* src = v + row_of(key) * p.v_stride + 2 * W * t;
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int c = 0; c < W / 8; ++c) {
                        const uint4 b = __ldg(reinterpret_cast<const uint4*>(src + W * h + 8 * c));
                        const uint32_t word[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                        for (int n = 0; n < 4; ++n) {
                            const float2 y = E::to2(word[n]);
                            const int e = 8 * c + 2 * n;
#pragma unroll
                            for (int r = 0; r < 2; ++r) {
                                acc[e][h + 2 * r] += seen[r] && !(fabsf(y.x) < INFINITY) ? y.x : 0.0f;
                                acc[e + 1][h + 2 * r] += seen[r] && !(fabsf(y.y) < INFINITY) ? y.y : 0.0f;
                            }
                        }
                    }
            }
        }
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
        l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
        if (!((rows >> (g + 8 * r)) & 1u))
            continue;
        T* dst = static_cast<T*>(p.out) + ((w.q_row + r0 + g + 8 * r) * p.q_heads + head) * DIM + 2 * W * t;
        const float f = hi[r] < 0 ? 0.0f : 1.0f / l[r];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int c = 0; c < W / 8; ++c) {
                uint32_t word[4];
#pragma unroll
                for (int n = 0; n < 4; ++n)
                    word[n] = E::pack2(acc[8 * c + 2 * n][h + 2 * r] * f, acc[8 * c + 2 * n + 1][h + 2 * r] * f);
                *reinterpret_cast<uint4*>(dst + W * h + 8 * c) = make_uint4(word[0], word[1], word[2], word[3]);
            }
    }
}

// The 32 rows of a warp in an item, after their outputs: those that are not finite are computed again
// if a value that a mask hides from some of them is not (a key tile's values are multiplied by the
// weights of all its rows, zeros among them).
template <class E, int DIM, bool WINDOW>
__device__ __forceinline__ void repair_rows(const PromptArgs& p, const Item<WINDOW>& w, int t, int r0, int head, int kv_head)
{
    using T = typename E::T;
    const int lane = threadIdx.x & 31;
    const uint4* out = reinterpret_cast<const uint4*>(static_cast<const T*>(p.out) + ((w.q_row + r0) * p.q_heads + head) * DIM);
    auto any_bad = [](const uint4& x) {
        return (not_finite<E>(x.x) | not_finite<E>(x.y) | not_finite<E>(x.z) | not_finite<E>(x.w)) != 0;
    };
    constexpr int LANES = DIM / 8;  // lanes that share a row
    uint32_t again = 0;
#pragma unroll 1
    for (int i = 0; i < 32; i += 32 / LANES) {
        const int r = i + lane / LANES;
        if (r0 + r < w.rows && any_bad(out[(int64_t)r * p.q_heads * LANES + lane % LANES]))
            again |= 1u << r;
    }
    again = __reduce_or_sync(0xffffffffu, again);
    if (again == 0)
        return;
    const T* v = static_cast<const T*>(p.v) + w.k_row * p.v_stride + (int64_t)kv_head * DIM + lane % LANES * 8;
    const Active<WINDOW> active = {w.heads(), w.begin(t), w.last(t)};
    bool found = false;
#pragma unroll 1
    for (int j = 0; j < w.count && !found; ++j) {
        const int k0 = w.key0(j);
        if (!active(j) || !w.partial(t, k0))
            continue;
        for (int key = k0 + lane / LANES; key < k0 + BM && w.k_row + key < p.total_k; key += 32 / LANES)
            found |= any_bad(__ldg(reinterpret_cast<const uint4*>(v + key * p.v_stride)));
        found = __any_sync(0xffffffffu, found);
    }
    if (!found)
        return;
#pragma unroll 1
    for (int i = 0; i < 32; i += 16)
        if ((again >> i) & 0xFFFFu)
            attend_rows<E, DIM, WINDOW>(p, w, r0 + i, (again >> i) & 0xFFFFu, head, kv_head);
}

template <class E, int DIM, bool WINDOW>
__global__ void __launch_bounds__(THREADS, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const PromptArgs p, unsigned int* err)
{
    using C = Cfg<DIM>;
    using T = typename E::T;
    using Item = ck::Item<WINDOW>;
    using Active = ck::Active<WINDOW>;
    constexpr int STAGES = C::STAGES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* s_q = smem;
    uint8_t* s_k0 = smem + C::Q_BYTES;
    uint8_t* s_ring = s_k0 + C::TILE_BYTES;
    uint64_t* bars = reinterpret_cast<uint64_t*>(s_ring + (size_t)2 * STAGES * C::TILE_BYTES);
    uint64_t* q_full = bars;             // [2]
    uint64_t* s_full = bars + 2;         // [2] S_t is complete (and every product before it)
    uint64_t* p_full = bars + 4;         // [2] P_t is written
    uint64_t* o_full = bars + 6;         // [2] O_t is final
    uint64_t* q_empty = bars + 8;        // [2] the item's last scores of tile t are computed
    uint64_t* k0_full = bars + 10;
    uint64_t* k0_empty = bars + 11;
    uint64_t* drain = bars + 12;
    uint64_t* p_half = bars + 13;        // [2] P_t is for its first keys, O_t may be added to
    uint64_t* full = bars + 15;          // [STAGES] V_j and K_{j+1} have landed
    uint64_t* empty = full + STAGES;     // [STAGES] their products are done
    uint64_t* item_full = empty + STAGES;       // [ITEMS]
    uint64_t* item_empty = item_full + ITEMS;   // [ITEMS]
    Item* s_items = reinterpret_cast<Item*>(item_empty + ITEMS);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(s_items + ITEMS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    static_assert((15 + 2 * STAGES + 2 * ITEMS) * 8 + ITEMS * sizeof(Item) + 8 <= C::STATE, "barriers and items");

    const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    if (warp == 0 && lane == 0) {
        for (int t = 0; t < 2; ++t) {
            mbar_init(&q_full[t], 1);
            mbar_init(&s_full[t], 1);
            mbar_init(&p_full[t], 4);
            mbar_init(&p_half[t], 4);
            mbar_init(&o_full[t], 1);
            mbar_init(&q_empty[t], 1);
        }
        mbar_init(k0_full, 1);
        mbar_init(k0_empty, 1);
        mbar_init(drain, 1);
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int s = 0; s < ITEMS; ++s) {
            mbar_init(&item_full[s], 1);
            mbar_init(&item_empty[s], ITEM_READERS);
        }
        *abort_flag = 0;
        fence_mbar_init();
        fence_proxy_async_smem();
        tma_prefetch_desc(&tmQ);
        tma_prefetch_desc(&tmK);
        tma_prefetch_desc(&tmV);
    }
    if (warp == 1) {
        tmem_alloc(tmem_slot, TMEM_COLS);
        tmem_relinquish();
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, *tmem_slot, 0);
    griddep_wait();

    // ---- the block's items.  Item i counts from the last slot down: causal prompts' longest
    // tiles first.
    const int units = p.pair ? p.q_heads / 2 : p.q_heads;
    auto item_at = [&](int64_t round) {
        const int64_t blocks = gridDim.x;
        const int64_t i = round * blocks + ((round & 1) ? blocks - 1 - blockIdx.x : blockIdx.x);
        Item w{};
        w.done = i >= p.items;
        if (w.done)
            return w;
        const int64_t slot = p.slots - 1 - i / units;
        w.head = (int)(i % units) << (p.pair ? 1 : 0);
        w.step = p.pair ? 0 : BM;
        const int64_t b = sequence_of_slot(p.cu_q, p.batch, p.rows_log2, slot);
        const int64_t q0 = __ldg(p.cu_q + b), q1 = __ldg(p.cu_q + b + 1);
        const int64_t k0 = __ldg(p.cu_k + b), k1 = __ldg(p.cu_k + b + 1);
        const bool bad_q = q0 < 0 || q1 < q0 || q1 > p.total_q;
        w.bad = bad_q || k0 < 0 || k1 < k0 || k1 > p.total_k;
        const int64_t start = max(q0, (int64_t)0);
        const int64_t r0 = (slot - ((start >> p.rows_log2) + b)) << p.rows_log2;
        w.q_row = start + r0;
        // (of a sequence with bounds out of range the rows inside the tensor)
        w.rows = r0 < 0 ? 0 : (int)min((int64_t)1 << p.rows_log2, max(min(q1, p.total_q) - w.q_row, (int64_t)0));
        w.k_row = k0;
        w.keys = w.bad ? 0 : (int)(k1 - k0);
        w.offset = w.bad ? 0 : (int)(r0 + (k1 - k0) - (q1 - q0));
        w.causal = p.causal;
        w.window = WINDOW ? (int)min(p.window, (int64_t)0x3FFFFFFF) : 0;
        w.sinks = WINDOW ? (int)min(p.sinks, (int64_t)0x3FFFFFFF) : 0;
        // key tiles: those of the first tokens, then those of the windows' union
        const int top = w.rows > 0 ? w.hi(w.rows - 1) : -1;
        w.prefix = w.first = w.count = 0;
        if (top >= 0) {
            w.first = w.lo(0) / BM;
            if (w.sinks > 0 && w.first > 0) {
                w.prefix = min((min(w.sinks, top + 1) + BM - 1) / BM, w.first);
                // (first tokens that reach into the windows' union lie in its tiles)
            }
            w.count = w.prefix + top / BM - w.first + 1;
        }
        return w;
    };
    // fn(w) for the block's items in order, by a whole warp or by one lane; stops where fn returns
    // false.  Where the items stop coming (a wait gave up), `anyway` goes on with its own.  True if
    // all were done.
    auto each_item = [&](auto whole_warp, auto anyway, auto fn) {
        bool coming = true;
        for (int64_t n = 0;; ++n) {
            const int s = (int)(n % ITEMS);
            Item w;
            coming = coming &&
                     mbar_wait(&item_full[s], (uint32_t)(n / ITEMS) & 1u, abort_flag, err, kErrWaitAttention, TIMEOUT_NS);
            if (whole_warp.value)
                coming = __all_sync(0xffffffffu, coming);
            if (coming) {
                w = s_items[s];
                if (whole_warp.value)
                    __syncwarp();
                if (!whole_warp.value || lane == 0)
                    mbar_arrive(&item_empty[s]);
                if (whole_warp.value)
                    __syncwarp();
            } else if (anyway.value) {
                w = item_at(n);
            } else {
                return false;
            }
            if (w.done)
                return true;
            if (!fn(w))
                return false;
        }
    };
    const int group = p.q_heads / p.kv_heads;

    if (warp < 4) {
        setmaxnreg_dec<REGS_LOAD>();
        if (warp == 0) {
            // ---------------------------------------------------------------- copies
            if (lane == 0) {
                auto load = [&](const CUtensorMap* map, uint8_t* dst, uint64_t* bar, int h, int64_t row) {
                    for (int x = 0; x < C::BOXES; ++x)
                        tma_load_3d(dst + x * C::BOX_BYTES, map, bar, x * 64, h, (int32_t)row);
                };
                auto wait = [&](uint64_t* bar, uint32_t parity) {
                    return mbar_wait(bar, parity, abort_flag, err, kErrWaitAttention, TIMEOUT_NS);
                };
                uint32_t uses = 0, k0_uses = 0, q_uses[2] = {0, 0};  // loads so far of the ring, K_0, Q_t
                const bool done = each_item(std::false_type(), std::false_type(), [&](const Item& w) {
                    if (w.count == 0)
                        return true;
                    auto load_q = [&](int t) {
                        if (!w.any(t))
                            return true;
                        if (!wait(&q_empty[t], (q_uses[t] + 1) & 1u))
                            return false;
                        ++q_uses[t];
                        mbar_arrive_expect_tx(&q_full[t], C::TILE_BYTES);
                        load(&tmQ, s_q + t * C::TILE_BYTES, &q_full[t], w.head + (p.pair ? t : 0), w.q_row + w.step * t);
                        return true;
                    };
                    const int kv_head = w.head / group;
                    bool ok = load_q(0) && wait(k0_empty, (k0_uses + 1) & 1u);
                    if (!ok)
                        return false;
                    ++k0_uses;
                    mbar_arrive_expect_tx(k0_full, C::TILE_BYTES);
                    load(&tmK, s_k0, k0_full, kv_head, w.k_row + w.key0(0));
                    ok = load_q(1);
                    for (int j = 0; ok && j < w.count; ++j) {
                        const int s = uses % STAGES;
                        ok = wait(&empty[s], (uses / STAGES + 1) & 1u);
                        if (!ok)
                            break;
                        ++uses;
                        const bool more = j + 1 < w.count;
                        uint8_t* dst = s_ring + (size_t)s * 2 * C::TILE_BYTES;
                        mbar_arrive_expect_tx(&full[s], more ? 2 * C::TILE_BYTES : C::TILE_BYTES);
                        load(&tmV, dst, &full[s], kv_head, w.k_row + w.key0(j));
                        if (more)
                            load(&tmK, dst + C::TILE_BYTES, &full[s], kv_head, w.k_row + w.key0(j + 1));
                    }
                    return ok;
                });
                if (!done) {  // aborting: every issued copy lands before shared memory is released
                    for (uint32_t i = uses > STAGES ? uses - STAGES : 0; i < uses; ++i)
                        wait_out(&full[i % STAGES], (i / STAGES) & 1u, err, kErrWaitAttention, TIMEOUT_NS);
                    if (k0_uses > 0)
                        wait_out(k0_full, (k0_uses - 1) & 1u, err, kErrWaitAttention, TIMEOUT_NS);
                    for (int t = 0; t < 2; ++t)
                        if (q_uses[t] > 0)
                            wait_out(&q_full[t], (q_uses[t] - 1) & 1u, err, kErrWaitAttention, TIMEOUT_NS);
                }
            }
            __syncwarp();
        } else if (warp == 1) {
            // -------------------------------------------------------------- products
            // The whole warp walks the tiles, so that descriptors stay uniform values, and one
            // elected lane issues; the others wait for it after each issue (left to run ahead into
            // the next barrier's polling loop they can keep it from being scheduled).
            {
                const uint32_t idesc_s = idesc_of<E>(BM, false) | (p.negate ? 1u << 13 : 0u);
                const uint32_t idesc_n = idesc_of<E>(NARROW, false) | (p.negate ? 1u << 13 : 0u);
                constexpr uint32_t idesc_o = idesc_of<E>(DIM, true);
                const uint64_t q_desc = desc_kmajor_sw128(smem_u32(s_q));
                const uint64_t k0_desc = desc_kmajor_sw128(smem_u32(s_k0));
                const uint64_t k_desc = desc_kmajor_sw128(smem_u32(s_ring) + C::TILE_BYTES);
                const uint64_t v_desc = desc_nmajor_sw128(smem_u32(s_ring), C::BOX_BYTES);
                constexpr uint64_t kTile = C::TILE_BYTES >> 4, kBox = C::BOX_BYTES >> 4;
                uint32_t uses = 0, k0_uses = 0, q_uses[2] = {0, 0};
                uint32_t p_phase[2] = {0, 0};
                bool started[2];
                auto wait = [&](uint64_t* bar, uint32_t parity) {
                    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity)))
                        return true;
                    const bool ok = mbar_wait(bar, parity, abort_flag, err, kErrWaitAttention, TIMEOUT_NS);
                    return __all_sync(0xffffffffu, ok) != 0;
                };
                const bool leader = elect_one();
                auto scores = [&](int t, uint64_t b, uint32_t idesc) {  // S_t = Q_t K^T
                    const uint64_t a = q_desc + t * kTile;
#pragma unroll
                    for (int k = 0; k < DIM / 16; ++k)
                        mma_ss(tmem + t * BM, a + (k / 4) * kBox + (k % 4) * 2, b + (k / 4) * kBox + (k % 4) * 2, idesc,
                               k > 0);
                    mma_commit(&s_full[t]);
                };
                auto values = [&](int t, uint64_t b, auto from, auto keys) {  // O_t += P_t V
#pragma unroll
                    for (int k = from.value / 16; k < keys.value / 16; ++k)
                        mma_ts(tmem + 2 * BM + t * DIM, tmem + t * BM + k * 8, b + k * (16 * 128 >> 4), idesc_o,
                               k > 0 || started[t]);
                };
                // The tensor core takes a product about as fast as one thread issues it and queues
                // only a few, and every step of this warp beside the busy softmax warps takes some
                // 100 cycles: so one wait and one branch stand between two groups of products.
                each_item(std::true_type(), std::false_type(), [&](Item w) {
                    // the same in every lane; said so, descriptors and bounds stay uniform values
                    w.rows = __shfl_sync(0xffffffffu, w.rows, 0);
                    w.keys = __shfl_sync(0xffffffffu, w.keys, 0);
                    w.offset = __shfl_sync(0xffffffffu, w.offset, 0);
                    w.prefix = __shfl_sync(0xffffffffu, w.prefix, 0);
                    w.first = __shfl_sync(0xffffffffu, w.first, 0);
                    w.count = __shfl_sync(0xffffffffu, w.count, 0);
                    if (w.count == 0)
                        return true;
                    const bool narrow = __shfl_sync(0xffffffffu, w.narrow(), 0);
                    const Active active[2] = {{w.heads(), w.begin(0), w.last(0)}, {w.heads(), w.begin(1), w.last(1)}};
                    bool q_seen[2] = {false, false};
                    auto q_here = [&](int t) {
                        if (!q_seen[t] && !wait(&q_full[t], q_uses[t] & 1u))
                            return false;
                        q_uses[t] += q_seen[t] ? 0 : 1;
                        q_seen[t] = true;
                        return true;
                    };
                    started[0] = started[1] = false;
                    if (!wait(k0_full, k0_uses & 1u))
                        return false;
                    ++k0_uses;
#pragma unroll
                    for (int t = 0; t < 2; ++t)
                        if (active[t](0)) {
                            if (!q_here(t))
                                return false;
                            tc_fence_after();
                            if (leader) {
                                scores(t, k0_desc, narrow ? idesc_n : idesc_s);
                                if (active[t].last == 0)
                                    mma_commit(&q_empty[t]);
                            }
                            __syncwarp();
                        }
                    if (leader)
                        mma_commit(k0_empty);
                    __syncwarp();
                    auto step = [&](int j, auto keys) {
                        const int s = uses % STAGES;
                        const uint32_t parity = (uses / STAGES) & 1u;
                        ++uses;
                        const uint64_t v = v_desc + s * 2 * kTile, k = k_desc + s * 2 * kTile;
                        const bool more = j + 1 < w.count;
                        if (!wait(&full[s], parity))
                            return false;
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            const bool now = active[t](j), next = more && active[t](j + 1);
                            if (next && !q_here(t))
                                return false;
                            constexpr int FIRST = keys.value < FIRST_KEYS<DIM> ? keys.value : FIRST_KEYS<DIM>;
                            if (now) {
                                if constexpr (FIRST > 0) {
                                    if (!wait(&p_half[t], p_phase[t]))
                                        return false;
                                    tc_fence_after();
                                    if (leader)
                                        values(t, v, std::integral_constant<int, 0>(), std::integral_constant<int, FIRST>());
                                    __syncwarp();
                                }
                                if (!wait(&p_full[t], p_phase[t]))
                                    return false;
                                p_phase[t] ^= 1u;
                            }
                            tc_fence_after();
                            if (leader) {
                                if (now) {
                                    values(t, v, std::integral_constant<int, FIRST>(), keys);
                                    if (j == active[t].last)
                                        mma_commit(&o_full[t]);
                                }
                                if (next) {
                                    scores(t, k, idesc_s);
                                    if (j + 1 == active[t].last)
                                        mma_commit(&q_empty[t]);
                                }
                                if (t == 1)
                                    mma_commit(&empty[s]);
                            }
                            __syncwarp();
                            started[t] |= now;
                        }
                        return true;
                    };
                    int j = 0;
                    if (narrow && !step(j++, std::integral_constant<int, NARROW>()))
                        return false;
                    for (; j < w.count; ++j)
                        if (!step(j, std::integral_constant<int, BM>()))
                            return false;
                    return true;
                });
                // every product must be complete before tensor and shared memory are released
                if (leader) {
                    mma_commit(drain);
                    wait_out(drain, 0, err, kErrWaitAttention, TIMEOUT_NS);
                }
            }
            __syncwarp();
        } else if (warp == 2) {
            // ----------------------------------------------------------------- items
            if (lane == 0) {
                for (int64_t n = 0;; ++n) {
                    const int s = (int)(n % ITEMS);
                    const Item w = item_at(n);
                    if (!mbar_wait(&item_empty[s], (uint32_t)(n / ITEMS + 1) & 1u, abort_flag, err, kErrWaitAttention, TIMEOUT_NS))
                        break;
                    s_items[s] = w;
                    mbar_arrive(&item_full[s]);
                    if (w.done)
                        break;
                }
            }
            __syncwarp();
        } else {
            // ---------------------------------------------------------------- bounds
            // every sequence's, by some block: where they descend there need be no item of it
            bool bad = false;
            for (int64_t b = (int64_t)blockIdx.x * 32 + lane; b < p.batch; b += (int64_t)gridDim.x * 32) {
                const int32_t q0 = __ldg(p.cu_q + b), q1 = __ldg(p.cu_q + b + 1);
                const int32_t k0 = __ldg(p.cu_k + b), k1 = __ldg(p.cu_k + b + 1);
                bad |= q0 < 0 || q1 < q0 || q1 > p.total_q || k0 < 0 || k1 < k0 || k1 > p.total_k;
            }
            if (bad)
                atomicOr(err, kErrIndex);
            __syncwarp();
        }
    } else {
        // ---------------------------------------------------------------------- softmax
        setmaxnreg_inc<REGS_SOFTMAX>();
        const int t = (warp - 4) >> 2;
        const int quarter = warp & 3;  // tensor memory lanes that this warp may access
        const int row = quarter * 32 + lane;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        const uint32_t s_addr = tmem + lanes + t * BM, o_addr = tmem + lanes + 2 * BM + t * DIM;
        const float c = p.c;
        uint32_t phase = 0, o_phase = 0;
        bool ok = true;  // once a wait has given up, the remaining rows become NaN
        bool again = false;  // some row of the warp is not finite
        each_item(std::true_type(), std::true_type(), [&](const Item& w) {
        const int r = w.step * t + row;  // row of the item
        const int head = w.head + (p.pair ? t : 0);
        const int hi = w.hi(r), lo = w.lo(r);
        const Active active = {w.heads(), w.begin(t), w.last(t)};
        const bool any = w.any(t);
        float m = -INFINITY;  // what the row's sums are relative to, in units of scores
        float l = 0.0f;
        bool started = false;
        // bring the row's sums to the maximum `top`, where `raise`
        auto raise_to = [&](float top, bool raise) {
            const float f = raise ? fast_exp2((m - top) * c) : 1.0f;
            if (raise)
                m = top;
            l *= f;
            if (!started)
                return;
#pragma unroll 1
            for (int i = 0; i < DIM / 16; ++i) {
                uint32_t v[16];
                tmem_ld_32x32b_x16(o_addr + 16 * i, v);
                tmem_wait_ld();
#pragma unroll
                for (int n = 0; n < 16; ++n)
                    v[n] = __float_as_uint(__uint_as_float(v[n]) * f);
                tmem_st_32x32b_x16(o_addr + 16 * i, v);
            }
        };
        auto weigh = [&](int j, auto keys) {  // tile j, of which the first `keys` matter
            constexpr int CHUNKS = keys.value / 32;
            const int k0 = w.key0(j);
            ok = mbar_wait(&s_full[t], phase, abort_flag, err, kErrWaitAttention, TIMEOUT_NS);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok)
                return;
            phase ^= 1u;
            tc_fence_after();
            const bool masked = w.partial(t, k0);
            uint32_t sr[CHUNKS][32];
            float tops[CHUNKS];
#pragma unroll
            for (int i = 0; i < CHUNKS; ++i)
                tmem_ld_max_32x32b_x32(s_addr + 32 * i, sr[i], tops[i]);
            tmem_wait_ld();
            if (masked) {
#pragma unroll
                for (int i = 0; i < CHUNKS; ++i) {
                    // bit n: key k0 + 32 i + n is seen (k <= hi and (k >= lo or k < sinks))
                    const int a = k0 + 32 * i;
                    const int nh = hi - a + 1, nl = lo - a, ns = w.sinks - a;
                    const uint32_t upto = nh <= 0 ? 0u : nh >= 32 ? 0xffffffffu : (1u << nh) - 1u;
                    const uint32_t below = nl <= 0 ? 0u : nl >= 32 ? 0xffffffffu : (1u << nl) - 1u;
                    const uint32_t head = ns <= 0 ? 0u : ns >= 32 ? 0xffffffffu : (1u << ns) - 1u;
                    const uint32_t seen = WINDOW ? upto & (~below | head) : upto;
                    tops[i] = -INFINITY;
#pragma unroll
                    for (int n = 0; n < 32; ++n) {
                        sr[i][n] = (seen >> n) & 1u ? sr[i][n] : 0xff800000u;
                        tops[i] = fmaxf(tops[i], __uint_as_float(sr[i][n]));
                    }
                }
            }
            float top = fmaxf(tops[0], m);
#pragma unroll
            for (int i = 1; i < CHUNKS; ++i)
                top = fmaxf(top, tops[i]);
            const bool raise = (top - m) * c > kLag;  // (m is -inf before the first key)
            if (__any_sync(0xffffffffu, raise))
                raise_to(top, raise);
            const float mc = m == -INFINITY ? 0.0f : -m * c;  // no key seen yet: weights 0
            const float2 c2 = make_float2(c, c), mc2 = make_float2(mc, mc);
            float2 sum = make_float2(0.0f, 0.0f);
            constexpr int FIRST = CHUNKS < FIRST_KEYS<DIM> / 32 ? CHUNKS : FIRST_KEYS<DIM> / 32;
            auto part = [&](auto from, auto to) {
                uint32_t packed[to.value - from.value][16];
#pragma unroll
                for (int i = from.value; i < to.value; ++i)
#pragma unroll
                    for (int n = 0; n < 16; ++n) {
                        float2 x = f2_fma_rn(make_float2(__uint_as_float(sr[i][2 * n]), __uint_as_float(sr[i][2 * n + 1])), c2, mc2);
                        x.x = fast_exp2(x.x);
                        x.y = fast_exp2(x.y);
                        sum = f2_add_rn(sum, x);
                        packed[i - from.value][n] = E::pack2(x.x, x.y);
                    }
#pragma unroll
                for (int i = from.value; i < to.value; ++i)
                    tmem_st_32x32b_x16(s_addr + 16 * i, packed[i - from.value]);
            };
            if constexpr (FIRST > 0) {
                part(std::integral_constant<int, 0>(), std::integral_constant<int, FIRST>());
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&p_half[t]);
            }
            if constexpr (FIRST < CHUNKS)
                part(std::integral_constant<int, FIRST>(), std::integral_constant<int, CHUNKS>());
            l += sum.x + sum.y;
            started = true;
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                mbar_arrive(&p_full[t]);
            __syncwarp();  // before the next wait, as for the products
        };
        int j = 0;
        if (w.narrow()) {
            if (ok && active(0))
                weigh(0, std::integral_constant<int, NARROW>());
            j = 1;
        }
        for (; ok && j < w.count; ++j)
            if (active(j))
                weigh(j, std::integral_constant<int, BM>());
        // ---- the rows' outputs
        const int64_t out_row = w.q_row + r;
        const bool mine = r < w.rows;
        const int rows = w.rows - (r - lane);  // of the warp
        const int64_t out_stride = (int64_t)p.q_heads * DIM;
        T* out = static_cast<T*>(p.out) + ((out_row - lane) * p.q_heads + head) * DIM;  // of lane 0
        if (ok && any) {
            ok = mbar_wait(&o_full[t], o_phase, abort_flag, err, kErrWaitAttention, TIMEOUT_NS);
            ok = __all_sync(0xffffffffu, ok);
            o_phase ^= 1u;
            tc_fence_after();
            if (ok) {
                const float f = hi < 0 ? 0.0f : 1.0f / l;  // (scores of -inf alone: 0 / 0, as they should)
                float check = 0.0f;  // 0 while all is finite, else NaN
#pragma unroll 1
                for (int i = 0; i < DIM / 32; ++i) {
                    uint32_t v[32];
                    tmem_ld_32x32b_x32(o_addr + 32 * i, v);
                    tmem_wait_ld();
                    float x[32];
#pragma unroll
                    for (int n = 0; n < 32; ++n) {
                        x[n] = __uint_as_float(v[n]);
                        check = fmaf(x[n], 0.0f, check);
                    }
                    store_rows<E>(out + 32 * i, out_stride, lane, rows, x, f);
                }
                if (mine && p.lse != nullptr)
                    p.lse[(int64_t)head * p.total_q + out_row] = (m * c + log2f(l)) * kLn2;
                // (l is NaN or infinite only through scores, which masks replace: not for this)
                again |= __any_sync(0xffffffffu, mine && check != check);
            }
        }
        if (__builtin_expect(!ok || w.bad || !any, 0)) {
            // no keys: zeros; bounds out of range or a wait that gave up: NaN
            const bool nan = w.bad || !ok;
            float x[32];
#pragma unroll
            for (int n = 0; n < 32; ++n)
                x[n] = nan ? NAN : 0.0f;
#pragma unroll 1
            for (int i = 0; i < DIM / 32; ++i)
                store_rows<E>(out + 32 * i, out_stride, lane, rows, x, 1.0f);
            if (mine && p.lse != nullptr)
                p.lse[(int64_t)head * p.total_q + out_row] = nan ? NAN : -INFINITY;
        }
        // O is read: the item's last hand-over of P was before that, so the next item's first one,
        // which lets O be written again, says so too
        tc_fence_before();
        return true;
        });
        // after all items, where no role waits for this one
        if (ok && __builtin_expect(again, 0)) {
            __syncwarp();  // the rows' own stores come first
#pragma unroll 1
            for (int64_t n = 0;; ++n) {
                const Item w = item_at(n);
                if (w.done)
                    break;
                const int r0 = w.step * t + quarter * 32, head = w.head + (p.pair ? t : 0);
                if (w.any(t) && r0 < w.rows)
                    repair_rows<E, DIM, WINDOW>(p, w, t, r0, head, head / group);
            }
        }
    }
    griddep_launch_dependents();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}

// [rows, heads, dim] with `stride` elements between rows, copied as boxes of 128 rows x 64
// values of one head.
bool make_map(CUtensorMap* map, const void* base, int64_t rows, int heads, int dim, int64_t stride, bool f16,
              std::string* why)
{
    const cuuint64_t dims[3] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)rows};
    const cuuint64_t strides[2] = {(cuuint64_t)dim * 2, (cuuint64_t)stride * 2};
    const cuuint32_t box[3] = {64, 1, BM};
    return make_box_map(map, base, 3, dims, strides, box, f16, why);
}

template <class E, int DIM, bool WINDOW>
cudaError_t launch(const PromptAttention& p, const DeviceInfo& dev, unsigned int* err, cudaStream_t s, std::string* why)
{
    using C = Cfg<DIM>;
    // a kernel attribute belongs to the context it was set in: set once per context
    static ContextCache<int> cache;
    int done = 0;
    cudaError_t e = cache.get(&done, [](int* d) {
        *d = 1;
        cudaFuncAttributes fa;
        cudaError_t a = cudaFuncGetAttributes(&fa, prompt_kernel<E, DIM, WINDOW>);
        if (a != cudaSuccess)
            return a;
        // the softmax warps claim what warps 0-3 give back: the launch must provide the sum
        if ((uint32_t)(fa.numRegs + 7) / 8 * 8 * THREADS < REGS_NEEDED_PER_BLOCK)
            return cudaErrorLaunchOutOfResources;
        return cudaFuncSetAttribute(prompt_kernel<E, DIM, WINDOW>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM);
    });
    if (e != cudaSuccess)
        return e;
    CUtensorMap q, k, v;
    if (!make_map(&q, p.q, p.total_q, p.q_heads, DIM, p.q_stride, p.f16, why))
        return cudaErrorInvalidValue;
    k = v = q;  // without keys no block copies any
    if (p.total_k > 0 && (!make_map(&k, p.k, p.total_k, p.kv_heads, DIM, p.k_stride, p.f16, why) ||
                          !make_map(&v, p.v, p.total_k, p.kv_heads, DIM, p.v_stride, p.f16, why)))
        return cudaErrorInvalidValue;
    PromptArgs a{};
    a.q = p.q, a.k = p.k, a.v = p.v;
    a.q_stride = p.q_stride, a.k_stride = p.k_stride, a.v_stride = p.v_stride;
    a.cu_q = p.cu_q, a.cu_k = p.cu_k;
    a.batch = p.batch, a.total_q = p.total_q, a.total_k = p.total_k;
    a.q_heads = p.q_heads, a.kv_heads = p.kv_heads;
    a.causal = p.causal;
    // the softmax wants a positive factor: a negative scale negates Q in the first product, and
    // for 0 the smallest factor that still keeps hidden scores (-inf) hidden stands in
    a.negate = p.scale < 0.0f;
    a.scale = p.scale;
    a.c = std::max(std::fabs(p.scale) * kLog2e, 1e-30f);
    a.window = p.causal ? p.window : 0;
    a.sinks = p.sinks;
    a.out = p.out;
    a.lse = p.lse;
    // Two heads that share their keys see the same key tiles; the next 128 queries see others at
    // both ends of theirs, where one tile then runs alone (16 heads on 4, pairs of heads against
    // 256 queries, when first tokens still took a whole tile: window of 1024 over 16000 tokens 148
    // against 159 us, six short prompts 18.7 against 20.2, 8192 causal tokens of 64 values 163
    // against 168).  Where there are no more tiles than multiprocessors, each has an item to itself:
    // its steps are shorter alone (1000 causal tokens of 16 heads: 14.3 us, 16.6 in pairs; 2000 of
    // 8: 22.6 and 27.0; 100 of 16: 6.3 and 6.7).
    const bool alone = ((p.total_q >> 7) + p.batch) * p.q_heads <= dev.sm_count;
    a.pair = !alone && p.q_heads / p.kv_heads % 2 == 0;
    a.rows_log2 = a.pair || alone ? 7 : 8;
    a.slots = (p.total_q >> a.rows_log2) + p.batch;
    a.items = a.slots * (a.pair ? p.q_heads / 2 : p.q_heads);
    const unsigned blocks = (unsigned)std::min<int64_t>(a.items, dev.sm_count);
    return launch_pdl(prompt_kernel<E, DIM, WINDOW>, dim3(blocks), dim3(THREADS), C::SMEM, s, q, k, v, a,
                      err);
}

}  // namespace

cudaError_t launch_attention(const PromptAttention& p, const DeviceInfo& dev, cudaStream_t s, std::string* why)
{
    unsigned int* err = nullptr;
    cudaError_t e = device_error_ptr(&err);
    if (e != cudaSuccess)
        return e;
    // A window has its own kernel: with its first tokens' tile in one for all, and before the loads
    // brought the maximum, 16384 causal tokens took 730 us instead of 716, 8192 that are not causal
    // 402 instead of 388.
    auto by_window = [&](auto type, auto dim) {
        using E = decltype(type);
        constexpr int DIM = decltype(dim)::value;
        return p.causal && p.window > 0 ? launch<E, DIM, true>(p, dev, err, s, why) : launch<E, DIM, false>(p, dev, err, s, why);
    };
    if (p.dim == 64)
        return p.f16 ? by_window(Fp16(), std::integral_constant<int, 64>()) : by_window(Bf16(), std::integral_constant<int, 64>());
    return p.f16 ? by_window(Fp16(), std::integral_constant<int, 128>()) : by_window(Bf16(), std::integral_constant<int, 128>());
}

}  // namespace ck
