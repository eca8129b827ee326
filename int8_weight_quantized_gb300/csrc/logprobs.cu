// logprobs.cu -- log probabilities of given tokens, the entropy and the top alternatives of rows of
// logits.
//
//   t_j = scale * (x_j - max x),  s = sum_j exp(t_j)
//   logprob = t_token - log s,  lse = scale * max x + log s,  entropy = log s - sum_j t_j exp(t_j) / s
//   top: the largest logits in order (NaN above all; of equal ones the lowest index first)
//
// Bound: HBM, each logit read once.
//
// A row is cut into pieces where there are few rows; a block of 8 warps takes a piece, 16 bytes a lane
// at a time, each warp with a maximum of its own that its sums are relative to.  A warp meets a new
// maximum seldom (once in the i-th of its steps with probability 1 / i): one vote a step finds it,
// together with what else is seldom.  Pieces of a row are joined by a second launch, always in the
// same order.
//
// Sums.  Terms above 1/4 (of the largest's 1) and the others have sums of their own, so that a sharp
// row's small rest, which is its entropy and the log probability of its likeliest token, does not lose
// its bits to the 1: log s = log1p((a - 1) + b).  With terms above 1/4 other than the 1 the rest is
// large itself.
//
// Top alternatives.  Each warp keeps its 32 best as (order of the logit, ~index) in one 64-bit number
// per lane, in descending order.  What exceeds its `top`-th goes to a buffer in shared memory; 32 of
// these are sorted and merged at a time (bitonic, 15 and 6 exchanges).  The first step's bar is the
// `top`-th of the lanes' largest, which as many logits reach.  So any order of the logits gives the
// same result, at most one merge for 32 logits (ascending ones).
#include <algorithm>
#include <cmath>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_common.cuh"
#include "transformer.h"
#include "warp_mma.cuh"

namespace ck {
namespace {

constexpr int WARPS = 8;
constexpr int THREADS = WARPS * 32;
constexpr int DEPTH = 4;                 // 16-byte loads of a lane in flight
constexpr int64_t kLeastPiece = 2048;    // logits
constexpr int64_t kPieces = 152 * 4;     // as many pieces as blocks fit at once
constexpr uint32_t FULL = 0xffffffffu;
constexpr float kNone = -160.0f;         // 2^-160 is 0 in fp32

// what a piece leaves: its maximum, sums relative to it, the 32 best
struct Part {
    uint64_t best[32];
    float m, a, b, w;  // w: sum of exp(t) t / ln 2
};

template <int TYPE>
struct Logit;
template <>
struct Logit<CK_OUT_F32> {
    using T = float;
    static constexpr int VEC = 4;
    static __device__ __forceinline__ float at(const T* p) { return __ldg(p); }
    static __device__ __forceinline__ void unpack(const uint4& v, float (&x)[VEC])
    {
        x[0] = __uint_as_float(v.x), x[1] = __uint_as_float(v.y), x[2] = __uint_as_float(v.z), x[3] = __uint_as_float(v.w);
    }
    static __device__ __forceinline__ float top(const uint4&, const float (&x)[VEC])
    {
        return max_nan(max_nan(x[0], x[1]), max_nan(x[2], x[3]));
    }
};
template <class E>
struct Logit16 {
    using T = typename E::T;
    static constexpr int VEC = 8;
    static __device__ __forceinline__ float at(const T* p) { return E::to(__ldg(p)); }
    static __device__ __forceinline__ void unpack(const uint4& v, float (&x)[VEC])
    {
        const uint32_t r[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = E::to2(r[i]);
            x[2 * i] = f.x, x[2 * i + 1] = f.y;
        }
    }
    static __device__ __forceinline__ float top(const uint4& v, const float (&)[VEC])
    {
        const uint32_t r[4] = {v.x, v.y, v.z, v.w};
        typename E::T2 h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            h[i] = *reinterpret_cast<const typename E::T2*>(&r[i]);
        const typename E::T2 m = __hmax2_nan(__hmax2_nan(h[0], h[1]), __hmax2_nan(h[2], h[3]));
        const float2 f = E::to2(*reinterpret_cast<const uint32_t*>(&m));
        return max_nan(f.x, f.y);
    }
};
template <>
struct Logit<CK_OUT_BF16> : Logit16<Bf16> {};
template <>
struct Logit<CK_OUT_F16> : Logit16<Fp16> {};

// Logits as integers in their order: NaN above +inf, -0 and +0 equal; never 0.
__device__ __forceinline__ uint32_t order_of(float x)
{
    if (x != x)
        return 0xffffffffu;
    const uint32_t u = x == 0.0f ? 0u : __float_as_uint(x);
    return (int32_t)u < 0 ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t order)
{
    return order == 0xffffffffu ? NAN : __uint_as_float((int32_t)order < 0 ? order & 0x7fffffffu : ~order);
}

// A bar that the logit of this order passes itself (NaN: everything passes).
__device__ __forceinline__ float below(uint32_t order)
{
    // (-0 is +0's equal)
    return order == 0xffffffffu ? NAN : value_of(order == 0x80000000u ? 0x7ffffffeu : order - 1u);
}

__device__ __forceinline__ uint64_t larger(uint64_t a, uint64_t b)
{
    return a > b ? a : b;
}

// One exchange of a bitonic network: the lane with bit `m` clear keeps the larger where `down`.
__device__ __forceinline__ uint64_t exchange(uint64_t k, int m, bool down)
{
    const uint64_t o = __shfl_xor_sync(FULL, k, m);
    const bool keep_larger = ((threadIdx.x & m) == 0) == down;
    return (o > k) == keep_larger ? o : k;
}

// 32 numbers in descending order over the lanes
__device__ __forceinline__ uint64_t sorted(uint64_t k)
{
#pragma unroll
    for (int size = 2; size <= 32; size *= 2)
#pragma unroll
        for (int m = size / 2; m > 0; m /= 2)
            k = exchange(k, m, size == 32 || (threadIdx.x & size) == 0);
    return k;
}

// The 32 largest of two descending sequences, descending
__device__ __forceinline__ uint64_t merged(uint64_t a, uint64_t b)
{
    uint64_t k = larger(a, __shfl_sync(FULL, b, 31 - (threadIdx.x & 31)));
#pragma unroll
    for (int m = 16; m > 0; m /= 2)
        k = exchange(k, m, true);
    return k;
}

__device__ __noinline__ uint64_t absorb(uint64_t best, uint64_t found)
{
    return merged(best, sorted(found));
}

// Sums of two sets of terms, the first brought from its reference to that of the second, `delta` =
// (first - second) c <= 0 above it in units of log 2 (what falls below 1/4 joins the small ones).
__device__ __forceinline__ void rescale(float& a, float& b, float& w, float delta)
{
    const float s = a + b;
    if (s == 0.0f)  // nothing yet; delta may be -inf
        return;
    const float f = fast_exp2(delta);
    w = f == 0.0f && delta == delta ? 0.0f : f * (w + delta * s);
    const bool small = f < 0.25f;
    b = small ? s * f : b * f;
    a = small ? 0.0f : a * f;
}

// A warp's way through its logits.
template <int TYPE, bool TOP>
struct Warp {
    using L = Logit<TYPE>;
    static constexpr int VEC = L::VEC;
    float c;         // scale / ln 2
    float near;      // what is above m - near is above 1/4
    float m = -INFINITY, ref = 0.0f;  // the maximum, and it or 0 where there is none yet
    float a = 0.0f, b = 0.0f, w = 0.0f;
    int top = 0;
    uint64_t best = 0;
    float bar = NAN;      // what is not <= bar goes to the buffer
    bool fresh = true;
    uint64_t* buffer = nullptr;  // [64]
    int waiting = 0;

    __device__ __forceinline__ void set_bar()
    {
        const uint64_t k = __shfl_sync(FULL, best, top - 1);
        bar = k == 0 ? NAN : value_of((uint32_t)(k >> 32));
    }
    __device__ __forceinline__ void merge_waiting()
    {
        __syncwarp();
        const int lane = threadIdx.x & 31;
        best = absorb(best, lane < waiting ? buffer[lane] : 0);
        const uint64_t rest = lane + 32 < waiting ? buffer[lane + 32] : 0;
        __syncwarp();
        buffer[lane] = rest;
        waiting = max(waiting - 32, 0);
        set_bar();
        __syncwarp();
    }
    // logits x[i] with index first + i, of which those in `valid` are there; largest: of these
    template <int N>
    __device__ __forceinline__ void take(const float (&x)[N], float largest, uint32_t first, uint32_t valid)
    {
        if (TOP) {
            if (fresh) {
                fresh = false;
                const uint64_t k = __shfl_sync(FULL, sorted(valid ? (uint64_t)order_of(largest) << 32 | 1u : 0), top - 1);
                if (k != 0)
                    bar = below((uint32_t)(k >> 32));
            }
            if (__any_sync(FULL, valid && !(largest <= bar))) {
                uint32_t found = 0;
#pragma unroll
                for (int i = 0; i < N; ++i)
                    found |= !(x[i] <= bar) ? 1u << i : 0u;
                found &= valid;
                while (__any_sync(FULL, found != 0)) {
                    const uint32_t with = __ballot_sync(FULL, found != 0);
                    if (found) {
                        const int i = __ffs(found) - 1;
                        found &= found - 1;
                        float v = x[0];
#pragma unroll
                        for (int n = 1; n < N; ++n)
                            v = n == i ? x[n] : v;
                        buffer[waiting + __popc(with & ((1u << (threadIdx.x & 31)) - 1u))] =
                            (uint64_t)order_of(v) << 32 | (FULL - (first + i));
                    }
                    waiting += __popc(with);
                    if (waiting >= 32)
                        merge_waiting();
                }
            }
        }
        if (__any_sync(FULL, !(largest <= m - near))) {
            float high = largest;
#pragma unroll
            for (int o = 16; o; o >>= 1)
                high = max_nan(high, __shfl_xor_sync(FULL, high, o));
            if (!(high <= m)) {
                rescale(a, b, w, (m - high) * c);
                m = ref = high;
            }
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float t = max_nan((x[i] - ref) * c, kNone);
                const float e = fast_exp2(t);
                a += e > 0.25f ? e : 0.0f;
                b += e > 0.25f ? 0.0f : e;  // (NaN too)
                w = fmaf(e, t, w);
            }
        } else {
            const float2 ref2 = make_float2(-ref, -ref), c2 = make_float2(c, c);
            float2 b2 = make_float2(b, 0.0f), w2 = make_float2(w, 0.0f);
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                float2 t = f2_mul_rn(f2_add_rn(make_float2(x[i], i + 1 < N ? x[i + 1] : -INFINITY), ref2), c2);
                t.x = max_nan(t.x, kNone), t.y = max_nan(t.y, kNone);
                const float2 e = make_float2(fast_exp2(t.x), fast_exp2(t.y));
                b2 = f2_add_rn(b2, e);
                w2 = f2_fma_rn(e, t, w2);
            }
            b = b2.x + b2.y;
            w = w2.x + w2.y;
        }
    }
};

// The parts of up to 32 pieces or warps, one a lane (m = -inf, zeros: none), as one.
__device__ __forceinline__ void join_sums(float& m, float& a, float& b, float& w, float c)
{
    float high = m;
#pragma unroll
    for (int o = 16; o; o >>= 1)
        high = max_nan(high, __shfl_xor_sync(FULL, high, o));
    rescale(a, b, w, (m - high) * c);
    m = high;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        a += __shfl_xor_sync(FULL, a, o);
        b += __shfl_xor_sync(FULL, b, o);
        w += __shfl_xor_sync(FULL, w, o);
    }
}

// A row's outputs, by one warp.
template <int TYPE>
__device__ __forceinline__ void leave(const TokenLogprobs& p, int64_t row, float m, float a, float b, float w, uint64_t best,
                                      unsigned int* err)
{
    using L = Logit<TYPE>;
    const int lane = threadIdx.x & 31;
    const bool finite = m - m == 0.0f;
    const float log_s = finite ? log1pf((a - 1.0f) + b) : NAN;
    if (lane == 0) {
        if (p.logprob) {
            const int token = __ldg(p.tokens + row);
            float r = 0.0f;
            if (token >= p.vocab) {
                r = NAN;
                atomicOr(err, kErrIndex);
            } else if (token >= 0) {
                const float x = L::at(static_cast<const typename L::T*>(p.logits) + row * p.stride + token);
                r = p.scale * (x - m) - log_s;
            }
            p.logprob[row] = r;
        }
        if (p.entropy)
            p.entropy[row] = log_s - w * kLn2 / (a + b);
        if (p.lse)
            p.lse[row] = finite ? p.scale * m + log_s : m;
    }
    if (lane < p.top) {
        p.top_index[row * p.top + lane] = (int32_t)(FULL - (uint32_t)best);
        p.top_logprob[row * p.top + lane] = p.scale * (value_of((uint32_t)(best >> 32)) - m) - log_s;
    }
}

template <int TYPE, bool TOP>
__global__ void __launch_bounds__(THREADS, 4) piece_kernel(const TokenLogprobs p, int pieces, int64_t piece, unsigned int* err)
{
    using L = Logit<TYPE>;
    using T = typename L::T;
    constexpr int VEC = L::VEC;
    griddep_wait();
    __shared__ uint64_t buffers[WARPS][64];
    __shared__ float sums[WARPS][4];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = blockIdx.x / pieces;
    const int number = (int)(blockIdx.x - row * pieces);
    const int64_t j0 = min(number * piece, p.vocab), j1 = min(j0 + piece, p.vocab);
    const T* x = static_cast<const T*>(p.logits) + row * p.stride;

    Warp<TYPE, TOP> me;
    me.c = p.scale * kLog2e;
    me.near = 2.0f / me.c;
    me.top = p.top;
    me.buffer = buffers[warp];

    // whole 16-byte vectors between v0 and v1; up to VEC - 1 logits on either side are warp 0's last step
    const int skew = (int)((reinterpret_cast<uintptr_t>(x + j0) / sizeof(T)) % VEC);
    const int64_t v0 = min(j0 + (skew ? VEC - skew : 0), j1), vectors = (j1 - v0) / VEC, v1 = v0 + vectors * VEC;
    const uint4* src = reinterpret_cast<const uint4*>(x + v0);
    const uint32_t low = (uint32_t)(TYPE == CK_OUT_F32 ? 0xff800000u : TYPE == CK_OUT_F16 ? 0xfc00fc00u : 0xff80ff80u);
    auto load = [&](int64_t v) {
        return v < vectors ? __ldcs(src + v) : make_uint4(low, low, low, low);
    };
    uint4 ahead[DEPTH];
    int64_t v = threadIdx.x;
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
        ahead[d] = load(v + d * THREADS);
    for (; v - lane < vectors; v += DEPTH * THREADS) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
            const uint4 now = ahead[d];
            const int64_t at = v + d * THREADS;
            ahead[d] = load(at + DEPTH * THREADS);
            if (at - lane < vectors) {  // the same for the warp
                float f[VEC];
                L::unpack(now, f);
                me.take(f, L::top(now, f), (uint32_t)(v0 + at * VEC), at < vectors ? (1u << VEC) - 1u : 0u);
            }
        }
    }
    if (warp == 0 && (v0 > j0 || j1 > v1)) {
        const int64_t j = lane < v0 - j0 ? j0 + lane : v1 + (lane - (v0 - j0));
        const bool there = lane < (v0 - j0) + (j1 - v1);
        if (TOP && !me.fresh && me.bar == me.bar)  // of equal ones these may come first
            me.bar = below(order_of(me.bar));
        const float f[1] = {there ? L::at(x + j) : -INFINITY};
        me.take(f, f[0], (uint32_t)j, there ? 1u : 0u);
    }
    if (TOP && me.waiting > 0)
        me.merge_waiting();

    // ---- the warps' parts as one
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        me.a += __shfl_xor_sync(FULL, me.a, o);
        me.b += __shfl_xor_sync(FULL, me.b, o);
        me.w += __shfl_xor_sync(FULL, me.w, o);
    }
    if (lane == 0)
        sums[warp][0] = me.m, sums[warp][1] = me.a, sums[warp][2] = me.b, sums[warp][3] = me.w;
    if (TOP)
        buffers[warp][lane] = me.best;
    __syncthreads();
    if (TOP)
#pragma unroll
        for (int n = WARPS / 2; n > 0; n /= 2) {
            if (warp < n) {
                me.best = merged(me.best, buffers[warp + n][lane]);
                buffers[warp][lane] = me.best;
            }
            __syncthreads();
        }
    if (warp == 0) {
        float m = -INFINITY, a = 0.0f, b = 0.0f, w = 0.0f;
        if (lane < WARPS)
            m = sums[lane][0], a = sums[lane][1], b = sums[lane][2], w = sums[lane][3];
        join_sums(m, a, b, w, me.c);
        if (pieces == 1) {
            leave<TYPE>(p, row, m, a, b, w, me.best, err);
        } else {
            Part* part = static_cast<Part*>(p.workspace) + blockIdx.x;
            if (TOP)
                part->best[lane] = me.best;
            if (lane == 0)
                *reinterpret_cast<float4*>(&part->m) = make_float4(m, a, b, w);
        }
    }
    griddep_launch_dependents();
}

// The pieces of a row as one: each of the block's warps takes every eighth, then the warps together.
template <int TYPE, bool TOP>
__global__ void __launch_bounds__(THREADS) join_kernel(const TokenLogprobs p, int pieces, unsigned int* err)
{
    griddep_wait();
    __shared__ uint64_t lists[WARPS][32];
    __shared__ float sums[WARPS][4];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = blockIdx.x;
    const Part* parts = static_cast<const Part*>(p.workspace) + row * pieces;
    const float c = p.scale * kLog2e;
    // (a lane takes pieces 32 apart: more than 256 pieces of a row only where it is longer than 2^19)
    float m = -INFINITY, a = 0.0f, b = 0.0f, w = 0.0f;
    for (int i = warp + lane * WARPS; i < pieces; i += 32 * WARPS) {
        const float4 f = __ldcg(reinterpret_cast<const float4*>(&parts[i].m));
        const float high = max_nan(m, f.x);
        float a2 = f.y, b2 = f.z, w2 = f.w;
        rescale(a, b, w, (m - high) * c);
        rescale(a2, b2, w2, (f.x - high) * c);
        m = high, a += a2, b += b2, w += w2;
    }
    join_sums(m, a, b, w, c);
    if (lane == 0)
        sums[warp][0] = m, sums[warp][1] = a, sums[warp][2] = b, sums[warp][3] = w;
    uint64_t best = 0;
    if (TOP) {
        for (int i = warp; i < pieces; i += WARPS)
            best = merged(best, __ldcg(reinterpret_cast<const unsigned long long*>(&parts[i].best[lane])));
        lists[warp][lane] = best;
    }
    __syncthreads();
    if (TOP)
#pragma unroll
        for (int n = WARPS / 2; n > 0; n /= 2) {
            if (warp < n) {
                best = merged(best, lists[warp + n][lane]);
                lists[warp][lane] = best;
            }
            __syncthreads();
        }
    if (warp != 0)
        return;
    m = -INFINITY, a = b = w = 0.0f;
    if (lane < WARPS)
        m = sums[lane][0], a = sums[lane][1], b = sums[lane][2], w = sums[lane][3];
    join_sums(m, a, b, w, c);
    leave<TYPE>(p, row, m, a, b, w, best, err);
}

// Pieces of a row: as many as fill the GPU, none below kLeastPiece.
int pieces_of(int64_t rows, int64_t vocab)
{
    const int64_t most = std::max<int64_t>(1, vocab / kLeastPiece);
    return (int)std::min(most, std::max<int64_t>(1, (kPieces + rows - 1) / std::max<int64_t>(rows, 1)));
}

}  // namespace

size_t logprobs_workspace(int64_t rows, int64_t vocab, int)
{
    const int pieces = pieces_of(rows, vocab);
    return pieces == 1 ? 0 : (size_t)rows * pieces * sizeof(Part);
}

int logprobs_launches(const TokenLogprobs& p)
{
    return pieces_of(p.rows, p.vocab) == 1 ? 1 : 2;
}

cudaError_t launch_token_logprobs(const TokenLogprobs& p, const DeviceInfo&, cudaStream_t s)
{
    unsigned int* err = nullptr;
    const cudaError_t e = device_error_ptr(&err);
    if (e != cudaSuccess)
        return e;
    const int pieces = pieces_of(p.rows, p.vocab);
    // whole vectors, so that rows that begin on one keep their pieces aligned
    const int64_t piece = ((p.vocab + pieces - 1) / pieces + 7) / 8 * 8;
    auto run = [&](auto type, auto top) {
        constexpr int TYPE = decltype(type)::value;
        constexpr bool TOP = decltype(top)::value;
        cudaError_t r = launch_pdl(piece_kernel<TYPE, TOP>, dim3((unsigned)(p.rows * pieces)), dim3(THREADS), 0, s, p, pieces,
                                   piece, err);
        if (r == cudaSuccess && pieces > 1)
            r = launch_pdl(join_kernel<TYPE, TOP>, dim3((unsigned)p.rows), dim3(THREADS), 0, s, p, pieces, err);
        return r;
    };
    auto by_top = [&](auto type) { return p.top > 0 ? run(type, std::true_type()) : run(type, std::false_type()); };
    return p.dtype == CK_OUT_F32   ? by_top(std::integral_constant<int, CK_OUT_F32>())
           : p.dtype == CK_OUT_F16 ? by_top(std::integral_constant<int, CK_OUT_F16>())
                                   : by_top(std::integral_constant<int, CK_OUT_BF16>());
}

}  // namespace ck
