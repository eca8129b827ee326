// adapter.cu -- low-rank adapters of many requests at once, beside a projection that they share.
//
//   h[m] = x[m] A_i^T,  y[m] = residual[m] + scaling[i] h[m] B_i^T,  i = index[m];  y[m] = residual[m] where i < 0
//
// Bound: HBM, the used adapters' A and B where the rows are few, x, residual and y where they are many.
//
// Two launches: h in parts of K (fp32, in the workspace), then h B^T onto the residual, the parts added
// in order.  The rows of a tile (up to 256) are put into groups of up to 16 of one adapter, whatever
// their order; a group is the 16 rows of the 16x8x16 matrix instruction.
//   few rows (up to 256): a block takes a group and a part of K; its 8 warps share the part out in steps
//     of 32 k, 16 bytes a lane straight from memory into the products' operands (the order of k within
//     a step is the same permutation on both sides), and add their sums up in shared memory.
//   many rows: a block takes 128 rows and a part of K on the fifth-generation tensor core, x and A by TMA
//     through a ring, h in tensor memory; once for every adapter that some of its rows have.
//   the second product: a warp takes a group and 32 columns at a time; columns are dealt to the
//     instruction's tiles so that a lane holds 8 neighbouring ones, and residual and y pass in 16 bytes.
//
// Rounding to fewer bits: h once, to the type of B, as the matrix instruction takes it; in fp16 relative
// to the power of two of the row's largest value, so that it neither overflows nor vanishes where the
// result does not.
#include <algorithm>
#include <cmath>
#include <string>
#include <type_traits>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_common.cuh"
#include "transformer.h"
#include "warp_mma.cuh"

namespace ck {
namespace {

constexpr int WARPS = 8;
constexpr int THREADS = WARPS * 32;
constexpr int kFewRows = 256;        // rows that one tile of groups holds
constexpr int TILE = 128;            // rows of a tile where there are more
constexpr uint32_t FULL = 0xffffffffu;
constexpr uint64_t TIMEOUT_NS = 2000000000ull;

// The rows of a tile by adapter, in groups of up to 16.
struct Groups {
    uint32_t key[kFewRows];            // adapter of each row; `adapters`: none, above: out of range
    int16_t row[kFewRows];             // rows in order of their adapters
    int16_t begin[kFewRows + 1];       // of each group, in `row`
    int count;
};

// By a whole block of THREADS: the groups of rows first .. first + rows - 1 (at most kFewRows).
__device__ __forceinline__ void make_groups(Groups& g, const int32_t* index, int64_t first, int rows, int64_t adapters)
{
    __shared__ int starts[WARPS];
    const int m = threadIdx.x, lane = m & 31, warp = m >> 5;
    uint32_t key = 0;
    if (m < rows) {
        const int32_t i = __ldg(index + first + m);
        key = i < 0 ? (uint32_t)adapters : (int64_t)i < adapters ? (uint32_t)i : (uint32_t)adapters + 1u;
        g.key[m] = key;
    }
    __syncthreads();
    const bool same = __syncthreads_and(m >= rows || key == g.key[0]);
    int at = m, of_mine = m;  // place in order, and among the rows of its own adapter
    if (!same && m < rows) {
        at = of_mine = 0;
        for (int n = 0; n < rows; ++n) {
            const uint32_t k = g.key[n];
            at += k < key || (k == key && n < m);
            of_mine += k == key && n < m;
        }
    }
    // which places begin a group
    __shared__ uint8_t begins[kFewRows];
    if (m < rows) {
        g.row[at] = (int16_t)m;
        begins[at] = of_mine % 16 == 0;
    }
    __syncthreads();
    const bool mine = m < rows && begins[m];
    const uint32_t some = __ballot_sync(FULL, mine);
    if (lane == 0)
        starts[warp] = __popc(some);
    __syncthreads();
    int before = 0, all = 0;
    for (int w = 0; w < WARPS; ++w) {
        before += w < warp ? starts[w] : 0;
        all += starts[w];
    }
    if (mine)
        g.begin[before + __popc(some & ((1u << lane) - 1u))] = (int16_t)m;
    if (m == 0) {
        g.count = all;
        g.begin[all] = (int16_t)rows;
    }
    __syncthreads();
}

// ---- few rows: h of one group over one part of K
template <class E, int RT>  // RT: tiles of 8 of the rank
__global__ void __launch_bounds__(THREADS) shrink_few_kernel(const AdapterLinear p, int splits, unsigned int* err)
{
    using T = typename E::T;
    __shared__ Groups groups;
    __shared__ float4 sums[4][16][RT * 2];
    griddep_wait();
    griddep_launch_dependents();
    const int number = blockIdx.x / splits, split = blockIdx.x - number * splits;
    make_groups(groups, p.index, 0, (int)p.M, p.adapters);
    if (number >= groups.count)
        return;
    const int begin = groups.begin[number], rows = groups.begin[number + 1] - begin;
    const uint32_t adapter = groups.key[groups.row[begin]];
    if (adapter >= p.adapters) {
        if (adapter > p.adapters && threadIdx.x == 0 && split == 0)
            atomicOr(err, kErrIndex);
        return;
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const T* x[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
        x[h] = g + 8 * h < rows ? static_cast<const T*>(p.x) + groups.row[begin + g + 8 * h] * p.K + 8 * t : nullptr;
    const T* a = static_cast<const T*>(p.a) + ((int64_t)adapter * p.rank + g) * p.K + 8 * t;
    const int64_t steps = (p.K + 31) / 32;
    const int64_t s0 = split * steps / splits, s1 = (split + 1) * steps / splits;
    float acc[RT][4] = {};
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll 2
    for (int64_t s = s0 + warp; s < s1; s += WARPS) {
        const int64_t k = 32 * s;
        const bool in = k + 8 * t < p.K;
        uint4 xv[2], av[RT];
#pragma unroll
        for (int h = 0; h < 2; ++h)
            xv[h] = x[h] && in ? __ldg(reinterpret_cast<const uint4*>(x[h] + k)) : zero;
#pragma unroll
        for (int j = 0; j < RT; ++j)
            av[j] = in && 8 * j < p.rank ? __ldg(reinterpret_cast<const uint4*>(a + (int64_t)8 * j * p.K + k)) : zero;
        const uint32_t lo[4] = {xv[0].x, xv[1].x, xv[0].y, xv[1].y}, hi[4] = {xv[0].z, xv[1].z, xv[0].w, xv[1].w};
#pragma unroll
        for (int j = 0; j < RT; ++j) {
            mma_16816<E>(acc[j], lo, av[j].x, av[j].y);
            mma_16816<E>(acc[j], hi, av[j].z, av[j].w);
        }
    }
    // the warps' sums: 4 to 7 onto 0 to 3, then these in order
    float* slab = reinterpret_cast<float*>(sums[warp & 3]);
    auto each = [&](auto fn) {
#pragma unroll
        for (int j = 0; j < RT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                fn(slab[(g + 8 * (i >> 1)) * RT * 8 + 8 * j + 2 * t + (i & 1)], acc[j][i]);
    };
    if (warp >= 4)
        each([](float& s, float v) { s = v; });
    __syncthreads();
    if (warp < 4)
        each([](float& s, float v) { s += v; });
    __syncthreads();
    float* out = static_cast<float*>(p.workspace) + (int64_t)split * p.M * p.rank;
    for (int i = threadIdx.x; i < rows * (p.rank / 4); i += THREADS) {
        const int r = i / (p.rank / 4), c = i - r * (p.rank / 4);
        float4 v = sums[0][r][c];
#pragma unroll
        for (int w = 1; w < 4; ++w) {
            const float4 u = sums[w][r][c];
            v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
        }
        *reinterpret_cast<float4*>(out + (int64_t)groups.row[begin + r] * p.rank + 4 * c) = v;
    }
}

// ---- many rows: one warp per (row, rank)
template <class E>
__global__ void __launch_bounds__(THREADS) shrink_many_kernel(const AdapterLinear p, unsigned int* err)
{
    using T = typename E::T;
    griddep_wait();
    griddep_launch_dependents();
    const int lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const int64_t m = unit / p.rank;
    const int r = (int)(unit - m * p.rank);
    if (m >= p.M)
        return;
    const int i = __ldg(p.index + m);
    if (i >= p.adapters) {
        if (lane == 0 && r == 0)
            atomicOr(err, kErrIndex);
    } else if (i >= 0) {
        const T* x = static_cast<const T*>(p.x) + m * p.K;
        const T* a = static_cast<const T*>(p.a) + ((int64_t)i * p.rank + r) * p.K;
        float sum = 0.0f;
        for (int64_t k = lane; k < p.K; k += 32)
            sum = fmaf(E::to(x[k]), E::to(a[k]), sum);
#pragma unroll
        for (int o = 16; o; o >>= 1)
            sum += __shfl_xor_sync(FULL, sum, o);
        if (lane == 0)
            static_cast<float*>(p.workspace)[m * p.rank + r] = sum;
    }
}

// ---- 8 neighbouring outputs of a lane
template <int OUT>
struct Eight;
template <>
struct Eight<CK_OUT_F32> {
    float4 v[2];
    static __device__ __forceinline__ Eight load(const void* base, int64_t i)
    {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
        return {{p[0], p[1]}};
    }
    __device__ __forceinline__ void store(void* base, int64_t i) const
    {
        float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + i);
        p[0] = v[0], p[1] = v[1];
    }
    __device__ __forceinline__ void add(const float (&d)[8])
    {
        v[0].x += d[0], v[0].y += d[1], v[0].z += d[2], v[0].w += d[3];
        v[1].x += d[4], v[1].y += d[5], v[1].z += d[6], v[1].w += d[7];
    }
};
template <class E>
struct Eight16 {
    uint4 v;
    static __device__ __forceinline__ uint4 read(const void* base, int64_t i)
    {
        return *reinterpret_cast<const uint4*>(static_cast<const typename E::T*>(base) + i);
    }
    __device__ __forceinline__ void store(void* base, int64_t i) const
    {
        *reinterpret_cast<uint4*>(static_cast<typename E::T*>(base) + i) = v;
    }
    __device__ __forceinline__ void add(const float (&d)[8])
    {
        uint32_t* w = &v.x;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const float2 f = E::to2(w[n]);
            w[n] = E::pack2(f.x + d[2 * n], f.y + d[2 * n + 1]);
        }
    }
};
template <>
struct Eight<CK_OUT_BF16> : Eight16<Bf16> {
    static __device__ __forceinline__ Eight load(const void* base, int64_t i) { return {{read(base, i)}}; }
};
template <>
struct Eight<CK_OUT_F16> : Eight16<Fp16> {
    static __device__ __forceinline__ Eight load(const void* base, int64_t i) { return {{read(base, i)}}; }
};

// Items are a tile's (group, 32 columns of the block's); a warp takes a run of them.
template <class E, int OUT, int KT>  // KT: steps of 32 of the rank
__global__ void __launch_bounds__(THREADS) expand_kernel(const AdapterLinear p, int tile, int chunk, int splits)
{
    using T = typename E::T;
    __shared__ Groups groups;
    const int64_t chunks = (p.N + chunk - 1) / chunk;
    const int64_t first = blockIdx.x / chunks * tile, n_first = blockIdx.x % chunks * chunk;
    const int rows = (int)min(p.M - first, (int64_t)tile);
    // (the first kernel lets this one begin when its blocks have seen the work before them complete)
    make_groups(groups, p.index, first, rows, p.adapters);
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
    const int steps = (int)((min(p.N - n_first, (int64_t)chunk) + 31) / 32);
    const int items = groups.count * steps;
    const int i0 = warp * items / WARPS, i1 = (warp + 1) * items / WARPS;
    const bool in_place = p.residual == p.y;
    int group = -1;
    uint32_t adapter = 0;
    int64_t row[2] = {-1, -1};
    uint32_t h[KT][2][4];
    float factor[2] = {0.0f, 0.0f};
    const T* b = nullptr;
    for (int i = i0; i < i1; ++i) {
        if (i / steps != group) {
            group = i / steps;
            const int begin = groups.begin[group], count = groups.begin[group + 1] - begin;
            adapter = groups.key[groups.row[begin]];
#pragma unroll
            for (int r = 0; r < 2; ++r)
                row[r] = g + 8 * r < count ? first + groups.row[begin + g + 8 * r] : -1;
            if (adapter < p.adapters) {
                const float scaling = p.scaling ? __ldg(p.scaling + adapter) : 1.0f;
                b = static_cast<const T*>(p.b) + (int64_t)adapter * p.N * p.rank + 8 * t;
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    float v[KT][8];
                    float top = 0.0f;
#pragma unroll
                    for (int k = 0; k < KT; ++k) {
#pragma unroll
                        for (int n = 0; n < 8; ++n)
                            v[k][n] = 0.0f;
                        if (row[r] >= 0 && 32 * k + 8 * t < p.rank) {
                            const float* src = static_cast<const float*>(p.workspace) + row[r] * p.rank + 32 * k + 8 * t;
                            for (int s = 0; s < splits; ++s) {
                                const float4* part = reinterpret_cast<const float4*>(src + (int64_t)s * p.M * p.rank);
                                const float4 lo = __ldcg(part), hi = __ldcg(part + 1);
                                v[k][0] += lo.x, v[k][1] += lo.y, v[k][2] += lo.z, v[k][3] += lo.w;
                                v[k][4] += hi.x, v[k][5] += hi.y, v[k][6] += hi.z, v[k][7] += hi.w;
                            }
                        }
#pragma unroll
                        for (int n = 0; n < 8; ++n)
                            top = fmaxf(top, fabsf(v[k][n]));
                    }
                    float down = 1.0f;
                    factor[r] = scaling;
                    if (std::is_same<E, Fp16>::value) {
                        top = fmaxf(top, __shfl_xor_sync(FULL, top, 1));
                        top = fmaxf(top, __shfl_xor_sync(FULL, top, 2));
                        // (both powers are floats for these e)
                        const int e = top > 0.0f && top < INFINITY ? max(ilogbf(top), -126) : 0;
                        down = ldexpf(1.0f, -e);
                        factor[r] = scaling * ldexpf(1.0f, e);
                    }
#pragma unroll
                    for (int k = 0; k < KT; ++k)
#pragma unroll
                        for (int s = 0; s < 2; ++s) {
                            h[k][s][r] = E::pack2(v[k][4 * s] * down, v[k][4 * s + 1] * down);
                            h[k][s][2 + r] = E::pack2(v[k][4 * s + 2] * down, v[k][4 * s + 3] * down);
                        }
                }
            }
        }
        const int64_t n0 = n_first + 32 * (i - group * steps), n = n0 + 8 * t;
        const bool here = n < p.N;
        if (adapter >= p.adapters) {  // none: the residual, or an index out of range: NaN
#pragma unroll
            for (int r = 0; r < 2; ++r)
                if (row[r] >= 0 && here && !(in_place && adapter == p.adapters)) {
                    Eight<OUT> y{};
                    if (p.residual)
                        y = Eight<OUT>::load(p.residual, row[r] * p.N + n);
                    if (adapter > p.adapters) {
                        const float nan[8] = {NAN, NAN, NAN, NAN, NAN, NAN, NAN, NAN};
                        y.add(nan);
                    }
                    y.store(p.y, row[r] * p.N + n);
                }
            continue;
        }
        Eight<OUT> y[2] = {};
        if (p.residual)
#pragma unroll
            for (int r = 0; r < 2; ++r)
                if (row[r] >= 0 && here)
                    y[r] = Eight<OUT>::load(p.residual, row[r] * p.N + n);
        float acc[4][4] = {};
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            uint4 bv[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t col = n0 + 8 * (g >> 1) + 2 * j + (g & 1);
                bv[j] = col < p.N && 32 * k + 8 * t < p.rank ? __ldg(reinterpret_cast<const uint4*>(b + col * p.rank + 32 * k))
                                                             : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                mma_16816<E>(acc[j], h[k][0], bv[j].x, bv[j].y);
                mma_16816<E>(acc[j], h[k][1], bv[j].z, bv[j].w);
            }
        }
#pragma unroll
        for (int r = 0; r < 2; ++r)
            if (row[r] >= 0 && here) {
                const float d[8] = {acc[0][2 * r] * factor[r], acc[0][2 * r + 1] * factor[r], acc[1][2 * r] * factor[r],
                                    acc[1][2 * r + 1] * factor[r], acc[2][2 * r] * factor[r], acc[2][2 * r + 1] * factor[r],
                                    acc[3][2 * r] * factor[r], acc[3][2 * r + 1] * factor[r]};
                y[r].add(d);
                y[r].store(p.y, row[r] * p.N + n);
            }
    }
    griddep_launch_dependents();
}

// Parts of K.
int splits_of(int64_t M, int64_t K)
{
    if (M > kFewRows)
        return 1;
    return (int)std::min<int64_t>(8, std::max<int64_t>(1, K / 512));
}

}  // namespace

size_t adapter_workspace(int64_t M, int64_t, int64_t K, int rank)
{
    return (size_t)splits_of(M, K) * M * rank * sizeof(float);
}

cudaError_t launch_adapter_linear(const AdapterLinear& p, const DeviceInfo& dev, cudaStream_t s)
{
    unsigned int* err = nullptr;
    const cudaError_t e = device_error_ptr(&err);
    if (e != cudaSuccess)
        return e;
    const bool few = p.M <= kFewRows;
    const int splits = splits_of(p.M, p.K);
    const int tile = few ? kFewRows : TILE;
    const int64_t tiles = (p.M + tile - 1) / tile;
    // columns of a block: about four blocks to an SM
    int64_t chunk = 32;
    while (chunk < 512 && tiles * ((p.N + 2 * chunk - 1) / (2 * chunk)) >= 4 * dev.sm_count)
        chunk *= 2;
    const unsigned expand = (unsigned)(tiles * ((p.N + chunk - 1) / chunk));
    auto shrink = [&](auto type) {
        using E = decltype(type);
        if (!few)
            return launch_pdl(shrink_many_kernel<E>, dim3((unsigned)((p.M * p.rank + 7) / 8)), dim3(THREADS), 0, s, p, err);
        auto by_rank = [&](auto rt) {
            return launch_pdl(shrink_few_kernel<E, decltype(rt)::value>, dim3((unsigned)(p.M * splits)), dim3(THREADS), 0, s, p,
                              splits, err);
        };
        if (p.rank <= 8)
            return by_rank(std::integral_constant<int, 1>());
        if (p.rank <= 16)
            return by_rank(std::integral_constant<int, 2>());
        if (p.rank <= 32)
            return by_rank(std::integral_constant<int, 4>());
        return p.rank <= 64 ? by_rank(std::integral_constant<int, 8>()) : by_rank(std::integral_constant<int, 16>());
    };
    auto grow = [&](auto type, auto out) {
        using E = decltype(type);
        constexpr int OUT = decltype(out)::value;
        auto by_rank = [&](auto kt) {
            return launch_pdl(expand_kernel<E, OUT, decltype(kt)::value>, dim3(expand), dim3(THREADS), 0, s, p, tile, (int)chunk,
                              splits);
        };
        if (p.rank <= 32)
            return by_rank(std::integral_constant<int, 1>());
        return p.rank <= 64 ? by_rank(std::integral_constant<int, 2>()) : by_rank(std::integral_constant<int, 4>());
    };
    auto run = [&](auto type) {
        const cudaError_t r = shrink(type);
        if (r != cudaSuccess)
            return r;
        if (p.out_dtype == CK_OUT_F32)
            return grow(type, std::integral_constant<int, CK_OUT_F32>());
        return p.out_dtype == CK_OUT_F16 ? grow(type, std::integral_constant<int, CK_OUT_F16>())
                                         : grow(type, std::integral_constant<int, CK_OUT_BF16>());
    };
    return p.f16 ? run(Fp16()) : run(Bf16());
}

}  // namespace ck
