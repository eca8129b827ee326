// int4.cu -- the linear layer with 4-bit weights and group scales, for few rows, and its
// weight preparation.
//
//   y[m,n] = out( sum_g scale[n,g] * (sum_{k in g} x[m,k] * c[n,k]) + bias[n] + residual[m,n] )
//   c = code - 8 in [-8, 7], eight codes to a 32-bit word: the code of k = 8 j + 2 i in bits
//   4 i .. 4 i + 3 of word j, that of k = 8 j + 2 i + 1 in bits 16 + 4 i .. (a pair of
//   neighbouring k is then one shift and one mask away from two 16-bit halves).
#include <algorithm>
#include <type_traits>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "attn_common.cuh"
#include "transformer.h"
#include "warp_mma.cuh"

namespace ck {
namespace {

__device__ __forceinline__ int code_shift(int e)
{
    return 4 * (e >> 1) + 16 * (e & 1);
}

// Bound: HBM, N K / 2 bytes of codes and 2 N K / group of scales, read once.
//
// A block's 8 warps are 8 / KW row groups of 16 RT weight rows each, and KW warps share out a
// group's K in chunks of 128, each a contiguous run; a warp streams its run's codes and scales through its own ring of
// asynchronous copies, with no block-wide barrier until the warps' sums are added, in a fixed
// order, at the end.  x, which every block reads whole, comes from L2 straight into the
// registers that the products take, a chunk ahead: in the ring it would take twice the codes'
// room at 8 rows.  Products run on the 16x8x16 matrix instruction,
// weight rows as its 16 rows and up to 8 rows of x as its 8 columns: at one row seven columns
// are idle, which costs nothing while HBM sets the pace, and up to 8 rows cost the same.  The
// codes are exact in bf16 and fp16 (nibble in the mantissa of 128 or 1024, minus that and 8),
// the products exact in fp32; a group's sum is scaled once, in fp32.
//
// Measured (GB300): one row, 28672 x 5376, groups of 128: 20.8 to 22.9 us, 3.5 to 3.8 TB/s, 52 to
// 57% of a copy's bandwidth, the ALU (shift and mask of each nibble pair) busy in 57% of the
// cycles, an instruction issued in 64%; in fp16, which takes two shifts less for a word, 21.1: the
// ALU alone is not what bounds it.  One row, 4096 x 4096: 4.4 us (launch and latency); 16 rows,
// 16384 x 4096, groups of 64: 15.2 us, 2.4 TB/s, waiting on the ring and on x; 32 rows, groups of
// 128: 23.0 us, 64 rows 42, 512 rows 267, 8192 rows 4.0 ms (272 TFLOP/s: beyond 32 rows each tile of
// them reads and widens the whole weight again).
constexpr int WARPS = 8;
constexpr int CHUNK = 128;                 // k of a ring unit
constexpr int STAGES = 4;
constexpr int W_LD = 80;                   // bytes of a unit's weight row: 64, padded so that 8 rows spread over the banks

// Blocks per SM that the compiler shares the registers out for (0: as it likes, which makes four).
// 32 rows of x need more than the 128 that two blocks leave (spilled: 32.9 us at 16384 x 4096, 23.3
// without); 16 rows do not, and two blocks hide more of their waits (18.6 us with one, 15.1 with
// two); one row at 16384 x 4096 took 13.2 us bound to four and 11.9 to two, 10.8 unbound.
template <int MT>
constexpr int kMinBlocks = MT == 4 ? 1 : MT == 2 ? 2 : 0;
template <int MT>
constexpr int kResident = MT == 4 ? 1 : MT == 2 ? 2 : 4;

// (w & MASK) | bits in one instruction (with both as constants the compiler made two of it)
template <uint32_t MASK>
__device__ __forceinline__ uint32_t and_or(uint32_t w, uint32_t bits)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(r) : "r"(w), "n"(MASK), "r"(bits));
    return r;
}

template <class E>
__device__ __forceinline__ uint32_t codes_of(uint32_t word, int i)
{
    // the pair k = 2 i, 2 i + 1 of the word's eight: code - 8 in two 16-bit floats
    if (std::is_same<E, Bf16>::value) {
        const uint32_t u = and_or<0x000F000Fu>(word >> (4 * i), 0x43004300u);  // 128 + code
        const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&u), __float2bfloat162_rn(136.0f));
        return *reinterpret_cast<const uint32_t*>(&v);
    }
    const uint32_t w = i < 2 ? word : word >> 8;
    if ((i & 1) == 0) {
        const uint32_t u = and_or<0x000F000Fu>(w, 0x64006400u);  // 1024 + code
        const __half2 v = __hsub2(*reinterpret_cast<const __half2*>(&u), __float2half2_rn(1032.0f));
        return *reinterpret_cast<const uint32_t*>(&v);
    }
    const uint32_t u = and_or<0x00F000F0u>(w, 0x64006400u);  // 1024 + 16 code, exact like the rest
    const __half2 v = __hfma2(*reinterpret_cast<const __half2*>(&u), __float2half2_rn(0.0625f), __float2half2_rn(-72.0f));
    return *reinterpret_cast<const uint32_t*>(&v);
}

template <int RT>
constexpr int kUnit = 16 * RT * (W_LD + 8);  // codes, then 8 bytes of scales a row

// PER_CHUNK: scales of a row in a chunk (4, 2 or 1 for groups of 32, 64, and 128 or 256)
template <class E, int RT, int MT, int PER_CHUNK, int KW>
__global__ void __launch_bounds__(WARPS * 32, kMinBlocks<MT>) int4_kernel(const Int4Linear p)
{
    using T = typename E::T;
    extern __shared__ __align__(128) uint8_t smem[];
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    constexpr int RW = WARPS / KW;             // row groups
    const int kw = warp % KW, rw = warp / KW;  // this warp's share of K, its row group
    const int64_t n0 = ((int64_t)blockIdx.x * RW + rw) * (16 * RT);
    const int64_t m0 = (int64_t)blockIdx.y * (8 * MT);
    const int rows = (int)min((int64_t)(8 * MT), p.M - m0);      // rows of x
    const int chunks = (int)(p.K / CHUNK);
    const int c0 = (int)((int64_t)kw * chunks / KW), c1 = (int)((int64_t)(kw + 1) * chunks / KW);
    const uint32_t ring = smem_u32(smem) + (uint32_t)(warp * STAGES * kUnit<RT>);
    const int64_t groups = p.K / p.group;
    const int log_chunks = p.group == 256 ? 1 : 0;  // chunks a group spans, PER_CHUNK == 1

    // where this lane's copies come from: row and 16 bytes of the codes, row of the scales
    const uint8_t* w_src[2 * RT];
    bool w_in[2 * RT];
#pragma unroll
    for (int i = 0; i < 2 * RT; ++i) {  // 8 rows of 4 x 16 bytes an instruction
        const int64_t n = n0 + i * 8 + g;
        w_in[i] = n < p.N;
        w_src[i] = reinterpret_cast<const uint8_t*>(p.w4) + (w_in[i] ? n : 0) * (p.K / 2) + t * 16;
    }
    constexpr int SI = (16 * RT + 31) / 32;  // instructions that copy a scale row per lane
    const __nv_bfloat16* s_src[SI];
    bool s_in[SI];
    int s_odd[SI];  // whether the row's first scale lies in an upper half
#pragma unroll
    for (int i = 0; i < SI; ++i) {
        const int64_t n = n0 + i * 32 + lane;
        s_in[i] = i * 32 + lane < 16 * RT && n < p.N;
        const int64_t first = (s_in[i] ? n : 0) * groups;
        s_src[i] = static_cast<const __nv_bfloat16*>(p.w_scale) + first;
        s_odd[i] = (int)(first & 1);
    }
    auto issue = [&](int c, int stage) {
        if (c < c1) {
            const uint32_t w = ring + stage * kUnit<RT> + g * W_LD + t * 16;
            const uint32_t sc = ring + stage * kUnit<RT> + 16 * RT * W_LD + lane * 8;
#pragma unroll
            for (int i = 0; i < 2 * RT; ++i)
                cp_async16(w + i * 8 * W_LD, w_src[i] + c * 64, w_in[i]);
            // the row's scales of this chunk: 8 bytes, 4, or the aligned 4 that hold the one
#pragma unroll
            for (int i = 0; i < SI; ++i)
                if (i * 32 + lane < 16 * RT) {
                    if (PER_CHUNK == 4)
                        cp_async_small<8>(sc + i * 256, s_src[i] + 4 * c, s_in[i]);
                    else if (PER_CHUNK == 2)
                        cp_async_small<4>(sc + i * 256, s_src[i] + 2 * c, s_in[i]);
                    else
                        cp_async_small<4>(sc + i * 256, s_src[i] + ((s_odd[i] + (c >> log_chunks)) & ~1) - s_odd[i], s_in[i]);
                }
        }
        cp_async_commit();
    };
    // this lane's part of 32 k of x: row g of each tile, k = 8 t .. + 7 (rows past M: 0)
    uint4 b[4][MT];
    const T* xl = static_cast<const T*>(p.x) + (m0 + g) * p.K + t * 8;
    auto load_x = [&](int c, int j) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
            if (8 * mt + g < rows)
                b[j][mt] = __ldg(reinterpret_cast<const uint4*>(xl + 8 * mt * p.K + c * CHUNK + j * 32));
    };
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s)
        issue(c0 + s, s);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
            b[j][mt] = make_uint4(0u, 0u, 0u, 0u);
        if (c0 < c1)
            load_x(c0, j);
    }
    // PER_CHUNK == 1: whether the first scale of this lane's rows (8 apart) lies in an upper half
    const int row_odd = (int)(((n0 + g) * groups) & 1);

    float sum[RT][MT][4] = {};
    float acc[RT][MT][4] = {};
    int stage = 0;
    for (int c = c0; c < c1; ++c) {
        issue(c + STAGES - 1, stage == 0 ? STAGES - 1 : stage - 1);
        cp_async_wait<STAGES - 1>();
        __syncwarp();
        const uint32_t w = ring + stage * kUnit<RT> + g * W_LD + t * 4;
        const uint32_t sc = ring + stage * kUnit<RT> + 16 * RT * W_LD + g * 8;
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // 32 k: word 4 j + t of a row is this lane's
#pragma unroll
            for (int rt = 0; rt < RT; ++rt) {
                const uint32_t lo = lds32(w + 16 * rt * W_LD + j * 16);
                const uint32_t hi = lds32(w + (16 * rt + 8) * W_LD + j * 16);
                const uint32_t a0[4] = {codes_of<E>(lo, 0), codes_of<E>(hi, 0), codes_of<E>(lo, 1), codes_of<E>(hi, 1)};
                const uint32_t a1[4] = {codes_of<E>(lo, 2), codes_of<E>(hi, 2), codes_of<E>(lo, 3), codes_of<E>(hi, 3)};
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    mma_16816<E>(acc[rt][mt], a0, b[j][mt].x, b[j][mt].y);
                    mma_16816<E>(acc[rt][mt], a1, b[j][mt].z, b[j][mt].w);
                }
            }
            if (c + 1 < c1)
                load_x(c + 1, j);  // the registers are free: the next chunk's
            // the end of a group: scale its sums
            if ((j + 1) % (4 / PER_CHUNK) == 0) {
#pragma unroll
                for (int rt = 0; rt < RT; ++rt)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int e = PER_CHUNK == 4 ? j : PER_CHUNK == 2 ? j >> 1 : 0;
                        const uint32_t pair = lds32(sc + (16 * rt + 8 * h) * 8 + (e >> 1) * 4);
                        const bool upper = PER_CHUNK == 1 ? (row_odd + (c >> log_chunks)) & 1 : e & 1;
                        const float s = __uint_as_float(upper ? pair & 0xFFFF0000u : pair << 16);
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) {
                            sum[rt][mt][2 * h] = fmaf(acc[rt][mt][2 * h], s, sum[rt][mt][2 * h]);
                            sum[rt][mt][2 * h + 1] = fmaf(acc[rt][mt][2 * h + 1], s, sum[rt][mt][2 * h + 1]);
                            acc[rt][mt][2 * h] = acc[rt][mt][2 * h + 1] = 0.0f;
                        }
                    }
            }
        }
        __syncwarp();
        stage = stage + 1 == STAGES ? 0 : stage + 1;
    }
    cp_async_wait<0>();
    griddep_launch_dependents();

    // add the warps' sums: [warp][m][n] in the ring's memory
    __syncthreads();
    float* red = reinterpret_cast<float*>(smem);
    constexpr int LD = 16 * RT + 1;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int m = 8 * mt + 2 * t + (i & 1);
                if (m < rows)
                    red[(warp * rows + m) * LD + 16 * rt + 8 * (i >> 1) + g] = sum[rt][mt][i];
            }
    __syncthreads();
    constexpr int BLOCK_ROWS = 16 * RT * RW;
    for (int i = threadIdx.x; i < rows * BLOCK_ROWS; i += WARPS * 32) {
        const int m = i / BLOCK_ROWS, r = i % BLOCK_ROWS;
        const int64_t n = (int64_t)blockIdx.x * BLOCK_ROWS + r;
        if (n >= p.N)
            continue;
        const int first = r / (16 * RT) * KW;  // the row group's first warp
        float v = 0.0f;
#pragma unroll
        for (int k = 0; k < KW; ++k)
            v += red[((first + k) * rows + m) * LD + r % (16 * RT)];
        if (p.bias != nullptr)
            v += E::to(static_cast<const T*>(p.bias)[n]);
        const int64_t at = (m0 + m) * p.N + n;
        if (p.out_dtype == CK_OUT_F32)
            static_cast<float*>(p.y)[at] = v + (p.residual ? static_cast<const float*>(p.residual)[at] : 0.0f);
        else if (p.out_dtype == CK_OUT_F16)
            static_cast<__half*>(p.y)[at] = Fp16::from(v + (p.residual ? Fp16::to(static_cast<const __half*>(p.residual)[at]) : 0.0f));
        else
            static_cast<__nv_bfloat16*>(p.y)[at] =
                Bf16::from(v + (p.residual ? Bf16::to(static_cast<const __nv_bfloat16*>(p.residual)[at]) : 0.0f));
    }
}

// Weight preparation: one thread per word for the codes; the group's scale is found by the
// group / 8 threads that share it (group <= 256: within a warp).  A group that holds a NaN or an
// infinity, which codes cannot, gets the scale NaN (and codes of zero).
__global__ void __launch_bounds__(256) int4_weight_kernel(const float* W, int64_t words, int group, uint32_t* w4,
                                                          __nv_bfloat16* w_scale)
{
    griddep_wait();
    const int lanes = group / 8;  // a power of two up to 32
    const int64_t j = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const bool in = j < words;  // words is a multiple of lanes: a group is all in or all out
    float v[8];
    float top = 0.0f;
    if (in) {
        const float4 a = __ldg(reinterpret_cast<const float4*>(W + 8 * j));
        const float4 b = __ldg(reinterpret_cast<const float4*>(W + 8 * j + 4));
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            top = max_nan(top, fabsf(v[e]));
    }
    for (int o = lanes >> 1; o; o >>= 1)
        top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (!in)
        return;
    const __nv_bfloat16 s16 = __float2bfloat16_rn(top < INFINITY ? __fdiv_rn(top, 7.0f) : NAN);
    const float s = __bfloat162float(s16);
    uint32_t word = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int c = s > 0.0f ? (int)fminf(fmaxf(rintf(__fdiv_rn(v[e], s)), -7.0f), 7.0f) : 0;
        word |= (uint32_t)(c + 8) << code_shift(e);
    }
    w4[j] = word;
    if (threadIdx.x % lanes == 0)
        w_scale[j / lanes] = s16;
}

__global__ void __launch_bounds__(256) int4_pack_kernel(const int8_t* codes, int64_t words, uint32_t* w4)
{
    griddep_wait();
    const int64_t j = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (j >= words)
        return;
    const uint2 r = __ldg(reinterpret_cast<const uint2*>(codes + 8 * j));
    uint32_t word = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int c = (int)(int8_t)(((e < 4 ? r.x : r.y) >> (8 * (e & 3))) & 255u);
        word |= (uint32_t)(min(max(c, -8), 7) + 8) << code_shift(e);
    }
    w4[j] = word;
}

}  // namespace

namespace {

template <class E, int RT, int MT, int PER_CHUNK, int KW>
cudaError_t launch(const Int4Linear& p, cudaStream_t s)
{
    constexpr size_t smem = std::max((size_t)WARPS * STAGES * kUnit<RT>,         // the rings
                                     (size_t)WARPS * 8 * MT * (16 * RT + 1) * 4);  // then the warps' sums
    // a kernel attribute belongs to the context it was set in: set once per context
    static ContextCache<int> cache;
    int done = 0;
    cudaError_t e = cache.get(&done, [](int* d) {
        *d = 1;
        return cudaFuncSetAttribute(int4_kernel<E, RT, MT, PER_CHUNK, KW>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    (int)smem);
    });
    if (e != cudaSuccess)
        return e;
    constexpr int ROWS = 16 * RT * WARPS / KW;
    const dim3 grid((unsigned)((p.N + ROWS - 1) / ROWS), (unsigned)((p.M + 8 * MT - 1) / (8 * MT)));
    return launch_pdl(int4_kernel<E, RT, MT, PER_CHUNK, KW>, grid, dim3(WARPS * 32), smem, s, p);
}

template <class E, int RT, int MT, int KW>
cudaError_t by_group(const Int4Linear& p, cudaStream_t s)
{
    return p.group == 32   ? launch<E, RT, MT, 4, KW>(p, s)
           : p.group == 64 ? launch<E, RT, MT, 2, KW>(p, s)
                           : launch<E, RT, MT, 1, KW>(p, s);
}

// KW: long runs of K per warp spread its set-up over more work and let a block's row groups share
// their reads of x in L1; short ones give a narrow layer enough warps and fill the last round of
// blocks better.  Rounds of blocks times (chunks of a run + 3 for what a block costs besides), at
// its least: KW = 2, 4, 8 took, in us, for 32 rows at 16384 x 4096 23.3, 24.7, 28.3, at 28672 x 5376
// 53.6, 45.0, 55.0, at 4096 x 16384 80.8, 40.9, 22.1; for 16 rows at 16384 x 4096 18.5, 15.2, 17.9.
template <class E, int RT, int MT>
cudaError_t by_split(const Int4Linear& p, const DeviceInfo& dev, cudaStream_t s)
{
    const int64_t chunks = p.K / CHUNK, slots = (int64_t)dev.sm_count * kResident<MT>;
    auto cost = [&](int kw) {
        const int64_t rows = 16 * RT * WARPS / kw;
        const int64_t blocks = (p.N + rows - 1) / rows * ((p.M + 8 * MT - 1) / (8 * MT));
        return (blocks + slots - 1) / slots * (chunks + 3 * kw) * (8 / kw);
    };
    const int64_t c2 = cost(2), c4 = cost(4), c8 = cost(8);
    if (c2 <= c4 && c2 <= c8)
        return by_group<E, RT, MT, 2>(p, s);
    if (c4 <= c8)
        return by_group<E, RT, MT, 4>(p, s);
    return by_group<E, RT, MT, 8>(p, s);
}

template <class E>
cudaError_t by_rows(const Int4Linear& p, const DeviceInfo& dev, cudaStream_t s)
{
    if (p.M <= 8)
        return by_split<E, 1, 1>(p, dev, s);
    if (p.M <= 16)
        return by_split<E, 2, 2>(p, dev, s);
    return by_split<E, 2, 4>(p, dev, s);
}

}  // namespace

cudaError_t launch_int4_linear(const Int4Linear& p, const DeviceInfo& dev, cudaStream_t s)
{
    return p.f16 ? by_rows<Fp16>(p, dev, s) : by_rows<Bf16>(p, dev, s);
}

cudaError_t launch_int4_weight(const float* W, int64_t N, int64_t K, int group, uint32_t* w4, void* w_scale,
                               const DeviceInfo& dev, cudaStream_t s)
{
    (void)dev;
    const int64_t words = N * (K / 8);
    return launch_pdl(int4_weight_kernel, dim3((unsigned)((words + 255) / 256)), dim3(256), 0, s, W, words, group, w4,
                      static_cast<__nv_bfloat16*>(w_scale));
}

cudaError_t launch_int4_pack(const int8_t* codes, int64_t N, int64_t K, uint32_t* w4, const DeviceInfo& dev,
                             cudaStream_t s)
{
    (void)dev;
    const int64_t words = N * (K / 8);
    return launch_pdl(int4_pack_kernel, dim3((unsigned)((words + 255) / 256)), dim3(256), 0, s, codes, words, w4);
}

}  // namespace ck
