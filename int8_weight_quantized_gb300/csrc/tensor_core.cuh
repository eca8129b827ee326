// tensor_core.cuh -- what the kernels of the operators around the linear layers that use the
// fifth-generation tensor core share beyond ck_device.cuh: copies, products, descriptors, tensor
// memory, and the way of a row from tensor memory to global memory.
#pragma once

#include <cstdint>
#include <mutex>
#include <string>
#include <type_traits>

#include <cuda.h>
#include <cudaTypedefs.h>

#include "attn_common.cuh"

namespace ck {

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int32_t c0, int32_t c1,
                                            int32_t c2)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
        : "memory");
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one()
{
    uint32_t yes;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(yes));
    return yes != 0;
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
}

__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t add)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(add)
        : "memory");
}

// 32 columns of the lane's row, and the largest of them (NaN left out).
__device__ __forceinline__ void tmem_ld_max_32x32b_x32(uint32_t taddr, uint32_t (&r)[32], float& top)
{
    asm volatile(
        "tcgen05.ld.red.sync.aligned.32x32b.x32.max.f32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, %32, [%33];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
          "=f"(top)
        : "r"(taddr));
}

__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void tmem_wait_st()
{
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

// Descriptor of a [keys][64 values] box with 128-byte swizzling as an operand whose N (the
// values) is contiguous: 8-key groups 1024 bytes apart (stride offset), 64-value boxes
// box_bytes apart (leading offset).
__device__ __forceinline__ uint64_t desc_nmajor_sw128(uint32_t smem_addr, uint32_t box_bytes)
{
    uint64_t d = 0;
    d |= (uint64_t)((smem_addr >> 4) & 0x3FFFu);
    d |= (uint64_t)(box_bytes >> 4) << 16;
    d |= (uint64_t)(1024u >> 4) << 32;
    d |= (uint64_t)1u << 46;
    d |= (uint64_t)2u << 61;
    return d;
}

// Instruction descriptor, fp32 accumulator: 16-bit types at bits 7 and 10 (1 = bf16), negated
// A at 13, B with N contiguous at 16, N / 8 at 17, M / 16 (of 128 rows) at 24.
template <class E>
__device__ __forceinline__ constexpr uint32_t idesc_of(int n, bool b_nmajor)
{
    return (1u << 4) | (std::is_same<E, Bf16>::value ? (1u << 7) | (1u << 10) : 0u) | (b_nmajor ? 1u << 16 : 0u) |
           ((uint32_t)(n >> 3) << 17) | (8u << 24);
}

// Bounded wait of teardown (raises no abort).
__device__ __forceinline__ void wait_out(uint64_t* bar, uint32_t parity, unsigned int* err, uint32_t code, uint64_t timeout_ns)
{
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t i = 1; !mbar_try_wait(bar, parity); ++i)
        if ((i & 255u) == 0 && globaltimer_ns() - t0 > timeout_ns) {
            atomicOr(err, code);
            return;
        }
}

// 32 values of each lane's row times f, to dst + lane * stride, for the first `rows` lanes.  Four
// lanes trade their 16-byte pieces, so that a store writes 64 bytes of each of 8 rows: with 16
// bytes of each of 32 the output of a tile took 2900 cycles.
template <class E>
__device__ __forceinline__ void store_rows(typename E::T* dst, int64_t stride, int lane, int rows, const float (&v)[32],
                                           float f)
{
    uint32_t r[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int n = 0; n < 4; ++n)
            r[i][n] = E::pack2(v[8 * i + 2 * n] * f, v[8 * i + 2 * n + 1] * f);
#pragma unroll
    for (int m = 1; m <= 2; m *= 2)
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (!(i & m))
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const bool up = lane & m;
                    const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? r[i][n] : r[i | m][n], m);
                    r[i][n] = up ? got : r[i][n];
                    r[i | m][n] = up ? r[i | m][n] : got;
                }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int row = (lane & ~3) + i;
        if (row < rows)
            *reinterpret_cast<uint4*>(dst + row * stride + (lane & 3) * 8) = make_uint4(r[i][0], r[i][1], r[i][2], r[i][3]);
    }
}

inline PFN_cuTensorMapEncodeTiled_v12000 encode_fn()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    });
    return fn;
}

// A tensor, the first dimension dense, copied as boxes with 128-byte swizzling.
inline bool make_box_map(CUtensorMap* map, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                         const cuuint32_t* box, CUtensorMapDataType type, std::string* why)
{
    auto fn = encode_fn();
    if (!fn) {
        *why = "cuTensorMapEncodeTiled is not available from the driver";
        return false;
    }
    const cuuint32_t estr[3] = {1, 1, 1};
    const CUresult r = fn(map, type, (cuuint32_t)rank,
                          const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                          CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS)
        *why = "cuTensorMapEncodeTiled failed (" + std::to_string((int)r) + ")";
    return r == CUDA_SUCCESS;
}

inline bool make_box_map(CUtensorMap* map, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                         const cuuint32_t* box, bool f16, std::string* why)
{
    return make_box_map(map, base, rank, dims, strides, box,
                        f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, why);
}

}  // namespace ck
