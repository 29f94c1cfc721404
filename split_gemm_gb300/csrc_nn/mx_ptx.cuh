// Inline-PTX wrappers for the 4-bit tensor-core path, written from the PTX ISA's
// instruction descriptions; the wrappers it has in common with the convolution
// kernels are in ptx.cuh.
#pragma once

#include "ptx.cuh"

namespace sgb {
namespace ptx {

// Instruction descriptor for kind::mxf4 (E2M1 operands, E8M0 scales, fp32 D):
// scale-factor id of B (bits 4-5) and of A (bits 29-30), the half of a 32-bit
// scale column (0 or 2) that the instruction's two blocks of 32 use; A and B format E2M1 (bits 7-9
// and 10-11 = 1), N >> 3 in bits 17-22, scale type E8M0 (bit 23 = 1), M >> 4 in bits 24-28.
__host__ __device__ constexpr uint32_t idesc_mxf4(int m, int n, int sf_id)
{
    return (static_cast<uint32_t>(sf_id) << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) | (1u << 23) |
           (static_cast<uint32_t>(m >> 4) << 24) | (static_cast<uint32_t>(sf_id) << 29);
}

// One stage of one CTA, up to 256 reduction elements, executed by a whole warp in uniform control flow: one elected
// lane copies the scales to tensor memory and issues the MMAs (128 x N x 64, N <= 128).  `mmas` is 1 .. 4; the scale
// tiles of 512 bytes lie at `sf_desc`, a's two in order of the reduction, then b's two, and go to the 16 columns
// from sfa in the same order; the second ones are read for more than two MMAs only.  b's rows begin at the 32 rows of
// column `sfb_from` of a tile.  In one block, so that the election and the operands' moves to uniform registers are paid once.
__device__ __forceinline__ void mma_mxf4_stage(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint64_t sf_desc, uint32_t sfa,
                                               uint32_t sfb_from, uint32_t idesc_lo, uint32_t idesc_hi, uint32_t accumulate,
                                               uint32_t mmas)
{
    asm volatile(
        "{\n\t.reg .pred p, e, t, m1, m2, m3;\n\t.reg .b64 a1, a2, a3, b1, b2, b3, s1, s2, s3;\n\t"
        ".reg .b32 f4, f8, f12, q8, q12;\n\t"
        "setp.ne.b32 p, %7, 0;\n\t"
        "setp.eq.b32 t, 0, 0;\n\t"
        "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\t"
        "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\t"
        "add.s64 s1, %3, 32;\n\tadd.s64 s2, %3, 64;\n\tadd.s64 s3, %3, 96;\n\t"
        "add.s32 f4, %4, 4;\n\tadd.s32 f8, %4, 8;\n\tadd.s32 f12, %4, 12;\n\t"
        "add.s32 q8, f8, %9;\n\tadd.s32 q12, f12, %9;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "setp.gt.and.u32 m1, %8, 1, e;\n\t"
        "setp.gt.and.u32 m2, %8, 2, e;\n\t"
        "setp.gt.and.u32 m3, %8, 3, e;\n\t"
        "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%4], %3;\n\t"
        "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [f8], s2;\n\t"
        "@m2 tcgen05.cp.cta_group::1.32x128b.warpx4 [f4], s1;\n\t"
        "@m2 tcgen05.cp.cta_group::1.32x128b.warpx4 [f12], s3;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %5, [%4], [q8], p;\n\t"
        "@m1 tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], a1, b1, %6, [%4], [q8], t;\n\t"
        "@m2 tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], a2, b2, %5, [f4], [q12], t;\n\t"
        "@m3 tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], a3, b3, %6, [f4], [q12], t;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "l"(sf_desc), "r"(sfa), "r"(idesc_lo), "r"(idesc_hi), "r"(accumulate), "r"(mmas), "r"(sfb_from)
        : "memory");
}

__device__ __forceinline__ void mma_commit_elect(uint64_t* bar)
{
    asm volatile(
        "{\n\t.reg .pred e;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_addr(bar))
        : "memory");
}

// Contiguous copy of a multiple of 16 bytes into this CTA's shared memory, counted on `bar`.
__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                     smem_addr(dst)),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_addr(bar))
                 : "memory");
}

// 32 lanes x 16 consecutive 32-bit columns.
__device__ __forceinline__ void tmem_ld_32x32b_x16(uint32_t taddr, uint32_t (&v)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr)
        : "memory");
}

// One stage of a CTA pair, 256 reduction elements, executed by a whole warp in uniform control flow: one elected
// lane copies the stage's scales to tensor memory (two tiles of a's rows to columns sfa.., four of b's to sfa+8..) and issues
// the four 256 x 256 x 64 MMAs.  A rows 0..127 and B rows 0..127 come from the leader's shared memory, the others from
// the peer's at the same addresses; each CTA's tensor memory takes its own shared memory's scales: of its
// 128 rows of a and of all 256 of b.  `sf_desc` describes the first of the scale tiles, 512 bytes each: a's two
// in order of the reduction, then two of b's first 128 rows, then two of the others.  In one block, so that the election and
// the operands' moves to uniform registers are paid once.
__device__ __forceinline__ void mma_mxf4_pair_stage(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint64_t sf_desc, uint32_t sfa,
                                                    uint32_t idesc_lo, uint32_t idesc_hi, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, e, t;\n\t.reg .b64 a1, a2, a3, b1, b2, b3, s1, s2, s3, s4, s5;\n\t"
        ".reg .b32 f4, f8, f12, f16, f20;\n\t"
        "setp.ne.b32 p, %7, 0;\n\t"
        "setp.eq.b32 t, 0, 0;\n\t"
        "add.s64 a1, %1, 2;\n\tadd.s64 a2, %1, 4;\n\tadd.s64 a3, %1, 6;\n\t"
        "add.s64 b1, %2, 2;\n\tadd.s64 b2, %2, 4;\n\tadd.s64 b3, %2, 6;\n\t"
        "add.s64 s1, %3, 32;\n\tadd.s64 s2, %3, 64;\n\tadd.s64 s3, %3, 96;\n\tadd.s64 s4, %3, 128;\n\tadd.s64 s5, %3, 160;\n\t"
        "add.s32 f4, %4, 4;\n\tadd.s32 f8, %4, 8;\n\tadd.s32 f12, %4, 12;\n\tadd.s32 f16, %4, 16;\n\tadd.s32 f20, %4, 20;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [%4], %3;\n\t"
        "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [f8], s2;\n\t"
        "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [f12], s4;\n\t"
        "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [f4], s1;\n\t"
        "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [f16], s3;\n\t"
        "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [f20], s5;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %5, [%4], [f8], p;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], a1, b1, %6, [%4], [f8], t;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], a2, b2, %5, [f4], [f16], t;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], a3, b3, %6, [f4], [f16], t;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "l"(sf_desc), "r"(sfa), "r"(idesc_lo), "r"(idesc_hi), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tma_load_2d_pair(void* dst, const void* map, uint32_t bar_cl, int32_t c0, int32_t c1)
{
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cl), "r"(c0), "r"(c1)
        : "memory");
}

// max(v, 0) of fp32 bits; NaN stays.
__device__ __forceinline__ uint32_t relu_nan(uint32_t v)
{
    float d;
    asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(d) : "f"(__uint_as_float(v)));
    return __float_as_uint(d);
}

__device__ __forceinline__ float4 ld_cluster_v4(uint32_t cluster_addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(cluster_addr)
                 : "memory");
    return v;
}

}  // namespace ptx
}  // namespace sgb
