// Inline-PTX wrappers of the adapter kernels, written from the PTX ISA's instruction descriptions; the others are in ptx.cuh and mx_ptx.cuh.
#pragma once

#include "mx_ptx.cuh"

namespace sgb {
namespace ptx {

// 16 lanes x 32 consecutive 32-bit columns of tensor memory: of column group j of 8, thread t gets columns 8j + 2(t%4) and the next, of
// lane t/4 in v[4j], v[4j+1] and of lane t/4 + 8 in v[4j+2], v[4j+3].
__device__ __forceinline__ void tmem_ld_16x256b_x4(uint32_t taddr, uint32_t (&v)[16])
{
    asm volatile(
        "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
          "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
        : "r"(taddr)
        : "memory");
}

// The same descriptor as plain_kmajor_desc for an MN-major operand without swizzle: core matrices of 8 reduction indices x 16 bytes of M (or N),
// the 8 indices 16 B apart; `sbo` is the distance of core matrices adjacent along M/N and `lbo` along the reduction.
__device__ __forceinline__ uint64_t plain_mnmajor_desc(uint32_t saddr, uint32_t lbo, uint32_t sbo) { return plain_kmajor_desc(saddr, lbo, sbo); }

// Four MMAs in turn into the same accumulator from one elected lane of a warp in uniform control flow, the descriptors `a_step` and
// `b_step` (16-byte units) apart; the first accumulates when `accumulate` is nonzero, the others always.  In one block, so that the election and the
// operands' moves to uniform registers are paid once: alone, an MMA costs its warp some 100 clocks, three times what a 128 x 64 x 16 takes.
__device__ __forceinline__ void mma_bf16_elect_x4(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint64_t a_step, uint64_t b_step, uint32_t idesc,
                                                  uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, e, t;\n\t.reg .b64 a1, a2, a3, b1, b2, b3;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "setp.eq.b32 t, 0, 0;\n\t"
        "add.s64 a1, %1, %3;\n\tadd.s64 a2, a1, %3;\n\tadd.s64 a3, a2, %3;\n\t"
        "add.s64 b1, %2, %4;\n\tadd.s64 b2, b1, %4;\n\tadd.s64 b3, b2, %4;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %5, p;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %5, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a2, b2, %5, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a3, b3, %5, t;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "l"(a_step), "l"(b_step), "r"(idesc), "r"(accumulate)
        : "memory");
}

// The same for two MMAs.
__device__ __forceinline__ void mma_bf16_elect_x2(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint64_t a_step, uint64_t b_step, uint32_t idesc,
                                                  uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, e, t;\n\t.reg .b64 a1, b1;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "setp.eq.b32 t, 0, 0;\n\t"
        "add.s64 a1, %1, %3;\n\tadd.s64 b1, %2, %4;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %5, p;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a1, b1, %5, t;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "l"(a_step), "l"(b_step), "r"(idesc), "r"(accumulate)
        : "memory");
}

// The same for A in tensor memory, in three parts: three MMAs with one B, A's columns `a_part` apart, and three with the next, 8 columns (16 of
// the reduction) and `b_step` on.
__device__ __forceinline__ void mma_bf16_parts_x2(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t a_part, uint64_t b_step, uint32_t idesc,
                                                  uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, e, t;\n\t.reg .b32 a1, a2, a3, a4, a5;\n\t.reg .b64 b1;\n\t"
        "setp.ne.b32 p, %6, 0;\n\t"
        "setp.eq.b32 t, 0, 0;\n\t"
        "add.s32 a1, %1, %3;\n\tadd.s32 a2, a1, %3;\n\tadd.s32 a3, %1, 8;\n\tadd.s32 a4, a1, 8;\n\tadd.s32 a5, a2, 8;\n\t"
        "add.s64 b1, %2, %4;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %5, p;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], %2, %5, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], %2, %5, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a3], b1, %5, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a4], b1, %5, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a5], b1, %5, t;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(a_part), "l"(b_step), "r"(idesc), "r"(accumulate)
        : "memory");
}

// The first three alone.
__device__ __forceinline__ void mma_bf16_parts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t a_part, uint32_t idesc, uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p, e, t;\n\t.reg .b32 a1, a2;\n\t"
        "setp.ne.b32 p, %5, 0;\n\t"
        "setp.eq.b32 t, 0, 0;\n\t"
        "add.s32 a1, %1, %3;\n\tadd.s32 a2, a1, %3;\n\t"
        "elect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %4, p;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a1], %2, %4, t;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [a2], %2, %4, t;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(a_part), "r"(idesc), "r"(accumulate)
        : "memory");
}

// 8 columns of the warp's 32 lanes from each thread's registers, and the wait for such stores.
__device__ __forceinline__ void tmem_st_32x32b_x8(uint32_t taddr, const uint32_t (&v)[8])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
                 "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Copies, loads and stores that a lane may skip, predicated: a branch costs a warp some 20 clocks.
__device__ __forceinline__ void cp_async_16_if(uint32_t dst, const void* src, bool p)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\t@p cp.async.cg.shared.global [%0], [%1], 16;\n\t}" ::"r"(dst), "l"(src), "r"(static_cast<uint32_t>(p))
                 : "memory");
}
__device__ __forceinline__ void cp_async_4_if(uint32_t dst, const void* src, bool p)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\t@p cp.async.ca.shared.global [%0], [%1], 4;\n\t}" ::"r"(dst), "l"(src), "r"(static_cast<uint32_t>(p))
                 : "memory");
}
__device__ __forceinline__ void cp_async_8_if(uint32_t dst, const void* src, bool p)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\t@p cp.async.ca.shared.global [%0], [%1], 8;\n\t}" ::"r"(dst), "l"(src), "r"(static_cast<uint32_t>(p))
                 : "memory");
}
__device__ __forceinline__ void cp_async_16_fill_if(uint32_t dst, const void* src, uint32_t src_bytes, bool p)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %3, 0;\n\t@p cp.async.cg.shared.global [%0], [%1], 16, %2;\n\t}" ::"r"(dst), "l"(src), "r"(src_bytes),
                 "r"(static_cast<uint32_t>(p))
                 : "memory");
}
__device__ __forceinline__ uint4 ld_v4_if(const void* src, bool p)
{
    uint4 v;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
        "@p ld.global.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
        : "l"(src), "r"(static_cast<uint32_t>(p))
        : "memory");
    return v;
}
__device__ __forceinline__ uint32_t ld_u8_if(const void* src, bool p)
{
    uint32_t v;
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %2, 0;\n\tmov.b32 %0, 0;\n\t@p ld.global.u8 %0, [%1];\n\t}" : "=&r"(v) : "l"(src), "r"(static_cast<uint32_t>(p))
                 : "memory");
    return v;
}
// Streaming: what is read or written once.
__device__ __forceinline__ uint4 ld_stream_v4_if(const void* src, bool p)
{
    uint4 v;
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\tmov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
        "@p ld.global.cs.v4.b32 {%0, %1, %2, %3}, [%4];\n\t}"
        : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w)
        : "l"(src), "r"(static_cast<uint32_t>(p))
        : "memory");
    return v;
}
__device__ __forceinline__ void st_stream_v4_if(void* dst, uint4 v, bool p)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t@p st.global.cs.v4.b32 [%0], {%1, %2, %3, %4};\n\t}" ::"l"(dst), "r"(v.x), "r"(v.y), "r"(v.z),
                 "r"(v.w), "r"(static_cast<uint32_t>(p))
                 : "memory");
}
__device__ __forceinline__ void st_stream_v2_if(void* dst, uint2 v, bool p)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %3, 0;\n\t@p st.global.cs.v2.b32 [%0], {%1, %2};\n\t}" ::"l"(dst), "r"(v.x), "r"(v.y),
                 "r"(static_cast<uint32_t>(p))
                 : "memory");
}
__device__ __forceinline__ uint2 ld_shared_v2(uint32_t addr)
{
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void mbar_arrive_if(uint64_t* bar, bool p)
{
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %1, 0;\n\t@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(smem_addr(bar)), "r"(static_cast<uint32_t>(p))
                 : "memory");
}

// The line that holds an address, to L2.
__device__ __forceinline__ void prefetch_l2(const void* src) { asm volatile("prefetch.global.L2 [%0];" ::"l"(src)); }

// A multiple of 16 bytes of this CTA's shared memory to another's of the cluster, counted on a barrier there.
__device__ __forceinline__ void bulk_to_cluster(uint32_t dst_cluster, uint32_t src, uint32_t bytes, uint32_t bar_cluster)
{
    asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst_cluster), "r"(src), "r"(bytes),
                 "r"(bar_cluster)
                 : "memory");
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t cluster_addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr) : "memory");
    return v;
}

// The cluster's barrier in two halves, the first without order of memory.
__device__ __forceinline__ void cluster_arrive_relaxed() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

}  // namespace ptx

namespace ad {

// A 32-bit value as three bf16 parts that add up to it exactly: its first 8 significant bits, the next 8 and the rest (each cut off, so
// that no part is larger than the value); what is not finite stays in the first alone.
__device__ __forceinline__ void split3(float v, uint32_t& hi, uint32_t& mid, uint32_t& lo)
{
    const uint32_t b = __float_as_uint(v);
    const bool finite = (b & 0x7f800000u) != 0x7f800000u;
    const float r = v - __uint_as_float(b & 0xffff0000u);
    const uint32_t rb = __float_as_uint(r);
    const float q = r - __uint_as_float(rb & 0xffff0000u);
    hi = finite ? b >> 16 : (b >> 16) | ((b & 0x7fffffu) ? 0x40u : 0u);  // a NaN stays one
    mid = finite ? rb >> 16 : 0u;
    lo = finite ? __float_as_uint(q) >> 16 : 0u;
}

}  // namespace ad
}  // namespace sgb
