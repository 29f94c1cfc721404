// The adapters' forward pass for few rows (a decoding step): pieces of up to 8 rows of one adapter, a cluster of S CTAs to each.
//
// What such a call takes is latency and the reading of a[e] and b[e]: 8 rows use each weight 8 times, two flops a byte.  So everything a thread reads is asked
// for at once: its columns of a and x for the first product, and its rows of b and of y for the second before the sums of the first are joined.  A warp takes
// 32 columns of x and of a's ranks at a time straight to registers (m16n8k16 products, a's 16 ranks the rows, x's 8 rows the columns; a lane's 16 bytes of each
// operand are neighbouring columns, the same in both, so their order within the product does not matter).  Its sums meet those of the CTA's 16 warps in
// shared memory and the cluster's in distributed shared memory, in a fixed order.  For the second product the rows of h (three bf16 parts of
// fp32, adapter_ptx.cuh) are the operand's 16 rows, half of them empty, and 32 columns of out its columns, in an order that leaves 8 neighbouring ones to a lane.
// The products go by registers (mma.sync): at 8 rows they are no part of the time, and tcgen05's would first have to lie in shared memory and come back from tensor memory.
//
// One row of 4096 x 4096, rank 16, in a graph: 4.0 to 4.2 us, of which the launch and two cluster barriers are most; 64 rows, 32 adapters: 5.3 us, 10 MB at 1.9 TB/s.
#include "conv2d.h"

#include "adapter_params.cuh"
#include "adapter_ptx.cuh"
#include "mxint8.cuh"

namespace sgb {
namespace ad {

constexpr int S_WARPS = 16, S_THREADS = 32 * S_WARPS;

__device__ __forceinline__ void mma_16n8k16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// 8 bf16 of a row, `valid` of them.
template <bool VEC>
__device__ __forceinline__ uint4 load8(const __nv_bfloat16* src, int valid)
{
    if constexpr (VEC) {
        return ptx::ld_v4_if(src, valid > 0);
    } else {
        uint32_t v[4] = {0u, 0u, 0u, 0u};
        if (valid > 0) mx::load_any<4, 2>(v, src, valid < 8 ? 2 * valid : 16);
        return make_uint4(v[0], v[1], v[2], v[3]);
    }
}

// 4 bf16 of a row of b.
template <bool VEC>
__device__ __forceinline__ uint2 load4(const __nv_bfloat16* src, int valid)
{
    if constexpr (VEC) {
        return valid > 0 ? __ldg(reinterpret_cast<const uint2*>(src)) : make_uint2(0u, 0u);
    } else {
        uint32_t v[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < valid) v[i] = __bfloat16_as_ushort(__ldg(src + i));
        return make_uint2(v[0] | v[1] << 16, v[2] | v[3] << 16);
    }
}

// RT: the rank in sixteens, at most.
template <int RT, bool VEC, typename TB, typename TO>
__global__ void __launch_bounds__(S_THREADS) pass_small(const __grid_constant__ PassParams p)
{
    constexpr int R = 16 * RT, PITCH = R + 4;
    __shared__ float partial[S_WARPS][8][PITCH];  // by warp, token, rank; the CTA's sums in the first
    __shared__ __align__(16) float h_all[8][PITCH];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
    const int rank_in = blockIdx.x % p.splits, warps = S_WARPS * p.splits, me = rank_in * S_WARPS + warp;
    ptx::grid_dependency_wait();
    const Piece piece = p.plan.small[blockIdx.x / p.splits];  // the same for the whole cluster
    if (piece.rows <= 0) return;
    const bool has = piece.adapter < p.adapters, mine = g < piece.rows;
    const int64_t e = has ? piece.adapter : 0, t = mine ? p.plan.order[piece.first + g] : 0;
    const __nv_bfloat16 *w1 = p.w1 + e * p.rank * p.from, *w2 = p.w2 + e * p.rank * p.to;
    const int units = (p.to + 31) / 32;
    const float scale = has && p.scale ? __ldg(p.scale + e) : 1.f;

    // The second product's operands of a unit of 32 columns: w2's rows 8(g/2) + 2j + (g&1), and base's 8 columns of token g.
    uint2 b[4][RT];
    const auto load_b = [&](int unit) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int c = 32 * unit + 8 * (g >> 1) + 2 * j + (g & 1);
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const int at = 16 * r + 4 * q;
                b[j][r] = load4<VEC>(w2 + static_cast<int64_t>(c) * p.rank + at, has && c < p.to ? p.rank - at : 0);
            }
        }
    };
    float base[8];
    const auto load_base = [&](int unit) {
        const int c = 32 * unit + 8 * q;
        const TB* src = static_cast<const TB*>(p.base) + t * p.base_stride + c;
        const int left = mine && p.base ? p.to - c : 0;
        if constexpr (VEC && sizeof(TB) == 2) {
            const uint4 v = ptx::ld_stream_v4_if(src, left > 0);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 8; ++i) base[i] = __uint_as_float(i % 2 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
        } else if constexpr (VEC) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint4 v = ptx::ld_stream_v4_if(src + 4 * i, left > 0);
                base[4 * i] = __uint_as_float(v.x), base[4 * i + 1] = __uint_as_float(v.y), base[4 * i + 2] = __uint_as_float(v.z), base[4 * i + 3] = __uint_as_float(v.w);
            }
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) base[i] = i < left ? mx::to_float(src[i]) : 0.f;
        }
    };

    if (has) {
        float acc[RT][4] = {};
        const __nv_bfloat16* x = p.in + t * p.in_stride;
        for (int c = 32 * me; c < p.from; c += 32 * warps) {
            const int k = c + 8 * q;
            const uint4 xv = load8<VEC>(x + k, mine ? p.from - k : 0);
            uint4 lo[RT], hi[RT];
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const int r0 = 16 * r + g;
                lo[r] = load8<VEC>(w1 + static_cast<int64_t>(r0) * p.from + k, r0 < p.rank ? p.from - k : 0);
                hi[r] = load8<VEC>(w1 + static_cast<int64_t>(r0 + 8) * p.from + k, r0 + 8 < p.rank ? p.from - k : 0);
            }
#pragma unroll
            for (int r = 0; r < RT; ++r) {
                const uint32_t first[4] = {lo[r].x, hi[r].x, lo[r].y, hi[r].y}, second[4] = {lo[r].z, hi[r].z, lo[r].w, hi[r].w};
                mma_16n8k16(acc[r], first, xv.x, xv.y);
                mma_16n8k16(acc[r], second, xv.z, xv.w);
            }
        }
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
            for (int i = 0; i < 4; ++i) partial[warp][2 * q + (i & 1)][16 * r + g + 8 * (i >> 1)] = acc[r][i];
    }
    if (me < units && p.out) {  // on their way while the sums are joined
        load_b(me);
        load_base(me);
    }
    __syncthreads();
    if (has) {
        for (int i = tid; i < 8 * R; i += S_THREADS) {
            float v[S_WARPS];
#pragma unroll
            for (int k = 0; k < S_WARPS; ++k) v[k] = partial[k][i / R][i % R];
#pragma unroll
            for (int k = 1; k < S_WARPS; ++k) v[0] += v[k];
            partial[0][i / R][i % R] = v[0];  // this thread's alone
        }
    }
    if (p.splits > 1)
        ptx::cluster_sync();
    else
        __syncthreads();
    for (int i = tid; i < 8 * R; i += S_THREADS) {
        const int row = i / R, r = i % R;
        float s = 0.f;
        if (has && r < p.rank) {
            for (int k = 0; k < p.splits; ++k) s += ptx::ld_cluster_f32(ptx::mapa_shared(ptx::smem_addr(&partial[0][row][r]), k));
            s *= scale;
        }
        h_all[row][r] = s;
        if (p.mid && rank_in == 0 && row < piece.rows && r < p.rank) p.mid[static_cast<int64_t>(p.plan.order[piece.first + row]) * p.rank + r] = s;
    }
    __syncthreads();
    if (p.splits > 1) ptx::cluster_arrive_relaxed();  // this CTA has read the others' sums
    if (p.out)
        for (int unit = me; unit < units; unit += warps) {
            if (unit != me) {
                load_b(unit);
                load_base(unit);
            }
            float d[4][4] = {};
            if (has)
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const float4 v = *reinterpret_cast<const float4*>(&h_all[g][16 * r + 4 * q]);
                    uint32_t s[4][3];
                    split3(v.x, s[0][0], s[0][1], s[0][2]);
                    split3(v.y, s[1][0], s[1][1], s[1][2]);
                    split3(v.z, s[2][0], s[2][1], s[2][2]);
                    split3(v.w, s[3][0], s[3][1], s[3][2]);
#pragma unroll
                    for (int part = 2; part >= 0; --part) {
                        const uint32_t a[4] = {s[0][part] | s[1][part] << 16, 0u, s[2][part] | s[3][part] << 16, 0u};
#pragma unroll
                        for (int j = 0; j < 4; ++j) mma_16n8k16(d[j], a, b[j][r].x, b[j][r].y);
                    }
                }
            float o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                o[i] = base[i] + d[i / 2][i % 2];
                if (p.relu && o[i] < 0.f) o[i] = 0.f;
            }
            const int c = 32 * unit + 8 * q;
            TO* dst = static_cast<TO*>(p.out) + t * p.out_stride + c;
            const int left = mine ? p.to - c : 0;
            if constexpr (!VEC) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (i < left) mx::from_float(dst[i], o[i]);
            } else if constexpr (sizeof(TO) == 4) {
                ptx::st_stream_v4_if(dst, make_uint4(__float_as_uint(o[0]), __float_as_uint(o[1]), __float_as_uint(o[2]), __float_as_uint(o[3])), left > 0);
                ptx::st_stream_v4_if(dst + 4, make_uint4(__float_as_uint(o[4]), __float_as_uint(o[5]), __float_as_uint(o[6]), __float_as_uint(o[7])), left > 0);
            } else {
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const __nv_bfloat162 v = __floats2bfloat162_rn(o[2 * i], o[2 * i + 1]);
                    w[i] = *reinterpret_cast<const uint32_t*>(&v);
                }
                ptx::st_stream_v4_if(dst, make_uint4(w[0], w[1], w[2], w[3]), left > 0);
            }
        }
    __syncwarp();
    if (p.splits > 1) ptx::cluster_wait();  // the others have read this CTA's sums
}

template <int RT, bool VEC, typename TB, typename TO>
int start_small(const PassParams& p, cudaStream_t stream)
{
    const int64_t grid = static_cast<int64_t>(p.plan.n_small) * p.splits;
    return mx::launch(pass_small<RT, VEC, TB, TO>, grid, S_THREADS, 0, stream, p.splits, p) == cudaSuccess ? CONV2D_OK : CONV2D_ERR_CUDA;
}

template <bool VEC, typename TB, typename TO>
int small_by_rank(const PassParams& p, cudaStream_t stream)
{
    if (p.rank <= 16) return start_small<1, VEC, TB, TO>(p, stream);
    if (p.rank <= 32) return start_small<2, VEC, TB, TO>(p, stream);
    return start_small<4, VEC, TB, TO>(p, stream);
}

template <bool VEC>
int small_by_types(const PassParams& p, int32_t base, int32_t out, cudaStream_t stream)
{
    using B = __nv_bfloat16;
    if (base == CONV2D_OUT_BF16) return out == CONV2D_OUT_BF16 ? small_by_rank<VEC, B, B>(p, stream) : small_by_rank<VEC, B, float>(p, stream);
    return out == CONV2D_OUT_BF16 ? small_by_rank<VEC, float, B>(p, stream) : small_by_rank<VEC, float, float>(p, stream);
}

int launch_small_fwd(PassParams& p, int32_t base_dtype, int32_t out_dtype, bool vec, cudaStream_t stream)
{
    // as many CTAs as leave each warp 32 columns of the longer side
    const int longest = p.from > p.to ? p.from : p.to;
    p.splits = 1;
    while (p.splits < 8 && longest > 32 * S_WARPS * p.splits) p.splits *= 2;
    return vec ? small_by_types<true>(p, base_dtype, out_dtype, stream) : small_by_types<false>(p, base_dtype, out_dtype, stream);
}

}  // namespace ad
}  // namespace sgb
