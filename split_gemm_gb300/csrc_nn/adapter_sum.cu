// The adapters' weight gradients: sums over an adapter's rows, out[e] (r, c) = sum of mid[t][r] * in[t][c], for da (mid = dh, in = x) and
// db (mid = h, in = dy) in one launch.
//
// HBM binds: `in` is read once, and with rank r there are 2r flops to its 1 or 2 bytes.  A CTA takes 256 columns of `in` (128 above
// rank 80, by tensor memory) and a piece of up to 32 of the plan's tiles, whatever adapters those belong to; an adapter's sum that lies in one piece goes straight
// to the result, else each piece's part goes to the workspace and a second launch adds the parts in order.
//
// The reduction runs over rows, so both operands are MN-major: in^T fills the accumulator's 128 lanes with columns, mid its columns
// with r, three times: the three bf16 parts of an fp32 mid (adapter_ptx.cuh) stand side by side, N = 3 * rank, and are added up as the accumulator is read.  Core
// matrices are 8 rows x 16 bytes, each column of them 16 bytes longer than it needs to be, so that 16-byte columns of one row, as they come
// from memory, fall into different banks.
//
// bf16 rows come by cp.async into the operand's place, ring stages ahead; checkpoints, rows that are not whole vectors, and mid come through
// registers, one or two stages ahead.  A checkpoint's integer becomes a bf16 number by bits: (m | 128) - 128 or 256, each with the scale in its exponent.
//
// Every wait is bounded, as in the pass (adapter_pass.cuh).
#include "adapter.h"

#include "adapter_params.cuh"
#include "adapter_ptx.cuh"
#include "mxint8.cuh"

namespace sgb {
namespace ad {

constexpr int U_WARPS = 16, U_LOADERS = 32 * U_WARPS, U_THREADS = U_LOADERS + 32;
constexpr uint64_t U_WAIT_NS = 1000000000ull;

// Shared memory of a stage of `tokens` rows: core matrices of a 16-byte column are `column` bytes, in's columns first, then mid's parts.
struct SumSmem {
    int rp, tokens, blocks;  // blocks of 128 columns
    __host__ __device__ constexpr SumSmem(int rank) : rp((rank + 15) / 16 * 16), tokens(rp <= 64 ? 64 : 32), blocks(rp <= 80 ? 2 : 1) {}
    __host__ __device__ constexpr int column() const { return tokens * 16 + 16; }
    __host__ __device__ constexpr int in_bytes() const { return 16 * blocks * column(); }
    __host__ __device__ constexpr int stage() const { return in_bytes() + 3 * rp / 8 * column(); }
    __host__ __device__ constexpr int stages() const { return 3; }
    // the plan's part: rows' numbers, tiles, stages
    __host__ __device__ constexpr int lists() const { return SUM_TILES * (TILE * 4 + 16) + SUM_TILES * 4 * 4; }
    __host__ __device__ constexpr int bytes() const { return stages() * stage() + lists() + 256; }
};

template <int MODE>  // 0: bf16 rows of whole vectors, 1: bf16, 2: a checkpoint
struct Sum {
    const SumParams& p;
    const SumJob& job;
    const SumSmem s;
    uint8_t* mem;
    int *ids, *steps;  // row numbers by tile (-1: none); stages: tile * 4 + part
    Piece* tiles;
    uint64_t *full, *empty, *done, *free_;
    volatile uint32_t* abort_flag;
    int tid, warp, lane, c0, n;

    __device__ __forceinline__ bool wait(uint64_t* bar, uint32_t parity, bool& ok) const
    {
        if (ok && !ptx::mbar_wait(bar, parity, U_WAIT_NS)) {
            ok = false;
            *abort_flag = 1u;
        }
        return ok;
    }
    __device__ __forceinline__ int row_at(int k, int t) const { return ids[(steps[k] >> 2) * TILE + (steps[k] & 3) * s.tokens + t]; }
    __device__ __forceinline__ int adapter_at(int k) const { return tiles[steps[k] >> 2].adapter; }
    __device__ __forceinline__ bool ends_run(int k) const { return k + 1 == n || adapter_at(k + 1) != adapter_at(k); }

    // What a thread holds of a stage on its way.
    struct Held {
        uint4 x[MODE == 2 ? 2 : MODE == 1 ? 4 : 1];
        uint32_t scale[MODE == 2 ? 2 : 1];
        float4 mid[2];
    };

    // The thread's 16-byte columns of mid: token and 8 r's; whether there is one.
    __device__ __forceinline__ bool mid_place(int& t, int& r8) const
    {
        const int per = s.rp >> 3;
        t = tid / per;
        r8 = tid - t * per;
        return t < s.tokens;
    }

    __device__ __forceinline__ void fetch(Held& h, int k) const
    {
        if constexpr (MODE == 2) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {  // 16 threads to a row
                const int t = (tid >> 4) + 32 * i, c = c0 + 16 * (tid & 15);
                h.x[i] = make_uint4(0, 0, 0, 0);
                h.scale[i] = 0u;
                if (t >= s.tokens || (s.blocks == 1 && (tid & 8))) continue;
                const int64_t row = row_at(k, t);
                if (row >= 0 && c < job.blocks * 32) {
                    h.x[i] = __ldg(reinterpret_cast<const uint4*>(job.data + row * (job.blocks * 32) + c));
                    h.scale[i] = __ldg(job.scales + row * job.blocks + (c >> 5));
                }
            }
        } else if constexpr (MODE == 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // a warp to a row
                const int t = warp + U_WARPS * i, c = c0 + 8 * lane;
                uint32_t v[4] = {0u, 0u, 0u, 0u};
                if (t < s.tokens && lane < 16 * s.blocks) {
                    const int64_t row = row_at(k, t);
                    if (row >= 0 && c < job.cols) mx::load_any<4, 2>(v, job.in + row * job.in_stride + c, job.cols - c < 8 ? 2 * (job.cols - c) : 16);
                }
                h.x[i] = make_uint4(v[0], v[1], v[2], v[3]);
            }
        }
        int t, r8;
        h.mid[0] = h.mid[1] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (mid_place(t, r8)) {
            const int64_t row = row_at(k, t);
            if (row >= 0) {
                const float* m = job.mid + row * p.rank + 8 * r8;
                if (job.mid_vec) {
                    if (8 * r8 < p.rank) h.mid[0] = __ldg(reinterpret_cast<const float4*>(m));
                    if (8 * r8 + 4 < p.rank) h.mid[1] = __ldg(reinterpret_cast<const float4*>(m) + 1);
                } else {
                    float* v = reinterpret_cast<float*>(h.mid);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        if (8 * r8 + i < p.rank) v[i] = __ldg(m + i);
                }
            }
        }
    }

    // Four integers of a checkpoint as bf16, `e` the exponent bits of 128 times their step, twice.
    __device__ __forceinline__ static uint2 widen(uint32_t word, uint32_t e)
    {
        const uint32_t u = word ^ 0x80808080u;
        uint32_t o[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t w = __byte_perm(u, 0u, i ? 0x4342 : 0x4140);
            const uint32_t a = (w & 0x007f007fu) | e, b = e + 0x00800080u - (w & 0x00800080u);
            const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
            o[i] = *reinterpret_cast<const uint32_t*>(&d);
        }
        return make_uint2(o[0], o[1]);
    }

    __device__ __forceinline__ void store(const Held& h, uint8_t* st) const
    {
        const uint32_t at = ptx::smem_addr(st);
        if constexpr (MODE == 2) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int t = (tid >> 4) + 32 * i;
                if (t >= s.tokens || (s.blocks == 1 && (tid & 8))) continue;
                const uint32_t w[4] = {h.x[i].x, h.x[i].y, h.x[i].z, h.x[i].w};
                uint32_t o[8];
                if (h.scale[i] <= 252u) {
                    const uint32_t e = (h.scale[i] + 1u) * 0x00800080u;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const uint2 d = widen(w[j], e);
                        o[2 * j] = d.x;
                        o[2 * j + 1] = d.y;
                    }
                } else {  // exponents past the trick's: the largest numbers, and NaN
                    const float f = mx::scale_value(h.scale[i]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float2 v[2];
                        mx::unpack_int8x4(v, w[j]);
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const __nv_bfloat162 d = __floats2bfloat162_rn(v[k].x * f, v[k].y * f);
                            o[2 * j + k] = *reinterpret_cast<const uint32_t*>(&d);
                        }
                    }
                }
                const uint32_t dst = at + t * 16 + 2 * (tid & 15) * s.column();
                ptx::st_shared_v4(dst, o[0], o[1], o[2], o[3]);
                ptx::st_shared_v4(dst + s.column(), o[4], o[5], o[6], o[7]);
            }
        } else if constexpr (MODE == 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = warp + U_WARPS * i;
                if (t < s.tokens && lane < 16 * s.blocks) ptx::st_shared_v4(at + t * 16 + lane * s.column(), h.x[i].x, h.x[i].y, h.x[i].z, h.x[i].w);
            }
        }
        int t, r8;
        if (mid_place(t, r8)) {
            const float v[8] = {h.mid[0].x, h.mid[0].y, h.mid[0].z, h.mid[0].w, h.mid[1].x, h.mid[1].y, h.mid[1].z, h.mid[1].w};
            uint32_t o[3][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t b[2][3];
#pragma unroll
                for (int j = 0; j < 2; ++j) {  // as split3; what is not finite makes its sums NaN
                    const float f = v[2 * i + j];
                    b[j][0] = __float_as_uint(f);
                    const float r = f - __uint_as_float(b[j][0] & 0xffff0000u);
                    b[j][1] = __float_as_uint(r);
                    b[j][2] = __float_as_uint(r - __uint_as_float(b[j][1] & 0xffff0000u));
                }
#pragma unroll
                for (int q = 0; q < 3; ++q) o[q][i] = __byte_perm(b[0][q], b[1][q], 0x7632);
            }
            const uint32_t dst = at + s.in_bytes() + t * 16 + r8 * s.column();
#pragma unroll
            for (int q = 0; q < 3; ++q) ptx::st_shared_v4(dst + q * (s.rp >> 3) * s.column(), o[q][0], o[q][1], o[q][2], o[q][3]);
        }
    }

    // bf16 rows straight into their place.
    __device__ __forceinline__ void copy(uint8_t* st, int k) const
    {
        const uint32_t at = ptx::smem_addr(st);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int t = warp + U_WARPS * i, c = c0 + 8 * lane;
            if (t < s.tokens && lane < 16 * s.blocks) {
                const int64_t row = row_at(k, t);
                const bool have = row >= 0 && c < job.cols;
                ptx::cp_async_16s(at + t * 16 + lane * s.column(), have ? job.in + row * job.in_stride + c : job.in, have ? 16 : 0);
            }
        }
    }

    // The finished accumulator of a run that ends with stage k: to the result, or to the piece's part of it.
    __device__ __forceinline__ void flush(uint32_t tmem, int k, int first, bool ok) const
    {
        const int e = adapter_at(k), piece = blockIdx.x / p.per_piece;
        const int t0 = piece * p.tiles_each + (steps[first] >> 2), t1 = piece * p.tiles_each + (steps[k] >> 2) + 1;
        const bool before = p.plan.tile_starts[e] < t0, after = p.plan.tile_starts[e + 1] > t1;
        const int64_t size = static_cast<int64_t>(p.rank) * job.cols;
        float* out = before || after ? job.part + (2 * piece + !before) * size : job.out + e * size;
        const int groups = s.rp >> 4;
        for (int item = warp >> 2; item < groups * s.blocks; item += U_WARPS / 4) {
            const int m = item / groups, r0 = (item - m * groups) * 16;
            const int c = c0 + 128 * m + 32 * (warp & 3) + lane;
            uint32_t v[3][16];
#pragma unroll
            for (int q = 0; q < 3; ++q) ptx::tmem_ld_32x32b_x16(tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + (3 * m + q) * s.rp + r0, v[q]);
            ptx::tmem_ld_wait();
            if (!ok || c >= job.cols) {
                __syncwarp();
                continue;
            }
            float f[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) f[i] = __uint_as_float(v[0][i]) + (__uint_as_float(v[1][i]) + __uint_as_float(v[2][i]));
            if (job.out_col == 1) {
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    if (r0 + i < p.rank) out[(r0 + i) * static_cast<int64_t>(job.cols) + c] = f[i];
            } else {
                float* at = out + static_cast<int64_t>(c) * p.rank + r0;
#pragma unroll
                for (int i = 0; i < 16; i += 4) {
                    if (job.out_vec && r0 + i < p.rank)
                        *reinterpret_cast<float4*>(at + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
                    else
#pragma unroll
                        for (int j = i; j < i + 4; ++j)
                            if (r0 + j < p.rank) at[j] = f[j];
                }
            }
            __syncwarp();
        }
    }

    __device__ __forceinline__ void load(uint32_t tmem)
    {
        bool ok = true;
        constexpr int DEPTH = MODE == 1 ? 1 : 2;
        Held held[DEPTH];
#pragma unroll
        for (int i = 0; i < DEPTH; ++i)
            if (i < n) fetch(held[i], i);
        int first = 0, runs = 0, told = 0;  // told: stages before it have been told of
        for (int k0 = 0; k0 < n; k0 += DEPTH)
#pragma unroll
            for (int i = 0; i < DEPTH; ++i) {
                const int k = k0 + i;
                if (k >= n) break;
                const int at = k % s.stages();
                uint8_t* st = mem + at * s.stage();
                wait(&empty[at], (static_cast<uint32_t>(k / s.stages()) & 1u) ^ 1u, ok);
                if constexpr (MODE == 0) {
                    copy(st, k);
                    ptx::cp_async_commit();
                }
                store(held[i], st);
                ptx::fence_proxy_async_smem();
                // One arrival to a warp (a barrier takes its arrivals one after another); copies' stages are told of a stage later.
                const bool last = ends_run(k);
                if constexpr (MODE == 0) {
                    if (last)
                        ptx::cp_async_wait<0>();
                    else
                        ptx::cp_async_wait<1>();
                }
                __syncwarp();
                if (lane == 0) {
                    if (MODE == 0 && k > told) ptx::mbar_arrive(&full[(k - 1) % s.stages()]);
                    if (MODE != 0 || last) ptx::mbar_arrive(&full[at]);
                }
                if (last) told = k + 1;
                if (k + DEPTH < n) fetch(held[i], k + DEPTH);
                if (last) {
                    wait(done, static_cast<uint32_t>(runs) & 1u, ok);
                    __syncwarp();
                    ptx::tc_fence_after();
                    flush(tmem, k, first, ok);
                    ptx::tc_fence_before();
                    __syncwarp();
                    if (lane == 0) ptx::mbar_arrive(free_);
                    first = k + 1;
                    ++runs;
                }
            }
        if constexpr (MODE == 0) ptx::cp_async_wait_all();
        if (!ok && p.status) atomicMax(p.status, 6u);
    }

    __device__ __forceinline__ void multiply(uint32_t tmem)
    {
        bool ok = true;
        int runs = 0;
        for (int k = 0; k < n; ++k) {
            const int at = k % s.stages();
            const bool begins = k == 0 || adapter_at(k - 1) != adapter_at(k);
            if (begins && runs > 0) wait(free_, static_cast<uint32_t>(runs - 1) & 1u, ok);
            wait(&full[at], static_cast<uint32_t>(k / s.stages()) & 1u, ok);
            ok = __all_sync(0xffffffffu, ok);  // what follows is the whole warp's
            if (!ok) break;
            ptx::fence_proxy_async_smem();
            ptx::tc_fence_after();
            const uint32_t a = ptx::smem_addr(mem + at * s.stage()), b = a + s.in_bytes();
            const uint64_t bd = ptx::plain_mnmajor_desc(b, 128, s.column());
            for (int m = 0; m < s.blocks; ++m) {
                const uint64_t ad = ptx::plain_mnmajor_desc(a + 16 * m * s.column(), 128, s.column());
                const uint32_t d = tmem + 3 * m * s.rp;
                if (s.tokens == 64) {  // rank 64 and below: all three parts in one
                    ptx::mma_bf16_elect_x4(d, ad, bd, 256 / 16, 256 / 16, ptx::idesc_bf16_f32_mn(128, 3 * s.rp), !begins);
                } else {
                    ptx::mma_bf16_elect_x2(d, ad, bd, 256 / 16, 256 / 16, ptx::idesc_bf16_f32_mn(128, 2 * s.rp), !begins);
                    ptx::mma_bf16_elect_x2(d + 2 * s.rp, ad, bd + (s.rp >> 2) * s.column() / 16, 256 / 16, 256 / 16, ptx::idesc_bf16_f32_mn(128, s.rp), !begins);
                }
            }
            ptx::mma_commit_elect(&empty[at]);
            if (ends_run(k)) {
                ptx::mma_commit_elect(done);
                ++runs;
            }
        }
    }
};

__global__ void __launch_bounds__(U_THREADS, 1) sum_tiles(const __grid_constant__ SumParams p)
{
    extern __shared__ __align__(1024) uint8_t raw[];
    const SumSmem s(p.rank);
    uint8_t* lists = raw + s.stages() * s.stage();
    Piece* tiles = reinterpret_cast<Piece*>(lists);
    int* ids = reinterpret_cast<int*>(tiles + SUM_TILES);
    int* steps = ids + SUM_TILES * TILE;
    uint64_t* full = reinterpret_cast<uint64_t*>(lists + s.lists());
    uint64_t *empty = full + 4, *done = empty + 4, *free_ = done + 1;
    uint32_t* slot = reinterpret_cast<uint32_t*>(free_ + 1);
    volatile uint32_t* abort_flag = slot + 1;
    volatile int* count = reinterpret_cast<volatile int*>(slot + 2);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    const int piece = blockIdx.x / p.per_piece, block = blockIdx.x % p.per_piece;
    const SumJob& job = p.jobs[block >= p.jobs[0].col_blocks];
    const int c0 = (block - (block >= p.jobs[0].col_blocks ? p.jobs[0].col_blocks : 0)) * 128 * s.blocks;
    if (tid == 0) {
        for (int i = 0; i < s.stages(); ++i) {
            ptx::mbar_init(&full[i], U_WARPS);
            ptx::mbar_init(&empty[i], 1);
        }
        ptx::mbar_init(done, 1);
        ptx::mbar_init(free_, U_WARPS);
        *abort_flag = 0u;
        ptx::mbar_init_fence();
    }
    ptx::grid_dependency_wait();
    // The piece's tiles, rows and stages; tiles without an adapter, which come last, are left out.
    const int first = piece * p.tiles_each, left = p.plan.tile_starts[p.adapters] - first;
    const int n_tiles = left < p.tiles_each ? left : p.tiles_each;
    if (n_tiles <= 0) return;
    if (warp == U_WARPS) {
        ptx::tmem_alloc(slot, 512);
        ptx::tmem_relinquish();
        Piece t{0, 0, 0, 0};
        if (lane < n_tiles) tiles[lane] = t = p.plan.tiles[first + lane];
        const int parts = (t.rows + s.tokens - 1) / s.tokens;
        int before = parts;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, before, o);
            if (lane >= o) before += up;
        }
        if (lane == 31) *count = before;
        before -= parts;
        for (int i = 0; i < parts; ++i) steps[before + i] = lane * 4 + i;
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    for (int i = tid; i < n_tiles * TILE; i += U_THREADS) ids[i] = (i & (TILE - 1)) < tiles[i / TILE].rows ? p.plan.order[tiles[i / TILE].first + (i & (TILE - 1))] : -1;
    __syncthreads();
    const uint32_t tmem = *slot;
    const auto run = [&](auto sum) {
        if (warp < U_WARPS)
            sum.load(tmem);
        else
            sum.multiply(tmem);
    };
    const int n = *count;
    if (job.mode == 0)
        run(Sum<0>{p, job, s, raw, ids, steps, tiles, full, empty, done, free_, abort_flag, tid, warp, lane, c0, n});
    else if (job.mode == 1)
        run(Sum<1>{p, job, s, raw, ids, steps, tiles, full, empty, done, free_, abort_flag, tid, warp, lane, c0, n});
    else
        run(Sum<2>{p, job, s, raw, ids, steps, tiles, full, empty, done, free_, abort_flag, tid, warp, lane, c0, n});
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == U_WARPS) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

constexpr int J_THREADS = 256;

// Adds the pieces' parts of adapters that lie in more than one, in the pieces' order, and clears those without rows.
__global__ void __launch_bounds__(J_THREADS) join_sums(const __grid_constant__ SumParams p)
{
    ptx::grid_dependency_wait();
    for (int j = 0; j < 2; ++j) {
        const SumJob& job = p.jobs[j];
        if (!job.out) continue;
        const int64_t size = static_cast<int64_t>(p.rank) * job.cols;
        for (int e = blockIdx.y; e < p.adapters; e += gridDim.y) {
            const int t0 = p.plan.tile_starts[e], t1 = p.plan.tile_starts[e + 1];
            const int first = t0 / p.tiles_each, last = (t1 - 1) / p.tiles_each;
            if (t1 > t0 && first == last) continue;
            float* out = job.out + e * size;
            if (job.join_vec) {
                for (int64_t i = static_cast<int64_t>(blockIdx.x) * J_THREADS + threadIdx.x; i < size / 4; i += static_cast<int64_t>(gridDim.x) * J_THREADS) {
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (t1 > t0) {
                        v = reinterpret_cast<const float4*>(job.part + (2 * first + 1) * size)[i];
#pragma unroll 8
                        for (int q = first + 1; q <= last; ++q) {
                            const float4 u = reinterpret_cast<const float4*>(job.part + 2 * static_cast<int64_t>(q) * size)[i];
                            v = make_float4(v.x + u.x, v.y + u.y, v.z + u.z, v.w + u.w);
                        }
                    }
                    reinterpret_cast<float4*>(out)[i] = v;
                }
            } else {
                for (int64_t i = static_cast<int64_t>(blockIdx.x) * J_THREADS + threadIdx.x; i < size; i += static_cast<int64_t>(gridDim.x) * J_THREADS) {
                    float v = 0.f;
                    if (t1 > t0) {
                        v = job.part[(2 * first + 1) * size + i];
#pragma unroll 8
                        for (int q = first + 1; q <= last; ++q) v += job.part[2 * static_cast<int64_t>(q) * size + i];
                    }
                    out[i] = v;
                }
            }
        }
    }
}

// How many tiles a CTA takes: as few as fill the SMs in whole waves, against some 4 us that a CTA costs beside its tiles' 1.2 us each.
int sum_tiles_each(int64_t rows, int64_t adapters, int rank, int64_t cols, int64_t outs)
{
    const SumSmem s(rank);
    const int64_t tiles = rows / TILE + (adapters < rows ? adapters : rows) / 2 + 1;
    const int64_t blocks = mx::cdiv<int64_t>(cols, 128 * s.blocks) + mx::cdiv<int64_t>(outs, 128 * s.blocks);
    int best = 1;
    double best_us = 1e30;
    for (int each = 1; each <= SUM_TILES; ++each) {
        const double us = static_cast<double>(mx::cdiv<int64_t>(mx::cdiv<int64_t>(tiles, each) * blocks, mx::SMS)) * (4.0 + 1.2 * each);
        if (us < best_us) best = each, best_us = us;
    }
    return best;
}

int64_t sum_pieces(const PlanLayout& l, int tiles_each) { return mx::cdiv<int64_t>(l.tiles, tiles_each); }

int launch_sums(SumParams& p, int64_t pieces, cudaStream_t stream)
{
    static std::atomic<uint64_t> done{0};
    const SumSmem s(p.rank);
    p.per_piece = 0;
    int64_t most = 0;
    for (SumJob& job : p.jobs) {
        job.col_blocks = job.out ? mx::cdiv(job.cols, 128 * s.blocks) : 0;
        p.per_piece += job.col_blocks;
        const int64_t size = static_cast<int64_t>(p.rank) * job.cols;
        job.mid_vec = p.rank % 4 == 0 && reinterpret_cast<uintptr_t>(job.mid) % 16 == 0;
        job.out_vec = p.rank % 4 == 0 && reinterpret_cast<uintptr_t>(job.out) % 16 == 0;
        job.join_vec = size % 4 == 0 && (reinterpret_cast<uintptr_t>(job.out) | reinterpret_cast<uintptr_t>(job.part)) % 16 == 0;
        if (job.out && size > most) most = size;
    }
    if (p.per_piece == 0) return CONV2D_OK;
    if (pieces * p.per_piece > INT32_MAX) return CONV2D_ERR_UNSUPPORTED;
    if (!mx::allow_smem(sum_tiles, 227 * 1024, done)) return CONV2D_ERR_CUDA;
    if (mx::launch(sum_tiles, pieces * p.per_piece, U_THREADS, s.bytes(), stream, 1, p) != cudaSuccess) return CONV2D_ERR_CUDA;
    const int64_t across = mx::cdiv<int64_t>(most, 4 * J_THREADS);
    const dim3 grid(static_cast<unsigned>(across < 4 * mx::SMS ? across : 4 * mx::SMS), static_cast<unsigned>(p.adapters < 8 ? p.adapters : 8));
    return mx::launch(join_sums, grid, J_THREADS, 0, stream, 1, p) == cudaSuccess ? CONV2D_OK : CONV2D_ERR_CUDA;
}

}  // namespace ad
}  // namespace sgb
