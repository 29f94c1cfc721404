// The adapters' weight gradients: sums over an adapter's rows, out[e] (r, c) = sum of mid[t][r] * in[t][c], for da (mid = dh, in = x) and
// db (mid = h, in = dy) in one launch.
//
// HBM would bind: `in` is read once, and with rank r there are 2r flops to its 1 or 2 bytes.  What is reached is half of its rate (db of 16384 x 4096, rank 64:
// 47 us for 20 of HBM's, with two launches): a stage's mid is converted by the warps that also see to its copies, some 1.2 us for 64 KB or less.  A CTA takes 256 columns of `in` (128 above
// rank 64, by tensor memory) and a piece of up to 32 of the plan's tiles, whatever adapters those belong to; an adapter's sum that lies in one piece goes straight
// to the result, else each piece's part goes to the workspace and a second launch adds the parts in order.
//
// The reduction runs over rows, so both operands are MN-major: in^T fills the accumulator's 128 lanes with columns, mid its columns
// with r, three times: the three bf16 parts of an fp32 mid (adapter_ptx.cuh) stand side by side, N = 3 * rank, and are added up as the accumulator is read.
// Matrix units cut their sums off at fp32's last bit, towards zero, so that a chain of them is off by half its length of such bits: the first parts, whose bits
// count, have two accumulators, taken by every other stage, with the small parts' between them: first | second | third | first.  An even stage's parts lie in
// this order in shared memory, an odd one's as second | third | first, and go to the accumulators one further on.
// in's rows keep their 128-byte lines (128-byte swizzle: copies that spread a line over shared memory are half as fast); mid's parts lie in core matrices of 8
// rows x 16 bytes, each column of them 16 bytes longer than it needs to be, so that neighbours fall into different banks.
//
// bf16 rows come by cp.async into the operand's place, ahead by all the stages that shared memory holds but two; checkpoints, rows that are not whole vectors, and mid come through
// registers, one or two stages ahead.  A checkpoint's integer becomes a bf16 number by bits: (m | 128) - 128 or 256, each with the scale in its exponent.
//
// db needs nothing of the pass before it, and its CTAs run beside that pass where it leaves SMs free; da's, which take dh, wait for it.  Both gradients of
// 16384 x 4096 -> 4096, rank 64, with dx take 184 us, where dx alone takes 96.
//
// Every wait is bounded, as in the pass (adapter_pass.cuh).
#include "adapter.h"

#include "adapter_params.cuh"
#include "adapter_ptx.cuh"
#include "mxint8.cuh"

namespace sgb {
namespace ad {

constexpr int U_WARPS = 16, U_LOADERS = 32 * U_WARPS, U_THREADS = U_LOADERS + 32;
constexpr int U_STAGES = 6;  // at most

// Shared memory of a stage of `tokens` rows: in by lines of 64 columns, then mid's parts, `column` bytes to a 16-byte column.
struct SumSmem {
    int rp, tokens, blocks;  // blocks of 128 columns
    __host__ __device__ constexpr SumSmem(int rank) : rp((rank + 15) / 16 * 16), tokens(rp <= 64 ? 64 : 32), blocks(rp <= 64 ? 2 : 1) {}
    __host__ __device__ constexpr int column() const { return tokens * 16 + 16; }
    __host__ __device__ constexpr int lines() const { return tokens * 128; }  // of 64 columns
    __host__ __device__ constexpr int in_bytes() const { return 2 * blocks * lines(); }
    __host__ __device__ constexpr int stage() const { return (in_bytes() + 3 * rp / 8 * column() + 1023) / 1024 * 1024; }
    // the plan's part: rows' numbers and each stage's tile by stage, the tiles
    __host__ __device__ constexpr int lists() const { return SUM_TILES * (TILE * 4 + 16) + SUM_TILES * 4 * 4 + 16; }
    __host__ __device__ constexpr int stages() const
    {
        const int fit = (227 * 1024 - lists() - 256) / stage();
        return fit < U_STAGES ? fit : U_STAGES;
    }
    __host__ __device__ constexpr int bytes() const { return stages() * stage() + lists() + 256; }
};

static_assert(SumSmem(16).stages() >= 3 && SumSmem(64).stages() >= 3 && SumSmem(128).stages() >= 3, "a stage filled, one multiplied and one on its way");
// (Asked of sum_blocks, the kernel was 1 to 2% slower.)
static_assert(SumSmem(64).blocks == sum_blocks(64) && SumSmem(65).blocks == sum_blocks(65), "as the rules have it");

template <int MODE>  // 0: bf16 rows of whole vectors, 1: bf16, 2: a checkpoint
struct Sum {
    const SumParams& p;
    const SumJob& job;
    const SumSmem s;
    uint8_t* mem;
    const int *ids, *steps;  // by stage: its rows' numbers (-1: none), its tile
    const Piece* tiles;
    uint64_t *full, *empty, *done, *free_, *last;
    int tid, warp, lane, c0, n, piece;

    // As in the pass: once a wait has run out, the thread waits no more.
    __device__ __forceinline__ void wait(uint64_t* bar, uint32_t parity, bool& ok) const
    {
        if (!ptx::mbar_try_wait(bar, parity) && ok && !ptx::mbar_wait(bar, parity, WAIT_NS)) {
            ok = false;
            atomicMax(p.status, 6u);
        }
    }
    __device__ __forceinline__ int adapter_at(int k) const { return tiles[steps[k]].adapter; }
    __device__ __forceinline__ bool ends_run(int k) const { return k + 1 == n || adapter_at(k + 1) != adapter_at(k); }

    // What a thread holds of a stage on its way.
    struct Held {
        uint4 x[MODE == 2 ? 2 : MODE == 1 ? 4 : 1];
        uint32_t scale[MODE == 2 ? 2 : 1];
        float4 mid[2];
    };

    // The thread's place in a stage: mid's token and 8 ranks, if it has any; in's columns and the four (two of a checkpoint) tokens from `row` on.
    int mid_token, mid_rank, row, col;
    bool has_mid, has_in;
    __device__ __forceinline__ void find_place()
    {
        const int per = s.rp >> 3;
        mid_token = tid / per;
        mid_rank = tid - mid_token * per;
        has_mid = mid_token < s.tokens;
        if constexpr (MODE == 2) {  // 16 threads to two rows
            row = 2 * (tid >> 4);
            col = c0 + 16 * (tid & 15);
            has_in = row < s.tokens && (s.blocks == 2 || (tid & 15) < 8) && col < job.blocks * 32;
        } else {  // a warp to four
            row = 4 * warp;
            col = c0 + 8 * lane;
            has_in = row < s.tokens && lane < 16 * s.blocks && col < job.cols;
        }
    }
    // Where in's 16-byte column c (of 8) of token t lies.
    __device__ __forceinline__ uint32_t in_at(int t, int c) const { return (c >> 3) * s.lines() + t * 128 + (((c ^ t) & 7) << 4); }
    // Whether the thread's part of in's place in a stage exists (it is zero where in has none).
    __device__ __forceinline__ bool stores_in() const
    {
        return row < s.tokens && (MODE == 2 ? s.blocks == 2 || (tid & 15) < 8 : lane < 16 * s.blocks);
    }

    __device__ __forceinline__ void fetch(Held& h, int k) const
    {
        const int* rows = ids + k * s.tokens;
        if constexpr (MODE == 2) {
            const int2 t = has_in ? *reinterpret_cast<const int2*>(rows + row) : make_int2(-1, -1);
            const int64_t pitch = job.blocks * 32;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int64_t r = i ? t.y : t.x;
                h.x[i] = ptx::ld_stream_v4_if(job.data + r * pitch + col, r >= 0);
                h.scale[i] = ptx::ld_u8_if(job.scales + r * job.blocks + (col >> 5), r >= 0);
            }
        } else if constexpr (MODE == 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int64_t r = has_in ? rows[row + i] : -1;
                uint32_t v[4] = {0u, 0u, 0u, 0u};
                if (r >= 0) mx::load_any<4, 2>(v, job.in + r * job.in_stride + col, job.cols - col < 8 ? 2 * (job.cols - col) : 16);
                h.x[i] = make_uint4(v[0], v[1], v[2], v[3]);
            }
        }
        const int64_t r = has_mid ? rows[mid_token] : -1;
        const float* m = job.mid + r * p.rank + 8 * mid_rank;
        if (job.mid_vec) {
            const uint4 a = ptx::ld_v4_if(m, r >= 0 && 8 * mid_rank < p.rank), b = ptx::ld_v4_if(m + 4, r >= 0 && 8 * mid_rank + 4 < p.rank);
            h.mid[0] = make_float4(__uint_as_float(a.x), __uint_as_float(a.y), __uint_as_float(a.z), __uint_as_float(a.w));
            h.mid[1] = make_float4(__uint_as_float(b.x), __uint_as_float(b.y), __uint_as_float(b.z), __uint_as_float(b.w));
        } else {
            float* v = reinterpret_cast<float*>(h.mid);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = r >= 0 && 8 * mid_rank + i < p.rank ? m[i] : 0.f;  // dh, which the pass beside writes: no __ldg
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

    __device__ __forceinline__ void store(const Held& h, uint32_t at, int turn) const
    {
        if constexpr (MODE == 2) {
            if (stores_in())
#pragma unroll
            for (int i = 0; i < 2; ++i) {
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
                ptx::st_shared_v4(at + in_at(row + i, 2 * (tid & 15)), o[0], o[1], o[2], o[3]);
                ptx::st_shared_v4(at + in_at(row + i, 2 * (tid & 15) + 1), o[4], o[5], o[6], o[7]);
            }
        } else if constexpr (MODE == 1) {
            if (stores_in())
#pragma unroll
                for (int i = 0; i < 4; ++i) ptx::st_shared_v4(at + in_at(row + i, lane), h.x[i].x, h.x[i].y, h.x[i].z, h.x[i].w);
        }
        if (has_mid) {
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
            const uint32_t part = (s.rp >> 3) * s.column(), dst = at + s.in_bytes() + mid_token * 16 + mid_rank * s.column();
            const uint32_t to[3] = {turn ? dst + 2 * part : dst, turn ? dst : dst + part, turn ? dst + part : dst + 2 * part};
#pragma unroll
            for (int q = 0; q < 3; ++q) ptx::st_shared_v4(to[q], o[q][0], o[q][1], o[q][2], o[q][3]);
        }
    }

    // bf16 rows straight into their place; zeros for what is not there.
    __device__ __forceinline__ void copy(uint32_t at, int k) const
    {
        const int4 t = row < s.tokens ? *reinterpret_cast<const int4*>(ids + k * s.tokens + row) : make_int4(-1, -1, -1, -1);
        const int rows[4] = {t.x, t.y, t.z, t.w};
        const bool mine = stores_in();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bool have = has_in && rows[i] >= 0;
            ptx::cp_async_16_fill_if(at + in_at(row + i, lane), have ? job.in + rows[i] * job.in_stride + col : job.in, have ? 16 : 0, mine);
        }
    }

    // The finished accumulator of a run that ends with stage k: to the result, or to the piece's part of it.
    __device__ __forceinline__ void flush(uint32_t tmem, int k, int first, bool ok) const
    {
        const int e = adapter_at(k);
        const int t0 = piece * job.tiles_each + steps[first], t1 = piece * job.tiles_each + steps[k] + 1;
        const bool before = p.plan.tile_starts[e] < t0, after = p.plan.tile_starts[e + 1] > t1;
        const int64_t size = static_cast<int64_t>(p.rank) * job.cols;
        float* out = before || after ? job.part + (2 * piece + !before) * size : job.out + e * size;
        const int groups = s.rp >> 4;
        for (int item = warp >> 2; item < groups * s.blocks; item += U_WARPS / 4) {
            const int m = item / groups, r0 = (item - m * groups) * 16;
            const int c = c0 + 128 * m + 32 * (warp & 3) + lane;
            float f[16];
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // the smallest parts first
                const int q = i < 2 ? 2 - i : 3 * (i - 2);
                if (q == 3 && k == first) continue;
                uint32_t v[16];
                ptx::tmem_ld_32x32b_x16(tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16) + (4 * m + q) * s.rp + r0, v);
                ptx::tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 16; ++j) f[j] = i == 0 ? __uint_as_float(v[j]) : __uint_as_float(v[j]) + f[j];
            }
            if (!ok || c >= job.cols) {
                __syncwarp();
                continue;
            }
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
        find_place();
        constexpr int DEPTH = MODE == 1 ? 1 : 2;
        Held held[DEPTH];
#pragma unroll
        for (int i = 0; i < DEPTH; ++i)
            if (i < n) fetch(held[i], i);
        int first = 0, runs = 0;
        int at = 0;  // the slot of this stage
        uint32_t free_phase = 1u;
        // Copies run ahead of the stage that is told of by all slots but one, whose products go on meanwhile, and the stage's own.
        const int ahead = s.stages() - 2;
        int to = 0;
        uint32_t to_phase = 1u;
        const auto copy_next = [&](int k) {
            if (k < n) {
                wait(&empty[to], to_phase, ok);
                copy(ptx::smem_addr(mem) + to * s.stage(), k);
            }
            ptx::cp_async_commit();
            to = to + 1 == s.stages() ? 0 : to + 1;
            to_phase = to ? to_phase : to_phase ^ 1u;
        };
        if constexpr (MODE == 0)
            for (int k = 0; k < ahead; ++k) copy_next(k);
        for (int k0 = 0; k0 < n; k0 += DEPTH)
#pragma unroll
            for (int i = 0; i < DEPTH; ++i) {
                const int k = k0 + i;
                if (k >= n) break;
                const uint32_t st = ptx::smem_addr(mem) + at * s.stage();
                const bool last = ends_run(k);
                if constexpr (MODE == 0)
                    copy_next(k + ahead);
                else
                    wait(&empty[at], free_phase, ok);
                store(held[i], st, (k - first) & 1);
                if (k + DEPTH < n) fetch(held[i], k + DEPTH);
                if constexpr (MODE == 0) {
                    switch (ahead) {
                        case 1: ptx::cp_async_wait<1>(); break;
                        case 2: ptx::cp_async_wait<2>(); break;
                        case 3: ptx::cp_async_wait<3>(); break;
                        default: ptx::cp_async_wait<4>();
                    }
                }
                ptx::fence_proxy_async_smem();
                // One arrival to a warp: a barrier takes its arrivals one after another.
                __syncwarp();
                ptx::mbar_arrive_if(&full[at], lane == 0);
                at = at + 1 == s.stages() ? 0 : at + 1;
                free_phase = at ? free_phase : free_phase ^ 1u;
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
    }

    __device__ __forceinline__ void multiply(uint32_t tmem)
    {
        bool ok = true;
        int runs = 0, at = 0;
        uint32_t phase = 0u;
        int turn = 0;  // of the run's stages
        for (int k = 0; k < n; ++k) {
            if (turn == 0 && runs > 0) wait(free_, static_cast<uint32_t>(runs - 1) & 1u, ok);
            const bool last = ends_run(k);
            wait(&full[at], phase, ok);
            __syncwarp();  // what follows is the whole warp's
            ptx::fence_proxy_async_smem();
            ptx::tc_fence_after();
            const uint32_t a = ptx::smem_addr(mem + at * s.stage()), b = a + s.in_bytes();
            const uint64_t bd = ptx::plain_mnmajor_desc(b, 128, s.column());
            for (int m = 0; m < s.blocks; ++m) {
                const uint64_t ad = ptx::sw128_mnmajor_desc(a + 2 * m * s.lines(), s.lines(), 1024);
                const uint32_t d = tmem + (4 * m + (turn & 1)) * s.rp;
                const uint64_t bd2 = bd + (s.rp >> 2) * s.column() / 16;
                if (s.tokens == 32) {  // ranks above 64
                    ptx::mma_bf16_elect_x2(d, ad, bd, 2048 / 16, 256 / 16, ptx::idesc_bf16_f32_mn(128, 2 * s.rp), turn > 0);
                    ptx::mma_bf16_elect_x2(d + 2 * s.rp, ad, bd2, 2048 / 16, 256 / 16, ptx::idesc_bf16_f32_mn(128, s.rp), turn > 1);
                } else if (turn == 1) {  // the second accumulator begins
                    ptx::mma_bf16_elect_x4(d, ad, bd, 2048 / 16, 256 / 16, ptx::idesc_bf16_f32_mn(128, 2 * s.rp), 1u);
                    ptx::mma_bf16_elect_x4(d + 2 * s.rp, ad, bd2, 2048 / 16, 256 / 16, ptx::idesc_bf16_f32_mn(128, s.rp), 0u);
                } else {
                    ptx::mma_bf16_elect_x4(d, ad, bd, 2048 / 16, 256 / 16, ptx::idesc_bf16_f32_mn(128, 3 * s.rp), turn > 0);
                }
            }
            ptx::mma_commit_elect(&empty[at]);
            at = at + 1 == s.stages() ? 0 : at + 1;
            phase = at ? phase : phase ^ 1u;
            turn = last ? 0 : turn + 1;
            if (last) {
                ptx::mma_commit_elect(done);
                ++runs;
            }
        }
        // as in the pass
        ptx::mma_commit_elect(last);
        if (!ptx::mbar_wait(last, 0, LAST_WAIT_NS)) atomicMax(p.status, 6u);
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
    uint64_t *empty = full + U_STAGES, *done = empty + U_STAGES, *free_ = done + 1, *last = free_ + 1;
    uint32_t* slot = reinterpret_cast<uint32_t*>(last + 1);
    volatile int* count = reinterpret_cast<volatile int*>(slot + 1);
    const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
    // db's CTAs first: they need nothing of the pass before them, and run beside it where it leaves SMs free.
    const bool late = static_cast<int>(blockIdx.x) >= p.first_late;
    const SumJob& job = p.jobs[late ? 0 : 1];
    const int number = static_cast<int>(blockIdx.x) - (late ? p.first_late : 0), piece = number / job.col_blocks;
    const int c0 = (number - piece * job.col_blocks) * 128 * s.blocks;
    if (tid == 0) {
        for (int i = 0; i < s.stages(); ++i) {
            ptx::mbar_init(&full[i], i == 0 ? U_WARPS + LOST_ROWS : U_WARPS);
            ptx::mbar_init(&empty[i], 1);
        }
        ptx::mbar_init(done, 1 + LOST_DONE);
        ptx::mbar_init(last, 1);
        ptx::mbar_init(free_, U_WARPS);
        ptx::mbar_init_fence();
    }
    // The pass has waited for what came before it, the plan with it, and lets this kernel start only then.
    if (!p.beside) ptx::grid_dependency_wait();
    // The piece's tiles, rows and stages; tiles without an adapter, which come last, are left out.
    const int first = piece * job.tiles_each, left = p.plan.tile_starts[p.adapters] - first;
    const int n_tiles = left < job.tiles_each ? left : job.tiles_each;
    // This kernel ends after the pass, so that whatever waits for it has waited for both.
    if (n_tiles <= 0) {
        if (p.beside) ptx::grid_dependency_wait();
        return;
    }
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
        for (int i = 0; i < parts; ++i) steps[before + i] = lane | i << 8;
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    const int n = *count;
    for (int i = tid; i < n * s.tokens; i += U_THREADS) {
        const int k = i / s.tokens, t = (steps[k] >> 8) * s.tokens + i - k * s.tokens;
        const Piece piece_of = tiles[steps[k] & 255];
        ids[i] = t < piece_of.rows ? p.plan.order[piece_of.first + t] : -1;
    }
    __syncthreads();
    if (tid < n) steps[tid] &= 255;
    if (late && p.beside) ptx::grid_dependency_wait();  // for dh
    __syncthreads();
    const uint32_t tmem = *slot;
    const auto run = [&](auto sum) {
        if (warp < U_WARPS)
            sum.load(tmem);
        else
            sum.multiply(tmem);
    };
    if (job.mode == 0)
        run(Sum<0>{p, job, s, raw, ids, steps, tiles, full, empty, done, free_, last, tid, warp, lane, c0, n, piece});
    else if (job.mode == 1)
        run(Sum<1>{p, job, s, raw, ids, steps, tiles, full, empty, done, free_, last, tid, warp, lane, c0, n, piece});
    else
        run(Sum<2>{p, job, s, raw, ids, steps, tiles, full, empty, done, free_, last, tid, warp, lane, c0, n, piece});
    ptx::tc_fence_before();
    __syncthreads();
    if (warp == U_WARPS) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
    if (!late && p.beside) ptx::grid_dependency_wait();
}

constexpr int J_THREADS = 256, J_SLICES = 8;

// The sum of an adapter's parts, V of type T at a time; parts first .. first + n - 1 in order.  From eight parts on a block's warps take an eighth of them each,
// all on their way at once, and the eighths are added in order.
template <typename T, typename Add>
__device__ __forceinline__ void join_parts_of(const SumJob& job, float* out, int64_t size, int first, int n, T* eighths, const Add& add)
{
    constexpr int V = sizeof(T) / 4;
    const int slices = n >= J_SLICES ? J_SLICES : 1, per = J_THREADS / slices, slice = threadIdx.x / per, lane = threadIdx.x - slice * per;
    const int q0 = n * slice / slices, q1 = n * (slice + 1) / slices;
    for (int64_t i0 = static_cast<int64_t>(blockIdx.x) * per; i0 < size / V; i0 += static_cast<int64_t>(gridDim.x) * per) {
        const int64_t i = i0 + lane;
        T v{};
        if (i < size / V)
#pragma unroll 8
            for (int q = q0; q < q1; ++q)  // an adapter that begins in a piece has the second of its parts there, one that goes on the first
                v = add(v, reinterpret_cast<const T*>(job.part + (2 * static_cast<int64_t>(first + q) + (q == 0)) * size)[i]);
        if (slices > 1) {
            __syncthreads();
            eighths[threadIdx.x] = v;
            __syncthreads();
            if (slice == 0)
#pragma unroll
                for (int k = 1; k < J_SLICES; ++k) v = add(v, eighths[k * per + lane]);
        }
        if (slice == 0 && i < size / V) reinterpret_cast<T*>(out)[i] = v;
    }
}

// Adds the pieces' parts of adapters that lie in more than one, in the pieces' order, and clears those without rows.
__global__ void __launch_bounds__(J_THREADS) join_sums(const __grid_constant__ SumParams p)
{
    __shared__ float4 eighths[J_THREADS];
    ptx::grid_dependency_wait();
    for (int j = 0; j < 2; ++j) {
        const SumJob& job = p.jobs[j];
        if (!job.out) continue;
        const int64_t size = static_cast<int64_t>(p.rank) * job.cols;
        for (int e = blockIdx.y; e < p.adapters; e += gridDim.y) {
            const int t0 = p.plan.tile_starts[e], t1 = p.plan.tile_starts[e + 1];
            const int first = t0 / job.tiles_each, n = t1 > t0 ? (t1 - 1) / job.tiles_each - first + 1 : 0;
            if (n == 1) continue;
            float* out = job.out + e * size;
            if (job.join_vec)
                join_parts_of(job, out, size, first, n, eighths, [](float4 a, float4 b) { return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w); });
            else
                join_parts_of(job, out, size, first, n, reinterpret_cast<float*>(eighths), [](float a, float b) { return a + b; });
        }
    }
}

int64_t sum_pieces(const PlanLayout& l, int tiles_each) { return mx::cdiv<int64_t>(l.tiles, tiles_each); }

int launch_sums(SumParams& p, const PlanLayout& l, cudaStream_t stream)
{
    static std::atomic<uint64_t> done{0};
    const SumSmem s(p.rank);
    int64_t most = 0, ctas = 0;
    bool many = false;  // parts to an adapter
    for (SumJob& job : p.jobs) {
        job.col_blocks = job.out ? mx::cdiv(job.cols, 128 * s.blocks) : 0;
        if (job.out) {
            ctas += sum_pieces(l, job.tiles_each) * job.col_blocks;
            many = many || sum_pieces(l, job.tiles_each) >= J_SLICES * p.adapters;
        }
        const int64_t size = static_cast<int64_t>(p.rank) * job.cols;
        job.mid_vec = p.rank % 4 == 0 && reinterpret_cast<uintptr_t>(job.mid) % 16 == 0;
        job.out_vec = p.rank % 4 == 0 && reinterpret_cast<uintptr_t>(job.out) % 16 == 0;
        job.join_vec = size % 4 == 0 && (reinterpret_cast<uintptr_t>(job.out) | reinterpret_cast<uintptr_t>(job.part)) % 16 == 0;
        const int64_t units = job.join_vec ? size / 4 : size;
        if (job.out && units > most) most = units;
    }
    if (ctas == 0) return CONV2D_OK;
    if (ctas > INT32_MAX) return CONV2D_ERR_UNSUPPORTED;
    p.first_late = p.jobs[1].out ? static_cast<int>(sum_pieces(l, p.jobs[1].tiles_each) * p.jobs[1].col_blocks) : 0;
    if (!mx::allow_smem(sum_tiles, 227 * 1024, done)) return CONV2D_ERR_CUDA;
    if (mx::launch(sum_tiles, ctas, U_THREADS, s.bytes(), stream, 1, p) != cudaSuccess) return CONV2D_ERR_CUDA;
    const int64_t across = mx::cdiv<int64_t>(most, many ? J_THREADS / J_SLICES : J_THREADS);
    const dim3 grid(static_cast<unsigned>(across < 4 * mx::SMS ? across : 4 * mx::SMS), static_cast<unsigned>(p.adapters < 8 ? p.adapters : 8));
    return mx::launch(join_sums, grid, J_THREADS, 0, stream, 1, p) == cudaSuccess ? CONV2D_OK : CONV2D_ERR_CUDA;
}

}  // namespace ad
}  // namespace sgb
