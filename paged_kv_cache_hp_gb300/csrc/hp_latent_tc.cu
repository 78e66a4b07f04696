// hp_latent_tc.cu -- attention over a paged cache of shared latent rows on the tensor cores
// (tcgen05): latent_dim 512, rope_dim 64, absorbed form.
//
// A CTA takes a tile of 64 (query, head) rows of one sequence and a range of its steps of 64
// tokens (hp_latent.cuh has the split).  Per step, with C the step's 64 cache rows of 576:
//   S [64 rows x 64 tokens]     = Q . C^T            36 products of 16 dims, M = N = 64
//   O^T [512 dims x 64 rows]   += C[:, :512]^T . P^T  4 tiles of 128 dims, 4 products each
// so the step's rows are loaded once (TMA, 128-byte swizzled, nine 64-dim chunks of 8 KiB) and
// serve as the B operand of S (K-major) and the A operand of O^T (M-major).  O^T rather than O:
// 64 rows of 512 fp32 sums are half of TMEM either way, but M = 128 products run at the full
// rate where M = 64 runs at half of it.  O^T stays in TMEM over the whole range: a row's
// reference maximum moves (and its column of O^T is rescaled) only when a score exceeds it by
// more than 2^kTau.  P (weights rounded to the element type) overwrites the step's rope chunk,
// which S has read.
//
// Shared memory: Q 72 KiB, two stages of C of 72 KiB -- 216 of 227 KiB; TMEM: O^T 256 columns,
// S 2 x 64.  Roles: warp 0 loads C, warp 6 the queries, warp 1 issues the products (S of a step
// ahead of O^T of the step before), warps 2-5 do the softmax and the epilogue.
//
// Above 64 heads a worker is two neighbouring CTAs whose tiles read the same tokens at the same
// time, so the second read of a row finds it in L2.
//
// Every wait is bounded (about 2 s) and reports HP_ERR_TIMEOUT; the softmax threads decide
// together, at their barrier, to stop, and operations in flight are waited for (bounded).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "hp_attn_merge.cuh"
#include "hp_internal.cuh"
#include "hp_latent.cuh"
#include "hp_resolve.cuh"
#include "hp_tcgen05.cuh"
#include "hp_tma.cuh"

namespace hp {
namespace {

using namespace tma;
using namespace tc;

constexpr int kW = 576, kR = 512;
constexpr uint32_t kRows = 64;                 // rows of a tile
constexpr uint32_t kTok = kLatentStep;         // tokens of a step
constexpr uint32_t kChunks = kW / 64, kVChunks = kR / 64;
constexpr uint32_t kChunk = 64 * 128;          // 64 rows x 64 dims
constexpr uint32_t kStage = kChunks * kChunk;
constexpr uint32_t kStages = 2;
constexpr uint32_t kOffC = kChunks * kChunk;   // Q first, then the stages
constexpr uint32_t kSmem = kOffC + kStages * kStage + 1024;
constexpr uint32_t kOCol = 0, kSCol = 256;     // TMEM columns
constexpr uint32_t kTmemCols = 512;
constexpr int kThreads = 7 * 32;
constexpr int kSoftmax = 128;
constexpr float kTau = 8.0f;

// A segment: steps k0 .. k1 - 1 of one tile, without those in which none of its rows sees a
// token (k0 >= k1: nothing to compute).
struct Segment {
    uint64_t s, len, q0, n, r0, k0, k1, ustart, steps;
    uint32_t rows;  // rows of the tile that exist, at least 1
};

struct Walk {
    const LatentArgs& a;
    uint64_t pos, end;
    uint32_t tile;  // this CTA's tile within the group
    __device__ bool next(Segment& g)
    {
        while (pos < end) {
            g.s = find_seq(a.units_off, a.num_seqs, pos);
            g.len = index_at(a.lens, a.idx64, g.s);
            g.q0 = a.q_ptr ? index_at(a.q_ptr, a.idx64, g.s) : g.s;
            g.n = (a.q_ptr ? index_at(a.q_ptr, a.idx64, g.s + 1) : g.s + 1) - g.q0;
            g.steps = (g.len + kTok - 1) / kTok;
            const uint64_t off = pos - a.units_off[g.s], grp = off / g.steps;
            g.ustart = a.units_off[g.s] + grp * g.steps;
            g.k0 = off % g.steps;
            g.k1 = umin(g.steps, g.k0 + (end - pos));
            pos += g.k1 - g.k0;
            g.r0 = grp * a.group_rows + tile * kRows;
            const uint64_t all = g.n * a.H;
            if (g.r0 >= all) continue;  // the group's last tile may have no rows
            g.rows = (uint32_t)umin(kRows, all - g.r0);
            const uint64_t last = (g.r0 + g.rows - 1) / a.H;  // the tile's last query sees most
            const uint64_t seen = g.len + 1 + last > g.n ? g.len + 1 + last - g.n : 0;
            g.k1 = umin(g.k1, (seen + kTok - 1) / kTok);
            return true;
        }
        return false;
    }
};

template <typename T> __device__ __forceinline__ uint32_t pack2(float a, float b);
template <> __device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <> __device__ __forceinline__ uint32_t pack2<__half>(float a, float b)
{
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <typename T> __device__ __forceinline__ T round1(float a);
template <> __device__ __forceinline__ __nv_bfloat16 round1<__nv_bfloat16>(float a) { return __float2bfloat16_rn(a); }
template <> __device__ __forceinline__ __half round1<__half>(float a) { return __float2half_rn(a); }

template <typename T>
__global__ void __launch_bounds__(kThreads, 1)
    latent_tc_kernel(const LatentArgs a, const __grid_constant__ CUtensorMap tmc,
                     const __grid_constant__ CUtensorMap tmq)
{
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    __shared__ __align__(8) unsigned long long c_full[kStages], c_free[kStages], s_full[2], s_free[2],
        p_full[2], o_done[2], o_free, q_full, q_free;
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag, fail_s[2];
    __shared__ float corr_s[kRows], inv_s[kRows];

    pdl_wait();
    if (a.hdr->verdict != kVerdictOk) return;
    const unsigned warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    T* out = static_cast<T*>(a.out);
    // queries of a sequence without tokens: zeros
    for (uint64_t s = (uint64_t)blockIdx.x * 7 + warp; s < a.num_seqs; s += (uint64_t)gridDim.x * 7)
        if (a.units_off[s] == a.units_off[s + 1]) {
            const uint64_t q0 = a.q_ptr ? index_at(a.q_ptr, a.idx64, s) : s;
            const uint64_t q1 = a.q_ptr ? index_at(a.q_ptr, a.idx64, s + 1) : s + 1;
            uint4* o = reinterpret_cast<uint4*>(out);
            for (uint64_t i = q0 * a.H * (kR / 8) + lane; i < q1 * a.H * (kR / 8); i += 32)
                o[i] = make_uint4(0, 0, 0, 0);
        }
    const uint32_t tiles = a.group_rows / kRows;
    const uint64_t total = a.hdr->total_units, Lw = (total + a.workers - 1) / a.workers;
    const uint64_t v = blockIdx.x / tiles, beg = umin(v * Lw, total), end = umin(beg + Lw, total);
    if (beg >= end) return;  // the whole CTA, before any barrier or TMEM

    const uint32_t sm0 = (smem_u32(smem_raw) + 1023u) & ~1023u;
    unsigned char* smem = smem_raw + (sm0 - smem_u32(smem_raw));
    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < kStages; ++i) {
            mbar_init(smem_u32(&c_full[i]), 1);
            mbar_init(smem_u32(&c_free[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&s_full[i]), 1);
            mbar_init(smem_u32(&s_free[i]), kSoftmax);
            mbar_init(smem_u32(&p_full[i]), kSoftmax);
            mbar_init(smem_u32(&o_done[i]), 1);
        }
        mbar_init(smem_u32(&o_free), kSoftmax);
        mbar_init(smem_u32(&q_full), 1);
        mbar_init(smem_u32(&q_free), 1);
        abort_flag = 0;
        fail_s[0] = fail_s[1] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tmem_alloc(smem_u32(&tmem_base), kTmemCols);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_base;
    Walk walk{a, beg, end, (uint32_t)(blockIdx.x % tiles)};
    Segment g;
    auto failed = [&](bool ok) {
        if (!ok) {
            abort_flag = 1;
            report(a.d_status, HP_ERR_TIMEOUT);
        }
        return !ok || *(volatile int*)&abort_flag;
    };

    if (warp == 0) {
        // ----------------------------------------------------------- cache rows of each step
        const uint32_t P = (uint32_t)a.page_size, box = P < kTok ? P : kTok, ppc = kTok / box;
        uint64_t j = 0;
        bool stop = false;
        while (!stop && walk.next(g)) {
            const uint64_t tab0 = index_at(a.seq_ptr, a.idx64, g.s);
            for (uint64_t k = g.k0; k < g.k1; ++k, ++j) {
                const uint32_t st = (uint32_t)(j % kStages);
                // lane i < ppc: the pool row of the step's i-th page, if a slot of it is live
                const uint64_t t = k * kTok + (uint64_t)lane * box;
                const bool live = lane < ppc && t < g.len;
                const uint32_t row =
                    live ? (uint32_t)(index_at(a.table, a.idx64, tab0 + t / P) * P + t % P) : 0u;
                const uint32_t pages = __popc(__ballot_sync(0xffffffffu, live));
                int ok = 1;
                if (lane == 0 && j >= kStages)
                    ok = mbar_wait(smem_u32(&c_free[st]), (uint32_t)((j / kStages - 1) & 1));
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (__any_sync(0xffffffffu, failed(ok != 0))) {
                    stop = true;
                    break;
                }
                const uint32_t bar = smem_u32(&c_full[st]), base = sm0 + kOffC + st * kStage;
                if (lane == 0) mbar_expect_tx(bar, pages * box * 128 * kChunks);
                __syncwarp();
                const uint32_t boxes = pages * kChunks;
                for (uint32_t b0 = 0; b0 < boxes; b0 += 32) {  // box b: chunk b / pages, page b % pages
                    const uint32_t b = b0 + lane, ch = b / pages, pg = b - ch * pages;
                    const uint32_t r = __shfl_sync(0xffffffffu, row, pg);
                    if (b < boxes && !(a.test_stall && j == 0))
                        tma_2d(base + ch * kChunk + pg * box * 128, &tmc, (int)(ch * 64), (int)r, bar);
                }
            }
        }
        if (lane == 0)  // the last loads land before the shared memory goes
            for (uint64_t x = j > kStages ? j - kStages : 0; x < j; ++x)
                mbar_wait(smem_u32(&c_full[x % kStages]), (uint32_t)((x / kStages) & 1));
        __syncwarp();
    } else if (warp == 6) {
        // ------------------------------------------------------------- queries of each tile
        if (lane == 0) {
            uint64_t seg = 0;
            while (walk.next(g)) {
                if (g.k0 >= g.k1) continue;
                const bool ok = seg == 0 || mbar_wait(smem_u32(&q_free), (uint32_t)((seg - 1) & 1));
                if (failed(ok)) break;
                mbar_expect_tx(smem_u32(&q_full), kChunks * kChunk);
                for (uint32_t c = 0; c < kChunks; ++c)
                    tma_2d(sm0 + c * kChunk, &tmq, (int)(c * 64), (int)(g.q0 * a.H + g.r0), smem_u32(&q_full));
                ++seg;
            }
            if (seg) mbar_wait(smem_u32(&q_full), (uint32_t)((seg - 1) & 1));
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---------------------------------------------------------------- products, one thread
        if (lane == 0) {
            const uint32_t id_s = f16_idesc(a.bf16 != 0, false, false, kRows, kTok);
            const uint32_t id_o = f16_idesc(a.bf16 != 0, true, false, 128, kRows);
            const uint64_t qd = sw128_desc(sm0, 16, 1024), cd0 = sw128_desc(sm0 + kOffC, 16, 1024);
            const uint64_t vd0 = sw128_desc(sm0 + kOffC, kChunk, 1024);
            uint64_t j = 0, seg = 0, done = 0;  // steps with S issued, segments, steps with O issued
            bool ok = true;
            // O^T of the step `done`; fresh: the first of its segment
            auto issue_o = [&](bool fresh) {
                const uint64_t x = done;
                ok = mbar_wait(smem_u32(&p_full[x % 2]), (uint32_t)((x / 2) & 1)) &&
                     (!fresh || seg == 0 || mbar_wait(smem_u32(&o_free), (uint32_t)((seg - 1) & 1)));
                if (failed(ok)) {
                    ok = false;
                    return;
                }
                fence_after();
                const uint32_t so = (uint32_t)(x % kStages) * kStage;
                const uint64_t vd = vd0 + (so >> 4), pd = cd0 + ((so + kVChunks * kChunk) >> 4);
#pragma unroll
                for (uint32_t m = 0; m < 4; ++m)
#pragma unroll
                    for (uint32_t kk = 0; kk < 4; ++kk)
                        mma_f16(tmem + kOCol + m * kRows, vd + ((m * 2 * kChunk + kk * 2048) >> 4),
                                pd + ((kk * 32) >> 4), id_o, !fresh || kk > 0);
                mma_commit(smem_u32(&c_free[x % kStages]));
                mma_commit(smem_u32(&o_done[x % 2]));
                ++done;
            };
            while (ok && walk.next(g)) {
                if (g.k0 >= g.k1) continue;
                for (uint64_t k = g.k0; ok && k < g.k1; ++k) {
                    ok = mbar_wait(smem_u32(&c_full[j % kStages]), (uint32_t)((j / kStages) & 1)) &&
                         (k != g.k0 || mbar_wait(smem_u32(&q_full), (uint32_t)(seg & 1))) &&
                         (j < 2 || mbar_wait(smem_u32(&s_free[j % 2]), (uint32_t)((j / 2 - 1) & 1)));
                    if (failed(ok)) {
                        ok = false;
                        break;
                    }
                    fence_after();
                    const uint64_t cd = cd0 + (((uint32_t)(j % kStages) * kStage) >> 4);
                    const uint32_t d = tmem + kSCol + (uint32_t)(j % 2) * kTok;
#pragma unroll
                    for (uint32_t u = 0; u < kChunks * 4; ++u) {
                        const uint32_t o = ((u >> 2) * kChunk + (u & 3) * 32) >> 4;
                        mma_f16(d, qd + o, cd + o, id_s, u);
                    }
                    mma_commit(smem_u32(&s_full[j % 2]));
                    if (k + 1 == g.k1) mma_commit(smem_u32(&q_free));
                    ++j;
                    if (k > g.k0) issue_o(k == g.k0 + 1);
                }
                if (ok) issue_o(g.k1 == g.k0 + 1);
                ++seg;
            }
            // everything issued has completed before the TMEM goes
            if (j) mbar_wait(smem_u32(&s_full[(j - 1) % 2]), (uint32_t)(((j - 1) / 2) & 1));
            if (done) mbar_wait(smem_u32(&o_done[(done - 1) % 2]), (uint32_t)(((done - 1) / 2) & 1));
        }
        __syncwarp();
    } else {
        // --------------------------------------------------------------- softmax, epilogue
        const uint32_t q4 = warp & 3, fr = lane >> 2, fc = lane & 3;  // fragment row, column
        const uint32_t row0 = q4 * 16 + fr;       // this thread's rows: row0, row0 + 8
        const uint32_t lane_addr = (q4 * 32) << 16;
        const float qscale = a.scale * 1.4426950408889634f;
        // a wait that runs out marks the window it falls in (the window of step w ends at that
        // step's vote) and the thread carries on to the vote with values it discards
        bool ok_w = true;
        auto wait_one = [&](uint32_t bar, uint32_t parity, uint64_t w) {
            if (!mbar_wait(bar, parity)) {
                fail_s[w % 2] = 1;
                abort_flag = 1;
                report(a.d_status, HP_ERR_TIMEOUT);
                ok_w = false;
            }
        };
        uint64_t j = 0;
        bool stop = false;
        while (!stop && walk.next(g)) {
            // tokens each of the thread's rows sees (0 for rows that do not exist)
            uint64_t vis[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint64_t r = row0 + 8 * i, qi = (g.r0 + r) / a.H;
                vis[i] = r < g.rows && g.len + 1 + qi > g.n ? g.len + 1 + qi - g.n : 0;
            }
            float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
            for (uint64_t k = g.k0; k < g.k1; ++k, ++j) {
                wait_one(smem_u32(&s_full[j % 2]), (uint32_t)((j / 2) & 1), j);
                fence_after();
                uint32_t xr[32];
                tmem_issue_frag(tmem + lane_addr + kSCol + (uint32_t)(j % 2) * kTok, xr);
                tmem_wait<32>(xr);
                fence_before();
                mbar_arrive(smem_u32(&s_free[j % 2]));
                const uint64_t t0 = k * kTok;
                float x[32], mx[2] = {-INFINITY, -INFINITY};
                const int lim0 = vis[0] > t0 ? (int)umin(vis[0] - t0, kTok) : 0;
                const int lim1 = vis[1] > t0 ? (int)umin(vis[1] - t0, kTok) : 0;
#pragma unroll
                for (int i = 0; i < 8; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int col = 8 * i + 2 * (int)fc + (e & 1);
                        const float y = __uint_as_float(xr[4 * i + e]) * qscale;
                        x[4 * i + e] = col < (e < 2 ? lim0 : lim1) ? y : -INFINITY;
                        mx[e >> 1] = fmaxf(mx[e >> 1], x[4 * i + e]);
                    }
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 1));
                    mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], 2));
                }
                const bool need = named_or(3, kSoftmax, mx[0] > m[0] + kTau || mx[1] > m[1] + kTau);
                ok_w = true;
                if (*(volatile int*)&fail_s[j % 2]) {
                    stop = true;
                    break;
                }
                if (need) {  // the same in every softmax thread
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const float mn = fmaxf(m[i], mx[i]);
                        const float f = m[i] == -INFINITY ? 0.0f : exp2_approx(m[i] - mn);
                        if (fc == 0) corr_s[row0 + 8 * i] = f;
                        l[i] *= f;
                        m[i] = mn;
                    }
                    if (k > g.k0) {
                        // rescale O^T, complete up to step j - 1
                        wait_one(smem_u32(&o_done[(j - 1) % 2]), (uint32_t)(((j - 1) / 2) & 1), j + 1);
                        named_sync(1, kSoftmax);
                        fence_after();
#pragma unroll 1
                        for (uint32_t c = 0; c < 256; c += 32) {
                            uint32_t o[32];
                            tmem_issue<32>(tmem + lane_addr + kOCol + c, o);
                            tmem_wait<32>(o);
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                o[i] = __float_as_uint(__uint_as_float(o[i]) * corr_s[(c & 32) + i]);
                            tmem_st32(tmem + lane_addr + kOCol + c, o);
                        }
                        tmem_st_wait();
                        fence_before();
                        named_sync(1, kSoftmax);  // corr_s is free again
                    }
                }
                // weights: summed in fp32, rounded to the element type for the product
                unsigned char* stage = smem + kOffC + (uint32_t)(j % kStages) * kStage;
                unsigned char* pb = stage + kVChunks * kChunk;
                const float m0 = m[0] == -INFINITY ? 0.0f : m[0], m1 = m[1] == -INFINITY ? 0.0f : m[1];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float p0 = exp2_approx(x[4 * i] - m0), p1 = exp2_approx(x[4 * i + 1] - m0);
                    const float p2 = exp2_approx(x[4 * i + 2] - m1), p3 = exp2_approx(x[4 * i + 3] - m1);
                    l[0] += p0 + p1;
                    l[1] += p2 + p3;
                    const uint32_t c = 8 * i + 2 * fc;
                    *reinterpret_cast<uint32_t*>(pb + sw128_off(row0, c)) = pack2<T>(p0, p1);
                    *reinterpret_cast<uint32_t*>(pb + sw128_off(row0 + 8, c)) = pack2<T>(p2, p3);
                }
                // rows past the sequence become zeros before they meet their zero weights
                if (t0 + kTok > g.len) {
                    const uint32_t t = threadIdx.x - 64;
                    for (uint32_t r = (uint32_t)(g.len - t0) + (t >> 6); r < kTok; r += 2)
                        *reinterpret_cast<uint4*>(stage + ((t & 63) >> 3) * kChunk + r * 128 + (t & 7) * 16) =
                            make_uint4(0, 0, 0, 0);
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                mbar_arrive(smem_u32(&p_full[j % 2]));
            }
            if (stop) break;
            const bool any = g.k0 < g.k1;
            if (any) wait_one(smem_u32(&o_done[(j - 1) % 2]), (uint32_t)(((j - 1) / 2) & 1), j);
            if (!named_and(2, kSoftmax, ok_w)) break;
            fence_after();
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
                l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
            }
            const bool whole = g.ustart >= beg && g.ustart + g.steps <= end;
            const uint64_t rec0 = (2 * v + (g.ustart <= beg ? 0 : 1)) * a.group_rows + walk.tile * kRows;
            if (fc == 0)
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    inv_s[row0 + 8 * i] = whole ? (l[i] == 0.0f ? 0.0f : 1.0f / l[i]) : 1.0f;
                    if (!whole) a.part_ml[rec0 + row0 + 8 * i] = make_float2(m[i], l[i]);
                }
            named_sync(1, kSoftmax);
            // O^T: lane = dim of a 128-dim tile, column = row
            const uint32_t dim0 = q4 * 32 + lane;
#pragma unroll 1
            for (uint32_t c = 0; c < 256; c += 32) {
                uint32_t o[32];
                if (any) {
                    tmem_issue<32>(tmem + lane_addr + kOCol + c, o);
                    tmem_wait<32>(o);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = 0u;
                }
                const uint32_t dim = (c >> 6) * 128 + dim0, rb = c & 32;
#pragma unroll
                for (uint32_t i = 0; i < 32; ++i)
                    if (rb + i < g.rows) {
                        const float y = __uint_as_float(o[i]) * inv_s[rb + i];
                        if (whole) out[(g.q0 * a.H + g.r0 + rb + i) * kR + dim] = round1<T>(y);
                        else a.part_acc[(rec0 + rb + i) * kR + dim] = y;
                    }
            }
            fence_before();
            if (any) mbar_arrive(smem_u32(&o_free));
            named_sync(1, kSoftmax);  // inv_s is rewritten by the next segment
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == 1) tmem_free(tmem, kTmemCols);
}

template <typename T>
int launch_t(const LatentArgs& a, cudaStream_t st)
{
    CUtensorMap mc, mq;
    const uint32_t box = a.page_size < kTok ? (uint32_t)a.page_size : kTok;
    if (!map_2d(&mc, a.pool, a.num_pages * a.page_size, kW, kW * 2, box, a.bf16) ||
        !map_2d(&mq, a.q, a.total_q * a.H, kW, kW * 2, kRows, a.bf16))
        return HP_ERR_CUDA;
    int dev = 0;
    if (current_sms(&dev) == 0 || !allow_dynamic_smem<latent_tc_kernel<T>>(dev, (int)kSmem))
        return HP_ERR_CUDA;
    return launch_dependent(latent_tc_kernel<T>, (unsigned)(a.workers * (a.group_rows / kRows)), kThreads,
                            (size_t)kSmem, st, a, mc, mq) == cudaSuccess
               ? HP_OK
               : HP_ERR_CUDA;
}

}  // namespace

bool latent_tc_fits(uint32_t latent_dim, uint64_t head_dim, uint64_t page_size, uint64_t num_pages,
                    uint64_t q_rows)
{
    return latent_dim == kR && head_dim == kW &&
           (page_size == 8 || page_size == 16 || page_size == 32 || page_size % 64 == 0) &&
           num_pages > 0 && num_pages * page_size < (1ull << 31) && q_rows < (1ull << 31);
}

int launch_latent_tc(const LatentArgs& a, void* stream)
{
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return a.bf16 ? launch_t<__nv_bfloat16>(a, st) : launch_t<__half>(a, st);
}

}  // namespace hp
