// hp_prefix_tc.cu -- attention of many queries to one shared prefix on the tensor cores (tcgen05), for
// head_dim 64 and 128: the first half of hp_attention_prefix.
//
// All queries of a group see all of its prefix, so for a K/V head the group's (query, head) rows,
// G to a query, form one dense product with the prefix's keys: S = Q K^T, O = P V.  A tile is up to
// 256 rows, a step 128 keys of a tile; the steps of all tiles, in order (group, head, tile, keys), are
// cut evenly among one CTA per SM, so a CTA has parts of one or a few tiles.  Each part leaves a record, the
// row's maximum, sum and unnormalised O in fp32, which hp_attn_rows.cu merges with the sequences' own tokens.
//
// A part is worked on as two halves of 128 rows, one after the other on the tensor cores and
// beside each other in the softmax.  More than 128 rows: both halves take every block of keys.  Up
// to 128 rows: both halves hold the same rows, half 0 takes the part's even blocks and half 1 its
// odd ones (a record each), so that the chain load -> S -> softmax -> O of one half still overlaps the other's.
// Per half and block:
//   S [128 x 128] = Q . K^T    operands in shared memory
//   O [128 x D] += P . V       P (16-bit) in TMEM over S, V N-major
// Two threads own a row of S, 64 scores each in registers; the row's reference maximum moves only when
// some score exceeds it by more than 2^kTau (the half's 256 threads vote, which also says that P may
// overwrite S).  K and V come page by page: a box is 64 dims of one head of up to 128 slots of a
// page, 128-byte swizzled, a lane's each.  The queries are laid out by the softmax threads themselves, for any
// number of heads to a group.
//
// A step of two full halves takes 3,600 cycles where its products need 2,048: a half's chain S, vote,
// softmax, O is as long, and two of them overlap (250 sequences of 8 heads, 3 prefixes of 20,000 to 40,000 tokens,
// 64 query heads on 8 of 128 dims: 211 us, 1.04 PFLOP/s, a seventh of the rows padding).  The warps that have no
// rows run a loop of their own: with one loop for all, 50 of the scores' registers a step went through
// local memory (410 us).
//
// The weights are rounded to T once (f16, the sequences above: the result is 2.9e-4 of its size from 64 bits, 2.1e-4
// of it by its own rounding).  As two parts, as in hp_attn_rows.cu, their share goes, for half as many
// tensor products again and 130 instructions more a thread and step, all in the chain that bounds the kernel: the whole
// call takes 323 us in place of 273.  HP_ATTN_CUDA_CORES is the caller's way to the two parts.
//
// Keys past the prefix's end in its last block have a score of -inf and a weight of zero; V's rows
// there are zeroed in shared memory first (they are not loaded, or belong to other tokens).  Every
// wait is bounded (about 2 s) and reports HP_ERR_TIMEOUT; what is in flight is waited for (bounded)
// before TMEM and shared memory go.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "hp_attn_merge.cuh"
#include "hp_prefix.cuh"
#include "hp_resolve.cuh"
#include "hp_rows.cuh"
#include "hp_scan.cuh"
#include "hp_tcgen05.cuh"
#include "hp_tma.cuh"

namespace hp {
namespace {

using namespace tma;
using namespace tc;

constexpr uint32_t kSlot = 128 * 128;  // 128 rows x 64 dims
constexpr uint32_t kTmemCols = 512, kSCol = 0, kOCol = 256;  // S (and P) of half t at 128 t, O at 256 + 128 t
constexpr int kThreads = 18 * 32;  // warps 0-7 half 0, 8-15 half 1, 16 TMA, 17 products
constexpr int kHalf = 256;         // softmax threads of a half: two to a row
constexpr float kTau = 8.0f;

template <int D> struct Ring {
    static constexpr uint32_t kS = D / 64;           // slots of a K or V block
    static constexpr uint32_t kBufs = D == 128 ? 2 : 4;
    static constexpr uint32_t kOffKv = 2 * kS * kSlot;  // behind the queries of both halves
    static constexpr uint32_t kSmem = kOffKv + kBufs * 2 * kS * kSlot + 1024;
};

// A part of a tile: blocks j0 .. j1 - 1 of its keys.
struct Part {
    uint64_t table, q_row, record;  // prefix's first entry; first query row; record row of the part's row 0
    uint32_t prefix, head, rows;    // rows of the tile
    uint32_t j0, j1;
    bool split;                     // both halves hold the same rows
    __device__ uint32_t blocks(int t) const
    {
        const uint32_t n = j1 - j0;
        return split ? (n + 1 - t) / 2 : n;
    }
};

// The part that begins at step pos of a range that ends at `end`, by a whole warp.
__device__ __forceinline__ Part part_at(const PrefixTcArgs& a, uint64_t pos, uint64_t end)
{
    const uint64_t g = warp_last(a.num_groups, [&](uint64_t i) { return a.groups[i].step0 <= pos; });
    const PrefixGroup gr = a.groups[g];
    const uint64_t local = pos - gr.step0, unit = quotient(local, gr.blocks);
    const uint32_t h = (uint32_t)quotient(unit, gr.tiles), tile = (uint32_t)(unit - (uint64_t)h * gr.tiles);
    const uint32_t qt = kPrefixRows / a.G;
    const uint32_t left = gr.rows - tile * qt;
    Part p;
    p.table = gr.table;
    p.prefix = gr.prefix;
    p.head = h;
    p.q_row = gr.row0 + (uint64_t)tile * qt;
    p.rows = (left < qt ? left : qt) * a.G;
    p.split = p.rows <= 128;
    p.j0 = (uint32_t)(local - unit * gr.blocks);
    p.j1 = (uint32_t)umin(gr.blocks, p.j0 + (end - pos));
    p.record = gr.rows0 + (uint64_t)h * gr.records + (uint64_t)tile * qt * a.G + (uint64_t)blockIdx.x * kPrefixRows;
    return p;
}

// Half of row x of the part's tile to its place in the S product's operand: zeros past the tile's rows.
template <typename T, int D>
__device__ __forceinline__ void load_queries(const PrefixTcArgs& a, const Part& p, uint32_t x, uint32_t half,
                                             unsigned char* dst)
{
    const uint32_t qi = x / a.G;
    const uint4* q = reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) +
                                                    ((p.q_row + qi) * a.H * a.G + p.head * a.G + (x - qi * a.G)) * D) +
                     half * (D / 16);
    uint4 v[D / 16];
#pragma unroll
    for (uint32_t i = 0; i < D / 16; ++i) v[i] = x < p.rows ? q[i] : uint4{};
#pragma unroll
    for (uint32_t i = 0; i < D / 16; ++i) {
        const uint32_t piece = D == 128 ? i : half * (D / 16) + i;
        *reinterpret_cast<uint4*>(dst + (D == 128 ? half * kSlot : 0) + ((piece ^ (threadIdx.x & 7)) << 4)) = v[i];
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_kernel(const PrefixTcArgs a, const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv)
{
    using R = Ring<D>;
    constexpr uint32_t kS = R::kS, kBufs = R::kBufs;
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    __shared__ __align__(8) unsigned long long k_full[kBufs], v_full[kBufs], k_free[kBufs], v_free[kBufs], q_full[2],
        s_full[2], p_full[2], o_done[2], all_done;
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag, fail_s[2][2];
    __shared__ float half_s[2][128];  // what a row's two threads tell each other
    pdl_wait();
    if (!plan_holds(a.hdr, a.num_keys, a.d_status, a.first && blockIdx.x == 0, a.first == 2)) return;
    const uint64_t steps = a.hdr->steps, lw = (steps + a.workers - 1) / a.workers;
    const uint64_t beg = umin(blockIdx.x * lw, steps), end = umin(beg + lw, steps);
    if (beg >= end) return;
    const unsigned warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t sm0 = (smem_u32(smem_raw) + 1023u) & ~1023u;
    unsigned char* const smem = smem_raw + (sm0 - smem_u32(smem_raw));
    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < kBufs; ++i) {
            mbar_init(smem_u32(&k_full[i]), 1);
            mbar_init(smem_u32(&v_full[i]), 1);
            mbar_init(smem_u32(&k_free[i]), 1);
            mbar_init(smem_u32(&v_free[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&q_full[i]), kHalf);
            mbar_init(smem_u32(&s_full[i]), 1);
            mbar_init(smem_u32(&p_full[i]), kHalf);
            mbar_init(smem_u32(&o_done[i]), 1);
            fail_s[i][0] = fail_s[i][1] = 0;
        }
        mbar_init(smem_u32(&all_done), 1);
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 17) tmem_alloc(smem_u32(&tmem_base), kTmemCols);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_base;
    // true unless the wait ran out or another role stopped; `warp_wait` for whole warps, whose
    // lanes then agree
    auto wait_for = [&](unsigned long long* bar, uint32_t parity) {
        if (mbar_wait_or(smem_u32(bar), parity, &abort_flag)) return true;
        abort_flag = 1;
        report(a.d_status, HP_ERR_TIMEOUT);
        return false;
    };
    auto warp_wait = [&](unsigned long long* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, wait_for(bar, parity)) != 0;
    };

    if (warp == 16) {
        // a lane's box: `sub` of the block's runs of a.box slots, 64 dims of the head
        const uint32_t nsub = 128 / a.box, sub = lane & (nsub - 1), half = lane / nsub;
        uint32_t n = 0, vn = 0;  // blocks whose K, whose V barrier has been armed
        bool stop = false;
        for (uint64_t pos = beg; pos < end && !stop;) {
            const Part p = part_at(a, pos, end);
            for (uint32_t j = p.j0; j < p.j1; ++j) {
                const uint32_t b = n % kBufs, t0 = j * 128 + sub * a.box;
                const bool live = half < kS && t0 < p.prefix;
                int row = 0;
                if (live) {
                    const uint32_t e = t0 / a.P;
                    row = (int)(index_at(a.table, a.idx64, p.table + e) * a.P + (t0 - e * a.P));
                }
                const uint32_t bytes = __popc(__ballot_sync(0xffffffffu, live)) * a.box * 128;
                const uint32_t dst = sm0 + R::kOffKv + (2 * b * kS + half) * kSlot + sub * a.box * 128;
                if (n >= kBufs && !warp_wait(&k_free[b], (n / kBufs - 1) & 1)) {
                    stop = true;
                    break;
                }
                if (lane == 0) mbar_expect_tx(smem_u32(&k_full[b]), bytes);
                __syncwarp();
                if (live && !(a.test_stall && n == 0)) tma_3d(dst, &tmk, (int)(half * 64), (int)p.head, row, smem_u32(&k_full[b]));
                __syncwarp();
                ++n;
                if (vn >= kBufs && !warp_wait(&v_free[b], (vn / kBufs - 1) & 1)) {
                    stop = true;
                    break;
                }
                ++vn;
                if (lane == 0) mbar_expect_tx(smem_u32(&v_full[b]), bytes);
                __syncwarp();
                if (live) tma_3d(dst + kS * kSlot, &tmv, (int)(half * 64), (int)p.head, row, smem_u32(&v_full[b]));
                __syncwarp();
            }
            pos += p.j1 - p.j0;
        }
        // the last loads land before the shared memory goes
        for (uint32_t x = n > kBufs ? n - kBufs : 0; x < n; ++x) mbar_wait(smem_u32(&k_full[x % kBufs]), (x / kBufs) & 1);
        for (uint32_t x = vn > kBufs ? vn - kBufs : 0; x < vn; ++x) mbar_wait(smem_u32(&v_full[x % kBufs]), (x / kBufs) & 1);
        __syncwarp();
    } else if (warp == 17) {
        const uint32_t id_s = f16_idesc(a.bf16 != 0, false, false, 128, 128);
        const uint32_t id_o = f16_idesc(a.bf16 != 0, false, true, 128, D);
        const uint64_t qd0 = sw128_desc(sm0, 16, 1024), kd0 = sw128_desc(sm0 + R::kOffKv, 16, 1024);
        const uint64_t vd0 = sw128_desc(sm0 + R::kOffKv + kS * kSlot, kSlot, 1024);
        bool ok = true;
        uint32_t n0 = 0, np = 0, c[2] = {0, 0};  // blocks before the part, parts, S issued for each half
        // S of half t for block n; K goes back behind it if `last`
        auto issue_s = [&](int t, uint32_t n, bool last) {
            const uint32_t b = n % kBufs;
            fence_after();
            const uint64_t qd = qd0 + ((t * kS * kSlot) >> 4), kd = kd0 + ((2 * b * kS * kSlot) >> 4);
            if (elect_one()) {
#pragma unroll
                for (uint32_t s = 0; s < kS; ++s)
#pragma unroll
                    for (uint32_t kk = 0; kk < 4; ++kk)
                        mma_f16(tmem + kSCol + t * 128, qd + (s * kSlot >> 4) + kk * 2, kd + (s * kSlot >> 4) + kk * 2, id_s, s | kk);
                mma_commit(smem_u32(&s_full[t]));
                if (last) mma_commit(smem_u32(&k_free[b]));
            }
            __syncwarp();
            ++c[t];
        };
        // O of half t for block n, the half's first of the part or not, its last or not; V goes back
        // behind it if `last`
        auto issue_o = [&](int t, uint32_t n, bool first, bool done, bool last) {
            const uint32_t b = n % kBufs;
            fence_after();
            const uint64_t vd = vd0 + ((2 * b * kS * kSlot) >> 4);
            if (elect_one()) {
#pragma unroll
                for (uint32_t kk = 0; kk < 8; ++kk)
                    mma_f16_ts(tmem + kOCol + t * 128, tmem + kSCol + t * 128 + kk * 8, vd + ((kk * 2048) >> 4), id_o,
                               first ? kk : 1u);
                if (done) mma_commit(smem_u32(&o_done[t]));
                if (last) mma_commit(smem_u32(&v_free[b]));
            }
            __syncwarp();
        };
        // What a round begins with: V of block n - back and P of half t (`has_o`), K of block n
        // (`has_s`).  A wait costs some 200 cycles even when its phase is complete, so the three are
        // polled together; K is waited for behind the O products.
        auto round = [&](int t, uint32_t n, uint32_t back, bool has_o, bool has_s, auto&& o, auto&& s) {
            const uint32_t nv = n - back;
            bool v_ok = !has_o, p_ok = !has_o, k_ok = !has_s;
            if (has_o) v_ok = mbar_try_wait(smem_u32(&v_full[nv % kBufs]), (nv / kBufs) & 1);
            if (has_s) k_ok = mbar_test(smem_u32(&k_full[n % kBufs]), (n / kBufs) & 1);
            if (has_o) p_ok = mbar_try_wait(smem_u32(&p_full[t]), (c[t] - 1) & 1);
            const unsigned polls = __reduce_and_sync(0xffffffffu, (v_ok ? 1u : 0u) | (k_ok ? 2u : 0u) | (p_ok ? 4u : 0u));
            if (!(polls & 1)) ok = warp_wait(&v_full[nv % kBufs], (nv / kBufs) & 1);
            if (ok && !(polls & 4)) ok = warp_wait(&p_full[t], (c[t] - 1) & 1);
            if (!ok) return;
            if (has_o) o();
            if (!(polls & 2)) ok = warp_wait(&k_full[n % kBufs], (n / kBufs) & 1);
            if (ok && has_s) s();
        };
        for (uint64_t pos = beg; pos < end && ok; ++np) {
            const Part p = part_at(a, pos, end);
            const uint32_t blocks = p.j1 - p.j0;
            for (int t = 0; t < 2; ++t)
                if (ok) ok = warp_wait(&q_full[t], np & 1);
            if (p.split) {
                for (uint32_t i = 0; i < blocks + 2 && ok; ++i) {
                    const int t = i & 1;
                    round(t, n0 + i, 2, i >= 2 && i - 2 < blocks, i < blocks,
                          [&] { issue_o(t, n0 + i - 2, i < 4, i >= blocks, true); }, [&] { issue_s(t, n0 + i, true); });
                }
            } else {
                for (uint32_t i = 0; i <= blocks && ok; ++i) {
                    const bool has_o = i > 0, has_s = i < blocks;
                    round(0, n0 + i, 1, has_o, has_s, [&] { issue_o(0, n0 + i - 1, i == 1, i == blocks, false); },
                          [&] { issue_s(0, n0 + i, false); });
                    if (ok && has_o) ok = warp_wait(&p_full[1], (c[1] - 1) & 1);
                    if (ok && has_o) issue_o(1, n0 + i - 1, i == 1, i == blocks, true);
                    if (ok && has_s) issue_s(1, n0 + i, true);
                }
            }
            n0 += blocks;
            pos += blocks;
        }
        // everything issued has completed before the TMEM goes: one more commit covers it
        if (elect_one()) mma_commit(smem_u32(&all_done));
        __syncwarp();
        mbar_wait(smem_u32(&all_done), 0);
    } else {
        const int t = warp >> 3;
        const uint32_t q4 = warp & 3, half = (warp >> 2) & 1, row = q4 * 32 + lane;
        const uint32_t sa = tmem + ((q4 * 32) << 16) + kSCol + t * 128 + 64 * half;
        const uint32_t oa = tmem + ((q4 * 32) << 16) + kOCol + t * 128 + half * (D / 2);
        float* const told = &half_s[t][row];  // the second one's value, then what the first made of it
        const float qscale = a.scale * 1.4426950408889634f;
        uint32_t c = 0, n0 = 0, done = 0;  // S taken, blocks before the part, parts with blocks for this half
        bool stop = false;
        // V past the prefix's end, `left` keys into block b of the part (the products of half 0 come
        // first where both take the block)
        auto clear_v = [&](uint32_t left, uint32_t n) {
            const uint32_t b = n % kBufs, r = threadIdx.x & 127, s = (threadIdx.x >> 7) & 1;
            if (warp_wait(&v_full[b], (n / kBufs) & 1) && r >= left && s < kS) {
                uint4* v = reinterpret_cast<uint4*>(smem + R::kOffKv + ((2 * b + 1) * kS + s) * kSlot + r * 128);
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = uint4{};
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            }
        };
        for (uint64_t pos = beg; pos < end && !stop;) {
            uint32_t blocks, stride, first, left;  // this half's blocks: first, first + stride, ... of the part's
            bool any, clears;                      // some row of the warp; this half clears V
            float m, l = 0.0f;
            {
                const Part p = part_at(a, pos, end);
                const uint32_t x = p.split ? row : 128 * t + row;  // row of the tile
                blocks = p.blocks(t);
                m = blocks ? kLowest : -INFINITY;  // (each of its blocks has a key)
                stride = p.split ? 2 : 1;
                first = p.split ? t : 0;
                left = p.prefix - (p.j0 + first) * 128;
                any = (x & ~31u) < p.rows;
                clears = p.split || t == 0;
                load_queries<T, D>(a, p, x, half, smem + t * kS * kSlot + row * 128);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                mbar_arrive(smem_u32(&q_full[t]));
            }
            if (!any) {  // 32 rows that nobody asked for: the warp votes and arrives, no more
                for (uint32_t i = 0; i < blocks; ++i, ++c, left -= 128 * stride) {
                    if (!warp_wait(&s_full[t], c & 1)) fail_s[t][c & 1] = 1;
                    const bool need = named_or(1 + t, kHalf, false);
                    if (*(volatile int*)&fail_s[t][c & 1]) {
                        stop = true;
                        break;
                    }
                    if (need) named_sync(1 + t, kHalf);
                    if (left < 128 && clears) clear_v(left, n0 + first + i * stride);
                    mbar_arrive(smem_u32(&p_full[t]));
                }
            } else {
                for (uint32_t i = 0; i < blocks; ++i, ++c, left -= 128 * stride) {  // left: keys from the block's first on
                    // a wait that runs out marks its block; the half's threads stop together, at the vote
                    if (!warp_wait(&s_full[t], c & 1)) fail_s[t][c & 1] = 1;
                    fence_after();
                    uint32_t xr[2][32];
                    tmem_issue<32>(sa, xr[0]);
                    tmem_issue<32>(sa + 32, xr[1]);
                    tmem_wait<32>(xr[0]);
                    tmem_wait<32>(xr[1]);
                    // the largest scaled score: the extreme of the raw ones on the scale's side; in the
                    // block in which the prefix ends, scaled scores with -inf past it
                    const int lim = left > 64 * half ? (int)(left - 64 * half) : 0;
                    float mx = -INFINITY, qs = qscale;
                    if (lim < 64) qs = 1.0f;
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float* s = reinterpret_cast<float*>(xr[h]);
                        if (lim < 64) {
#pragma unroll
                            for (int k = 0; k < 32; ++k) {
                                s[k] = 32 * h + k < lim ? s[k] * qscale : -INFINITY;
                                mx = fmaxf(mx, s[k]);
                            }
                        } else if (qscale >= 0.0f) {
                            float e0 = s[0], e1 = s[1];
#pragma unroll
                            for (int k = 2; k < 30; k += 4) {
                                e0 = max3(e0, s[k], s[k + 1]);
                                e1 = max3(e1, s[k + 2], s[k + 3]);
                            }
                            mx = fmaxf(mx, fmaxf(max3(e0, s[30], s[31]), e1) * qscale);
                        } else {
                            float e0 = s[0], e1 = s[1];
#pragma unroll
                            for (int k = 2; k < 30; k += 4) {
                                e0 = min3(e0, s[k], s[k + 1]);
                                e1 = min3(e1, s[k + 2], s[k + 3]);
                            }
                            mx = fmaxf(mx, fminf(min3(e0, s[30], s[31]), e1) * qscale);
                        }
                    }
                    // (past this barrier every thread of the half has its scores, and P may overwrite them)
                    if (half) *told = mx;
                    fence_before();
                    const bool need = named_or(1 + t, kHalf, mx > m + kTau);
                    fence_after();
                    if (*(volatile int*)&fail_s[t][c & 1]) {
                        stop = true;
                        break;
                    }
                    if (need) {  // the same in the whole half
                        float mn;
                        if (!half) *told = mn = fmaxf(m, fmaxf(mx, *told));
                        named_sync(1 + t, kHalf);
                        if (half) mn = *told;
                        const float f = exp2_approx(m - mn);
                        m = mn;
                        l *= f;
                        if (i > 0) {  // the scores of this block are complete, so O of the last one is
#pragma unroll 1
                            for (uint32_t k = 0; k < D / 2; k += 16) {
                                uint32_t o[16];
                                tmem_issue<16>(oa + k, o);
                                tmem_wait<16>(o);
#pragma unroll
                                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                tmem_st16(oa + k, o);
                            }
                        }
                    }
                    const float base = kWeightLift<T> - m;
                    const uint64_t qs2 = pair_of(qs, qs), base2 = pair_of(base, base);
                    uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t w16[16];
                        const float* s = reinterpret_cast<const float*>(xr[h]);
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            float2 w = of_pair(fma2(pair_of(s[2 * k], s[2 * k + 1]), qs2, base2));
                            w.x = exp2_approx(w.x);
                            w.y = exp2_approx(w.y);
                            sum[k & 1] = add2(sum[k & 1], pair_of(w.x, w.y));
                            w16[k] = pack2<T>(w.x, w.y);
                        }
                        tmem_st16(sa - 32 * half + 16 * h, w16);
                    }
                    const float2 sums = of_pair(add2(sum[0], sum[1]));
                    l += sums.x + sums.y;
                    tmem_st_wait();
                    fence_before();
                    if (left < 128 && clears) clear_v(left, n0 + first + i * stride);
                    mbar_arrive(smem_u32(&p_full[t]));
                }
            }
            const Part p = part_at(a, pos, end);
            if (!stop && blocks) {
                const bool ok = warp_wait(&o_done[t], done & 1);
                ++done;
                if (half) *told = l;
                stop = !named_and(1 + t, kHalf, ok);
                fence_after();
                if (!half) l += *told;
            }
            if (!stop && any) {
                const uint32_t x = p.split ? row : 128 * t + row;
                const bool real = x < p.rows;
                const uint64_t rec = p.record + (p.split && t ? p.rows + x : x);
                if (real && !half) a.rec.ml[rec] = make_float2(m, l);
                if (blocks) {
                    float4* o4 = reinterpret_cast<float4*>(a.rec.acc + rec * D + half * (D / 2));
#pragma unroll 1
                    for (uint32_t k = 0; k < D / 2; k += 32) {
                        uint32_t o[32];
                        tmem_issue<32>(oa + k, o);
                        tmem_wait<32>(o);
                        if (real)
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                o4[k / 4 + e] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                                            __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
                    }
                    fence_before();
                }
            }
            n0 += p.j1 - p.j0;
            pos += p.j1 - p.j0;
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == 17) tmem_free(tmem, kTmemCols);
}

// A pool as boxes of 64 dims of one head of `box` slots.
bool pool_map(CUtensorMap* m, const void* pool, const PrefixTcArgs& a, uint32_t D)
{
    EncodeFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {D, a.H, a.num_pages * a.P};
    const cuuint64_t strides[2] = {D * 2ull, (uint64_t)a.H * D * 2};
    const cuuint32_t box[3] = {64, 1, a.box};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, a.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, const_cast<void*>(pool),
              dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int D>
int launch_d(const PrefixTcArgs& a, cudaStream_t st)
{
    CUtensorMap mk, mv;
    if (!pool_map(&mk, a.k_pool, a, D) || !pool_map(&mv, a.v_pool, a, D)) return HP_ERR_CUDA;
    int dev = 0;
    if (current_sms(&dev) == 0 || !allow_dynamic_smem<prefix_kernel<T, D>>(dev, (int)Ring<D>::kSmem)) return HP_ERR_CUDA;
    return launch_dependent(prefix_kernel<T, D>, (unsigned)a.workers, kThreads, (size_t)Ring<D>::kSmem, st, a, mk, mv) ==
                   cudaSuccess
               ? HP_OK
               : HP_ERR_CUDA;
}

}  // namespace

bool prefix_tc_shape(uint64_t head_dim, uint64_t page_size)
{
    return (head_dim == 64 || head_dim == 128) && page_size % 8 == 0;
}

bool prefix_tc_fits(uint64_t head_dim, uint64_t page_size, uint64_t num_pages)
{
    return prefix_tc_shape(head_dim, page_size) && num_pages > 0 && num_pages * page_size < (1ull << 31);
}

uint32_t prefix_tc_box(uint64_t page_size)
{
    uint32_t box = 8;
    while (box < 128 && page_size % (2 * box) == 0) box *= 2;
    return box;
}

int launch_prefix_tc(const PrefixTcArgs& a, uint32_t head_dim, void* stream)
{
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (a.bf16) return head_dim == 64 ? launch_d<__nv_bfloat16, 64>(a, st) : launch_d<__nv_bfloat16, 128>(a, st);
    return head_dim == 64 ? launch_d<__half, 64>(a, st) : launch_d<__half, 128>(a, st);
}

}  // namespace hp
