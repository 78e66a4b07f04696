// hp_latent_tc.cu -- attention over a paged cache of shared latent rows on the tensor cores
// (tcgen05): latent_dim 512, rope_dim 64, absorbed form.
//
// A CTA takes a tile of 64 (query, head) rows of one sequence and a range of its steps of 64
// tokens (hp_latent.cuh has the split).  Per step, with C the step's 64 cache rows of 576:
//   S [64 rows x 64 tokens]     = Q . C^T            36 products of 16 dims, M = N = 64
//   O^T [512 dims x 64 rows]   += C[:, :512]^T . P^T  4 tiles of 128 dims, 4 products each
// so the step's rows are loaded once and serve as the B operand of S (K-major) and the A operand of
// O^T (M-major).  O^T rather than O: 64 rows of 512 fp32 sums are half of TMEM either way, but M =
// 128 products run at the full rate where M = 64 runs at half of it (34 cycles for M = N = 64, 50
// for M = 128, N = 64, which its shared-memory reads set: 2,024 a step).  O^T stays in TMEM over
// the whole range: a row's reference maximum moves (and its column of O^T is rescaled) only when
// a score exceeds it by more than 2^kTau.
//
// A TMA box is 8 tokens: [9 chunks of 64 dims][8 rows][128 bytes], 128-byte swizzled, 9 KiB, so
// that eight rows are one swizzle atom for every chunk and the operands' 8-row groups lie 9 KiB
// apart whatever the page size (a multiple of 8).  Eight boxes a step: issuing a box takes the
// loader about 100 cycles, and boxes of one chunk (36 a step on 16-slot pages) held it to 4,400
// a step.  Slots of four boxes go back to the loader as the products of their 32 tokens end.
//
// A step takes 3,150 cycles: two in flight, each the chain slots free -> loaded 1,400 -> S and the
// other step's O^T side by side 2,000 -> softmax 1,300 -> O^T 1,500.  The next step's rows are
// prefetched into L2 while this one waits for its slots (decode of 64 x 128 heads 119 -> 115 us,
// 16 long sequences 319 -> 308 us: 5.9 TB/s).  Putting O^T(j) before the rest of S(j + 1), by polls
// or at a fixed place, gained nothing (117 to 120 us): S then ends later by as much.
//
// Shared memory: Q 72 KiB, two steps of C 144 KiB, P (weights rounded to the element type)
// 8 KiB.  TMEM: O^T 256 columns, S 2 x 64.  Roles: warp 0 loads C, warp 7 the queries, warp 1
// issues S, warp 6 O^T (apart, so that neither waits for the other's operands), warps 2-5 do
// the softmax and the epilogue.
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
#include "hp_latent_plan.cuh"
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
constexpr uint32_t kChunks = kW / 64;
constexpr uint32_t kChunk = 64 * 128;          // 64 rows x 64 dims
constexpr uint32_t kGroup = kChunks * 1024;    // 8 tokens
constexpr uint32_t kSlots = 4;                 // of four groups each: two steps
constexpr uint32_t kOffC = kChunks * kChunk;   // Q first, then the slots, then P
constexpr uint32_t kOffP = kOffC + kSlots * 4 * kGroup;
constexpr uint32_t kSmem = kOffP + kRows * 128 + 1024;
constexpr uint32_t kOCol = 0, kSCol = 256;     // TMEM columns
constexpr uint32_t kTmemCols = 512;
constexpr int kThreads = 8 * 32;
constexpr int kSoftmax = 128;
constexpr float kTau = 8.0f;

// A segment: steps k0 .. k1 - 1 of one tile, without those in which none of its rows sees a
// token (k0 >= k1: nothing to compute).
struct Segment {
    uint64_t s, len, q0, n, r0, k0, k1, ustart, steps;
    uint64_t seen;  // tokens that the tile's last row sees, the most of its rows
    uint32_t rows;  // rows of the tile that exist, at least 1
};

// The segments of a worker's range in order; every role walks them, whole warps at a time.  The
// first search takes 32 sums at a time, the rest go forward, and a segment's facts are loaded
// together: three trips to memory to the first segment, one or two to each next.
struct Walk {
    const LatentArgs& a;
    const uint32_t* small;  // the CTA's own sums, or NULL
    uint64_t pos, end;
    uint32_t tile;  // this CTA's tile within the group
    uint64_t s, first, past;  // the current sequence and its units
    __device__ uint64_t units(uint64_t i) const { return small ? small[i] : a.units_off[i]; }
    __device__ Walk(const LatentArgs& args, const uint32_t* sums, uint64_t beg, uint64_t e, uint32_t t, unsigned lane)
        : a(args), small(sums), pos(beg), end(e), tile(t)
    {
        uint64_t lo = 0, hi = a.num_seqs;
        while (hi - lo > 1) {  // the last sequence whose units start at or before beg
            const uint64_t step = (hi - lo + 31) / 32, i = lo + lane * step;
            const unsigned below = __ballot_sync(0xffffffffu, i < hi && units(i) <= beg);
            lo += (uint64_t)(31 - __clz(below)) * step;
            hi = umin(hi, lo + step);
        }
        s = lo;
        first = units(s);
        past = units(s + 1);
    }
    __device__ bool next(Segment& g)
    {
        while (pos < end) {
            while (pos >= past) {  // sequences without units are passed over
                if (++s >= a.num_seqs) return false;  // (not with a plan of this batch)
                first = past;
                past = units(s + 1);
            }
            g.s = s;
            g.len = index_at(a.lens, a.idx64, s);
            g.q0 = a.q_ptr ? index_at(a.q_ptr, a.idx64, s) : s;
            g.n = (a.q_ptr ? index_at(a.q_ptr, a.idx64, s + 1) : s + 1) - g.q0;
            g.steps = (g.len + kTok - 1) / kTok;
            if (g.steps == 0) return false;  // (nor this)
            const uint64_t off = pos - first;
            // (the usual group is the sequence's only one)
            const uint64_t grp = off < g.steps ? 0 : off / g.steps;
            g.ustart = first + grp * g.steps;
            g.k0 = off - grp * g.steps;
            g.k1 = umin(g.steps, g.k0 + (end - pos));
            pos += g.k1 - g.k0;
            g.r0 = grp * a.group_rows + tile * kRows;
            const uint64_t all = g.n * a.H;
            if (g.r0 >= all) continue;  // the group's last tile may have no rows
            g.rows = (uint32_t)umin(kRows, all - g.r0);
            const uint64_t last = (uint32_t)(g.r0 + g.rows - 1) / a.H;  // the tile's last query sees most
            g.seen = g.len + 1 + last > g.n ? g.len + 1 + last - g.n : 0;
            g.k1 = umin(g.k1, (g.seen + kTok - 1) / kTok);
            return true;
        }
        return false;
    }
};

// Page of a sequence's group of 8 tokens.
__device__ __forceinline__ uint64_t div_groups(const LatentArgs& a, uint64_t group)
{
    return group < (1ull << 32) ? div_invariant((uint32_t)group, a.g_m, a.g_l) : group / (a.page_size / 8);
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1)
    latent_tc_kernel(const LatentArgs a, const __grid_constant__ CUtensorMap tmc,
                     const __grid_constant__ CUtensorMap tmq)
{
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    __shared__ __align__(8) unsigned long long c_full[2], c_free[kSlots], s_full[2], s_free[2], p_full[2], o_done[2], o_free, q_full, q_free, s_end, o_end;
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag, fail_s[2];
    __shared__ float corr_s[kRows], inv_s[kRows];
    __shared__ uint32_t units_s[kSmallSeqs + 1];

    const unsigned warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    T* out = static_cast<T*>(a.out);
    // what does not depend on the plan, while the plan runs
    const uint32_t sm0 = (smem_u32(smem_raw) + 1023u) & ~1023u;
    unsigned char* smem = smem_raw + (sm0 - smem_u32(smem_raw));
    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < kSlots; ++i) mbar_init(smem_u32(&c_free[i]), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&c_full[i]), 2);  // a step's two slots
            mbar_init(smem_u32(&s_full[i]), 1);
            mbar_init(smem_u32(&s_free[i]), kSoftmax);
            mbar_init(smem_u32(&p_full[i]), kSoftmax);
            mbar_init(smem_u32(&o_done[i]), 1);
        }
        mbar_init(smem_u32(&o_free), kSoftmax);
        mbar_init(smem_u32(&q_full), 1);
        mbar_init(smem_u32(&q_free), 1);
        mbar_init(smem_u32(&s_end), 1);
        mbar_init(smem_u32(&o_end), 1);
        abort_flag = 0;
        fail_s[0] = fail_s[1] = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (threadIdx.x == 64) {
        prefetch_map(&tmc);
        prefetch_map(&tmq);
    }
    if (warp == 1) tmem_alloc(smem_u32(&tmem_base), kTmemCols);
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_base;
    pdl_wait();
    bool planned;
    uint64_t total;
    if (a.small) {
        const SmallPlan sp = small_plan(a.plan, a.idx64, units_s, nullptr);
        if (blockIdx.x == 0) {  // (whole, as a planned call may follow)
            if (threadIdx.x == 0) store_plan(a.plan, sp);
            if (threadIdx.x <= a.num_seqs) a.plan.ws.units_off[threadIdx.x] = units_s[threadIdx.x];
        }
        planned = sp.key == kVerdictOk;
        total = planned ? sp.units : 0;
    } else {
        planned = a.hdr->verdict == kVerdictOk;
        total = planned ? a.hdr->total_units : 0;
    }
    auto units = [&](uint64_t s) { return a.small ? (uint64_t)units_s[s] : (uint64_t)a.units_off[s]; };
    // queries of sequences without tokens: zeros, 32 sequences to a warp at a time
    auto zero_empty = [&](uint64_t w, uint64_t warps) {
        for (uint64_t k = w;; k += warps) {  // the CTA's k-th 32 sequences, whichever warps share them
            const uint64_t s0 = (blockIdx.x + k * gridDim.x) * 32, s = s0 + lane;
            if (s0 >= a.num_seqs) break;
            unsigned empty = __ballot_sync(0xffffffffu, s < a.num_seqs && units(s) == units(s + 1));
            for (; empty; empty &= empty - 1) {
                const uint64_t e = s0 + __ffs(empty) - 1;
                const uint64_t q0 = a.q_ptr ? index_at(a.q_ptr, a.idx64, e) : e;
                const uint64_t q1 = a.q_ptr ? index_at(a.q_ptr, a.idx64, e + 1) : e + 1;
                uint4* o = reinterpret_cast<uint4*>(out);
                for (uint64_t i = q0 * a.H * (kR / 8) + lane; i < q1 * a.H * (kR / 8); i += 32)
                    o[i] = make_uint4(0, 0, 0, 0);
            }
        }
    };
    const uint32_t tiles = a.group_rows / kRows;
    const uint64_t Lw = (total + a.workers - 1) / a.workers;
    const uint64_t v = blockIdx.x / tiles, beg = umin(v * Lw, total), end = umin(beg + Lw, total);
    if (planned && threadIdx.x == 96 && blockIdx.x % tiles == 0) write_merge(a, v, total, units);  // (a softmax thread, idle yet)
    if (beg >= end) {  // the whole CTA
        if (planned) zero_empty(warp, 8);
        if (warp == 1) tmem_free(tmem, kTmemCols);
        return;
    }

    Walk walk(a, a.small ? units_s : nullptr, beg, end, (uint32_t)(blockIdx.x % tiles), lane);
    Segment g;
    // true unless the wait ran out or another role stopped; warp_wait for whole warps
    auto wait_for = [&](unsigned long long* bar, uint32_t parity) {
        if (mbar_wait_or(smem_u32(bar), parity, &abort_flag)) return true;
        abort_flag = 1;
        report(a.d_status, HP_ERR_TIMEOUT);
        return false;
    };
    auto warp_wait = [&](unsigned long long* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, wait_for(bar, parity)) != 0;
    };

    if (warp == 0) {
        // ----------------------------------------------------------- cache rows of each step
        const uint32_t P = (uint32_t)a.page_size;
        uint64_t j = 0, armed = 0;  // steps, slots given to loads
        bool ok = true;
        while (ok && walk.next(g)) {
            const uint64_t tab0 = index_at(a.seq_ptr, a.idx64, g.s);
            // The slice's entries 64 at a time, two per lane, the next 32 on their way before they
            // are needed: a lookup is a shuffle (a load per step cost 1,500 cycles of it).
            const uint64_t npages = g.len ? div_groups(a, (g.len - 1) / 8) + 1 : 0;
            auto entries = [&](uint64_t i) {
                return i + lane < npages ? index_at(a.table, a.idx64, tab0 + i + lane) : 0ull;
            };
            uint64_t base = div_groups(a, g.k0 * 8);
            unsigned long long cur = entries(base), nxt = entries(base + 32);
            // lane i: the pool row of step k's i-th (mod 8) group of 8 tokens
            auto row_of = [&](uint64_t k) {
                const uint64_t gi = k * 8 + (lane & 7), page = div_groups(a, gi);
                const uint32_t rel = (uint32_t)(page - base);  // below 64: two steps span 16 pages at most
                const unsigned long long e0 = __shfl_sync(0xffffffffu, cur, (int)(rel & 31));
                const unsigned long long e1 = __shfl_sync(0xffffffffu, nxt, (int)(rel & 31));
                return (int)((rel < 32 ? e0 : e1) * P + (gi * 8 - page * P));
            };
            auto groups_of = [&](uint64_t k) { return (uint32_t)umin(8, (g.len - k * kTok + 7) / 8); };  // with a token
            for (uint64_t k = g.k0; ok && k < g.k1; ++k, ++j) {
                if (div_groups(a, k * 8) >= base + 32) {
                    base += 32;
                    cur = nxt;
                    nxt = entries(base + 32);
                }
                const int row = row_of(k);
                const uint32_t live = groups_of(k);
                // the next step's rows start for the L2 while this one waits for its slots, a pair's
                // CTAs half of them each
                if (k + 1 < g.k1) {
                    const int ahead = row_of(k + 1);
                    if (lane < 8 && lane < groups_of(k + 1) && lane % tiles == walk.tile) prefetch_3d(&tmc, 0, ahead, 0);
                    __syncwarp();
                }
                for (uint32_t p = 0; p < 2; ++p) {
                    const uint64_t c = 2 * j + p;
                    const uint32_t sl = (uint32_t)(c % kSlots), n = live > 4 * p ? (uint32_t)umin(4, live - 4 * p) : 0;
                    if (c >= kSlots) ok = warp_wait(&c_free[sl], (uint32_t)((c / kSlots - 1) & 1));
                    if (!ok) break;
                    const uint32_t bar = smem_u32(&c_full[j % 2]);
                    if (lane == 0) mbar_expect_tx(bar, n * kGroup);
                    armed = c + 1;
                    __syncwarp();
                    if (lane >> 2 == p && (lane & 3) < n && !(a.test_stall && c == 0))
                        tma_3d(sm0 + kOffC + (sl * 4 + (lane & 3)) * kGroup, &tmc, 0, row, 0, bar);
                }
            }
        }
        // the last loads land before the shared memory goes (a step that a wait cut short arrives for
        // its missing slot here, so that its barrier's phase can end)
        for (; armed % 2; ++armed)
            if (lane == 0) mbar_arrive(smem_u32(&c_full[armed / 2 % 2]));
        __syncwarp();
        for (uint64_t x = armed / 2 > 2 ? armed / 2 - 2 : 0; x < armed / 2; ++x)
            mbar_wait(smem_u32(&c_full[x % 2]), (uint32_t)((x / 2) & 1));
        __syncwarp();
    } else if (warp == 7) {
        // ------------------------------------------------------------- queries of each tile
        uint64_t seg = 0;
        while (walk.next(g)) {
            if (g.k0 >= g.k1) continue;
            if (seg && !warp_wait(&q_free, (uint32_t)((seg - 1) & 1))) break;
            if (lane == 0) mbar_expect_tx(smem_u32(&q_full), kChunks * kChunk);
            __syncwarp();
            if (lane < kChunks)
                tma_2d(sm0 + lane * kChunk, &tmq, (int)(lane * 64), (int)(g.q0 * a.H + g.r0), smem_u32(&q_full));
            ++seg;
        }
        zero_empty(0, 1);
        if (seg) mbar_wait(smem_u32(&q_full), (uint32_t)((seg - 1) & 1));
        __syncwarp();
    } else if (warp == 1) {
        // -------------------------------------------------------------------- S = Q . C^T
        const uint32_t id_s = f16_idesc(a.bf16 != 0, false, false, kRows, kTok);
        const uint64_t qd = sw128_desc(sm0, 16, 1024), cd0 = sw128_desc(sm0 + kOffC, 16, kGroup);
        uint64_t j = 0, seg = 0;
        bool ok = true;
        while (ok && walk.next(g)) {
            if (g.k0 >= g.k1) continue;
            ok = warp_wait(&q_full, (uint32_t)(seg & 1));
            for (uint64_t k = g.k0; ok && k < g.k1; ++k, ++j) {
                if (j >= 2) ok = warp_wait(&s_free[j % 2], (uint32_t)((j / 2 - 1) & 1));
                if (ok) ok = warp_wait(&c_full[j % 2], (uint32_t)((j / 2) & 1));
                if (!ok) break;
                fence_after();
                const uint32_t d = tmem + kSCol + (uint32_t)(j % 2) * kTok;
                const uint64_t cd = cd0 + (((uint32_t)(j % 2) * 8 * kGroup) >> 4);
                if (elect_one()) {
#pragma unroll 4  // (all 36 in a row cost more in instruction fetches)
                    for (uint32_t u = 0; u < kChunks * 4; ++u)
                        mma_f16(d, qd + (((u >> 2) * kChunk + (u & 3) * 32) >> 4),
                                cd + (((u >> 2) * 1024 + (u & 3) * 32) >> 4), id_s, u);
                    mma_commit(smem_u32(&s_full[j % 2]));
                    if (k + 1 == g.k1) mma_commit(smem_u32(&q_free));
                }
                __syncwarp();
            }
            ++seg;
        }
        // every S issued has completed before the TMEM goes
        if (elect_one()) mma_commit(smem_u32(&s_end));
        __syncwarp();
        mbar_wait(smem_u32(&s_end), 0);
    } else if (warp == 6) {
        // ------------------------------------------------------------------- O^T += C^T . P^T
        const uint32_t id_o = f16_idesc(a.bf16 != 0, true, false, 128, kRows);
        const uint64_t vd0 = sw128_desc(sm0 + kOffC, 1024, kGroup), pd = sw128_desc(sm0 + kOffP, 16, 1024);
        uint64_t j = 0, seg = 0;
        bool ok = true;
        while (ok && walk.next(g)) {
            if (g.k0 >= g.k1) continue;
            for (uint64_t k = g.k0; ok && k < g.k1; ++k, ++j) {
                // (complete since S has read them; waited for here too, as their reader)
                ok = warp_wait(&c_full[j % 2], (uint32_t)((j / 2) & 1));
                if (ok && k == g.k0 && seg) ok = warp_wait(&o_free, (uint32_t)((seg - 1) & 1));
                if (ok) ok = warp_wait(&p_full[j % 2], (uint32_t)((j / 2) & 1));
                if (!ok) break;
                fence_after();
                const uint32_t acc = k > g.k0, half = (uint32_t)(j % 2);
                const uint64_t vd = vd0 + ((half * 8 * kGroup) >> 4);
                if (elect_one()) {
#pragma unroll
                    for (uint32_t kk = 0; kk < 4; ++kk) {  // 16 tokens, half a slot
#pragma unroll
                        for (uint32_t m = 0; m < 4; ++m)   // 128 dims
                            mma_f16(tmem + kOCol + m * kRows, vd + ((kk * 2 * kGroup + m * 2048) >> 4), pd + kk * 2,
                                    id_o, acc | kk);
                        if (kk & 1) mma_commit(smem_u32(&c_free[half * 2 + kk / 2]));
                    }
                    mma_commit(smem_u32(&o_done[half]));
                }
                __syncwarp();
            }
            ++seg;
        }
        if (elect_one()) mma_commit(smem_u32(&o_end));
        __syncwarp();
        mbar_wait(smem_u32(&o_end), 0);
    } else {
        // --------------------------------------------------------------- softmax, epilogue
        const uint32_t q4 = warp & 3, fr = lane >> 2, fc = lane & 3;  // fragment row, column
        const uint32_t row0 = q4 * 16 + fr;       // this thread's rows: row0, row0 + 8
        const uint32_t lane_addr = (q4 * 32) << 16;
        const float qscale = a.scale * 1.4426950408889634f;
        // a wait that runs out marks the window it falls in (the window of step w ends at that
        // step's vote) and the thread carries on to the vote with values it discards
        bool ok_w = true;
        auto wait_one = [&](unsigned long long* bar, uint32_t parity, uint64_t w) {
            if (!wait_for(bar, parity)) {
                fail_s[w % 2] = 1;
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
            // tokens that all of them see
            const uint64_t first = g.n > 1 ? (uint32_t)g.r0 / a.H : 0;
            const uint64_t all = g.len + 1 + first > g.n ? g.len + 1 + first - g.n : 0;
            float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
            for (uint64_t k = g.k0; k < g.k1; ++k, ++j) {
                wait_one(&s_full[j % 2], (uint32_t)((j / 2) & 1), j);
                fence_after();
                uint32_t xr[32];
                tmem_issue_frag(tmem + lane_addr + kSCol + (uint32_t)(j % 2) * kTok, xr);
                tmem_wait<32>(xr);
                fence_before();
                mbar_arrive(smem_u32(&s_free[j % 2]));
                const uint64_t t0 = k * kTok;
                // The rows' largest scaled scores.  Elements 4 i + 0, 1 are of the first row, 2, 3 of the
                // second.  A step that a row does not see whole takes scaled scores, -inf where it
                // sees none; others stay raw, and their extreme on the scale's side is scaled.
                float* x = reinterpret_cast<float*>(xr);
                float mx[2], qs = qscale;
                const int lim0 = vis[0] > t0 ? (int)umin(vis[0] - t0, kTok) : 0;
                const int lim1 = vis[1] > t0 ? (int)umin(vis[1] - t0, kTok) : 0;
                if (__any_sync(0xffffffffu, lim0 < (int)kTok || lim1 < (int)kTok)) {
                    qs = 1.0f;
                    mx[0] = mx[1] = -INFINITY;
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const int col = 8 * (i / 4) + 2 * (int)fc + (i & 1);
                        x[i] = col < (i & 2 ? lim1 : lim0) ? x[i] * qscale : -INFINITY;
                        mx[i >> 1 & 1] = fmaxf(mx[i >> 1 & 1], x[i]);
                    }
                } else if (qscale >= 0.0f) {
                    mx[0] = fmaxf(x[0], x[1]);
                    mx[1] = fmaxf(x[2], x[3]);
#pragma unroll
                    for (int i = 4; i < 32; i += 2) mx[i >> 1 & 1] = max3(mx[i >> 1 & 1], x[i], x[i + 1]);
                    mx[0] = fmaxf(-INFINITY, mx[0] * qscale);
                    mx[1] = fmaxf(-INFINITY, mx[1] * qscale);
                } else {
                    mx[0] = fminf(x[0], x[1]);
                    mx[1] = fminf(x[2], x[3]);
#pragma unroll
                    for (int i = 4; i < 32; i += 2) mx[i >> 1 & 1] = min3(mx[i >> 1 & 1], x[i], x[i + 1]);
                    mx[0] = fmaxf(-INFINITY, mx[0] * qscale);
                    mx[1] = fmaxf(-INFINITY, mx[1] * qscale);
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
                        wait_one(&o_done[(j - 1) % 2], (uint32_t)(((j - 1) / 2) & 1), j + 1);
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
                // weights (times 2^kWeightLift): summed in fp32, rounded to the element type for the product
                const float m0 = m[0] == -INFINITY ? 0.0f : m[0], m1 = m[1] == -INFINITY ? 0.0f : m[1];
                const float b0 = kWeightLift<T> - m0, b1 = kWeightLift<T> - m1;
                const uint64_t qs2 = pair_of(qs, qs), n0 = pair_of(b0, b0), n1 = pair_of(b1, b1);
                uint64_t sum0 = 0ull, sum1 = 0ull;
                uint32_t w[16];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float2 p0 = of_pair(fma2(pair_of(x[4 * i], x[4 * i + 1]), qs2, n0));
                    float2 p1 = of_pair(fma2(pair_of(x[4 * i + 2], x[4 * i + 3]), qs2, n1));
                    p0 = make_float2(exp2_approx(p0.x), exp2_approx(p0.y));
                    p1 = make_float2(exp2_approx(p1.x), exp2_approx(p1.y));
                    sum0 = add2(sum0, pair_of(p0.x, p0.y));
                    sum1 = add2(sum1, pair_of(p1.x, p1.y));
                    w[2 * i] = pack2<T>(p0.x, p0.y);
                    w[2 * i + 1] = pack2<T>(p1.x, p1.y);
                }
                l[0] += of_pair(sum0).x + of_pair(sum0).y;
                l[1] += of_pair(sum1).x + of_pair(sum1).y;
                // P is free once O^T of the step before has read it
                if (k > g.k0) wait_one(&o_done[(j - 1) % 2], (uint32_t)(((j - 1) / 2) & 1), j + 1);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t c = 8 * i + 2 * fc;
                    *reinterpret_cast<uint32_t*>(smem + kOffP + sw128_off(row0, c)) = w[2 * i];
                    *reinterpret_cast<uint32_t*>(smem + kOffP + sw128_off(row0 + 8, c)) = w[2 * i + 1];
                }
                // Values that meet zero weights have to be finite.  Tokens that no row of the tile sees, those
                // past the sequence among them, become zeros; of tokens that some see, what is not finite
                // does (the score of such a token is not finite either, so a row that sees it has its NaN
                // from there, or the weight zero of a score of -inf).  With one query a sequence only
                // the former occur.
                if (t0 + kTok > all) {
                    const uint32_t t = threadIdx.x - 64;  // chunk (t & 63) / 8, 16-byte piece t & 7
                    unsigned char* base = smem + kOffC + (uint32_t)(j % 2) * 8 * kGroup + ((t & 63) >> 3) * 1024 + (t & 7) * 16;
                    auto piece = [&](uint32_t r) { return reinterpret_cast<uint4*>(base + (r >> 3) * kGroup + (r & 7) * 128); };
                    const uint32_t r1 = g.seen < t0 + kTok ? (uint32_t)(g.seen - t0) : kTok;  // (seen > t0)
                    for (uint32_t r = r1 + (t >> 6); r < kTok; r += 2) *piece(r) = make_uint4(0, 0, 0, 0);
                    if (all < g.seen) {
                        wait_one(&c_full[j % 2], (uint32_t)((j / 2) & 1), j + 1);  // (its reader too)
                        for (uint32_t r = (all > t0 ? (uint32_t)(all - t0) : 0u) + (t >> 6); r < r1; r += 2)
                            *piece(r) = finite_only<T>(*piece(r));
                    }
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                mbar_arrive(smem_u32(&p_full[j % 2]));
            }
            if (stop) break;
            const bool any = g.k0 < g.k1;
            if (any) wait_one(&o_done[(j - 1) % 2], (uint32_t)(((j - 1) / 2) & 1), j);
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
                    inv_s[row0 + 8 * i] = l[i] == 0.0f ? 0.0f : 1.0f / l[i];
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
                if (whole) {
                    // lanes 2x, 2x + 1 hold dims d, d + 1: the even one stores both of an even row,
                    // the odd one of the odd row after it
                    T* o0 = out + (g.q0 * a.H + g.r0 + rb + (lane & 1)) * kR + (dim & ~1u);
#pragma unroll
                    for (uint32_t i = 0; i < 32; i += 2) {
                        const float e = __uint_as_float(o[i]) * inv_s[rb + i];
                        const float f = __uint_as_float(o[i + 1]) * inv_s[rb + i + 1];
                        const float y = __shfl_xor_sync(0xffffffffu, lane & 1 ? e : f, 1);
                        if (rb + i + (lane & 1) < g.rows)
                            *reinterpret_cast<uint32_t*>(o0 + i * kR) = lane & 1 ? pack2<T>(y, f) : pack2<T>(e, y);
                    }
                } else {
#pragma unroll
                    for (uint32_t i = 0; i < 32; ++i)
                        if (rb + i < g.rows) a.part_acc[(rec0 + rb + i) * kR + dim] = __uint_as_float(o[i]);
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

// The pool [rows, 576] as [chunk 9][row][64 dims]: boxes of 64 dims x 8 rows x 9 chunks.
bool pool_map(CUtensorMap* m, const LatentArgs& a)
{
    EncodeFn fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[3] = {64, a.num_pages * a.page_size, kChunks};
    const cuuint64_t strides[2] = {kW * 2, 128};
    const cuuint32_t box[3] = {64, 8, kChunks};
    const cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, a.bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3,
              const_cast<void*>(a.pool), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T>
int launch_t(const LatentArgs& a, cudaStream_t st)
{
    CUtensorMap mc, mq;
    if (!pool_map(&mc, a) || !map_2d(&mq, a.q, a.total_q * a.H, kW, kW * 2, kRows, a.bf16)) return HP_ERR_CUDA;
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
           page_size % 8 == 0 && num_pages > 0 && num_pages * page_size < (1ull << 31) && q_rows < (1ull << 31);
}

int launch_latent_tc(const LatentArgs& a, void* stream)
{
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return a.bf16 ? launch_t<__nv_bfloat16>(a, st) : launch_t<__half>(a, st);
}

}  // namespace hp
