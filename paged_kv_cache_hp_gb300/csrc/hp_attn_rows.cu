// hp_attn_rows.cu -- attention of single query rows over some pages of their sequences: the pages of
// a list (hp_attention_pages), or the stretch behind a prefix that is shared (hp_attention_prefix).
//
// For query row r and K/V head g, the G query heads of g at once:
//   x_t = scale q . K(t),  m = max x_t,  o = sum_t 2^((x_t - m) log2 e) V(t) / sum_t 2^(...)
// over the tokens t that the row's pages hold and it sees; one pass, with a maximum, a sum and a
// value sum that are rescaled together.  (A part that saw a token has a maximum of at least kLowest, even where
// all its scores are -inf: its value sum counts, 0 times infinities and all, and a row of such parts is 0 / 0.
// Only a part without tokens has -inf.)  Each element of K and V is used G times only, so what bounds it
// is memory: 4 D bytes a token and head.  The two products keep up on mma.sync with the tokens as its
// 16 rows and the queries as its 8 columns (S^T = K Q^T, O^T = V^T P^T), which wastes nothing at G = 8
// and needs neither TMEM nor more than a warp; the weights go from one product's accumulators to the
// other's operand by a transposed move inside the warp.
//
// A cluster of 1 to 8 CTAs takes a (row, head): its pages, cut into as many runs, and each run's
// blocks of kTokens tokens to the CTA's four warps in turn.  Each warp has its own ring (cp.async) of
// three units, K or V of a block, refilled as each has been read, and its own maximum, sum and value
// sum; they meet in the CTA's shared memory, the CTAs' in distributed shared memory (the answer is the
// same whichever finishes first, and no workspace is needed), and what the prefix's kernel left joins
// there.  Start and merge are 6 us of a CTA, so four of them share an SM (head_dim 64 and 128: 48 KiB of rings and
// 128 registers each; two at 256, with 96 KiB, and with more than 8 query heads a K/V
// head): 64 sequences x 8 heads x 2,048 tokens of 128 dims take 83 us, 5.9 TB/s; 128 x 8 x 540 tokens behind a
// prefix 58 us, 5.1 TB/s (two CTAs with rings half as large again: 61).
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "hp_attn_merge.cuh"
#include "hp_mma.cuh"
#include "hp_prefix.cuh"
#include "hp_resolve.cuh"
#include "hp_rows.cuh"
#include "hp_tcgen05.cuh"
#include "hp_tma.cuh"

namespace hp {
namespace {

namespace cg = cooperative_groups;
using tc::kWeightLift;
using tc::pack2;
using tc::split2;
using tma::smem_u32;

constexpr int kRowWarps = 4, kThreads = kRowWarps * 32;
constexpr uint32_t kWindow = 256;  // pages whose places lie in shared memory (a multiple of kTokens)
constexpr float kTau = 8.0f;       // log2 units a score may exceed its query's reference by

template <int D> struct Shape {
    static constexpr int kTokens = D == 64 ? 32 : 16;     // of a block
    static constexpr int kRow = D * 2, kPieces = kRow / 16;
    static constexpr int kUnit = kTokens * kRow;          // its rows of K, or of V
    static constexpr int kUnits = 3;                      // of a warp's ring
    static constexpr int kRing = kRowWarps * kUnits * kUnit;
    static constexpr int kPad = D + 4;                    // floats of a row of the merge
};

// a / b, in 32 bits where both fit.
__device__ __forceinline__ uint64_t small_quotient(uint64_t a, uint64_t b)
{
    return (a | b) >> 32 ? a / b : (uint32_t)a / (uint32_t)b;
}

struct Place {      // a page of the row's tokens
    uint64_t row0;  // its first slot in the pool
    uint32_t lo, hi;  // the slots that count
};

// Where the row's tokens lie: pages 0 .. count - 1 of a list or of up to two stretches.
struct Source {
    uint64_t lo, hi;           // the sequence's slice (list)
    const int32_t* list;
    uint32_t len, seen;
    uint64_t table[2];         // stretches: entry of page 0 of each slice
    uint32_t from, mid;        // tokens [0, mid) of the first if from is 0, [mid, seen) of the second
    uint32_t first_pages;      // pages of the first stretch
    uint32_t mid_page;         // mid / P
};

template <bool LIST>
__device__ __forceinline__ int place_at(const RowsArgs& a, const Source& s, uint32_t e, Place* p)
{
    *p = Place{0, 0, 0};
    uint64_t phys;
    if (LIST) {
        const int32_t j = s.list[e];
        if (j < 0) return HP_OK;
        const uint64_t t0 = (uint64_t)(uint32_t)j * a.P;
        if (t0 >= s.len) return HP_ERR_LEN;
        const int code = page_at(a.t, a.q.idx64, s.lo, s.hi, (uint32_t)j, &phys);
        if (code != HP_OK) return code;
        p->hi = t0 < s.seen ? (uint32_t)umin(a.P, s.seen - t0) : 0u;
    } else {
        const bool own = e >= s.first_pages;
        const uint32_t j = own ? s.mid_page + (e - s.first_pages) : e, t0 = j * a.P;
        const uint32_t t_lo = own ? s.mid : 0u, t_hi = own ? s.seen : s.mid;
        phys = index_at(a.t.table, a.q.idx64, (own ? s.table[1] : s.table[0]) + j);
        if (phys >= a.t.num_pages) return HP_ERR_PAGE_ID;  // (the plan has looked)
        p->lo = t_lo > t0 ? t_lo - t0 : 0u;
        p->hi = t_hi > t0 ? (t_hi - t0 < a.P ? t_hi - t0 : a.P) : 0u;
    }
    p->row0 = phys * a.P;
    return HP_OK;
}

template <typename T, int D, int NT, bool LIST>
__global__ void __launch_bounds__(kThreads, D == 256 || NT == 2 ? 2 : 4) rows_kernel(const RowsArgs a)
{
    using Sh = Shape<D>;
    constexpr int kTokens = Sh::kTokens, kSub = kTokens / 16;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ Place window[kWindow];
    __shared__ float s_m[kRowWarps][8 * NT], s_l[kRowWarps][8 * NT];
    __shared__ float2 s_ml[8 * NT];  // the CTA's
    __shared__ int s_code;
    const unsigned warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t4 = lane & 3;
    pdl_wait();
    const uint32_t unit = blockIdx.x / a.cluster, rank = blockIdx.x % a.cluster, h = unit % a.H;
    const uint64_t r = unit / a.H;
    if (LIST && r >= a.q.total_q) {  // the extra cluster's first CTA
        if (rank) return;
        int code = offsets_code(a.q.q_ptr, a.q.idx64, a.q.num_seqs, a.q.total_q);
        if (a.check_all) {
            Source* const rows = reinterpret_cast<Source*>(smem);  // (kRowsChecked of them; the ring is larger)
            for_each_query(a.q, [&](uint64_t i, const Query& q) {
                Source s{};  // (no list: nothing to look at)
                code = lower(code, q.code);
                if (q.seq < a.q.num_seqs && q.code == HP_OK) {
                    s.lo = index_at(a.t.seq_ptr, a.q.idx64, q.seq);
                    s.hi = index_at(a.t.seq_ptr, a.q.idx64, q.seq + 1);
                    s.len = (uint32_t)q.len;
                    s.seen = q.seen;
                    s.list = a.selected + i * a.H * a.k;
                }
                rows[i] = s;
            });
            __syncthreads();
            const uint32_t each = a.H * a.k;
            Place p;
#pragma unroll 4
            for (uint32_t e = threadIdx.x; e < (uint32_t)a.q.total_q * each; e += kThreads) {
                const Source& s = rows[e / each];
                if (s.list) code = lower(code, place_at<true>(a, s, e % each, &p));
            }
        }
        report_codes(code, a.d_status, a.check_all);
        return;
    }
    // what the row reads
    Source src{};
    uint32_t count = 0, skip = 0, last = a.P;  // pages; slots before the first token, up to the last
    PrefixRow row{};
    if (LIST) {
        const Query q = find_query(a.q, r);
        if (q.code != HP_OK && a.d_status && !a.check_all && rank == 0 && threadIdx.x == 0)
            atomicMin(a.d_status, q.code);
        if (q.seq >= a.q.num_seqs || q.code != HP_OK) return;  // (the whole cluster)
        src.lo = index_at(a.t.seq_ptr, a.q.idx64, q.seq);
        src.hi = index_at(a.t.seq_ptr, a.q.idx64, q.seq + 1);
        src.len = (uint32_t)q.len;
        src.seen = q.seen;
        src.list = a.selected + (uint64_t)unit * a.k;
        count = a.k;
    } else {
        row = a.rows[r];
        if (!plan_holds(a.hdr, a.num_keys, a.d_status, a.first && blockIdx.x == 0, a.first == 2) || row.group == 0xFFFFFFFFu) return;
        src.seen = row.seen;
        src.mid = row.prefix < row.seen ? row.prefix : row.seen;
        src.table[1] = row.table;
        if (a.rec.workers == 0 && src.mid) {
            src.table[0] = a.groups[row.group].table;
            src.first_pages = div_invariant(src.mid - 1, a.p_m, a.p_l) + 1;
        }
        src.mid_page = div_invariant(src.mid, a.p_m, a.p_l);
        const uint32_t end = src.seen > src.mid ? src.seen : src.mid;  // the last token is end - 1
        const uint32_t end_page = end ? div_invariant(end - 1, a.p_m, a.p_l) : 0u;
        const uint32_t own = src.seen > src.mid ? end_page + 1 - src.mid_page : 0u;
        count = src.first_pages + own;
        if (end) last = end - end_page * a.P;
        if (src.first_pages == 0 && own) skip = src.mid - src.mid_page * a.P;
    }
    if (threadIdx.x == 0) s_code = HP_OK;
    // the prefix's records of query head 0: first, count, and where a second of each lies
    uint64_t rec = 0;
    uint32_t recs = 0, second = 0;
    if (!LIST && a.rec.workers && row.prefix) {
        const PrefixGroup gr = a.groups[row.group];
        const uint32_t qt = kPrefixRows / a.G, tile = row.local / qt, left = gr.rows - tile * qt;
        const uint32_t rows = (left < qt ? left : qt) * a.G;
        const uint64_t lw = small_quotient(a.hdr->steps + a.rec.workers - 1, a.rec.workers);
        const uint64_t s0 = gr.step0 + ((uint64_t)h * gr.tiles + tile) * gr.blocks;
        const uint64_t v0 = small_quotient(s0, lw), v1 = small_quotient(s0 + gr.blocks - 1, lw);
        rec = gr.rows0 + h * gr.records + (uint64_t)tile * qt * a.G + v0 * kPrefixRows + row.local % qt * a.G;
        recs = (uint32_t)(v1 - v0 + 1);
        if (rows <= kPrefixRows / 2) {
            second = rows;
            recs *= 2;
        }
    }
    // the queries: rows dims 2 t4 + {0, 1} and + 8 of every 16, columns the heads
    uint32_t qb[NT][D / 16][2];
    {
        const T* q = static_cast<const T*>(a.queries) + (r * a.H + h) * a.G * D;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < D / 16; ++c)
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    qb[nt][c][x] = 8 * nt + g < a.G ? *reinterpret_cast<const uint32_t*>(
                                                          q + (8 * nt + g) * D + 16 * c + 8 * x + 2 * t4)
                                                    : 0u;
    }
    float o[NT][D / 16][4], m[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int c = 0; c < D / 16; ++c)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[nt][c][e] = 0.0f;
        m[nt][0] = m[nt][1] = -INFINITY;
        l[nt][0] = l[nt][1] = 0.0f;
    }
    const float qs = a.scale * 1.4426950408889634f;
    const uint64_t row_bytes = (uint64_t)a.H * Sh::kRow;
    const char* kp = static_cast<const char*>(a.k_pool) + (uint64_t)h * Sh::kRow;
    const char* vp = static_cast<const char*>(a.v_pool) + (uint64_t)h * Sh::kRow;
    const uint32_t ring = smem_u32(smem) + warp * Sh::kUnits * Sh::kUnit;

    // this CTA's blocks: places x of all pages' slots, kTokens to a block
    // (all below 2^32: the pages' slots number at most 2^31 and two pages more)
    const uint32_t x_end = count ? (count - 1) * a.P + last : 0u;
    const uint32_t b0 = skip / kTokens, b1 = (x_end + kTokens - 1) / kTokens, all = b1 > b0 ? b1 - b0 : 0u;
    const uint32_t per = (all + a.cluster - 1) / a.cluster, at0 = rank * per;
    const uint32_t bb = b0 + (at0 < all ? at0 : all), be = bb + per < b0 + all ? bb + per : b0 + all;
    const uint32_t wblocks = kWindow * a.P / kTokens;
    for (uint32_t win = bb / wblocks, w0 = win * wblocks; bb < be && w0 < be; ++win, w0 += wblocks) {
        const uint32_t wb = bb > w0 ? bb : w0, we = be - w0 < wblocks ? be : w0 + wblocks;
        const uint32_t page0 = win * kWindow;
        {
            const uint32_t e0 = div_invariant(wb * kTokens, a.p_m, a.p_l);
            const uint32_t e_last = div_invariant(we * kTokens - 1, a.p_m, a.p_l), e1 = e_last < count ? e_last + 1 : count;
            __syncthreads();  // (the last window has been read)
            int code = HP_OK;
            for (uint32_t e = e0 + threadIdx.x; e < e1; e += kThreads)
                code = lower(code, place_at<LIST>(a, src, e, &window[e - page0]));
            if (code != HP_OK) {
                atomicMin(&s_code, code);
                if (LIST && a.d_status && !a.check_all) atomicMin(a.d_status, code);
            }
            __syncthreads();
        }
        const uint32_t x_base = page0 * a.P;  // (x below 2^32)
        const uint32_t pages = count - page0 < kWindow ? count - page0 : kWindow;
        const uint32_t nb = we - wb, iters = nb > warp ? (nb - warp + kRowWarps - 1) / kRowWarps : 0;
        uint64_t off = 0;  // this lane's token of the block placed last: where its rows begin
        auto place = [&](uint32_t it) {  // which tokens of the warp's block `it` count
            if (it >= iters) return 0u;
            const uint32_t x = (wb + warp + it * kRowWarps) * kTokens - x_base + (lane % kTokens);
            const uint32_t e = div_invariant(x, a.p_m, a.p_l), slot = x - e * a.P;
            const Place p = e < pages ? window[e] : Place{0, 0, 0};
            const bool in = slot >= p.lo && slot < p.hi;
            off = in ? (p.row0 + slot) * row_bytes : 0;
            return __ballot_sync(0xffffffffu, in);
        };
        auto copy = [&](const char* pool, uint32_t unit, uint32_t mask) {  // that block's rows
            if (mask) {
                constexpr int kLanes = Sh::kPieces, kAt = kLanes >= 32 ? 1 : 32 / kLanes;
#pragma unroll
                for (int i = 0; i < kTokens / kAt; ++i) {
                    const uint32_t tok = i * kAt + lane / kLanes, piece = lane % kLanes;
                    const uint64_t at = __shfl_sync(0xffffffffu, off, tok) + piece * 16;
                    mma::copy16(ring + unit * Sh::kUnit + tok * Sh::kRow + ((piece ^ (tok & 7)) << 4), pool + at,
                                (mask >> tok & 1) ? 16u : 0u);
                }
            }
            mma::copies_commit();
        };
        // units in flight: K of a block goes where V of the one before the last was, V where K of the
        // last was, each as soon as it has been read
        uint32_t mask = place(0), next, at = 0;  // at: the unit of this block's K, its V's at + 1
        copy(kp, 0, mask);
        copy(vp, 1, mask);
        next = place(1);
        copy(kp, 2, next);
        for (uint32_t it = 0; it < iters; ++it) {
            const uint32_t at_v = at == 2 ? 0 : at + 1;
            const uint32_t sk = ring + at * Sh::kUnit, sv = ring + at_v * Sh::kUnit;
            float s[kSub][NT][4];
            mma::copies_wait<2>();
            __syncwarp();
            if (mask) {
                // S^T: 16 tokens x 8 queries each
#pragma unroll
                for (int b = 0; b < kSub; ++b)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[b][nt][e] = 0.0f;
#pragma unroll
                for (int c = 0; c < D / 16; ++c)
#pragma unroll
                    for (int b = 0; b < kSub; ++b) {
                        uint32_t k4[4];
                        const uint32_t tok = 16 * b + (lane & 15), piece = 2 * c + (lane >> 4);
                        mma::load4(k4, sk + tok * Sh::kRow + ((piece ^ (tok & 7)) << 4));
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            mma::product<T>(s[b][nt], k4[0], k4[1], k4[2], k4[3], qb[nt][c][0], qb[nt][c][1]);
                    }
            }
            __syncwarp();  // K has been read
            copy(vp, at, next);
            if (mask) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int x = 0; x < 2; ++x) m[nt][x] = fmaxf(m[nt][x], kLowest);
                bool move = false;
#pragma unroll
                for (int b = 0; b < kSub; ++b)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const bool in = mask >> (16 * b + g + 8 * (e >> 1)) & 1;
                            s[b][nt][e] = in ? s[b][nt][e] * qs : -INFINITY;
                            move |= s[b][nt][e] > m[nt][e & 1] + kTau;
                        }
                if (__any_sync(0xffffffffu, move)) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            float top = m[nt][x];
#pragma unroll
                            for (int b = 0; b < kSub; ++b) top = fmaxf(top, fmaxf(s[b][nt][x], s[b][nt][x + 2]));
#pragma unroll
                            for (int w = 4; w < 32; w <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
                            const float f = exp2_approx(m[nt][x] - top);
                            m[nt][x] = top;
                            l[nt][x] *= f;
#pragma unroll
                            for (int c = 0; c < D / 16; ++c) {
                                o[nt][c][x] *= f;
                                o[nt][c][x + 2] *= f;
                            }
                        }
                }
                // weights, as two parts of T for the value product, which takes 16-bit operands only (rounded
                // once, two weights a step of T apart are equal; the second part's products are 1% of the
                // time: 82.3 us without and 83.2 with them at the lists above)
                uint32_t p[kSub][NT][2], rest[kSub][NT][2];
#pragma unroll
                for (int b = 0; b < kSub; ++b)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        float w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            w[e] = exp2_approx(s[b][nt][e] - m[nt][e & 1] + kWeightLift<T>);
                            l[nt][e & 1] += w[e];
                        }
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            uint32_t hi, lo;
                            split2<T>(w[2 * x], w[2 * x + 1], hi, lo);
                            p[b][nt][x] = mma::transposed(hi);
                            rest[b][nt][x] = mma::transposed(lo);
                        }
                    }
                mma::copies_wait<2>();
                __syncwarp();
#pragma unroll
                for (int b = 0; b < kSub; ++b) {
                    // O^T += V^T P^T
#pragma unroll
                    for (int c = 0; c < D / 16; ++c) {
                        uint32_t v4[4];
                        const uint32_t tok = 16 * b + (lane & 7) + ((lane >> 4) << 3), piece = 2 * c + ((lane >> 3) & 1);
                        mma::load4_transposed(v4, sv + tok * Sh::kRow + ((piece ^ (tok & 7)) << 4));
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            mma::product<T>(o[nt][c], v4[0], v4[1], v4[2], v4[3], p[b][nt][0], p[b][nt][1]);
                            mma::product<T>(o[nt][c], v4[0], v4[1], v4[2], v4[3], rest[b][nt][0], rest[b][nt][1]);
                        }
                    }
                }
            }
            __syncwarp();  // V has been read
            mask = next;
            next = place(it + 2);
            copy(kp, at_v, next);
            at = at == 0 ? 2 : at - 1;
        }
        mma::copies_wait<0>();
    }
    // ---- the warps' parts meet
    __syncthreads();
    float* part = reinterpret_cast<float*>(smem);  // [warp][query][kPad]
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            float sum = l[nt][x];
#pragma unroll
            for (int w = 4; w < 32; w <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
            const int n = 8 * nt + 2 * t4 + x;
            if (g == 0) {
                s_m[warp][n] = m[nt][x];
                s_l[warp][n] = sum;
            }
            float* dst = part + (warp * 8 * NT + n) * Sh::kPad + g;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) {
                dst[16 * c] = o[nt][c][x];
                dst[16 * c + 8] = o[nt][c][x + 2];
            }
        }
    __syncthreads();
    if (threadIdx.x < 8 * NT) {
        float top = -INFINITY, sum = 0.0f;
        for (int w = 0; w < kRowWarps; ++w) top = fmaxf(top, s_m[w][threadIdx.x]);
        for (int w = 0; w < kRowWarps; ++w) {
            const float f = s_m[w][threadIdx.x] == -INFINITY ? 0.0f : exp2_approx(s_m[w][threadIdx.x] - top);
            sum += s_l[w][threadIdx.x] * f;
            s_m[w][threadIdx.x] = f;  // the warp's factor
        }
        s_ml[threadIdx.x] = make_float2(top, sum);
    }
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < a.G * (D / 4); i += kThreads) {
        const uint32_t n = i / (D / 4), d = i % (D / 4) * 4;
        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < kRowWarps; ++w) {
            const float4 y = *reinterpret_cast<const float4*>(part + (w * 8 * NT + n) * Sh::kPad + d);
            const float f = s_m[w][n];
            x.x += y.x * f, x.y += y.y * f, x.z += y.z * f, x.w += y.w * f;
        }
        *reinterpret_cast<float4*>(part + n * Sh::kPad + d) = x;  // (only this thread reads these places)
    }
    // ---- the CTAs' parts meet, each CTA finishing a share of the dimensions
    cg::cluster_group cluster = cg::this_cluster();
    if (a.cluster > 1) cluster.sync();
    else __syncthreads();
    int code = s_code;
    for (uint32_t c = 0; c < a.cluster; ++c) code = lower(code, *cluster.map_shared_rank(&s_code, c));
    const uint32_t share = (a.G * (D / 4) + a.cluster - 1) / a.cluster;
    const uint32_t i0 = rank * share, i1 = (uint32_t)umin(i0 + share, a.G * (D / 4));
    auto record = [&](uint32_t v) {  // the v-th record's row of query head 0
        return second ? rec + (uint64_t)(v >> 1) * kPrefixRows + (v & 1) * second : rec + (uint64_t)v * kPrefixRows;
    };
    // each source's weight for each query head (negative: it saw no token), the CTAs' first, and one over
    // the heads' sums (0 where no source saw one); a warp a head
    const uint32_t sources = a.cluster + recs;
    float* const weight = reinterpret_cast<float*>(smem) + kRowWarps * 8 * NT * Sh::kPad;  // [head][sources]
    for (uint32_t n = warp; n < a.G; n += kRowWarps) {
        auto source = [&](uint32_t v) {
            return v < a.cluster ? cluster.map_shared_rank(s_ml, v)[n] : a.rec.ml[record(v - a.cluster) + n];
        };
        float top = -INFINITY, sum = 0.0f;
        for (uint32_t v = lane; v < sources; v += 32) top = fmaxf(top, source(v).x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        for (uint32_t v = lane; v < sources; v += 32) {
            const float2 ml = source(v);
            const bool none = ml.x == -INFINITY;
            const float f = none ? -1.0f : exp2_approx(ml.x - top);
            weight[n * sources + v] = f;
            if (!none) sum += ml.y * f;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) s_l[0][n] = top == -INFINITY ? 0.0f : 1.0f / sum;
    }
    __syncthreads();
    if (code == HP_OK)
        for (uint32_t i = i0 + threadIdx.x; i < i1; i += kThreads) {
            const uint32_t n = i / (D / 4), d = i % (D / 4) * 4;
            const float* w = weight + n * sources;
            float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            auto add = [&](float f, const float4& y) {
                if (f < 0.0f) return;
                x.x += y.x * f, x.y += y.y * f, x.z += y.z * f, x.w += y.w * f;
            };
            for (uint32_t c = 0; c < a.cluster; ++c)
                add(w[c], *reinterpret_cast<const float4*>(cluster.map_shared_rank(part, c) + n * Sh::kPad + d));
            for (uint32_t v0 = 0; v0 < recs; v0 += 8) {  // eight records in flight
                float4 y[8];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (v0 + e < recs && !(w[a.cluster + v0 + e] < 0.0f))
                        y[e] = *reinterpret_cast<const float4*>(a.rec.acc + (record(v0 + e) + n) * D + d);
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (v0 + e < recs) add(w[a.cluster + v0 + e], y[e]);
            }
            const float inv = s_l[0][n];
            uint2 y;
            y.x = pack2<T>(x.x * inv, x.y * inv);
            y.y = pack2<T>(x.z * inv, x.w * inv);
            *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + ((r * a.H + h) * a.G + n) * D + d) = y;
        }
    if (a.cluster > 1) cluster.sync();  // (the others have read this CTA's)
}

template <typename T, int D, int NT, bool LIST>
int launch_k(const RowsArgs& a, cudaStream_t st)
{
    int dev = 0;
    // the merge: the warps' parts, then a weight for each source and query head
    constexpr int kMerge = (kRowWarps * 8 * NT * Shape<D>::kPad + kPagesMaxGroup * (8 + 2 * (int)kPrefixMaxSms)) * 4;
    constexpr int kSmem = Shape<D>::kRing > kMerge ? Shape<D>::kRing : kMerge;
    if (current_sms(&dev) == 0 || !allow_dynamic_smem<rows_kernel<T, D, NT, LIST>>(dev, kSmem)) return HP_ERR_CUDA;
    cudaLaunchConfig_t cfg{};
    const uint64_t units = a.q.total_q * a.H;
    cfg.gridDim = dim3((unsigned)((units + (LIST && a.d_status != nullptr)) * a.cluster));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim = {a.cluster, 1, 1};
    cfg.attrs = attr;
    cfg.numAttrs = a.cluster > 1 ? 2 : 1;
    if (cfg.gridDim.x == 0) return HP_OK;
    return cudaLaunchKernelEx(&cfg, rows_kernel<T, D, NT, LIST>, a) == cudaSuccess ? HP_OK : HP_ERR_CUDA;
}

template <typename T, int D>
int launch_d(const RowsArgs& a, cudaStream_t st)
{
    if (a.selected) return a.G <= 8 ? launch_k<T, D, 1, true>(a, st) : launch_k<T, D, 2, true>(a, st);
    return a.G <= 8 ? launch_k<T, D, 1, false>(a, st) : launch_k<T, D, 2, false>(a, st);
}

template <typename T>
int launch_t(const RowsArgs& a, cudaStream_t st)
{
    return a.D == 64 ? launch_d<T, 64>(a, st) : a.D == 128 ? launch_d<T, 128>(a, st) : launch_d<T, 256>(a, st);
}

}  // namespace

int launch_rows(const RowsArgs& a, void* stream)
{
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (a.selected && a.d_status && !a.check_all) {
        const int rc = launch_clear_status(a.d_status, stream);
        if (rc) return rc;
    }
    return a.bf16 ? launch_t<__nv_bfloat16>(a, st) : launch_t<__half>(a, st);
}

}  // namespace hp
