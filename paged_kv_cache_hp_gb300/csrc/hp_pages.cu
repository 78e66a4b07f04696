// hp_pages.cu -- which pages of a long sequence a query should read: bounds of a page's keys, upper
// bounds of its scores, the selection.
//
// Bounds.  hi_d = max_t K(t)_d and lo_d = min_t K(t)_d over the page's tokens.  For any query q
//   q . K(t) = sum_d q_d K(t)_d <= sum_d max(q_d hi_d, q_d lo_d),
// so a page whose sum is low holds no token that scores high.  bounds_kernel reads the rows of the
// pages that new tokens fell into and stores both rows: pure data movement.
//
// Scores.  max(q_d hi_d, q_d lo_d) is q_d hi_d where q_d > 0 and q_d lo_d elsewhere, so the sum is the
// product of the page's 2 D numbers with the row (max(q, 0), min(q, 0)), which a matrix product takes
// for 16 pages and 8 queries at a time.  Both rows are exact in the pool's type, products and sums
// are fp32.  Where an infinity meets a zero of the other half, the sum is not a number: such a page
// (rare) is summed again from the definition.
//
// Selection.  Scores as integers in the order of the numbers; the threshold's 11 high bits by a histogram in
// shared memory, the others by ranking the few scores that share those (or, where they are many, by two more
// histograms of 11 and 10 bits), then one pass that writes the pages above it and the first of those at
// it, in ascending order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "hp_mma.cuh"
#include "hp_pages.cuh"
#include "hp_resolve.cuh"

namespace hp {
namespace {

// -------------------------------------------------------------------------- bounds
constexpr int kBoundsThreads = 128;

template <typename T> struct Two;
template <> struct Two<__nv_bfloat16> { using V = __nv_bfloat162; };
template <> struct Two<__half> { using V = __half2; };

// Two elements, NaN if either operand is.
template <typename T> __device__ __forceinline__ uint32_t most2(uint32_t a, uint32_t b)
{
    using V = typename Two<T>::V;
    const V r = __hmax2_nan(*reinterpret_cast<V*>(&a), *reinterpret_cast<V*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}
template <typename T> __device__ __forceinline__ uint32_t least2(uint32_t a, uint32_t b)
{
    using V = typename Two<T>::V;
    const V r = __hmin2_nan(*reinterpret_cast<V*>(&a), *reinterpret_cast<V*>(&b));
    return *reinterpret_cast<const uint32_t*>(&r);
}
template <typename T> __device__ __forceinline__ void meet(uint4& hi, uint4& lo, const uint4& x, const uint4& y)
{
    hi.x = most2<T>(hi.x, x.x), hi.y = most2<T>(hi.y, x.y), hi.z = most2<T>(hi.z, x.z), hi.w = most2<T>(hi.w, x.w);
    lo.x = least2<T>(lo.x, y.x), lo.y = least2<T>(lo.y, y.y), lo.z = least2<T>(lo.z, y.z), lo.w = least2<T>(lo.w, y.w);
}

struct BoundsUnit {
    uint64_t phys;
    uint32_t rows;  // 0: no page
    int code;
};

// Page k of those that sequence s's new tokens touch.  n0, n1: their offsets.
__device__ __forceinline__ BoundsUnit bounds_unit(const BoundsArgs& a, uint64_t s, uint64_t k)
{
    BoundsUnit u{0, 0, HP_OK};
    const uint64_t n0 = a.q.q_ptr ? index_at(a.q.q_ptr, a.q.idx64, s) : 0;
    const uint64_t n1 = a.q.q_ptr ? index_at(a.q.q_ptr, a.q.idx64, s + 1) : 1;
    const uint64_t len = index_at(a.q.lens, a.q.idx64, s);
    if (n0 >= n1 || (a.q.q_ptr ? n1 > a.q.total_q : len == 0)) return u;
    if (n1 - n0 > len || len >= kPagesMaxTokens) {
        u.code = HP_ERR_LEN;
        return u;
    }
    const uint64_t j = (uint32_t)(len - (n1 - n0)) / a.P + k, t0 = j * a.P;
    if (t0 >= len) return u;
    u.code = page_at(a.t, a.q.idx64, index_at(a.t.seq_ptr, a.q.idx64, s), index_at(a.t.seq_ptr, a.q.idx64, s + 1), j,
                     &u.phys);
    if (u.code == HP_OK) u.rows = (uint32_t)umin(a.P, len - t0);
    return u;
}

// A CTA takes one page and up to 128 of its row's 16-byte columns; where a row has fewer, several
// threads share a column's tokens and meet in shared memory.  Page k of sequence s is unit
// new_ptr[s] / P + 2 s + k: n tokens touch at most n / P + 2 pages, so no two sequences' units meet
// and no sums over the sequences are needed.  (11 prompts of 36,000 tokens, 4 heads of 128 in pages of 64: 8.7 us,
// 4.3 TB/s in one wave; 64 decode steps: 4.2 us, the host's time for a call.)
template <typename T>
__global__ void __launch_bounds__(kBoundsThreads) bounds_kernel(const BoundsArgs a)
{
    __shared__ uint4 s_hi[kBoundsThreads], s_lo[kBoundsThreads];
    pdl_wait();
    const uint32_t parts = (a.columns + kBoundsThreads - 1) / kBoundsThreads;
    const uint64_t u = blockIdx.x / parts;
    const bool offsets = a.q.q_ptr != nullptr;
    auto first = [&](uint64_t i) { return index_at(a.q.q_ptr, a.q.idx64, i) / a.P + 2 * i; };
    if (u >= a.units) {  // the extra CTA
        int code = offsets_code(a.q.q_ptr, a.q.idx64, a.q.num_seqs, a.q.total_q);
        if (a.check_all)
            for (uint64_t i = threadIdx.x; i < a.units; i += kBoundsThreads) {
                uint64_t s = i, lo = 0;
                if (offsets) {
                    uint64_t end = a.q.num_seqs;
                    for (s = 0; end - s > 1;) {
                        const uint64_t mid = (s + end) >> 1;
                        if (first(mid) <= i) s = mid;
                        else end = mid;
                    }
                    lo = first(s);
                }
                if (!offsets || lo <= i) code = lower(code, bounds_unit(a, s, offsets ? i - lo : 0).code);
            }
        report_codes(code, a.d_status, a.check_all);
        return;
    }
    uint64_t s = u, k = 0;
    if (offsets) {
        s = warp_last(a.q.num_seqs, [&](uint64_t i) { return first(i) <= u; });
        if (first(s) > u) return;
        k = u - first(s);
    }
    const BoundsUnit un = bounds_unit(a, s, k);
    if (un.code != HP_OK && a.d_status && !a.check_all && threadIdx.x == 0) atomicMin(a.d_status, un.code);
    if (un.rows == 0) return;
    const uint32_t c0 = (uint32_t)(blockIdx.x % parts) * kBoundsThreads;
    const uint32_t cols = a.columns - c0 < kBoundsThreads ? a.columns - c0 : kBoundsThreads;
    const uint32_t lanes = kBoundsThreads / cols, mine = threadIdx.x / cols, c = c0 + threadIdx.x % cols;
    const uint4* rows = static_cast<const uint4*>(a.pool) + un.phys * a.P * a.columns + c;
    const uint32_t stop = mine < lanes ? un.rows : 0;
    uint4 hi{}, lo{};
    if (mine < stop) {
        hi = lo = rows[(uint64_t)mine * a.columns];
        // eight rows in flight
        uint32_t t = mine + lanes;
        for (; t + 7 * lanes < stop; t += 8 * lanes) {
            uint4 x[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = rows[(uint64_t)(t + i * lanes) * a.columns];
#pragma unroll
            for (int i = 0; i < 8; ++i) meet<T>(hi, lo, x[i], x[i]);
        }
        uint4 x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = t + i * lanes < stop ? rows[(uint64_t)(t + i * lanes) * a.columns] : hi;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (t + i * lanes < stop) meet<T>(hi, lo, x[i], x[i]);
    }
    if (lanes > 1) {
        s_hi[threadIdx.x] = hi;
        s_lo[threadIdx.x] = lo;
        __syncthreads();
        if (mine == 0)
            for (uint32_t m = 1; m < lanes && m < un.rows; ++m)
                meet<T>(hi, lo, s_hi[threadIdx.x + m * cols], s_lo[threadIdx.x + m * cols]);
    }
    if (mine == 0) {
        uint4* out = static_cast<uint4*>(a.bounds) + 2 * un.phys * a.columns;
        const uint32_t h = c / a.row_half, d = c % a.row_half;
        out[(2 * h) * a.row_half + d] = hi;
        out[(2 * h + 1) * a.row_half + d] = lo;
    }
}

// -------------------------------------------------------------------------- scores
constexpr int kScoreWarps = 8;

__device__ __forceinline__ float larger(float a, float b)  // NaN if either is
{
    return a != a ? a : (b != b ? b : fmaxf(a, b));
}

template <typename T> __device__ __forceinline__ float widen(T x);
template <> __device__ __forceinline__ float widen(__nv_bfloat16 x) { return __bfloat162float(x); }
template <> __device__ __forceinline__ float widen(__half x) { return __half2float(x); }

struct ScoreRow {
    uint64_t lo;  // first table entry
    uint32_t n;   // pages
    int code;
};

__device__ __forceinline__ ScoreRow score_row(const ScoreArgs& a, const Query& q)
{
    ScoreRow row{0, 0, q.code};
    if (q.seq >= a.q.num_seqs || q.code != HP_OK || q.seen == 0) return row;
    const uint64_t lo = index_at(a.t.seq_ptr, a.q.idx64, q.seq), hi = index_at(a.t.seq_ptr, a.q.idx64, q.seq + 1);
    const uint32_t n = (q.seen + a.P - 1) / a.P;
    if (n > a.max_pages) row.code = HP_ERR_OUT_SIZE;
    else if (lo > hi || hi > a.t.table_len || n > hi - lo) row.code = HP_ERR_LEN;
    else row.lo = lo, row.n = n;
    return row;
}

// A warp takes 16 pages of a K/V head at a time: lane l loads 16 bytes (l % 4) of every 64 of pages
// l / 4 and l / 4 + 8, straight into the registers of the product's A operand.  (The order of a
// product's inner dimension is free: the queries' registers are filled in the same order, from the
// same 16 bytes of q.)  The warps of a CTA take the heads of the same pages, whose bounds lie
// together.  What bounds it is memory: 512 bytes a page and head at D = 128 (300,000 pages of 8 heads: 203 us,
// 6.05 TB/s).  A row's loads of up to 256 elements are in flight together, two CTAs an SM: half as many at a time
// and three CTAs took 222 us.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(32 * kScoreWarps, D == 256 || NT == 2 ? 1 : D == 128 ? 2 : 3) scores_kernel(const ScoreArgs a)
{
    constexpr int kSeg = D / 32;   // 64-byte segments of a row of D elements
    constexpr int kPart = 2 * kSeg < 8 ? 2 * kSeg : 8;
    pdl_wait();
    const uint64_t r = blockIdx.x / a.chunks;
    const unsigned warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    if (r >= a.q.total_q) {  // the extra CTA
        int code = offsets_code(a.q.q_ptr, a.q.idx64, a.q.num_seqs, a.q.total_q);
        if (a.check_all) {
            __shared__ ScoreRow rows[kRowsChecked];
            for_each_query(a.q, [&](uint64_t i, const Query& q) {
                rows[i] = score_row(a, q);
                code = lower(code, rows[i].code);
            });
            __syncthreads();
            for (uint64_t i = warp; i < a.q.total_q; i += kScoreWarps)
                for (uint32_t j = lane; j < rows[i].n; j += 32)
                    if (index_at(a.t.table, a.q.idx64, rows[i].lo + j) >= a.t.num_pages) code = lower(code, HP_ERR_PAGE_ID);
        }
        report_codes(code, a.d_status, a.check_all);
        return;
    }
    const uint32_t first = (uint32_t)umin((blockIdx.x % a.chunks) * a.chunk_blocks * 16ull, 0xFFFFFFFFull);
    const ScoreRow row = score_row(a, find_query(a.q, r));
    const bool tell = a.d_status && !a.check_all;
    if (row.code != HP_OK && tell && first == 0 && threadIdx.x == 0) atomicMin(a.d_status, row.code);
    if (first >= row.n) return;
    const uint32_t end = (uint32_t)umin(row.n, (uint64_t)first + a.chunk_blocks * 16ull);
    const uint32_t blocks = (end - first + 15) / 16;
    const T* queries = static_cast<const T*>(a.queries) + r * a.H * a.G * D;
    uint4 up[NT][kSeg], dn[NT][kSeg];
    uint32_t head = 0xFFFFFFFFu;
    // the pages of this lane's two rows of an item (16 pages, a head), as the table has them
    const uint32_t items = blocks * a.H;  // (a CTA's: the host holds them below 2^31)
    auto pages_of = [&](uint32_t i, uint64_t (&phys)[2]) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const uint32_t j = first + i / a.H * 16 + g + 8 * x;
            phys[x] = i < items && j < end ? index_at(a.t.table, a.q.idx64, row.lo + j) : 0;
        }
    };
    uint64_t next[2];
    pages_of(warp, next);
    for (uint32_t i = warp; i < items; i += kScoreWarps) {
        const uint32_t block = i / a.H, h = i - block * a.H, p0 = first + block * 16;
        const uint64_t phys[2] = {next[0], next[1]};
        const bool ok[2] = {p0 + g < end && phys[0] < a.t.num_pages, p0 + g + 8 < end && phys[1] < a.t.num_pages};
        if (tell && t == 0 && ((p0 + g < end && !ok[0]) || (p0 + g + 8 < end && !ok[1])))
            atomicMin(a.d_status, (int)HP_ERR_PAGE_ID);
        pages_of(i + kScoreWarps, next);  // (on its way while this item is summed)
        if (!__any_sync(0xffffffffu, ok[0] || ok[1])) continue;
        if (h != head) {
            head = h;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < kSeg; ++c) {
                    const uint32_t n = 8 * nt + g;
                    uint4 x{};
                    if (n < a.G)
                        x = *reinterpret_cast<const uint4*>(queries + (uint64_t)(h * a.G + n) * D + c * 32 + t * 8);
                    up[nt][c] = uint4{most2<T>(x.x, 0u), most2<T>(x.y, 0u), most2<T>(x.z, 0u), most2<T>(x.w, 0u)};
                    dn[nt][c] = uint4{least2<T>(x.x, 0u), least2<T>(x.y, 0u), least2<T>(x.z, 0u), least2<T>(x.w, 0u)};
                }
        }
        const uint4* at[2];  // (a row without a page reads the pool's first, for nothing)
#pragma unroll
        for (int x = 0; x < 2; ++x)
            at[x] = reinterpret_cast<const uint4*>(static_cast<const T*>(a.bounds) +
                                                   ((ok[x] ? phys[x] : 0) * a.H + h) * 2 * D) + t;
        float acc[NT][4] = {};
        // a row's 2 D numbers in parts, the loads of each in flight together
#pragma unroll
        for (int c0 = 0; c0 < 2 * kSeg; c0 += kPart) {
            uint4 x[kPart], y[kPart];
#pragma unroll
            for (int c = 0; c < kPart; ++c) {
                x[c] = at[0][(c0 + c) * 4];
                y[c] = at[1][(c0 + c) * 4];
            }
#pragma unroll
            for (int c = 0; c < kPart; ++c)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const uint4 b = c0 + c < kSeg ? up[nt][c0 + c] : dn[nt][c0 + c - kSeg];
                    mma::product<T>(acc[nt], x[c].x, y[c].x, x[c].y, y[c].y, b.x, b.y);
                    mma::product<T>(acc[nt], x[c].z, y[c].z, x[c].w, y[c].w, b.z, b.w);
                }
        }
        // the largest of the group's queries: columns 2 t and 2 t + 1 here, the others in the lane's quad
        float best[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (8 * nt + 2 * t + (e & 1) < a.G) best[e >> 1] = larger(best[e >> 1], acc[nt][e]);
#pragma unroll
        for (int o = 1; o < 4; o <<= 1)
#pragma unroll
            for (int x = 0; x < 2; ++x) best[x] = larger(best[x], __shfl_xor_sync(0xffffffffu, best[x], o));
        float* out = a.scores + (r * a.H + h) * a.max_pages + p0;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const unsigned bad = __ballot_sync(0xffffffffu, t == 0 && ok[x] && best[x] != best[x]);
            if (ok[x] && t == 0 && best[x] == best[x]) out[g + 8 * x] = best[x] * a.scale;
            for (unsigned left = bad; left; left &= left - 1) {  // from the definition
                const int src = __ffs(left) - 1;
                const uint64_t pg = __shfl_sync(0xffffffffu, phys[x], src);
                const T* b = static_cast<const T*>(a.bounds) + (pg * a.H + h) * 2 * D;
                float top = -INFINITY;
                for (uint32_t n = 0; n < a.G; ++n) {
                    float sum = 0.0f;
                    for (int d = lane; d < D; d += 32) {
                        const float qd = widen(queries[(uint64_t)(h * a.G + n) * D + d]);
                        sum += larger(qd * widen(b[d]), qd * widen(b[D + d]));
                    }
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    top = larger(top, sum);
                }
                if (lane == 0) out[src / 4 + 8 * x] = top * a.scale;
            }
        }
    }
}

// ----------------------------------------------------------------------- selection
constexpr uint32_t kBins = 2048;

// Scores in the order of their keys; all NaN above everything and alike, both zeros alike.
__device__ __forceinline__ uint32_t score_key(float x)
{
    if (x != x) return 0xFFFFFFFFu;
    const uint32_t b = __float_as_uint(x + 0.0f);
    return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}

// The sum over the warps before this one, and over all, of a warp's number; `room` has kWarps words.
// (Two barriers: before the words are written and before they are read.)
template <int kWarps>
__device__ __forceinline__ uint32_t warps_before(uint32_t mine, uint32_t* room, uint32_t& all)
{
    const unsigned warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __syncthreads();
    if (lane == 0) room[warp] = mine;
    __syncthreads();
    const uint32_t x = lane < kWarps ? room[lane] : 0u;
    uint32_t sum = x;
#pragma unroll
    for (int o = 1; o < kWarps; o <<= 1) {
        const uint32_t up = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= (unsigned)o) sum += up;
    }
    all = __shfl_sync(0xffffffffu, sum, kWarps - 1);
    return __shfl_sync(0xffffffffu, sum - x, warp);
}

// One CTA a (query, K/V head).  Warp w holds the scores w * 32 * PER ... of a tile, score i * 32 + lane
// of them in register i: coalesced loads, and ballots give their order.  Only the first pass counts
// all scores; those in its threshold bin (a few hundred) are gathered in shared memory.
// In the last one lane i of a warp writes what ballot i found: few bits are set where few pages are
// taken.  Rows of more than a tile are read again each time (they lie in L2).  What bounds it is issue
// and barriers: 1,900 instructions a warp of 1,024 scores and a dozen barriers (2,048 rows of up to 8,192 scores: 45
// us; 512 threads of 16 scores: 48).
template <int THREADS, int PER>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) select_kernel(const SelectArgs a)
{
    constexpr int kWarps = THREADS / 32, kPerThread = kBins / THREADS;
    constexpr uint32_t kTile = THREADS * PER, kCand = 2048;
    static_assert(PER <= 32 && kPerThread % 4 == 0, "a lane a ballot, bins in vectors");
    __shared__ __align__(16) uint32_t hist[kBins];
    __shared__ __align__(16) uint32_t cand[kCand];
    __shared__ uint32_t s_room[kWarps], s_bin, s_left, s_cand;
    pdl_wait();
    const uint64_t r = blockIdx.x / a.H;
    const unsigned warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (r >= a.q.total_q) {  // the extra CTA
        int code = offsets_code(a.q.q_ptr, a.q.idx64, a.q.num_seqs, a.q.total_q);
        if (a.check_all)
            for_each_query(a.q, [&](uint64_t, const Query& q) {
                code = lower(code, q.code != HP_OK ? q.code
                                   : q.seen && (q.seen + a.P - 1) / a.P > a.max_pages ? HP_ERR_OUT_SIZE : HP_OK);
            });
        report_codes(code, a.d_status, a.check_all);
        return;
    }
    const Query q = find_query(a.q, r);
    const uint32_t n = (q.seen + a.P - 1) / a.P;
    const int code = q.code != HP_OK ? q.code : n > a.max_pages ? HP_ERR_OUT_SIZE : HP_OK;
    if (code != HP_OK && a.d_status && !a.check_all && threadIdx.x == 0) atomicMin(a.d_status, code);
    if (q.seq >= a.q.num_seqs || code != HP_OK) return;
    int32_t* out = a.selected + (r * a.H + blockIdx.x % a.H) * a.k;
    if (n <= a.k) {
        for (uint32_t i = threadIdx.x; i < a.k; i += THREADS) out[i] = i < n ? (int32_t)i : -1;
        return;
    }
    for (uint32_t i = threadIdx.x; i < a.sinks; i += THREADS) out[i] = (int32_t)i;
    for (uint32_t i = threadIdx.x; i < a.recent; i += THREADS)
        out[a.k - a.recent + i] = (int32_t)(n - a.recent + i);
    const uint32_t count = n - a.sinks - a.recent;  // more than
    uint32_t need = a.k - a.sinks - a.recent;
    if (need == 0) return;
    const float* scores = a.scores + (r * a.H + blockIdx.x % a.H) * a.max_pages + a.sinks;
    const bool one = count <= kTile;
    const uint32_t mine = warp * (PER * 32) + lane;
    uint32_t key[PER];
    auto load = [&](uint32_t base) {  // (places past the end are told apart by their index)
        const float* from = scores + base + mine;
        const uint32_t left = count - base > mine ? count - base - mine : 0u;
        float x[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) x[i] = 32u * i < left ? from[32 * i] : 0.0f;
#pragma unroll
        for (int i = 0; i < PER; ++i) key[i] = score_key(x[i]);
        return left;
    };
    // f(key, place within the thread's 32 PER of the tile) for every score
    auto every = [&](auto&& f) {
        for (uint32_t base = 0; base < count; base += kTile) {
            uint32_t left = count - base > mine ? count - base - mine : 0u;
            if (!one) left = load(base);
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (32u * i < left) f(key[i]);
        }
    };
    if (one) load(0);
    uint32_t prefix = 0;
    int shift = 32;
    bool gathered = false;
    for (int pass = 0; pass < 3; ++pass) {
        const int bits = pass < 2 ? 11 : 10, down = shift - bits;
        for (uint32_t i = threadIdx.x; i < kBins / 4; i += THREADS) reinterpret_cast<uint4*>(hist)[i] = uint4{};
        if (threadIdx.x == 0 && pass == 0) s_cand = 0;
        __syncthreads();
        const uint32_t low = (1u << bits) - 1;
        if (pass == 0) every([&](uint32_t x) { atomicAdd(&hist[x >> down], 1u); });
        else if (gathered)
            for (uint32_t i = threadIdx.x; i < s_cand; i += THREADS) {
                if (cand[i] >> shift == prefix) atomicAdd(&hist[cand[i] >> down & low], 1u);
            }
        else every([&](uint32_t x) {
                if (x >> shift == prefix) atomicAdd(&hist[x >> down & low], 1u);
            });
        __syncthreads();
        // from the highest bin down: thread i has bins kBins - 1 - i * kPerThread ...
        uint32_t h[kPerThread], part = 0;
#pragma unroll
        for (int i = 0; i < kPerThread / 4; ++i) {
            const uint4 v = reinterpret_cast<const uint4*>(hist)[(kBins - (threadIdx.x + 1) * kPerThread) / 4 + kPerThread / 4 - 1 - i];
            h[4 * i] = v.w, h[4 * i + 1] = v.z, h[4 * i + 2] = v.y, h[4 * i + 3] = v.x;
            part += v.x + v.y + v.z + v.w;
        }
        uint32_t sum = part, all;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t up = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= (unsigned)o) sum += up;
        }
        const uint32_t total = __shfl_sync(0xffffffffu, sum, 31);
        uint32_t before = warps_before<kWarps>(total, s_room, all) + sum - part;
        if (before < need && need <= before + part) {  // one thread's
            uint32_t b = kBins - 1 - threadIdx.x * kPerThread;
#pragma unroll
            for (int i = 0; i < kPerThread; ++i) {
                if (before < need && need <= before + h[i]) {
                    s_bin = b - i;
                    s_left = need - before;
                }
                before += h[i];
            }
        }
        __syncthreads();
        prefix = (prefix << bits) | s_bin;
        need = s_left;
        shift = down;
        if (pass == 0) {
            const uint32_t in = hist[prefix];  // scores in the threshold's bin
            gathered = in <= kCand;
            if (gathered)
                every([&](uint32_t x) {
                    if (x >> down == prefix) cand[atomicAdd(&s_cand, 1u)] = x;
                });
            __syncthreads();  // (the bin has been read, the scores are gathered)
            if (in <= THREADS) {
                // few: a thread each counts those above and those equal (0 is no score's key)
                if (threadIdx.x < 4) cand[in + threadIdx.x] = 0;
                __syncthreads();
                const uint32_t x = cand[threadIdx.x];
                if (warp * 32 < in) {
                    uint32_t above = 0, equal = 0;
                    for (uint32_t j = 0; j < in; j += 4) {
                        const uint4 y = *reinterpret_cast<const uint4*>(cand + j);
                        above += (y.x > x) + (y.y > x) + (y.z > x) + (y.w > x);
                        equal += (y.x == x) + (y.y == x) + (y.z == x) + (y.w == x);
                    }
                    if (threadIdx.x < in && above < need && need <= above + equal) {  // equal ones all say the same
                        s_bin = x;
                        s_left = need - above;
                    }
                }
                __syncthreads();
                prefix = s_bin;
                need = s_left;
                break;
            }
        }
    }
    // above the threshold `prefix`, and the first `need` at it, in order
    uint32_t above_base = 0, equal_base = 0;
    for (uint32_t base = 0; base < count; base += kTile) {
        uint32_t left = count - base > mine ? count - base - mine : 0u;
        if (!one) left = load(base);
        uint32_t ma = 0, me = 0;  // of ballot `lane`
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const unsigned va = __ballot_sync(0xffffffffu, 32u * i < left && key[i] > prefix);
            const unsigned ve = __ballot_sync(0xffffffffu, 32u * i < left && key[i] == prefix);
            if (lane == (unsigned)i) ma = va, me = ve;
        }
        // counts of both, packed: a tile has at most 2^14 scores
        const uint32_t both = __popc(ma) << 16 | __popc(me);
        uint32_t sum = both, all;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t up = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= (unsigned)o) sum += up;
        }
        const uint32_t total = __shfl_sync(0xffffffffu, sum, 31);
        const uint32_t at = warps_before<kWarps>(total, s_room, all) + sum - both;
        uint32_t pa = above_base + (at >> 16), pe = equal_base + (at & 0xFFFF);
        above_base += all >> 16;
        equal_base += all & 0xFFFF;
        if (pe >= need) me = 0;
        for (unsigned taken = ma | me; taken; taken &= taken - 1) {
            const unsigned bit = __ffs(taken) - 1;
            const bool equal = me >> bit & 1;
            if (!equal || pe < need)
                out[a.sinks + pa + (pe < need ? pe : need)] = (int32_t)(a.sinks + base + warp * (PER * 32) + 32 * lane + bit);
            if (equal) ++pe;
            else ++pa;
        }
    }
}

// (a dependent launch on either side: a memset takes 3 us of a stream of such calls)
__global__ void clear_status_kernel(int* d_status)
{
    pdl_wait();
    *d_status = HP_OK;
}

int start_status(bool all, int* d_status, cudaStream_t st)
{
    return !d_status || all ? (int)HP_OK : launch_clear_status(d_status, st);
}

template <typename T, int D>
int launch_scores_d(const ScoreArgs& a, unsigned grid, cudaStream_t st)
{
    return (a.G <= 8 ? launch_dependent(scores_kernel<T, D, 1>, grid, 32 * kScoreWarps, 0, st, a)
                     : launch_dependent(scores_kernel<T, D, 2>, grid, 32 * kScoreWarps, 0, st, a)) == cudaSuccess
               ? HP_OK
               : HP_ERR_CUDA;
}

template <typename T>
int launch_scores_t(const ScoreArgs& a, unsigned grid, cudaStream_t st)
{
    return a.D == 64 ? launch_scores_d<T, 64>(a, grid, st)
                     : a.D == 128 ? launch_scores_d<T, 128>(a, grid, st) : launch_scores_d<T, 256>(a, grid, st);
}

}  // namespace

int launch_clear_status(int* d_status, void* stream)
{
    return launch_dependent(clear_status_kernel, 1, 1, 0, static_cast<cudaStream_t>(stream), d_status) == cudaSuccess
               ? HP_OK
               : HP_ERR_CUDA;
}

int launch_page_bounds(const BoundsArgs& a, void* stream)
{
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int rc = start_status(a.check_all, a.d_status, st);
    if (rc) return rc;
    const uint32_t parts = (a.columns + kBoundsThreads - 1) / kBoundsThreads;
    const unsigned grid = (unsigned)(a.units * parts + (a.d_status != nullptr));
    if (grid == 0) return HP_OK;
    return (a.bf16 ? launch_dependent(bounds_kernel<__nv_bfloat16>, grid, kBoundsThreads, 0, st, a)
                   : launch_dependent(bounds_kernel<__half>, grid, kBoundsThreads, 0, st, a)) == cudaSuccess
               ? HP_OK
               : HP_ERR_CUDA;
}

int launch_page_scores(const ScoreArgs& a, void* stream)
{
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int rc = start_status(a.check_all, a.d_status, st);
    if (rc) return rc;
    const unsigned grid = (unsigned)(a.q.total_q * a.chunks + (a.d_status != nullptr));
    if (grid == 0) return HP_OK;
    return a.bf16 ? launch_scores_t<__nv_bfloat16>(a, grid, st) : launch_scores_t<__half>(a, grid, st);
}

int launch_select_pages(const SelectArgs& a, void* stream)
{
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int rc = start_status(a.check_all, a.d_status, st);
    if (rc) return rc;
    const unsigned grid = (unsigned)(a.q.total_q * a.H + (a.d_status != nullptr));
    if (grid == 0) return HP_OK;
    cudaError_t e;
    if (a.max_pages <= 512) e = launch_dependent(select_kernel<128, 4>, grid, 128, 0, st, a);
    else if (a.max_pages <= 2048) e = launch_dependent(select_kernel<256, 8>, grid, 256, 0, st, a);
    else e = launch_dependent(select_kernel<256, 32>, grid, 256, 0, st, a);
    return e == cudaSuccess ? HP_OK : HP_ERR_CUDA;
}

}  // namespace hp
