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
// Selection.  Scores as integers in the order of the numbers; the threshold by three passes over 11,
// 11 and 10 bits of them (a histogram in shared memory each), then one pass that writes the pages
// above it and the first of those at it, in ascending order.
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
// and no sums over the sequences are needed.
template <typename T>
__global__ void __launch_bounds__(kBoundsThreads) bounds_kernel(const BoundsArgs a)
{
    __shared__ uint4 s_hi[kBoundsThreads], s_lo[kBoundsThreads];
    pdl_wait();
    const uint32_t parts = (a.columns + kBoundsThreads - 1) / kBoundsThreads;
    const uint64_t u = blockIdx.x / parts;
    const bool offsets = a.q.q_ptr != nullptr;
    if (u >= a.units) {  // the extra CTA
        int code = offsets_code(a.q.q_ptr, a.q.idx64, a.q.num_seqs, a.q.total_q);
        if (a.check_all)
            for (uint64_t s = threadIdx.x >> 5; s < a.q.num_seqs; s += kBoundsThreads / 32) {
                const uint64_t n = offsets ? index_at(a.q.q_ptr, a.q.idx64, s + 1) - index_at(a.q.q_ptr, a.q.idx64, s) : 1;
                const uint64_t pages = n <= a.q.total_q ? n / a.P + 2 : 0;
                for (uint64_t k = threadIdx.x & 31; k < pages; k += 32) code = lower(code, bounds_unit(a, s, k).code);
            }
        report_codes(code, a.d_status, a.check_all);
        return;
    }
    uint64_t s = u, k = 0;
    if (offsets) {
        auto first = [&](uint64_t i) { return index_at(a.q.q_ptr, a.q.idx64, i) / a.P + 2 * i; };
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
// together.  What bounds it is memory: 512 bytes a page and head at D = 128.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(32 * kScoreWarps) scores_kernel(const ScoreArgs a)
{
    constexpr int kSeg = D / 32;   // 64-byte segments of a row of D elements
    constexpr int kPart = kSeg < 4 ? kSeg : 4;
    pdl_wait();
    const uint64_t r = blockIdx.x / a.chunks;
    const unsigned warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    if (r >= a.q.total_q) {  // the extra CTA
        int code = offsets_code(a.q.q_ptr, a.q.idx64, a.q.num_seqs, a.q.total_q);
        if (a.check_all)
            for (uint64_t i = warp; i < a.q.total_q; i += kScoreWarps) {
                const ScoreRow row = score_row(a, find_query(a.q, i));
                code = lower(code, row.code);
                for (uint32_t j = lane; j < row.n; j += 32)
                    if (index_at(a.t.table, a.q.idx64, row.lo + j) >= a.t.num_pages) code = lower(code, HP_ERR_PAGE_ID);
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
    for (uint64_t i = warp; i < (uint64_t)blocks * a.H; i += kScoreWarps) {
        const uint32_t h = (uint32_t)(i % a.H), p0 = first + (uint32_t)(i / a.H) * 16;
        uint64_t phys[2];
        bool ok[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const uint32_t j = p0 + g + 8 * x;
            phys[x] = j < end ? index_at(a.t.table, a.q.idx64, row.lo + j) : 0;
            ok[x] = j < end && phys[x] < a.t.num_pages;
            if (j < end && !ok[x]) {
                if (tell && t == 0) atomicMin(a.d_status, (int)HP_ERR_PAGE_ID);
            }
        }
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
        const uint4* at[2];
#pragma unroll
        for (int x = 0; x < 2; ++x)
            at[x] = reinterpret_cast<const uint4*>(static_cast<const T*>(a.bounds) +
                                                   ((ok[x] ? phys[x] : 0) * a.H + h) * 2 * D) + t;
        float acc[NT][4] = {};
#pragma unroll
        for (int half = 0; half < 2; ++half)
#pragma unroll
            for (int c0 = 0; c0 < kSeg; c0 += kPart) {
                uint4 x[kPart], y[kPart];
#pragma unroll
                for (int c = 0; c < kPart; ++c) {
                    const int at16 = half * (D / 8) + (c0 + c) * 4;
                    x[c] = ok[0] ? at[0][at16] : uint4{};
                    y[c] = ok[1] ? at[1][at16] : uint4{};
                }
#pragma unroll
                for (int c = 0; c < kPart; ++c)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        const uint4 b = half ? dn[nt][c0 + c] : up[nt][c0 + c];
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

// One CTA a (query, K/V head).  Warp w holds the scores w * 32 * PER ... of a tile, score i * 32 + lane
// of them in register i: coalesced loads, and ballots give their order.  Rows of more than a tile
// are read again in each pass (they lie in L2).
template <int THREADS, int PER>
__global__ void __launch_bounds__(THREADS) select_kernel(const SelectArgs a)
{
    constexpr int kWarps = THREADS / 32, kPerThread = kBins / THREADS;
    constexpr uint32_t kTile = THREADS * PER;
    __shared__ uint32_t hist[kBins];
    __shared__ uint32_t s_warp[2][kWarps], s_bin, s_left;
    pdl_wait();
    const uint64_t r = blockIdx.x / a.H;
    const unsigned warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (r >= a.q.total_q) {  // the extra CTA
        int code = offsets_code(a.q.q_ptr, a.q.idx64, a.q.num_seqs, a.q.total_q);
        if (a.check_all)
            for (uint64_t i = warp; i < a.q.total_q; i += kWarps) {
                const Query q = find_query(a.q, i);
                code = lower(code, q.code != HP_OK ? q.code
                                   : q.seen && (q.seen + a.P - 1) / a.P > a.max_pages ? HP_ERR_OUT_SIZE : HP_OK);
            }
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
    uint32_t key[PER];
    auto load = [&](uint32_t base) {  // (places past the end are told apart by their index)
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const uint32_t at = base + (warp * PER + i) * 32 + lane;
            key[i] = at < count ? score_key(scores[at]) : 0u;
        }
    };
    if (one) load(0);
    uint32_t prefix = 0;
    int shift = 32;
    for (int pass = 0; pass < 3; ++pass) {
        const int bits = pass < 2 ? 11 : 10;
        for (uint32_t i = threadIdx.x; i < kBins; i += THREADS) hist[i] = 0;
        __syncthreads();
        for (uint32_t base = 0; base < count; base += kTile) {
            if (!one) load(base);
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const uint32_t at = base + (warp * PER + i) * 32 + lane;
                if (at < count && (pass == 0 || key[i] >> shift == prefix))
                    atomicAdd(&hist[(key[i] >> (shift - bits)) & ((1u << bits) - 1)], 1u);
            }
        }
        __syncthreads();
        // from the highest bin down: thread i has bins kBins - 1 - i * kPerThread ...
        uint32_t mine = 0;
#pragma unroll
        for (int i = 0; i < kPerThread; ++i) mine += hist[kBins - 1 - threadIdx.x * kPerThread - i];
        uint32_t sum = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t up = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= (unsigned)o) sum += up;
        }
        if (lane == 31) s_warp[0][warp] = sum;
        __syncthreads();
        uint32_t before = sum - mine;
        for (unsigned w = 0; w < warp; ++w) before += s_warp[0][w];
        if (before < need && need <= before + mine) {  // one thread's
            uint32_t b = kBins - 1 - threadIdx.x * kPerThread;
            while (before + hist[b] < need) before += hist[b--];
            s_bin = b;
            s_left = need - before;
        }
        __syncthreads();
        prefix = (prefix << bits) | s_bin;
        need = s_left;
        shift -= bits;
    }
    // above the threshold `prefix`, and the first `need` at it, in order
    uint32_t above_base = 0, equal_base = 0;
    for (uint32_t base = 0; base < count; base += kTile) {
        if (!one) load(base);
        uint32_t above = 0, equal = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const bool in = base + (warp * PER + i) * 32 + lane < count;
            above += __popc(__ballot_sync(0xffffffffu, in && key[i] > prefix));
            equal += __popc(__ballot_sync(0xffffffffu, in && key[i] == prefix));
        }
        __syncthreads();  // (the last tile's sums have been read)
        if (lane == 0) {
            s_warp[0][warp] = above;
            s_warp[1][warp] = equal;
        }
        __syncthreads();
        uint32_t pa = above_base, pe = equal_base;
        for (unsigned w = 0; w < kWarps; ++w) {
            if (w < warp) pa += s_warp[0][w], pe += s_warp[1][w];
            above_base += s_warp[0][w];
            equal_base += s_warp[1][w];
        }
        const unsigned below = (1u << lane) - 1u;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const uint32_t at = base + (warp * PER + i) * 32 + lane;
            const unsigned ma = __ballot_sync(0xffffffffu, at < count && key[i] > prefix);
            const unsigned me = __ballot_sync(0xffffffffu, at < count && key[i] == prefix);
            const uint32_t xa = pa + __popc(ma & below), xe = pe + __popc(me & below);
            if ((ma >> lane & 1) || ((me >> lane & 1) && xe < need))
                out[a.sinks + xa + (xe < need ? xe : need)] = (int32_t)(a.sinks + at);
            pa += __popc(ma);
            pe += __popc(me);
        }
    }
}

int start_status(bool all, int* d_status, cudaStream_t st)
{
    if (!d_status || all) return HP_OK;
    return cudaMemsetAsync(d_status, 0, sizeof(int), st) == cudaSuccess ? HP_OK : HP_ERR_CUDA;
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
    else e = launch_dependent(select_kernel<512, 16>, grid, 512, 0, st, a);
    return e == cudaSuccess ? HP_OK : HP_ERR_CUDA;
}

}  // namespace hp
