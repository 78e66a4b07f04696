// hp_latent.cu -- attention over a paged cache of shared latent rows on the CUDA cores (the
// shapes the tensor-core kernels do not take), the merge of the absorbed form's records, and
// the gather of the latent rows in front of the expanded form.
//
// Absorbed form: row r = (query, head) of a sequence scores every token it sees against the
// whole cache row, s_t = scale q_r . C_t over W dims, and sums the row's first R dims,
// o_r = sum_t p_t C_t[:R] with p the softmax of s: the row is read once for both.  Running
// maximum and sum (fp32, log2 units); a worker takes an equal range of (row group, step of 64
// tokens) units, so one long sequence spreads over the whole GPU and its partial results are
// joined by latent_merge_kernel in the order of the workers.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "hp_attn_merge.cuh"
#include "hp_internal.cuh"
#include "hp_latent.cuh"
#include "hp_latent_plan.cuh"
#include "hp_resolve.cuh"

namespace hp {
namespace {

// (Pool rows are read by plain loads: a kernel behind an append is resident while that one still writes
// them, and the read-only path is for memory that does not change over a kernel's life.)
constexpr float kLog2e = 1.4426950408889634f;

template <typename T> struct Pair;
template <> struct Pair<__half> {
    __device__ static float2 up(uint32_t u) { return __half22float2(*reinterpret_cast<const __half2*>(&u)); }
    __device__ static uint32_t down(float a, float b)
    {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    __device__ static __half one(float x) { return __float2half_rn(x); }
};
template <> struct Pair<__nv_bfloat16> {
    __device__ static float2 up(uint32_t u) { return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u)); }
    __device__ static uint32_t down(float a, float b)
    {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    __device__ static __nv_bfloat16 one(float x) { return __float2bfloat16_rn(x); }
};

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

constexpr int kRowsWarp = 2;   // rows of a warp
constexpr int kMaxPairs = 9;   // element pairs per lane: W <= 576
constexpr int kAccPairs = 8;   // R <= 512
constexpr int kKeys = 4;       // tokens per pass

template <typename T>
__global__ void __launch_bounds__(256, 2) latent_cc_kernel(const LatentArgs a)
{
    pdl_wait();
    if (a.hdr->verdict != kVerdictOk) return;
    const unsigned warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t pairs = a.W / 2, accp = a.R / 64;
    uint32_t* out = static_cast<uint32_t*>(a.out);
    for (uint64_t s = (uint64_t)blockIdx.x * 8 + warp; s < a.num_seqs; s += (uint64_t)gridDim.x * 8)
        if (a.units_off[s] == a.units_off[s + 1]) {  // no token: zeros for its queries
            const uint64_t q0 = a.q_ptr ? index_at(a.q_ptr, a.idx64, s) : s;
            const uint64_t q1 = a.q_ptr ? index_at(a.q_ptr, a.idx64, s + 1) : s + 1;
            for (uint64_t i = q0 * a.H * (a.R / 2) + lane; i < q1 * a.H * (a.R / 2); i += 32) out[i] = 0u;
        }
    const uint64_t total = a.hdr->total_units, Lw = (total + a.workers - 1) / a.workers;
    const uint64_t v = blockIdx.x, beg = umin(v * Lw, total), end = umin(beg + Lw, total);
    if (threadIdx.x == 255) write_merge(a, v, total, [&](uint64_t s) { return (uint64_t)a.units_off[s]; });
    const float qscale = a.scale * kLog2e;
    uint64_t pos = beg;
    while (pos < end) {
        const uint64_t s = find_seq(a.units_off, a.num_seqs, pos);
        const uint64_t len = index_at(a.lens, a.idx64, s), tab0 = index_at(a.seq_ptr, a.idx64, s);
        const uint64_t q0 = a.q_ptr ? index_at(a.q_ptr, a.idx64, s) : s;
        const uint64_t n = (a.q_ptr ? index_at(a.q_ptr, a.idx64, s + 1) : s + 1) - q0;
        const uint64_t steps = (len + kLatentStep - 1) / kLatentStep, off = pos - a.units_off[s];
        const uint64_t g = off / steps, k0 = off % steps, k1 = umin(steps, k0 + (end - pos));
        const uint64_t ustart = a.units_off[s] + g * steps;
        pos += k1 - k0;
        // this warp's rows, and the tokens each sees
        const uint64_t r0 = g * a.group_rows + warp * kRowsWarp;
        uint64_t vis[kRowsWarp];
        float q[kRowsWarp][2 * kMaxPairs], acc[kRowsWarp][2 * kAccPairs], m[kRowsWarp], l[kRowsWarp];
#pragma unroll
        for (int i = 0; i < kRowsWarp; ++i) {
            const uint64_t r = r0 + i, qi = r / a.H;
            const bool on = r < n * a.H;
            vis[i] = on && len + 1 + qi > n ? len + 1 + qi - n : 0;
            const uint32_t* src = static_cast<const uint32_t*>(a.q) + (q0 * a.H + r) * pairs;
#pragma unroll
            for (int j = 0; j < kMaxPairs; ++j) {
                const uint32_t p = lane + 32 * j;
                const float2 x = Pair<T>::up(on && p < pairs ? src[p] : 0u);
                q[i][2 * j] = x.x * qscale;
                q[i][2 * j + 1] = x.y * qscale;
            }
#pragma unroll
            for (int j = 0; j < 2 * kAccPairs; ++j) acc[i][j] = 0.0f;
            m[i] = -INFINITY;
            l[i] = 0.0f;
        }
        uint64_t tend = 0;
#pragma unroll
        for (int i = 0; i < kRowsWarp; ++i) tend = umax(tend, vis[i]);
        tend = umin(tend, umin(k1 * kLatentStep, len));
        for (uint64_t t0 = k0 * kLatentStep; t0 < tend; t0 += 32) {
            // the pool rows of 32 tokens, one per lane
            unsigned long long at = 0;
            if (t0 + lane < tend) {
                const uint64_t t = t0 + lane;
                at = index_at(a.table, a.idx64, tab0 + t / a.page_size) * a.page_size + t % a.page_size;
            }
            const uint32_t cnt = (uint32_t)umin(32, tend - t0);
            for (uint32_t c = 0; c < cnt; c += kKeys) {
                uint32_t kv[kKeys][kMaxPairs];
                float sc[kRowsWarp][kKeys];
#pragma unroll
                for (int u = 0; u < kKeys; ++u) {
                    const unsigned long long row = __shfl_sync(0xffffffffu, at, (int)umin(c + u, cnt - 1));
                    const uint32_t* src = static_cast<const uint32_t*>(a.pool) + row * pairs;
#pragma unroll
                    for (int j = 0; j < kMaxPairs; ++j) {
                        const uint32_t p = lane + 32 * j;
                        kv[u][j] = p < pairs ? src[p] : 0u;
                    }
                }
#pragma unroll
                for (int u = 0; u < kKeys; ++u) {
                    float d[kRowsWarp];
#pragma unroll
                    for (int i = 0; i < kRowsWarp; ++i) d[i] = 0.0f;
#pragma unroll
                    for (int j = 0; j < kMaxPairs; ++j) {
                        const float2 x = Pair<T>::up(kv[u][j]);
#pragma unroll
                        for (int i = 0; i < kRowsWarp; ++i)
                            d[i] = fmaf(q[i][2 * j + 1], x.y, fmaf(q[i][2 * j], x.x, d[i]));
                    }
#pragma unroll
                    for (int i = 0; i < kRowsWarp; ++i)
                        sc[i][u] = warp_sum(d[i]);
                }
#pragma unroll
                for (int i = 0; i < kRowsWarp; ++i) {
                    float mn = m[i];
#pragma unroll
                    for (int u = 0; u < kKeys; ++u) {
                        if (c + u >= cnt || t0 + c + u >= vis[i]) sc[i][u] = -INFINITY;
                        mn = fmaxf(mn, sc[i][u]);
                    }
                    // (no token seen yet: weights of zero, but a NaN score keeps its NaN)
                    const float base = mn == -INFINITY ? 0.0f : mn, f = exp2_approx(m[i] - base);
                    m[i] = mn;
                    l[i] *= f;
#pragma unroll
                    for (int u = 0; u < kKeys; ++u) {
                        sc[i][u] = exp2_approx(sc[i][u] - base);
                        l[i] += sc[i][u];
                    }
#pragma unroll
                    for (int j = 0; j < 2 * kAccPairs; ++j) acc[i][j] *= f;
                }
#pragma unroll
                for (int u = 0; u < kKeys; ++u)
#pragma unroll
                    for (int j = 0; j < kAccPairs; ++j)
                        if ((uint32_t)j < accp) {
                            const float2 x = Pair<T>::up(kv[u][j]);
#pragma unroll
                            for (int i = 0; i < kRowsWarp; ++i)
                                // a token the row does not see is absent, not of weight zero
                                if (sc[i][u] != 0.0f) {
                                    acc[i][2 * j] = fmaf(sc[i][u], x.x, acc[i][2 * j]);
                                    acc[i][2 * j + 1] = fmaf(sc[i][u], x.y, acc[i][2 * j + 1]);
                                }
                        }
            }
        }
        const bool whole = ustart >= beg && ustart + steps <= end;
        const uint64_t slot = 2 * v + (ustart <= beg ? 0 : 1);
#pragma unroll
        for (int i = 0; i < kRowsWarp; ++i) {
            const uint64_t r = r0 + i;
            if (r >= n * a.H) continue;
            if (whole) {
                const float inv = l[i] == 0.0f ? 0.0f : 1.0f / l[i];
                uint32_t* o = out + (q0 * a.H + r) * (a.R / 2);
#pragma unroll
                for (int j = 0; j < kAccPairs; ++j)
                    if ((uint32_t)j < accp)
                        o[lane + 32 * j] = Pair<T>::down(acc[i][2 * j] * inv, acc[i][2 * j + 1] * inv);
            } else {
                const uint64_t rec = slot * a.group_rows + warp * kRowsWarp + i;
                float2* o = reinterpret_cast<float2*>(a.part_acc + rec * a.R);
#pragma unroll
                for (int j = 0; j < kAccPairs; ++j)
                    if ((uint32_t)j < accp) o[lane + 32 * j] = make_float2(acc[i][2 * j], acc[i][2 * j + 1]);
                if (lane == 0) a.part_ml[rec] = make_float2(m[i], l[i]);
            }
        }
    }
}

// CTA (v, y): rows of the group that begins in worker v's range and goes on past it, SPLIT warps
// to a row (each a stretch of its sums).  With few rows four warps share one, so that a long
// sequence's many records are read by more of the GPU; with many, one warp's fixed part (the
// entry, the maxima and sums) is paid once a row (GB300, 128 heads: 16 us against 85 with four).
// Records of the range's workers that saw no token of the row have maximum -inf and sum 0; one of
// NaN scores has maximum -inf and a NaN sum, which stays.
template <typename T, int SPLIT>
__global__ void __launch_bounds__(256, 4) latent_merge_kernel(const LatentArgs a)
{
    constexpr int kRowsCta = 8 / SPLIT, kQuads = 4 / SPLIT, kBatch = 2 * SPLIT;  // kQuads float4s a lane
    pdl_wait();
    if (a.hdr->verdict != kVerdictOk) return;
    const unsigned warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const LatentMerge mg = a.merge[blockIdx.x];
    const uint32_t gr = blockIdx.y * kRowsCta + warp / SPLIT;
    if (gr >= mg.rows) return;
    const uint32_t v = blockIdx.x, last = mg.last;
    // worker w's record row
    auto rec = [&](uint32_t w) { return (uint64_t)(2 * w + (w == v ? mg.slot : 0)) * a.group_rows + gr; };
    // float4s of the row: this warp's stretch of R / 4 / SPLIT, kQuads per lane.  The first records'
    // are on their way while the maxima are looked at.
    const uint32_t stretch = a.R / 4 / SPLIT, q0 = (warp % SPLIT) * stretch;
    float4 x[kBatch][kQuads], acc[kQuads];
    auto fetch = [&](uint32_t w) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
#pragma unroll
            for (int j = 0; j < kQuads; ++j)
                x[i][j] = lane + 32 * j < stretch && w + i <= last
                              ? reinterpret_cast<const float4*>(a.part_acc + rec(w + i) * a.R)[q0 + lane + 32 * j]
                              : make_float4(0, 0, 0, 0);
    };
    fetch(v);
    // maximum and sum over the records, a lane per record, then pairwise
    float M = -INFINITY, L = 0.0f, mine = -INFINITY;  // mine: the maximum of record v + lane
    for (uint32_t w = v + lane; w <= last; w += 32) {
        const float2 ml = a.part_ml[rec(w)];
        if (w == v + lane) mine = ml.x;
        const float mn = fmaxf(M, ml.x), base = mn == -INFINITY ? 0.0f : mn;
        L = L * exp2_approx(M - base) + ml.y * exp2_approx(ml.x - base);
        M = mn;
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const float om = __shfl_xor_sync(0xffffffffu, M, o), ol = __shfl_xor_sync(0xffffffffu, L, o);
        const float mn = fmaxf(M, om), base = mn == -INFINITY ? 0.0f : mn;
        L = L * exp2_approx(M - base) + ol * exp2_approx(om - base);
        M = mn;
    }
    const float top = M == -INFINITY ? 0.0f : M;
    float fl = exp2_approx(mine - top);  // the factors of 32 records, one per lane
#pragma unroll
    for (int j = 0; j < kQuads; ++j) acc[j] = make_float4(0, 0, 0, 0);
    for (uint32_t w = v; w <= last;) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const float f = __shfl_sync(0xffffffffu, fl, (int)(w - v + i) & 31);  // (0 past the last)
#pragma unroll
            for (int j = 0; j < kQuads; ++j) {
                acc[j].x = fmaf(f, x[i][j].x, acc[j].x);
                acc[j].y = fmaf(f, x[i][j].y, acc[j].y);
                acc[j].z = fmaf(f, x[i][j].z, acc[j].z);
                acc[j].w = fmaf(f, x[i][j].w, acc[j].w);
            }
        }
        w += kBatch;
        if (w > last) break;
        fetch(w);
        if ((w - v) % 32 == 0) fl = exp2_approx((w + lane <= last ? a.part_ml[rec(w + lane)].x : -INFINITY) - top);
    }
    const float inv = L == 0.0f ? 0.0f : 1.0f / L;
    uint2* o = reinterpret_cast<uint2*>(static_cast<T*>(a.out) + (mg.out_row + gr) * a.R);
#pragma unroll
    for (int j = 0; j < kQuads; ++j)
        if (lane + 32 * j < stretch)
            o[q0 + lane + 32 * j] = make_uint2(Pair<T>::down(acc[j].x * inv, acc[j].y * inv),
                                               Pair<T>::down(acc[j].z * inv, acc[j].w * inv));
}

// --------------------------------------------------------------------- expanded form

// The latent rows of each sequence in order, padded with zeros to a multiple of kLatentPad, so
// that a block of 128 rows lies in one sequence.  Four rows per warp, 16 bytes per lane.  For the
// tensor cores (blocked) the latent part is a matrix of its own, the rope keys lie as shared memory
// holds them, and the kernel describes each block of queries (a search per CTA of the attention
// would be ten dependent loads); for a small batch it makes the plan first (hp_latent_plan.cuh).
__global__ void __launch_bounds__(256) latent_rows_kernel(const LatentPrefillArgs a)
{
    constexpr int kRowsWarp4 = 4;  // rows of a warp, looked up and loaded together
    __shared__ uint32_t units_s[kSmallSeqs + 1], rows_s[kSmallSeqs + 1];
    pdl_wait();
    uint64_t units, rows;
    if (a.small) {
        const SmallPlan sp = small_plan(a.plan, a.idx64, units_s, rows_s);
        if (blockIdx.x == 0 && threadIdx.x == 0) store_plan(a.plan, sp);
        if (sp.key != kVerdictOk) return;
        units = sp.units;
        rows = sp.rows;
    } else {
        if (a.hdr->verdict != kVerdictOk) return;
        units = a.hdr->total_units;
        rows = a.hdr->total_rows;
    }
    auto units_at = [&](uint64_t s) { return a.small ? (uint64_t)units_s[s] : (uint64_t)a.units_off[s]; };
    auto rows_at = [&](uint64_t s) { return a.small ? (uint64_t)rows_s[s] : (uint64_t)a.rows_off[s]; };
    auto find = [&](auto sums, uint64_t u) {  // the last sequence whose sum is at most u
        uint64_t lo = 0, hi = a.num_seqs;
        while (hi - lo > 1) {
            const uint64_t mid = (lo + hi) >> 1;
            if (sums(mid) <= u) lo = mid;
            else hi = mid;
        }
        return lo;
    };
    const unsigned warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (a.blocked) {  // the attention's units, from the last to the first: late queries see most
        if (blockIdx.x == 0 && threadIdx.x == 0) a.plan.ws.hdr->spoilt = 0;  // (the expansion sets it)
        for (uint64_t e = (uint64_t)blockIdx.x * 256 + threadIdx.x; e < a.max_units; e += (uint64_t)gridDim.x * 256) {
            LatentUnit un{};
            if (e < units) {
                const uint64_t u = units - 1 - e, s = find(units_at, u);
                const uint64_t q0 = a.q_ptr ? index_at(a.q_ptr, a.idx64, s) : s;
                const uint64_t n = (a.q_ptr ? index_at(a.q_ptr, a.idx64, s + 1) : s + 1) - q0;
                const uint64_t i0 = (u - units_at(s)) * a.q_block;
                un.block = rows_at(s) / kLatentPad;
                un.q_row = q0 + i0;
                un.seen0 = (int64_t)(index_at(a.lens, a.idx64, s) + 1 + i0) - (int64_t)n;
                un.queries = (uint32_t)umin(n - i0, a.q_block);
            }
            a.units[e] = un;
        }
    }
    const uint32_t vecs = a.W / 8, lvecs = a.R / 8;
    for (uint64_t row0 = ((uint64_t)blockIdx.x * 8 + warp) * kRowsWarp4; row0 < rows;
         row0 += (uint64_t)gridDim.x * 8 * kRowsWarp4) {
        const uint64_t s = find(rows_at, row0);  // (128 divides its first row)
        const uint64_t t0 = row0 - rows_at(s);
        const uint64_t len = index_at(a.lens, a.idx64, s), tab0 = index_at(a.seq_ptr, a.idx64, s);
        const uint4* src[kRowsWarp4];
#pragma unroll
        for (int i = 0; i < kRowsWarp4; ++i) {
            const uint64_t t = t0 + i;
            src[i] = nullptr;
            if (t < len)
                src[i] = static_cast<const uint4*>(a.pool) +
                         (index_at(a.table, a.idx64, tab0 + t / a.page_size) * a.page_size + t % a.page_size) * vecs;
        }
#pragma unroll 3
        for (uint32_t c = lane; c < vecs; c += 32) {
            uint4 x[kRowsWarp4];
#pragma unroll
            for (int i = 0; i < kRowsWarp4; ++i) x[i] = src[i] ? src[i][c] : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int i = 0; i < kRowsWarp4; ++i) {
                const uint64_t r = row0 + i;
                if (!a.blocked) static_cast<uint4*>(a.rows)[r * vecs + c] = x[i];
                else if (c < lvecs) static_cast<uint4*>(a.rows)[r * lvecs + c] = x[i];
                else  // 128-byte rows, 16-byte pieces swizzled by the row
                    static_cast<uint4*>(a.rope_blocks)[r * 8 + ((c - lvecs) ^ (r & 7))] = x[i];
            }
        }
    }
}

// kv[row, n] = sum_d rows[row, d] w_kv[n, d]: 64 x 64 tiles, 4 x 4 per thread.
template <typename T>
__global__ void __launch_bounds__(256) latent_expand_cc_kernel(const LatentPrefillArgs a)
{
    pdl_wait();
    if (a.hdr->verdict != kVerdictOk) return;
    const uint64_t row0 = (uint64_t)blockIdx.x * 64;
    const uint32_t N = a.H * (a.Dn + a.Dv), n0 = blockIdx.y * 64;
    if (row0 >= a.hdr->total_rows) return;
    __shared__ float sa[32][65], sb[32][65];  // [k][row], [k][n]
    const uint32_t tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    for (uint32_t k0 = 0; k0 < a.R; k0 += 32) {
        for (uint32_t i = threadIdx.x; i < 64 * 16; i += 256) {  // 16 pairs of 64 rows
            const uint32_t r = i / 16, p = i % 16;
            const float2 x = Pair<T>::up(*reinterpret_cast<const uint32_t*>(
                static_cast<const T*>(a.rows) + (row0 + r) * a.W + k0 + 2 * p));
            sa[2 * p][r] = x.x;
            sa[2 * p + 1][r] = x.y;
            const float2 y = Pair<T>::up(n0 + r < N ? *reinterpret_cast<const uint32_t*>(
                static_cast<const T*>(a.w_kv) + (uint64_t)(n0 + r) * a.R + k0 + 2 * p) : 0u);
            sb[2 * p][r] = y.x;
            sb[2 * p + 1][r] = y.y;
        }
        __syncthreads();
#pragma unroll 8
        for (int k = 0; k < 32; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    acc[i][j] = fmaf(sa[k][ty + 16 * i], sb[k][tx + 16 * j], acc[i][j]);
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (n0 + tx + 16 * j < N)
                static_cast<T*>(a.kv)[(row0 + ty + 16 * i) * N + n0 + tx + 16 * j] =
                    Pair<T>::one(acc[i][j]);
}

constexpr int kQ = 4;   // queries of a warp
constexpr int kDp = 4;  // element pairs per lane of a head's nope part or value: up to 256 dims

// CTA (u, h): block u of 32 queries, head h.
template <typename T>
__global__ void __launch_bounds__(256) latent_prefill_cc_kernel(const LatentPrefillArgs a)
{
    pdl_wait();
    if (a.hdr->verdict != kVerdictOk) return;
    const uint64_t u = blockIdx.x;
    if (u >= a.hdr->total_units) return;
    const unsigned warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t h = blockIdx.y, Dr = a.W - a.R;
    const uint64_t s = find_seq(a.units_off, a.num_seqs, u);
    const uint64_t len = index_at(a.lens, a.idx64, s);
    const uint64_t q0 = a.q_ptr ? index_at(a.q_ptr, a.idx64, s) : s;
    const uint64_t n = (a.q_ptr ? index_at(a.q_ptr, a.idx64, s + 1) : s + 1) - q0;
    const uint64_t i0 = (u - a.units_off[s]) * a.q_block + warp * kQ;
    const uint32_t np = a.Dn / 2, rp = Dr / 2, vp = a.Dv / 2;
    const float qscale = a.scale * kLog2e;
    uint64_t vis[kQ], tend = 0;
    float q[kQ][2 * kDp + 2], acc[kQ][2 * kDp], m[kQ], l[kQ];
#pragma unroll
    for (int i = 0; i < kQ; ++i) {
        const bool on = i0 + i < n;
        vis[i] = on && len + 1 + i0 + i > n ? len + 1 + i0 + i - n : 0;
        tend = umax(tend, vis[i]);
        const uint32_t* src =
            static_cast<const uint32_t*>(a.q) + ((q0 + i0 + i) * a.H + h) * (np + rp);
#pragma unroll
        for (int j = 0; j < kDp; ++j) {
            const uint32_t p = lane + 32 * j;
            const float2 x = Pair<T>::up(on && p < np ? src[p] : 0u);
            q[i][2 * j] = x.x * qscale;
            q[i][2 * j + 1] = x.y * qscale;
        }
        const float2 x = Pair<T>::up(on && lane < rp ? src[np + lane] : 0u);
        q[i][2 * kDp] = x.x * qscale;
        q[i][2 * kDp + 1] = x.y * qscale;
#pragma unroll
        for (int j = 0; j < 2 * kDp; ++j) acc[i][j] = 0.0f;
        m[i] = -INFINITY;
        l[i] = 0.0f;
    }
    const uint64_t row0 = a.rows_off[s];
    for (uint64_t t = 0; t < tend; ++t) {
        const uint32_t* kv = static_cast<const uint32_t*>(a.kv) +
                             ((row0 + t) * a.H + h) * (uint64_t)(np + vp);
        const uint32_t* kr = static_cast<const uint32_t*>(a.rows) + (row0 + t) * (a.W / 2) + a.R / 2;
        float d[kQ];
        float2 x = Pair<T>::up(lane < rp ? kr[lane] : 0u);
#pragma unroll
        for (int i = 0; i < kQ; ++i) d[i] = q[i][2 * kDp] * x.x + q[i][2 * kDp + 1] * x.y;
#pragma unroll
        for (int j = 0; j < kDp; ++j) {
            const uint32_t p = lane + 32 * j;
            x = Pair<T>::up(p < np ? kv[p] : 0u);
#pragma unroll
            for (int i = 0; i < kQ; ++i)
                d[i] = fmaf(q[i][2 * j + 1], x.y, fmaf(q[i][2 * j], x.x, d[i]));
        }
#pragma unroll
        for (int i = 0; i < kQ; ++i) {
            d[i] = warp_sum(d[i]);
            if (t >= vis[i]) continue;  // (the same in every lane)
            const float mn = fmaxf(m[i], d[i]), base = mn == -INFINITY ? 0.0f : mn;
            const float f = exp2_approx(m[i] - base), w = exp2_approx(d[i] - base);
            m[i] = mn;
            l[i] = l[i] * f + w;
#pragma unroll
            for (int j = 0; j < kDp; ++j) {
                const uint32_t p = lane + 32 * j;
                const float2 y = Pair<T>::up(p < vp ? kv[np + p] : 0u);
                acc[i][2 * j] = fmaf(w, y.x, acc[i][2 * j] * f);
                acc[i][2 * j + 1] = fmaf(w, y.y, acc[i][2 * j + 1] * f);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kQ; ++i) {
        if (i0 + i >= n) continue;
        const float inv = l[i] == 0.0f ? 0.0f : 1.0f / l[i];
        uint32_t* o = static_cast<uint32_t*>(a.out) + ((q0 + i0 + i) * a.H + h) * vp;
#pragma unroll
        for (int j = 0; j < kDp; ++j)
            if (lane + 32 * j < vp)
                o[lane + 32 * j] = Pair<T>::down(acc[i][2 * j] * inv, acc[i][2 * j + 1] * inv);
    }
}

template <typename T> int launch_prefill_t(const LatentPrefillArgs& a, cudaStream_t st)
{
    const uint32_t N = a.H * (a.Dn + a.Dv);
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.blockDim = dim3(256);
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.gridDim = dim3((unsigned)(a.cap_rows / 64), (N + 63) / 64);
    if (cudaLaunchKernelEx(&cfg, latent_expand_cc_kernel<T>, a) != cudaSuccess) return HP_ERR_CUDA;
    cfg.gridDim = dim3((unsigned)a.max_units, a.H);
    return cudaLaunchKernelEx(&cfg, latent_prefill_cc_kernel<T>, a) == cudaSuccess ? HP_OK : HP_ERR_CUDA;
}

}  // namespace

int launch_latent_cc(const LatentArgs& a, void* stream)
{
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const cudaError_t e =
        a.bf16 ? launch_dependent(latent_cc_kernel<__nv_bfloat16>, (unsigned)a.workers, 256, 0, st, a)
               : launch_dependent(latent_cc_kernel<__half>, (unsigned)a.workers, 256, 0, st, a);
    return e == cudaSuccess ? HP_OK : HP_ERR_CUDA;
}

int launch_latent_merge(const LatentArgs& a, void* stream)
{
    const bool few = a.total_q * a.H <= 2048;  // rows in all
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.gridDim = dim3((unsigned)a.workers, (a.group_rows + (few ? 1 : 7)) / (few ? 2 : 8));
    cfg.blockDim = dim3(256);
    cfg.stream = static_cast<cudaStream_t>(stream);
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e =
        a.bf16 ? (few ? cudaLaunchKernelEx(&cfg, latent_merge_kernel<__nv_bfloat16, 4>, a)
                      : cudaLaunchKernelEx(&cfg, latent_merge_kernel<__nv_bfloat16, 1>, a))
               : (few ? cudaLaunchKernelEx(&cfg, latent_merge_kernel<__half, 4>, a)
                      : cudaLaunchKernelEx(&cfg, latent_merge_kernel<__half, 1>, a));
    return e == cudaSuccess ? HP_OK : HP_ERR_CUDA;
}

int launch_latent_rows(const LatentPrefillArgs& a, void* stream)
{
    int dev = 0;
    const int sms = current_sms(&dev);
    if (sms == 0) return HP_ERR_CUDA;
    // (each CTA that makes the plan itself makes it once: no more of them than reside)
    const uint64_t ctas = a.cap_rows / 32, cap = (uint64_t)sms * (a.small ? 4 : 32);
    const uint64_t grid = ctas == 0 ? 1 : (ctas < cap ? ctas : cap);
    return launch_dependent(latent_rows_kernel, (unsigned)grid, 256, 0,
                            static_cast<cudaStream_t>(stream), a) == cudaSuccess
               ? HP_OK
               : HP_ERR_CUDA;
}

int launch_latent_prefill_cc(const LatentPrefillArgs& a, void* stream)
{
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return a.bf16 ? launch_prefill_t<__nv_bfloat16>(a, st) : launch_prefill_t<__half>(a, st);
}

}  // namespace hp
