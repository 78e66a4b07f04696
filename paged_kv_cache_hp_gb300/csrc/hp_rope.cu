// hp_rope.cu -- norm, position rotation and append in one pass over a projection's output.
//
// A head's vector x becomes y_d = x_d * rsqrt(mean x^2 + eps) * w_d, its pairs (a, b) turn to
// (a cos - b sin, b cos + a sin), and the result goes to q_out or to the token's slot of the
// pool.  Every element is read and written once, so the pass is bound by memory: a head takes a
// group of L lanes, 8 elements each (16 bytes of a 16-bit type), L the power of two that covers
// its dimensions; a warp takes one token (or a share of its heads when tokens are few) and
// keeps that token's cosines and sines in registers over all the heads.  Sums, norm and
// rotation are fp32, rounded once.
//
// Errors: a token is skipped by the warp that meets it.  *d_status comes from one extra CTA that
// looks at every token's slot and positions while the others work (no launch of its own; a
// batch of 64 tokens takes 3.5 us in a graph), or from a memset before the kernel and atomicMin over
// the codes where that CTA would be the last to finish: it takes 2 ns a token, the others 0.23 ns a
// KiB, so batches of more than kReportTokens go by the bytes of a token (8,193 tokens of 25 KiB:
// 42.7 us against 47.2 with the memset; 16,001 of 6.7 KiB: 30.6 against 28.8).  Either way it is the
// smallest code of the batch, whatever the order.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "hp_internal.cuh"
#include "hp_resolve.cuh"
#include "hp_step.cuh"

namespace hp {
namespace {

constexpr int kThreads = 256;
constexpr int kWarpsRope = kThreads / 32;

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float x, float& y) { y = x; }
__device__ __forceinline__ void from_f(float x, __half& y) { y = __float2half_rn(x); }
__device__ __forceinline__ void from_f(float x, __nv_bfloat16& y) { y = __float2bfloat16_rn(x); }

// 16 bytes of what the call only reads.  Not by the read-only path (__ldg): a CTA is resident while the
// kernel before it still writes these bytes, and that path is for memory that does not change over a
// kernel's life; nor would the wait hold such a load back.  A volatile one stays behind the wait, and may
// pass the call's own stores (a plain load may not: 32.6 us for 16,001 latent rows against 28.8).
__device__ __forceinline__ uint4 load16(const void* p)
{
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ float4 load4(const float* p)
{
    const uint4 v = load16(p);
    return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
}

// 8 elements in 16-byte pieces
template <typename T> struct Vec8 {
    static constexpr int N = 8 * sizeof(T) / 16;
    uint4 u[N];
    __device__ __forceinline__ void load(const T* p)
    {
#pragma unroll
        for (int i = 0; i < N; ++i) u[i] = load16(reinterpret_cast<const uint4*>(p) + i);
    }
    // (q_out may be q)
    __device__ __forceinline__ void load_rw(const T* p)
    {
#pragma unroll
        for (int i = 0; i < N; ++i) u[i] = *(reinterpret_cast<const uint4*>(p) + i);
    }
    __device__ __forceinline__ void store(T* p) const
    {
#pragma unroll
        for (int i = 0; i < N; ++i) *(reinterpret_cast<uint4*>(p) + i) = u[i];
    }
    __device__ __forceinline__ void unpack(float (&x)[8]) const
    {
        const T* e = reinterpret_cast<const T*>(u);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = to_f(e[i]);
    }
    __device__ __forceinline__ void pack(const float (&x)[8])
    {
        T* e = reinterpret_cast<T*>(u);
#pragma unroll
        for (int i = 0; i < 8; ++i) from_f(x[i], e[i]);
    }
};

__device__ __forceinline__ uint64_t position(const RopeArgs& r, uint64_t tokens, uint32_t axis,
                                             uint64_t t)
{
    const uint64_t i = axis * tokens + t;
    return r.idx64 ? static_cast<const unsigned long long*>(r.positions)[i]
                   : (uint64_t)static_cast<const unsigned int*>(r.positions)[i];
}

// HP_OK, or why a token of slot `slot` is not processed (a padding token: HP_OK); far: one of its
// positions is past the table.
__device__ __forceinline__ int code_of(const AppendArgs& a, int64_t slot, bool far)
{
    if (slot < 0) return HP_OK;
    return far ? HP_ERR_LEN : ((uint64_t)slot >= a.num_slots ? HP_ERR_PAGE_ID : HP_OK);
}

__device__ __forceinline__ int token_error(const AppendArgs& a, uint64_t t, int64_t slot)
{
    bool far = false;
    if (a.rope.rot)
        for (uint32_t x = 0; x < a.rope.axes; ++x) far |= position(a.rope, a.tokens, x, t) >= a.rope.max_pos;
    return code_of(a, slot, far);
}

constexpr uint64_t kReportTokens = 2048, kReportBytes = 12288;

// The extra CTA, the grid's first: the smallest code of all tokens, eight of each thread's looked at
// together (one by one they took 69 us for 16,001).
__device__ __forceinline__ void report_all(const AppendArgs& a)
{
    constexpr int kTogether = 8;
    __shared__ int s_code;
    if (threadIdx.x == 0) s_code = HP_OK;
    __syncthreads();
    int code = HP_OK;
    for (uint64_t t0 = threadIdx.x; t0 < a.tokens; t0 += kTogether * kThreads) {
        int64_t slot[kTogether];
        bool far[kTogether];
#pragma unroll
        for (int u = 0; u < kTogether; ++u) {
            const uint64_t t = t0 + u * kThreads;
            slot[u] = t < a.tokens ? a.slot_map[t] : -1;
            far[u] = false;
#pragma unroll
            for (uint32_t x = 0; x < 4; ++x)
                if (t < a.tokens && a.rope.rot && x < a.rope.axes)
                    far[u] |= position(a.rope, a.tokens, x, t) >= a.rope.max_pos;
        }
#pragma unroll
        for (int u = 0; u < kTogether; ++u) code = min(code, code_of(a, slot[u], far[u]));
    }
    if (code != HP_OK) atomicMin(&s_code, code);
    __syncthreads();
    if (threadIdx.x == 0) *a.d_status = s_code;
}

// Whether token t is to be processed; a large batch's warps report its error themselves.
__device__ __forceinline__ bool admit(const AppendArgs& a, uint64_t t, int64_t slot, unsigned lane, bool report_here)
{
    const int code = token_error(a, t, slot);
    if (code != HP_OK && report_here && lane == 0) atomicMin(a.d_status, code);
    return slot >= 0 && code == HP_OK;
}

// The rotation of the 8 dimensions d0 .. d0 + 7 of token t: y_j = c_j x_j + s_j partner_j.
struct Turn {
    float c[8], s[8];
    bool on;      // these dimensions turn (else they stay as they are, infinities included)
    int partner;  // lanes to the partner's 8 dimensions; 0: pairs lie within the 8
    __device__ __forceinline__ void load(const RopeArgs& r, uint64_t tokens, uint64_t t, uint32_t d0)
    {
        partner = 0;
        on = d0 < r.rot;
        if (!on) {
#pragma unroll
            for (int j = 0; j < 8; ++j) c[j] = 1.0f, s[j] = 0.0f;
            return;
        }
        const uint32_t half = r.rot / 2;
        uint64_t pos[4];
#pragma unroll
        for (uint32_t x = 0; x < 4; ++x) pos[x] = x < r.axes ? position(r, tokens, x, t) : 0;
        const bool high = !r.inter && d0 >= half;
        if (!r.inter) partner = high ? -(int)(half / 8) : (int)(half / 8);
        if (r.axes == 1) {  // 16-byte pieces of the token's one row
            const float* row = r.cos_sin + pos[0] * r.rot;
            if (r.inter) {
                const float4 cv = load4(row + d0 / 2), sv = load4(row + half + d0 / 2);
                const float ce[4] = {cv.x, cv.y, cv.z, cv.w}, se[4] = {sv.x, sv.y, sv.z, sv.w};
#pragma unroll
                for (int j = 0; j < 8; ++j) c[j] = ce[j / 2], s[j] = (j & 1) == 0 ? -se[j / 2] : se[j / 2];
            } else {
                const float *cr = row + d0 - (high ? half : 0), *sr = cr + half;
                const float4 c0 = load4(cr), c1 = load4(cr + 4), s0 = load4(sr), s1 = load4(sr + 4);
                const float ce[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
                const float se[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
                for (int j = 0; j < 8; ++j) c[j] = ce[j], s[j] = high ? se[j] : -se[j];
            }
            return;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t i = r.inter ? (d0 + j) / 2 : d0 + j - (high ? half : 0);
            uint64_t p = pos[0];
#pragma unroll
            for (int x = 1; x < 4; ++x)
                if (i >= r.first[x]) p = pos[x];
            const float* row = r.cos_sin + p * r.rot;
            c[j] = row[i];
            const float sn = row[half + i];
            s[j] = (r.inter ? (j & 1) == 0 : !high) ? -sn : sn;
        }
    }
};

// 8 elements of the lane `from`, in this lane's place (whole warps).
template <typename T> __device__ __forceinline__ Vec8<T> shuffled(const Vec8<T>& v, int from)
{
    Vec8<T> r;
#pragma unroll
    for (int i = 0; i < Vec8<T>::N; ++i) {
        r.u[i].x = __shfl_sync(0xffffffffu, v.u[i].x, from);
        r.u[i].y = __shfl_sync(0xffffffffu, v.u[i].y, from);
        r.u[i].z = __shfl_sync(0xffffffffu, v.u[i].z, from);
        r.u[i].w = __shfl_sync(0xffffffffu, v.u[i].w, from);
    }
    return r;
}

// The partners y of the elements x of v (whole warps; `lane`: this lane's number).
template <typename T>
__device__ __forceinline__ void partners(const Turn& turn, bool inter, const Vec8<T>& v, unsigned lane,
                                         const float (&x)[8], float (&y)[8])
{
    if (inter) {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = x[j ^ 1];
    } else {
        shuffled(v, (int)lane + turn.partner).unpack(y);
    }
}

// x <- x c + y s; dimensions that do not turn keep x c, infinities included (all: every
// dimension turns)
__device__ __forceinline__ void turned(bool all, bool on, float (&x)[8], const float (&y)[8], const float (&c)[8],
                                       const float (&s)[8])
{
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float z = fmaf(y[j], s[j], x[j] * c[j]);
        x[j] = all || on ? z : x[j] * c[j];
    }
}

template <int L> __device__ __forceinline__ float group_sum(float v)
{
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Heads a lane group loads before it works on them: 2 KiB in flight per warp.
template <typename T> constexpr int kBatch = sizeof(T) == 2 ? 4 : 2;

template <typename T> struct Batch {
    Vec8<T> v[kBatch<T>];
    // heads h, h + step, ... of `count`, element d0 of the lane's at src + head * dim
    __device__ __forceinline__ void load(const T* src, uint32_t h, uint32_t step, uint32_t count, uint32_t dim, bool live)
    {
#pragma unroll
        for (int u = 0; u < kBatch<T>; ++u)
            if (live && h + u * step < count) v[u].load_rw(src + (uint64_t)(h + u * step) * dim);
    }
};

// The factors of a head's elements with the gains folded in: c_j w_j, and s_j w_partner.
template <typename T>
__device__ __forceinline__ void fold(const Turn& turn, bool inter, const T* weight, uint32_t d0, bool live, unsigned lane,
                                     float (&c)[8], float (&s)[8])
{
    float g[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) g[j] = 1.0f;
    if (live && weight) {
        Vec8<T> w;
        w.load(weight + d0);
        w.unpack(g);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float p = inter ? g[j ^ 1] : __shfl_sync(0xffffffffu, g[j], (int)lane + turn.partner);
        c[j] = turn.c[j] * g[j];
        s[j] = turn.s[j] * p;
    }
}

// Heads h0 + sub, + step, ... of `count` (h0 the same in the warp; the first batch is loaded):
// y_j = r (c_j x_j + s_j x_partner) with r the head's inverse root mean square where NORM.
template <typename T, int L, bool NORM>
__device__ __forceinline__ void heads_out(const AppendArgs& a, const Turn& turn, Batch<T>& b, const T* src, T* dst,
                                          uint32_t h0, uint32_t sub, uint32_t step, uint32_t count, bool live,
                                          unsigned lane, const float (&c)[8], const float (&s)[8])
{
    const bool inter = a.rope.inter, all = a.rope.rot == a.dim;
    const float inv_dim = 1.0f / (float)a.dim;
    while (h0 < count) {
#pragma unroll
        for (int u = 0; u < kBatch<T>; ++u, h0 += step) {
            if (h0 >= count) break;  // (the same in every lane)
            float x[8], y[8];
            b.v[u].unpack(x);
            partners(turn, inter, b.v[u], lane, x, y);
            float r = 1.0f;
            if (NORM) {
                float ss = 0.0f;
                if (live) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
                }
                r = rsqrtf(group_sum<L>(ss) * inv_dim + a.eps);
            }
            turned(all, turn.on, x, y, c, s);
            if (NORM)
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] *= r;
            b.v[u].pack(x);
            if (live && h0 + sub < count) b.v[u].store(dst + (uint64_t)(h0 + sub) * a.dim);
        }
        b.load(src, h0 + sub, step, count, a.dim, live);
    }
}

// Warp w of the grid takes token w / parts and, of its query, key and value heads each, every
// parts-th group of 32 / L.  A token's first queries are loaded before its slot and positions
// are looked at, so their latencies overlap.
template <typename T, int L>
__global__ void __launch_bounds__(kThreads, 3) qk_append_kernel(const AppendArgs a, uint32_t parts, bool report_here)
{
    pdl_wait();
    const unsigned extra = !report_here && a.d_status != nullptr;
    if (extra && blockIdx.x == 0) {
        report_all(a);
        return;
    }
    const unsigned lane = threadIdx.x & 31, sub = lane / L, l = lane % L;
    const uint64_t warps = (uint64_t)(gridDim.x - extra) * kWarpsRope;
    const uint32_t d0 = l * 8, step = parts * (32 / L);
    const bool live = d0 < a.dim, inter = a.rope.inter;
    for (uint64_t w = (uint64_t)(blockIdx.x - extra) * kWarpsRope + (threadIdx.x >> 5); w < a.tokens * parts;
         w += warps) {
        const uint64_t t = w / parts;
        const uint32_t h0 = (uint32_t)(w % parts) * (32 / L);
        const T* src = static_cast<const T*>(a.q) + t * a.q_stride + d0;
        Batch<T> b;
        b.load(src, h0 + sub, step, a.hq, a.dim, live);
        const int64_t slot = a.slot_map[t];
        if (!admit(a, t, slot, lane, report_here)) continue;
        Turn turn;
        turn.load(a.rope, a.tokens, t, live ? d0 : a.rope.rot);
        float c[8], s[8];
        fold(turn, inter, static_cast<const T*>(a.q_weight), d0, live, lane, c, s);
        T* dst = static_cast<T*>(a.q_out) + t * a.qo_stride + d0;
        if (a.q_weight) heads_out<T, L, true>(a, turn, b, src, dst, h0, sub, step, a.hq, live, lane, c, s);
        else heads_out<T, L, false>(a, turn, b, src, dst, h0, sub, step, a.hq, live, lane, c, s);
        const uint64_t row = (uint64_t)slot * a.hkv * a.dim + d0;
        src = static_cast<const T*>(a.k) + t * a.k_stride + d0;
        b.load(src, h0 + sub, step, a.hkv, a.dim, live);
        fold(turn, inter, static_cast<const T*>(a.k_weight), d0, live, lane, c, s);
        dst = static_cast<T*>(a.k_pool) + row;
        if (a.k_weight) heads_out<T, L, true>(a, turn, b, src, dst, h0, sub, step, a.hkv, live, lane, c, s);
        else heads_out<T, L, false>(a, turn, b, src, dst, h0, sub, step, a.hkv, live, lane, c, s);
        src = static_cast<const T*>(a.v) + t * a.v_stride + d0;
        dst = static_cast<T*>(a.v_pool) + row;
        for (uint32_t h = h0 + sub; h < a.hkv; h += kBatch<T> * step) {  // values keep their bits
            b.load(src, h, step, a.hkv, a.dim, live);
#pragma unroll
            for (int u = 0; u < kBatch<T>; ++u)
                if (live && h + u * step < a.hkv) b.v[u].store(dst + (uint64_t)(h + u * step) * a.dim);
        }
    }
}

// As above; part 0 of a token also takes its latent row (the whole warp, kLatVec vectors of 8
// elements a lane: latent_dim up to 256 kLatVec) and shared key.
template <typename T, int L, int kLatVec>
__global__ void __launch_bounds__(kThreads, 3) latent_append_kernel(const AppendArgs a, uint32_t parts, bool report_here)
{
    pdl_wait();
    const unsigned extra = !report_here && a.d_status != nullptr;
    if (extra && blockIdx.x == 0) {
        report_all(a);
        return;
    }
    constexpr int U = kBatch<T>;
    const unsigned lane = threadIdx.x & 31, sub = lane / L, l = lane % L;
    const uint64_t warps = (uint64_t)(gridDim.x - extra) * kWarpsRope;
    const uint32_t d0 = l * 8, R = a.latent_dim, D = a.rope.rot, step = parts * (32 / L);
    const bool live = d0 < D;
    for (uint64_t w = (uint64_t)(blockIdx.x - extra) * kWarpsRope + (threadIdx.x >> 5); w < a.tokens * parts;
         w += warps) {
        const uint64_t t = w / parts;
        const uint32_t part = (uint32_t)(w % parts);
        uint32_t h = part * (32 / L) + sub;
        Vec8<T> v[U], c[kLatVec], k;
        auto load = [&](int u, uint32_t hh) {
            if (live && hh < a.hq)
                v[u].load_rw(static_cast<const T*>(a.q) + t * a.q_stride + (uint64_t)hh * a.q_head + d0);
        };
#pragma unroll
        for (int u = 0; u < U; ++u) load(u, h + u * step);
        if (part == 0) {
            const T* src = static_cast<const T*>(a.latent) + t * a.latent_stride;
#pragma unroll
            for (int i = 0; i < kLatVec; ++i)
                if ((i * 32 + lane) * 8 < R) c[i].load(src + (i * 32 + lane) * 8);
            if (live && sub == 0) k.load(static_cast<const T*>(a.k) + t * a.k_stride + d0);
        }
        const int64_t slot = a.slot_map[t];
        if (!admit(a, t, slot, lane, report_here)) continue;
        Turn turn;
        turn.load(a.rope, a.tokens, t, live ? d0 : D);
        if (part == 0) {
            T* row = static_cast<T*>(a.k_pool) + (uint64_t)slot * (R + D);
            if (a.latent_weight) {
                float ss = 0.0f;
#pragma unroll
                for (int i = 0; i < kLatVec; ++i)
                    if ((i * 32 + lane) * 8 < R) {
                        float x[8];
                        c[i].unpack(x);
#pragma unroll
                        for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
                    }
                const float r = rsqrtf(group_sum<32>(ss) / (float)R + a.eps);
#pragma unroll
                for (int i = 0; i < kLatVec; ++i)
                    if ((i * 32 + lane) * 8 < R) {
                        float x[8], g[8];
                        Vec8<T> wv;
                        wv.load(static_cast<const T*>(a.latent_weight) + (i * 32 + lane) * 8);
                        c[i].unpack(x);
                        wv.unpack(g);
#pragma unroll
                        for (int j = 0; j < 8; ++j) x[j] = x[j] * r * g[j];
                        c[i].pack(x);
                    }
            }
#pragma unroll
            for (int i = 0; i < kLatVec; ++i)
                if ((i * 32 + lane) * 8 < R) c[i].store(row + (i * 32 + lane) * 8);
            float kx[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) kx[j] = 0.0f;
            if (live && sub == 0) k.unpack(kx);
            float ky[8];
            partners(turn, a.rope.inter, k, lane, kx, ky);
            turned(true, true, kx, ky, turn.c, turn.s);
            if (live && sub == 0) {
                k.pack(kx);
                k.store(row + R + d0);
            }
        }
        while (h - sub < a.hq) {
#pragma unroll
            for (int u = 0; u < U; ++u, h += step) {
                if (h - sub >= a.hq) break;  // (the same in every lane)
                const bool on = live && h < a.hq;
                float x[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = 0.0f;
                if (on) v[u].unpack(x);
                float y[8];
                partners(turn, a.rope.inter, v[u], lane, x, y);
                turned(true, true, x, y, turn.c, turn.s);
                if (on) {
                    v[u].pack(x);
                    v[u].store(static_cast<T*>(a.q_out) + t * a.qo_stride + (uint64_t)h * a.qo_head + d0);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) load(u, h + u * step);
        }
    }
}

// Warps per token: all the heads in one while that gives every SM 16 warps, else enough
// shares of a token to come near it.
template <typename T, int L, bool LATENT>
int launch_l(const AppendArgs& a, cudaStream_t st)
{
    int dev = 0;
    const int sms = current_sms(&dev);
    if (sms == 0) return HP_ERR_CUDA;
    const uint64_t groups = LATENT ? (a.hq + 32 / L - 1) / (32 / L)
                                   : (a.hq + 2 * a.hkv + 32 / L - 1) / (32 / L);
    const uint64_t want = ((uint64_t)sms * 16 + a.tokens - 1) / a.tokens;
    const uint64_t parts = want < 1 ? 1 : (want < groups ? want : (groups ? groups : 1));
    const uint64_t warps = a.tokens * parts, ctas = (warps + kWarpsRope - 1) / kWarpsRope;
    const uint64_t cap = (uint64_t)sms * 64;
    const uint64_t row = sizeof(T) * (LATENT ? 2ull * a.hq * a.dim + 2ull * (a.latent_dim + a.dim)
                                             : (2ull * a.hq + 4ull * a.hkv) * a.dim);  // read and written
    const bool report_here = a.d_status && a.tokens > kReportTokens && row < kReportBytes;
    if (report_here && cudaMemsetAsync(a.d_status, 0, sizeof(int), st) != cudaSuccess) return HP_ERR_CUDA;
    const unsigned grid = (unsigned)(ctas < cap ? ctas : cap) + (a.d_status && !report_here);
    // A dependent launch: the CTAs are there when the stream's last kernel ends, which each waits for
    // before it looks at memory.
    auto kernel = LATENT ? (a.latent_dim <= 512 ? latent_append_kernel<T, L, 2> : latent_append_kernel<T, L, 4>)
                         : qk_append_kernel<T, L>;
    return launch_dependent(kernel, grid, kThreads, 0, st, a, (uint32_t)parts, report_here) == cudaSuccess ? HP_OK
                                                                                                        : HP_ERR_CUDA;
}

template <typename T, bool LATENT>
int launch_d(uint32_t dim, const AppendArgs& a, cudaStream_t st)
{
    const uint32_t lanes = (dim + 7) / 8;
    if (lanes <= 8) return launch_l<T, 8, LATENT>(a, st);
    if (lanes <= 16) return launch_l<T, 16, LATENT>(a, st);
    return launch_l<T, 32, LATENT>(a, st);
}

template <bool LATENT>
int launch_append(uint32_t dtype, uint32_t dim, const AppendArgs& a, void* stream)
{
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    switch (dtype) {
    case HP_F32: return launch_d<float, LATENT>(dim, a, st);
    case HP_F16: return launch_d<__half, LATENT>(dim, a, st);
    default: return launch_d<__nv_bfloat16, LATENT>(dim, a, st);
    }
}

}  // namespace

int launch_qk_append(uint32_t dtype, const AppendArgs& a, void* stream)
{
    return launch_append<false>(dtype, a.dim, a, stream);
}

int launch_latent_append(uint32_t dtype, const AppendArgs& a, void* stream)
{
    return launch_append<true>(dtype, a.rope.rot, a, stream);
}

}  // namespace hp
