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
// Errors come from one extra CTA that looks at every token's slot and positions and stores the
// first error (or HP_OK); the others skip the tokens it names.  So *d_status costs no launch of
// its own and does not depend on the order of the CTAs.
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

// 8 elements in 16-byte pieces
template <typename T> struct Vec8 {
    static constexpr int N = 8 * sizeof(T) / 16;
    uint4 u[N];
    __device__ __forceinline__ void load(const T* p)
    {
#pragma unroll
        for (int i = 0; i < N; ++i) u[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
    }
    // (q_out may be q: such loads bypass the read-only path)
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

// HP_OK, or why token t is not processed (a padding token: HP_OK, by its slot).
__device__ __forceinline__ int token_error(const AppendArgs& a, uint64_t t)
{
    const int64_t slot = a.slot_map[t];
    if (slot < 0) return HP_OK;
    if ((uint64_t)slot >= a.num_slots) return HP_ERR_PAGE_ID;
    if (a.rope.rot)
        for (uint32_t x = 0; x < a.rope.axes; ++x)
            if (position(a.rope, a.tokens, x, t) >= a.rope.max_pos) return HP_ERR_LEN;
    return HP_OK;
}

// The extra CTA: the first token with an error, its code.
__device__ __forceinline__ void report_first(const AppendArgs& a)
{
    __shared__ unsigned long long s_first;
    if (threadIdx.x == 0) s_first = ~0ull;
    __syncthreads();
    for (uint64_t t = threadIdx.x; t < a.tokens; t += kThreads)
        if (token_error(a, t) != HP_OK) {
            atomicMin(&s_first, (unsigned long long)t);
            break;  // t only grows
        }
    __syncthreads();
    if (threadIdx.x == 0) *a.d_status = s_first == ~0ull ? HP_OK : token_error(a, s_first);
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
        if (!on) return;
        const uint32_t half = r.rot / 2;
        uint64_t pos[4];
#pragma unroll
        for (uint32_t x = 0; x < 4; ++x) pos[x] = x < r.axes ? position(r, tokens, x, t) : 0;
        const bool high = !r.inter && d0 >= half;
        if (!r.inter) partner = high ? -(int)(half / 8) : (int)(half / 8);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const uint32_t i = r.inter ? (d0 + j) / 2 : d0 + j - (high ? half : 0);
            uint64_t p = pos[0];
#pragma unroll
            for (int x = 1; x < 4; ++x)
                if (i >= r.first[x]) p = pos[x];
            const float* row = r.cos_sin + p * r.rot;
            c[j] = __ldg(row + i);
            const float sn = __ldg(row + half + i);
            s[j] = (r.inter ? (j & 1) == 0 : !high) ? -sn : sn;
        }
    }
    // every lane of the warp calls it; lane: this lane's number
    __device__ __forceinline__ void apply(float (&x)[8], bool inter, unsigned lane) const
    {
        float y[8];
        if (inter) {
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = x[j ^ 1];
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = __shfl_sync(0xffffffffu, x[j], (int)lane + partner);
        }
        if (on)
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = x[j] * c[j] + y[j] * s[j];
    }
};

template <int L> __device__ __forceinline__ float group_sum(float v)
{
#pragma unroll
    for (int o = L / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Warp w of the grid takes token w / parts and, of its heads (queries, keys, values in that
// order), every parts-th group of 32 / L.
template <typename T, int L>
__global__ void __launch_bounds__(kThreads) qk_append_kernel(const AppendArgs a, uint32_t parts)
{
    if (a.d_status && blockIdx.x == gridDim.x - 1) {
        report_first(a);
        return;
    }
    const unsigned lane = threadIdx.x & 31, sub = lane / L, l = lane % L;
    const uint64_t warps = (uint64_t)(gridDim.x - (a.d_status != nullptr)) * kWarpsRope;
    const uint32_t heads = a.hq + 2 * a.hkv, d0 = l * 8;
    const bool live = d0 < a.dim;
    float qw[8], kw[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) qw[j] = kw[j] = 1.0f;
    if (live && a.q_weight) {
        Vec8<T> v;
        v.load(static_cast<const T*>(a.q_weight) + d0);
        v.unpack(qw);
    }
    if (live && a.k_weight) {
        Vec8<T> v;
        v.load(static_cast<const T*>(a.k_weight) + d0);
        v.unpack(kw);
    }
    for (uint64_t w = (uint64_t)blockIdx.x * kWarpsRope + (threadIdx.x >> 5); w < a.tokens * parts;
         w += warps) {
        const uint64_t t = w / parts;
        const int64_t slot = a.slot_map[t];
        if (slot < 0 || token_error(a, t) != HP_OK) continue;
        Turn turn;
        turn.load(a.rope, a.tokens, t, live ? d0 : a.rope.rot);
        for (uint32_t h0 = (uint32_t)(w % parts) * (32 / L); h0 < heads; h0 += parts * (32 / L)) {
            const uint32_t h = h0 + sub;
            const bool on = live && h < heads;
            const bool is_q = h < a.hq, is_k = !is_q && h < a.hq + a.hkv;
            const uint32_t g = is_q ? h : (is_k ? h - a.hq : h - a.hq - a.hkv);  // head of its kind
            const T* src = static_cast<const T*>(is_q ? a.q : (is_k ? a.k : a.v)) +
                           t * (is_q ? a.q_stride : (is_k ? a.k_stride : a.v_stride)) +
                           (uint64_t)g * a.dim + d0;
            Vec8<T> v;
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = 0.0f;
            if (on) {
                v.load_rw(src);
                v.unpack(x);
            }
            const bool norm = is_q ? a.q_weight != nullptr : a.k_weight != nullptr;
            float ss = 0.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
            ss = group_sum<L>(ss);
            const float r = norm ? rsqrtf(ss / (float)a.dim + a.eps) : 1.0f;
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = x[j] * r * (is_q ? qw[j] : kw[j]);
            turn.apply(x, a.rope.inter, lane);
            if (!on) continue;
            if (is_q) {
                v.pack(x);
                v.store(static_cast<T*>(a.q_out) + t * a.qo_stride + (uint64_t)g * a.dim + d0);
            } else {
                if (is_k) v.pack(x);  // a value keeps its bits
                v.store(static_cast<T*>(is_k ? a.k_pool : a.v_pool) +
                        ((uint64_t)slot * a.hkv + g) * a.dim + d0);
            }
        }
    }
}

constexpr int kLatVec = 4;  // 32 lanes x 8 elements x 4: latent vectors up to 1024

// As above; part 0 of a token also takes its latent row (the whole warp) and shared key.
template <typename T, int L>
__global__ void __launch_bounds__(kThreads) latent_append_kernel(const AppendArgs a, uint32_t parts)
{
    if (a.d_status && blockIdx.x == gridDim.x - 1) {
        report_first(a);
        return;
    }
    const unsigned lane = threadIdx.x & 31, sub = lane / L, l = lane % L;
    const uint64_t warps = (uint64_t)(gridDim.x - (a.d_status != nullptr)) * kWarpsRope;
    const uint32_t d0 = l * 8, R = a.latent_dim, D = a.rope.rot;
    const bool live = d0 < D;
    for (uint64_t w = (uint64_t)blockIdx.x * kWarpsRope + (threadIdx.x >> 5); w < a.tokens * parts;
         w += warps) {
        const uint64_t t = w / parts;
        const uint32_t part = (uint32_t)(w % parts);
        const int64_t slot = a.slot_map[t];
        if (slot < 0 || token_error(a, t) != HP_OK) continue;
        Turn turn;
        turn.load(a.rope, a.tokens, t, live ? d0 : D);
        if (part == 0) {
            T* row = static_cast<T*>(a.k_pool) + (uint64_t)slot * (R + D);
            const T* src = static_cast<const T*>(a.latent) + t * a.latent_stride;
            Vec8<T> v[kLatVec], k;
            float ss = 0.0f;
#pragma unroll
            for (int i = 0; i < kLatVec; ++i) {
                const uint32_t d = (i * 32 + lane) * 8;
                if (d < R) v[i].load(src + d);
            }
            float kx[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) kx[j] = 0.0f;
            if (live && sub == 0) {
                k.load(static_cast<const T*>(a.k) + t * a.k_stride + d0);
                k.unpack(kx);
            }
#pragma unroll
            for (int i = 0; i < kLatVec; ++i)
                if ((i * 32 + lane) * 8 < R) {
                    float x[8];
                    v[i].unpack(x);
#pragma unroll
                    for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
                }
            ss = group_sum<32>(ss);
            const float r = a.latent_weight ? rsqrtf(ss / (float)R + a.eps) : 1.0f;
#pragma unroll
            for (int i = 0; i < kLatVec; ++i) {
                const uint32_t d = (i * 32 + lane) * 8;
                if (d < R) {
                    if (a.latent_weight) {
                        float x[8], g[8];
                        Vec8<T> wv;
                        wv.load(static_cast<const T*>(a.latent_weight) + d);
                        v[i].unpack(x);
                        wv.unpack(g);
#pragma unroll
                        for (int j = 0; j < 8; ++j) x[j] = x[j] * r * g[j];
                        v[i].pack(x);
                    }
                    v[i].store(row + d);
                }
            }
            turn.apply(kx, a.rope.inter, lane);
            if (live && sub == 0) {
                k.pack(kx);
                k.store(row + R + d0);
            }
        }
        for (uint32_t h0 = part * (32 / L); h0 < a.hq; h0 += parts * (32 / L)) {
            const uint32_t h = h0 + sub;
            const bool on = live && h < a.hq;
            Vec8<T> v;
            float x[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) x[j] = 0.0f;
            if (on) {
                v.load_rw(static_cast<const T*>(a.q) + t * a.q_stride + (uint64_t)h * a.q_head + d0);
                v.unpack(x);
            }
            turn.apply(x, a.rope.inter, lane);
            if (on) {
                v.pack(x);
                v.store(static_cast<T*>(a.q_out) + t * a.qo_stride + (uint64_t)h * a.qo_head + d0);
            }
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
    const uint64_t cap = (uint64_t)sms * 8;
    const unsigned grid = (unsigned)(ctas < cap ? ctas : cap) + (a.d_status != nullptr);
    if (LATENT)
        latent_append_kernel<T, L><<<grid, kThreads, 0, st>>>(a, (uint32_t)parts);
    else
        qk_append_kernel<T, L><<<grid, kThreads, 0, st>>>(a, (uint32_t)parts);
    return cudaGetLastError() == cudaSuccess ? HP_OK : HP_ERR_CUDA;
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
