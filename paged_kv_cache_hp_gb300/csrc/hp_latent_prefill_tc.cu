// hp_latent_prefill_tc.cu -- the expanded form of latent attention on the tensor cores (tcgen05):
// latent_dim 512, rope_dim 64, nope_dim 128, v_dim 128.
//
// latent_expand_kernel: KV [rows, H * 256] = C [rows, 512] . W^T, a plain product.  Persistent
// CTAs, tiles of 128 x 256, eight 64-wide slices of the 512 through a ring of four stages (A 16
// KiB, B 32 KiB, TMA, 128-byte swizzled), two accumulators of 256 TMEM columns so that a tile's
// epilogue (TMEM -> registers -> shared memory -> bulk store, eight warps) overlaps the next
// tile's products.  The SM's reads bound it: 384 KiB a tile arrive at 49 bytes a cycle where the
// tensor pipe would take 94 (tiles of 256 x 256 read a third less and gain nothing, their
// epilogue standing between the tiles: 144 against 139 us at 21,000 rows and 32 heads).  A CTA's
// tiles are consecutive, so all the columns of a few row blocks are in flight at once and both
// operands come from L2.  KV goes to the workspace in blocks of 128 rows x 64 columns laid out as
// shared memory will hold them (head, row block, K0 K1 V0 V1), so that the attention below loads
// 16 KiB pieces with untiled bulk copies; the rope keys likewise (hp_latent.cu).  K and V are rounded
// to 16 bits there, as the attention's products take them (in 32 bits they would be twice the traffic and
// a product of split operands twice the time): against 64 bits the whole is off by 1.5 to 1.6 times
// what the result's own rounding is.
//
// latent_prefill_kernel: softmax(scale Q K^T) V for one head and 256 queries of a sequence, as
// two tiles of 128 queries that share the keys' 128-row blocks: K = [expanded 128 | rope 64], V =
// expanded 128.  Per tile and block:
//   S [128 x 128] = Q . K^T      12 products of K = 16, operands in shared memory
//   O [128 x 128] += P . V        8 products; P (16-bit) in TMEM over S, V N-major
// Two threads own a query's row of S, 64 scores each, all in registers: a barrier of the tile's 256
// threads says whether any score exceeds its row's reference maximum by more than 2^kTau (only
// then the two compare their maxima, and rescale half of the row of O each) and that P may
// overwrite S.  While one tile's softmax runs, the other tile's products do: the issue order is
// O0(j-1) S0(j) O1(j-1) S1(j), from one thread, whose products execute in order.  A round of 128 keys
// takes 3,600 cycles where its products need 2,640 (the S operands' reads fill shared memory's
// bandwidth): a tile's chain S 790, 380 until its threads know, softmax 1,500, 220 until the issuer
// knows, O 500.  One thread to a query took 3,900 (1,783 against 1,867 us at 21,000 tokens and 32
// heads); an issuing warp for each tile lets the two fall into step (1,996).  K and V pass through
// a ring of eight 16 KiB slots (128 keys x 64 dims).  Sequences are padded to 128 rows of zeros in
// the workspace (hp_latent.cu), so no block reads another sequence's rows.
//
// Every wait is bounded (about 2 s) and reports HP_ERR_TIMEOUT; operations in flight are waited
// for (bounded) before TMEM and shared memory go.
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

constexpr uint32_t kR = 512, kW = 576, kDn = 128, kDv = 128, kDq = 192, kKv = kDn + kDv;
constexpr uint32_t kSlot = 128 * 128;  // 128 rows x 64 dims
constexpr uint32_t kTmemCols = 512;

// ------------------------------------------------------------------------ expansion
constexpr uint32_t kGSlices = kR / 64;
constexpr int kGThreads = 10 * 32;  // warp 0 TMA, 1 products, 2-9 epilogue

constexpr uint32_t kGStages = 4, kGStage = 3 * kSlot;   // A 128 x 64, B 256 x 64
constexpr uint32_t kGOut = kGStages * kGStage;          // then 4 KiB for each epilogue warp
constexpr uint32_t kGSmem = kGOut + 8 * 4096 + 1024;

template <typename T>
__global__ void __launch_bounds__(kGThreads, 1)
    latent_expand_kernel(const LatentPrefillArgs a, const __grid_constant__ CUtensorMap tma_a,
                         const __grid_constant__ CUtensorMap tma_b)
{
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    __shared__ __align__(8) unsigned long long full[kGStages], freed[kGStages], t_full[2], t_free[2];
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag;
    pdl_wait();
    if (a.hdr->verdict != kVerdictOk) return;
    const unsigned warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t nt = a.H;  // column tiles: a head each
    const uint64_t rblocks = a.hdr->total_rows / 128;
    const uint64_t tiles = rblocks * nt;
    const uint64_t per = (tiles + gridDim.x - 1) / gridDim.x;
    const uint64_t beg = umin(blockIdx.x * per, tiles), end = umin(beg + per, tiles);
    if (beg >= end) return;
    const uint32_t sm0 = (smem_u32(smem_raw) + 1023u) & ~1023u;
    unsigned char* smem = smem_raw + (sm0 - smem_u32(smem_raw));
    if (threadIdx.x == 0) {
        for (uint32_t i = 0; i < kGStages; ++i) {
            mbar_init(smem_u32(&full[i]), 1);
            mbar_init(smem_u32(&freed[i]), 1);
        }
        for (uint32_t i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&t_full[i]), 1);
            mbar_init(smem_u32(&t_free[i]), 256);
        }
        abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 1) tmem_alloc(smem_u32(&tmem_base), kTmemCols);
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
    if (warp == 0) {
        if (lane == 0) {
            uint64_t i = 0;
            bool stop = false;
            for (uint64_t t = beg; t < end && !stop; ++t) {
                const int row = (int)(t / nt * 128), col = (int)(t % nt * kKv);
                for (uint32_t s = 0; s < kGSlices; ++s, ++i) {
                    const uint32_t st = (uint32_t)(i % kGStages), bar = smem_u32(&full[st]);
                    if (i >= kGStages && !wait_for(&freed[st], (uint32_t)((i / kGStages - 1) & 1))) {
                        stop = true;
                        break;
                    }
                    mbar_expect_tx(bar, kGStage);
                    const uint32_t d = sm0 + st * kGStage;
                    tma_2d(d, &tma_a, (int)(s * 64), row, bar);
                    tma_2d(d + kSlot, &tma_b, (int)(s * 64), col, bar);
                    tma_2d(d + 2 * kSlot, &tma_b, (int)(s * 64), col + 128, bar);
                }
            }
            for (uint64_t x = i > kGStages ? i - kGStages : 0; x < i; ++x)
                mbar_wait(smem_u32(&full[x % kGStages]), (uint32_t)((x / kGStages) & 1));
        }
        __syncwarp();
    } else if (warp == 1) {
        const uint32_t id = f16_idesc(a.bf16 != 0, false, false, 128, 256);
        const uint64_t ad0 = sw128_desc(sm0, 16, 1024), bd0 = sw128_desc(sm0 + kSlot, 16, 1024);
        uint64_t i = 0, n = 0;
        bool stop = false;
        for (uint64_t t = beg; t < end && !stop; ++t, ++n) {
            const uint32_t buf = (uint32_t)(n & 1);
            if (n >= 2 && !warp_wait(&t_free[buf], (uint32_t)((n / 2 - 1) & 1))) break;
            for (uint32_t s = 0; s < kGSlices; ++s, ++i) {
                const uint32_t st = (uint32_t)(i % kGStages);
                if (!warp_wait(&full[st], (uint32_t)((i / kGStages) & 1))) {
                    stop = true;
                    break;
                }
                fence_after();
                const uint64_t ad = ad0 + ((st * kGStage) >> 4), bd = bd0 + ((st * kGStage) >> 4);
                if (elect_one()) {
#pragma unroll
                    for (uint32_t kk = 0; kk < 4; ++kk)
                        mma_f16(tmem + buf * 256, ad + kk * 2, bd + kk * 2, id, s | kk);
                    mma_commit(smem_u32(&freed[st]));
                    if (s + 1 == kGSlices) mma_commit(smem_u32(&t_full[buf]));
                }
                __syncwarp();
            }
        }
        // every product issued has completed before the TMEM goes
        if (i) mbar_wait(smem_u32(&freed[(i - 1) % kGStages]), (uint32_t)(((i - 1) / kGStages) & 1));
    } else {
        // Epilogue: a warp takes 32 rows (its TMEM quarter) of two of the tile's 64-column pieces; a
        // piece's 32 rows lie 4 KiB together in the workspace's 16 KiB block, stored by the warp
        // alone.
        const uint32_t q4 = warp & 3, g = (warp - 2) >> 2, lane_addr = (q4 * 32) << 16;
        const uint32_t stage = kGOut + (warp - 2) * 4096;
        unsigned char* row = smem + stage + lane * 128;
        uint64_t n = 0;
        for (uint64_t t = beg; t < end; ++t, ++n) {
            const uint32_t buf = (uint32_t)(n & 1);
            if (!warp_wait(&t_full[buf], (uint32_t)((n / 2) & 1))) break;
            fence_after();
            char* out = static_cast<char*>(a.kv) + (t % nt * (a.cap_rows / 128) + t / nt) * 4 * kSlot + q4 * 4096;
#pragma unroll 1
            for (uint32_t c = 2 * g; c < 2 * g + 2; ++c) {
                uint32_t o[2][32];
                const uint32_t src = tmem + lane_addr + buf * 256 + c * 64;
                tmem_issue<32>(src, o[0]);
                tmem_issue<32>(src + 32, o[1]);
                tmem_wait<32>(o[0]);
                tmem_wait<32>(o[1]);
                // (the warp's last store has read the stage)
                if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
                __syncwarp();
                uint32_t spoilt = 0;
#pragma unroll
                for (uint32_t v = 0; v < 8; ++v) {
                    const uint32_t* e = o[v >> 2] + 8 * (v & 3);
                    uint4 w;
                    w.x = pack2<T>(__uint_as_float(e[0]), __uint_as_float(e[1]));
                    w.y = pack2<T>(__uint_as_float(e[2]), __uint_as_float(e[3]));
                    w.z = pack2<T>(__uint_as_float(e[4]), __uint_as_float(e[5]));
                    w.w = pack2<T>(__uint_as_float(e[6]), __uint_as_float(e[7]));
                    *reinterpret_cast<uint4*>(row + ((v ^ (lane & 7)) << 4)) = w;
                    spoilt |= spoilt_bits<T>(w.x) | spoilt_bits<T>(w.y) | spoilt_bits<T>(w.z) | spoilt_bits<T>(w.w);
                }
                if (spoilt) a.plan.ws.hdr->spoilt = 1;  // (of K as well: nothing but time)
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) bulk_store(out + c * kSlot, sm0 + stage, 4096, 0);
            }
            fence_before();
            mbar_arrive(smem_u32(&t_free[buf]));
        }
        if (lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
        __syncwarp();
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == 1) tmem_free(tmem, kTmemCols);
}

// ------------------------------------------------------------------------ attention
constexpr uint32_t kSlots = 8;
constexpr uint32_t kOffKv = 2 * 3 * kSlot;  // Q: two tiles of three 128 x 64 blocks
constexpr uint32_t kSmem = kOffKv + kSlots * kSlot + 1024;
constexpr uint32_t kSCol = 0, kOCol = 256;  // S (and P) of tile t at 128 t, O at 256 + 128 t
constexpr int kThreads = 18 * 32;           // warps 0-7 tile 0, 8-15 tile 1, 16 TMA, 17 products
constexpr int kTile = 256;                  // softmax threads of a tile: two to a query
constexpr float kTau = 8.0f;

// Values that meet zero weights have to be finite.  Of the rows from `first` on of a block of V in its two
// slots, which some query of the unit does not see, what is not finite becomes zero; true if there
// was any.  By the 256 threads of a tile, a row of 64 dims each.  Looked at where the expansion
// found such a value anywhere in the batch (in every call it cost 570 cycles of each of a unit's last
// three blocks: 2% of prompts of 2,000 tokens).
template <typename T>
__device__ __noinline__ bool clear_spoilt(unsigned char* slot0, unsigned char* slot1, uint32_t first)
{
    const uint32_t r = threadIdx.x & 127;
    unsigned char* row = (threadIdx.x & 128 ? slot1 : slot0) + r * 128;
    if (r < first) return false;
    uint32_t any = 0;
#pragma unroll
    for (uint32_t v = 0; v < 8; ++v) {  // (pieces in an order that keeps the banks apart)
        const uint4 x = *reinterpret_cast<const uint4*>(row + ((v ^ (r & 7)) << 4));
        any |= spoilt_bits<T>(x.x) | spoilt_bits<T>(x.y) | spoilt_bits<T>(x.z) | spoilt_bits<T>(x.w);
    }
    if (!any) return false;
    for (uint32_t v = 0; v < 8; ++v) {
        uint4* at = reinterpret_cast<uint4*>(row + (v << 4));
        *at = finite_only<T>(*at);
    }
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    return true;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 1)
    latent_prefill_kernel(const LatentPrefillArgs a, const __grid_constant__ CUtensorMap tmq)
{
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    __shared__ __align__(8) unsigned long long k_full[2], v_full[2], k_free[2], v_free[2], q_full[2],
        s_full[2], p_full[2], o_done[2], all_done;
    __shared__ uint32_t tmem_base;
    __shared__ int abort_flag, fail_s[2][2], spoilt;
    __shared__ float half_s[2][128];  // what a query's two threads tell each other
    pdl_wait();
    // everything the CTA needs to know, in one trip to memory (hp_latent.cu wrote the units, the
    // last queries of the batch first)
    const LatentUnit un = a.units[blockIdx.x % a.max_units];
    if (a.hdr->verdict != kVerdictOk || un.queries == 0) return;
    const bool look = a.hdr->spoilt != 0;
    const uint32_t h = (uint32_t)(blockIdx.x / a.max_units);
    const unsigned warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // blocks of 128 keys that each tile's last query reaches
    uint32_t nblk[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        const uint32_t q = un.queries > 128u * t ? (un.queries < 128u * t + 128 ? un.queries : 128u * t + 128) : 0;
        const int64_t seen = un.seen0 + (int64_t)q - 1;  // by the tile's last query
        nblk[t] = q && seen > 0 ? (uint32_t)((seen + 127) / 128) : 0;
    }
    const uint32_t blocks = nblk[0] > nblk[1] ? nblk[0] : nblk[1];

    const uint32_t sm0 = (smem_u32(smem_raw) + 1023u) & ~1023u;
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(smem_u32(&k_full[i]), 1);
            mbar_init(smem_u32(&v_full[i]), 1);
            mbar_init(smem_u32(&k_free[i]), 1);
            mbar_init(smem_u32(&v_free[i]), 1);
            mbar_init(smem_u32(&q_full[i]), 1);
            mbar_init(smem_u32(&s_full[i]), 1);
            mbar_init(smem_u32(&p_full[i]), kTile);
            fail_s[i][0] = fail_s[i][1] = 0;
            mbar_init(smem_u32(&o_done[i]), 1);
        }
        mbar_init(smem_u32(&all_done), 1);
        abort_flag = 0;
        spoilt = 0;
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
        if (lane == 0) {
            for (int t = 0; t < 2; ++t)
                if (nblk[t]) {
                    mbar_expect_tx(smem_u32(&q_full[t]), 3 * kSlot);
                    for (uint32_t c = 0; c < 3; ++c)
                        tma_2d(sm0 + (3 * t + c) * kSlot, &tmq, (int)(h * kDq + c * 64), (int)(un.q_row + 128 * t),
                               smem_u32(&q_full[t]));
                }
            const char* kv = static_cast<const char*>(a.kv) + (h * (a.cap_rows / 128) + un.block) * 4 * kSlot;
            const char* rope = static_cast<const char*>(a.rope_blocks) + un.block * kSlot;
            // Piece c = 5 j + i (K: 0, 1 expanded, 2 rope; V: 3, 4) goes to slot c mod 8, where piece
            // c - 8 was: K's first after the rope keys of block j - 2, its others after V of j - 2,
            // V after the first keys of j - 1.  One barrier for the three pieces of K, one for V.
            auto piece = [&](uint32_t j, uint32_t i, unsigned long long* bar) {
                if (a.test_stall && j == 0 && i == 0) return;
                bulk_load(sm0 + kOffKv + (5 * j + i) % kSlots * kSlot,
                          i == 2 ? rope + (uint64_t)j * kSlot : kv + ((uint64_t)j * 4 + (i < 2 ? i : i - 1)) * kSlot,
                          kSlot, smem_u32(bar));
            };
            uint32_t ka = 0, va = 0;  // blocks whose K, whose V barrier has been armed
            for (uint32_t j = 0; j < blocks; ++j) {
                unsigned long long *kb = &k_full[j & 1], *vb = &v_full[j & 1];
                if (j >= 2 && !wait_for(&k_free[j & 1], (j / 2 - 1) & 1)) break;
                mbar_expect_tx(smem_u32(kb), 3 * kSlot);
                ++ka;
                piece(j, 0, kb);
                if (j >= 2 && !wait_for(&v_free[j & 1], (j / 2 - 1) & 1)) break;
                piece(j, 1, kb);
                piece(j, 2, kb);
                if (j >= 1 && !wait_for(&k_free[(j - 1) & 1], ((j - 1) / 2) & 1)) break;
                mbar_expect_tx(smem_u32(vb), 2 * kSlot);
                ++va;
                piece(j, 3, vb);
                piece(j, 4, vb);
            }
            // the last loads land before the shared memory goes
            for (int t = 0; t < 2; ++t)
                if (nblk[t]) mbar_wait(smem_u32(&q_full[t]), 0);
            for (uint32_t x = ka > 2 ? ka - 2 : 0; x < ka; ++x) mbar_wait(smem_u32(&k_full[x & 1]), (x / 2) & 1);
            for (uint32_t x = va > 2 ? va - 2 : 0; x < va; ++x) mbar_wait(smem_u32(&v_full[x & 1]), (x / 2) & 1);
        }
        __syncwarp();
    } else if (warp == 17) {
        const uint32_t id_s = f16_idesc(a.bf16 != 0, false, false, 128, 128);
        const uint32_t id_o = f16_idesc(a.bf16 != 0, false, true, 128, 128);
        const uint32_t id_o64 = f16_idesc(a.bf16 != 0, false, true, 128, 64);
        const uint64_t qd0 = sw128_desc(sm0, 16, 1024), kd0 = sw128_desc(sm0 + kOffKv, 16, 1024);
        const uint64_t vd0 = sw128_desc(sm0 + kOffKv, kSlot, 1024);
        bool ok = true;
        for (int t = 0; t < 2; ++t)
            if (ok && nblk[t]) ok = warp_wait(&q_full[t], 0);
        // round j: O of block j - 1 and S of block j, tile after tile.  A wait costs some 200 cycles
        // even when its phase is complete, so each operand is waited for once a round, and where the
        // products issued before it are still running; V goes back before S of the second tile.
        for (uint32_t j = 0; j <= blocks && ok; ++j) {
            // the round's first polls together: each is a trip to shared memory and back
            bool v_ok = j == 0, p_ok = j == 0 || j - 1 >= nblk[0], k_ok = j >= blocks;
            if (!v_ok) v_ok = mbar_try_wait(smem_u32(&v_full[(j - 1) & 1]), ((j - 1) / 2) & 1);
            if (!k_ok) k_ok = mbar_test(smem_u32(&k_full[j & 1]), (j / 2) & 1);
            if (!p_ok) p_ok = mbar_try_wait(smem_u32(&p_full[0]), (j - 1) & 1);
            const unsigned polls = __reduce_and_sync(0xffffffffu, (v_ok ? 1u : 0u) | (k_ok ? 2u : 0u) | (p_ok ? 4u : 0u));
            if (!(polls & 1)) ok = warp_wait(&v_full[(j - 1) & 1], ((j - 1) / 2) & 1);
#pragma unroll
            for (int t = 0; t < 2; ++t) {
                const bool has_o = j > 0 && j - 1 < nblk[t], has_s = j < nblk[t];
                if (ok && has_o && (t == 1 || !(polls & 4))) ok = warp_wait(&p_full[t], (j - 1) & 1);
                if (!ok) break;
                fence_after();
                // V of block j - 1 is two slots of 64 dims: neighbours, but for the ring's last and first
                const uint32_t v0 = (5 * j - 2) % kSlots, pa = tmem + kSCol + t * 128, od = tmem + kOCol + t * 128;
                const uint32_t acc = j > 1, sd = tmem + kSCol + t * 128;
                const uint64_t vd = vd0 + ((v0 * kSlot) >> 4), qd = qd0 + ((3 * t * kSlot) >> 4);
                const uint64_t k0 = kd0 + ((((5 * j) % kSlots) * kSlot) >> 4);
                const uint64_t k1 = kd0 + ((((5 * j + 1) % kSlots) * kSlot) >> 4);
                const uint64_t k2 = kd0 + ((((5 * j + 2) % kSlots) * kSlot) >> 4);
                if (elect_one()) {
                    if (has_o) {
                        if (v0 + 1 < kSlots) {
#pragma unroll
                            for (uint32_t kk = 0; kk < 8; ++kk)
                                mma_f16_ts(od, pa + kk * 8, vd + ((kk * 2048) >> 4), id_o, acc | kk);
                        } else {
#pragma unroll
                            for (uint32_t kk = 0; kk < 8; ++kk) {
                                mma_f16_ts(od, pa + kk * 8, vd + ((kk * 2048) >> 4), id_o64, acc | kk);
                                mma_f16_ts(od + 64, pa + kk * 8, vd0 + ((kk * 2048) >> 4), id_o64, acc | kk);
                            }
                        }
                        if (j == nblk[t]) mma_commit(smem_u32(&o_done[t]));
                    }
                    if (t == 1 && j > 0) mma_commit(smem_u32(&v_free[(j - 1) & 1]));  // both tiles have read it
                }
                __syncwarp();
                if (t == 0 && !(polls & 2)) ok = warp_wait(&k_full[j & 1], (j / 2) & 1);
                if (!ok) break;
                fence_after();
                if (elect_one()) {
                    if (has_s) {
#pragma unroll
                        for (uint32_t kk = 0; kk < 4; ++kk) mma_f16(sd, qd + kk * 2, k0 + kk * 2, id_s, kk);
#pragma unroll
                        for (uint32_t kk = 0; kk < 4; ++kk)
                            mma_f16(sd, qd + (kSlot >> 4) + kk * 2, k1 + kk * 2, id_s, 1u);
#pragma unroll
                        for (uint32_t kk = 0; kk < 4; ++kk)
                            mma_f16(sd, qd + (2 * kSlot >> 4) + kk * 2, k2 + kk * 2, id_s, 1u);
                        mma_commit(smem_u32(&s_full[t]));
                    }
                    if (t == 1 && j < blocks) mma_commit(smem_u32(&k_free[j & 1]));
                }
                __syncwarp();
            }
        }
        // everything issued has completed before the TMEM goes: one more commit covers it
        if (elect_one()) mma_commit(smem_u32(&all_done));
        __syncwarp();
        mbar_wait(smem_u32(&all_done), 0);
    } else {
        const int t = warp >> 3;
        const uint32_t q4 = warp & 3, half = (warp >> 2) & 1, row = q4 * 32 + lane;
        const uint32_t sa = tmem + ((q4 * 32) << 16) + kSCol + t * 128;
        const uint32_t oa = tmem + ((q4 * 32) << 16) + kOCol + t * 128 + half * 64;
        float* const told = &half_s[t][row];  // the second one's value, then what the first made of it
        const uint32_t qi = 128 * t + row;  // query of the unit
        const bool real = qi < un.queries;
        const uint64_t vis = real && un.seen0 + qi > 0 ? (uint64_t)(un.seen0 + qi) : 0;
        const float qscale = a.scale * 1.4426950408889634f;
        const int64_t every = un.seen0 > 0 ? un.seen0 : 0;  // tokens that all queries of the unit see
        float m = -INFINITY, l = 0.0f;
        bool stop = false;
        for (uint32_t j = 0; j < nblk[t]; ++j) {
            // a wait that runs out marks its block; the tile's threads stop together, at the vote
            if (!warp_wait(&s_full[t], j & 1)) fail_s[t][j & 1] = 1;
            fence_after();
            uint32_t xr[2][32];
            tmem_issue<32>(sa + 64 * half, xr[0]);
            tmem_issue<32>(sa + 64 * half + 32, xr[1]);
            const uint64_t t0 = (uint64_t)j * 128 + 64 * half;
            const int lim = vis > t0 ? (int)umin(vis - t0, 64) : 0;
            const bool masked = __any_sync(0xffffffffu, lim < 64);
            tmem_wait<32>(xr[0]);
            tmem_wait<32>(xr[1]);
            // the largest scaled score: the extreme of the raw ones on the scale's side; a block that
            // ends or is masked inside takes scaled scores with -inf in the places not seen
            float mx = -INFINITY, qs = qscale;
            if (masked) qs = 1.0f;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float* x = reinterpret_cast<float*>(xr[c]);
                if (masked) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        x[i] = 32 * c + i < lim ? x[i] * qscale : -INFINITY;
                        mx = fmaxf(mx, x[i]);
                    }
                } else if (qscale >= 0.0f) {
                    float e0 = x[0], e1 = x[1];
#pragma unroll
                    for (int i = 2; i < 30; i += 4) {
                        e0 = max3(e0, x[i], x[i + 1]);
                        e1 = max3(e1, x[i + 2], x[i + 3]);
                    }
                    mx = fmaxf(mx, fmaxf(max3(e0, x[30], x[31]), e1) * qscale);
                } else {
                    float e0 = x[0], e1 = x[1];
#pragma unroll
                    for (int i = 2; i < 30; i += 4) {
                        e0 = min3(e0, x[i], x[i + 1]);
                        e1 = min3(e1, x[i + 2], x[i + 3]);
                    }
                    mx = fmaxf(mx, fminf(min3(e0, x[30], x[31]), e1) * qscale);
                }
            }
            // (past this barrier every thread of the tile has its scores, and P may overwrite them)
            if (half) *told = mx;
            fence_before();
            const bool need = named_or(1 + t, kTile, mx > m + kTau);
            fence_after();
            if (*(volatile int*)&fail_s[t][j & 1]) {
                stop = true;
                break;
            }
            if (need) {  // the same in the whole tile
                float mn;
                if (!half) *told = mn = fmaxf(m, fmaxf(mx, *told));
                named_sync(1 + t, kTile);
                if (half) mn = *told;
                const float f = m == -INFINITY ? 0.0f : exp2_approx(m - mn);
                m = mn;
                l *= f;
                if (j > 0) {  // the scores of this block are complete, so O of the last one is
#pragma unroll 1
                    for (uint32_t c = 0; c < 64; c += 16) {
                        uint32_t o[16];
                        tmem_issue<16>(oa + c, o);
                        tmem_wait<16>(o);
#pragma unroll
                        for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                        tmem_st16(oa + c, o);
                    }
                }
            }
            const float base = kWeightLift<T> - (m == -INFINITY ? 0.0f : m);
            const uint64_t qs2 = pair_of(qs, qs), base2 = pair_of(base, base);
            uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t p[16];
                const float* x = reinterpret_cast<const float*>(xr[c]);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    float2 w = of_pair(fma2(pair_of(x[2 * i], x[2 * i + 1]), qs2, base2));
                    w.x = exp2_approx(w.x);
                    w.y = exp2_approx(w.y);
                    sum[i & 1] = add2(sum[i & 1], pair_of(w.x, w.y));
                    p[i] = pack2<T>(w.x, w.y);
                }
                tmem_st16(sa + 32 * half + 16 * c, p);
            }
            const float2 sums = of_pair(add2(sum[0], sum[1]));
            l += sums.x + sums.y;
            tmem_st_wait();
            fence_before();
            // (the first tile's products of a block come first, so its threads look at V for both)
            if (look && (int64_t)(j + 1) * 128 > every && (t == 0 || j >= nblk[0]) &&
                warp_wait(&v_full[j & 1], (j / 2) & 1)) {
                const int64_t first = every - (int64_t)j * 128;
                unsigned char* kv = smem_raw + (sm0 - smem_u32(smem_raw)) + kOffKv;
                if (clear_spoilt<T>(kv + (5 * j + 3) % kSlots * kSlot, kv + (5 * j + 4) % kSlots * kSlot,
                                    first > 0 ? (uint32_t)first : 0u))
                    *(volatile int*)&spoilt = 1;
            }
            mbar_arrive(smem_u32(&p_full[t]));
        }
        if (!stop && nblk[t]) {
            const bool ok = warp_wait(&o_done[t], 0);
            if (half) *told = l;
            stop = !named_and(1 + t, kTile, ok);
            if (!half) *told = l += *told;
            named_sync(1 + t, kTile);
            if (half) l = *told;
            fence_after();
        }
        if (!stop) {
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
            uint4* o4 = reinterpret_cast<uint4*>(static_cast<T*>(a.out) + ((un.q_row + qi) * a.H + h) * kDv + half * 64);
#pragma unroll 1
            for (uint32_t c = 0; c < 64; c += 32) {
                uint32_t o[32];
                if (nblk[t]) {
                    tmem_issue<32>(oa + c, o);
                    tmem_wait<32>(o);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = 0u;
                }
                // what was cleared, for the queries that see it
                if (*(volatile int*)&spoilt)
                    for (int64_t k = every; k < (int64_t)vis; ++k) {
                        const char* v = static_cast<const char*>(a.kv) +
                                        ((h * (a.cap_rows / 128) + un.block + k / 128) * 4 + 2 + half) * kSlot + k % 128 * 128;
#pragma unroll
                        for (uint32_t p = 0; p < 4; ++p) {
                            const uint4 x = *reinterpret_cast<const uint4*>(v + (((c / 8 + p) ^ (uint32_t)(k & 7)) << 4));
                            const T* e = reinterpret_cast<const T*>(&x);
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                const float f = (float)e[i];
                                if (!isfinite(f)) o[8 * p + i] = __float_as_uint(__uint_as_float(o[8 * p + i]) + f);
                            }
                        }
                    }
                if (real) {
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        uint4 w;
                        uint32_t* wp = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            wp[e] = pack2<T>(__uint_as_float(o[8 * v + 2 * e]) * inv,
                                             __uint_as_float(o[8 * v + 2 * e + 1]) * inv);
                        o4[c / 8 + v] = w;
                    }
                }
            }
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    if (warp == 17) tmem_free(tmem, kTmemCols);
}

template <typename T>
int launch_t(const LatentPrefillArgs& a, cudaStream_t st)
{
    CUtensorMap ma, mb, mq;
    if (!map_2d(&ma, a.rows, a.cap_rows, kR, kR * 2, 128, a.bf16) ||
        !map_2d(&mb, a.w_kv, (uint64_t)a.H * kKv, kR, kR * 2, 128, a.bf16) ||
        !map_2d(&mq, a.q, a.total_q, (uint64_t)a.H * kDq, (uint64_t)a.H * kDq * 2, 128, a.bf16))
        return HP_ERR_CUDA;
    int dev = 0;
    const int sms = current_sms(&dev);
    if (sms == 0 || !allow_dynamic_smem<latent_expand_kernel<T>>(dev, (int)kGSmem) ||
        !allow_dynamic_smem<latent_prefill_kernel<T>>(dev, (int)kSmem))
        return HP_ERR_CUDA;
    const uint64_t tiles = a.cap_rows / 128 * a.H;
    const unsigned grid = (unsigned)(tiles < (uint64_t)sms ? tiles : (uint64_t)sms);
    if (launch_dependent(latent_expand_kernel<T>, grid, kGThreads, (size_t)kGSmem, st, a, ma, mb) != cudaSuccess)
        return HP_ERR_CUDA;
    return launch_dependent(latent_prefill_kernel<T>, (unsigned)(a.max_units * a.H), kThreads, (size_t)kSmem, st, a,
                            mq) == cudaSuccess
               ? HP_OK
               : HP_ERR_CUDA;
}

}  // namespace

bool latent_prefill_tc_fits(uint32_t latent_dim, uint64_t head_dim, uint32_t nope, uint32_t v,
                            uint64_t cap_rows, uint64_t total_q, uint32_t heads)
{
    return latent_dim == kR && head_dim == kW && nope == kDn && v == kDv && cap_rows > 0 &&
           cap_rows < (1ull << 31) && total_q < (1ull << 31) && 2 * total_q * heads < (1ull << 31);
}

int launch_latent_prefill_tc(const LatentPrefillArgs& a, void* stream)
{
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return a.bf16 ? launch_t<__nv_bfloat16>(a, st) : launch_t<__half>(a, st);
}

}  // namespace hp
