// hp_step.cu -- the block tables of one serving step, from the requests' lengths.
//
// need_s = max(have_s, ceil((len_s + new_s) / P)); the grown slices lie at the exclusive prefix
// sums of need, the new tokens at those of new, and sequence s takes its new pages from the
// free list at prefix(need) - prefix(have), the latter being seq_ptr itself.  Every output is
// then a function of one entry or token index and these sums: a scan by one CTA (four
// sequences per thread), which also applies every rule, and a fill that writes nothing when a
// rule failed and finds an entry's or token's sequence by a binary search of the sums.
//
// A step of up to kFusedSeqs sequences and kFusedItems entries and tokens runs as one CTA with
// the sums in shared memory: one launch, and searches of 30 cycles a step instead of the L2's
// hundreds.  A larger one spreads its fill over the GPU, 1024 entries or tokens per CTA, each CTA
// searching the stretch of sums that its own entries meet, copied to shared memory when it fits.
#include <cuda_runtime.h>

#include "hp_internal.cuh"
#include "hp_resolve.cuh"
#include "hp_scan.cuh"
#include "hp_step.cuh"

namespace hp {
namespace {

constexpr unsigned long long kMaxTokens = 1ull << 58;
constexpr int kPer = 4;                    // sequences per thread and chunk of the scan
constexpr uint32_t kFusedSeqs = 1024;
constexpr uint64_t kFusedItems = 16384;
constexpr uint32_t kStretch = 1536;        // sums a fill CTA keeps in shared memory
constexpr uint32_t kFillItems = 1024;      // entries or tokens of a fill CTA

__device__ __forceinline__ unsigned long long page_of(const StepArgs& a, unsigned long long x)
{
    return a.div_ok && x < (1ull << 32) ? div_invariant((uint32_t)x, a.div_m, a.div_l) : x / a.d.page_size;
}

// Prefix sums of the new tokens (tok) and pages, entries 0 .. S, and the verdict: one CTA of
// kPlanThreads.  KEEP: the inputs seq_ptr and seq_lens are left in sp_copy and len_copy.
template <typename IndexT, bool KEEP, typename SumT>
__device__ unsigned long long scan_step(const StepArgs& a, SumT* tok, SumT* pages, SumT* sp_copy = nullptr,
                                        unsigned long long* len_copy = nullptr)
{
    const hp_step_desc& d = a.d;
    const IndexT* sp = static_cast<const IndexT*>(d.seq_ptr);
    const IndexT* lens = static_cast<const IndexT*>(d.seq_lens);
    const IndexT* nw = static_cast<const IndexT*>(d.new_lens);
    const uint64_t S = d.num_seqs;
    const unsigned long long most = sizeof(IndexT) == 4 ? 0xFFFFFFFFull : kMaxTokens;
    __shared__ unsigned long long s_key;
    if (threadIdx.x == 0) s_key = kVerdictOk;
    __syncthreads();
    const unsigned long long sp_first = sp[0], sp_last = sp[S];
    unsigned long long ct = 0, cp = 0;  // sums before this chunk, the same in every thread
    for (uint64_t base = 0; base < S; base += kPlanThreads * kPer) {
        const uint64_t s0 = base + threadIdx.x * kPer;
        unsigned long long t[kPer], p[kPer], st = 0, sg = 0;
        unsigned long long lo[kPer + 1], len[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) t[i] = p[i] = len[i] = lo[i] = 0;
        if (base + (threadIdx.x & ~31u) * kPer < S) {  // warps past the last sequence only scan
#pragma unroll
            for (int i = 0; i <= kPer; ++i) lo[i] = s0 + i <= S ? (unsigned long long)sp[s0 + i] : 0;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                len[i] = s0 + i < S ? (unsigned long long)lens[s0 + i] : 0;
                t[i] = s0 + i < S ? (unsigned long long)nw[s0 + i] : 0;
            }
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                if (s0 + i < S) {
                    const unsigned long long end = len[i] + t[i], have = lo[i + 1] - lo[i];
                    if (lo[i] > lo[i + 1]) {
                        atomicMin(&s_key, verdict_key(kRankSeqPtrOrder, s0 + i));
                    } else if (end < len[i] || end > most || (len[i] && page_of(a, len[i] - 1) >= have)) {
                        atomicMin(&s_key, verdict_key(kRankLen, s0 + i));
                    } else {
                        const unsigned long long want = end ? page_of(a, end - 1) + 1 : 0;
                        p[i] = want > have ? want : have;
                    }
                }
                st = sat_add(st, t[i]);
                sg = sat_add(sg, p[i]);
            }
        }
        unsigned long long ex_t, ex_p, tot_t, tot_p;
        block_scan2(st, sg, ex_t, ex_p, tot_t, tot_p);
        ex_t = sat_add(ct, ex_t);
        ex_p = sat_add(cp, ex_p);
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (s0 + i < S) {
                tok[s0 + i] = (SumT)ex_t;
                pages[s0 + i] = (SumT)ex_p;
                if (KEEP) {
                    sp_copy[s0 + i] = (SumT)lo[i];
                    len_copy[s0 + i] = len[i];
                }
                ex_t = sat_add(ex_t, t[i]);
                ex_p = sat_add(ex_p, p[i]);
            }
        ct = sat_add(ct, tot_t);
        cp = sat_add(cp, tot_p);
    }
    __syncthreads();
    unsigned long long key = s_key;
    if (sp_first != 0) key = min(key, verdict_key(kRankSeqPtrStart, 0));
    if (sp_last != d.table_len) key = min(key, verdict_key(kRankSeqPtrEnd, S));
    // (with the rules above satisfied, the slices add up to table_len)
    if (cp > d.table_len && cp - d.table_len > d.num_free) key = min(key, verdict_key(kRankCapacity, 0));
    if (cp > d.table_cap || ct > d.token_cap || cp > most || ct > most)
        key = min(key, verdict_key(kRankOutSize, 0));
    if (threadIdx.x == 0) {
        tok[S] = (SumT)ct;
        pages[S] = (SumT)cp;
        if (KEEP) sp_copy[S] = (SumT)sp_last;
        if (a.d_status) *a.d_status = key_status(key);
    }
    return key;
}

// Largest s in [lo, hi) with sums[s] <= u, given sums[lo] <= u < sums[hi].
template <typename SumT, typename Int>
__device__ __forceinline__ Int find_in(const SumT* sums, Int lo, Int hi, SumT u)
{
    while (hi - lo > 1) {
        const Int mid = (lo + hi) >> 1;
        if (sums[mid] <= u) lo = mid;
        else hi = mid;
    }
    return lo;
}

// The same by a whole warp, 32 sums at a time: 3 loads deep for 32,768 sequences.
__device__ __forceinline__ uint64_t find_wide(const unsigned long long* sums, uint64_t hi, uint64_t u, unsigned lane)
{
    uint64_t lo = 0;
    while (hi - lo > 1) {
        const uint64_t step = (hi - lo + 31) / 32, i = lo + lane * step;
        const unsigned below = __ballot_sync(0xffffffffu, i < hi && sums[i] <= u);
        lo += (uint64_t)(31 - __clz(below)) * step;  // lane 0's sum is not above u
        hi = umin(hi, lo + step);
    }
    return lo;
}

// Page j of a sequence whose old slice is the `have` entries from `lo` and whose grown slice starts
// at entry `at`.
template <typename IndexT>
__device__ __forceinline__ IndexT page_entry(const hp_step_desc& d, unsigned long long lo, unsigned long long have,
                                             unsigned long long at, uint64_t j)
{
    return j < have ? static_cast<const IndexT*>(d.block_table)[lo + j]
                    : static_cast<const IndexT*>(d.free_pages)[at - lo + j - have];
}

// Row t: the token at position pos of that sequence.
template <typename IndexT>
__device__ __forceinline__ void put_token(const StepArgs& a, uint64_t t, unsigned long long pos, unsigned long long lo,
                                          unsigned long long have, unsigned long long at)
{
    const unsigned long long j = page_of(a, pos), page = page_entry<IndexT>(a.d, lo, have, at, j);
    a.d.slot_map[t] = (int64_t)(page * a.d.page_size + (pos - j * a.d.page_size));
    static_cast<IndexT*>(a.d.positions)[t] = (IndexT)pos;
}

template <typename IndexT>
__device__ __forceinline__ void put_none(const StepArgs& a, uint64_t t)
{
    a.d.slot_map[t] = -1;
    static_cast<IndexT*>(a.d.positions)[t] = 0;
}

// The sequences' own outputs; s <= S.
template <typename IndexT>
__device__ __forceinline__ void put_sequence(const hp_step_desc& d, uint64_t s, unsigned long long tok,
                                             unsigned long long pages)
{
    static_cast<IndexT*>(d.seq_ptr_out)[s] = (IndexT)pages;
    static_cast<IndexT*>(d.new_ptr_out)[s] = (IndexT)tok;
    if (s < d.num_seqs)
        static_cast<IndexT*>(d.lens_out)[s] = static_cast<const IndexT*>(d.seq_lens)[s] +
                                              static_cast<const IndexT*>(d.new_lens)[s];
    if (s == d.num_seqs && d.totals) {
        d.totals[0] = pages;
        d.totals[1] = tok;
        d.totals[2] = pages - d.table_len;
    }
}

template <typename IndexT>
__global__ void __launch_bounds__(kPlanThreads) step_fused_kernel(const StepArgs a)
{
    // (sums of at most kFusedItems once the rules hold: 32 bits)
    __shared__ uint32_t tok[kFusedSeqs + 1], pages[kFusedSeqs + 1], sp[kFusedSeqs + 1];
    __shared__ unsigned long long len[kFusedSeqs + 1];
    if (scan_step<IndexT, true, uint32_t>(a, tok, pages, sp, len) != kVerdictOk) return;  // the same in every thread
    __syncthreads();
    const hp_step_desc& d = a.d;
    const uint32_t S = (uint32_t)d.num_seqs, cap = (uint32_t)d.token_cap;
    const uint32_t tokens = tok[S], entries = pages[S];
    for (uint32_t s = threadIdx.x; s <= S; s += kPlanThreads) put_sequence<IndexT>(d, s, tok[s], pages[s]);
    for (uint32_t t = threadIdx.x; t < cap; t += kPlanThreads) {
        if (t >= tokens) {
            put_none<IndexT>(a, t);
        } else {
            const uint32_t s = find_in(tok, 0u, S, t);
            put_token<IndexT>(a, t, len[s] + (t - tok[s]), sp[s], sp[s + 1] - sp[s], pages[s]);
        }
    }
#pragma unroll 4
    for (uint32_t e = threadIdx.x; e < entries; e += kPlanThreads) {
        const uint32_t s = find_in(pages, 0u, S, e);
        static_cast<IndexT*>(d.table_out)[e] = page_entry<IndexT>(d, sp[s], sp[s + 1] - sp[s], pages[s], e - pages[s]);
    }
}

template <typename IndexT>
__global__ void __launch_bounds__(kPlanThreads) step_scan_kernel(const StepArgs a)
{
    pdl_trigger();
    const unsigned long long key = scan_step<IndexT, false, unsigned long long>(a, a.ws.rows_off, a.ws.units_off);
    if (threadIdx.x == 0) a.ws.hdr->verdict = key;
}

// CTA b of the first entry_ctas takes table entries, the others tokens and sequences.
template <typename IndexT>
__global__ void __launch_bounds__(256) step_fill_kernel(const StepArgs a, uint64_t entry_ctas, uint64_t token_ctas)
{
    __shared__ uint32_t part[kStretch + 1];
    __shared__ uint64_t s_lo, s_hi;
    pdl_wait();
    if (a.ws.hdr->verdict != kVerdictOk) return;
    const hp_step_desc& d = a.d;
    const IndexT* sp = static_cast<const IndexT*>(d.seq_ptr);
    const IndexT* lens = static_cast<const IndexT*>(d.seq_lens);
    const uint64_t S = d.num_seqs;
    if (blockIdx.x >= entry_ctas + token_ctas) {
        const uint64_t s = (blockIdx.x - entry_ctas - token_ctas) * 256ull + threadIdx.x;
        if (s <= S) put_sequence<IndexT>(d, s, a.ws.rows_off[s], a.ws.units_off[s]);
        return;
    }
    const bool entries = blockIdx.x < entry_ctas;
    const unsigned long long* sums = entries ? a.ws.units_off : a.ws.rows_off;
    const unsigned long long total = sums[S];
    const uint64_t u0 = (entries ? blockIdx.x : blockIdx.x - entry_ctas) * (uint64_t)kFillItems;
    const uint64_t u1 = umin(u0 + kFillItems, total);
    const unsigned lane = threadIdx.x & 31;
    if (u0 < u1) {  // the same in every thread
        if (threadIdx.x < 32) {
            const uint64_t s = find_wide(sums, S, u0, lane);
            if (lane == 0) s_lo = s;
        } else if (threadIdx.x < 64) {
            const uint64_t s = find_wide(sums, S, u1 - 1, lane);
            if (lane == 0) s_hi = s + 1;
        }
        __syncthreads();
    }
    const uint64_t lo = u0 < u1 ? s_lo : 0, hi = u0 < u1 ? s_hi : 0;
    const unsigned long long first_sum = u0 < u1 ? sums[lo] : 0;
    const bool near = hi - lo <= kStretch;
    if (near && u0 < u1) {  // the sums relative to u0; that of lo, which may lie before it, apart
        for (uint32_t i = threadIdx.x; i <= (uint32_t)(hi - lo); i += 256)
            part[i] = i == 0 ? 0u : (uint32_t)umin(sums[lo + i] - u0, 1u << 30);
        __syncthreads();
    }
#pragma unroll
    for (uint32_t i = 0; i < kFillItems; i += 256) {
        const uint32_t x = i + threadIdx.x;
        const uint64_t u = u0 + x;
        if (u >= u1) {
            if (!entries && u < d.token_cap) put_none<IndexT>(a, u);
            continue;
        }
        uint64_t s, off;
        if (near) {
            const uint32_t r = find_in(part, 0u, (uint32_t)(hi - lo), x);
            s = lo + r;
            off = r == 0 ? u - first_sum : x - part[r];
        } else {
            s = find_in(sums, lo, hi, (unsigned long long)u);
            off = u - sums[s];
        }
        const unsigned long long first = sp[s], have = sp[s + 1] - first;
        if (entries)
            static_cast<IndexT*>(d.table_out)[u] = page_entry<IndexT>(d, first, have, u - off, off);
        else
            put_token<IndexT>(a, u, lens[s] + off, first, have, a.ws.units_off[s]);
    }
}

template <typename IndexT>
int launch_t(const StepArgs& a, cudaStream_t st)
{
    const hp_step_desc& d = a.d;
    if (d.num_seqs <= kFusedSeqs && d.table_cap + d.token_cap <= kFusedItems) {
        step_fused_kernel<IndexT><<<1, kPlanThreads, 0, st>>>(a);
        return cudaGetLastError() == cudaSuccess ? HP_OK : HP_ERR_CUDA;
    }
    const uint64_t ec = (d.table_cap + kFillItems - 1) / kFillItems, tc = (d.token_cap + kFillItems - 1) / kFillItems;
    const uint64_t grid = ec + tc + d.num_seqs / 256 + 1;
    if (grid >= (1ull << 31)) return HP_ERR_OVERFLOW;
    step_scan_kernel<IndexT><<<1, kPlanThreads, 0, st>>>(a);
    if (cudaGetLastError() != cudaSuccess) return HP_ERR_CUDA;
    return launch_dependent(step_fill_kernel<IndexT>, (unsigned)grid, 256, 0, st, a, ec, tc) == cudaSuccess
               ? HP_OK
               : HP_ERR_CUDA;
}

}  // namespace

int launch_step_tables(const StepArgs& a, void* stream)
{
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return a.d.index_type == HP_IDX_U64 ? launch_t<unsigned long long>(a, st)
                                        : launch_t<unsigned int>(a, st);
}

}  // namespace hp
