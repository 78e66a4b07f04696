// hp_step.cu -- the block tables of one serving step, from the requests' lengths.
//
// need_s = max(have_s, ceil((len_s + new_s) / P)); the grown slices lie at the exclusive prefix
// sums of need, the new tokens at those of new, and sequence s takes its new pages from the
// free list at prefix(need) - prefix(have), the latter being seq_ptr itself.  Every output is
// then a function of one entry or token index and these sums, whose sequence a binary search
// finds.  Bytes bound it for a large step, latency for a small one.
//
// A step of up to kFusedSeqs sequences and kFusedItems entries and tokens runs as one CTA with
// the sums in shared memory: one launch, and searches of 30 cycles a step instead of the L2's
// hundreds.  A larger one takes two kernels.  The scan's CTAs (up to kMaxBlocks, 1,024 sequences
// each, more where the sequences are more) leave sums local to their sequences, their totals and
// the first rule that failed; every CTA of the fill adds the totals up again (a load and a scan of
// at most 256 numbers), so nothing waits for a CTA, and writes nothing when a rule failed.  One
// CTA scanning 4,096 sequences took 12.6 us of a step's 24.
#include <cuda_runtime.h>

#include "hp_internal.cuh"
#include "hp_resolve.cuh"
#include "hp_scan.cuh"
#include "hp_step.cuh"

namespace hp {
namespace {

constexpr unsigned long long kMaxTokens = 1ull << 58;
constexpr uint32_t kFusedSeqs = 1024;
constexpr uint64_t kFusedItems = 16384;
constexpr uint32_t kStretch = 2560;        // sums a fill CTA keeps in shared memory
constexpr uint32_t kFillItems = 2048;      // entries or tokens of a fill CTA
constexpr uint32_t kMaxBlocks = kStepBlocks;

__device__ __forceinline__ unsigned long long page_of(const StepArgs& a, unsigned long long x)
{
    return a.div_ok && x < (1ull << 32) ? div_invariant((uint32_t)x, a.div_m, a.div_l) : x / a.d.page_size;
}

struct Sums {
    unsigned long long tok, pages, key;  // totals, and the verdict key of the sequences' own rules
};

// Exclusive prefix sums of the new tokens and pages over sequences s0 .. s1 - 1, at tok[s - s0] and
// pages[s - s0]; a CTA of kPlanThreads, the result the same in every thread.  KEEP: seq_ptr and
// seq_lens are left in sp_copy and len_copy.
template <typename IndexT, bool KEEP, typename SumT>
__device__ Sums scan_range(const StepArgs& a, uint64_t s0, uint64_t s1, SumT* tok, SumT* pages,
                           SumT* sp_copy = nullptr, unsigned long long* len_copy = nullptr)
{
    const IndexT* sp = static_cast<const IndexT*>(a.d.seq_ptr);
    const IndexT* lens = static_cast<const IndexT*>(a.d.seq_lens);
    const IndexT* nw = static_cast<const IndexT*>(a.d.new_lens);
    const unsigned long long most = sizeof(IndexT) == 4 ? 0xFFFFFFFFull : kMaxTokens;
    __shared__ unsigned long long s_key;
    if (threadIdx.x == 0) s_key = kVerdictOk;
    __syncthreads();
    unsigned long long ct = 0, cp = 0;  // sums before this round
    for (uint64_t base = s0; base < s1; base += kPlanThreads) {
        const uint64_t s = base + threadIdx.x;
        unsigned long long t = 0, p = 0;
        if (s < s1) {
            const unsigned long long lo = sp[s], hi = sp[s + 1], len = lens[s];
            t = nw[s];
            const unsigned long long end = len + t, have = hi - lo;
            if (lo > hi) {
                atomicMin(&s_key, verdict_key(kRankSeqPtrOrder, s));
            } else if (end < len || end > most || (len && page_of(a, len - 1) >= have)) {
                atomicMin(&s_key, verdict_key(kRankLen, s));
            } else {
                const unsigned long long want = end ? page_of(a, end - 1) + 1 : 0;
                p = want > have ? want : have;
            }
            if (KEEP) {
                sp_copy[s - s0] = (SumT)lo;
                len_copy[s - s0] = len;
            }
        }
        unsigned long long ex_t, ex_p, tot_t, tot_p;
        block_scan2(t, p, ex_t, ex_p, tot_t, tot_p);
        if (s < s1) {
            tok[s - s0] = (SumT)sat_add(ct, ex_t);
            pages[s - s0] = (SumT)sat_add(cp, ex_p);
        }
        ct = sat_add(ct, tot_t);
        cp = sat_add(cp, tot_p);
    }
    __syncthreads();
    return Sums{ct, cp, s_key};
}

// The verdict of the step, given all the sums and the ends of seq_ptr.
template <typename IndexT>
__device__ __forceinline__ unsigned long long verdict(const hp_step_desc& d, const Sums& all,
                                                      unsigned long long sp_first, unsigned long long sp_last)
{
    const unsigned long long most = sizeof(IndexT) == 4 ? 0xFFFFFFFFull : kMaxTokens;
    unsigned long long key = all.key;
    if (sp_first != 0) key = min(key, verdict_key(kRankSeqPtrStart, 0));
    if (sp_last != d.table_len) key = min(key, verdict_key(kRankSeqPtrEnd, d.num_seqs));
    // (with the rules above satisfied, the slices add up to table_len)
    if (all.pages > d.table_len && all.pages - d.table_len > d.num_free)
        key = min(key, verdict_key(kRankCapacity, 0));
    if (all.pages > d.table_cap || all.tok > d.token_cap || all.pages > most || all.tok > most)
        key = min(key, verdict_key(kRankOutSize, 0));
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

// The same by a whole warp over sums(0) .. sums(hi - 1), 32 at a time: 3 loads deep for 32,768.
template <typename F>
__device__ __forceinline__ uint64_t find_wide(F sums, uint64_t hi, uint64_t u, unsigned lane)
{
    uint64_t lo = 0;
    while (hi - lo > 1) {
        const uint64_t step = (hi - lo + 31) / 32, i = lo + lane * step;
        const unsigned below = __ballot_sync(0xffffffffu, i < hi && sums(i) <= u);
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

// Row t: the token at position pos of that sequence.  A page whose slots reach past 2^63 - 1 gives that
// number, which is in no pool (a product that wraps could name some other page's slot, or a padding row).
template <typename IndexT>
__device__ __forceinline__ void put_token(const StepArgs& a, uint64_t t, unsigned long long pos, unsigned long long lo,
                                          unsigned long long have, unsigned long long at)
{
    const unsigned long long j = page_of(a, pos), page = page_entry<IndexT>(a.d, lo, have, at, j);
    const unsigned long long slot = page * a.d.page_size + (pos - j * a.d.page_size);
    a.d.slot_map[t] = page < a.page_limit ? (int64_t)slot : INT64_MAX;
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
    const hp_step_desc& d = a.d;
    pdl_wait();
    const unsigned long long sp_first = static_cast<const IndexT*>(d.seq_ptr)[0];
    const unsigned long long sp_last = static_cast<const IndexT*>(d.seq_ptr)[d.num_seqs];
    const Sums all = scan_range<IndexT, true, uint32_t>(a, 0, d.num_seqs, tok, pages, sp, len);
    const unsigned long long key = verdict<IndexT>(d, all, sp_first, sp_last);
    if (threadIdx.x == 0 && a.d_status) *a.d_status = key_status(key);
    if (key != kVerdictOk) return;  // the same in every thread
    if (threadIdx.x == 0) {
        tok[d.num_seqs] = (uint32_t)all.tok;
        pages[d.num_seqs] = (uint32_t)all.pages;
        sp[d.num_seqs] = (uint32_t)sp_last;
    }
    __syncthreads();
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
    pdl_wait();
    const uint64_t s0 = (uint64_t)blockIdx.x << a.block_log, s1 = umin(s0 + (1ull << a.block_log), a.d.num_seqs);
    const Sums r = scan_range<IndexT, false, unsigned long long>(a, s0, s1, a.ws.rows_off + s0, a.ws.units_off + s0);
    if (threadIdx.x == 0) {
        a.blocks[blockIdx.x] = r.tok;
        a.blocks[kMaxBlocks + blockIdx.x] = r.pages;
        a.blocks[2 * kMaxBlocks + blockIdx.x] = r.key;
    }
}

// CTA b of the first entry_ctas takes table entries, the next token_ctas tokens, the others
// sequences.
template <typename IndexT>
__global__ void __launch_bounds__(256) step_fill_kernel(const StepArgs a, uint32_t blocks, uint64_t entry_ctas,
                                                        uint64_t token_ctas)
{
    __shared__ uint32_t part[kStretch + 1];
    __shared__ uint64_t s_lo, s_hi;
    __shared__ unsigned long long tok0[kMaxBlocks + 1], pages0[kMaxBlocks + 1], w_tok[8], w_pages[8], w_key[8];
    const hp_step_desc& d = a.d;
    const IndexT* sp = static_cast<const IndexT*>(d.seq_ptr);
    const IndexT* lens = static_cast<const IndexT*>(d.seq_lens);
    const uint64_t S = d.num_seqs;
    const unsigned lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    pdl_wait();
    // the sums before each block of sequences, the totals and the verdict: a block per thread
    const unsigned long long sp_first = sp[0], sp_last = sp[S];
    const bool mine = threadIdx.x < blocks;
    const unsigned long long bt = mine ? a.blocks[threadIdx.x] : 0;
    const unsigned long long bp = mine ? a.blocks[kMaxBlocks + threadIdx.x] : 0;
    unsigned long long it = bt, ip = bp, key = mine ? a.blocks[2 * kMaxBlocks + threadIdx.x] : kVerdictOk;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long nt = __shfl_up_sync(0xffffffffu, it, o), np = __shfl_up_sync(0xffffffffu, ip, o);
        if (lane >= (unsigned)o) {
            it = sat_add(nt, it);
            ip = sat_add(np, ip);
        }
        key = min(key, __shfl_xor_sync(0xffffffffu, key, o));
    }
    if (lane == 31) {
        w_tok[warp] = it;
        w_pages[warp] = ip;
        w_key[warp] = key;
    }
    __syncthreads();
    Sums all{0, 0, kVerdictOk};
    unsigned long long ct = 0, cp = 0;  // sums of the warps before this one
#pragma unroll
    for (unsigned w = 0; w < 8; ++w) {
        if (w == warp) {
            ct = all.tok;
            cp = all.pages;
        }
        all.tok = sat_add(all.tok, w_tok[w]);
        all.pages = sat_add(all.pages, w_pages[w]);
        all.key = min(all.key, w_key[w]);
    }
    if (mine) {  // (nothing saturates once the rules hold)
        tok0[threadIdx.x] = ct + it - bt;
        pages0[threadIdx.x] = cp + ip - bp;
    }
    __syncthreads();
    key = verdict<IndexT>(d, all, sp_first, sp_last);
    if (blockIdx.x == 0 && threadIdx.x == 0 && a.d_status) *a.d_status = key_status(key);
    if (key != kVerdictOk) return;  // the same in every thread
    auto tok_at = [&](uint64_t s) { return s < S ? tok0[s >> a.block_log] + a.ws.rows_off[s] : all.tok; };
    auto pages_at = [&](uint64_t s) { return s < S ? pages0[s >> a.block_log] + a.ws.units_off[s] : all.pages; };
    if (blockIdx.x >= entry_ctas + token_ctas) {
        const uint64_t s = (blockIdx.x - entry_ctas - token_ctas) * 256ull + threadIdx.x;
        if (s <= S) put_sequence<IndexT>(d, s, tok_at(s), pages_at(s));
        return;
    }
    const bool entries = blockIdx.x < entry_ctas;
    auto sums = [&](uint64_t s) { return entries ? pages_at(s) : tok_at(s); };
    const unsigned long long total = entries ? all.pages : all.tok;
    const uint64_t u0 = (entries ? blockIdx.x : blockIdx.x - entry_ctas) * (uint64_t)kFillItems;
    const uint64_t u1 = umin(u0 + kFillItems, total);
    if (u0 < u1) {  // the same in every thread
        if (warp == 0) {
            const uint64_t s = find_wide(sums, S, u0, lane);
            if (lane == 0) s_lo = s;
        } else if (warp == 1) {
            const uint64_t s = find_wide(sums, S, u1 - 1, lane);
            if (lane == 0) s_hi = s + 1;
        }
        __syncthreads();
    }
    const uint64_t lo = u0 < u1 ? s_lo : 0, hi = u0 < u1 ? s_hi : 0;
    const unsigned long long first_sum = u0 < u1 ? sums(lo) : 0;
    const bool near = hi - lo <= kStretch;
    if (near && u0 < u1) {  // the sums relative to u0; that of lo, which may lie before it, apart
        for (uint32_t i = threadIdx.x; i <= (uint32_t)(hi - lo); i += 256)
            part[i] = i == 0 ? 0u : (uint32_t)umin(sums(lo + i) - u0, 1u << 30);
        __syncthreads();
    }
#pragma unroll 4
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
            uint64_t l = lo, h = hi;
            while (h - l > 1) {
                const uint64_t mid = (l + h) >> 1;
                if (sums(mid) <= u) l = mid;
                else h = mid;
            }
            s = l;
            off = u - sums(s);
        }
        const unsigned long long first = sp[s], have = sp[s + 1] - first;
        if (entries)
            static_cast<IndexT*>(d.table_out)[u] = page_entry<IndexT>(d, first, have, u - off, off);
        else
            put_token<IndexT>(a, u, lens[s] + off, first, have, pages_at(s));
    }
}

template <typename IndexT>
int launch_t(const StepArgs& a, cudaStream_t st)
{
    const hp_step_desc& d = a.d;
    if (d.num_seqs <= kFusedSeqs && d.table_cap + d.token_cap <= kFusedItems) {
        // (a dependent launch, as the scan: there when the stream's last kernel ends, and waiting for it)
        return launch_dependent(step_fused_kernel<IndexT>, 1, kPlanThreads, 0, st, a) == cudaSuccess ? HP_OK
                                                                                                  : HP_ERR_CUDA;
    }
    const uint64_t ec = (d.table_cap + kFillItems - 1) / kFillItems, tc = (d.token_cap + kFillItems - 1) / kFillItems;
    const uint64_t grid = ec + tc + d.num_seqs / 256 + 1;
    StepArgs b = a;
    b.block_log = 10;
    while ((d.num_seqs >> b.block_log) >= kMaxBlocks) ++b.block_log;
    const unsigned blocks = (unsigned)(d.num_seqs >> b.block_log) + 1;
    if (launch_dependent(step_scan_kernel<IndexT>, blocks, kPlanThreads, 0, st, b) != cudaSuccess) return HP_ERR_CUDA;
    return launch_dependent(step_fill_kernel<IndexT>, (unsigned)grid, 256, 0, st, b, blocks, ec, tc) == cudaSuccess
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
