// hp_step.cu -- the block tables of one serving step, from the requests' lengths.
//
// need_s = max(have_s, ceil((len_s + new_s) / P)); the grown slices lie at the exclusive prefix
// sums of need, the new tokens at those of new, and sequence s takes its new pages from the
// free list at prefix(need) - prefix(have), the latter being seq_ptr itself.  Every output is
// then a function of one entry or token index and these sums, so two kernels do it: a scan by
// one CTA, which also applies every rule, and a fill by the whole grid that writes nothing
// when a rule failed.
#include <cuda_runtime.h>

#include "hp_internal.cuh"
#include "hp_resolve.cuh"
#include "hp_scan.cuh"
#include "hp_step.cuh"

namespace hp {
namespace {

constexpr unsigned long long kMaxTokens = 1ull << 58;

template <typename IndexT>
__global__ void __launch_bounds__(kPlanThreads) step_scan_kernel(const StepArgs a)
{
    const hp_step_desc& d = a.d;
    const IndexT* sp = static_cast<const IndexT*>(d.seq_ptr);
    const IndexT* lens = static_cast<const IndexT*>(d.seq_lens);
    const IndexT* nw = static_cast<const IndexT*>(d.new_lens);
    const uint64_t S = d.num_seqs, P = d.page_size;
    const unsigned long long most = sizeof(IndexT) == 4 ? 0xFFFFFFFFull : kMaxTokens;
    __shared__ unsigned long long s_key, s_tok, s_pages;
    pdl_trigger();
    if (threadIdx.x == 0) {
        s_key = kVerdictOk;
        s_tok = s_pages = 0;
    }
    __syncthreads();
    for (uint64_t base = 0; base < S; base += kPlanThreads) {
        const uint64_t s = base + threadIdx.x;
        unsigned long long tok = 0, pages = 0;
        if (s < S) {
            const unsigned long long lo = sp[s], hi = sp[s + 1], len = lens[s];
            tok = nw[s];
            const unsigned long long end = len + tok;
            if (lo > hi) {
                atomicMin(&s_key, verdict_key(kRankSeqPtrOrder, s));
            } else if (end < len || end > most || len / P + (len % P != 0) > hi - lo) {
                atomicMin(&s_key, verdict_key(kRankLen, s));
            } else {
                const unsigned long long want = end / P + (end % P != 0);
                pages = want > hi - lo ? want : hi - lo;
            }
        }
        unsigned long long ex_t, ex_p, tot_t, tot_p;
        block_scan2(tok, pages, ex_t, ex_p, tot_t, tot_p);
        const unsigned long long ct = s_tok, cp = s_pages;
        if (s < S) {
            a.ws.rows_off[s] = sat_add(ct, ex_t);
            a.ws.units_off[s] = sat_add(cp, ex_p);
        }
        __syncthreads();
        if (threadIdx.x == 0) {
            s_tok = sat_add(ct, tot_t);
            s_pages = sat_add(cp, tot_p);
        }
        __syncthreads();
    }
    if (threadIdx.x == 0) {
        unsigned long long key = s_key;
        if (sp[0] != 0) key = min(key, verdict_key(kRankSeqPtrStart, 0));
        if ((unsigned long long)sp[S] != d.table_len) key = min(key, verdict_key(kRankSeqPtrEnd, S));
        // (with the rules above satisfied, the slices add up to table_len)
        if (s_pages > d.table_len && s_pages - d.table_len > d.num_free)
            key = min(key, verdict_key(kRankCapacity, 0));
        if (s_pages > d.table_cap || s_tok > d.token_cap || s_pages > most || s_tok > most)
            key = min(key, verdict_key(kRankOutSize, 0));
        a.ws.rows_off[S] = s_tok;
        a.ws.units_off[S] = s_pages;
        a.ws.hdr->total_rows = s_tok;
        a.ws.hdr->total_units = s_pages;
        a.ws.hdr->verdict = key;
        if (a.d_status) *a.d_status = key_status(key);
    }
}

// One table entry, token or sequence per thread, grid-stride; the sequence of an entry or
// token by a binary search of its prefix sums.
template <typename IndexT>
__global__ void __launch_bounds__(256) step_fill_kernel(const StepArgs a)
{
    pdl_wait();
    if (a.ws.hdr->verdict != kVerdictOk) return;
    const hp_step_desc& d = a.d;
    const IndexT* sp = static_cast<const IndexT*>(d.seq_ptr);
    const IndexT* lens = static_cast<const IndexT*>(d.seq_lens);
    const IndexT* nw = static_cast<const IndexT*>(d.new_lens);
    const IndexT* old = static_cast<const IndexT*>(d.block_table);
    const IndexT* fr = static_cast<const IndexT*>(d.free_pages);
    IndexT* pos_out = static_cast<IndexT*>(d.positions);
    const uint64_t S = d.num_seqs, P = d.page_size;
    const unsigned long long tokens = a.ws.hdr->total_rows, pages = a.ws.hdr->total_units;
    const uint64_t first = (uint64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const uint64_t stride = (uint64_t)gridDim.x * blockDim.x;
    for (uint64_t e = first; e < pages; e += stride) {
        const uint64_t s = find_seq(a.ws.units_off, S, e);
        const unsigned long long lo = sp[s], have = sp[s + 1] - lo, at = a.ws.units_off[s];
        const uint64_t j = e - at;
        static_cast<IndexT*>(d.table_out)[e] = j < have ? old[lo + j] : fr[at - lo + j - have];
    }
    for (uint64_t t = first; t < d.token_cap; t += stride) {
        if (t >= tokens) {
            d.slot_map[t] = -1;
            pos_out[t] = 0;
            continue;
        }
        const uint64_t s = find_seq(a.ws.rows_off, S, t);
        const unsigned long long pos = lens[s] + (t - a.ws.rows_off[s]);
        const unsigned long long lo = sp[s], have = sp[s + 1] - lo, j = pos / P;
        const unsigned long long page = j < have ? old[lo + j] : fr[a.ws.units_off[s] - lo + j - have];
        d.slot_map[t] = (int64_t)(page * P + pos % P);
        pos_out[t] = (IndexT)pos;
    }
    for (uint64_t s = first; s <= S; s += stride) {
        static_cast<IndexT*>(d.seq_ptr_out)[s] = (IndexT)a.ws.units_off[s];
        static_cast<IndexT*>(d.new_ptr_out)[s] = (IndexT)a.ws.rows_off[s];
        if (s < S) static_cast<IndexT*>(d.lens_out)[s] = (IndexT)(lens[s] + nw[s]);
        if (s == S && d.totals) {
            d.totals[0] = pages;
            d.totals[1] = tokens;
            d.totals[2] = pages - d.table_len;
        }
    }
}

template <typename IndexT>
int launch_t(const StepArgs& a, cudaStream_t st)
{
    int dev = 0;
    const int sms = current_sms(&dev);
    if (sms == 0) return HP_ERR_CUDA;
    step_scan_kernel<IndexT><<<1, kPlanThreads, 0, st>>>(a);
    if (cudaGetLastError() != cudaSuccess) return HP_ERR_CUDA;
    uint64_t n = a.d.num_seqs + 1;
    if (a.d.table_cap > n) n = a.d.table_cap;
    if (a.d.token_cap > n) n = a.d.token_cap;
    const uint64_t cap = (uint64_t)sms * 8, want = (n + 255) / 256;
    return launch_dependent(step_fill_kernel<IndexT>, (unsigned)(want < cap ? want : cap), 256, 0,
                            st, a) == cudaSuccess
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
