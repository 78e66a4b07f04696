// hp_latent_plan.cuh -- the plan of a small batch (hp_plan.cu's kPlanLatent), made by every CTA of the
// first kernel for itself instead of by a launch before it.
//
// A launch in a stream of small kernels is 6 us, the plan of up to kSmallSeqs sequences and a block
// table of kPlanTable entries 1 to 2 us of every CTA's start (five loads a sequence and 16 table
// entries a thread, in one trip to memory): decode of one sequence 20.6 -> 16 us, a prompt of
// three short sequences 24.6 -> 19.4 us.
//
// That first kernel is launched as a dependent of whatever the stream holds before it and waits for
// its completion before it reads or writes memory (2.5 us less than a plain launch, its barriers and
// TMEM being made ready meanwhile).  Every dependent launch of this library waits so, so what came
// before the kernel before is complete too.
#pragma once

#include "hp_latent.cuh"
#include "hp_scan.cuh"

namespace hp {

struct SmallPlan {
    unsigned long long key;  // the verdict
    uint32_t rows, units;    // totals
};

// The sums of `p` (1 <= p.num_seqs <= kSmallSeqs, p.table_len <= kPlanTable, sums below 2^31 once the rules
// hold) at units[0 .. S] and, where wanted, rows[0 .. S], in shared memory; by a whole CTA of at least
// kSmallSeqs threads, the result the same in all.
__device__ __forceinline__ SmallPlan small_plan(const PlanArgs& p, int idx64, uint32_t* units, uint32_t* rows)
{
    __shared__ unsigned long long s_key, s_len;
    __shared__ uint32_t w_units[kSmallSeqs / 32], w_rows[kSmallSeqs / 32];
    const uint32_t S = (uint32_t)p.num_seqs, t = threadIdx.x, lane = t & 31, warp = t >> 5;
    unsigned long long lo = 0, hi = 0, len = 0, n0 = t, n1 = t + 1, bad = ~0ull;
    if (t < S) {
        lo = index_at(p.seq_ptr, idx64, t);
        hi = index_at(p.seq_ptr, idx64, t + 1);
        len = index_at(p.lens, idx64, t);
        if (p.new_ptr) {
            n0 = index_at(p.new_ptr, idx64, t);
            n1 = index_at(p.new_ptr, idx64, t + 1);
        }
    }
#pragma unroll 8
    for (uint32_t k = t; k < (uint32_t)p.table_len; k += blockDim.x)
        if (index_at(p.table, idx64, k) >= p.num_pages && bad == ~0ull) bad = k;
    if (t == 0) {
        s_key = kVerdictOk;
        s_len = 0;
    }
    __syncthreads();
    if (bad != ~0ull) atomicMin(&s_key, verdict_key(kRankPageId, bad));
    uint32_t u = 0, r = 0;
    if (t < S) {
        unsigned long long pages = quotient(len, p.page_size);
        pages += pages * p.page_size != len;
        if (lo > hi) atomicMin(&s_key, verdict_key(kRankSeqPtrOrder, t));
        else if (pages > hi - lo) atomicMin(&s_key, verdict_key(kRankLen, t));
        if (n0 > n1) atomicMin(&s_key, verdict_key(kRankNewPtrOrder, t));
        const unsigned long long n = n0 <= n1 && n1 <= p.total_new ? n1 - n0 : 0;
        // (truncated only where a rule fails)
        if (p.heads) {
            u = (uint32_t)(quotient(n * p.heads + p.group_rows - 1, p.group_rows) *
                           quotient(len + p.step_tokens - 1, p.step_tokens));
        } else {
            u = (uint32_t)quotient(n + p.group_rows - 1, p.group_rows);
            r = (uint32_t)(quotient(len + p.row_round - 1, p.row_round) * p.row_round);
            atomicAdd(&s_len, len);  // (wraps only past HP_ERR_LEN, an earlier rule)
        }
    }
    if (t == 0) {
        if (lo != 0) atomicMin(&s_key, verdict_key(kRankSeqPtrStart, 0));
        if (n0 != 0) atomicMin(&s_key, verdict_key(kRankNewPtrStart, 0));
    }
    if (t + 1 == S) {
        if (hi != p.table_len) atomicMin(&s_key, verdict_key(kRankSeqPtrEnd, S));
        if (n1 > p.total_new) atomicMin(&s_key, verdict_key(kRankNewPtrEnd, S));
    }
    uint32_t iu = u, ir = r;
    if (t < kSmallSeqs) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t nu = __shfl_up_sync(0xffffffffu, iu, o), nr = __shfl_up_sync(0xffffffffu, ir, o);
            if (lane >= (uint32_t)o) {
                iu += nu;
                ir += nr;
            }
        }
        if (lane == 31) {
            w_units[warp] = iu;
            w_rows[warp] = ir;
        }
    }
    __syncthreads();
    SmallPlan out{s_key, 0, 0};
    uint32_t bu = 0, br = 0;
#pragma unroll
    for (uint32_t w = 0; w < kSmallSeqs / 32; ++w) {
        if (w == warp) {
            bu = out.units;
            br = out.rows;
        }
        out.units += w_units[w];
        out.rows += w_rows[w];
    }
    if (!p.heads && s_len > p.out_tokens) out.key = min(out.key, verdict_key(kRankOutSize, 0));
    if (t < S) {
        units[t] = bu + iu - u;
        if (rows) rows[t] = br + ir - r;
    }
    if (t == 0) {
        units[S] = out.units;
        if (rows) rows[S] = out.rows;
    }
    __syncthreads();
    return out;
}

// Stored for the kernels after, by one thread of the grid.
__device__ __forceinline__ void store_plan(const PlanArgs& p, const SmallPlan& s)
{
    p.ws.hdr->total_rows = s.rows;
    p.ws.hdr->total_units = s.units;
    p.ws.hdr->verdict = s.key;
    if (p.d_status) *p.d_status = key_status(s.key);
}

}  // namespace hp
