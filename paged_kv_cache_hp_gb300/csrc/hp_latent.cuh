// hp_latent.cuh -- launch interface of attention over a paged cache of shared latent rows
// (hp_latent.cu on the CUDA cores, hp_latent_tc.cu and hp_latent_prefill_tc.cu on the tensor
// cores).
#pragma once

#include <cstdint>

#include "hp_internal.cuh"

namespace hp {

constexpr uint32_t kLatentStep = 64;        // tokens per step of the absorbed form
constexpr uint32_t kLatentMaxSms = 160;     // workers are counted for at most this many SMs
constexpr uint32_t kLatentRecordRows = 128; // record rows per SM
constexpr uint32_t kLatentCcRows = 16;      // (query, head) rows per group, CUDA cores
constexpr uint32_t kLatentPad = 128;        // expanded form: rows a sequence is padded to
constexpr uint32_t kLatentCcQueries = 32;   // queries per block, CUDA cores
constexpr uint32_t kLatentTcQueries = 256;  // queries per block, tensor cores
constexpr uint32_t kSmallSeqs = 128;        // batches up to this many sequences, and
constexpr uint64_t kPlanTable = 4096;       // this many table entries, need no plan launch

// Absorbed form, after a kPlanLatent plan on the same stream.  The plan's units are, sequence
// after sequence and row group after row group, the steps of kLatentStep tokens: a group is
// group_rows of the sequence's n * H rows (row r: query r / H, head r % H).  The units are
// split evenly over `workers`; a group that several workers share leaves a record per worker:
// its first worker's in slot 1 of that worker's two unless the group starts its range, the
// others' in slot 0 (a range has at most one group that began before it and one that goes on
// after it).
struct LatentMerge {          // the group that begins in a worker's range and goes on past it
    uint64_t out_row;         // row of out of the group's first row
    uint32_t rows;            // rows of the group; 0: no such group
    uint32_t last;            // its last worker
    uint32_t slot;            // the worker's own record slot (the others': 0)
    uint32_t pad[3];
};

struct LatentArgs {
    const void* pool;
    const void* q;            // [total_q, H, W]
    const void* q_ptr;        // NULL: query s is sequence s's
    const void* table;
    const void* seq_ptr;
    const void* lens;
    uint64_t num_seqs, page_size, num_pages;
    uint64_t total_q;
    uint32_t H, R, W;         // heads, latent_dim, latent_dim + rope_dim
    uint32_t group_rows;
    uint32_t g_m, g_l;        // div_invariant constants of page_size / 8 (tensor cores)
    uint64_t workers;
    float scale;
    int bf16, idx64, test_stall;
    int small;                // tensor cores: the kernel makes the plan itself (hp_latent_plan.cuh)
    PlanArgs plan;
    const WsHeader* hdr;
    const unsigned long long* units_off;
    float* part_acc;          // [2 * workers * group_rows, R]
    float2* part_ml;          // their maxima (log2 units) and sums (tensor cores: sums and accumulators
                              // times 2^kWeightLift)
    LatentMerge* merge;       // [workers], written by the attention kernel for the merge
    void* out;                // [total_q, H, R]
    int* d_status;
};
int launch_latent_cc(const LatentArgs& a, void* stream);
int launch_latent_tc(const LatentArgs& a, void* stream);
bool latent_tc_fits(uint32_t latent_dim, uint64_t head_dim, uint64_t page_size, uint64_t num_pages,
                    uint64_t q_rows);
int launch_latent_merge(const LatentArgs& a, void* stream);

// Expanded form, after a kPlanLatent plan (rows padded to kLatentPad per sequence, units of
// q_block queries).
struct LatentUnit {           // a block of queries, for the tensor-core attention
    uint64_t block;           // its sequence's first block of 128 rows in the workspace
    uint64_t q_row;           // its first query
    int64_t seen0;            // tokens that query sees (not positive: none)
    uint32_t queries;         // 0: no unit
    uint32_t pad;
};

struct LatentPrefillArgs {
    const void* pool;
    const void* w_kv;         // [H, Dn + Dv, R]
    const void* q;            // [total_q, H, Dn + W - R]
    const void* q_ptr;
    const void* table;
    const void* seq_ptr;
    const void* lens;
    uint64_t num_seqs, page_size, num_pages;
    uint64_t total_q, cap_rows, max_units;
    uint32_t H, R, W, Dn, Dv, q_block;
    float scale;
    int bf16, idx64, test_stall;
    int small;                // blocked: the gather makes the plan itself (hp_latent_plan.cuh)
    PlanArgs plan;
    const WsHeader* hdr;
    const unsigned long long* rows_off;
    const unsigned long long* units_off;
    int blocked;              // tensor cores: the buffers below in blocks (hp_latent_prefill_tc.cu)
    void* rows;               // [cap_rows, W]: the latent rows, zeros behind each sequence; blocked:
                              // [cap_rows, R]
    LatentUnit* units;        // blocked: [max_units]
    void* rope_blocks;        // blocked: the rope keys, 128 x 64 per 128 rows, swizzled
    void* kv;                 // [cap_rows, H, Dn + Dv]; blocked: [H, cap_rows / 128, 4, 128 x 64]
    void* out;                // [total_q, H, Dv]
    int* d_status;
};
int launch_latent_rows(const LatentPrefillArgs& a, void* stream);
int launch_latent_prefill_cc(const LatentPrefillArgs& a, void* stream);
int launch_latent_prefill_tc(const LatentPrefillArgs& a, void* stream);
bool latent_prefill_tc_fits(uint32_t latent_dim, uint64_t head_dim, uint32_t nope, uint32_t v,
                            uint64_t cap_rows, uint64_t total_q, uint32_t heads);

__device__ __forceinline__ unsigned long long index_at(const void* p, int idx64, uint64_t i)
{
    return idx64 ? (unsigned long long)static_cast<const unsigned long long*>(p)[i]
                 : (unsigned long long)static_cast<const unsigned int*>(p)[i];
}

// Worker v's entry of a.merge, by one thread of the attention kernel; units(s): the plan's sums,
// total = units(num_seqs).
template <typename F>
__device__ __forceinline__ void write_merge(const LatentArgs& a, uint64_t v, uint64_t total, F units)
{
    const uint64_t Lw = (total + a.workers - 1) / a.workers;
    const uint64_t b = v * Lw, beg = b < total ? b : total, e = beg + Lw, end = e < total ? e : total;
    LatentMerge m{};
    if (beg < end && end < total) {
        uint64_t lo = 0, hi = a.num_seqs;  // the sequence of the range's last unit
        while (hi - lo > 1) {
            const uint64_t mid = (lo + hi) >> 1;
            if (units(mid) <= end - 1) lo = mid;
            else hi = mid;
        }
        const uint64_t len = index_at(a.lens, a.idx64, lo);
        const uint64_t q0 = a.q_ptr ? index_at(a.q_ptr, a.idx64, lo) : lo;
        const uint64_t n = (a.q_ptr ? index_at(a.q_ptr, a.idx64, lo + 1) : lo + 1) - q0;
        const uint64_t steps = (len + kLatentStep - 1) / kLatentStep;
        const uint64_t first = units(lo), g = (end - 1 - first) / steps, start = first + g * steps;
        if (start >= beg && start + steps > end) {
            const uint64_t left = n * a.H - g * a.group_rows;
            m.out_row = q0 * a.H + g * a.group_rows;
            m.rows = (uint32_t)(left < a.group_rows ? left : a.group_rows);
            m.last = (uint32_t)((start + steps - 1) / Lw);
            m.slot = start > beg ? 1 : 0;
        }
    }
    a.merge[v] = m;
}

}  // namespace hp
