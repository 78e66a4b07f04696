// hp_prefix.cu -- the plan of attention behind shared prefixes (hp_attention_prefix): validation, and
// what the kernels behind it need to know of each query row and each group.
//
// One launch: the block table, the sequences and the rows are spread over all its CTAs (one more for
// every 8,192 table entries: a thread's eight are in flight together), the sums over the groups are the
// first one's.  Each CTA leaves a verdict of its own, which every CTA of the next kernel reads and
// meets (hp_prefix.cuh), so no CTA waits for another and nothing has to be cleared first.
#include <cuda_runtime.h>

#include "hp_prefix.cuh"
#include "hp_resolve.cuh"
#include "hp_rows.cuh"
#include "hp_scan.cuh"

namespace hp {
namespace {

__global__ void __launch_bounds__(kPlanThreads) prefix_plan_kernel(const PrefixPlanArgs a)
{
    __shared__ unsigned long long s_key;
    pdl_wait();
    const unsigned rank = blockIdx.x;
    const uint64_t tid = rank * (uint64_t)kPlanThreads + threadIdx.x, threads = a.ctas * (uint64_t)kPlanThreads;
    const uint64_t S = a.num_seqs, N = a.num_groups;
    if (threadIdx.x == 0) s_key = kVerdictOk;
    __syncthreads();
    auto fail = [&](unsigned rule, uint64_t at) { atomicMin(&s_key, verdict_key(rule, at)); };
    auto q_at = [&](uint64_t s) { return a.q_ptr ? index_at(a.q_ptr, a.idx64, s) : (unsigned long long)s; };

    // invariant (3): a thread's entries, eight in flight
    for (uint64_t k = tid; k < a.table_len; k += 8 * threads) {
        unsigned long long e[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) e[i] = k + i * threads < a.table_len ? index_at(a.table, a.idx64, k + i * threads) : 0ull;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (k + i * threads < a.table_len && e[i] >= a.num_pages) fail(kRankPageId, k + i * threads);
    }
    if (tid == 0) {
        if (index_at(a.seq_ptr, a.idx64, 0) != 0) fail(kRankSeqPtrStart, 0);
        if (index_at(a.seq_ptr, a.idx64, S) != a.table_len) fail(kRankSeqPtrEnd, S);
        if (q_at(0) != 0) fail(kRankNewPtrStart, 0);
        if (q_at(S) > a.total_q) fail(kRankNewPtrEnd, S);
        if (index_at(a.group_ptr, a.idx64, 0) != 0 || index_at(a.group_ptr, a.idx64, N) != S) fail(kRankGroup, 0);
    }
    for (uint64_t g = tid; g < N; g += threads)
        if (index_at(a.group_ptr, a.idx64, g) > index_at(a.group_ptr, a.idx64, g + 1)) fail(kRankGroup, g);
    // sequences and their rows: a thread each where they have one row, a warp each otherwise
    const uint64_t wide = a.q_ptr ? 32 : 1, lane = tid % wide;
    for (uint64_t s = tid / wide; s < S; s += threads / wide) {
        const uint64_t lo = index_at(a.seq_ptr, a.idx64, s), hi = index_at(a.seq_ptr, a.idx64, s + 1);
        const uint64_t len = index_at(a.lens, a.idx64, s), n0 = q_at(s), n1 = q_at(s + 1);
        uint64_t pages = quotient(len, a.P);
        pages += pages * a.P != len;
        if (lo > hi) fail(kRankSeqPtrOrder, s);
        else if (pages > hi - lo || len >= kPagesMaxTokens) fail(kRankLen, s);
        if (n0 > n1) fail(kRankNewPtrOrder, s);
        uint64_t g = 0, end = N;  // the last group that begins at or before s (num_groups > 0)
        while (end - g > 1) {
            const uint64_t mid = (g + end) >> 1;
            if (index_at(a.group_ptr, a.idx64, mid) <= s) g = mid;
            else end = mid;
        }
        const uint64_t prefix = index_at(a.prefix_lens, a.idx64, g);
        const uint64_t n = n0 <= n1 && n1 <= a.total_q ? n1 - n0 : 0;
        // every query sees the whole prefix
        if (prefix && (prefix > len || (n ? n - 1 : 0) > len - prefix)) fail(kRankPrefix, g);
        const uint64_t first = umin(index_at(a.group_ptr, a.idx64, g), S), r0 = q_at(first);
        for (uint64_t i = lane; i < n; i += wide) {
            const uint64_t behind = n - 1 - i;
            PrefixRow row;
            row.table = lo;
            row.prefix = (uint32_t)prefix;
            row.seen = len > behind ? (uint32_t)(len - behind) : 0u;
            row.group = (uint32_t)g;
            row.local = (uint32_t)(n0 + i - r0);
            a.rows[n0 + i] = row;
        }
    }
    for (uint64_t r = q_at(S) + tid; r < a.total_q; r += threads) a.rows[r].group = 0xFFFFFFFFu;
    // groups: steps and record rows before each
    uint64_t steps = 0;
    if (rank == 0) {
        uint64_t c_steps = 0, c_rows = 0;
        const uint64_t qt = kPrefixRows / a.G;
        for (uint64_t base = 0; base < N; base += kPlanThreads) {
            const uint64_t g = base + threadIdx.x;
            PrefixGroup gr{};
            uint64_t st = 0, rr = 0;
            if (g < N) {
                const uint64_t s0 = umin(index_at(a.group_ptr, a.idx64, g), S);
                const uint64_t s1 = umin(index_at(a.group_ptr, a.idx64, g + 1), S);
                const uint64_t r0 = umin(q_at(s0), a.total_q), r1 = umin(q_at(s1), a.total_q);
                const uint64_t prefix = umin(index_at(a.prefix_lens, a.idx64, g), kPagesMaxTokens);
                gr.table = index_at(a.seq_ptr, a.idx64, s0);
                gr.row0 = r0;
                gr.rows = r1 > r0 ? (uint32_t)(r1 - r0) : 0u;
                gr.prefix = (uint32_t)prefix;
                gr.blocks = (uint32_t)((prefix + kPrefixKeys - 1) / kPrefixKeys);
                gr.tiles = (uint32_t)((gr.rows + qt - 1) / qt);
                st = (uint64_t)a.H * gr.tiles * gr.blocks;
                const uint64_t last = gr.tiles ? (gr.rows - (gr.tiles - 1) * qt) * a.G : 0;
                gr.records = gr.tiles ? (gr.tiles - 1) * qt * a.G + (last <= kPrefixRows / 2 ? 2 * last : last) : 0;
                rr = a.H * gr.records;
            }
            unsigned long long es, er, ts, tr;
            block_scan2(st, rr, es, er, ts, tr);
            if (g < N) {
                gr.step0 = c_steps + es;
                gr.rows0 = c_rows + er;
                a.groups[g] = gr;
            }
            c_steps += ts;
            c_rows += tr;
        }
        steps = c_steps;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        a.hdr->keys[rank] = s_key;
        if (rank == 0) a.hdr->steps = steps;
    }
}

__global__ void __launch_bounds__(kPrefixPlanCtas) prefix_status_kernel(const PrefixHeader* hdr, uint32_t n, int* d_status)
{
    pdl_wait();
    plan_holds(hdr, n, d_status, true, false);
}

}  // namespace

int launch_prefix_plan(const PrefixPlanArgs& a, void* stream)
{
    return launch_dependent(prefix_plan_kernel, a.ctas, kPlanThreads, 0, static_cast<cudaStream_t>(stream), a) == cudaSuccess
               ? HP_OK
               : HP_ERR_CUDA;
}

int launch_prefix_status(const PrefixHeader* hdr, uint32_t ctas, int* d_status, void* stream)
{
    if (!d_status) return HP_OK;
    return launch_dependent(prefix_status_kernel, 1, kPrefixPlanCtas, 0, static_cast<cudaStream_t>(stream), hdr, ctas,
                            d_status) == cudaSuccess
               ? HP_OK
               : HP_ERR_CUDA;
}

}  // namespace hp
