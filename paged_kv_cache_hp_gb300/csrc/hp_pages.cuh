// hp_pages.cuh -- launch interface of the operators that read only some of a long sequence's
// pages (hp_pages.cu: bounds, scores, selection; hp_attn_rows.cu: attention), and the pieces that
// they share: which sequence a query belongs to, and how errors reach the status word.
#pragma once

#include <cstdint>

#include "hp_internal.cuh"
#include "hp_latent.cuh"  // index_at

namespace hp {

constexpr uint32_t kPagesMaxPage = 4096;        // slots of a page
constexpr uint32_t kPagesMaxGroup = 16;         // query heads of a K/V head
constexpr uint64_t kPagesMaxTokens = 1u << 31;  // tokens of a sequence stay below (32-bit token numbers)
// Up to this many entries (pages, list entries) of up to so many rows one extra CTA looks at them all,
// beside the others, and stores the status (under 5 us); beyond it a kernel of one thread before
// this one clears the word, and whoever meets an error lowers it.
constexpr uint64_t kPagesChecked = 1024, kRowsChecked = 128;

// The queries of a batch: sequence s has q_ptr[s] .. q_ptr[s+1], its last tokens in order (q_ptr
// NULL: one each).
struct QueryArgs {
    const void* q_ptr;
    const void* lens;
    uint64_t num_seqs, total_q;
    int idx64;
};

struct PageTable {
    const void* seq_ptr;
    const void* table;
    uint64_t table_len, num_pages;
};

struct BoundsArgs {
    QueryArgs q;              // q_ptr: the new tokens' offsets, total_q their count
    PageTable t;
    const void* pool;
    void* bounds;             // [num_pages, H, 2, D]
    uint64_t units;           // pages that the new tokens can touch
    uint32_t P, columns;      // slots of a page, 16-byte columns of a row (H * D / 8)
    uint32_t row_half;        // D / 8: columns of a head
    int bf16;
    int check_all;            // the extra CTA looks at everything
    int* d_status;
};
int launch_page_bounds(const BoundsArgs& a, void* stream);

struct ScoreArgs {
    QueryArgs q;
    PageTable t;
    const void* bounds;
    const void* queries;      // [total_q, H * G, D]
    float* scores;            // [total_q, H, max_pages]
    uint64_t max_pages;
    uint32_t P, H, G, D;
    uint32_t chunk_blocks;    // a CTA's pages, in blocks of 16
    uint64_t chunks;          // of a row
    float scale;
    int bf16;
    int check_all;
    int* d_status;
};
int launch_page_scores(const ScoreArgs& a, void* stream);

struct SelectArgs {
    QueryArgs q;
    const float* scores;      // [total_q, H, max_pages]
    int32_t* selected;        // [total_q, H, k]
    uint64_t max_pages;
    uint32_t P, H, sinks, recent, k;
    int check_all;
    int* d_status;
};
int launch_select_pages(const SelectArgs& a, void* stream);

// Clears the status word ahead of a kernel whose CTAs report what they meet.
int launch_clear_status(int* d_status, void* stream);

#ifdef __CUDACC__

// The largest s of [0, n) up to which f holds from 0 on (f(0) is taken to hold), by a whole warp;
// the same in all lanes.  Ends for any f.
template <typename F>
__device__ __forceinline__ uint64_t warp_last(uint64_t n, F f)
{
    const unsigned lane = threadIdx.x & 31;
    uint64_t lo = 0, hi = n;
    while (hi - lo > 1) {
        const uint64_t step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step;
        const unsigned holds = __ballot_sync(0xffffffffu, at < hi && f(at));
        const unsigned run = holds == 0xffffffffu ? 32u : (unsigned)__ffs(~holds) - 1u;
        const uint64_t end = lo + (run + 1) * step;
        lo += run * step;
        hi = end < hi ? end : hi;
    }
    return lo;
}

struct Query {
    uint64_t seq;   // num_seqs: no sequence has it
    uint64_t len;
    uint32_t seen;  // tokens it sees
    int code;       // HP_ERR_LEN: more tokens than these operators take
};

__device__ __forceinline__ Query query_of(const QueryArgs& a, uint64_t s, uint64_t r, uint64_t n0, uint64_t n1)
{
    Query q{a.num_seqs, 0, 0, HP_OK};
    if (n0 > r || r >= n1 || n1 > a.total_q) return q;
    q.seq = s;
    q.len = index_at(a.lens, a.idx64, s);
    if (q.len >= kPagesMaxTokens) {
        q.code = HP_ERR_LEN;
        return q;
    }
    const uint64_t behind = n1 - 1 - r;  // queries of the sequence after this one
    q.seen = q.len > behind ? (uint32_t)(q.len - behind) : 0u;
    return q;
}

// Query r, by a whole warp.
__device__ __forceinline__ Query find_query(const QueryArgs& a, uint64_t r)
{
    if (!a.q_ptr) return query_of(a, r, r, r, r + 1);
    if (a.num_seqs == 0) return Query{0, 0, 0, HP_OK};
    const uint64_t s = warp_last(a.num_seqs, [&](uint64_t i) { return index_at(a.q_ptr, a.idx64, i) <= r; });
    return query_of(a, s, r, index_at(a.q_ptr, a.idx64, s), index_at(a.q_ptr, a.idx64, s + 1));
}

// f(r, query r) for every row, each by one thread of the CTA.
template <typename F>
__device__ __forceinline__ void for_each_query(const QueryArgs& a, F f)
{
    if (!a.q_ptr) {
        for (uint64_t r = threadIdx.x; r < a.total_q; r += blockDim.x) f(r, query_of(a, r, r, r, r + 1));
    } else {
        for (uint64_t r = threadIdx.x >> 5; r < a.total_q; r += blockDim.x >> 5) {
            const Query q = find_query(a, r);
            if ((threadIdx.x & 31) == 0) f(r, q);
        }
    }
}

__device__ __forceinline__ int lower(int a, int b) { return a < b ? a : b; }

// What is wrong with the offsets p[0 .. S], as this thread of the CTA sees it.
__device__ __forceinline__ int offsets_code(const void* p, int idx64, uint64_t S, uint64_t total)
{
    int code = HP_OK;
    if (!p) return code;
    for (uint64_t s = threadIdx.x; s <= S; s += blockDim.x) {
        const uint64_t x = index_at(p, idx64, s);
        if (s == 0 && x != 0) code = lower(code, HP_ERR_NEW_PTR_START);
        if (s < S && x > index_at(p, idx64, s + 1)) code = lower(code, HP_ERR_NEW_PTR_ORDER);
        if (s == S && x > total) code = lower(code, HP_ERR_NEW_PTR_END);
    }
    return code;
}

// The lowest of the CTA's codes: stored (the CTA looked at everything), or met with what others
// report.
__device__ __forceinline__ void report_codes(int code, int* d_status, bool all)
{
    __shared__ int s_code;
    if (threadIdx.x == 0) s_code = HP_OK;
    __syncthreads();
    if (code != HP_OK) atomicMin(&s_code, code);
    __syncthreads();
    if (threadIdx.x) return;
    if (all) *d_status = s_code;
    else if (s_code != HP_OK) atomicMin(d_status, s_code);
}

// The page that entry j of sequence s names, or a code.
__device__ __forceinline__ int page_at(const PageTable& t, int idx64, uint64_t lo, uint64_t hi, uint64_t j,
                                       uint64_t* phys)
{
    if (lo > hi || hi > t.table_len || j >= hi - lo) return HP_ERR_LEN;
    *phys = index_at(t.table, idx64, lo + j);
    return *phys < t.num_pages ? HP_OK : HP_ERR_PAGE_ID;
}

#endif  // __CUDACC__

}  // namespace hp
