// hp_abi_pages.cu -- the entry points of long contexts (include/hp.h): page bounds, page scores, page
// selection, attention over selected pages, attention behind shared prefixes.  Host-side checks,
// then launches on the caller's stream.
#include <cuda_runtime.h>

#include <algorithm>

#include "hp_abi_checks.cuh"
#include "hp_rows.cuh"

namespace {

constexpr u64 kGrid = (1ull << 31) - 1;

u64 index_bytes(uint32_t index_type) { return index_type == HP_IDX_U64 ? 8 : 4; }

// The descriptor as these operators take it: what they read is checked on the device.
int check_pages(const hp_paged_desc* desc, const void* pool, hp_paged_desc* d)
{
    if (!desc) return HP_ERR_NULL;
    *d = *desc;
    if (pool) d->page_pool = pool;
    d->flags &= ~(HP_PERMISSIVE | HP_HAS_QUANT);
    const int rc = check_desc(d);
    if (rc) return rc;
    if (d->dtype != HP_F16 && d->dtype != HP_BF16) return HP_ERR_DTYPE;
    if ((d->head_dim != 64 && d->head_dim != 128 && d->head_dim != 256) || d->page_size > hp::kPagesMaxPage ||
        d->num_heads > (1u << 16))
        return HP_ERR_ARG;
    return HP_OK;
}

int check_heads(const hp_paged_desc& d, uint32_t num_q_heads, float scale)
{
    if (num_q_heads == 0 || num_q_heads % d.num_heads || num_q_heads / d.num_heads > hp::kPagesMaxGroup ||
        !(scale == scale))
        return HP_ERR_ARG;
    return HP_OK;
}

// Offsets of queries or new tokens: NULL for one a sequence.
int check_offsets(const hp_paged_desc& d, const void* ptr, u64 total)
{
    if (total >> 40) return HP_ERR_OVERFLOW;
    if (!ptr) return total == d.num_seqs ? HP_OK : HP_ERR_ARG;
    return misaligned(ptr, index_bytes(d.index_type)) ? HP_ERR_ALIGN : HP_OK;
}

hp::QueryArgs query_args(const hp_paged_desc& d, const void* q_ptr, u64 total_q)
{
    return hp::QueryArgs{q_ptr, d.seq_lens, d.num_seqs, total_q, d.index_type == HP_IDX_U64};
}

hp::PageTable page_table(const hp_paged_desc& d)
{
    return hp::PageTable{d.seq_ptr, d.block_table, d.table_len, d.num_pages};
}

// (A call without rows, whose offsets say so, launches its extra CTA alone: they may not hold.)
int reset_status(int* d_status, void* stream)
{
    if (!d_status) return HP_OK;
    return cudaMemsetAsync(d_status, 0, sizeof(int), static_cast<cudaStream_t>(stream)) == cudaSuccess ? HP_OK
                                                                                                       : HP_ERR_CUDA;
}

// CTAs of a (row, K/V head), up to eight: doubled while the grid has fewer than four to an SM (it can end at almost
// eight; an SM holds four, two at head_dim 256 or more than 8 query heads a K/V head) and each then has 64 tokens.
uint32_t cluster_of(u64 units, u64 tokens, int sms)
{
    uint32_t c = 1;
    while (c < 8 && units * c < 4 * (u64)sms && tokens / (2 * c) >= 64) c *= 2;
    return c;
}

}  // namespace

HP_API int hp_page_bounds(const hp_paged_desc* desc, const void* new_ptr, uint64_t total_new, void* bounds,
                          int* d_status, void* stream)
{
    hp_paged_desc d;
    int rc = check_pages(desc, nullptr, &d);
    if (rc) return rc;
    rc = check_offsets(d, new_ptr, total_new);
    if (rc) return rc;
    if (d.num_pages && !bounds) return HP_ERR_NULL;
    if (misaligned(bounds, 64)) return HP_ERR_ALIGN;
    hp::BoundsArgs a{};
    a.q = query_args(d, new_ptr, total_new);
    a.t = page_table(d);
    a.pool = d.page_pool;
    a.bounds = bounds;
    a.P = (uint32_t)d.page_size;
    a.row_half = (uint32_t)d.head_dim / 8;
    a.columns = (uint32_t)d.num_heads * a.row_half;
    a.units = d.num_seqs == 0 ? 0 : new_ptr ? total_new / a.P + 2 * d.num_seqs : d.num_seqs;
    if ((u128)a.units * ((a.columns + 127) / 128) + 1 > kGrid) return HP_ERR_OVERFLOW;
    if (!new_ptr && a.units == 0) return reset_status(d_status, stream);
    a.bf16 = d.dtype == HP_BF16;
    a.check_all = a.units <= hp::kPagesChecked;
    a.d_status = d_status;
    return hp::launch_page_bounds(a, stream);
}

HP_API int hp_page_scores(const hp_paged_desc* desc, const void* bounds, const void* q, const void* q_ptr,
                          uint64_t total_q, uint32_t num_q_heads, float scale, float* scores, uint64_t max_pages,
                          int* d_status, void* stream)
{
    if (desc && desc->num_pages && !bounds) return HP_ERR_NULL;
    hp_paged_desc d;
    int rc = check_pages(desc, bounds, &d);
    if (rc) return rc;
    rc = check_heads(d, num_q_heads, scale);
    if (rc) return rc;
    if (scale < 0.0f) return HP_ERR_ARG;
    rc = check_offsets(d, q_ptr, total_q);
    if (rc) return rc;
    if (max_pages >> 31 || total_q >= kGrid || ((u128)total_q * d.num_heads * max_pages) >> 60) return HP_ERR_OVERFLOW;
    if (total_q && (!q || (max_pages && !scores))) return HP_ERR_NULL;
    if (misaligned(q, 16) || misaligned(scores, 4)) return HP_ERR_ALIGN;
    if (!q_ptr && total_q == 0) return reset_status(d_status, stream);
    int dev = 0;
    const u64 sms = (u64)hp::current_sms(&dev);
    if (sms == 0) return HP_ERR_CUDA;
    hp::ScoreArgs a{};
    a.q = query_args(d, q_ptr, total_q);
    a.t = page_table(d);
    a.bounds = bounds;
    a.queries = q;
    a.scores = scores;
    a.max_pages = max_pages;
    a.P = (uint32_t)d.page_size;
    a.H = (uint32_t)d.num_heads;
    a.G = num_q_heads / a.H;
    a.D = (uint32_t)d.head_dim;
    // a CTA's eight warps take (16 pages, head) pairs: one each while the SMs are not filled twice
    // over, then up to sixteen (eight: 212 us where sixteen take 206, at 300,000 pages of 8 heads of 128)
    const u64 blocks = std::max<u64>(1, (max_pages + 15) / 16);
    const u64 each = std::min<u64>(16, std::max<u64>(1, total_q * blocks * a.H / (sms * 32)));
    a.chunk_blocks = (uint32_t)std::max<u64>(1, (each * 8 + a.H - 1) / a.H);
    a.chunks = (blocks + a.chunk_blocks - 1) / a.chunk_blocks;
    if ((u128)total_q * a.chunks + 1 > kGrid) return HP_ERR_OVERFLOW;
    a.scale = scale;
    a.bf16 = d.dtype == HP_BF16;
    a.check_all = total_q <= hp::kRowsChecked && total_q * max_pages <= 4 * hp::kPagesChecked;
    a.d_status = d_status;
    return hp::launch_page_scores(a, stream);
}

HP_API int hp_select_pages(const hp_paged_desc* desc, const void* q_ptr, uint64_t total_q, const float* scores,
                           uint64_t max_pages, uint32_t sinks, uint32_t recent, uint32_t k, int32_t* selected,
                           int* d_status, void* stream)
{
    hp_paged_desc d;
    int rc = check_pages(desc, nullptr, &d);
    if (rc) return rc;
    rc = check_offsets(d, q_ptr, total_q);
    if (rc) return rc;
    if (k == 0 || k >> 31 || (u64)sinks + recent > k) return HP_ERR_ARG;
    if (max_pages >> 31 || ((u128)total_q * d.num_heads * std::max<u64>(max_pages, k)) >> 60) return HP_ERR_OVERFLOW;
    if (total_q && ((max_pages && !scores) || !selected)) return HP_ERR_NULL;
    if (misaligned(scores, 4) || misaligned(selected, 4)) return HP_ERR_ALIGN;
    if ((u128)total_q * d.num_heads + 1 > kGrid) return HP_ERR_OVERFLOW;
    if (!q_ptr && total_q == 0) return reset_status(d_status, stream);
    hp::SelectArgs a{};
    a.q = query_args(d, q_ptr, total_q);
    a.scores = scores;
    a.selected = selected;
    a.max_pages = max_pages;
    a.P = (uint32_t)d.page_size;
    a.H = (uint32_t)d.num_heads;
    a.sinks = sinks;
    a.recent = recent;
    a.k = k;
    a.check_all = q_ptr ? total_q <= hp::kRowsChecked : total_q <= hp::kPagesChecked;
    a.d_status = d_status;
    return hp::launch_select_pages(a, stream);
}

namespace {

// Checks and arguments that the two attention calls share.
int rows_args(const hp_paged_desc& d, const void* v_pool, const void* q, const void* q_ptr, u64 total_q,
              uint32_t num_q_heads, float scale, void* out, hp::RowsArgs* a)
{
    int rc = check_heads(d, num_q_heads, scale);
    if (rc) return rc;
    rc = check_offsets(d, q_ptr, total_q);
    if (rc) return rc;
    if ((u128)total_q * num_q_heads >> 40 || (u128)total_q * d.num_heads * 8 + 8 > kGrid) return HP_ERR_OVERFLOW;
    if ((d.num_pages && !v_pool) || (total_q && (!q || !out))) return HP_ERR_NULL;
    if (misaligned(v_pool, 64) || misaligned(q, 16) || misaligned(out, 16)) return HP_ERR_ALIGN;
    a->q = query_args(d, q_ptr, total_q);
    a->t = page_table(d);
    a->k_pool = d.page_pool;
    a->v_pool = v_pool;
    a->queries = q;
    a->out = out;
    a->P = (uint32_t)d.page_size;
    hp::invariant_divisor(a->P, &a->p_m, &a->p_l);
    a->H = (uint32_t)d.num_heads;
    a->G = num_q_heads / a->H;
    a->D = (uint32_t)d.head_dim;
    a->scale = scale;
    a->bf16 = d.dtype == HP_BF16;
    return HP_OK;
}

}  // namespace

HP_API int hp_attention_pages(const hp_paged_desc* k_desc, const void* v_pool, const void* q, const void* q_ptr,
                              uint64_t total_q, uint32_t num_q_heads, float scale, const int32_t* selected,
                              uint32_t k, void* out, int* d_status, void* stream)
{
    hp_paged_desc d;
    int rc = check_pages(k_desc, nullptr, &d);
    if (rc) return rc;
    hp::RowsArgs a{};
    rc = rows_args(d, v_pool, q, q_ptr, total_q, num_q_heads, scale, out, &a);
    if (rc) return rc;
    if (k == 0 || (u64)k * d.page_size >> 31) return HP_ERR_ARG;
    if (total_q && !selected) return HP_ERR_NULL;
    if (misaligned(selected, 4)) return HP_ERR_ALIGN;
    if (!q_ptr && total_q == 0) return reset_status(d_status, stream);
    int dev = 0;
    const int sms = hp::current_sms(&dev);
    if (sms == 0) return HP_ERR_CUDA;
    a.selected = selected;
    a.k = k;
    a.cluster = cluster_of(total_q * a.H, (u64)k * a.P, sms);
    a.check_all = total_q <= hp::kRowsChecked && total_q * a.H * k <= hp::kPagesChecked;
    a.d_status = d_status;
    return hp::launch_rows(a, stream);
}

namespace {

// Byte offsets of the workspace of hp_attention_prefix.
struct PrefixWs {
    u64 rows, groups, ml, acc, total;
};

int prefix_ws(u64 num_groups, u64 total_q, uint32_t num_q_heads, u64 head_dim, u64 page_size, PrefixWs* w)
{
    if (num_groups >> 32 || total_q >> 32 || ((u128)total_q * num_q_heads) >> 40 || head_dim > 256) return HP_ERR_OVERFLOW;
    // (the tensor cores' kernel alone leaves records: two of a row where a tile has up to 128 of them)
    const u64 records = hp::prefix_tc_shape(head_dim, page_size)
                            ? 2 * total_q * num_q_heads + (u64)hp::kPrefixMaxSms * hp::kPrefixRows
                            : 0;
    w->rows = hp::round_up_256(sizeof(hp::PrefixHeader));
    w->groups = w->rows + hp::round_up_256(total_q * sizeof(hp::PrefixRow));
    w->ml = w->groups + hp::round_up_256(num_groups * sizeof(hp::PrefixGroup));
    w->acc = w->ml + hp::round_up_256(records * sizeof(float2));
    w->total = w->acc + hp::round_up_256(records * head_dim * 4);
    return HP_OK;
}

struct PrefixCall {
    hp_paged_desc d;
    hp::RowsArgs rows;
    hp::PrefixPlanArgs plan;
};

int prefix_prepare(const hp_paged_desc* k_desc, const void* v_pool, const void* group_ptr, const void* prefix_lens,
                   u64 num_groups, const void* q, const void* q_ptr, u64 total_q, uint32_t num_q_heads, float scale,
                   void* out, void* workspace, u64 workspace_bytes, int* d_status, PrefixCall* c)
{
    int rc = check_pages(k_desc, nullptr, &c->d);
    if (rc) return rc;
    const hp_paged_desc& d = c->d;
    c->rows = hp::RowsArgs{};
    rc = rows_args(d, v_pool, q, q_ptr, total_q, num_q_heads, scale, out, &c->rows);
    if (rc) return rc;
    if (num_groups > d.num_seqs || (num_groups == 0 && d.num_seqs)) return HP_ERR_ARG;
    if (!group_ptr || (num_groups && !prefix_lens)) return HP_ERR_NULL;
    if (misaligned(group_ptr, index_bytes(d.index_type)) || misaligned(prefix_lens, index_bytes(d.index_type)))
        return HP_ERR_ALIGN;
    PrefixWs w;
    rc = prefix_ws(num_groups, total_q, num_q_heads, d.head_dim, d.page_size, &w);
    if (rc) return rc;
    if (!workspace || misaligned(workspace, 256) || workspace_bytes < w.total) return HP_ERR_WORKSPACE;
    char* ws = static_cast<char*>(workspace);
    hp::PrefixPlanArgs& p = c->plan;
    p = hp::PrefixPlanArgs{};
    p.seq_ptr = d.seq_ptr;
    p.lens = d.seq_lens;
    p.table = d.block_table;
    p.q_ptr = q_ptr;
    p.group_ptr = group_ptr;
    p.prefix_lens = prefix_lens;
    p.num_seqs = d.num_seqs;
    p.num_groups = num_groups;
    p.total_q = total_q;
    p.table_len = d.table_len;
    p.num_pages = d.num_pages;
    p.P = c->rows.P;
    p.H = c->rows.H;
    p.G = c->rows.G;
    p.idx64 = d.index_type == HP_IDX_U64;
    p.hdr = reinterpret_cast<hp::PrefixHeader*>(ws);
    p.rows = reinterpret_cast<hp::PrefixRow*>(ws + w.rows);
    p.groups = reinterpret_cast<hp::PrefixGroup*>(ws + w.groups);
    p.ctas = hp::prefix_plan_ctas(d.table_len);
    hp::RowsArgs& a = c->rows;
    a.hdr = p.hdr;
    a.num_keys = p.ctas;
    a.rows = p.rows;
    a.groups = p.groups;
    a.rec.ml = reinterpret_cast<float2*>(ws + w.ml);
    a.rec.acc = reinterpret_cast<float*>(ws + w.acc);
    a.d_status = d_status;
    return HP_OK;
}

// The kernels behind the plan; the first of them stores the status (first 1: in any case, 2: an error).
int prefix_run(PrefixCall& c, int first, void* stream)
{
    hp::RowsArgs& a = c.rows;
    if (c.d.num_seqs == 0 || a.q.total_q == 0)
        return first == 1 ? hp::launch_prefix_status(c.plan.hdr, c.plan.ctas, a.d_status, stream) : HP_OK;
    a.first = first;
    int dev = 0;
    const int sms = hp::current_sms(&dev);
    if (sms == 0) return HP_ERR_CUDA;
    a.cluster = cluster_of(a.q.total_q * a.H, c.d.table_len * c.d.page_size / c.d.num_seqs, sms);
    // Each query reads its prefix by itself (through L2) while that is little: a launch, the records and their
    // merge are 8 us and more.  The host knows neither the prefixes nor who shares them, so this takes the table for
    // one of prefixes that many share; where it is not, the tensor cores lose (below), and HP_ATTN_CUDA_CORES helps.  One group, 16-slot pages, 128 dims, a few tokens behind the prefix, us on the
    // tensor cores and without (by the bytes of K and V that the table's slots hold): 8 sequences and 8 K/V
    // heads at 67 MB 26 and 18, at 264 MB 36 and 33; 16 at 527 MB 51 and 58; 64 at 145 MB 38 and 30, at 538 MB 41 and
    // 57, at 2.1 GB 57 and 159; 64 with one head at 67 MB 32 and 19, at 264 MB 41 and 34.  Sequences so long that
    // eight CTAs a (query, head) are few: one sequence with 2 heads at 16,000 tokens 41 and 35, at 30,000 44 and 54, at
    // 60,000 48 and 95; with one head 50 and 34, 55 and 54, 59 and 95.  Little shared, 8 K/V heads: 256 sequences of 1,024
    // tokens behind 16 shared ones 191 and 169, behind 128 189 and 174, of 450 with 8
    // query heads each behind 16 114 and 88, of 500 behind 512 123 and 125, of 100 behind
    // 900 68 and 95; groups of one: 64 of 2,000 tokens 132 and 94, 256 of 400 167 and 85, 4 of 33,000 122 and 92;
    // prefixes of 0: 64 of 2,000 96 and 93, 256 of 500 101 and 98.
    const u128 bytes = (u128)c.d.table_len * c.d.page_size * c.d.num_heads * c.d.head_dim * 4;
    if (!(c.d.flags & (HP_ATTN_CUDA_CORES | HP_HOST_MEMORY)) &&
        ((c.d.flags & HP_ATTN_TENSOR_CORES) || bytes >= HP_PREFIX_TC_MIN_BYTES ||
         (u128)c.d.table_len * c.d.page_size >= (u128)HP_PREFIX_TC_MIN_TOKENS * c.d.num_seqs) &&
        hp::prefix_tc_fits(c.d.head_dim, c.d.page_size, c.d.num_pages)) {
        a.rec.workers = std::min<u64>((u64)sms, hp::kPrefixMaxSms);
        hp::PrefixTcArgs t{};
        t.k_pool = a.k_pool;
        t.v_pool = a.v_pool;
        t.q = a.queries;
        t.table = c.d.block_table;
        t.num_groups = c.plan.num_groups;
        t.num_pages = c.d.num_pages;
        t.workers = a.rec.workers;
        t.P = a.P;
        t.H = a.H;
        t.G = a.G;
        t.box = hp::prefix_tc_box(a.P);
        t.scale = a.scale;
        t.bf16 = a.bf16;
        t.idx64 = a.q.idx64;
        t.test_stall = (c.d.flags & HP_TEST_STALL) != 0;
        t.hdr = a.hdr;
        t.groups = a.groups;
        t.num_keys = a.num_keys;
        t.first = first;
        a.first = 0;
        t.rec = a.rec;
        t.d_status = a.d_status;
        const int rc = hp::launch_prefix_tc(t, a.D, stream);
        if (rc) return rc;
    }
    return hp::launch_rows(a, stream);
}

}  // namespace

HP_API int hp_attention_prefix_workspace_bytes(const hp_paged_desc* k_desc, uint64_t num_groups, uint64_t total_q,
                                               uint32_t num_q_heads, uint64_t* bytes)
{
    if (!k_desc || !bytes) return HP_ERR_NULL;
    PrefixWs w;
    const int rc = prefix_ws(num_groups, total_q, num_q_heads, k_desc->head_dim, k_desc->page_size, &w);
    if (rc) return rc;
    *bytes = w.total;
    return HP_OK;
}

HP_API int hp_attention_prefix_plan(const hp_paged_desc* k_desc, const void* group_ptr, const void* prefix_lens,
                                    uint64_t num_groups, const void* q_ptr, uint64_t total_q, uint32_t num_q_heads,
                                    void* workspace, uint64_t workspace_bytes, int* d_status, void* stream)
{
    PrefixCall c;
    // (no buffers of a layer: the descriptor's pool stands in for them in the checks)
    const void* any = k_desc ? k_desc->page_pool : nullptr;
    void* stand_in = const_cast<void*>(any ? any : workspace);
    int rc = prefix_prepare(k_desc, any, group_ptr, prefix_lens, num_groups, stand_in, q_ptr, total_q,
                                  num_q_heads, 1.0f, stand_in, workspace, workspace_bytes, d_status, &c);
    if (rc) return rc;
    rc = hp::launch_prefix_plan(c.plan, stream);
    return rc ? rc : hp::launch_prefix_status(c.plan.hdr, c.plan.ctas, d_status, stream);
}

HP_API int hp_attention_prefix_planned(const hp_paged_desc* k_desc, const void* v_pool, const void* group_ptr,
                                       const void* prefix_lens, uint64_t num_groups, const void* q, const void* q_ptr,
                                       uint64_t total_q, uint32_t num_q_heads, float scale, void* out,
                                       void* workspace, uint64_t workspace_bytes, int* d_status, void* stream)
{
    PrefixCall c;
    const int rc = prefix_prepare(k_desc, v_pool, group_ptr, prefix_lens, num_groups, q, q_ptr, total_q, num_q_heads,
                                  scale, out, workspace, workspace_bytes, d_status, &c);
    return rc ? rc : prefix_run(c, 2, stream);
}

HP_API int hp_attention_prefix(const hp_paged_desc* k_desc, const void* v_pool, const void* group_ptr,
                               const void* prefix_lens, uint64_t num_groups, const void* q, const void* q_ptr,
                               uint64_t total_q, uint32_t num_q_heads, float scale, void* out, void* workspace,
                               uint64_t workspace_bytes, int* d_status, void* stream)
{
    PrefixCall c;
    int rc = prefix_prepare(k_desc, v_pool, group_ptr, prefix_lens, num_groups, q, q_ptr, total_q, num_q_heads, scale,
                            out, workspace, workspace_bytes, d_status, &c);
    if (rc) return rc;
    rc = hp::launch_prefix_plan(c.plan, stream);
    return rc ? rc : prefix_run(c, 1, stream);
}
