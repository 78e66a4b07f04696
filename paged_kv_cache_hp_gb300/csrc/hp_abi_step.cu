// hp_abi_step.cu -- the entry points of a serving step (include/hp.h): step tables, norm +
// rotation + append, latent attention.  Host-side checks, then launches on the caller's stream.
#include <cuda_runtime.h>

#include <algorithm>

#include "hp_abi_checks.cuh"
#include "hp_latent.cuh"
#include "hp_step.cuh"

namespace {

constexpr u64 kMost = 1ull << 58;

u64 index_bytes(uint32_t index_type) { return index_type == HP_IDX_U64 ? 8 : 4; }

int reset_status(int* d_status, void* stream)
{
    if (!d_status) return HP_OK;
    return cudaMemsetAsync(d_status, 0, sizeof(int), static_cast<cudaStream_t>(stream)) ==
                   cudaSuccess
               ? HP_OK
               : HP_ERR_CUDA;
}

u64 step_ws_bytes(u64 num_seqs)
{
    return hp::kWsHeaderBytes + 2 * hp::round_up_256(8 * (num_seqs + 1)) + 3 * 8 * hp::kStepBlocks;
}

}  // namespace

HP_API int hp_step_tables_workspace_bytes(uint64_t num_seqs, uint64_t* bytes)
{
    if (!bytes) return HP_ERR_NULL;
    if (num_seqs >= kMost) return HP_ERR_OVERFLOW;
    *bytes = step_ws_bytes(num_seqs);
    return HP_OK;
}

HP_API int hp_step_tables(const hp_step_desc* step, void* workspace, uint64_t workspace_bytes,
                          int* d_status, void* stream)
{
    if (!step) return HP_ERR_NULL;
    const hp_step_desc& d = *step;
    if (d.index_type != HP_IDX_U32 && d.index_type != HP_IDX_U64) return HP_ERR_INDEX_TYPE;
    if (!d.page_size) return HP_ERR_ZERO_PAGE_SIZE;
    if (d.reserved) return HP_ERR_ARG;
    if (d.num_seqs >= kMost || d.page_size >= kMost || d.table_len >= kMost ||
        d.num_free >= kMost || d.table_cap >= kMost || d.token_cap >= kMost ||
        d.table_cap + d.token_cap > (1ull << 41) || d.num_seqs > (1ull << 37))
        return HP_ERR_OVERFLOW;  // (2,048 entries or tokens or 256 sequences a CTA: 1.5 2^30 CTAs of 2^31 - 1)
    if (!d.seq_ptr || !d.seq_ptr_out || !d.new_ptr_out ||
        (d.num_seqs && (!d.seq_lens || !d.new_lens || !d.lens_out)) ||
        (d.table_len && !d.block_table) || (d.num_free && !d.free_pages) ||
        (d.table_cap && !d.table_out) || (d.token_cap && (!d.slot_map || !d.positions)))
        return HP_ERR_NULL;
    const u64 w = index_bytes(d.index_type);
    for (const void* p : {d.block_table, d.seq_ptr, d.seq_lens, d.new_lens, d.free_pages,
                          (const void*)d.table_out, (const void*)d.seq_ptr_out,
                          (const void*)d.lens_out, (const void*)d.new_ptr_out,
                          (const void*)d.positions})
        if (misaligned(p, w)) return HP_ERR_ALIGN;
    if (misaligned(d.slot_map, 8) || misaligned(d.totals, 8)) return HP_ERR_ALIGN;
    if (!workspace || misaligned(workspace, 256) || workspace_bytes < step_ws_bytes(d.num_seqs))
        return HP_ERR_WORKSPACE;
    hp::StepArgs a{};
    a.d = d;
    a.ws = hp::ws_view(workspace, d.num_seqs);
    a.blocks = a.ws.units_off + hp::round_up_256(8 * (d.num_seqs + 1)) / 8;
    a.div_ok = d.page_size <= (1ull << 31);
    if (a.div_ok) hp::invariant_divisor(d.page_size, &a.div_m, &a.div_l);
    a.page_limit = (1ull << 63) / d.page_size;
    a.d_status = d_status;
    return hp::launch_step_tables(a, stream);
}

namespace {

// The rotation's own checks; `tokens` rows of positions.
int check_rope(const hp_rope_desc* r, u64 tokens, hp::RopeArgs* out)
{
    if (r->index_type != HP_IDX_U32 && r->index_type != HP_IDX_U64) return HP_ERR_INDEX_TYPE;
    if (r->rot_dim == 0 || r->rot_dim % 16 || r->rot_dim > 256) return HP_ERR_ARG;
    if (r->axes < 1 || r->axes > 4 || r->interleaved > 1) return HP_ERR_ARG;
    u64 pairs = 0;
    for (uint32_t x = 0; x < r->axes; ++x) pairs += r->section[x];
    if (pairs != r->rot_dim / 2) return HP_ERR_ARG;
    if (((u128)r->max_pos * r->rot_dim * 4) >> 63) return HP_ERR_OVERFLOW;
    if (tokens && (!r->positions || (r->max_pos && !r->cos_sin))) return HP_ERR_NULL;
    if (misaligned(r->cos_sin, 16) || misaligned(r->positions, index_bytes(r->index_type)))
        return HP_ERR_ALIGN;
    out->cos_sin = r->cos_sin;
    out->positions = r->positions;
    out->max_pos = r->max_pos;
    out->rot = r->rot_dim;
    out->axes = r->axes;
    out->inter = r->interleaved;
    out->idx64 = r->index_type == HP_IDX_U64;
    uint32_t first = 0;
    for (uint32_t x = 0; x < 4; ++x) {
        out->first[x] = x < r->axes ? first : 0xFFFFFFFFu;
        if (x < r->axes) first += r->section[x];
    }
    return HP_OK;
}

// A pool of num_pages x page_size rows of row_bytes; *slots receives the slot count.
int check_pool(u64 num_pages, u64 page_size, u64 row_bytes, u64* slots)
{
    if (!page_size) return HP_ERR_ZERO_DIM;
    const u128 n = (u128)num_pages * page_size;
    if (n >> 63 || (n * row_bytes) >> 63) return HP_ERR_OVERFLOW;
    *slots = (u64)n;
    return HP_OK;
}

// `tokens` rows at `stride` elements each must be addressable and 16-byte steps.
int check_rows(const void* p, u64 tokens, u64 stride, u64 es)
{
    if (misaligned(p, 16) || (stride * es) % 16) return HP_ERR_ALIGN;
    if (((u128)tokens * stride * es) >> 63) return HP_ERR_OVERFLOW;
    return HP_OK;
}

bool float_type(uint32_t dtype) { return dtype == HP_F32 || dtype == HP_F16 || dtype == HP_BF16; }

}  // namespace

HP_API int hp_qk_norm_rope_append(const hp_qk_desc* qk, const hp_rope_desc* rope, int* d_status,
                                  void* stream)
{
    if (!qk) return HP_ERR_NULL;
    const hp_qk_desc& d = *qk;
    if (!float_type(d.dtype)) return HP_ERR_DTYPE;
    if (!d.num_kv_heads || !d.head_dim) return HP_ERR_ZERO_DIM;
    if (d.head_dim % 8 || d.head_dim > 256 || d.reserved || d.num_q_heads > (1u << 20) ||
        d.num_kv_heads > (1u << 20) || d.num_tokens >= kMost)
        return HP_ERR_ARG;
    hp::AppendArgs a{};
    if (rope) {
        const int rc = check_rope(rope, d.num_tokens, &a.rope);
        if (rc) return rc;
        if (rope->rot_dim > d.head_dim) return HP_ERR_ARG;
    }
    const u64 es = elem_bytes(d.dtype);
    int rc = check_pool(d.num_pages, d.page_size, (u64)d.num_kv_heads * d.head_dim * es, &a.num_slots);
    if (rc) return rc;
    if (d.num_tokens && (!d.k || !d.v || !d.slot_map || (d.num_q_heads && (!d.q || !d.q_out))))
        return HP_ERR_NULL;
    if (d.num_pages && (!d.k_pool || !d.v_pool)) return HP_ERR_NULL;
    if ((rc = check_rows(d.k, d.num_tokens, d.k_stride, es)) ||
        (rc = check_rows(d.v, d.num_tokens, d.v_stride, es)))
        return rc;
    if (d.num_q_heads && ((rc = check_rows(d.q, d.num_tokens, d.q_stride, es)) ||
                          (rc = check_rows(d.q_out, d.num_tokens, d.q_out_stride, es))))
        return rc;
    if (misaligned(d.k_pool, 16) || misaligned(d.v_pool, 16) || misaligned(d.q_weight, 16) ||
        misaligned(d.k_weight, 16) || misaligned(d.slot_map, 8))
        return HP_ERR_ALIGN;
    if (d.num_tokens == 0) return reset_status(d_status, stream);
    a.tokens = d.num_tokens;
    a.slot_map = d.slot_map;
    a.eps = d.eps;
    a.q = d.q;
    a.q_out = d.q_out;
    a.q_stride = d.q_stride;
    a.qo_stride = d.q_out_stride;
    a.q_head = a.qo_head = d.head_dim;
    a.hq = d.num_q_heads;
    a.dim = d.head_dim;
    a.q_weight = d.q_weight;
    a.hkv = d.num_kv_heads;
    a.k = d.k;
    a.v = d.v;
    a.k_stride = d.k_stride;
    a.v_stride = d.v_stride;
    a.k_weight = d.k_weight;
    a.k_pool = d.k_pool;
    a.v_pool = d.v_pool;
    a.d_status = d_status;
    return hp::launch_qk_append(d.dtype, a, stream);
}

HP_API int hp_latent_append(const hp_latent_desc* latent, const hp_rope_desc* rope, int* d_status,
                            void* stream)
{
    if (!latent || !rope) return HP_ERR_NULL;
    const hp_latent_desc& d = *latent;
    if (!float_type(d.dtype)) return HP_ERR_DTYPE;
    if (!d.latent_dim) return HP_ERR_ZERO_DIM;
    if (d.latent_dim % 8 || d.latent_dim > 1024 || d.num_q_heads > (1u << 20) ||
        d.num_tokens >= kMost)
        return HP_ERR_ARG;
    hp::AppendArgs a{};
    int rc = check_rope(rope, d.num_tokens, &a.rope);
    if (rc) return rc;
    const u64 es = elem_bytes(d.dtype);
    rc = check_pool(d.num_pages, d.page_size, (u64)(d.latent_dim + rope->rot_dim) * es, &a.num_slots);
    if (rc) return rc;
    if (d.num_tokens && (!d.latent || !d.k_rope || !d.slot_map ||
                         (d.num_q_heads && (!d.q_rope || !d.q_out))))
        return HP_ERR_NULL;
    if (d.num_pages && !d.pool) return HP_ERR_NULL;
    if ((rc = check_rows(d.latent, d.num_tokens, d.latent_stride, es)) ||
        (rc = check_rows(d.k_rope, d.num_tokens, d.k_rope_stride, es)))
        return rc;
    if (d.num_q_heads &&
        ((rc = check_rows(d.q_rope, d.num_tokens, d.q_stride, es)) ||
         (rc = check_rows(d.q_out, d.num_tokens, d.q_out_stride, es)) ||
         (rc = check_rows(d.q_rope, d.num_q_heads, d.q_head_stride, es)) ||
         (rc = check_rows(d.q_out, d.num_q_heads, d.q_out_head_stride, es))))
        return rc;
    if (misaligned(d.pool, 16) || misaligned(d.latent_weight, 16) || misaligned(d.slot_map, 8))
        return HP_ERR_ALIGN;
    if (d.num_tokens == 0) return reset_status(d_status, stream);
    a.tokens = d.num_tokens;
    a.slot_map = d.slot_map;
    a.eps = d.eps;
    a.q = d.q_rope;
    a.q_out = d.q_out;
    a.q_stride = d.q_stride;
    a.q_head = d.q_head_stride;
    a.qo_stride = d.q_out_stride;
    a.qo_head = d.q_out_head_stride;
    a.hq = d.num_q_heads;
    a.dim = rope->rot_dim;
    a.k = d.k_rope;
    a.k_stride = d.k_rope_stride;
    a.k_pool = d.pool;
    a.latent = d.latent;
    a.latent_stride = d.latent_stride;
    a.latent_weight = d.latent_weight;
    a.latent_dim = d.latent_dim;
    a.d_status = d_status;
    return hp::launch_latent_append(d.dtype, a, stream);
}

namespace {

// Checks shared by the latent-attention entry points, on a strict copy of the descriptor.
int check_latent(const hp_paged_desc* desc, uint32_t latent_dim, u64 total_q, uint32_t heads,
                 hp_paged_desc* d)
{
    if (!desc) return HP_ERR_NULL;
    *d = *desc;
    d->flags &= ~(HP_PERMISSIVE | HP_HAS_QUANT);
    const int rc = check_desc(d);
    if (rc) return rc;
    if (d->dtype != HP_F16 && d->dtype != HP_BF16) return HP_ERR_DTYPE;
    if (d->num_heads != 1 || latent_dim == 0 || latent_dim % 64 || latent_dim > 512)
        return HP_ERR_ARG;
    if (d->head_dim < (u64)latent_dim + 8 || d->head_dim > (u64)latent_dim + 64 ||
        d->head_dim % 8 || d->page_size > (1u << 26) || heads == 0 || heads > 4096)
        return HP_ERR_ARG;
    // unit indices (row groups x steps), element indices and byte offsets fit 64 bits
    const u128 rows = (u128)total_q * heads;
    const u128 steps = (u128)d->table_len * d->page_size / hp::kLatentStep + 1;
    if (rows >> 48 || steps >> 56 || (rows + d->num_seqs) * steps >> 62) return HP_ERR_OVERFLOW;
    return HP_OK;
}

int check_q_ptr(const hp_paged_desc& d, const void* q_ptr, u64 total_q)
{
    if (!q_ptr) return total_q == d.num_seqs ? HP_OK : HP_ERR_ARG;
    return misaligned(q_ptr, index_bytes(d.index_type)) ? HP_ERR_ALIGN : HP_OK;
}

bool latent_on_tensor_cores(const hp_paged_desc& d, uint32_t latent_dim, u64 q_rows)
{
    return !(d.flags & (HP_ATTN_CUDA_CORES | HP_HOST_MEMORY)) &&
           hp::latent_tc_fits(latent_dim, d.head_dim, d.page_size, d.num_pages, q_rows);
}

// Tensor cores: tiles of 64 rows; above 64 heads a worker is a pair of CTAs whose two tiles
// read the same tokens at the same time.
uint32_t latent_group_rows(bool tc, uint32_t heads)
{
    return !tc ? hp::kLatentCcRows : (heads > 64 ? 128 : 64);
}

u64 latent_records(uint32_t latent_dim)
{
    return (u64)hp::kLatentMaxSms * hp::kLatentRecordRows * (latent_dim + 2) * 4 +
           2 * (u64)hp::kLatentMaxSms * sizeof(hp::LatentMerge);
}

// Whether the first kernel of a call makes the plan itself (hp_latent_plan.cuh): few sequences, a
// short table, and sums that fit 32 bits.
bool plans_itself(const hp_paged_desc& d, u64 total_q, uint32_t heads, uint32_t group_rows)
{
    const u128 groups = (u128)total_q * heads / group_rows + d.num_seqs;
    const u128 steps = (u128)d.table_len * d.page_size / hp::kLatentStep + 1;
    return d.num_seqs > 0 && d.num_seqs <= hp::kSmallSeqs && d.table_len <= hp::kPlanTable && total_q > 0 &&
           (groups * steps) >> 31 == 0 && (steps * hp::kLatentStep + (u128)hp::kLatentPad * d.num_seqs) >> 31 == 0;
}

// The plan of the absorbed form (q_ptr: see hp_latent_decode).  Block tables up to kPlanTable
// entries are checked by the plan's one CTA (four loads a thread) instead of a launch of their own,
// which is 2.5 us.
hp::PlanArgs decode_plan(const hp_paged_desc& d, const void* q_ptr, u64 total_q, uint32_t heads, uint32_t group_rows,
                         void* workspace, int* d_status)
{
    hp::PlanArgs pa = plan_args(&d, workspace, d_status);
    pa.new_ptr = q_ptr;
    pa.total_new = total_q;
    pa.step_tokens = hp::kLatentStep;
    pa.heads = heads;
    pa.group_rows = group_rows;
    pa.row_round = 1;
    pa.check_table = d.table_len <= hp::kPlanTable;
    return pa;
}

int latent_prepare(const hp_paged_desc* desc, uint32_t latent_dim, const void* q_ptr, u64 total_q,
                   uint32_t heads, const void* ws, u64 ws_bytes_, hp_paged_desc* d, u64* plan_bytes)
{
    int rc = check_latent(desc, latent_dim, total_q, heads, d);
    if (rc) return rc;
    rc = check_q_ptr(*d, q_ptr, total_q);
    if (rc) return rc;
    rc = ws_bytes(d, plan_bytes);
    if (rc) return rc;
    if (!ws || misaligned(ws, 256) || ws_bytes_ < *plan_bytes + latent_records(latent_dim))
        return HP_ERR_WORKSPACE;
    return HP_OK;
}

int latent_buffers(const void* q, const void* out, u64 total_q)
{
    if (total_q && (!q || !out)) return HP_ERR_NULL;
    return misaligned(q, 16) || misaligned(out, 16) ? HP_ERR_ALIGN : HP_OK;
}

}  // namespace

HP_API int hp_latent_decode_workspace_bytes(const hp_paged_desc* desc, uint32_t latent_dim,
                                            uint64_t total_q, uint32_t num_q_heads, uint64_t* bytes)
{
    (void)total_q;
    (void)num_q_heads;
    if (!desc || !bytes) return HP_ERR_NULL;
    u64 plan = 0;
    const int rc = ws_bytes(desc, &plan);
    if (rc) return rc;
    if (plan > (1ull << 62)) return HP_ERR_OVERFLOW;
    *bytes = plan + latent_records(latent_dim);
    return HP_OK;
}

HP_API int hp_latent_plan(const hp_paged_desc* desc, uint32_t latent_dim, const void* q_ptr,
                          uint64_t total_q, uint32_t num_q_heads, void* workspace,
                          uint64_t workspace_bytes, int* d_status, void* stream)
{
    hp_paged_desc d;
    u64 plan = 0;
    const int rc = latent_prepare(desc, latent_dim, q_ptr, total_q, num_q_heads, workspace,
                                  workspace_bytes, &d, &plan);
    if (rc) return rc;
    const uint32_t gr = latent_group_rows(latent_on_tensor_cores(d, latent_dim, total_q * num_q_heads), num_q_heads);
    const hp::PlanArgs pa = decode_plan(d, q_ptr, total_q, num_q_heads, gr, workspace, d_status);
    return hp::launch_plan(hp::kPlanLatent, d.index_type == HP_IDX_U64, pa, stream);
}

namespace {

// The absorbed form behind a plan in the workspace, or, with `alone`, with its own.
int decode(const hp_paged_desc* desc, uint32_t latent_dim, const void* q, const void* q_ptr, uint64_t total_q,
           uint32_t num_q_heads, float scale, void* out, void* workspace, uint64_t workspace_bytes, int* d_status,
           void* stream, bool alone)
{
    hp_paged_desc d;
    u64 plan = 0;
    int rc = latent_prepare(desc, latent_dim, q_ptr, total_q, num_q_heads, workspace,
                            workspace_bytes, &d, &plan);
    if (rc) return rc;
    rc = latent_buffers(q, out, total_q);
    if (rc) return rc;
    const bool tc = latent_on_tensor_cores(d, latent_dim, total_q * num_q_heads);
    const uint32_t gr = latent_group_rows(tc, num_q_heads);
    const bool small = alone && tc && plans_itself(d, total_q, num_q_heads, gr);
    if (alone && !small) {
        rc = hp_latent_plan(desc, latent_dim, q_ptr, total_q, num_q_heads, workspace, workspace_bytes, d_status,
                            stream);
        if (rc) return rc;
    }
    if (d.num_seqs == 0 || total_q == 0) return HP_OK;
    int dev = 0;
    const u64 sms = std::min<u64>((u64)hp::current_sms(&dev), hp::kLatentMaxSms);
    if (sms == 0) return HP_ERR_CUDA;
    const hp::WsView ws = hp::ws_view(workspace, d.num_seqs);
    hp::LatentArgs a{};
    a.pool = d.page_pool;
    a.q = q;
    a.q_ptr = q_ptr;
    a.table = d.block_table;
    a.seq_ptr = d.seq_ptr;
    a.lens = d.seq_lens;
    a.num_seqs = d.num_seqs;
    a.page_size = d.page_size;
    a.num_pages = d.num_pages;
    a.total_q = total_q;
    a.H = num_q_heads;
    a.R = latent_dim;
    a.W = (uint32_t)d.head_dim;
    a.group_rows = gr;
    if (tc) hp::invariant_divisor(d.page_size / 8, &a.g_m, &a.g_l);
    a.workers = tc ? sms / (a.group_rows / 64) : 2 * sms;
    a.scale = scale;
    a.bf16 = d.dtype == HP_BF16;
    a.idx64 = d.index_type == HP_IDX_U64;
    a.test_stall = (d.flags & HP_TEST_STALL) != 0;
    a.small = small;
    a.plan = decode_plan(d, q_ptr, total_q, num_q_heads, gr, workspace, d_status);
    a.hdr = ws.hdr;
    a.units_off = ws.units_off;
    a.part_acc = reinterpret_cast<float*>(static_cast<char*>(workspace) + plan);
    a.part_ml = reinterpret_cast<float2*>(a.part_acc +
                                          (u64)hp::kLatentMaxSms * hp::kLatentRecordRows * latent_dim);
    a.merge = reinterpret_cast<hp::LatentMerge*>(a.part_ml + (u64)hp::kLatentMaxSms * hp::kLatentRecordRows);
    a.out = out;
    a.d_status = d_status;
    rc = tc ? hp::launch_latent_tc(a, stream) : hp::launch_latent_cc(a, stream);
    return rc ? rc : hp::launch_latent_merge(a, stream);
}

}  // namespace

HP_API int hp_latent_decode_planned(const hp_paged_desc* desc, uint32_t latent_dim, const void* q,
                                    const void* q_ptr, uint64_t total_q, uint32_t num_q_heads,
                                    float scale, void* out, void* workspace,
                                    uint64_t workspace_bytes, int* d_status, void* stream)
{
    return decode(desc, latent_dim, q, q_ptr, total_q, num_q_heads, scale, out, workspace, workspace_bytes, d_status,
                  stream, false);
}

HP_API int hp_latent_decode(const hp_paged_desc* desc, uint32_t latent_dim, const void* q,
                            const void* q_ptr, uint64_t total_q, uint32_t num_q_heads, float scale,
                            void* out, void* workspace, uint64_t workspace_bytes, int* d_status,
                            void* stream)
{
    return decode(desc, latent_dim, q, q_ptr, total_q, num_q_heads, scale, out, workspace, workspace_bytes, d_status,
                  stream, true);
}

namespace {

// Byte offsets of the expanded form's buffers behind the plan.
struct PrefillWs {
    u64 plan, cap_rows, rows_bytes, kv_bytes, unit_bytes;
    u64 total() const { return plan + rows_bytes + kv_bytes + unit_bytes; }
};

// Blocks of `block` queries that total_q queries of num_seqs sequences can make.
u64 most_units(u64 total_q, u64 num_seqs, uint32_t block)
{
    return total_q / block + std::min<u64>(num_seqs, total_q);
}

int prefill_ws(const hp_paged_desc* d, uint32_t nope, uint32_t v, u64 total_q, uint32_t heads, u64 kv_tokens,
               PrefillWs* w)
{
    const int rc = ws_bytes(d, &w->plan);
    if (rc) return rc;
    const u128 rows = ((u128)kv_tokens + (u128)(hp::kLatentPad - 1) * d->num_seqs + hp::kLatentPad - 1) /
                      hp::kLatentPad * hp::kLatentPad;
    const u128 row = (u128)d->head_dim * 2, kv = (u128)heads * ((u64)nope + v) * 2;
    if (rows >> 36 || row >> 24 || (rows * (row + kv)) >> 60 || total_q >> 48) return HP_ERR_OVERFLOW;
    w->cap_rows = (u64)rows;
    w->rows_bytes = hp::round_up_256((u64)(rows * row));
    w->kv_bytes = hp::round_up_256((u64)(rows * kv));
    w->unit_bytes =
        hp::round_up_256(most_units(total_q, d->num_seqs, hp::kLatentTcQueries) * sizeof(hp::LatentUnit));
    return HP_OK;
}

}  // namespace

HP_API int hp_latent_prefill_workspace_bytes(const hp_paged_desc* desc, uint32_t latent_dim,
                                             uint32_t nope_dim, uint32_t v_dim, uint64_t total_q,
                                             uint32_t num_q_heads, uint64_t kv_tokens,
                                             uint64_t* bytes)
{
    (void)latent_dim;
    if (!desc || !bytes) return HP_ERR_NULL;
    PrefillWs w;
    const int rc = prefill_ws(desc, nope_dim, v_dim, total_q, num_q_heads, kv_tokens, &w);
    if (rc) return rc;
    *bytes = w.total();
    return HP_OK;
}

HP_API int hp_latent_prefill(const hp_paged_desc* desc, uint32_t latent_dim, const void* w_kv,
                             uint32_t nope_dim, uint32_t v_dim, const void* q, const void* q_ptr,
                             uint64_t total_q, uint32_t num_q_heads, float scale, void* out,
                             uint64_t kv_tokens, void* workspace, uint64_t workspace_bytes,
                             int* d_status, void* stream)
{
    hp_paged_desc d;
    int rc = check_latent(desc, latent_dim, total_q, num_q_heads, &d);
    if (rc) return rc;
    if (nope_dim == 0 || nope_dim % 16 || nope_dim > 256 || v_dim == 0 || v_dim % 16 || v_dim > 256)
        return HP_ERR_ARG;
    rc = check_q_ptr(d, q_ptr, total_q);
    if (rc) return rc;
    PrefillWs w;
    rc = prefill_ws(&d, nope_dim, v_dim, total_q, num_q_heads, kv_tokens, &w);
    if (rc) return rc;
    if (!workspace || misaligned(workspace, 256) || workspace_bytes < w.total())
        return HP_ERR_WORKSPACE;
    if (!w_kv) return HP_ERR_NULL;
    if (misaligned(w_kv, 16)) return HP_ERR_ALIGN;
    rc = latent_buffers(q, out, total_q);
    if (rc) return rc;
    const bool tc = !(d.flags & HP_ATTN_CUDA_CORES) &&
                    hp::latent_prefill_tc_fits(latent_dim, d.head_dim, nope_dim, v_dim, w.cap_rows,
                                               total_q, num_q_heads);
    const uint32_t block = tc ? hp::kLatentTcQueries : hp::kLatentCcQueries;
    const u64 max_units = most_units(total_q, d.num_seqs, block);
    if (max_units >= (1ull << 31)) return HP_ERR_OVERFLOW;
    hp::PlanArgs pa = plan_args(&d, workspace, d_status);
    pa.new_ptr = q_ptr;
    pa.total_new = total_q;
    pa.step_tokens = hp::kLatentStep;
    pa.heads = 0;
    pa.group_rows = block;
    pa.row_round = hp::kLatentPad;
    pa.out_tokens = kv_tokens;
    pa.check_table = d.table_len <= hp::kPlanTable;
    const bool small = tc && plans_itself(d, total_q, 1, block);
    if (!small) {
        rc = hp::launch_plan(hp::kPlanLatent, d.index_type == HP_IDX_U64, pa, stream);
        if (rc) return rc;
        if (d.num_seqs == 0 || total_q == 0) return HP_OK;
    }
    const hp::WsView ws = hp::ws_view(workspace, d.num_seqs);
    hp::LatentPrefillArgs a{};
    a.pool = d.page_pool;
    a.w_kv = w_kv;
    a.q = q;
    a.q_ptr = q_ptr;
    a.table = d.block_table;
    a.seq_ptr = d.seq_ptr;
    a.lens = d.seq_lens;
    a.num_seqs = d.num_seqs;
    a.page_size = d.page_size;
    a.num_pages = d.num_pages;
    a.total_q = total_q;
    a.cap_rows = w.cap_rows;
    a.max_units = max_units;
    a.H = num_q_heads;
    a.R = latent_dim;
    a.W = (uint32_t)d.head_dim;
    a.Dn = nope_dim;
    a.Dv = v_dim;
    a.q_block = block;
    a.scale = scale;
    a.bf16 = d.dtype == HP_BF16;
    a.idx64 = d.index_type == HP_IDX_U64;
    a.test_stall = (d.flags & HP_TEST_STALL) != 0;
    a.small = small;
    a.plan = pa;
    a.hdr = ws.hdr;
    a.rows_off = ws.rows_off;
    a.units_off = ws.units_off;
    a.rows = static_cast<char*>(workspace) + w.plan;
    a.blocked = tc;
    a.rope_blocks = static_cast<char*>(a.rows) + w.cap_rows * latent_dim * 2;
    a.kv = static_cast<char*>(a.rows) + w.rows_bytes;
    a.units = reinterpret_cast<hp::LatentUnit*>(static_cast<char*>(a.kv) + w.kv_bytes);
    a.out = out;
    a.d_status = d_status;
    rc = hp::launch_latent_rows(a, stream);
    if (rc) return rc;
    return tc ? hp::launch_latent_prefill_tc(a, stream) : hp::launch_latent_prefill_cc(a, stream);
}
