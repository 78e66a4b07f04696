// hp_abi_checks.cuh -- host-side argument checks shared by the entry points (hp_abi.cu,
// hp_abi_step.cu).
#pragma once

#include <cstdint>

#include "hp_internal.cuh"

#define HP_API extern "C" __attribute__((visibility("default")))

namespace {

using u64 = uint64_t;
using u128 = unsigned __int128;

inline u64 elem_bytes(uint32_t dtype)
{
    switch (dtype) {
    case HP_F32: return 4;
    case HP_F16: return 2;
    case HP_BF16: return 2;
    case HP_I8: return 1;
    case HP_U8: return 1;
    case HP_F64: return 8;
    default: return 0;
    }
}

inline bool misaligned(const void* p, u64 a) { return reinterpret_cast<uintptr_t>(p) % a != 0; }

inline int check_desc(const hp_paged_desc* d)
{
    if (!d) return HP_ERR_NULL;
    if (d->rank != 3) return HP_ERR_RANK;
    if (d->paged_axis != 0) return HP_ERR_PAGED_AXIS;
    if (d->has_shard) return HP_ERR_SHARD;
    if (d->index_type != HP_IDX_U32 && d->index_type != HP_IDX_U64) return HP_ERR_INDEX_TYPE;
    if (d->index_type == HP_IDX_U32 && (d->num_pages > (1ull << 32) || d->table_len > 0xFFFFFFFFull))
        return HP_ERR_INDEX_TYPE;
    const u64 es = elem_bytes(d->dtype);
    if (!es) return HP_ERR_DTYPE;
    if (!d->page_size || !d->num_heads || !d->head_dim) return HP_ERR_ZERO_DIM;
    const bool quant = d->flags & HP_HAS_QUANT;
    if (quant && (!d->scales || (u128)d->scales_len != (u128)d->num_pages * d->page_size))
        return HP_ERR_SCALES;
    if ((d->num_pages && !d->page_pool) || !d->seq_ptr || (d->num_seqs && !d->seq_lens) ||
        (d->table_len && !d->block_table))
        return HP_ERR_NULL;
    if (misaligned(d->page_pool, 64) || misaligned(d->block_table, 64) ||
        misaligned(d->seq_ptr, 64) || misaligned(d->seq_lens, 64) ||
        (quant && misaligned(d->scales, 64)))
        return HP_ERR_ALIGN;
    u128 bytes = (u128)d->num_pages * d->page_size;
    bytes *= d->num_heads;
    if (bytes >> 64) return HP_ERR_OVERFLOW;
    bytes *= d->head_dim;
    if (bytes >> 64) return HP_ERR_OVERFLOW;
    bytes *= es;
    if (bytes >> 64) return HP_ERR_OVERFLOW;
    return HP_OK;
}

inline u64 row_bytes_of(const hp_paged_desc* d)
{
    return d->num_heads * d->head_dim * elem_bytes(d->dtype);
}

inline int ws_bytes(const hp_paged_desc* d, u64* out)
{
    if (d->num_seqs >= (1ull << 58)) return HP_ERR_OVERFLOW;
    *out = hp::kWsHeaderBytes + 2 * hp::round_up_256(8 * (d->num_seqs + 1));
    return HP_OK;
}

inline int check_ws(const hp_paged_desc* d, const void* ws, u64 have)
{
    u64 need = 0;
    int rc = ws_bytes(d, &need);
    if (rc) return rc;
    if (!ws || misaligned(ws, 256) || have < need) return HP_ERR_WORKSPACE;
    return HP_OK;
}

// Widest power-of-two vector (<= 16 bytes) that divides the row and both bases.
inline int pick_vec(u64 row_bytes, const void* a, const void* b)
{
    const uintptr_t m = static_cast<uintptr_t>(row_bytes) | reinterpret_cast<uintptr_t>(a) |
                        reinterpret_cast<uintptr_t>(b);
    for (int v = 16; v > 1; v >>= 1)
        if (m % v == 0) return v;
    return 1;
}

inline hp::PlanArgs plan_args(const hp_paged_desc* d, void* ws, int* d_status)
{
    hp::PlanArgs a{};
    a.seq_ptr = d->seq_ptr;
    a.lens = d->seq_lens;
    a.table = d->block_table;
    a.num_seqs = d->num_seqs;
    a.page_size = d->page_size;
    a.table_len = d->table_len;
    a.num_pages = d->num_pages;
    a.strict = !(d->flags & HP_PERMISSIVE);
    a.d_status = d_status;
    a.ws = hp::ws_view(ws, d->num_seqs);
    return a;
}

}  // namespace
