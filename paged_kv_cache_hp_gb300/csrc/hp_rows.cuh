// hp_rows.cuh -- launch interface of attention for single query rows over lists or stretches of
// pages (hp_attn_rows.cu) and of the shared prefix in front of them (hp_prefix.cu, hp_prefix_tc.cu).
#pragma once

#include <cfloat>
#include <cstdint>

#include "hp_pages.cuh"

namespace hp {

// The least reference maximum (log2 units) of a part that saw a token; -inf where it saw none.
constexpr float kLowest = -FLT_MAX;
constexpr uint32_t kPrefixKeys = 128;      // keys of a step of the shared prefix
constexpr uint32_t kPrefixRows = 256;      // (query, head) rows of a tile: two tiles of 128 to the tensor core
constexpr uint32_t kPrefixMaxSms = 160;    // workers are counted for at most this many SMs
constexpr uint32_t kPrefixPlanCtas = 128;  // at most, and as many verdicts
constexpr uint64_t kPrefixPlanPart = 8192; // table entries that a CTA of the plan looks at (more in a longer table)

// A query row of hp_attention_prefix, as the plan leaves it.
struct PrefixRow {
    uint64_t table;      // first entry of its sequence's slice
    uint32_t prefix;     // tokens that its group shares
    uint32_t seen;       // tokens it sees (of its whole sequence)
    uint32_t group;      // 0xFFFFFFFF: no sequence has this row
    uint32_t local;      // row within its group
};

// A group: its prefix is read through the slice of its first sequence.
struct PrefixGroup {
    uint64_t table;      // first entry of that slice
    uint64_t row0;       // first query row
    uint64_t step0;      // steps before it: tile after tile (head after head), the blocks of keys of each
    uint64_t rows0;      // record rows before it
    uint32_t rows;       // query rows
    uint32_t prefix;
    uint32_t blocks;     // of kPrefixKeys keys
    uint32_t tiles;      // of a head
    uint64_t records;    // record rows of a head: a tile's rows, twice those of a tile of up to 128
};

struct PrefixHeader {
    unsigned long long steps;  // of all groups
    unsigned long long keys[kPrefixPlanCtas];  // the verdict of each of the plan's CTAs
};

inline uint32_t prefix_plan_ctas(uint64_t table_len)
{
    const uint64_t n = 1 + table_len / kPrefixPlanPart;
    return n < kPrefixPlanCtas ? (uint32_t)n : kPrefixPlanCtas;
}

struct PrefixPlanArgs {
    const void *seq_ptr, *lens, *table, *q_ptr, *group_ptr, *prefix_lens;
    uint64_t num_seqs, num_groups, total_q, table_len, num_pages;
    uint32_t P, H, G;
    int idx64;
    PrefixHeader* hdr;
    PrefixRow* rows;
    PrefixGroup* groups;   // [num_groups]
    uint32_t ctas;         // prefix_plan_ctas(table_len)
};
int launch_prefix_plan(const PrefixPlanArgs& a, void* stream);
// The plan's verdict to the status word (a call that runs the plan alone, or has no rows).
int launch_prefix_status(const PrefixHeader* hdr, uint32_t ctas, int* d_status, void* stream);

// The records that the prefix's workers leave: worker v's part of a tile whose record rows begin at R
// (of all tiles, in order) at rows R + v * kPrefixRows ..., no two of them in one place since a part has at
// most kPrefixRows record rows.  A tile of up to 128 rows has two records a part, one behind the other.
struct PrefixRecords {
    float* acc;            // [rows, D]
    float2* ml;            // [rows]: maximum (log2 units) and sum
    uint64_t workers;      // 0: no records (the rows read their prefixes themselves)
};

struct PrefixTcArgs {
    const void *k_pool, *v_pool, *q, *table;
    uint64_t num_groups, num_pages, workers;
    uint32_t P, H, G;
    uint32_t box;          // slots of a load: the largest power of two up to 128 that divides P
    float scale;
    int bf16, idx64, test_stall;
    const PrefixHeader* hdr;
    const PrefixGroup* groups;
    uint32_t num_keys;     // verdicts in hdr
    int first;             // the call's first kernel behind its plan: it stores the status
    PrefixRecords rec;
    int* d_status;
};
bool prefix_tc_shape(uint64_t head_dim, uint64_t page_size);
bool prefix_tc_fits(uint64_t head_dim, uint64_t page_size, uint64_t num_pages);
uint32_t prefix_tc_box(uint64_t page_size);
int launch_prefix_tc(const PrefixTcArgs& a, uint32_t head_dim, void* stream);

struct RowsArgs {
    QueryArgs q;           // lists
    PageTable t;
    const void *k_pool, *v_pool, *queries;
    void* out;             // [total_q, H * G, D]
    uint32_t P, p_m, p_l;  // page size and its div_invariant constants
    uint32_t H, G, D;
    float scale;
    int bf16;
    uint32_t cluster;      // CTAs of a (row, K/V head)
    // lists
    const int32_t* selected;  // [total_q, H, k]; NULL: stretches
    uint32_t k;
    int check_all;
    int* d_status;
    // stretches behind a plan
    const PrefixHeader* hdr;
    uint32_t num_keys;
    int first;
    const PrefixRow* rows;
    const PrefixGroup* groups;
    PrefixRecords rec;
};
int launch_rows(const RowsArgs& a, void* stream);

}  // namespace hp
