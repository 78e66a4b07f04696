// hp_step.cuh -- launch interface of the serving-step kernels: block tables (hp_step.cu) and
// the norm + rotation + append kernels (hp_rope.cu).
#pragma once

#include <cstdint>

#include "hp_internal.cuh"

namespace hp {

constexpr uint32_t kStepBlocks = 256;  // blocks of sequences whose sums are local

struct StepArgs {
    hp_step_desc d;
    WsView ws;  // rows_off: prefix of the new tokens, units_off of the pages, within each block
    unsigned long long* blocks;  // [3][kStepBlocks]: each block's tokens, pages, verdict key
    uint64_t page_limit;         // 2^63 / page_size: the slots of pages below it fit an int64
    uint32_t block_log;          // log2 of a block's sequences
    uint32_t div_ok, div_m, div_l;  // div_invariant constants of page_size, where it fits
    int* d_status;
};
int launch_step_tables(const StepArgs& a, void* stream);

// The rotation, with the host's checks done: per-axis first pair, 0xFFFFFFFF past the last.
struct RopeArgs {
    const float* cos_sin;
    const void* positions;
    uint64_t max_pos;
    uint32_t rot, axes, inter, idx64;
    uint32_t first[4];
};

struct AppendArgs {
    RopeArgs rope;
    uint64_t tokens, num_slots;
    const int64_t* slot_map;
    float eps;
    // heads to rotate (queries): (t, h, d) at t * q_stride + h * q_head
    const void* q;
    void* q_out;
    uint64_t q_stride, q_head, qo_stride, qo_head;
    uint32_t hq, dim;
    const void* q_weight;
    // K/V heads (hp_qk_norm_rope_append)
    uint32_t hkv;
    const void *k, *v;
    uint64_t k_stride, v_stride;
    const void* k_weight;
    void *k_pool, *v_pool;
    // latent rows (hp_latent_append)
    const void* latent;
    uint64_t latent_stride;
    const void* latent_weight;
    uint32_t latent_dim;
    int* d_status;
};
int launch_qk_append(uint32_t dtype, const AppendArgs& a, void* stream);
int launch_latent_append(uint32_t dtype, const AppendArgs& a, void* stream);

}  // namespace hp
