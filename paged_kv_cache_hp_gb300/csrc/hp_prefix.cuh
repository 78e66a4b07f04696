// hp_prefix.cuh -- how the kernels behind a plan of hp_attention_prefix learn its verdict.
#pragma once

#include "hp_rows.cuh"

namespace hp {

// Whether the plan holds, the same in the whole CTA, by all its threads (at least kPrefixPlanCtas of them).  `tell`: one CTA of
// the call's first kernel stores the status, HP_OK or the first failing rule's; of a planned call only the latter.
__device__ __forceinline__ bool plan_holds(const PrefixHeader* hdr, uint32_t n, int* d_status, bool tell, bool planned)
{
    __shared__ unsigned long long s_first;
    const unsigned long long key = threadIdx.x < n ? hdr->keys[threadIdx.x] : kVerdictOk;
    const bool bad = __syncthreads_or(key != kVerdictOk);
    if (tell && d_status) {  // (the same in the whole CTA)
        if (threadIdx.x == 0) s_first = kVerdictOk;
        __syncthreads();
        if (key != kVerdictOk) atomicMin(&s_first, key);
        __syncthreads();
        if (threadIdx.x == 0 && (bad || !planned)) *d_status = key_status(s_first);
    }
    return !bad;
}

}  // namespace hp
