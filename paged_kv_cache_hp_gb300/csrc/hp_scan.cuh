// hp_scan.cuh -- helpers of the planning kernels (hp_plan.cu, hp_step.cu, hp_latent_plan.cuh): the
// saturating block scan of the one-CTA ones, a division.
#pragma once

#include <cuda_runtime.h>

namespace hp {

constexpr int kPlanThreads = 1024;
constexpr int kWarps = kPlanThreads / 32;

__device__ __forceinline__ unsigned long long sat_add(unsigned long long a, unsigned long long b)
{
    unsigned long long c = a + b;
    return c < a ? ~0ull : c;
}

// a / b, in 32 bits where both fit (a 64-bit division is some hundred instructions).
__device__ __forceinline__ unsigned long long quotient(unsigned long long a, unsigned long long b)
{
    return (a | b) >> 32 ? a / b : (unsigned long long)((unsigned)a / (unsigned)b);
}

// Exclusive block scan of two counters at once with saturating addition (which is
// associative: it is min(a + b, 2^64 - 1) over the naturals).  Returns the
// exclusive prefixes; *tot receives the block totals.
__device__ __forceinline__ void block_scan2(unsigned long long v0, unsigned long long v1,
                                            unsigned long long& ex0, unsigned long long& ex1,
                                            unsigned long long& tot0, unsigned long long& tot1)
{
    __shared__ unsigned long long w0[kWarps], w1[kWarps];
    const int lane = threadIdx.x & 31, wid = threadIdx.x >> 5;
    unsigned long long i0 = v0, i1 = v1;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        unsigned long long n0 = __shfl_up_sync(0xffffffffu, i0, o);
        unsigned long long n1 = __shfl_up_sync(0xffffffffu, i1, o);
        if (lane >= o) {
            i0 = sat_add(n0, i0);
            i1 = sat_add(n1, i1);
        }
    }
    unsigned long long e0 = __shfl_up_sync(0xffffffffu, i0, 1);
    unsigned long long e1 = __shfl_up_sync(0xffffffffu, i1, 1);
    if (lane == 0) e0 = e1 = 0;
    if (lane == 31) {
        w0[wid] = i0;
        w1[wid] = i1;
    }
    __syncthreads();
    if (wid == 0) {
        unsigned long long a0 = w0[lane], a1 = w1[lane];  // kWarps == 32
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            unsigned long long n0 = __shfl_up_sync(0xffffffffu, a0, o);
            unsigned long long n1 = __shfl_up_sync(0xffffffffu, a1, o);
            if (lane >= o) {
                a0 = sat_add(n0, a0);
                a1 = sat_add(n1, a1);
            }
        }
        w0[lane] = a0;
        w1[lane] = a1;
    }
    __syncthreads();
    unsigned long long p0 = wid ? w0[wid - 1] : 0, p1 = wid ? w1[wid - 1] : 0;
    ex0 = sat_add(p0, e0);
    ex1 = sat_add(p1, e1);
    tot0 = w0[kWarps - 1];
    tot1 = w1[kWarps - 1];
    __syncthreads();  // w0/w1 are reused by the next call
}

}  // namespace hp
