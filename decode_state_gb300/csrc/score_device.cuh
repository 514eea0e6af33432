// Device helpers of the routing and its balance loss: masked logits, exponentials below a maximum, sums over lanes.
#pragma once

#include <stdint.h>

#include "sdm.h"
#include "sdm_device.cuh"

namespace sdm {

constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ float minus_inf() { return __uint_as_float(0xff800000u); }
__device__ __forceinline__ bool masked(float x) { return !(x > minus_inf()); }  // NaN too

// exp(x - m) with m the largest of the logits; several +inf are the largest together
__device__ __forceinline__ float exp_below(float x, float m) {
    return masked(x) ? 0.0f : x == m ? 1.0f : expf(x - m);
}

// Over the LANES lanes of a warp that lie together (a power of two), the same bits in each of them.
template <int LANES = 32>
__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) x += __shfl_xor_sync(kAll, x, o);
    return x;
}
template <int LANES = 32>
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(kAll, x, o));
    return x;
}

}  // namespace sdm
