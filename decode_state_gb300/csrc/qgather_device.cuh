// Shared by the kernels that gather rows for many tokens (qgather_ring.cu) and for few (qgather.cu).
#pragma once

#include "quant_device.cuh"
#include "sdm_internal.h"

namespace sdm {

__device__ __forceinline__ bool padding(const QGatherArgs& a, int64_t t) {
    if (a.chunk == 1 && a.chunk_valid == nullptr) return a.valid == 0;
    const int vt = a.chunk_valid != nullptr ? __ldg(a.chunk_valid + t / a.chunk) : a.valid;
    return (int)(t % a.chunk) >= vt;
}

__device__ __forceinline__ void store_dw(const QGatherArgs& a, int op, int64_t i, float x) {
    if (a.w_bf16)
        static_cast<uint16_t*>(a.dw[op])[i] = from_f32<uint16_t>(x);
    else
        static_cast<float*>(a.dw[op])[i] = x;
}

template <typename F>
__device__ __forceinline__ float dot_piece(const float* d, const uint4& v) {
    f32x2 x[F::C / 2], sum = 0;
    F::unpack2(v, x);
#pragma unroll
    for (int i = 0; i < F::C / 2; ++i) sum = fma2(pair(d[2 * i], d[2 * i + 1]), x[i], sum);
    float lo, hi;
    split(sum, lo, hi);
    return lo + hi;
}

}  // namespace sdm
