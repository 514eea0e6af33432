// Rows into and out of a quantised bank.
//
// Math (include/sdm.h): for every group of 32, 64 or 128 columns, scale = max|x| / L and
// code = round(x * (L / max|x|)); reading back gives scale * code.
//
// Design. A lane owns one 16-byte piece of a row's codes (16 columns, or 32 of 4 bits). The lanes
// of a scale group are neighbours, so the group's maximum is one to three shuffles, and a row that
// is ragged gets whole groups of lanes, the ones behind its end holding zeros. One pass: the
// columns stay in registers between the maximum and the rounding. The copy of a row is bound by
// memory; nothing is shared between rows, so there is neither shared memory nor a barrier.
#include <algorithm>
#include <climits>

#include "quant_device.cuh"
#include "sdm_internal.h"

namespace sdm {
namespace {

__device__ unsigned int g_quant_status;

constexpr int kThreads = 256;

// the slot of row r, or -1 (flagged) when it lies outside the bank
__device__ __forceinline__ int64_t row_slot(const QuantRowsArgs& a, int64_t r) {
    if (a.slots == nullptr) return r;
    const int64_t s = a.idx64 ? __ldg(static_cast<const int64_t*>(a.slots) + r) : __ldg(static_cast<const int32_t*>(a.slots) + r);
    if (s >= 0 && s < a.n_slots) return s;
    atomicOr(&g_quant_status, SDM_DEV_BAD_INDEX);
    return -1;
}

template <typename E, int C>
__device__ __forceinline__ void load_columns(const E* p, int n, bool vec, float* x) {
    if (vec && n >= C) {
        constexpr int PER = 16 / sizeof(E);
#pragma unroll
        for (int i = 0; i < C / PER; ++i) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(p) + i);
            if constexpr (sizeof(E) == 2)
                unpack<Bf16>(v, x + PER * i);
            else
                unpack<F32>(v, x + PER * i);
        }
    } else {
#pragma unroll
        for (int i = 0; i < C; ++i) x[i] = i < n ? to_f32(__ldg(p + i)) : 0.0f;
    }
}

template <typename E, int C>
__device__ __forceinline__ void store_columns(E* p, int n, bool vec, const float* x) {
    if (vec && n >= C) {
#pragma unroll
        for (int i = 0; i < C * (int)sizeof(E) / 16; ++i) {
            uint4 v;
            if constexpr (sizeof(E) == 2) {
                uint32_t w[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const __nv_bfloat162 b = __floats2bfloat162_rn(x[8 * i + 2 * j], x[8 * i + 2 * j + 1]);
                    w[j] = *reinterpret_cast<const uint32_t*>(&b);
                }
                v = make_uint4(w[0], w[1], w[2], w[3]);
            } else {
                v = make_uint4(__float_as_uint(x[4 * i]), __float_as_uint(x[4 * i + 1]), __float_as_uint(x[4 * i + 2]),
                               __float_as_uint(x[4 * i + 3]));
            }
            reinterpret_cast<uint4*>(p)[i] = v;
        }
    } else {
#pragma unroll
        for (int i = 0; i < C; ++i)
            if (i < n) p[i] = from_f32<E>(x[i]);
    }
}

template <typename F, typename E>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const QuantRowsArgs a) {
    constexpr int C = F::C;
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t r = a.small ? (int64_t)((uint32_t)id / (uint32_t)a.lanes) : id / a.lanes;
    const int p = (int)(id - r * a.lanes), n = a.hd - p * C;  // this lane's piece; columns from its first one on
    const bool live = r < a.n_rows;
    const int64_t slot = live ? row_slot(a, r) : -1;
    float x[C];
    load_columns<E, C>(static_cast<const E*>(a.rows) + (live ? r * a.row_stride + p * C : 0), live ? n : 0, a.vec, x);
    float scale;
    f32x2 x2[C / 2];
#pragma unroll
    for (int i = 0; i < C / 2; ++i) x2[i] = pair(x[2 * i], x[2 * i + 1]);
    const float top = piece_top<F>(x2);
    float inv;
    group_scales<F, 1>(&top, a.group / C, &scale, &inv);
    const uint4 codes = pack_piece<F>(x2, inv);
    if (slot < 0) return;
    if (p < a.pieces) reinterpret_cast<uint4*>(a.codes)[slot * a.pieces + p] = codes;
    if (p % (a.group / C) == 0) a.scales[slot * a.groups + p / (a.group / C)] = scale;
}

template <typename F, typename E>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const QuantRowsArgs a) {
    constexpr int C = F::C;
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
    const int64_t r = a.small ? (int64_t)((uint32_t)id / (uint32_t)a.lanes) : id / a.lanes;
    if (r >= a.n_rows) return;
    const int p = (int)(id - r * a.lanes), n = a.hd - p * C;
    const int64_t slot = row_slot(a, r);
    float x[C];
    if (slot >= 0) {
        unpack<F>(__ldg(reinterpret_cast<const uint4*>(a.codes) + slot * a.pieces + p), x);
        const float s = __ldg(a.scales + slot * a.groups + p * C / a.group);
#pragma unroll
        for (int i = 0; i < C; ++i) x[i] *= s;
    } else {
#pragma unroll
        for (int i = 0; i < C; ++i) x[i] = 0.0f;
    }
    store_columns<E, C>(static_cast<E*>(a.rows) + r * a.row_stride + p * C, n, a.vec, x);
}

template <typename F>
const void* kernel_of(int row_dtype, bool write) {
    if (write)
        return row_dtype == SDM_BF16 ? (const void*)quantize_kernel<F, uint16_t> : (const void*)quantize_kernel<F, float>;
    return row_dtype == SDM_BF16 ? (const void*)dequantize_kernel<F, uint16_t> : (const void*)dequantize_kernel<F, float>;
}

}  // namespace

int launch_quant_rows(const QuantRowsArgs& a0, int format, int row_dtype, bool write, cudaStream_t stream) {
    QuantRowsArgs a = a0;
    const int C = format == SDM_INT4 ? Int4::C : 16;
    a.pieces = (a.hd + C - 1) / C;
    a.groups = (a.hd + a.group - 1) / a.group;
    // the write gives every group all its lanes (their shuffles are aligned), the read only the pieces
    a.lanes = write ? a.groups * (a.group / C) : a.pieces;
    const int es = row_dtype == SDM_BF16 ? 2 : 4;
    a.vec = reinterpret_cast<uintptr_t>(a.rows) % 16 == 0 && a.row_stride * es % 16 == 0;
    const int64_t blocks = (a.n_rows * a.lanes + kThreads - 1) / kThreads;
    if (blocks > INT_MAX) return SDM_ECOUNT;
    a.small = blocks * kThreads <= INT_MAX;
    const void* fn = format == SDM_INT8  ? kernel_of<Int8>(row_dtype, write)
                     : format == SDM_FP8 ? kernel_of<Fp8>(row_dtype, write)
                                         : kernel_of<Int4>(row_dtype, write);
    void* args[] = {&a};
    return launch_pdl_raw(fn, dim3((unsigned)blocks), dim3(kThreads), 0, stream, args);
}

int quant_status(unsigned int* word, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(word, g_quant_status, sizeof(unsigned int));
    if (e == cudaSuccess && clear) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_quant_status, &zero, sizeof(unsigned int));
    }
    return (int)e;
}

}  // namespace sdm
