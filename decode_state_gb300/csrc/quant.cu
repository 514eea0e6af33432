// Rows into and out of a quantised bank.
//
// Math (include/sdm.h): for every group of 32, 64 or 128 columns, scale = max|x| / L and
// code = round(x * (L / max|x|)); reading back gives scale * code.
//
// Design. A lane owns 16 columns of a row: 16 bytes of codes, or 8 of 4 bits. The lanes of a scale
// group are neighbours, so the group's maximum is one to three shuffles, and a row that is ragged gets
// whole groups of lanes, the ones behind its end holding zeros. One pass: the columns stay in registers
// between the maximum and the rounding. The copy of a row is bound by memory: 2^20 rows of 128 float32
// into int8 slots in order run at 7.1 TB/s, at random slots at 5.9 (128-byte rows and their scales are
// scattered). 32 columns a lane for 4 bits (whole 16-byte pieces) ran at 5.3.
//
// Contiguous rows whose columns do not start on 16-byte boundaries go through shared memory, a run of
// whole rows for each block, so that global memory still sees 16-byte accesses: 2^20 rows of 100 bf16
// were read back at 0.6 TB/s by columns.
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

constexpr int kCols = 16;           // columns of a lane
constexpr int kRunBytes = 16 * 1024;  // rows that a block takes through shared memory

// A lane's codes in a bank row: 16 bytes, or 8 of 4 bits.
template <typename F>
struct Share {
    using Codes = uint4;
    static __device__ __forceinline__ void unpack2(const Codes& v, f32x2* x) { F::unpack2(v, x); }
    static __device__ __forceinline__ Codes pack2(const f32x2* y) { return F::pack2(y); }
};
template <>
struct Share<Int4> {
    using Codes = uint2;
    static __device__ __forceinline__ void unpack2(const Codes& v, f32x2* x) {
        Int4::unpack_word(v.x, x);
        Int4::unpack_word(v.y, x + 4);
    }
    static __device__ __forceinline__ Codes pack2(const f32x2* y) { return make_uint2(Int4::pack_word(y), Int4::pack_word(y + 4)); }
};

// n columns from p on (a lane's 16 at most), zeros behind them
template <typename E>
__device__ __forceinline__ void load_columns(const E* p, int n, bool vec, float* x) {
    if (vec && n >= kCols) {
        constexpr int PER = 16 / sizeof(E);
#pragma unroll
        for (int i = 0; i < kCols / PER; ++i) {
            const uint4 v = *(reinterpret_cast<const uint4*>(p) + i);
            if constexpr (sizeof(E) == 2)
                unpack<Bf16>(v, x + PER * i);
            else
                unpack<F32>(v, x + PER * i);
        }
    } else {
#pragma unroll
        for (int i = 0; i < kCols; ++i) x[i] = i < n ? to_f32(p[i]) : 0.0f;
    }
}

template <typename E>
__device__ __forceinline__ void store_columns(E* p, int n, bool vec, const float* x) {
    if (vec && n >= kCols) {
#pragma unroll
        for (int i = 0; i < kCols * (int)sizeof(E) / 16; ++i) {
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
        for (int i = 0; i < kCols; ++i)
            if (i < n) p[i] = from_f32<E>(x[i]);
    }
}

// The rows of a block's run as they lie in memory, bytes [begin, end) of the row array; in shared memory
// they keep their position within 16 bytes.
template <typename E>
struct Run {
    unsigned char *global, *shared;  // of the run's first byte
    int bytes, head;                 // head: bytes before the first boundary

    __device__ __forceinline__ Run(const QuantRowsArgs& a, unsigned char* smem, int64_t row0, int rows) {
        global = reinterpret_cast<unsigned char*>(a.rows) + row0 * a.hd * (int64_t)sizeof(E);
        const int off = (int)(reinterpret_cast<uintptr_t>(global) & 15u);
        shared = smem + off;
        bytes = rows * a.hd * (int)sizeof(E);
        head = min(bytes, (16 - off) & 15);
    }
    // f16(i): copy the 16 bytes from i on; f1(i): the element from i on
    template <typename F16, typename F1>
    __device__ __forceinline__ void each(const F16& f16, const F1& f1) const {
        const int whole = head + (bytes - head) / 16 * 16;
        for (int i = head + (int)threadIdx.x * 16; i < whole; i += kThreads * 16) f16(i);
        const int rest = (head + bytes - whole) / (int)sizeof(E);
        if ((int)threadIdx.x < rest) {
            const int i = threadIdx.x * (int)sizeof(E);
            f1(i < head ? i : whole + i - head);
        }
    }
};

template <typename F, typename E, bool RUN>
__global__ void __launch_bounds__(kThreads) quantize_kernel(const QuantRowsArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    using Codes = typename Share<F>::Codes;
    const int gl = a.group / kCols;
    grid_dependency_wait();
    grid_launch_dependents();
    const auto one = [&](int64_t r, int p, bool there, const E* from, bool vec) {
        const int64_t slot = there ? row_slot(a, r) : -1;
        float x[kCols];
        load_columns<E>(from + p * kCols, there ? a.hd - p * kCols : 0, vec, x);
        f32x2 x2[kCols / 2];
#pragma unroll
        for (int i = 0; i < kCols / 2; ++i) x2[i] = pair(x[2 * i], x[2 * i + 1]);
        const float top = piece_top<kCols>(x2);
        float scale, inv;
        group_scales<F, 1>(&top, gl, &scale, &inv);
        const f32x2 f = pair(inv, inv);
#pragma unroll
        for (int i = 0; i < kCols / 2; ++i) x2[i] = mul2(x2[i], f);
        Codes codes = Share<F>::pack2(x2);
        if (!(inv > 0.0f)) codes = Codes{};
        if (slot < 0) return;
        if (p < a.pieces) reinterpret_cast<Codes*>(a.codes)[slot * a.pieces + p] = codes;
        if (p % gl == 0) a.scales[slot * a.groups + p / gl] = scale;
    };
    if constexpr (RUN) {
        const int64_t row0 = (int64_t)blockIdx.x * a.run_rows;
        const int rows = (int)min((int64_t)a.run_rows, a.n_rows - row0);
        const Run<E> run(a, smem, row0, rows);
        run.each([&](int i) { *reinterpret_cast<uint4*>(run.shared + i) = __ldg(reinterpret_cast<const uint4*>(run.global + i)); },
                 [&](int i) { *reinterpret_cast<E*>(run.shared + i) = __ldg(reinterpret_cast<const E*>(run.global + i)); });
        __syncthreads();
        for (int i0 = 0; i0 < rows * a.lanes; i0 += kThreads) {  // all threads, for the shuffles
            const int i = i0 + threadIdx.x, r = i / a.lanes;
            one(row0 + r, i - r * a.lanes, r < rows, reinterpret_cast<const E*>(run.shared) + min(r, rows - 1) * a.hd, false);
        }
    } else {
        const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
        const int64_t r = a.small ? (int64_t)((uint32_t)id / (uint32_t)a.lanes) : id / a.lanes;
        const bool there = r < a.n_rows;
        one(r, (int)(id - r * a.lanes), there, static_cast<const E*>(a.rows) + (there ? r : 0) * a.row_stride, a.vec);
    }
}

template <typename F, typename E, bool RUN>
__global__ void __launch_bounds__(kThreads) dequantize_kernel(const QuantRowsArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    using Codes = typename Share<F>::Codes;
    grid_dependency_wait();
    grid_launch_dependents();
    const auto one = [&](int64_t r, int p, E* to, bool vec) {
        const int64_t slot = row_slot(a, r);
        float x[kCols];
#pragma unroll
        for (int i = 0; i < kCols; ++i) x[i] = 0.0f;
        if (slot >= 0) {
            const Codes codes = __ldg(reinterpret_cast<const Codes*>(a.codes) + slot * a.pieces + p);
            const float s = __ldg(a.scales + slot * a.groups + p * kCols / a.group);
            f32x2 x2[kCols / 2];
            Share<F>::unpack2(codes, x2);
#pragma unroll
            for (int i = 0; i < kCols / 2; ++i) split(mul2(x2[i], pair(s, s)), x[2 * i], x[2 * i + 1]);
        }
        store_columns<E>(to + p * kCols, a.hd - p * kCols, vec, x);
    };
    if constexpr (RUN) {
        const int64_t row0 = (int64_t)blockIdx.x * a.run_rows;
        const int rows = (int)min((int64_t)a.run_rows, a.n_rows - row0);
        const Run<E> run(a, smem, row0, rows);
        for (int i = threadIdx.x; i < rows * a.lanes; i += kThreads) {
            const int r = i / a.lanes;
            one(row0 + r, i - r * a.lanes, reinterpret_cast<E*>(run.shared) + r * a.hd, false);
        }
        __syncthreads();
        run.each([&](int i) { *reinterpret_cast<uint4*>(run.global + i) = *reinterpret_cast<const uint4*>(run.shared + i); },
                 [&](int i) { *reinterpret_cast<E*>(run.global + i) = *reinterpret_cast<const E*>(run.shared + i); });
    } else {
        const int64_t id = (int64_t)blockIdx.x * kThreads + threadIdx.x;
        const int64_t r = a.small ? (int64_t)((uint32_t)id / (uint32_t)a.lanes) : id / a.lanes;
        if (r < a.n_rows) one(r, (int)(id - r * a.lanes), static_cast<E*>(a.rows) + r * a.row_stride, a.vec);
    }
}

template <typename F, typename E>
const void* kernel_of(bool write, bool run) {
    if (write) return run ? (const void*)quantize_kernel<F, E, true> : (const void*)quantize_kernel<F, E, false>;
    return run ? (const void*)dequantize_kernel<F, E, true> : (const void*)dequantize_kernel<F, E, false>;
}

template <typename F>
const void* kernel_of(int row_dtype, bool write, bool run) {
    return row_dtype == SDM_BF16 ? kernel_of<F, uint16_t>(write, run) : kernel_of<F, float>(write, run);
}

}  // namespace

int launch_quant_rows(const QuantRowsArgs& a0, int format, int row_dtype, bool write, cudaStream_t stream) {
    QuantRowsArgs a = a0;
    a.pieces = format == SDM_INT4 ? ((a.hd + 1) / 2 + 15) / 16 * 2 : (a.hd + 15) / 16;  // shares of a row of codes, its padding with them
    a.groups = (a.hd + a.group - 1) / a.group;
    // the write gives every group all its lanes (their shuffles are aligned), the read those with columns
    a.lanes = write ? a.groups * (a.group / kCols) : (a.hd + kCols - 1) / kCols;
    const int es = row_dtype == SDM_BF16 ? 2 : 4;
    a.vec = reinterpret_cast<uintptr_t>(a.rows) % 16 == 0 && a.row_stride * es % 16 == 0;
    a.run_rows = kRunBytes / (a.hd * es);
    const bool run = !a.vec && a.row_stride == a.hd && a.run_rows > 0;
    const int64_t blocks = run ? (a.n_rows + a.run_rows - 1) / a.run_rows : (a.n_rows * a.lanes + kThreads - 1) / kThreads;
    if (blocks > INT_MAX) return SDM_ECOUNT;
    a.small = blocks * kThreads <= INT_MAX;
    const void* fn = format == SDM_INT8  ? kernel_of<Int8>(row_dtype, write, run)
                     : format == SDM_FP8 ? kernel_of<Fp8>(row_dtype, write, run)
                                         : kernel_of<Int4>(row_dtype, write, run);
    void* args[] = {&a};
    return launch_pdl_raw(fn, dim3((unsigned)blocks), dim3(kThreads), run ? kRunBytes + 16 : 0, stream, args);
}

cudaError_t quant_status(void** word) { return cudaGetSymbolAddress(word, g_quant_status); }

}  // namespace sdm
