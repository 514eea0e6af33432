// Write-then-read tokens on a quantised bank.
//
// Math (include/sdm.h), per stream and token, row = scale * code, d_w = exp(g_w):
//     retrieved = sum_w k_w d_w row_w,  delta = beta (v - retrieved)
//     row_w <- quantised(d_w row_w + k_w delta),  out = sum_r q_r row_r  (after the write)
//
// Design. Everything but a group's scale is independent by columns, so one block owns a (stream,
// slice of 8 pieces = 128 columns, a whole number of scale groups) for all T tokens, and a block
// barrier orders a token's writes before its reads: no other block touches those bytes. LR lanes
// hold a row's slice, 16 bytes each, so a thread keeps its few rows' codes in registers from the
// retrieval to the write-back: each row is read once and written once, and the group's maximum is
// a shuffle among neighbouring lanes. The sums over rows go through shuffles within a warp and
// shared memory across warps, in a fixed order.
#include <algorithm>
#include <climits>

#include "quant_device.cuh"
#include "sdm_internal.h"

namespace sdm {
namespace {

__device__ unsigned int g_qdecode_status;

constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ int64_t bank_slot(const QDecodeArgs& a, const void* idx, int64_t i) {
    const int64_t s = a.idx64 ? __ldg(static_cast<const int64_t*>(idx) + i) : __ldg(static_cast<const int32_t*>(idx) + i);
    if (s >= 0 && s < a.n_slots) return s;
    atomicOr(&g_qdecode_status, SDM_DEV_BAD_INDEX);
    return -1;
}

// Sum x[0..16) over the row slots of a warp (lanes LR apart); x[0 .. 16 * LR / 32) then holds the
// columns from the returned one on.
template <int LR>
__device__ __forceinline__ int reduce_rows(float* x, int lane) {
    int first = 0, half = 8;
#pragma unroll
    for (int o = 16; o >= LR; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i < half) {
                const float keep = up ? x[i + half] : x[i], give = up ? x[i] : x[i + half];
                x[i] = keep + __shfl_xor_sync(kAll, give, o);
            }
        }
        first += up ? half : 0;
        half /= 2;
    }
    return first;
}

// F: Int8 or Fp8. LR: lanes of a row slice (its columns: 16 * LR). NT: threads. RPT: rows a thread holds.
template <typename F, int LR, int NT, int RPT>
__global__ void __launch_bounds__(NT) qdecode_kernel(const QDecodeArgs a) {
    static_assert(F::C == 16, "pieces of 16 columns");
    constexpr int COLS = 16 * LR, RS = NT / LR, WARPS = NT / 32, KEEP = 16 * LR / 32;
    __shared__ __align__(16) float part_k[WARPS][COLS];
    __shared__ __align__(16) float part_q[WARPS][COLS];
    __shared__ __align__(16) float delta[COLS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rs = tid / LR, lp = tid % LR;
    const int64_t s = blockIdx.x / a.slices;
    const int slice = (int)(blockIdx.x % a.slices);
    const int p = slice * LR + lp, c0 = slice * COLS, hd = a.hd;
    const bool active = p < a.pieces;
    const int gl = min(a.group / 16, LR);  // lanes of a scale group
    const int64_t group = p * 16 / a.group;
    uint4* codes = reinterpret_cast<uint4*>(a.codes) + p;
    float* scales = a.scales + group;
    grid_dependency_wait();
    grid_launch_dependents();

    for (int t = 0; t < a.T; ++t) {
        const int64_t ts = t * a.tstride + s * a.sstride;
        // the write rows, and their decayed sum
        int64_t slot[RPT];
        uint4 code[RPT];
        float ds[RPT], kv[RPT], x[16], acc[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < RPT; ++j) {
            const int w = rs + j * RS;
            slot[j] = -1;
            kv[j] = ds[j] = 0.0f;
            code[j] = make_uint4(0u, 0u, 0u, 0u);
            if (w < a.W) {
                slot[j] = bank_slot(a, a.k_idx, ts * a.W + w);
                kv[j] = __ldg(a.k_val + ts * a.W + w);
                if (slot[j] >= 0 && active) {
                    code[j] = __ldcg(codes + slot[j] * a.pieces);
                    ds[j] = __ldcg(scales + slot[j] * a.groups) * expf(__ldg(a.g + ts * a.G + (a.G == 1 ? 0 : w)));
                }
            }
        }
#pragma unroll
        for (int j = 0; j < RPT; ++j) {
            F::unpack(code[j], x);
            const float f = kv[j] * ds[j];
#pragma unroll
            for (int i = 0; i < 16; ++i) acc[i] = fmaf(f, x[i], acc[i]);
        }
        int first = reduce_rows<LR>(acc, lane);
#pragma unroll
        for (int i = 0; i < KEEP; ++i) part_k[warp][lp * 16 + first + i] = acc[i];
        __syncthreads();
        for (int c = tid; c < COLS; c += NT) {
            float r = part_k[0][c];
#pragma unroll
            for (int q = 1; q < WARPS; ++q) r += part_k[q][c];
            const bool in = c0 + c < hd;
            delta[c] = in ? __ldg(a.beta + ts) * (__ldg(a.v + ts * hd + c0 + c) - r) : 0.0f;
        }
        __syncthreads();
        // the new rows
        float dl[16];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 f = *reinterpret_cast<const float4*>(&delta[lp * 16 + 4 * i]);
            dl[4 * i] = f.x, dl[4 * i + 1] = f.y, dl[4 * i + 2] = f.z, dl[4 * i + 3] = f.w;
        }
#pragma unroll
        for (int j = 0; j < RPT; ++j) {
            F::unpack(code[j], x);
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = fmaf(kv[j], dl[i], ds[j] * x[i]);
            float sc;
            const uint4 n = quantise_piece<F>(x, gl, &sc);
            if (slot[j] >= 0 && active) {
                codes[slot[j] * a.pieces] = n;
                if (lp % gl == 0) scales[slot[j] * a.groups] = sc;
            }
        }
        __syncthreads();  // the rows are written: the reads below, and the next token, may touch them
        // the readings
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[i] = 0.0f;
        for (int r0 = rs; r0 < a.R; r0 += RPT * RS) {
            uint4 v[RPT];
            float qs[RPT];
#pragma unroll
            for (int j = 0; j < RPT; ++j) {
                const int r = r0 + j * RS;
                v[j] = make_uint4(0u, 0u, 0u, 0u);
                qs[j] = 0.0f;
                if (r < a.R) {
                    const int64_t sl = bank_slot(a, a.q_idx, ts * a.R + r);
                    if (sl >= 0 && active) {
                        v[j] = __ldcg(codes + sl * a.pieces);
                        qs[j] = __ldg(a.q_val + ts * a.R + r) * __ldcg(scales + sl * a.groups);
                    }
                }
            }
#pragma unroll
            for (int j = 0; j < RPT; ++j) {
                F::unpack(v[j], x);
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[i] = fmaf(qs[j], x[i], acc[i]);
            }
        }
        first = reduce_rows<LR>(acc, lane);
#pragma unroll
        for (int i = 0; i < KEEP; ++i) part_q[warp][lp * 16 + first + i] = acc[i];
        __syncthreads();
        for (int c = tid; c < COLS; c += NT) {
            if (c0 + c >= hd) break;
            float r = part_q[0][c];
#pragma unroll
            for (int q = 1; q < WARPS; ++q) r += part_q[q][c];
            if (a.out_bf16)
                static_cast<uint16_t*>(a.out)[ts * hd + c0 + c] = from_f32<uint16_t>(r);
            else
                static_cast<float*>(a.out)[ts * hd + c0 + c] = r;
        }
        // part_k, delta and part_q of the next token are written behind barriers that follow their
        // last reads here
    }
}

struct Chosen {
    const void* fn;
    int threads;
};

template <typename F, int LR>
Chosen choose(int W) {
    constexpr int S = 128 / LR;  // row slots of 128 threads
    if (W <= 2 * S) return {(const void*)qdecode_kernel<F, LR, 128, 2>, 128};
    if (W <= 4 * S) return {(const void*)qdecode_kernel<F, LR, 128, 4>, 128};
    if (W <= 8 * S) return {(const void*)qdecode_kernel<F, LR, 128, 8>, 128};
    return {(const void*)qdecode_kernel<F, LR, 256, 8>, 256};
}

}  // namespace

int launch_qdecode(const QDecodeArgs& a0, int format, cudaStream_t stream) {
    QDecodeArgs a = a0;
    a.pieces = (a.hd + 15) / 16;
    a.groups = (a.hd + a.group - 1) / a.group;
    const bool narrow = a.pieces <= 4;
    a.slices = narrow ? 1 : (a.pieces + 7) / 8;
    const int64_t blocks = a.n_streams * a.slices;
    if (blocks > INT_MAX) return SDM_ECOUNT;
    const Chosen c = format == SDM_INT8 ? (narrow ? choose<Int8, 4>(a.W) : choose<Int8, 8>(a.W))
                                        : (narrow ? choose<Fp8, 4>(a.W) : choose<Fp8, 8>(a.W));
    void* args[] = {&a};
    return launch_pdl_raw(c.fn, dim3((unsigned)blocks), dim3((unsigned)c.threads), 0, stream, args);
}

int qdecode_status(unsigned int* word, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(word, g_qdecode_status, sizeof(unsigned int));
    if (e == cudaSuccess && clear) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_qdecode_status, &zero, sizeof(unsigned int));
    }
    return (int)e;
}

}  // namespace sdm
