// Gather over a quantised bank, and the gradient of a gather's weights.
//
// Math (include/sdm.h): out[t] = sum_n w[t, n] * row(idx[t, n]) and
// dw[t, n] = <dout[t], row(idx[t, n])>, row = scale * code (or the row of a bf16 / float32 bank).
//
// Design. A warp owns a token's entries over a slice of at most 32 pieces (16 bytes each) of the
// row. LR lanes hold one row, so 32 / LR rows are read at once, and the rows of 32 entries are
// requested ahead of their use: the lanes first load 32 indices and weights (coalesced), then hand
// them round by shuffles. Rows go from memory to registers; there is no shared memory and no
// barrier unless warps share a token. The bound is the row reads: 128-byte rows at random places.
//
// Few tokens would leave most of the machine idle while each warp waits for one batch of rows after
// another, so below kSplitUnits warps' worth of work four warps share a token and join their sums
// through shared memory. The rule looks at the sizes only, so that results do not depend on the GPU.
#include <algorithm>
#include <climits>

#include "quant_device.cuh"
#include "sdm_internal.h"

namespace sdm {
namespace {

__device__ unsigned int g_qgather_status;

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int64_t kSplitUnits = 4096;
constexpr unsigned kAll = 0xffffffffu;

// A unit of work: one operand of one token over one column slice.
struct Unit {
    int64_t t;
    int op, slice, part;  // part: this warp's share of the entries
    bool live;            // there is such a unit (blocks of unshared warps may have spare ones)
};

__device__ __forceinline__ Unit unit_of(const QGatherArgs& a) {
    const int warp = threadIdx.x >> 5;
    const int64_t u = a.split > 1 ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * kWarps + warp;
    Unit r;
    r.part = a.split > 1 ? warp : 0;
    r.slice = a.slices > 1 ? (int)(u % a.slices) : 0;
    const int64_t v = a.slices > 1 ? u / a.slices : u;
    r.op = a.n_ops == 2 ? (int)(v & 1) : 0;
    r.t = a.n_ops == 2 ? v >> 1 : v;
    r.live = r.t < a.tokens;
    return r;
}

__device__ __forceinline__ bool padding(const QGatherArgs& a, int64_t t) {
    if (a.chunk == 1 && a.chunk_valid == nullptr) return a.valid == 0;
    const int vt = a.chunk_valid != nullptr ? __ldg(a.chunk_valid + t / a.chunk) : a.valid;
    return (int)(t % a.chunk) >= vt;
}

// the slot of entry i, or -1 (flagged) when it lies outside the bank
__device__ __forceinline__ int entry_slot(const QGatherArgs& a, const void* idx, int64_t i) {
    const int64_t s = a.idx64 ? __ldg(static_cast<const int64_t*>(idx) + i) : __ldg(static_cast<const int32_t*>(idx) + i);
    if (s >= 0 && s < a.n_slots) return (int)s;
    atomicOr(&g_qgather_status, SDM_DEV_BAD_INDEX);
    return -1;
}

// 16 bytes of a row; `n` columns from the piece's first one on. Unaligned rows are read by columns.
template <typename F, bool ALIGNED>
__device__ __forceinline__ uint4 load_piece(const unsigned char* p, int n, bool on) {
    if constexpr (ALIGNED) {
        return load16_if(p, on);
    } else {
        uint32_t w[4] = {0u, 0u, 0u, 0u};
        if (!on) n = 0;
        using E = typename F::E;
        const E* e = reinterpret_cast<const E*>(p);
#pragma unroll
        for (int i = 0; i < F::C; ++i) {
            if (i >= n) break;
            if constexpr (sizeof(E) == 2)
                w[i / 2] |= (uint32_t)__ldg(e + i) << (16 * (i & 1));
            else
                w[i] = __float_as_uint(__ldg(e + i));
        }
        return make_uint4(w[0], w[1], w[2], w[3]);
    }
}

// Sum x[0..N) over the 32 / LR row slots of a warp, leaving each slot with a share of the columns:
// half of them are handed over at every step, so N - N / slots shuffles do it instead of N * log2.
// x[0 .. N / slots) then holds the columns from the returned one on.
template <int N, int LR>
__device__ __forceinline__ int reduce_scatter(float* x, int lane) {
    int first = 0;
    int half = N / 2;
#pragma unroll
    for (int o = 16; o >= LR; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
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

template <typename F, int LR>
__global__ void __launch_bounds__(kThreads) qgather_kernel(const QGatherArgs a) {
    constexpr int C = F::C, SLOTS = 32 / LR, KEEP = C / SLOTS;
    static_assert(KEEP >= 1, "every row slot keeps columns");
    extern __shared__ __align__(16) float joined[];
    grid_dependency_wait();
    grid_launch_dependents();
    const Unit u = unit_of(a);
    if (!u.live) return;  // unshared units only: a shared one fills its block
    const int lane = threadIdx.x & 31, rs = lane / LR, p = u.slice * LR + lane % LR;
    const int hd = a.hd, NR = a.width[u.op];
    f32x2 acc2[C / 2];
#pragma unroll
    for (int i = 0; i < C / 2; ++i) acc2[i] = 0;

    if (!padding(a, u.t)) {
        const bool active = p < a.pieces;
        const unsigned char* bank = static_cast<const unsigned char*>(a.bank) + (int64_t)p * 16;
        const float* scales = a.scales + (p * C) / a.group;
        const int64_t e0 = u.t * NR;
        for (int base = u.part * 32; base < NR; base += 32 * a.split) {
            int slot = -1;
            float w = 0.0f;
            if (base + lane < NR) {
                slot = entry_slot(a, a.idx[u.op], e0 + base + lane);
                w = a.w_bf16 ? to_f32(__ldg(static_cast<const uint16_t*>(a.w[u.op]) + e0 + base + lane))
                             : __ldg(static_cast<const float*>(a.w[u.op]) + e0 + base + lane);
            }
            constexpr int BATCH = LR < 8 ? LR : 8;  // rows requested at once by a lane
#pragma unroll
            for (int s0 = 0; s0 < LR; s0 += BATCH) {
                if (base + s0 * SLOTS >= NR) break;
                uint4 v[BATCH];
                float ws[BATCH], sc[BATCH];
#pragma unroll
                for (int s = 0; s < BATCH; ++s) {
                    const int src = (s0 + s) * SLOTS + rs;
                    const int sl = __shfl_sync(kAll, slot, src);
                    ws[s] = __shfl_sync(kAll, w, src);
                    const bool on = sl >= 0 && active;
                    v[s] = load16_if(bank + sl * a.row_bytes, on);
                    sc[s] = load4_if(scales + (int64_t)sl * a.groups, on);
                }
#pragma unroll
                for (int s = 0; s < BATCH; ++s) {
                    f32x2 x[C / 2];
                    F::unpack2(v[s], x);
                    const float fs = ws[s] * sc[s];
                    const f32x2 f = pair(fs, fs);
#pragma unroll
                    for (int i = 0; i < C / 2; ++i) acc2[i] = fma2(f, x[i], acc2[i]);
                }
            }
        }
    }

    float acc[C];
#pragma unroll
    for (int i = 0; i < C / 2; ++i) split(acc2[i], acc[2 * i], acc[2 * i + 1]);
    const int first = reduce_scatter<C, LR>(acc, lane);
    if (a.split > 1) {  // the other warps' sums of the same columns
        float* mine = joined + (threadIdx.x) * KEEP;
#pragma unroll
        for (int i = 0; i < KEEP; ++i) mine[i] = acc[i];
        __syncthreads();
        if (u.part != 0) return;
#pragma unroll
        for (int i = 0; i < KEEP; ++i) {
            acc[i] = joined[lane * KEEP + i];
            for (int q = 1; q < kWarps; ++q) acc[i] += joined[(q * 32 + lane) * KEEP + i];
        }
    }
    const int c0 = p * C + first;
    float* out = a.out[u.op] + u.t * hd + c0;
    if (KEEP % 4 == 0 && a.vec_out && c0 + KEEP <= hd) {
#pragma unroll
        for (int i = 0; i < KEEP / 4; ++i)
            reinterpret_cast<float4*>(out)[i] = make_float4(acc[4 * i], acc[4 * i + 1], acc[4 * i + 2], acc[4 * i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < KEEP; ++i)
            if (c0 + i < hd) out[i] = acc[i];
    }
}

template <typename F, int LR, bool ALIGNED>
__global__ void __launch_bounds__(kThreads) gather_dw_kernel(const QGatherArgs a) {
    constexpr int C = F::C;
    grid_dependency_wait();
    grid_launch_dependents();
    const Unit u = unit_of(a);  // a.slices is 1 here: the warp walks the slices of a row itself
    if (!u.live) return;
    const int lane = threadIdx.x & 31, rs = lane / LR;
    const int hd = a.hd, NR = a.width[u.op];
    const int64_t e0 = u.t * NR;
    const bool pad = padding(a, u.t);
    const int slices = (a.pieces + LR - 1) / LR;
    const float* dout = a.dout[u.op] + u.t * hd;

    float d[C];
    const auto load_dout = [&](int p) {
        if (a.vec_out && p * C + C <= hd) {
#pragma unroll
            for (int i = 0; i < C / 4; ++i) {
                const float4 f = __ldg(reinterpret_cast<const float4*>(dout + p * C) + i);
                d[4 * i] = f.x, d[4 * i + 1] = f.y, d[4 * i + 2] = f.z, d[4 * i + 3] = f.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < C; ++i) d[i] = p * C + i < hd ? __ldg(dout + p * C + i) : 0.0f;
        }
    };
    if (!pad && slices == 1) load_dout(lane % LR);

    for (int base = u.part * 32; base < NR; base += 32 * a.split) {
        float dot[LR];  // the lanes of row slot rs hold partial dots of entries base + rs * LR + 0 .. LR - 1
#pragma unroll
        for (int s = 0; s < LR; ++s) dot[s] = 0.0f;
        if (!pad) {
            const int slot = base + lane < NR ? entry_slot(a, a.idx[u.op], e0 + base + lane) : -1;
            for (int slice = 0; slice < slices; ++slice) {
                const int p = slice * LR + lane % LR;
                if (slices > 1) load_dout(p);
                constexpr int BATCH = LR < 8 ? LR : 8;
#pragma unroll
                for (int s0 = 0; s0 < LR; s0 += BATCH) {
                    uint4 v[BATCH];
                    float sc[BATCH];
#pragma unroll
                    for (int s = 0; s < BATCH; ++s) {
                        const int sl = __shfl_sync(kAll, slot, rs * LR + s0 + s);
                        const bool on = sl >= 0 && p < a.pieces;
                        v[s] = load_piece<F, ALIGNED>(static_cast<const unsigned char*>(a.bank) + sl * a.row_bytes + (int64_t)p * 16,
                                                      hd - p * C, on);
                        if constexpr (F::kQuantised) sc[s] = load4_if(a.scales + (int64_t)sl * a.groups + p * C / a.group, on);
                    }
#pragma unroll
                    for (int s = 0; s < BATCH; ++s) {
                        f32x2 x[C / 2], sum2 = 0;
                        F::unpack2(v[s], x);
#pragma unroll
                        for (int i = 0; i < C / 2; ++i) sum2 = fma2(pair(d[2 * i], d[2 * i + 1]), x[i], sum2);
                        float sum, odd;
                        split(sum2, sum, odd);
                        sum += odd;
                        if constexpr (F::kQuantised)
                            dot[s0 + s] = fmaf(sum, sc[s], dot[s0 + s]);
                        else
                            dot[s0 + s] += sum;
                    }
                }
            }
            // the sums over the lanes of a row, lane j of them keeping entry j's
#pragma unroll
            for (int h = LR / 2; h >= 1; h /= 2) {
                const bool up = lane & h;
#pragma unroll
                for (int i = 0; i < LR / 2; ++i) {
                    if (i < h) {
                        const float keep = up ? dot[i + h] : dot[i], give = up ? dot[i] : dot[i + h];
                        dot[i] = keep + __shfl_xor_sync(kAll, give, h);
                    }
                }
            }
        }
        if (base + lane < NR) {
            if (a.w_bf16)
                static_cast<uint16_t*>(a.dw[u.op])[e0 + base + lane] = from_f32<uint16_t>(dot[0]);
            else
                static_cast<float*>(a.dw[u.op])[e0 + base + lane] = dot[0];
        }
    }
}

template <typename F>
const void* qgather_of(int lr) {
    switch (lr) {
        case 4: return (const void*)qgather_kernel<F, 4>;
        case 8: return (const void*)qgather_kernel<F, 8>;
        case 16: return (const void*)qgather_kernel<F, 16>;
        default: return (const void*)qgather_kernel<F, 32>;
    }
}

template <typename F, bool ALIGNED = true>
const void* dw_of(int lr) {
    switch (lr) {
        case 4: return (const void*)gather_dw_kernel<F, 4, ALIGNED>;
        case 8: return (const void*)gather_dw_kernel<F, 8, ALIGNED>;
        case 16: return (const void*)gather_dw_kernel<F, 16, ALIGNED>;
        default: return (const void*)gather_dw_kernel<F, 32, ALIGNED>;
    }
}

int columns(int format) { return format == SDM_INT4 ? 32 : format == SDM_BF16 ? 8 : format == SDM_F32 ? 4 : 16; }

// lanes that hold one row of `pieces` pieces, or of one slice of a longer row
int row_lanes(int pieces) { return pieces <= 4 ? 4 : pieces <= 8 ? 8 : pieces <= 16 ? 16 : 32; }

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

int run(const void* fn, QGatherArgs& a, size_t smem, cudaStream_t stream) {
    const int64_t units = a.tokens * a.n_ops * a.slices;
    a.split = units < kSplitUnits && std::max(a.width[0], a.n_ops == 2 ? a.width[1] : 0) > 32 ? kWarps : 1;
    const int64_t blocks = a.split > 1 ? units : (units + kWarps - 1) / kWarps;
    if (blocks > INT_MAX) return SDM_ECOUNT;
    void* args[] = {&a};
    return launch_pdl_raw(fn, dim3((unsigned)blocks), dim3(kThreads), a.split > 1 ? smem : 0, stream, args);
}

}  // namespace

int launch_qgather(const QGatherArgs& a0, int format, cudaStream_t stream) {
    QGatherArgs a = a0;
    const int C = columns(format);
    a.pieces = (a.hd + C - 1) / C;
    a.groups = (a.hd + a.group - 1) / a.group;
    a.row_bytes = (int64_t)a.pieces * 16;
    const int lr = row_lanes(a.pieces);
    a.slices = (a.pieces + lr - 1) / lr;
    a.vec_out = a.hd % 4 == 0 && aligned16(a.out[0]) && (a.n_ops == 1 || aligned16(a.out[1]));
    const void* fn = format == SDM_INT8 ? qgather_of<Int8>(lr) : format == SDM_FP8 ? qgather_of<Fp8>(lr) : qgather_of<Int4>(lr);
    return run(fn, a, sizeof(float) * kThreads * C * lr / 32, stream);
}

int launch_gather_dw(const QGatherArgs& a0, int format, cudaStream_t stream) {
    QGatherArgs a = a0;
    const int C = columns(format);
    a.pieces = (a.hd + C - 1) / C;
    const bool quantised = format != SDM_BF16 && format != SDM_F32;
    a.groups = quantised ? (a.hd + a.group - 1) / a.group : 0;
    a.row_bytes = quantised ? (int64_t)a.pieces * 16 : (int64_t)a.hd * (format == SDM_BF16 ? 2 : 4);
    a.slices = 1;
    a.vec_out = a.hd % 4 == 0 && aligned16(a.dout[0]) && (a.n_ops == 1 || aligned16(a.dout[1]));
    const int lr = row_lanes(a.pieces);
    const bool al = quantised || (a.row_bytes % 16 == 0 && aligned16(a.bank));
    const void* fn = format == SDM_INT8   ? dw_of<Int8>(lr)
                     : format == SDM_FP8  ? dw_of<Fp8>(lr)
                     : format == SDM_INT4 ? dw_of<Int4>(lr)
                     : format == SDM_BF16 ? (al ? dw_of<Bf16>(lr) : dw_of<Bf16, false>(lr))
                                          : (al ? dw_of<F32>(lr) : dw_of<F32, false>(lr));
    return run(fn, a, 0, stream);
}

int qgather_status(unsigned int* word, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(word, g_qgather_status, sizeof(unsigned int));
    if (e == cudaSuccess && clear) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_qgather_status, &zero, sizeof(unsigned int));
    }
    return (int)e;
}

}  // namespace sdm
