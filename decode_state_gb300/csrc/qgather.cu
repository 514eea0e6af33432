// Gather over a quantised bank, and the gradient of a gather's weights.
//
// Math (include/sdm.h): out[t] = sum_n w[t, n] * row(idx[t, n]) and
// dw[t, n] = <dout[t], row(idx[t, n])>, row = scale * code (or the row of a bf16 / float32 bank).
//
// Design. Here are the kernels for few tokens, and for banks whose rows are not 16-byte aligned, and the
// choice between them and those for many (qgather_ring.cu). LR lanes hold one row or a slice of it, 16
// bytes each, so a warp reads 32 / LR rows at once. A block of four warps shares a token's entries, rows
// go straight to registers, and the sums are joined through shared memory; with few tokens the machine
// is idle otherwise, and a ring has nothing to run ahead of. The rule between them looks at the sizes
// only, so that results do not depend on the GPU. Bound by latency: 256 tokens with 64 int8 rows of 128
// columns take 2.6 us from a graph, a launch and two loads that wait for one another, the index and the row.
#include <algorithm>
#include <climits>

#include "qgather_device.cuh"

namespace sdm {
namespace {

__device__ unsigned int g_qgather_status;

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int64_t kRingUnits = 4096;  // units from which on the ring kernel is used
// Chunks whose prefix sums the ring kernel keeps in shared memory; a call with chunk_valid and more of them
// stays here, whatever its tokens: 65536 tokens of 64 and 64 fp8 rows (the gradient of 64 int8 rows) take 215 us (138) in
// 16384 chunks of 4 and 440 (253) in 32768 of 2.
constexpr int kMaxChunks = 16384;
constexpr unsigned kAll = 0xffffffffu;

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

template <int C>
__device__ __forceinline__ void load_dout(const float* dout, int c0, int hd, bool vec, float* d) {
    if (vec && c0 + C <= hd) {
#pragma unroll
        for (int i = 0; i < C / 4; ++i) {
            const float4 f = __ldg(reinterpret_cast<const float4*>(dout + c0) + i);
            d[4 * i] = f.x, d[4 * i + 1] = f.y, d[4 * i + 2] = f.z, d[4 * i + 3] = f.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < C; ++i) d[i] = c0 + i < hd ? __ldg(dout + c0 + i) : 0.0f;
    }
}

// x[0 .. KEEP) to the columns c0 .. of a float32 row
template <int KEEP>
__device__ __forceinline__ void store_columns(float* row, int c0, int hd, bool vec, const float* x) {
    if (KEEP % 4 == 0 && vec && c0 + KEEP <= hd) {
#pragma unroll
        for (int i = 0; i < KEEP / 4; ++i)
            reinterpret_cast<float4*>(row + c0)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < KEEP; ++i)
            if (c0 + i < hd) row[c0 + i] = x[i];
    }
}

template <typename F>
__device__ __forceinline__ void add_piece(float weight, const uint4& v, f32x2* acc) {
    f32x2 x[F::C / 2];
    F::unpack2(v, x);
    const f32x2 f = pair(weight, weight);
#pragma unroll
    for (int i = 0; i < F::C / 2; ++i) acc[i] = fma2(f, x[i], acc[i]);
}

// ---------------------------------------------------------------- direct: four warps for a token

// the block's unit, and its warp's share [e0, e1) of the entries: even, in whole rows of `slots`
struct Share {
    int64_t t;
    int op, slice, e0, e1;
};

__device__ __forceinline__ Share share_of(const QGatherArgs& a, int slots) {
    Share r;
    const int64_t u = blockIdx.x;
    r.slice = a.slices > 1 ? (int)(u % a.slices) : 0;
    const int64_t v = a.slices > 1 ? u / a.slices : u;
    r.op = a.n_ops == 2 ? (int)(v & 1) : 0;
    r.t = a.n_ops == 2 ? v >> 1 : v;
    const int n = a.width[r.op], per = ((n + kWarps - 1) / kWarps + slots - 1) / slots * slots;
    r.e0 = min(n, (int)(threadIdx.x >> 5) * per);
    r.e1 = min(n, r.e0 + per);
    return r;
}

template <typename F, int LR>
__global__ void __launch_bounds__(kThreads) qgather_direct(const QGatherArgs a) {
    constexpr int C = F::C, SLOTS = 32 / LR, KEEP = C / SLOTS, BATCH = LR < 8 ? LR : 8;
    static_assert(KEEP >= 1, "every row slot keeps columns");
    __shared__ __align__(16) float joined[kThreads * KEEP];
    grid_dependency_wait();
    grid_launch_dependents();
    const Share u = share_of(a, SLOTS);
    const int lane = threadIdx.x & 31, rs = lane / LR, p = u.slice * LR + lane % LR;
    const int hd = a.hd, NR = a.width[u.op];
    f32x2 acc2[C / 2];
#pragma unroll
    for (int i = 0; i < C / 2; ++i) acc2[i] = 0;

    if (!padding(a, u.t)) {
        const bool active = p < a.pieces;
        const unsigned char* bank = static_cast<const unsigned char*>(a.bank) + (int64_t)p * 16;
        const float* scales = a.scales + (p * C) / a.group;
        const int64_t first = u.t * NR;
        for (int base = u.e0; base < u.e1; base += 32) {
            int slot = -1;
            float w = 0.0f;
            if (base + lane < u.e1) {
                slot = entry_slot(a, a.idx[u.op], first + base + lane);
                w = a.w_bf16 ? to_f32(__ldg(static_cast<const uint16_t*>(a.w[u.op]) + first + base + lane))
                             : __ldg(static_cast<const float*>(a.w[u.op]) + first + base + lane);
                w = slot >= 0 ? w : 0.0f;  // a skipped entry's may be anything
            }
#pragma unroll
            for (int s0 = 0; s0 < LR; s0 += BATCH) {
                if (base + s0 * SLOTS >= u.e1) break;
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
                for (int s = 0; s < BATCH; ++s) add_piece<F>(ws[s] * sc[s], v[s], acc2);
            }
        }
    }

    float acc[C];
#pragma unroll
    for (int i = 0; i < C / 2; ++i) split(acc2[i], acc[2 * i], acc[2 * i + 1]);
    const int first = reduce_scatter<C, LR>(acc, lane);
#pragma unroll
    for (int i = 0; i < KEEP; ++i) joined[threadIdx.x * KEEP + i] = acc[i];
    __syncthreads();
    if (threadIdx.x >= 32) return;
#pragma unroll
    for (int i = 0; i < KEEP; ++i) {
        for (int q = 1; q < kWarps; ++q) acc[i] += joined[(q * 32 + lane) * KEEP + i];
    }
    store_columns<KEEP>(a.out[u.op] + u.t * hd, p * C + first, hd, a.vec_out, acc);
}

// The warp walks the slices of its rows itself (a.slices is 1).
template <typename F, int LR, bool ALIGNED>
__global__ void __launch_bounds__(kThreads) gather_dw_direct(const QGatherArgs a) {
    constexpr int C = F::C, SLOTS = 32 / LR, BATCH = LR < 8 ? LR : 8;
    grid_dependency_wait();
    grid_launch_dependents();
    const Share u = share_of(a, SLOTS);
    const int lane = threadIdx.x & 31, rs = lane / LR;
    const int hd = a.hd, NR = a.width[u.op];
    const int64_t first = u.t * NR;
    const bool pad = padding(a, u.t);
    const int slices = (a.pieces + LR - 1) / LR;
    const float* dout = a.dout[u.op] + u.t * hd;
    float d[C];
    if (!pad && slices == 1) load_dout<C>(dout, lane % LR * C, hd, a.vec_out, d);

    for (int base = u.e0; base < u.e1; base += 32) {
        int slot = -1;
        float dot[LR];  // row slot rs, step s: entry base + s * SLOTS + rs
#pragma unroll
        for (int s = 0; s < LR; ++s) dot[s] = 0.0f;
        if (!pad) {
            if (base + lane < u.e1) slot = entry_slot(a, a.idx[u.op], first + base + lane);
            for (int slice = 0; slice < slices; ++slice) {
                const int p = slice * LR + lane % LR;
                if (slices > 1) load_dout<C>(dout, p * C, hd, a.vec_out, d);
#pragma unroll
                for (int s0 = 0; s0 < LR; s0 += BATCH) {
                    if (base + s0 * SLOTS >= u.e1) break;
                    uint4 v[BATCH];
                    float sc[BATCH];
#pragma unroll
                    for (int s = 0; s < BATCH; ++s) {
                        const int sl = __shfl_sync(kAll, slot, (s0 + s) * SLOTS + rs);
                        const bool on = sl >= 0 && p < a.pieces;
                        v[s] = load_piece<F, ALIGNED>(static_cast<const unsigned char*>(a.bank) + sl * a.row_bytes + (int64_t)p * 16,
                                                      hd - p * C, on);
                        if constexpr (F::kQuantised) sc[s] = load4_if(a.scales + (int64_t)sl * a.groups + p * C / a.group, on);
                    }
#pragma unroll
                    for (int s = 0; s < BATCH; ++s) {
                        const float sum = dot_piece<F>(d, v[s]);
                        if constexpr (F::kQuantised)
                            dot[s0 + s] = fmaf(sum, sc[s], dot[s0 + s]);
                        else
                            dot[s0 + s] += sum;
                    }
                }
            }
            // the sums over the lanes of a row, lane j of them keeping step j's
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
        const int at = lane % LR * SLOTS + rs, e = base + at;
        const bool read = __shfl_sync(kAll, slot, at) >= 0;  // a skipped entry's is 0 whatever dout holds
        if (e < u.e1) store_dw(a, u.op, first + e, read ? dot[0] : 0.0f);
    }
}

// ---------------------------------------------------------------- choice

template <typename F, bool GRAD, bool ALIGNED, int LR>
const void* direct_lr() {
    if constexpr (GRAD)
        return (const void*)gather_dw_direct<F, LR, ALIGNED>;
    else
        return (const void*)qgather_direct<F, LR>;
}

template <typename F, bool GRAD, bool ALIGNED = true>
const void* direct(int lr) {
    return lr == 4    ? direct_lr<F, GRAD, ALIGNED, 4>()
           : lr == 8  ? direct_lr<F, GRAD, ALIGNED, 8>()
           : lr == 16 ? direct_lr<F, GRAD, ALIGNED, 16>()
                      : direct_lr<F, GRAD, ALIGNED, 32>();
}

int columns(int format) { return format == SDM_INT4 ? 32 : format == SDM_BF16 ? 8 : format == SDM_F32 ? 4 : 16; }

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Lanes of a row in the direct kernels, whose time is the loads that wait for one another: a warp's
// entries by batches of 8 rows a lane, and in the gradient by slices. Of equals the fewest lanes over.
// The gradient of 1000 tokens with 37 bf16 rows of 33 pieces: 8.1 us by this rule (3 slices of 16 lanes),
// 14.0 by the fewest lanes over alone (nine slices of 4).
int direct_lanes(const QGatherArgs& a, bool grad) {
    const int entries = (std::max(a.width[0], a.n_ops == 2 ? a.width[1] : 0) + kWarps - 1) / kWarps;
    int best = 0, best_waits = 0, best_lanes = 0;
    for (int lr = 32; lr >= 4; lr /= 2) {
        const int slices = (a.pieces + lr - 1) / lr, steps = (entries + 32 / lr - 1) / (32 / lr), batch = std::min(lr, 8);
        const int waits = (steps + batch - 1) / batch * (grad ? slices : 1);
        if (best == 0 || waits < best_waits || (waits == best_waits && slices * lr < best_lanes)) best = lr, best_waits = waits, best_lanes = slices * lr;
    }
    return best;
}

// fn(lr): the direct kernel. `ring`: the rows are 16-byte aligned.
template <typename Fn>
int run(const Fn& fn, QGatherArgs& a, int format, bool grad, bool ring, cudaStream_t stream) {
    const int64_t chunks = a.tokens / a.chunk;
    if (ring && a.tokens * a.n_ops >= kRingUnits && a.tokens * a.pieces <= INT_MAX && (!a.chunk_valid || chunks <= kMaxChunks))
        return launch_gather_ring(a, format, grad, stream);
    const int lr = direct_lanes(a, grad);
    a.slices = grad ? 1 : (a.pieces + lr - 1) / lr;
    const int64_t units = a.tokens * a.n_ops * a.slices;
    if (units > INT_MAX) return SDM_ECOUNT;
    void* args[] = {&a};
    return launch_pdl_raw(fn(lr), dim3((unsigned)units), dim3(kThreads), 0, stream, args);
}

}  // namespace

int row_lanes(int pieces, int most) {
    int best = most;
    for (int lr = most; lr >= 4; lr /= 2)
        if ((pieces + lr - 1) / lr * lr < (pieces + best - 1) / best * best) best = lr;
    return best;
}

int launch_qgather(const QGatherArgs& a0, int format, cudaStream_t stream) {
    QGatherArgs a = a0;
    const int C = columns(format);
    a.pieces = (a.hd + C - 1) / C;
    a.groups = (a.hd + a.group - 1) / a.group;
    a.row_bytes = (int64_t)a.pieces * 16;
    a.vec_out = a.hd % 4 == 0 && aligned16(a.out[0]) && (a.n_ops == 1 || aligned16(a.out[1]));
    const auto fn = [&](int lr) {
        return format == SDM_INT8 ? direct<Int8, false>(lr) : format == SDM_FP8 ? direct<Fp8, false>(lr) : direct<Int4, false>(lr);
    };
    return run(fn, a, format, false, true, stream);
}

int launch_gather_dw(const QGatherArgs& a0, int format, cudaStream_t stream) {
    QGatherArgs a = a0;
    const int C = columns(format);
    a.pieces = (a.hd + C - 1) / C;
    const bool quantised = format != SDM_BF16 && format != SDM_F32;
    a.groups = quantised ? (a.hd + a.group - 1) / a.group : 0;
    a.row_bytes = quantised ? (int64_t)a.pieces * 16 : (int64_t)a.hd * (format == SDM_BF16 ? 2 : 4);
    a.vec_out = a.hd % 4 == 0 && aligned16(a.dout[0]) && (a.n_ops == 1 || aligned16(a.dout[1]));
    const bool al = quantised || (a.row_bytes % 16 == 0 && aligned16(a.bank));
    const auto fn = [&](int lr) {
        return format == SDM_INT8   ? direct<Int8, true>(lr)
               : format == SDM_FP8  ? direct<Fp8, true>(lr)
               : format == SDM_INT4 ? direct<Int4, true>(lr)
               : format == SDM_BF16 ? (al ? direct<Bf16, true>(lr) : direct<Bf16, true, false>(lr))
                                    : (al ? direct<F32, true>(lr) : direct<F32, true, false>(lr));
    };
    return run(fn, a, format, true, al, stream);
}

cudaError_t qgather_status(void** word) { return cudaGetSymbolAddress(word, g_qgather_status); }

}  // namespace sdm
