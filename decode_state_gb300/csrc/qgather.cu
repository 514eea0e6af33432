// Gather over a quantised bank, and the gradient of a gather's weights.
//
// Math (include/sdm.h): out[t] = sum_n w[t, n] * row(idx[t, n]) and
// dw[t, n] = <dout[t], row(idx[t, n])>, row = scale * code (or the row of a bf16 / float32 bank).
//
// Design. Rows of 128 bytes at random places are what bounds both: at 7 TB/s every SM has to have
// some 50 KB of them on their way all the time. LR lanes hold one row (or a slice of it), 16 bytes
// each, so a warp reads 32 / LR rows at once.
//
// ring kernel (many tokens): persistent warps walk over the live tokens in steps of up to 32 entries.
// While a step is summed from shared memory, the rows of the next two are on their way by cp.async,
// and the indices of the one behind them by plain loads; no registers wait for rows, and the only
// barriers are within a warp. A block finds the live tokens by the prefix sums of chunk_valid, so
// that every warp gets as many of them: by token number, warps whose tokens mostly lay at the end of
// their chunks were done long before the others.
//
// direct kernel (few tokens, or a bank whose rows are not 16-byte aligned): a block of four warps
// shares a token's entries, rows go straight to registers, and the sums are joined through shared
// memory; with few tokens the machine is idle otherwise, and a ring has nothing to run ahead of.
// The rule between them looks at the sizes only, so that results do not depend on the GPU.
#include <algorithm>
#include <climits>

#include "quant_device.cuh"
#include "sdm_internal.h"

namespace sdm {
namespace {

__device__ unsigned int g_qgather_status;

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int64_t kRingUnits = 4096;  // units from which on the ring kernel is used
constexpr int kMaxChunks = 16384;     // chunks whose prefix sums the ring kernel keeps in shared memory
constexpr int kRingWarps = 16;        // warps of its blocks at most
constexpr unsigned kAll = 0xffffffffu;

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
__device__ __forceinline__ float dot_piece(const float* d, const uint4& v) {
    f32x2 x[F::C / 2], sum = 0;
    F::unpack2(v, x);
#pragma unroll
    for (int i = 0; i < F::C / 2; ++i) sum = fma2(pair(d[2 * i], d[2 * i + 1]), x[i], sum);
    float lo, hi;
    split(sum, lo, hi);
    return lo + hi;
}

template <typename F>
__device__ __forceinline__ void add_piece(float weight, const uint4& v, f32x2* acc) {
    f32x2 x[F::C / 2];
    F::unpack2(v, x);
    const f32x2 f = pair(weight, weight);
#pragma unroll
    for (int i = 0; i < F::C / 2; ++i) acc[i] = fma2(f, x[i], acc[i]);
}

__device__ __forceinline__ void store_dw(const QGatherArgs& a, int op, int64_t i, float x) {
    if (a.w_bf16)
        static_cast<uint16_t*>(a.dw[op])[i] = from_f32<uint16_t>(x);
    else
        static_cast<float*>(a.dw[op])[i] = x;
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
        float dot[LR];  // row slot rs, step s: entry base + s * SLOTS + rs
#pragma unroll
        for (int s = 0; s < LR; ++s) dot[s] = 0.0f;
        if (!pad) {
            const int slot = base + lane < u.e1 ? entry_slot(a, a.idx[u.op], first + base + lane) : -1;
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
        const int e = base + lane % LR * SLOTS + rs;
        if (e < u.e1) store_dw(a, u.op, first + e, dot[0]);
    }
}

// ---------------------------------------------------------------- ring: persistent warps

constexpr int kAhead = 2;  // steps whose rows are on their way while one is summed

__device__ __forceinline__ void copy16_if(void* dst, const void* src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4_if(void* dst, const void* src, bool on) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(on ? 4 : 0) : "memory");
}

// One step's share of shared memory: the rows' slices by 16-byte pieces, the entries' scales, and for
// the gradient the slice of dout. ONE: a row's slice has one scale.
template <typename F, int LR, bool GRAD, bool ONE>
struct RingStage {
    static constexpr int ENTRIES = LR <= 8 ? 32 : 256 / LR;  // of a step, so that its rows are 4 KB
    static constexpr int STEPS = ENTRIES * LR / 32;          // rows of a row slot
    static constexpr int COLS = LR * F::C;
    static constexpr int GROUPS = !F::kQuantised ? 0 : ONE ? 1 : (COLS + 31) / 32;  // scales of a row's slice at most
    uint4 rows[ENTRIES * LR];
    float dout[GRAD ? COLS : 4];
    float scale[GROUPS > 0 ? ENTRIES * GROUPS : 4];
};

// Where a step is: token, column slice, operand, its first entry; token -1: none.
struct Step {
    int t, slice, op, base;
};

// F: format. LR: lanes of a row. GRAD: the weights' gradient.
template <typename F, int LR, bool GRAD, bool ONE>
__global__ void __launch_bounds__(kRingWarps * 32, 1) gather_ring(const QGatherArgs a) {
    using S = RingStage<F, LR, GRAD, ONE>;
    constexpr int C = F::C, SLOTS = 32 / LR, KEEP = C / SLOTS > 0 ? C / SLOTS : 1, STEPS = S::STEPS, ENTRIES = S::ENTRIES;
    extern __shared__ __align__(16) unsigned char ring[];
    __shared__ int warp_sums[kRingWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    const int rs = lane / LR, lp = lane % LR, hd = a.hd;
    const int tokens = (int)a.tokens, chunks = tokens / a.chunk;
    int* prefix = reinterpret_cast<int*>(ring);  // [chunks + 1] live tokens ahead of a chunk, with chunk_valid
    S* stages = reinterpret_cast<S*>(ring + (a.chunk_valid ? ((size_t)chunks + 4) / 4 * 16 : 0)) + warp * (kAhead + 1);
    const int slices = (a.pieces + LR - 1) / LR;
    const int unit_slices = GRAD ? 1 : slices;  // the gradient's steps walk over the slices themselves
    grid_dependency_wait();
    grid_launch_dependents();

    int live = chunks * a.valid;  // live tokens
    if (a.chunk_valid != nullptr) {
        const int per = (chunks + blockDim.x - 1) / blockDim.x, c0 = min(chunks, tid * per), c1 = min(chunks, c0 + per);
        int own = 0;
        for (int c = c0; c < c1; ++c) own += min(max(__ldg(a.chunk_valid + c), 0), a.chunk);
        int sum = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kAll, sum, o);
            if (lane >= o) sum += y;
        }
        if (lane == 31) warp_sums[warp] = sum;
        __syncthreads();
        sum -= own;
        live = 0;
        for (int w = 0; w < warps; ++w) {
            if (w < warp) sum += warp_sums[w];
            live += warp_sums[w];
        }
        for (int c = c0; c < c1; ++c) {
            prefix[c] = sum;
            sum += min(max(__ldg(a.chunk_valid + c), 0), a.chunk);
        }
        if (tid == 0) prefix[chunks] = live;
        __syncthreads();
    }
    // the k-th live token
    const auto live_token = [&](int k) {
        if (a.chunk_valid == nullptr) return a.valid == a.chunk ? k : k / a.valid * a.chunk + k % a.valid;
        int lo = 0, hi = chunks - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (prefix[mid] <= k)
                lo = mid;
            else
                hi = mid - 1;
        }
        return lo * a.chunk + k - prefix[lo];
    };

    const int me = blockIdx.x * warps + warp, stride = gridDim.x * warps;
    const int64_t units = (int64_t)live * unit_slices;
    int64_t next = me;  // the unit behind the 32 that the lanes hold
    int held_t = 0, held_slice = 0, held = 0, taken = 0;
    Step at{-1, 0, 0, 0};
    // the next step of this warp's walk
    const auto advance = [&]() {
        if (at.t >= 0) {
            if (GRAD && ++at.slice < slices) return;
            if (GRAD) at.slice = 0;
            at.base += ENTRIES;
            if (at.base < a.width[at.op]) return;
            at.base = 0;
            if (++at.op < a.n_ops) return;
        }
        at.op = at.base = 0;
        if (taken == held) {
            const int64_t u = next + (int64_t)lane * stride;
            held = __popc(__ballot_sync(kAll, u < units));
            taken = 0;
            next += 32 * (int64_t)stride;
            if (u < units) {
                const int k = (int)(unit_slices > 1 ? u / unit_slices : u);
                held_slice = unit_slices > 1 ? (int)(u - (int64_t)k * unit_slices) : 0;
                held_t = live_token(k);
            }
        }
        if (taken < held) {
            at.t = __shfl_sync(kAll, held_t, taken);
            at.slice = __shfl_sync(kAll, held_slice, taken);
            ++taken;
        } else {
            at.t = -1;
            held = taken = 0;
            next = units;
        }
    };
    // a step's indices and weights as they are in memory, an entry for each lane
    uint32_t raw_lo = 0, raw_hi = 0, raw_w = 0;
    const auto load_entries = [&]() {
        const int e = at.base + lane;
        if (at.t < 0 || lane >= ENTRIES || e >= a.width[at.op]) return;
        const int64_t i = (int64_t)at.t * a.width[at.op] + e;
        const uint32_t* word = static_cast<const uint32_t*>(a.idx[at.op]) + (a.idx64 ? 2 * i : i);
        raw_lo = __ldg(word);
        if (a.idx64) raw_hi = __ldg(word + 1);
        if (!GRAD) raw_w = a.w_bf16 ? __ldg(static_cast<const uint16_t*>(a.w[at.op]) + i) : __ldg(static_cast<const uint32_t*>(a.w[at.op]) + i);
    };
    // request the step's rows (one commit for every step, requested or not); returns the lane's weight
    const auto request = [&](S& st) {
        float weight = 0.0f;
        if (at.t >= 0) {
            const int n = a.width[at.op] - at.base;
            int slot = -1;
            if (lane < min(n, ENTRIES)) {
                const int64_t x = a.idx64 ? (int64_t)((uint64_t)raw_hi << 32 | raw_lo) : (int64_t)(int32_t)raw_lo;
                if (x >= 0 && x < a.n_slots)
                    slot = (int)x;
                else
                    atomicOr(&g_qgather_status, SDM_DEV_BAD_INDEX);
                weight = a.w_bf16 ? __uint_as_float(raw_w << 16) : __uint_as_float(raw_w);
            }
            const int p = at.slice * LR + lp, g0 = ONE ? 0 : at.slice * LR * C / a.group;
            const unsigned char* bank = static_cast<const unsigned char*>(a.bank) + p * 16;
            const bool active = p < a.pieces;
            uint4* to = st.rows + lane;
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                const int sl = __shfl_sync(kAll, slot, s * SLOTS + rs);
                copy16_if(to + s * 32, bank + sl * a.row_bytes, sl >= 0 && active);
            }
            if constexpr (F::kQuantised) {
                const float* scales = a.scales + (int64_t)slot * a.groups + g0;
                if (ONE) {
                    if (lane < ENTRIES) copy4_if(&st.scale[lane], scales, slot >= 0);
                } else if (lane < ENTRIES) {
                    const int ng = min(a.groups - g0, (LR * C + a.group - 1) / a.group);
                    for (int g = 0; g < ng; ++g) copy4_if(&st.scale[lane * S::GROUPS + g], scales + g, slot >= 0);
                }
            }
            if (GRAD) {
                const float* d = a.dout[at.op] + (int64_t)at.t * hd + at.slice * LR * C;
                const int left = hd - at.slice * LR * C;
                if (a.vec_out) {
                    for (int c = lane; c < LR * C / 4; c += 32) copy16_if(&st.dout[4 * c], d + 4 * c, 4 * c < left);
                } else {
                    for (int c = lane; c < LR * C; c += 32) copy4_if(&st.dout[c], d + c, c < left);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        return weight;
    };

    Step steps[kAhead + 1];  // the steps of the ring, the oldest first, and their weights
    float weights[kAhead + 1];
    int head = 0;  // the stage of the oldest
    advance();
    load_entries();
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
        steps[i] = at;
        weights[i] = request(stages[i]);
        if (at.t >= 0) advance();
        load_entries();
    }
    // padding tokens: zeros, while the first rows are on their way
    if (live < tokens) {
        for (int64_t t0 = (int64_t)me * 32; t0 < tokens; t0 += (int64_t)stride * 32) {
            for (uint32_t pads = __ballot_sync(kAll, t0 + lane < tokens && padding(a, t0 + lane)); pads; pads &= pads - 1) {
                const int64_t t = t0 + __ffs(pads) - 1;
                for (int op = 0; op < a.n_ops; ++op) {
                    if (GRAD) {
                        for (int i = lane; i < a.width[op]; i += 32) store_dw(a, op, t * a.width[op] + i, 0.0f);
                    } else if (a.vec_out) {
                        for (int c = 4 * lane; c < hd; c += 128) *reinterpret_cast<float4*>(a.out[op] + t * hd + c) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    } else {
                        for (int c = lane; c < hd; c += 32) a.out[op][t * hd + c] = 0.0f;
                    }
                }
            }
        }
    }
    f32x2 acc2[C / 2];
    float dot[STEPS];
    while (steps[0].t >= 0) {
        steps[kAhead] = at;
        weights[kAhead] = request(stages[head == 0 ? kAhead : head - 1]);
        if (at.t >= 0) advance();
        load_entries();
        asm volatile("cp.async.wait_group %0;" ::"n"(kAhead) : "memory");
        __syncwarp();
        const S& st = stages[head];
        const Step now = steps[0];
        const int width = a.width[now.op], n = width - now.base;  // entries from here on
        const int p = now.slice * LR + lp;
        const int gi = ONE || S::GROUPS == 0 ? 0 : min(p * C / a.group - now.slice * LR * C / a.group, S::GROUPS - 1);
        if constexpr (GRAD) {
            if (now.slice == 0) {
#pragma unroll
                for (int s = 0; s < STEPS; ++s) dot[s] = 0.0f;
            }
            float d[C];
#pragma unroll
            for (int i = 0; i < C; i += 4) {
                const float4 f = *reinterpret_cast<const float4*>(&st.dout[lp * C + i]);
                d[i] = f.x, d[i + 1] = f.y, d[i + 2] = f.z, d[i + 3] = f.w;
            }
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                if (s * SLOTS >= n) break;
                const float sum = dot_piece<F>(d, st.rows[s * 32 + lane]);
                if constexpr (F::kQuantised && !ONE)  // scales of lanes behind the row's end are not there
                    dot[s] = fmaf(sum, p < a.pieces ? st.scale[(s * SLOTS + rs) * S::GROUPS + gi] : 0.0f, dot[s]);
                else
                    dot[s] += sum;
            }
            if (now.slice + 1 == slices) {
                // the sums over the lanes of a row: halves of the steps are handed over while there are any
                int left = STEPS;
#pragma unroll
                for (int h = LR / 2; h >= 1; h /= 2) {
                    const bool up = lane & h;
                    if (left > 1) {
                        left /= 2;
#pragma unroll
                        for (int i = 0; i < STEPS / 2; ++i) {
                            if (i < left) {
                                const float keep = up ? dot[i + left] : dot[i], give = up ? dot[i] : dot[i + left];
                                dot[i] = keep + __shfl_xor_sync(kAll, give, h);
                            }
                        }
                    } else {
                        dot[0] += __shfl_xor_sync(kAll, dot[0], h);
                    }
                }
                constexpr int PER = LR / STEPS;  // lanes that hold the same step's sum
                const int e = lp / PER * SLOTS + rs;
                if (lp % PER == 0 && e < n) {
                    if constexpr (F::kQuantised && ONE) dot[0] *= st.scale[e];
                    store_dw(a, now.op, (int64_t)now.t * width + now.base + e, dot[0]);
                }
            }
        } else {
            if (now.base == 0) {
#pragma unroll
                for (int i = 0; i < C / 2; ++i) acc2[i] = 0;
            }
            const float own = ONE && lane < ENTRIES ? weights[0] * st.scale[lane] : weights[0];
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                if (s * SLOTS >= n) break;
                const int e = s * SLOTS + rs;
                float f = __shfl_sync(kAll, own, e);
                if (!ONE) f = p < a.pieces ? f * st.scale[e * S::GROUPS + gi] : 0.0f;
                add_piece<F>(f, st.rows[s * 32 + lane], acc2);
            }
            if (n <= ENTRIES) {
                float acc[C];
#pragma unroll
                for (int i = 0; i < C / 2; ++i) split(acc2[i], acc[2 * i], acc[2 * i + 1]);
                const int first = reduce_scatter<C, LR>(acc, lane);
                store_columns<KEEP>(a.out[now.op] + (int64_t)now.t * hd, p * C + first, hd, a.vec_out, acc);
            }
        }
        __syncwarp();  // the stage may be filled again
        head = head == kAhead ? 0 : head + 1;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            steps[i] = steps[i + 1];
            weights[i] = weights[i + 1];
        }
    }
}

// ---------------------------------------------------------------- choice

struct Kernels {
    const void *direct, *ring;
    size_t stage_bytes;
};

template <typename F, int LR, bool GRAD, bool ALIGNED>
Kernels kernels_lr(bool one) {
    const void* direct;
    if constexpr (GRAD)
        direct = (const void*)gather_dw_direct<F, LR, ALIGNED>;
    else
        direct = (const void*)qgather_direct<F, LR>;
    if constexpr (!ALIGNED) return {direct, nullptr, 0};
    if constexpr (F::kQuantised) {
        if (!one) return {direct, (const void*)gather_ring<F, LR, GRAD, false>, sizeof(RingStage<F, LR, GRAD, false>)};
    }
    return {direct, (const void*)gather_ring<F, LR, GRAD, true>, sizeof(RingStage<F, LR, GRAD, true>)};
}

template <typename F, bool GRAD, bool ALIGNED = true>
Kernels kernels(int lr, bool one) {
    return lr == 4    ? kernels_lr<F, 4, GRAD, ALIGNED>(one)
           : lr == 8  ? kernels_lr<F, 8, GRAD, ALIGNED>(one)
           : lr == 16 ? kernels_lr<F, 16, GRAD, ALIGNED>(one)
                      : kernels_lr<F, 32, GRAD, ALIGNED>(one);
}

int columns(int format) { return format == SDM_INT4 ? 32 : format == SDM_BF16 ? 8 : format == SDM_F32 ? 4 : 16; }

// Lanes that hold a row or a slice of it: the number that leaves the fewest lanes over, the larger of
// equals (its rows come in longer runs).
int row_lanes(int pieces) {
    int best = 32;
    for (int lr = 32; lr >= 4; lr /= 2)
        if ((pieces + lr - 1) / lr * lr < (pieces + best - 1) / best * best) best = lr;
    return best;
}

bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

int run(const Kernels& k, QGatherArgs& a, cudaStream_t stream) {
    const int64_t units = a.tokens * a.n_ops * a.slices, chunks = a.tokens / a.chunk;
    void* args[] = {&a};
    if (units < kRingUnits || k.ring == nullptr || a.tokens * a.slices > INT_MAX || (a.chunk_valid && chunks > kMaxChunks)) {
        if (units > INT_MAX) return SDM_ECOUNT;
        return launch_pdl_raw(k.direct, dim3((unsigned)units), dim3(kThreads), 0, stream, args);
    }
    // one block for every SM, of as many warps as find room for their stages
    const size_t prefix = a.chunk_valid ? ((size_t)chunks + 4) / 4 * 16 : 0, per_warp = k.stage_bytes * (kAhead + 1);
    const size_t room = smem_per_sm() - smem_reserved_per_block() - kRingWarps * 4 - prefix;
    const int warps = (int)std::min<size_t>(kRingWarps, room / per_warp);
    const size_t smem = prefix + per_warp * warps;
    const int rc = allow_smem(k.ring, smem);
    if (rc != 0) return rc;
    const int64_t blocks = std::min((int64_t)sm_count(), (a.tokens * a.slices + warps - 1) / warps);
    return launch_pdl_raw(k.ring, dim3((unsigned)blocks), dim3(warps * 32), smem, stream, args);
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
    const bool one = a.groups == 1;
    return run(format == SDM_INT8  ? kernels<Int8, false>(lr, one)
               : format == SDM_FP8 ? kernels<Fp8, false>(lr, one)
                                   : kernels<Int4, false>(lr, one),
               a, stream);
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
    const bool al = quantised || (a.row_bytes % 16 == 0 && aligned16(a.bank)), one = a.groups <= 1;
    return run(format == SDM_INT8   ? kernels<Int8, true>(lr, one)
               : format == SDM_FP8  ? kernels<Fp8, true>(lr, one)
               : format == SDM_INT4 ? kernels<Int4, true>(lr, one)
               : format == SDM_BF16 ? (al ? kernels<Bf16, true>(lr, one) : kernels<Bf16, true, false>(lr, one))
                                    : (al ? kernels<F32, true>(lr, one) : kernels<F32, true, false>(lr, one)),
               a, stream);
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
