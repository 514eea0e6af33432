// The balance loss of a router, the counts of its entries, and the gradient of its logits.
//
// Math (include/sdm.h): with p the shares of a token's scores and c the counts of its sequence,
//     loss = scale * n / (T C) * sum_t sum_j c_j p_tj,   dx_j = dloss * scale * n / (T C) * p_j (c_j - sum_i c_i p_i) [(1 - s_j)].
// The counts come first, from the indices alone; then one pass over the logits has both the loss and the
// gradient, since the loss is a sum over tokens of <c, p> and the gradient of a token needs no other token. Column
// sums of p, which a mean over tokens asks for at first sight, would hold n sums for every block and a second
// pass for the gradient.
//
// Counts enter without their mean, c' = c - C / n: as the p of a token sum to one, <c, p> = C / n + <c', p> and
// c_j - <c, p> = c'_j - <c', p>. Near balance the c' are small, and so are then the errors of the differences.
#include <algorithm>
#include <climits>

#include "score_device.cuh"
#include "sdm_internal.h"

namespace sdm {
namespace {

__device__ unsigned int g_balance_status;

constexpr int kCountThreads = 256;
constexpr int kCountBins = 4096;  // entries of a row that a block counts in shared memory

// The sequence of token t: its number (-1: none) and the tokens around t that share it (offsets out of order give
// some such range, empty perhaps).
struct Sequence {
    int64_t s;
    int64_t begin, end;
};
__device__ __forceinline__ Sequence sequence_of(const int32_t* offsets, int64_t sequences, int64_t tokens, int64_t t) {
    if (offsets == nullptr) return {0, 0, tokens};
    int64_t lo = 0, hi = sequences + 1;  // the first offset beyond t
    while (lo < hi) {
        const int64_t mid = (lo + hi) >> 1;
        if (__ldg(offsets + mid) > t)
            hi = mid;
        else
            lo = mid + 1;
    }
    const int64_t begin = lo > 0 ? __ldg(offsets + lo - 1) : 0, end = lo <= sequences ? __ldg(offsets + lo) : tokens;
    return {lo > 0 && lo <= sequences ? lo - 1 : -1, begin, end < tokens ? end : tokens};
}

__global__ void __launch_bounds__(kCountThreads) balance_zero_kernel(const BalanceArgs a) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t all = a.sequences * a.n, step = (int64_t)gridDim.x * kCountThreads;
    for (int64_t i = (int64_t)blockIdx.x * kCountThreads + threadIdx.x; i < all; i += step) a.counts[i] = 0;
    for (int64_t i = (int64_t)blockIdx.x * kCountThreads + threadIdx.x; i < a.sequences; i += step) a.totals[i] = 0;
}

// The column of entry e of token t, or -1: an entry of weight 0, or an index outside the row (flagged).
__device__ __forceinline__ int counted_column(const BalanceArgs& a, int64_t e, int64_t t) {
    int64_t j = a.idx64 ? __ldg(static_cast<const int64_t*>(a.idx) + e) : __ldg(static_cast<const int32_t*>(a.idx) + e);
    if (a.base != nullptr) j -= a.idx64 ? __ldg(static_cast<const int64_t*>(a.base) + t) : __ldg(static_cast<const int32_t*>(a.base) + t);
    if (j < 0 || j >= a.n) {
        atomicOr(&g_balance_status, SDM_DEV_BAD_INDEX);
        return -1;
    }
    return a.w != nullptr && __ldg(a.w + e) == 0.0f ? -1 : (int)j;
}

// Each block counts the entries of a run of tokens. LOCAL: in shared memory, one sequence of the run after the
// other, so that few entries of a short row do not queue up at the same words of L2.
template <bool LOCAL>
__global__ void __launch_bounds__(kCountThreads) balance_count_kernel(const BalanceArgs a, int64_t run) {
    __shared__ int bins[LOCAL ? kCountBins : 1];
    __shared__ int all;
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t first = blockIdx.x * run, last = first + run < a.tokens ? first + run : a.tokens;
    const int tid = threadIdx.x;
    if constexpr (LOCAL) {
        for (int64_t t = first; t < last;) {
            const Sequence q = sequence_of(a.offsets, a.sequences, a.tokens, t);
            const int64_t end = q.end < t + 1 ? t + 1 : q.end < last ? q.end : last;
            if (q.s >= 0) {
                for (int j = tid; j < a.n; j += kCountThreads) bins[j] = 0;
                if (tid == 0) all = 0;
                __syncthreads();
                int mine = 0;
                for (int64_t e = t * a.k + tid; e < end * a.k; e += kCountThreads) {
                    const int j = counted_column(a, e, a.base != nullptr ? (int64_t)((uint32_t)e / (uint32_t)a.k) : 0);
                    if (j >= 0) {
                        atomicAdd(&bins[j], 1);
                        ++mine;
                    }
                }
                mine = __reduce_add_sync(kAll, mine);
                if ((tid & 31) == 0 && mine) atomicAdd(&all, mine);
                __syncthreads();
                for (int j = tid; j < a.n; j += kCountThreads)
                    if (bins[j]) atomicAdd(a.counts + q.s * a.n + j, bins[j]);
                if (tid == 0 && all) atomicAdd(a.totals + q.s, all);
                __syncthreads();
            }
            t = end;
        }
    } else {
        const int64_t from = first * a.k, to = last * a.k;
        for (int64_t e0 = from; e0 < to; e0 += kCountThreads) {  // whole warps stay together
            const int64_t e = e0 + tid;
            int64_t s = -1;
            if (e < to) {
                const int64_t t = (uint32_t)e / (uint32_t)a.k;
                s = sequence_of(a.offsets, a.sequences, a.tokens, t).s;
                const int j = s >= 0 ? counted_column(a, e, t) : -1;
                if (j >= 0)
                    atomicAdd(a.counts + s * a.n + j, 1);
                else
                    s = -1;
            }
            const unsigned same = __match_any_sync(kAll, s);
            if (s >= 0 && (tid & 31) == __ffs(same) - 1) atomicAdd(a.totals + s, __popc(same));
        }
    }
}

// exp(x) for x <= 0. Of bf16 logits by the hardware's 2^x, 2 ulp of it and |x| roundings of the product: 1e-6 at
// x = -10, far below the logits' own 2^-9; of float32 logits by expf. A row of 256 bf16 logits spends a third less on it.
template <typename L>
__device__ __forceinline__ float exp_score(float x) {
    if constexpr (sizeof(L) == 4) return expf(x);
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x * 1.4426950408889634f));
    return y;
}

// A token's row for a team of TEAM threads (lanes of a warp, or a block), E logits a thread from one read to the
// gradient's write (E 0: rows too long for that are read again). VEC: 16 bytes an access, for rows that start on
// 16-byte boundaries; else 4. An access holds V consecutive entries, thread tid has those from (i * TEAM + tid) * V on.
template <int TEAM, int E, bool VEC, typename L>
struct Row {
    static constexpr int V = (VEC ? 16 : 4) / sizeof(L), W = V * sizeof(L) / 4, LANES = TEAM <= 32 ? TEAM : 32, WARPS = TEAM <= 32 ? 1 : TEAM / 32;
    static constexpr int R = E > 0 ? E : V, RAW = R / V * W;

    int n, tid;
    bool softmax, words;  // words: 4-byte accesses of two bf16 are aligned

    __device__ __forceinline__ Row(const BalanceArgs& a, int tid_) : n(a.n), tid(tid_), softmax(a.score == SDM_SOFTMAX) {
        words = VEC || V == 1 ||
                ((reinterpret_cast<uintptr_t>(a.logits) | reinterpret_cast<uintptr_t>(a.dlogits) | reinterpret_cast<uintptr_t>(a.add)) % 4 == 0 &&
                 ((a.row_stride | (a.dlogits ? a.dlogits_stride : 0) | (a.add ? a.add_stride : 0)) * sizeof(L)) % 4 == 0);
    }
    __device__ __forceinline__ int column(int i) const { return (i * TEAM + tid) * V; }  // of access i

    // the V entries from j on as they lie in memory; behind the end of the row, `fill` (the bits of an entry)
    __device__ __forceinline__ void get(const L* row, int j, uint32_t* w, uint32_t fill) const {
        if (words && j + V <= n) {
            if constexpr (VEC) {
                const uint4 v = *reinterpret_cast<const uint4*>(row + j);
                w[0] = v.x, w[1] = v.y, w[2] = v.z, w[W - 1] = v.w;
            } else {
                w[0] = *reinterpret_cast<const uint32_t*>(row + j);
            }
        } else {
#pragma unroll
            for (int i = 0; i < W; ++i) {
                if constexpr (sizeof(L) == 4)
                    w[i] = j + i < n ? reinterpret_cast<const uint32_t*>(row)[j + i] : fill;
                else
                    w[i] = (j + 2 * i < n ? (uint32_t)reinterpret_cast<const uint16_t*>(row)[j + 2 * i] : fill) |
                           (j + 2 * i + 1 < n ? (uint32_t)reinterpret_cast<const uint16_t*>(row)[j + 2 * i + 1] : fill) << 16;
            }
        }
    }
    static constexpr uint32_t kNone = sizeof(L) == 4 ? 0xff800000u : 0xff80u;  // -inf
    static __device__ __forceinline__ void unpack(const uint32_t* w, float* x) {
#pragma unroll
        for (int i = 0; i < W; ++i) {
            if constexpr (sizeof(L) == 4) {
                x[i] = __uint_as_float(w[i]);
            } else {
                x[2 * i] = __uint_as_float(w[i] << 16);
                x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
            }
        }
    }
    __device__ __forceinline__ void put(L* row, int j, const float* d) const {
        if (words && j + V <= n) {
            uint32_t w[W];
#pragma unroll
            for (int i = 0; i < W; ++i) {
                if constexpr (sizeof(L) == 4) {
                    w[i] = __float_as_uint(d[i]);
                } else {
                    const __nv_bfloat162 b = __floats2bfloat162_rn(d[2 * i], d[2 * i + 1]);
                    w[i] = *reinterpret_cast<const uint32_t*>(&b);
                }
            }
            if constexpr (VEC)
                *reinterpret_cast<uint4*>(row + j) = make_uint4(w[0], w[1], w[2], w[W - 1]);
            else
                *reinterpret_cast<uint32_t*>(row + j) = w[0];
        } else {
#pragma unroll
            for (int c = 0; c < V; ++c)
                if (j + c < n) row[j + c] = from_f32<L>(d[c]);
        }
    }
    // all of a thread's share of a row (none of it where the team has no row)
    __device__ __forceinline__ void get_all(const L* row, bool on, uint32_t* w, uint32_t fill) const {
#pragma unroll
        for (int i = 0; i < R / V; ++i) get(row, on ? column(i) : n, w + i * W, fill);
    }

    // the largest m of the team, the sums z and d of what is relative to each thread's own m
    __device__ __forceinline__ void join(bool soft, float& m, float& z, float& d, float (*joint)[WARPS]) const {
        if (TEAM < 32 ? __any_sync(kAll, soft) : soft) {
            const float mine = m;
            m = warp_max<LANES>(m);
            const float scale = soft ? exp_below(mine, m) : 1.0f;
            z *= scale;
            d *= scale;
        }
        z = warp_sum<LANES>(z);
        d = warp_sum<LANES>(d);
        if constexpr (TEAM > 32) {
            if ((tid & 31) == 0) {
                joint[0][tid >> 5] = m;
                joint[1][tid >> 5] = z;
                joint[2][tid >> 5] = d;
            }
            __syncthreads();
            const int lane = tid & 31, w = lane % WARPS;  // every warp for itself
            const float theirs = joint[0][w];
            m = warp_max<WARPS>(theirs);
            const float scale = lane >= WARPS ? 0.0f : soft ? exp_below(theirs, m) : 1.0f;
            z = warp_sum(joint[1][w] * scale);
            d = warp_sum(joint[2][w] * scale);
        }
    }

    // What the row adds to its sequence's loss, and its gradient where GRAD. `raw` holds the row (E 0: nothing); counts(i, j, c)
    // gives the counts less their mean of the V entries of access i, which start with entry j; `joint` is
    // shared memory that the team is done with.
    template <bool GRAD, typename C>
    __device__ __forceinline__ float pass(const L* row, uint32_t* raw, bool on, const C& counts, float unit, float g, L* out, const L* add,
                                          float (*joint)[WARPS]) const {
        uint32_t adds[RAW];
        constexpr bool EARLY = GRAD && E > 0 && TEAM <= 32 && RAW <= 8;  // what is added is on its way meanwhile
        if (EARLY && add != nullptr) get_all(add, on, adds, 0u);
        // Sigmoid scores so small that their sum loses bits are shares of exp(x) instead, as for a softmax.
        bool soft = softmax;
        float x[GRAD && E > 0 ? R : 1];  // scores; s (1 - s) of a sigmoid
        float m, mine, z, d;
        for (;;) {
            m = minus_inf();
            z = d = 0.0f;
            // f(access, first column, its V logits)
            const auto each = [&](const auto& f) {
                if constexpr (E > 0) {
#pragma unroll
                    for (int i = 0; i < R / V; ++i) {
                        float y[V];
                        unpack(raw + i * W, y);
                        f(i, column(i), y);
                    }
                } else {
#pragma unroll 4
                    for (int i = 0; column(i) < n; ++i) {
                        uint32_t w[W];
                        float y[V];
                        get(row, column(i), w, kNone);
                        unpack(w, y);
                        f(i, column(i), y);
                    }
                }
            };
            if (soft)
                each([&](int, int, const float* y) {
#pragma unroll
                    for (int c = 0; c < V; ++c) m = fmaxf(m, y[c]);  // NaN is left out
                });
            const bool plain = fabsf(m) <= 3.402823466e38f;  // neither +inf nor masked throughout
            const float below = plain ? m : 0.0f;
            each([&](int i, int j, const float* y) {
                float c[V];
                counts(i, j, c);
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float logit = fmaxf(y[v], minus_inf());  // NaN is masked
                    float s, kept;
                    if (soft) {
                        s = kept = plain ? exp_score<L>(logit - below) : exp_below(logit, m);
                    } else {  // t = 0 and s = 0 where masked
                        const float t = exp_score<L>(-fabsf(logit));
                        float r;
                        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + t));
                        const float tr = t * r;
                        s = logit < 0.0f ? tr : r;
                        kept = tr * r;
                    }
                    if constexpr (GRAD && E > 0) x[i * V + v] = kept;
                    z += s;
                    d = fmaf(s, c[v], d);
                }
            });
            mine = m;
            join(soft, m, z, d, joint);
            const bool low = on && !soft && z < 0x1p-100f;
            if (!(TEAM <= 32 ? __any_sync(kAll, low) : low)) break;
            if constexpr (TEAM > 32) __syncthreads();  // joint is written again
            soft |= low;
        }
        const float mean = z > 0.0f ? __fdiv_rn(d, z) : 0.0f;
        if constexpr (GRAD) {
            if (on) {
                const float gz = z > 0.0f ? __fdiv_rn(g, z) * (soft ? exp_below(mine, m) : 1.0f) : 0.0f, gm = -gz * mean;
                const auto write = [&](int i, int j, const float* kept) {
                    float c[V], y[V];
                    counts(i, j, c);
                    if (add != nullptr) {
                        if constexpr (EARLY) {
                            unpack(adds + i * W, y);
                        } else {
                            uint32_t w[W];
                            get(add, j, w, 0u);
                            unpack(w, y);
                        }
                    } else {
#pragma unroll
                        for (int v = 0; v < V; ++v) y[v] = 0.0f;
                    }
#pragma unroll
                    for (int v = 0; v < V; ++v) y[v] = fmaf(kept[v], fmaf(gz, c[v], gm), y[v]);
                    put(out, j, y);
                };
                if constexpr (E > 0) {
#pragma unroll
                    for (int i = 0; i < R / V; ++i) write(i, column(i), x + i * V);
                } else {
                    for (int i = 0; column(i) < n; ++i) {
                        uint32_t w[W];
                        float y[V];
                        get(row, column(i), w, kNone);
                        unpack(w, y);
#pragma unroll
                        for (int v = 0; v < V; ++v) {
                            const float logit = fmaxf(y[v], minus_inf());
                            if (soft) {
                                y[v] = exp_below(logit, mine);
                            } else {
                                const float t = exp_score<L>(-fabsf(logit)), r = __frcp_rn(1.0f + t);
                                y[v] = t * r * r;
                            }
                        }
                        write(i, column(i), y);
                    }
                }
            }
        }
        return z > 0.0f ? fmaf(unit, mean, 1.0f) : 0.0f;
    }
};

// A sequence's factors: the mean of its counts, its inverse, and what its gradient is multiplied by.
struct Factors {
    float centre, unit, g;
};
__device__ __forceinline__ Factors factors_of(const BalanceArgs& a, int64_t s, int64_t length, int total) {
    Factors f{0.0f, 0.0f, 0.0f};
    if (total > 0 && length > 0) {
        const double per = (double)a.n / total;
        f.centre = (float)(1.0 / per);
        f.unit = (float)per;
        if (a.dlogits != nullptr) f.g = (float)((double)a.scale * per / (double)length) * (a.dloss ? __ldg(a.dloss + s) : 1.0f);
    }
    return f;
}

// The counts from column j on less their mean, from memory that this launch only reads.
template <int V>
__device__ __forceinline__ void centred(const int32_t* counts, int n, bool whole, float centre, int j, float* c) {
    if (V >= 4 && whole && j + V <= n) {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const int4 v = __ldg(reinterpret_cast<const int4*>(counts + j + i));
            c[i] = (float)v.x - centre;
            c[(i + 1) % V] = (float)v.y - centre;
            c[(i + 2) % V] = (float)v.z - centre;
            c[(i + 3) % V] = (float)v.w - centre;
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) c[i] = j + i < n ? (float)__ldg(counts + j + i) - centre : 0.0f;
    }
}

// Blocks an SM that the registers are bounded for.
constexpr int rows_blocks(int team, int e) { return team <= 128 ? (team <= 32 && e >= 32 ? 6 : 8) : team == 256 ? 4 : 2; }

// A team takes a run of consecutive tokens; rows of the next token are on their way while a warp works on one.
template <int TEAM, int E, bool VEC, bool GRAD, typename L>
__global__ void __launch_bounds__(TEAM <= 32 ? 128 : TEAM, rows_blocks(TEAM, E)) balance_rows_kernel(const BalanceArgs a) {
    using R = Row<TEAM, E, VEC, L>;
    constexpr int NT = TEAM <= 32 ? 128 : TEAM, TEAMS = NT / TEAM, V = R::V;
    constexpr bool KEPT = TEAM <= 32 && E <= 16;          // the sequence's counts stay in registers
    constexpr bool AHEAD = TEAM <= 32 && R::RAW <= 8;     // the next row is loaded early
    __shared__ float joint[2][3][R::WARPS];
    grid_dependency_wait();
    grid_launch_dependents();
    const R r(a, threadIdx.x % TEAM);
    const int64_t team = (int64_t)blockIdx.x * TEAMS + threadIdx.x / TEAM, first = team * a.rows;
    const bool whole = reinterpret_cast<uintptr_t>(a.counts) % 16 == 0 && a.n % 4 == 0;
    Sequence q{-1, 0, 0};
    Factors f{0.0f, 0.0f, 0.0f};
    float sum = 0.0f;
    float kept[KEPT ? R::R : 1];
    uint32_t raw[R::RAW], next[AHEAD ? R::RAW : 1];
    const auto row_of = [&](int64_t t) { return static_cast<const L*>(a.logits) + (t < a.tokens ? t : 0) * a.row_stride; };
    if constexpr (AHEAD) r.get_all(row_of(first), first < a.tokens, next, R::kNone);
    for (int64_t i = 0; i < a.rows; ++i) {
        const int64_t t = first + i;
        const bool on = t < a.tokens;
        if (TEAM >= 32 && !on) break;  // lanes of a warp that hold several teams stay together
        if constexpr (AHEAD) {
#pragma unroll
            for (int w = 0; w < R::RAW; ++w) raw[w] = next[w];
            r.get_all(row_of(t + 1), i + 1 < a.rows && t + 1 < a.tokens, next, R::kNone);
        } else if constexpr (E > 0) {
            r.get_all(row_of(t), on, raw, R::kNone);
        }
        if (on && (t < q.begin || t >= q.end)) {
            if (q.s >= 0 && r.tid == 0) a.parts[team + q.s] = sum;
            sum = 0.0f;
            q = sequence_of(a.offsets, a.sequences, a.tokens, t);
            f = q.s >= 0 ? factors_of(a, q.s, q.end - q.begin, __ldg(a.totals + q.s)) : Factors{0.0f, 0.0f, 0.0f};
            if constexpr (KEPT) {
#pragma unroll
                for (int e = 0; e < R::R; e += V) {
                    if (q.s >= 0) {
                        centred<V>(a.counts + q.s * a.n, a.n, whole, f.centre, r.column(e / V), kept + e);
                    } else {
#pragma unroll
                        for (int c = 0; c < V; ++c) kept[e + c] = 0.0f;
                    }
                }
            }
        }
        __syncwarp();
        const int32_t* from = q.s >= 0 ? a.counts + q.s * a.n : nullptr;
        const auto counts = [&](int access, int j, float* c) {
            if constexpr (KEPT) {
#pragma unroll
                for (int v = 0; v < V; ++v) c[v] = kept[access * V + v];
            } else if (from != nullptr) {
                centred<V>(from, a.n, whole, f.centre, j, c);
            } else {
#pragma unroll
                for (int v = 0; v < V; ++v) c[v] = 0.0f;
            }
        };
        L* out = GRAD ? static_cast<L*>(a.dlogits) + t * a.dlogits_stride : nullptr;
        const L* add = GRAD && a.add != nullptr ? static_cast<const L*>(a.add) + t * a.add_stride : nullptr;
        sum += r.template pass<GRAD>(row_of(t), raw, on, counts, f.unit, f.g, out, add, joint[t & 1]);
    }
    if (q.s >= 0 && r.tid == 0) a.parts[team + q.s] = sum;
}

// A sequence's loss out of its parts: those of the teams that met it lie side by side.
__global__ void __launch_bounds__(kCountThreads) balance_loss_kernel(const BalanceArgs a) {
    __shared__ double sums[kCountThreads / 32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t s = blockIdx.x;
    int64_t begin = 0, end = a.tokens;
    if (a.offsets != nullptr) {
        begin = max((int64_t)__ldg(a.offsets + s), (int64_t)0);
        end = min((int64_t)__ldg(a.offsets + s + 1), a.tokens);
    }
    const bool any = end > begin && a.totals[s] > 0;
    double sum = 0.0;
    if (any)
        for (int64_t p = begin / a.rows + s + threadIdx.x; p <= (end - 1) / a.rows + s; p += kCountThreads) sum += a.parts[p];
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = sum;
    __syncthreads();
    if (threadIdx.x == 0) {
        double all = 0.0;
        for (int w = 0; w < kCountThreads / 32; ++w) all += sums[w];
        a.loss[s] = any ? (float)(a.scale * all / (double)(end - begin)) : 0.0f;
    }
}

struct Team {
    const void* fn;
    int threads, teams;
};

// Without the gradient a row need not stay in registers, and a block reads it at the pace of memory. Teams as in
// the routing's gradient.
template <bool VEC, bool GRAD, typename L>
Team rows_kernel(int n) {
    if (n <= 32) return {(const void*)balance_rows_kernel<4, 8, VEC, GRAD, L>, 128, 32};
    if (n <= 64) return {(const void*)balance_rows_kernel<8, 8, VEC, GRAD, L>, 128, 16};
    if (n <= 128) return {(const void*)balance_rows_kernel<16, 8, VEC, GRAD, L>, 128, 8};
    if (n <= 256) return {(const void*)balance_rows_kernel<32, 8, VEC, GRAD, L>, 128, 4};
    if (n <= 512) return {(const void*)balance_rows_kernel<32, 16, VEC, GRAD, L>, 128, 4};
    if (n <= 1024) return {(const void*)balance_rows_kernel<32, 32, VEC, GRAD, L>, 128, 4};
    if (n <= 2048) return {(const void*)balance_rows_kernel<128, 16, VEC, GRAD, L>, 128, 1};
    if (n <= 4096) return {(const void*)balance_rows_kernel<128, 32, VEC, GRAD, L>, 128, 1};
    if (n <= 6144) return {(const void*)balance_rows_kernel<128, 48, VEC, GRAD, L>, 128, 1};
    if (n <= 8192) return {(const void*)balance_rows_kernel<256, 32, VEC, GRAD, L>, 256, 1};
    if (n <= 16384) return {(const void*)balance_rows_kernel<512, 32, VEC, GRAD, L>, 512, 1};
    return {(const void*)balance_rows_kernel<512, 0, VEC, GRAD, L>, 512, 1};
}
template <typename L>
Team rows_kernel(int n, bool vec, bool grad) {
    return vec ? (grad ? rows_kernel<true, true, L>(n) : rows_kernel<true, false, L>(n))
               : (grad ? rows_kernel<false, true, L>(n) : rows_kernel<false, false, L>(n));
}

}  // namespace

int64_t balance_workspace(int64_t sequences) { return 4 * ((sequences + 63) / 64 * 64 + kBalanceTeams + sequences); }

int launch_balance(const BalanceArgs& a0, cudaStream_t stream) {
    BalanceArgs a = a0;
    a.totals = static_cast<int32_t*>(a.workspace);
    a.parts = reinterpret_cast<float*>(a.totals + (a.sequences + 63) / 64 * 64);
    const size_t es = a.logit_bf16 ? 2 : 4;
    const auto whole = [&](const void* p, int64_t stride) {
        return p == nullptr || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride * es % 16 == 0);
    };
    const bool vec = whole(a.logits, a.row_stride) && whole(a.dlogits, a.dlogits_stride) && whole(a.add, a.add_stride), grad = a.dlogits != nullptr;
    const Team team = a.logit_bf16 ? rows_kernel<uint16_t>(a.n, vec, grad) : rows_kernel<float>(a.n, vec, grad);
    const int64_t sms = sm_count();
    if (a.sequences > 0) {
        const int64_t zeros = std::min<int64_t>((a.sequences * a.n + 4 * kCountThreads - 1) / (4 * kCountThreads), 8 * sms);
        void* args[] = {&a};
        int rc = launch_pdl_raw((const void*)balance_zero_kernel, dim3((unsigned)zeros), dim3(kCountThreads), 0, stream, args);
        if (rc != 0) return rc;
    }
    if (a.sequences > 0 && a.tokens > 0) {
        const int64_t entries = a.tokens * a.k;
        int64_t blocks = std::min<int64_t>(std::min<int64_t>((entries + 4 * kCountThreads - 1) / (4 * kCountThreads), 4 * sms), a.tokens);
        int64_t run = (a.tokens + blocks - 1) / blocks;
        blocks = (a.tokens + run - 1) / run;
        const bool local = a.n <= kCountBins && entries >= 2 * a.n * (blocks + a.sequences);
        void* args[] = {&a, &run};
        const int rc = launch_pdl_raw(local ? (const void*)balance_count_kernel<true> : (const void*)balance_count_kernel<false>,
                                      dim3((unsigned)blocks), dim3(kCountThreads), 0, stream, args);
        if (rc != 0) return rc;
    }
    a.rows = 1;
    if (a.tokens > 0) {
        // runs that fill the GPU once
        const int64_t most = std::min<int64_t>(kBalanceTeams, sms * std::max(1, blocks_per_sm(team.fn, team.threads, 0)) * team.teams);
        a.rows = (a.tokens + most - 1) / most;
        const int64_t teams = (a.tokens + a.rows - 1) / a.rows;
        void* args[] = {&a};
        const int rc = launch_pdl_raw(team.fn, dim3((unsigned)((teams + team.teams - 1) / team.teams)), dim3(team.threads), 0, stream, args);
        if (rc != 0) return rc;
    }
    if (a.sequences == 0) return 0;
    void* args[] = {&a};
    return launch_pdl_raw((const void*)balance_loss_kernel, dim3((unsigned)a.sequences), dim3(kCountThreads), 0, stream, args);
}

cudaError_t balance_status(void** word) { return cudaGetSymbolAddress(word, g_balance_status); }

}  // namespace sdm
