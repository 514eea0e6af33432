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
    int s, begin, end;
};
__device__ __forceinline__ Sequence sequence_at(const BalanceArgs& a, int beyond) {  // `beyond`: the first offset beyond the token
    const int begin = beyond > 0 ? __ldg(a.offsets + beyond - 1) : 0, end = beyond <= a.sequences ? __ldg(a.offsets + beyond) : a.tokens;
    return {beyond > 0 && beyond <= a.sequences ? beyond - 1 : -1, begin, min(end, a.tokens)};
}
__device__ __forceinline__ Sequence sequence_of(const BalanceArgs& a, int t) {
    if (a.offsets == nullptr) return {0, 0, a.tokens};
    int lo = 0, hi = a.sequences + 1;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(a.offsets + mid) > t)
            hi = mid;
        else
            lo = mid + 1;
    }
    return sequence_at(a, lo);
}
// The same by a whole warp, 32 offsets at a time.
__device__ __forceinline__ Sequence warp_sequence_of(const BalanceArgs& a, int t) {
    if (a.offsets == nullptr) return {0, 0, a.tokens};
    const int lane = threadIdx.x & 31;
    int lo = 0, len = a.sequences + 1;  // the answer is in [lo, lo + len]
    while (len > 0) {
        const int step = (len + 31) / 32, at = min((lane + 1) * step, len) - 1;  // the last of each of 32 shares
        const int shares = __popc(__ballot_sync(kAll, __ldg(a.offsets + lo + at) <= t));
        const int skip = min(shares * step, len);
        lo += skip;
        len = shares == 32 ? 0 : min(step, len - skip) - 1;  // the last of the share is beyond t
    }
    return sequence_at(a, lo);
}

__global__ void __launch_bounds__(kCountThreads) balance_zero_kernel(const BalanceArgs a) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t all = (int64_t)a.sequences * a.n, step = (int64_t)gridDim.x * kCountThreads;
    for (int64_t i = (int64_t)blockIdx.x * kCountThreads + threadIdx.x; i < all; i += step) a.counts[i] = 0;
    for (int64_t i = (int64_t)blockIdx.x * kCountThreads + threadIdx.x; i < a.sequences; i += step) a.totals[i] = 0;
}

// The columns of N entries e, e + step, ... below `end`, or -1: of weight 0, or an index outside the row (flagged). Their
// loads are on their way together.
template <int N>
__device__ __forceinline__ void counted_columns(const BalanceArgs& a, uint32_t e, uint32_t step, uint32_t end, int* column) {
    int64_t j[N];
    float w[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint32_t at = e + i * step;
        j[i] = -1;
        w[i] = 1.0f;
        if (at < end) {
            j[i] = a.idx64 ? __ldg(static_cast<const int64_t*>(a.idx) + at) : __ldg(static_cast<const int32_t*>(a.idx) + at);
            if (a.w != nullptr) w[i] = __ldg(a.w + at);
            if (a.base != nullptr) {
                const uint32_t t = at / (uint32_t)a.k;
                j[i] -= a.idx64 ? __ldg(static_cast<const int64_t*>(a.base) + t) : __ldg(static_cast<const int32_t*>(a.base) + t);
            }
        }
    }
    bool outside = false;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const bool in = j[i] >= 0 && j[i] < a.n;
        outside |= !in && e + i * step < end;
        column[i] = in && w[i] != 0.0f ? (int)j[i] : -1;
    }
    if (outside) atomicOr(&g_balance_status, SDM_DEV_BAD_INDEX);
}

// Each block counts the entries of a run of tokens. LOCAL: in shared memory, one sequence of the run after the
// other, so that few entries of a short row do not queue up at the same words of L2.
template <bool LOCAL>
__global__ void __launch_bounds__(kCountThreads) balance_count_kernel(const BalanceArgs a, int run) {
    __shared__ int bins[LOCAL ? kCountBins : 1];
    __shared__ int all;
    constexpr int N = 4;
    grid_dependency_wait();
    grid_launch_dependents();
    const int first = blockIdx.x * run, last = min(first + run, a.tokens), tid = threadIdx.x;
    if constexpr (LOCAL) {
        for (int t = first; t < last;) {
            const Sequence q = warp_sequence_of(a, t);
            const int end = max(t + 1, min(q.end, last));
            if (q.s >= 0) {
                for (int j = tid; j < a.n; j += kCountThreads) bins[j] = 0;
                if (tid == 0) all = 0;
                __syncthreads();
                int mine = 0;
                const uint32_t until = (uint32_t)end * a.k;
                for (uint32_t e = (uint32_t)t * a.k + tid; e < until; e += N * kCountThreads) {
                    int column[N];
                    counted_columns<N>(a, e, kCountThreads, until, column);
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        if (column[i] >= 0) {
                            atomicAdd(&bins[column[i]], 1);
                            ++mine;
                        }
                    }
                }
                mine = __reduce_add_sync(kAll, mine);
                if ((tid & 31) == 0 && mine) atomicAdd(&all, mine);
                __syncthreads();
                for (int j = tid; j < a.n; j += kCountThreads)
                    if (bins[j]) atomicAdd(a.counts + (int64_t)q.s * a.n + j, bins[j]);
                if (tid == 0 && all) atomicAdd(a.totals + q.s, all);
                __syncthreads();
            }
            t = end;
        }
    } else {
        const uint32_t from = (uint32_t)first * a.k, to = (uint32_t)last * a.k;
        for (uint32_t e0 = from; e0 < to; e0 += kCountThreads) {  // whole warps stay together
            const uint32_t e = e0 + tid;
            int s = -1, column = -1;
            if (e < to) {
                s = sequence_of(a, (int)(e / (uint32_t)a.k)).s;
                if (s >= 0) counted_columns<1>(a, e, 0, to, &column);
                if (column >= 0)
                    atomicAdd(a.counts + (int64_t)s * a.n + column, 1);
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

// A token's row for a team of TEAM threads (lanes of a warp, or a block). VEC: 16 bytes an access, for rows that start
// on 16-byte boundaries; else 4. An access holds V consecutive entries, thread tid has those from (i * TEAM + tid) * V on.
// Lanes of a warp keep the row in registers, E logits each, a block in shared memory (each thread what is its own).
template <int TEAM, int E, bool VEC, typename L>
struct Row {
    static constexpr int V = (VEC ? 16 : 4) / sizeof(L), W = V * sizeof(L) / 4, WARPS = TEAM <= 32 ? 1 : TEAM / 32;
    static constexpr int RAW = E / V * W;  // words of a lane's share

    int n, tid;
    bool words;  // 4-byte accesses of two bf16 are aligned

    __device__ __forceinline__ Row(const BalanceArgs& a, int tid_) : n(a.n), tid(tid_) {
        words = VEC || V == 1 ||
                ((reinterpret_cast<uintptr_t>(a.logits) | reinterpret_cast<uintptr_t>(a.dlogits) | reinterpret_cast<uintptr_t>(a.add)) % 4 == 0 &&
                 ((a.row_stride | (a.dlogits ? a.dlogits_stride : 0) | (a.add ? a.add_stride : 0)) * sizeof(L)) % 4 == 0);
    }
    __device__ __forceinline__ int column(int i) const { return (i * TEAM + tid) * V; }  // of access i

    // the V entries from j on as they lie in memory; behind the end of the row, `fill` (the bits of an entry)
    __device__ __forceinline__ void get_inside(const L* row, int j, uint32_t* w) const {
        if constexpr (VEC) {
            const uint4 v = *reinterpret_cast<const uint4*>(row + j);
            w[0] = v.x, w[1] = v.y, w[2] = v.z, w[W - 1] = v.w;
        } else {
            w[0] = *reinterpret_cast<const uint32_t*>(row + j);
        }
    }
    __device__ __forceinline__ void get(const L* row, int j, uint32_t* w, uint32_t fill) const {
        if (words && j + V <= n) {
            get_inside(row, j, w);
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
    __device__ __forceinline__ void put_inside(L* row, int j, const float* d) const {
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
    }
    __device__ __forceinline__ void put(L* row, int j, const float* d) const {
        if (words && j + V <= n) {
            put_inside(row, j, d);
        } else {
#pragma unroll
            for (int c = 0; c < V; ++c)
                if (j + c < n) row[j + c] = from_f32<L>(d[c]);
        }
    }

    // Of N logits: their scores, those of a softmax relative to m, added to z and, times their counts, to d; `kept` is what
    // the gradient takes of each: the score, times what a sigmoid leaves to one.
    template <int N>
    static __device__ __forceinline__ void soft_scores(const float* y, float m, const float* c, float* kept, float& z, float& d) {
        if (fabsf(m) <= 3.402823466e38f) {
#pragma unroll
            for (int v = 0; v < N; ++v) kept[v] = exp_score<L>(fmaxf(y[v], minus_inf()) - m);  // NaN is masked
        } else {  // +inf, or masked throughout
#pragma unroll
            for (int v = 0; v < N; ++v) kept[v] = exp_below(y[v], m);
        }
#pragma unroll
        for (int v = 0; v < N; ++v) {
            z += kept[v];
            d = fmaf(kept[v], c[v], d);
        }
    }
    template <int N>
    static __device__ __forceinline__ void sigmoid_scores(const float* y, const float* c, float* kept, float& z, float& d) {
#pragma unroll
        for (int v = 0; v < N; ++v) {
            const float logit = fmaxf(y[v], minus_inf()), t = exp_score<L>(-fabsf(logit));  // t = 0 and s = 0 where masked
            float r;
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + t));  // 1 ulp
            const float tr = t * r, s = logit < 0.0f ? tr : r;
            kept[v] = tr * r;
            z += s;
            d = fmaf(s, c[v], d);
        }
    }
    // The gradient of N logits, from what was kept of them.
    template <int N>
    static __device__ __forceinline__ void gradient(float* kept, const float* c, float gz, float gm, const float* add) {
#pragma unroll
        for (int v = 0; v < N; ++v) kept[v] = fmaf(kept[v], fmaf(gz, c[v], gm), add[v]);
    }
};

// 1 / z of a sum of scores, which is at least 2^-60 or 0 (1 ulp).
__device__ __forceinline__ float inverse_of(float z) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(z));
    return z > 0.0f ? r : 0.0f;
}

// Sums of sigmoid scores below this lose bits; the row's shares are then those of exp(x), as for a softmax.
constexpr float kLowScores = 0x1p-60f;

// A sequence's factors: the mean of its counts, its inverse, and what its gradient is multiplied by.
struct Factors {
    float centre, unit, g;
};
__device__ __forceinline__ Factors factors_of(const BalanceArgs& a, int s, int length, int total) {
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

// What the tokens of a team's run share: the sequence that they are in, and the sum of their parts of its loss.
struct Run {
    Sequence q{-1, 0, 0};
    Factors f{0.0f, 0.0f, 0.0f};
    float sum = 0.0f;

    // Token t is next; true where another sequence begins.
    __device__ __forceinline__ bool next(const BalanceArgs& a, int t, int team, bool writes) {
        if (t >= q.begin && t < q.end) return false;
        done(a, team, writes);
        sum = 0.0f;
        q = sequence_of(a, t);
        f = q.s >= 0 ? factors_of(a, q.s, q.end - q.begin, __ldg(a.totals + q.s)) : Factors{0.0f, 0.0f, 0.0f};
        return true;
    }
    __device__ __forceinline__ void done(const BalanceArgs& a, int team, bool writes) const {
        if (q.s >= 0 && writes) a.parts[team + q.s] = sum;
    }
};

// Rows of up to 512 entries: TEAM lanes a row, E logits each. The next token's row is on its way while a warp
// works on one, and the counts of the sequence stay in registers. Half as many lanes with twice the logits spend less on
// what a row costs whatever its length: 65536 rows of 256 bf16 with the gradient, 16 lanes TIME16 us, 32 lanes 33.
template <int TEAM, int E, bool VEC, bool GRAD, typename L>
__global__ void __launch_bounds__(128, 5) balance_lanes_kernel(const BalanceArgs a) {
    using R = Row<TEAM, E, VEC, L>;
    constexpr int TEAMS = 128 / TEAM, V = R::V, ACCESSES = E / V;
    constexpr bool AHEAD = R::RAW <= 8;
    grid_dependency_wait();
    grid_launch_dependents();
    const R r(a, threadIdx.x % TEAM);
    const int team = blockIdx.x * TEAMS + threadIdx.x / TEAM, first = (int)min((int64_t)team * a.rows, (int64_t)a.tokens);
    const int count = min(a.rows, a.tokens - first), steps = __reduce_max_sync(kAll, count);
    const bool whole = reinterpret_cast<uintptr_t>(a.counts) % 16 == 0 && a.n % 4 == 0, softmax = a.score == SDM_SOFTMAX;
    Run run;
    float counts[E];
#pragma unroll
    for (int e = 0; e < E; ++e) counts[e] = 0.0f;
    uint32_t raw[R::RAW], next[AHEAD ? R::RAW : 1];
    const auto get_all = [&](const L* row, bool on, uint32_t* w, uint32_t fill) {
#pragma unroll
        for (int i = 0; i < ACCESSES; ++i) r.get(row, on ? r.column(i) : r.n, w + i * R::W, fill);
    };
    const L *row = static_cast<const L*>(a.logits) + first * a.row_stride, *add = static_cast<const L*>(a.add) + (a.add ? first * a.add_stride : 0);
    L* out = static_cast<L*>(a.dlogits) + (GRAD ? first * a.dlogits_stride : 0);
    if constexpr (AHEAD) get_all(row, count > 0, next, R::kNone);
    for (int i = 0; i < steps; ++i) {  // lanes of a warp that hold several teams stay together
        const bool on = i < count;
        if constexpr (AHEAD) {
#pragma unroll
            for (int w = 0; w < R::RAW; ++w) raw[w] = next[w];
            get_all(row + a.row_stride, i + 1 < count, next, R::kNone);
        } else {
            get_all(row, on, raw, R::kNone);
        }
        uint32_t adds[GRAD ? R::RAW : 1];
        if (GRAD && a.add != nullptr) get_all(add, on, adds, 0u);
        if (on && run.next(a, first + i, team, r.tid == 0)) {
#pragma unroll
            for (int e = 0; e < E; e += V) {
                if (run.q.s >= 0) {
                    centred<V>(a.counts + (int64_t)run.q.s * a.n, a.n, whole, run.f.centre, r.column(e / V), counts + e);
                } else {
#pragma unroll
                    for (int v = 0; v < V; ++v) counts[e + v] = 0.0f;
                }
            }
        }
        __syncwarp();
        float kept[E], z = 0.0f, d = 0.0f;
        // the shares of exp(x); every lane of the warp takes part, `mine` says whose team means it
        const auto soft = [&](bool mine) {
            float top = minus_inf(), zs = 0.0f, ds = 0.0f, y[V], e[V];
#pragma unroll
            for (int i2 = 0; i2 < ACCESSES; ++i2) {
                R::unpack(raw + i2 * R::W, y);
#pragma unroll
                for (int v = 0; v < V; ++v) top = fmaxf(top, y[v]);  // NaN is left out
            }
            top = warp_max<TEAM>(top);
#pragma unroll
            for (int i2 = 0; i2 < ACCESSES; ++i2) {
                R::unpack(raw + i2 * R::W, y);
                R::template soft_scores<V>(y, top, counts + i2 * V, e, zs, ds);
#pragma unroll
                for (int v = 0; v < V; ++v)
                    if (mine) kept[i2 * V + v] = e[v];
            }
            zs = warp_sum<TEAM>(zs);
            ds = warp_sum<TEAM>(ds);
            if (mine) z = zs, d = ds;
        };
        if (softmax) {
            soft(true);
        } else {
#pragma unroll
            for (int i2 = 0; i2 < ACCESSES; ++i2) {
                float y[V];
                R::unpack(raw + i2 * R::W, y);
                R::template sigmoid_scores<V>(y, counts + i2 * V, kept + i2 * V, z, d);
            }
            z = warp_sum<TEAM>(z);
            d = warp_sum<TEAM>(d);
            const bool low = on && z < kLowScores;
            if (__any_sync(kAll, low)) soft(low);
        }
        const float inverse = inverse_of(z), mean = d * inverse;
        if (z > 0.0f) run.sum += fmaf(run.f.unit, mean, 1.0f);
        if (GRAD && on) {
            const float gz = run.f.g * inverse, gm = -gz * mean;
#pragma unroll
            for (int i2 = 0; i2 < ACCESSES; ++i2) {
                float more[V];
#pragma unroll
                for (int v = 0; v < V; ++v) more[v] = 0.0f;
                if (a.add != nullptr) R::unpack(adds + i2 * R::W, more);
                R::template gradient<V>(kept + i2 * V, counts + i2 * V, gz, gm, more);
                r.put(out, r.column(i2), kept + i2 * V);
            }
            out += a.dlogits_stride;
            add += a.add_stride;
        }
        row += a.row_stride;
    }
    run.done(a, team, r.tid == 0);
}

// Longer rows: a block a row, 16 logits a thread at a time. What the loss alone needs is summed in one pass, relative
// to a maximum that grows. For the gradient the logits of a softmax, or what it takes of a sigmoid's, wait in shared
// memory (STAGED), and with them the counts of the sequence (COUNTED), each thread's own; rows too long for that are read
// again.
template <int TEAM, bool VEC, bool GRAD, bool STAGED, bool COUNTED, typename L>
__global__ void __launch_bounds__(TEAM, 1024 / TEAM) balance_block_kernel(const BalanceArgs a) {
    using R = Row<TEAM, 0, VEC, L>;
    constexpr int V = R::V, N = 16, U = N / V;
    extern __shared__ float stage[];
    __shared__ float joints[2][3][R::WARPS];
    int half = 0;
    grid_dependency_wait();
    grid_launch_dependents();
    const R r(a, threadIdx.x);
    const int first = (int)min((int64_t)blockIdx.x * a.rows, (int64_t)a.tokens), last = first + min(a.rows, a.tokens - first);
    const bool whole = reinterpret_cast<uintptr_t>(a.counts) % 16 == 0 && a.n % 4 == 0, softmax = a.score == SDM_SOFTMAX;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, chunks = (a.n + TEAM * N - 1) / (TEAM * N), full = r.words ? a.n / (TEAM * N) : 0;
    float* kept_counts = stage + (STAGED ? (a.n + TEAM * V - 1) / (TEAM * V) * (TEAM * V) : 0);
    Run run;
    for (int t = first; t < last; ++t) {
        const bool begins = run.next(a, t, blockIdx.x, threadIdx.x == 0);
        const L* row = static_cast<const L*>(a.logits) + t * a.row_stride;
        const int32_t* from = run.q.s >= 0 ? a.counts + (int64_t)run.q.s * a.n : nullptr;
        // the N values of a chunk of a thread in shared memory, which ends with the row's last access
        const auto put_shared = [&](float* to, int chunk, const float* x) {
            to += chunk * N * TEAM + threadIdx.x;
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (chunk >= full && r.column(chunk * U + u) >= a.n) continue;
#pragma unroll
                for (int v = 0; v < V; ++v) to[(u * V + v) * TEAM] = x[u * V + v];
            }
        };
        const auto get_shared = [&](const float* at, int chunk, float* x, float fill) {
            at += chunk * N * TEAM + threadIdx.x;
            if (chunk < full) {
#pragma unroll
                for (int i = 0; i < N; ++i) x[i] = at[i * TEAM];
            } else {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const bool in = r.column(chunk * U + u) < a.n;
#pragma unroll
                    for (int v = 0; v < V; ++v) x[u * V + v] = in ? at[(u * V + v) * TEAM] : fill;
                }
            }
        };
        const auto load_counts = [&](int chunk, float* c) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (from != nullptr) {
                    centred<V>(from, a.n, whole, run.f.centre, r.column(chunk * U + u), c + u * V);
                } else {
#pragma unroll
                    for (int v = 0; v < V; ++v) c[u * V + v] = 0.0f;
                }
            }
        };
        if (COUNTED && begins) {
            for (int chunk = 0; chunk < chunks; ++chunk) {
                float c[N];
                load_counts(chunk, c);
                put_shared(kept_counts, chunk, c);
            }
        }
        const auto counts = [&](int chunk, float* c) {
            if constexpr (COUNTED)
                get_shared(kept_counts, chunk, c, 0.0f);
            else
                load_counts(chunk, c);
        };
        // the logits of a chunk (NaN as masked), or other values that lie like them
        const auto get = [&](const L* from_row, int chunk, float* x, uint32_t fill) {
            uint32_t w[U][R::W];
            if (chunk < full) {
#pragma unroll
                for (int u = 0; u < U; ++u) r.get_inside(from_row, r.column(chunk * U + u), w[u]);
            } else {
#pragma unroll
                for (int u = 0; u < U; ++u) r.get(from_row, r.column(chunk * U + u), w[u], fill);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) R::unpack(w[u], x + u * V);
        };
        float m = minus_inf(), z = 0.0f, d = 0.0f;
        bool soft = softmax;
        for (;;) {
            if (soft) {
#pragma unroll 2
                for (int chunk = 0; chunk < chunks; ++chunk) {
                    float x[N], c[N], top = m;
                    get(row, chunk, x, R::kNone);
                    counts(chunk, c);
                    if (STAGED) put_shared(stage, chunk, x);
#pragma unroll
                    for (int i = 0; i < N; ++i) top = fmaxf(top, x[i]);  // NaN is left out
                    if (top > m) {
                        const float scale = exp_below(m, top);
                        z *= scale;
                        d *= scale;
                        m = top;
                    }
                    R::template soft_scores<N>(x, m, c, x, z, d);
                }
                const float mine = m;
                m = warp_max(m);
                const float scale = exp_below(mine, m);
                z *= scale;
                d *= scale;
            } else {
#pragma unroll 2
                for (int chunk = 0; chunk < chunks; ++chunk) {
                    float x[N], c[N];
                    get(row, chunk, x, R::kNone);
                    counts(chunk, c);
                    R::template sigmoid_scores<N>(x, c, x, z, d);
                    if (STAGED && GRAD) put_shared(stage, chunk, x);
                }
            }
            z = warp_sum(z);
            d = warp_sum(d);
            float(*joint)[R::WARPS] = joints[half ^= 1];  // the other half may still be read
            if (lane == 0) {
                joint[0][warp] = m;
                joint[1][warp] = z;
                joint[2][warp] = d;
            }
            __syncthreads();
            const int w = lane % R::WARPS;  // every warp for itself
            const float theirs = joint[0][w];
            m = warp_max<R::WARPS>(theirs);
            const float scale = lane >= R::WARPS ? 0.0f : soft ? exp_below(theirs, m) : 1.0f;
            z = warp_sum(joint[1][w] * scale);
            d = warp_sum(joint[2][w] * scale);
            if (soft || z >= kLowScores) break;
            soft = true;
            m = minus_inf();
            z = d = 0.0f;
        }
        const float inverse = inverse_of(z), mean = d * inverse;
        if (z > 0.0f) run.sum += fmaf(run.f.unit, mean, 1.0f);
        if constexpr (GRAD) {
            L* out = static_cast<L*>(a.dlogits) + t * a.dlogits_stride;
            const L* add = a.add != nullptr ? static_cast<const L*>(a.add) + t * a.add_stride : nullptr;
            const float gz = run.f.g * inverse, gm = -gz * mean;
            for (int chunk = 0; chunk < chunks; ++chunk) {
                float x[N], c[N], adds[N];
                counts(chunk, c);
                float unused = 0.0f;
                if constexpr (STAGED)
                    get_shared(stage, chunk, x, minus_inf());
                else
                    get(row, chunk, x, R::kNone);
                if (soft)
                    R::template soft_scores<N>(x, m, c, x, unused, unused);
                else if (!STAGED)
                    R::template sigmoid_scores<N>(x, c, x, unused, unused);
                if (add != nullptr) {
                    get(add, chunk, adds, 0u);
                } else {
#pragma unroll
                    for (int i = 0; i < N; ++i) adds[i] = 0.0f;
                }
                R::template gradient<N>(x, c, gz, gm, adds);
                if (chunk < full) {
#pragma unroll
                    for (int u = 0; u < U; ++u) r.put_inside(out, r.column(chunk * U + u), x + u * V);
                } else {
#pragma unroll
                    for (int u = 0; u < U; ++u) r.put(out, r.column(chunk * U + u), x + u * V);
                }
            }
        }
    }
    run.done(a, blockIdx.x, threadIdx.x == 0);
}

// A sequence's loss out of its parts: those of the teams that met it lie side by side.
__global__ void __launch_bounds__(kCountThreads) balance_loss_kernel(const BalanceArgs a) {
    __shared__ double sums[kCountThreads / 32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int s = blockIdx.x;
    int begin = 0, end = a.tokens;
    if (a.offsets != nullptr) {
        begin = max(__ldg(a.offsets + s), 0);
        end = min(__ldg(a.offsets + s + 1), a.tokens);
    }
    const bool any = end > begin && a.totals[s] > 0;
    double sum = 0.0;
    if (any)
        for (int p = begin / a.rows + s + threadIdx.x; p <= (end - 1) / a.rows + s; p += kCountThreads) sum += a.parts[p];
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
    size_t smem;
};

// Sixteen logits a lane up to 512 entries, in fewer lanes for shorter rows; then blocks of 128 to 512 threads. For the
// gradient they stage the counts up to 8192 entries, and rows up to 48 K.
constexpr int kStaged = 48 * 1024, kCounted = 8192;
template <int TEAM, bool VEC, bool GRAD, typename L>
Team block_team(int n) {
    constexpr int V = (VEC ? 16 : 4) / sizeof(L);
    const size_t smem = (size_t)(n + TEAM * V - 1) / (TEAM * V) * (TEAM * V) * sizeof(float);
    if constexpr (!GRAD) {
        return {(const void*)balance_block_kernel<TEAM, VEC, false, false, false, L>, TEAM, 1, 0};
    } else if constexpr (TEAM < 512) {  // rows of at most kCounted entries
        return {(const void*)balance_block_kernel<TEAM, VEC, true, true, true, L>, TEAM, 1, 2 * smem};
    } else {
        if (n <= kStaged) return {(const void*)balance_block_kernel<TEAM, VEC, true, true, false, L>, TEAM, 1, smem};
        return {(const void*)balance_block_kernel<TEAM, VEC, true, false, false, L>, TEAM, 1, 0};
    }
}
template <bool VEC, bool GRAD, typename L>
Team rows_team(int n) {
    if (n <= 32) return {(const void*)balance_lanes_kernel<2, 16, VEC, GRAD, L>, 128, 64, 0};
    if (n <= 64) return {(const void*)balance_lanes_kernel<4, 16, VEC, GRAD, L>, 128, 32, 0};
    if (n <= 128) return {(const void*)balance_lanes_kernel<8, 16, VEC, GRAD, L>, 128, 16, 0};
    if (n <= 256) return {(const void*)balance_lanes_kernel<16, 16, VEC, GRAD, L>, 128, 8, 0};
    if (n <= 512) return {(const void*)balance_lanes_kernel<32, 16, VEC, GRAD, L>, 128, 4, 0};
    if (n <= 2048) return block_team<128, VEC, GRAD, L>(n);
    return n <= kCounted ? block_team<256, VEC, GRAD, L>(n) : block_team<512, VEC, GRAD, L>(n);
}
template <typename L>
Team rows_team(int n, bool vec, bool grad) {
    return vec ? (grad ? rows_team<true, true, L>(n) : rows_team<true, false, L>(n)) : (grad ? rows_team<false, true, L>(n) : rows_team<false, false, L>(n));
}

}  // namespace

int64_t balance_workspace(int64_t sequences) { return 4 * ((sequences + 63) / 64 * 64 + kBalanceTeams + sequences); }

int launch_balance(const BalanceArgs& a0, cudaStream_t stream) {
    BalanceArgs a = a0;
    a.totals = static_cast<int32_t*>(a.workspace);
    a.parts = reinterpret_cast<float*>(a.totals + ((int64_t)a.sequences + 63) / 64 * 64);
    const size_t es = a.logit_bf16 ? 2 : 4;
    const auto whole = [&](const void* p, int64_t stride) {
        return p == nullptr || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && stride * es % 16 == 0);
    };
    const bool vec = whole(a.logits, a.row_stride) && whole(a.dlogits, a.dlogits_stride) && whole(a.add, a.add_stride), grad = a.dlogits != nullptr;
    const Team team = a.logit_bf16 ? rows_team<uint16_t>(a.n, vec, grad) : rows_team<float>(a.n, vec, grad);
    const int sms = sm_count();
    if (a.sequences > 0) {
        const int64_t zeros = std::min<int64_t>(((int64_t)a.sequences * a.n + 4 * kCountThreads - 1) / (4 * kCountThreads), 8 * sms);
        void* args[] = {&a};
        int rc = launch_pdl_raw((const void*)balance_zero_kernel, dim3((unsigned)zeros), dim3(kCountThreads), 0, stream, args);
        if (rc != 0) return rc;
    }
    if (a.sequences > 0 && a.tokens > 0) {
        const int64_t entries = (int64_t)a.tokens * a.k;
        int blocks = (int)std::min<int64_t>(std::min<int64_t>((entries + 4 * kCountThreads - 1) / (4 * kCountThreads), 4 * sms), a.tokens);
        int run = (a.tokens + blocks - 1) / blocks;
        blocks = (a.tokens + run - 1) / run;
        const bool local = a.n <= kCountBins && entries >= (int64_t)2 * a.n * (blocks + a.sequences);
        void* args[] = {&a, &run};
        const int rc = launch_pdl_raw(local ? (const void*)balance_count_kernel<true> : (const void*)balance_count_kernel<false>,
                                      dim3(blocks), dim3(kCountThreads), 0, stream, args);
        if (rc != 0) return rc;
    }
    a.rows = 1;
    if (a.tokens > 0) {
        // runs that fill the GPU once
        int rc = allow_smem(team.fn, team.smem + 1024);  // and what the kernel has besides
        if (rc != 0) return rc;
        const int most = std::min(kBalanceTeams, sms * std::max(1, blocks_per_sm(team.fn, team.threads, team.smem)) * team.teams);
        a.rows = (a.tokens - 1) / most + 1;
        const int teams = (a.tokens - 1) / a.rows + 1;
        void* args[] = {&a};
        rc = launch_pdl_raw(team.fn, dim3((unsigned)((teams + team.teams - 1) / team.teams)), dim3(team.threads), team.smem, stream, args);
        if (rc != 0) return rc;
    }
    if (a.sequences == 0) return 0;
    void* args[] = {&a};
    return launch_pdl_raw((const void*)balance_loss_kernel, dim3((unsigned)a.sequences), dim3(kCountThreads), 0, stream, args);
}

cudaError_t balance_status(void** word) { return cudaGetSymbolAddress(word, g_balance_status); }

}  // namespace sdm
