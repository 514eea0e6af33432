// The balance loss over rows of logits, for balance.cu and the translation units that hold its kernels over rows of
// each type of logits.
#pragma once

#include <algorithm>
#include <type_traits>

#include "balance_internal.h"
#include "cluster_device.cuh"
#include "quant_device.cuh"
#include "score_device.cuh"
#include "sdm_internal.h"

namespace sdm {
namespace {

__device__ unsigned int g_balance_status;  // only kernels of balance.cu raise it

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

// exp(x - m) for x <= m is 2^((x - m) * log2(e)) by the hardware's 2^x, which is good for 2 ulp. Its argument is rounded
// twice, and log2(e) once: 2.5 steps of 2^-24 of the result for each unit of x - m. With expf in its place 1024 float32 rows
// of 16384 take 29 us for 26, and 4097 of 4099 with the gradient 64 for 60. (x * log2(e) - m * log2(e) in one operation is
// off by what m, not x - m, amounts to.)
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float exp2_of(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
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
    // the gradient takes of each: the score, times what a sigmoid leaves to one. Two at a time where the hardware has
    // one instruction for two.
    template <int N>
    static __device__ __forceinline__ void soft_scores(const float* y, float m, const float* c, float* kept, float& z, float& d) {
        if (fabsf(m) <= 3.402823466e38f) {
            if constexpr (N > 1) {
                f32x2 z2 = pair(0.0f, 0.0f), d2 = z2;
                const f32x2 log2e = pair(kLog2e, kLog2e), below = pair(-m, -m);
#pragma unroll
                for (int v = 0; v < N; v += 2) {
                    float a0, a1;
                    split(mul2(add2(pair(fmaxf(y[v], minus_inf()), fmaxf(y[v + 1], minus_inf())), below), log2e), a0, a1);  // NaN is masked
                    kept[v] = exp2_of(a0);
                    kept[v + 1] = exp2_of(a1);
                    const f32x2 s = pair(kept[v], kept[v + 1]);
                    z2 = add2(z2, s);
                    d2 = fma2(s, pair(c[v], c[v + 1]), d2);
                }
                add_pairs(z2, d2, z, d);
                return;
            }
            kept[0] = exp2_of((fmaxf(y[0], minus_inf()) - m) * kLog2e);
            z += kept[0];
            d = fmaf(kept[0], c[0], d);
            return;
        }
#pragma unroll
        for (int v = 0; v < N; ++v) {  // +inf, or masked throughout
            kept[v] = exp_below(y[v], m);
            z += kept[v];
            d = fmaf(kept[v], c[v], d);
        }
    }
    template <int N>
    static __device__ __forceinline__ void sigmoid_scores(const float* y, const float* c, float* kept, float& z, float& d) {
        // t = exp(-|x|), r = 1 / (1 + t): s is r or t * r, s * (1 - s) is t * r * r; t = 0 and s = 0 where masked
        const auto exponential = [](float logit) { return exp2_of(-fabsf(logit) * kLog2e); };
        const auto reciprocal = [](float x) {
            float r;
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));  // 1 ulp
            return r;
        };
        if constexpr (N > 1) {
            f32x2 z2 = pair(0.0f, 0.0f), d2 = z2;
#pragma unroll
            for (int v = 0; v < N; v += 2) {
                const float x0 = fmaxf(y[v], minus_inf()), x1 = fmaxf(y[v + 1], minus_inf());
                const f32x2 t = pair(exponential(x0), exponential(x1));
                float a0, a1, tr0, tr1;
                split(add2(t, pair(1.0f, 1.0f)), a0, a1);
                const float r0 = reciprocal(a0), r1 = reciprocal(a1);
                const f32x2 r = pair(r0, r1), tr = mul2(t, r);
                split(tr, tr0, tr1);
                split(mul2(tr, r), kept[v], kept[v + 1]);
                const f32x2 s = pair(x0 < 0.0f ? tr0 : r0, x1 < 0.0f ? tr1 : r1);
                z2 = add2(z2, s);
                d2 = fma2(s, pair(c[v], c[v + 1]), d2);
            }
            add_pairs(z2, d2, z, d);
        } else {
            const float x = fmaxf(y[0], minus_inf()), t = exponential(x), r = reciprocal(1.0f + t), tr = t * r, s = x < 0.0f ? tr : r;
            kept[0] = tr * r;
            z += s;
            d = fmaf(s, c[0], d);
        }
    }
    static __device__ __forceinline__ void add_pairs(f32x2 z2, f32x2 d2, float& z, float& d) {
        float z0, z1, d0, d1;
        split(z2, z0, z1);
        split(d2, d0, d1);
        z += z0 + z1;
        d += d0 + d1;
    }
    // The gradient of N logits, from what was kept of them.
    template <int N>
    static __device__ __forceinline__ void gradient(float* kept, const float* c, float gz, float gm, const float* add) {
        if constexpr (N > 1) {
            const f32x2 gz2 = pair(gz, gz), gm2 = pair(gm, gm);
#pragma unroll
            for (int v = 0; v < N; v += 2)
                split(fma2(pair(kept[v], kept[v + 1]), fma2(gz2, pair(c[v], c[v + 1]), gm2), pair(add[v], add[v + 1])), kept[v], kept[v + 1]);
        } else {
            kept[0] = fmaf(kept[0], fmaf(gz, c[0], gm), add[0]);
        }
    }
};

// 1 / z of a sum of scores, which is at least 2^-30 or 0 (1 ulp).
__device__ __forceinline__ float inverse_of(float z) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(z));
    return z > 0.0f ? r : 0.0f;
}

// Where a row's sigmoid scores sum to less than this, its shares are those of exp(x), as for a softmax: what the scores leave to
// one is one then, but for 2^-30, and scores that are 0 in float32 have their shares (above it, 0 is below 2^-96 of the sum).
constexpr float kLowScores = 0x1p-30f;

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
    float sum = 0.0f, lost = 0.0f;

    // A row's part. Parts that are nearly alike would all be rounded the same way as the sum grows, by 280 steps of 2^-24 of
    // it after 1850 rows, so what each addition loses goes into the next (Kahan).
    __device__ __forceinline__ void add(float part) {
        const float y = part - lost, t = sum + y;
        lost = (t - sum) - y;
        sum = t;
    }
    // Token t is next; true where another sequence begins.
    __device__ __forceinline__ bool next(const BalanceArgs& a, int t, int team, bool writes) {
        if (t >= q.begin && t < q.end) return false;
        done(a, team, writes);
        sum = lost = 0.0f;
        q = sequence_of(a, t);
        f = q.s >= 0 ? factors_of(a, q.s, q.end - q.begin, __ldg(a.totals + q.s)) : Factors{0.0f, 0.0f, 0.0f};
        return true;
    }
    __device__ __forceinline__ void done(const BalanceArgs& a, int team, bool writes) const {
        if (q.s >= 0 && writes) a.parts[team + q.s] = sum;
    }
};

// What a row adds to its sequence's loss, by TEAM lanes that hold it in `raw`, E logits each, and the counts less their
// mean in `counts`; GRAD: writes its gradient, to which `adds` is added. All lanes of the warp come here, `on` those
// that have a row.
template <bool GRAD, int TEAM, int E, bool VEC, typename L>
__device__ __forceinline__ float lanes_pass(const Row<TEAM, E, VEC, L>& r, const uint32_t* raw, const uint32_t* adds, const float* counts, bool on,
                                            bool softmax, const Factors& f, bool adding, L* out) {
    using R = Row<TEAM, E, VEC, L>;
    constexpr int V = R::V, ACCESSES = E / V;
    float kept[E], z = 0.0f, d = 0.0f;
    // the shares of exp(x); every lane of the warp takes part, `mine` says whose team means it
    const auto soft = [&](bool mine) {
        float top = minus_inf(), zs = 0.0f, ds = 0.0f, y[V], e[V];
#pragma unroll
        for (int i = 0; i < ACCESSES; ++i) {
            R::unpack(raw + i * R::W, y);
#pragma unroll
            for (int v = 0; v < V; ++v) top = fmaxf(top, y[v]);  // NaN is left out
        }
        top = warp_max<TEAM>(top);
#pragma unroll
        for (int i = 0; i < ACCESSES; ++i) {
            R::unpack(raw + i * R::W, y);
            R::template soft_scores<V>(y, top, counts + i * V, e, zs, ds);
#pragma unroll
            for (int v = 0; v < V; ++v)
                if (mine) kept[i * V + v] = e[v];
        }
        zs = warp_sum<TEAM>(zs);
        ds = warp_sum<TEAM>(ds);
        if (mine) z = zs, d = ds;
    };
    if (softmax) {
        soft(true);
    } else {
#pragma unroll
        for (int i = 0; i < ACCESSES; ++i) {
            float y[V];
            R::unpack(raw + i * R::W, y);
            R::template sigmoid_scores<V>(y, counts + i * V, kept + i * V, z, d);
        }
        z = warp_sum<TEAM>(z);
        d = warp_sum<TEAM>(d);
        const bool low = on && z < kLowScores;
        if (__any_sync(kAll, low)) soft(low);
    }
    const float inverse = inverse_of(z), mean = d * inverse;
    if (GRAD && on) {
        const float gz = f.g * inverse, gm = -gz * mean;
#pragma unroll
        for (int i = 0; i < ACCESSES; ++i) {
            float more[V];
#pragma unroll
            for (int v = 0; v < V; ++v) more[v] = 0.0f;
            if (adding) R::unpack(adds + i * R::W, more);
            R::template gradient<V>(kept + i * V, counts + i * V, gz, gm, more);
            r.put(out, r.column(i), kept + i * V);
        }
    }
    return z > 0.0f ? fmaf(f.unit, mean, 1.0f) : 0.0f;
}

// Rows of up to 512 entries: TEAM lanes a row, E logits each. The next token's row is on its way while a warp
// works on one, and the counts of the sequence stay in registers. Sixteen logits a lane spend less than eight on what a row
// costs whatever its length: a call with 65536 rows of 256 bf16 and the gradient takes 37 us, with eight 42. Its registers
// fit four blocks an SM; with five (43 us) some are spilled, three (39 us) hide less latency.
template <int TEAM, int E, bool VEC, bool GRAD, typename L>
__global__ void __launch_bounds__(128, 4) balance_lanes_kernel(const BalanceArgs a) {
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
        const float part = lanes_pass<GRAD>(r, raw, adds, counts, on, softmax, run.f, GRAD && a.add != nullptr, out);
        run.add(part);
        if (GRAD && on) {
            out += a.dlogits_stride;
            add += a.add_stride;
        }
        row += a.row_stride;
    }
    run.done(a, team, r.tid == 0);
}

// Few tokens: one launch, with a cluster of blocks for each sequence. Each of its blocks counts all of the sequence's
// entries in shared memory and goes over its share of the rows; the first has the counts and the loss. The last cluster, of a
// call with offsets, writes the rows of the tokens that are in no sequence. 64 rows of 256 bf16: 6.2 us, in four launches 8.0.
// (Float32 logits with the gradient spill 36 bytes a thread.)
constexpr int kSmallCluster = 8, kSmallThreads = 256, kSmallBins = 512;
template <int TEAM, bool GRAD, typename L>
__global__ void __launch_bounds__(kSmallThreads) balance_small_kernel(const BalanceArgs a) {
    using R = Row<TEAM, 16, false, L>;
    constexpr int TEAMS = kSmallThreads / TEAM, V = R::V, N = 4;
    __shared__ int bins[kSmallBins];
    __shared__ int total;
    __shared__ float sums[kSmallThreads / 32];
    __shared__ float sum_of_block;
    grid_dependency_wait();
    grid_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, s = blockIdx.x / kSmallCluster;
    const int block = (int)cluster_rank();
    const bool outside = s == a.sequences, softmax = a.score == SDM_SOFTMAX;
    // the cluster's tokens: begin .. end, or all but those
    int begin = 0, end = a.tokens;
    if (a.offsets != nullptr) {
        begin = min(max(__ldg(a.offsets + (outside ? 0 : s)), 0), a.tokens);
        end = min(max(__ldg(a.offsets + (outside ? s : s + 1)), begin), a.tokens);
    }
    const int rows = outside ? a.tokens - (end - begin) : end - begin;
    const R r(a, tid % TEAM);
    uint32_t raw[R::RAW], adds[GRAD ? R::RAW : 1];
    int64_t t = 0;
    bool on = false;
    const auto load = [&](int i) {  // row i of the cluster's
        on = i < rows;
        t = !on ? 0 : outside ? (i < begin ? i : end + i - begin) : begin + i;
#pragma unroll
        for (int x = 0; x < 16 / V; ++x) r.get(static_cast<const L*>(a.logits) + t * a.row_stride, on ? r.column(x) : r.n, raw + x * R::W, R::kNone);
        if (GRAD && a.add != nullptr) {
#pragma unroll
            for (int x = 0; x < 16 / V; ++x) r.get(static_cast<const L*>(a.add) + t * a.add_stride, on ? r.column(x) : r.n, adds + x * R::W, 0u);
        }
    };
    const int first = block * TEAMS + tid / TEAM;
    load(first);  // on its way while the entries are counted
    for (int j = tid; j < a.n; j += kSmallThreads) bins[j] = 0;
    if (tid == 0) total = 0;
    __syncthreads();
    int own = 0;
    const uint32_t until = outside ? 0u : (uint32_t)end * a.k;
    for (uint32_t e = (uint32_t)begin * a.k + tid; e < until; e += N * kSmallThreads) {
        int column[N];
        counted_columns<N>(a, e, kSmallThreads, until, column);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (column[i] >= 0) {
                atomicAdd(&bins[column[i]], 1);
                ++own;
            }
        }
    }
    own = __reduce_add_sync(kAll, own);
    if (lane == 0 && own) atomicAdd(&total, own);
    __syncthreads();
    Factors f{0.0f, 0.0f, 0.0f};
    if (!outside) {
        f = factors_of(a, s, end - begin, total);
        if (block == 0)
            for (int j = tid; j < a.n; j += kSmallThreads) a.counts[(int64_t)s * a.n + j] = bins[j];
    }
    float counts[16], sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 16 / V; ++i) {
#pragma unroll
        for (int v = 0; v < V; ++v) counts[i * V + v] = !outside && r.column(i) + v < a.n ? (float)bins[r.column(i) + v] - f.centre : 0.0f;
    }
    for (int i0 = first - tid / TEAM; i0 < rows; i0 += kSmallCluster * TEAMS) {
        const float part = lanes_pass<GRAD>(r, raw, adds, counts, on, softmax, f, GRAD && a.add != nullptr,
                                            GRAD ? static_cast<L*>(a.dlogits) + t * a.dlogits_stride : nullptr);
        if (r.tid == 0) sum += part;
        load(i0 + kSmallCluster * TEAMS + tid / TEAM);
    }
    sum = warp_sum(sum);
    if (lane == 0) sums[tid >> 5] = sum;
    __syncthreads();
    if (tid == 0) {
        sum = 0.0f;
        for (int w = 0; w < kSmallThreads / 32; ++w) sum += sums[w];
        sum_of_block = sum;
    }
    cluster_sync();
    if (block == 0 && tid == 0 && !outside) {
        double all = 0.0;
        for (uint32_t q = 0; q < kSmallCluster; ++q) all += __uint_as_float(cluster_load(cluster_address(&sum_of_block, q)));
        a.loss[s] = end > begin && total > 0 ? (float)(a.scale * all / (double)(end - begin)) : 0.0f;
    }
    cluster_sync();  // the sums are read
}

// Longer rows: a block a row, 8 logits a thread at a time. What the loss alone needs is summed in one pass, relative
// to a maximum that grows. For the gradient the logits of a softmax, or what it takes of a sigmoid's, wait in shared
// memory (STAGED), and with them the counts of the sequence (COUNTED), each thread's own; rows too long for that are read
// again (of float32 that start anywhere, 100 bytes a thread are spilled there). How many rows a block has follows from what
// fits an SM, with the gradient fewer than without, so that the two losses may differ in their last bit.
template <int TEAM, bool VEC, bool GRAD, bool STAGED, bool COUNTED, typename L>
__global__ void __launch_bounds__(TEAM, 1024 / TEAM) balance_block_kernel(const BalanceArgs a) {
    using R = Row<TEAM, 0, VEC, L>;
    constexpr int V = R::V, N = 8, U = N / V;
    extern __shared__ float stage[];
    __shared__ float joints[2][3][R::WARPS];
    int half = 0;
    grid_dependency_wait();
    grid_launch_dependents();
    const R r(a, threadIdx.x);
    const int first = (int)min((int64_t)blockIdx.x * a.rows, (int64_t)a.tokens), last = first + min(a.rows, a.tokens - first);
    const bool whole = reinterpret_cast<uintptr_t>(a.counts) % 16 == 0 && a.n % 4 == 0, softmax = a.score == SDM_SOFTMAX;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, full = r.words ? a.n / (TEAM * N) * U : 0;
    float* kept_counts = stage + (STAGED ? (a.n + TEAM * V - 1) / (TEAM * V) * (TEAM * V) : 0);
    Run run;
    for (int t = first; t < last; ++t) {
        const bool begins = run.next(a, t, blockIdx.x, threadIdx.x == 0);
        const L* row = static_cast<const L*>(a.logits) + t * a.row_stride;
        const int32_t* from = run.q.s >= 0 ? a.counts + (int64_t)run.q.s * a.n : nullptr;
        // f(accesses, first access) over this thread's share of the row: U accesses at a time as far as all threads
        // have them, then one by one
        const auto each = [&](const auto& f) {
#pragma unroll 2
            for (int i = 0; i < full; i += U) f(std::integral_constant<int, U>{}, i);
            for (int i = full; r.column(i) < a.n; ++i) f(std::integral_constant<int, 1>{}, i);
        };
        const auto get = [&](auto count, const L* from_row, int i, float* x, uint32_t fill) {
            constexpr int A = decltype(count)::value;
            uint32_t w[A][R::W];
#pragma unroll
            for (int u = 0; u < A; ++u) {
                if constexpr (A > 1)
                    r.get_inside(from_row, r.column(i + u), w[u]);
                else
                    r.get(from_row, r.column(i + u), w[u], fill);
            }
#pragma unroll
            for (int u = 0; u < A; ++u) R::unpack(w[u], x + u * V);
        };
        const auto put_shared = [&](auto count, float* to, int i, const float* x) {
#pragma unroll
            for (int v = 0; v < decltype(count)::value * V; ++v) to[(i * V + v) * TEAM + threadIdx.x] = x[v];
        };
        const auto get_shared = [&](auto count, const float* at, int i, float* x) {
#pragma unroll
            for (int v = 0; v < decltype(count)::value * V; ++v) x[v] = at[(i * V + v) * TEAM + threadIdx.x];
        };
        const auto load_counts = [&](auto count, int i, float* c) {
#pragma unroll
            for (int u = 0; u < decltype(count)::value; ++u) {
                if (from != nullptr) {
                    centred<V>(from, a.n, whole, run.f.centre, r.column(i + u), c + u * V);
                } else {
#pragma unroll
                    for (int v = 0; v < V; ++v) c[u * V + v] = 0.0f;
                }
            }
        };
        if (COUNTED && begins)
            each([&](auto count, int i) {
                float c[decltype(count)::value * V];
                load_counts(count, i, c);
                put_shared(count, kept_counts, i, c);
            });
        const auto counts = [&](auto count, int i, float* c) {
            if constexpr (COUNTED)
                get_shared(count, kept_counts, i, c);
            else
                load_counts(count, i, c);
        };
        float m = minus_inf(), z = 0.0f, d = 0.0f;
        bool soft = softmax;
        for (;;) {
            if (soft) {
                each([&](auto count, int i) {
                    constexpr int M = decltype(count)::value * V;
                    float x[M], c[M], top = m;
                    get(count, row, i, x, R::kNone);
                    counts(count, i, c);
                    if (STAGED) put_shared(count, stage, i, x);
#pragma unroll
                    for (int v = 0; v < M; ++v) top = fmaxf(top, x[v]);  // NaN is left out
                    if (top > m) {
                        const float scale = exp_below(m, top);
                        z *= scale;
                        d *= scale;
                        m = top;
                    }
                    R::template soft_scores<M>(x, m, c, x, z, d);
                });
                const float mine = m;
                m = warp_max(m);
                const float scale = exp_below(mine, m);
                z *= scale;
                d *= scale;
            } else {
                each([&](auto count, int i) {
                    constexpr int M = decltype(count)::value * V;
                    float x[M], c[M];
                    get(count, row, i, x, R::kNone);
                    counts(count, i, c);
                    R::template sigmoid_scores<M>(x, c, x, z, d);
                    if (STAGED) put_shared(count, stage, i, x);
                });
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
        if (z > 0.0f) run.add(fmaf(run.f.unit, mean, 1.0f));
        if constexpr (GRAD) {
            L* out = static_cast<L*>(a.dlogits) + t * a.dlogits_stride;
            const L* add = a.add != nullptr ? static_cast<const L*>(a.add) + t * a.add_stride : nullptr;
            const float gz = run.f.g * inverse, gm = -gz * mean;
            each([&](auto count, int i) {
                constexpr int A = decltype(count)::value, M = A * V;
                float x[M], c[M], adds[M], unused = 0.0f;
                counts(count, i, c);
                if constexpr (STAGED)
                    get_shared(count, stage, i, x);
                else
                    get(count, row, i, x, R::kNone);
                if (soft)
                    R::template soft_scores<M>(x, m, c, x, unused, unused);
                else if (!STAGED)
                    R::template sigmoid_scores<M>(x, c, x, unused, unused);
#pragma unroll
                for (int v = 0; v < M; ++v) adds[v] = 0.0f;
                if (add != nullptr) get(count, add, i, adds, 0u);
                R::template gradient<M>(x, c, gz, gm, adds);
#pragma unroll
                for (int u = 0; u < A; ++u) {
                    if constexpr (A > 1)
                        r.put_inside(out, r.column(i + u), x + u * V);
                    else
                        r.put(out, r.column(i + u), x + u * V);
                }
            });
        }
    }
    run.done(a, blockIdx.x, threadIdx.x == 0);
}

// Sixteen logits a lane up to 512 entries, in fewer lanes for shorter rows; then blocks of 128 to 512 threads. For the
// gradient they stage the counts up to 8192 entries, and rows up to 48 K.
constexpr int kStaged = 48 * 1024, kCounted = 8192;
template <int TEAM, bool VEC, bool GRAD, typename L>
BalanceTeam block_team(int n) {
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
BalanceTeam rows_team(int n) {
    if (n <= 32) return {(const void*)balance_lanes_kernel<2, 16, VEC, GRAD, L>, 128, 64, 0};
    if (n <= 64) return {(const void*)balance_lanes_kernel<4, 16, VEC, GRAD, L>, 128, 32, 0};
    if (n <= 128) return {(const void*)balance_lanes_kernel<8, 16, VEC, GRAD, L>, 128, 16, 0};
    if (n <= 256) return {(const void*)balance_lanes_kernel<16, 16, VEC, GRAD, L>, 128, 8, 0};
    if (n <= 512) return {(const void*)balance_lanes_kernel<32, 16, VEC, GRAD, L>, 128, 4, 0};
    if (n <= 2048) return block_team<128, VEC, GRAD, L>(n);
    return n <= kCounted ? block_team<256, VEC, GRAD, L>(n) : block_team<512, VEC, GRAD, L>(n);
}
template <typename L>
BalanceTeam rows_team(int n, bool vec, bool grad) {
    return vec ? (grad ? rows_team<true, true, L>(n) : rows_team<true, false, L>(n)) : (grad ? rows_team<false, true, L>(n) : rows_team<false, false, L>(n));
}


// The kernel that takes a whole call of few tokens, for rows of up to kSmallBins entries.
template <bool GRAD, typename L>
const void* small_kernel(int n) {
    if (n <= 64) return (const void*)balance_small_kernel<4, GRAD, L>;
    return n <= 256 ? (const void*)balance_small_kernel<16, GRAD, L> : (const void*)balance_small_kernel<32, GRAD, L>;
}

}  // namespace
}  // namespace sdm
