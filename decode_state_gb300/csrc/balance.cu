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

// A score of a sigmoid with what it leaves to one, in one register: s below one half, else -(1 - s), each with all
// of its bits. 0 for a masked logit.
__device__ __forceinline__ float sigmoid_pair(float x) {
    const float t = expf(-fabsf(x)), r = __frcp_rn(1.0f + t);
    return masked(x) ? 0.0f : x < 0.0f ? t * r : -(t * r);
}
__device__ __forceinline__ bool upper(float y) { return __float_as_int(y) < 0; }  // -0 too
__device__ __forceinline__ float pair_score(float y) { return upper(y) ? 1.0f + y : y; }
__device__ __forceinline__ float pair_rest(float y) { return upper(y) ? -y : 1.0f - y; }

// A team of TEAM threads (lanes of a warp, or a block) takes a run of consecutive tokens, E logits a thread in
// registers from the read to the gradient's write (E 0: rows too long for that are read again). VEC: 16 bytes an
// access, for rows that start on 16-byte boundaries; else 4.
template <int TEAM, int E, bool VEC, typename L>
__global__ void __launch_bounds__(TEAM <= 32 ? 128 : TEAM) balance_rows_kernel(const BalanceArgs a) {
    constexpr int NT = TEAM <= 32 ? 128 : TEAM, TEAMS = NT / TEAM, WARPS = TEAM <= 32 ? 1 : TEAM / 32;
    constexpr int V = (VEC ? 16 : 4) / sizeof(L), LANES = TEAM <= 32 ? TEAM : 32, R = E > 0 ? E : 1;
    constexpr bool KEPT = TEAM <= 32;  // the sequence's counts stay in registers too
    __shared__ float joint[2][3][WARPS];
    grid_dependency_wait();
    grid_launch_dependents();
    const int tid = threadIdx.x % TEAM, n = a.n;
    const int64_t team = (int64_t)blockIdx.x * TEAMS + threadIdx.x / TEAM, first = team * a.rows;
    const bool softmax = a.score == SDM_SOFTMAX, grad = a.dlogits != nullptr;
    const bool words = VEC || V == 1 ||
                       ((reinterpret_cast<uintptr_t>(a.logits) | reinterpret_cast<uintptr_t>(a.dlogits) | reinterpret_cast<uintptr_t>(a.add)) % 4 == 0 &&
                        ((a.row_stride | (grad ? a.dlogits_stride : 0) | (a.add ? a.add_stride : 0)) * sizeof(L)) % 4 == 0);

    const auto get = [&](const L* row, int j, float* x, float fill) {  // V elements from j on
        if (words && j + V <= n) {
            if constexpr (VEC) {
                const uint4 v = *reinterpret_cast<const uint4*>(row + j);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if constexpr (sizeof(L) == 2) {
                        x[2 * c] = __uint_as_float(w[c] << 16);
                        x[2 * c + 1] = __uint_as_float(w[c] & 0xffff0000u);
                    } else {
                        x[c] = __uint_as_float(w[c]);
                    }
                }
            } else if constexpr (V == 2) {
                const uint32_t w = *reinterpret_cast<const uint32_t*>(row + j);
                x[0] = __uint_as_float(w << 16);
                x[V - 1] = __uint_as_float(w & 0xffff0000u);
            } else {
                x[0] = to_f32(row[j]);
            }
        } else {
#pragma unroll
            for (int c = 0; c < V; ++c) x[c] = j + c < n ? to_f32(row[j + c]) : fill;
        }
    };
    const auto put = [&](L* row, int j, const float* d) {
        if (words && j + V <= n) {
            if constexpr (sizeof(L) == 2) {
                uint32_t w[V / 2];
#pragma unroll
                for (int c = 0; c < V / 2; ++c) {
                    const __nv_bfloat162 b = __floats2bfloat162_rn(d[2 * c], d[2 * c + 1]);
                    w[c] = *reinterpret_cast<const uint32_t*>(&b);
                }
                if constexpr (VEC)
                    *reinterpret_cast<uint4*>(row + j) = make_uint4(w[0], w[1], w[2], w[V / 2 - 1]);
                else
                    *reinterpret_cast<uint32_t*>(row + j) = w[0];
            } else if constexpr (VEC) {
                *reinterpret_cast<float4*>(row + j) = make_float4(d[0], d[1], d[2], d[V - 1]);
            } else {
                row[j] = from_f32<L>(d[0]);
            }
        } else {
#pragma unroll
            for (int c = 0; c < V; ++c)
                if (j + c < n) row[j + c] = from_f32<L>(d[c]);
        }
    };

    Sequence q{-1, 0, 0};
    float centre = 0.0f, unit = 0.0f, g = 0.0f, sum = 0.0f;
    float kept[KEPT ? R : 1];
    // the counts less their mean of the V entries from j on; 0 where there is no sequence
    const auto count = [&](int j, float* c) {
        const int32_t* from = a.counts + q.s * n;
        if (VEC && n % 4 == 0 && j + V <= n) {
#pragma unroll
            for (int i = 0; i < V; i += 4) {
                const int4 v = __ldg(reinterpret_cast<const int4*>(from + j + i));
                c[i] = (float)v.x - centre;
                c[(i + 1) % V] = (float)v.y - centre;
                c[(i + 2) % V] = (float)v.z - centre;
                c[(i + 3) % V] = (float)v.w - centre;
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) c[i] = j + i < n ? (float)__ldg(from + j + i) - centre : 0.0f;
        }
    };
    // of a token's team: the largest m, the sums z and d of what is relative to each thread's own m
    const auto join = [&](bool soft, float& m, float& z, float& d, int64_t t) {
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
            float(*to)[WARPS] = joint[t & 1];  // the other half is still read for the token before
            if ((tid & 31) == 0) {
                to[0][tid >> 5] = m;
                to[1][tid >> 5] = z;
                to[2][tid >> 5] = d;
            }
            __syncthreads();
            const int lane = tid & 31, w = lane % WARPS;  // every warp for itself
            const float theirs = to[0][w];
            m = warp_max<WARPS>(theirs);
            const float scale = lane >= WARPS ? 0.0f : soft ? exp_below(theirs, m) : 1.0f;
            z = warp_sum(to[1][w] * scale);
            d = warp_sum(to[2][w] * scale);
        }
    };

    for (int64_t i = 0; i < a.rows; ++i) {
        const int64_t t = first + i;
        const bool on = t < a.tokens;
        if (TEAM >= 32 && !on) break;  // lanes of a warp that hold several teams stay together
        if (on && (t < q.begin || t >= q.end)) {
            if (q.s >= 0 && tid == 0) a.parts[team + q.s] = sum;
            sum = 0.0f;
            q = sequence_of(a.offsets, a.sequences, a.tokens, t);
            centre = unit = g = 0.0f;
            const int total = q.s >= 0 ? __ldg(a.totals + q.s) : 0;
            if (total > 0 && q.end > q.begin) {
                const double per = (double)a.n / total;
                centre = (float)(1.0 / per);
                unit = (float)per;
                g = grad ? (float)((double)a.scale * per / (double)(q.end - q.begin)) * (a.dloss ? __ldg(a.dloss + q.s) : 1.0f) : 0.0f;
            }
            if constexpr (KEPT) {
#pragma unroll
                for (int e = 0; e < R; e += V) {
                    if (q.s >= 0) {
                        count((e / V * TEAM + tid) * V, kept + e);
                    } else {
#pragma unroll
                        for (int c = 0; c < V; ++c) kept[e + c] = 0.0f;
                    }
                }
            }
        }
        __syncwarp();
        const L* row = static_cast<const L*>(a.logits) + (on ? t : 0) * a.row_stride;
        float x[R];
        float m = minus_inf(), z = 0.0f, d = 0.0f;
        const auto counts_at = [&](int e, float* c) {
            if constexpr (KEPT) {
#pragma unroll
                for (int i2 = 0; i2 < V; ++i2) c[i2] = kept[e + i2];
            } else if (q.s >= 0) {
                count((e / V * TEAM + tid) * V, c);
            } else {
#pragma unroll
                for (int i2 = 0; i2 < V; ++i2) c[i2] = 0.0f;
            }
        };
        // f(first column, V logits) over this thread's columns of a row that is not kept
        const auto each = [&](const auto& f) {
            for (int j = tid * V; j < n; j += TEAM * V) {
                float y[V];
                get(row, j, y, minus_inf());
                f(j, y);
            }
        };
        const auto largest = [&] {
            if constexpr (E > 0) {
#pragma unroll
                for (int e = 0; e < E; ++e) m = fmaxf(m, x[e]);
            } else {
                each([&](int, const float* y) {
#pragma unroll
                    for (int c = 0; c < V; ++c) m = fmaxf(m, y[c]);
                });
            }
        };
        // Sigmoid scores so small that their sum loses bits are shares of exp(x) instead, as for a softmax.
        bool soft = softmax;
        float mine;
        for (;;) {
            if constexpr (E > 0) {
#pragma unroll
                for (int e = 0; e < E; e += V) get(row, on ? (e / V * TEAM + tid) * V : n, x + e, minus_inf());
#pragma unroll
                for (int e = 0; e < E; ++e) x[e] = fmaxf(x[e], minus_inf());  // NaN is masked
            }
            if (soft) {
                largest();
                const bool plain = fabsf(m) <= 3.402823466e38f;  // neither +inf nor masked throughout
                if constexpr (E > 0) {
#pragma unroll
                    for (int e = 0; e < E; e += V) {
                        float c[V];
                        counts_at(e, c);
#pragma unroll
                        for (int i2 = 0; i2 < V; ++i2) {
                            x[e + i2] = plain ? expf(x[e + i2] - m) : exp_below(x[e + i2], m);
                            z += x[e + i2];
                            d = fmaf(x[e + i2], c[i2], d);
                        }
                    }
                } else {
                    each([&](int j, const float* y) {
                        float c[V];
                        counts_at(j / (TEAM * V) * V, c);
#pragma unroll
                        for (int i2 = 0; i2 < V; ++i2) {
                            const float s = exp_below(y[i2], m);
                            z += s;
                            d = fmaf(s, c[i2], d);
                        }
                    });
                }
            } else if constexpr (E > 0) {
#pragma unroll
                for (int e = 0; e < E; e += V) {
                    float c[V];
                    counts_at(e, c);
#pragma unroll
                    for (int i2 = 0; i2 < V; ++i2) {
                        x[e + i2] = sigmoid_pair(x[e + i2]);
                        const float s = pair_score(x[e + i2]);
                        z += s;
                        d = fmaf(s, c[i2], d);
                    }
                }
            } else {
                each([&](int j, const float* y) {
                    float c[V];
                    counts_at(j / (TEAM * V) * V, c);
#pragma unroll
                    for (int i2 = 0; i2 < V; ++i2) {
                        const float s = pair_score(sigmoid_pair(y[i2]));
                        z += s;
                        d = fmaf(s, c[i2], d);
                    }
                });
            }
            mine = m;
            join(soft, m, z, d, t);
            const bool low = on && !soft && z < 0x1p-100f;
            if (!(TEAM <= 32 ? __any_sync(kAll, low) : low)) break;
            if constexpr (TEAM > 32) __syncthreads();  // joint is written again
            soft |= low;
            m = minus_inf();
            z = d = 0.0f;
        }
        const float mean = z > 0.0f ? __fdiv_rn(d, z) : 0.0f;
        if (z > 0.0f) sum += fmaf(unit, mean, 1.0f);
        if (grad && on) {
            L* out = static_cast<L*>(a.dlogits) + t * a.dlogits_stride;
            const L* add = a.add ? static_cast<const L*>(a.add) + t * a.add_stride : nullptr;
            const float gz = z > 0.0f ? __fdiv_rn(g, z) * (soft ? exp_below(mine, m) : 1.0f) : 0.0f;
            const auto write = [&](int j, const float* s, const float* c) {
                float y[V];
#pragma unroll
                for (int i2 = 0; i2 < V; ++i2) {
                    if (soft)
                        y[i2] = gz * s[i2] * (c[i2] - mean);
                    else
                        y[i2] = gz * pair_score(s[i2]) * pair_rest(s[i2]) * (c[i2] - mean);
                }
                if (add != nullptr) {
                    float b[V];
                    get(add, j, b, 0.0f);
#pragma unroll
                    for (int i2 = 0; i2 < V; ++i2) y[i2] += b[i2];
                }
                put(out, j, y);
            };
            if constexpr (E > 0) {
#pragma unroll
                for (int e = 0; e < E; e += V) {
                    float c[V];
                    counts_at(e, c);
                    write((e / V * TEAM + tid) * V, x + e, c);
                }
            } else {
                each([&](int j, const float* y) {
                    float c[V], s[V];
                    counts_at(j / (TEAM * V) * V, c);
#pragma unroll
                    for (int i2 = 0; i2 < V; ++i2) s[i2] = soft ? exp_below(y[i2], mine) : sigmoid_pair(y[i2]);
                    write(j, s, c);
                });
            }
        }
    }
    if (q.s >= 0 && tid == 0) a.parts[team + q.s] = sum;
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

template <bool VEC, typename L>
Team rows_kernel(int n) {
    if (n <= 32) return {(const void*)balance_rows_kernel<4, 8, VEC, L>, 128, 32};
    if (n <= 64) return {(const void*)balance_rows_kernel<8, 8, VEC, L>, 128, 16};
    if (n <= 128) return {(const void*)balance_rows_kernel<16, 8, VEC, L>, 128, 8};
    if (n <= 256) return {(const void*)balance_rows_kernel<32, 8, VEC, L>, 128, 4};
    if (n <= 512) return {(const void*)balance_rows_kernel<32, 16, VEC, L>, 128, 4};
    if (n <= 1024) return {(const void*)balance_rows_kernel<32, 32, VEC, L>, 128, 4};
    if (n <= 2048) return {(const void*)balance_rows_kernel<128, 16, VEC, L>, 128, 1};
    if (n <= 4096) return {(const void*)balance_rows_kernel<128, 32, VEC, L>, 128, 1};
    if (n <= 8192) return {(const void*)balance_rows_kernel<256, 32, VEC, L>, 256, 1};
    if (n <= 16384) return {(const void*)balance_rows_kernel<512, 32, VEC, L>, 512, 1};
    return {(const void*)balance_rows_kernel<512, 0, VEC, L>, 512, 1};
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
    const bool vec = whole(a.logits, a.row_stride) && whole(a.dlogits, a.dlogits_stride) && whole(a.add, a.add_stride) &&
                     reinterpret_cast<uintptr_t>(a.counts) % 16 == 0;
    const Team team = a.logit_bf16 ? (vec ? rows_kernel<true, uint16_t>(a.n) : rows_kernel<false, uint16_t>(a.n))
                                   : (vec ? rows_kernel<true, float>(a.n) : rows_kernel<false, float>(a.n));
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
        const int64_t most = std::min<int64_t>(kBalanceTeams, sms * (2048 / team.threads) * team.teams);
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
