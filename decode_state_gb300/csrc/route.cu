// Routing: the k best of n entries a token, with their weights, and the gradient of the logits.
//
// Math (include/sdm.h): scores s = softmax(x) or 1 / (1 + exp(-x)); entries ranked by x, s or
// s + bias; best groups, then best entries, ties to the lower index; weights s, renormalised.
//
// Ranks are compared as 32-bit integers in the order of the floats, 1 for masked entries and more for
// all others.
//
// Both forward kernels find a lower bound of the k-th rank first: of the largest ranks of 32 lanes, or
// of all threads of a block, the k-th largest is one, since k entries at least reach it. The entries
// that reach it are few more than k; they are collected in shared memory and ranked by counting.
// Where they are too many (equal ranks), or fewer than k entries are not masked, a slower path
// follows that takes any ranks.
//
// route_warp_kernel (n <= 1024, k <= 32): a warp for each token, its ranks in registers, lane l the
// consecutive entries from l * E on, so that lane order is index order. Bound by instructions (an
// exponential and a reciprocal for every entry of a biased sigmoid), not by its 2 or 4 bytes.
// route_block_kernel: a block for each token, its ranks staged in shared memory. The slower path
// narrows the k-th rank down by histograms of its leading 11, then 11, then 10 bits.
#include <algorithm>
#include <climits>
#include <cmath>

#include "quant_device.cuh"
#include "sdm_internal.h"

namespace sdm {
namespace {

__device__ unsigned int g_route_status;

constexpr unsigned kAll = 0xffffffffu;
constexpr uint32_t kMasked = 1;
constexpr int kMaxGroups = 256, kMaxK = 256;
constexpr int kCandidates = 512;
constexpr size_t kStagedBytes = 192 * 1024;  // ranks a block keeps in shared memory

__device__ __forceinline__ float minus_inf() { return __uint_as_float(0xff800000u); }
__device__ __forceinline__ bool masked(float x) { return !(x > minus_inf()); }  // NaN too

// exp(x - m) with m the largest of the logits; several +inf are the largest together
__device__ __forceinline__ float exp_below(float x, float m) {
    return masked(x) ? 0.0f : x == m ? 1.0f : expf(x - m);
}
__device__ __forceinline__ float sigmoid(float x) { return masked(x) ? 0.0f : __frcp_rn(__fadd_rn(1.0f, expf(-x))); }

// Scores of N logits: sigmoid() bit by bit (any value for masked ones), but without a branch for each,
// so that they overlap. A reciprocal of a float in [1, 2^126] is correctly rounded by one Newton step from the
// hardware's approximation (checked for every significand); the rare others are done again.
template <int N>
__device__ __forceinline__ void sigmoids(const float* x, float* s) {
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float y = __fadd_rn(1.0f, expf(masked(x[i]) ? 0.0f : -x[i]));
        float r;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(y));
        s[i] = fmaf(fmaf(-y, r, 1.0f), r, r);
        most = fmaxf(most, y);
    }
    if (most > 0x1p126f) {
#pragma unroll
        for (int i = 0; i < N; ++i) s[i] = __frcp_rn(__fadd_rn(1.0f, expf(-x[i])));
    }
}

// A float as an unsigned integer in the same order (-0 and +0 alike); masked ranks become kMasked.
__device__ __forceinline__ uint32_t ordered(float r) {
    if (masked(r)) return kMasked;
    const uint32_t b = __float_as_uint(r + 0.0f);
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}

__device__ __forceinline__ void put_index(const RouteArgs& a, int64_t t, int i, int j) {
    if (a.idx64)
        static_cast<int64_t*>(a.idx)[t * a.k + i] = j + (a.base ? __ldg(static_cast<const int64_t*>(a.base) + t) : 0);
    else
        static_cast<int32_t*>(a.idx)[t * a.k + i] = j + (a.base ? __ldg(static_cast<const int32_t*>(a.base) + t) : 0);
}

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(kAll, x, o);
    return x;
}
__device__ __forceinline__ float warp_max(float x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(kAll, x, o));
    return x;
}

// The two largest values of a set as it grows; empty places hold -inf.
struct Top2 {
    float a, b;
    __device__ __forceinline__ Top2() : a(minus_inf()), b(minus_inf()) {}
    __device__ __forceinline__ void add(float x) {
        const float low = fminf(a, x);
        a = fmaxf(a, x);
        b = fmaxf(b, low);
    }
    __device__ __forceinline__ void join(float oa, float ob) {  // the two largest of another set
        add(oa);
        b = fmaxf(b, ob);  // ob <= oa: it is second at best
    }
    // a group's score, as an ordered integer: 0 for a group of masked entries
    __device__ __forceinline__ uint32_t score(int group_top) const {
        if (a == minus_inf()) return 0;
        return ordered(group_top == 1 ? a : a + (b == minus_inf() ? 0.0f : b));
    }
};

// Whether group g is among the `top` best of scores[0 .. groups), ties to the lower index.
__device__ __forceinline__ bool group_stays(const uint32_t* scores, int groups, int top, int g) {
    const uint32_t mine = scores[g];
    int better = 0;
    for (int o = 0; o < groups; ++o) better += scores[o] > mine || (scores[o] == mine && o < g);
    return better < top;
}

// The inputs of a rank as 64 bits that order first by rank, then by the lower index.
__device__ __forceinline__ uint64_t candidate(uint32_t rank, int j) { return (uint64_t)rank << 32 | (uint32_t)~j; }
__device__ __forceinline__ int candidate_index(uint64_t c) { return (int)~(uint32_t)c; }

// ---------------------------------------------------------------- a warp for each token

constexpr int kWarpThreads = 256;
constexpr int kWarpCandidates = 64;

// The k-th largest of the 32 lanes' values, and the largest, on every lane (a bitonic sort).
__device__ __forceinline__ float kth_of_lanes(float x, int k, float* most) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int size = 2; size <= 32; size *= 2) {
#pragma unroll
        for (int o = size / 2; o >= 1; o /= 2) {
            const float y = __shfl_xor_sync(kAll, x, o);
            const bool larger = ((lane & o) == 0) == ((lane & size) == 0);  // falling order
            x = larger ? fmaxf(x, y) : fminf(x, y);
        }
    }
    *most = __shfl_sync(kAll, x, 0);
    return __shfl_sync(kAll, x, k - 1);
}

__device__ __forceinline__ int lanes_before(int own, int* all) {
    const int lane = threadIdx.x & 31;
    int sum = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kAll, sum, o);
        if (lane >= o) sum += y;
    }
    *all = __shfl_sync(kAll, sum, 31);
    return sum - own;
}

// E: entries of a lane. L: uint16_t (bf16) or float logits.
template <int E, typename L>
__global__ void __launch_bounds__(kWarpThreads) route_warp_kernel(const RouteArgs a) {
    constexpr int WARPS = kWarpThreads / 32;
    extern __shared__ float staged[];  // groups that are no whole lanes: every warp's group values [n] and scores [n_groups]
    __shared__ uint64_t found[WARPS][kWarpCandidates];
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = (int64_t)blockIdx.x * WARPS + warp;
    if (t >= a.tokens) return;
    const int n = a.n, k = a.k, j0 = lane * E;
    const L* row = static_cast<const L*>(a.logits) + t * a.row_stride;

    float x[E];
    if ((reinterpret_cast<uintptr_t>(row) & 15u) == 0 && j0 + E <= n) {
#pragma unroll
        for (int i = 0; i < E * (int)sizeof(L) / 16; ++i) {
            const uint4 v = __ldg(reinterpret_cast<const uint4*>(row + j0) + i);
            if constexpr (sizeof(L) == 2)
                unpack<Bf16>(v, x + 8 * i);
            else
                unpack<F32>(v, x + 4 * i);
        }
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) x[i] = j0 + i < n ? to_f32(__ldg(row + j0 + i)) : minus_inf();
    }

    const bool softmax = a.score == SDM_SOFTMAX, biased = a.bias != nullptr;
    const bool grouped = a.n_groups > 1 && a.top_groups < a.n_groups, by_sum = grouped && a.group_top == 2;
    float m = minus_inf(), total = 1.0f;
    if (softmax && (biased || !a.renorm || by_sum)) {
#pragma unroll
        for (int i = 0; i < E; ++i) m = fmaxf(m, x[i]);  // NaN takes no part
        m = warp_max(m);
        if (biased || !a.renorm) {
            total = 0.0f;
#pragma unroll
            for (int i = 0; i < E; ++i) total += exp_below(x[i], m);
            total = warp_sum(total);
        }
    }
    // ranks, -inf where masked
    float r[E];
    if (!softmax) {
        sigmoids<E>(x, r);
    } else if (biased) {
#pragma unroll
        for (int i = 0; i < E; ++i) r[i] = __fdiv_rn(exp_below(x[i], m), total);
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) r[i] = x[i];
    }
    if (biased) {
        if ((reinterpret_cast<uintptr_t>(a.bias) & 15u) == 0 && j0 + E <= n) {
#pragma unroll
            for (int i = 0; i < E / 4; ++i) {
                const float4 f = __ldg(reinterpret_cast<const float4*>(a.bias + j0) + i);
                r[4 * i] += f.x, r[4 * i + 1] += f.y, r[4 * i + 2] += f.z, r[4 * i + 3] += f.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i)
                if (j0 + i < n) r[i] += __ldg(a.bias + j0 + i);
        }
    }
#pragma unroll
    for (int i = 0; i < E; ++i) r[i] = masked(x[i]) || masked(r[i]) ? minus_inf() : r[i];

    if (grouped) {
        const bool sums = by_sum && softmax && !biased;  // judged by exp(x - m), not by the ranks
        const int per = n / a.n_groups, lanes = per / E;
        if (per % E == 0 && lanes <= 32 && (lanes & (lanes - 1)) == 0) {
            // whole lanes, a power of two of them: by shuffles
            Top2 top;
#pragma unroll
            for (int i = 0; i < E; ++i) top.add(sums ? (r[i] == minus_inf() ? minus_inf() : exp_below(x[i], m)) : r[i]);
            for (int o = 1; o < lanes; o <<= 1) top.join(__shfl_xor_sync(kAll, top.a, o), __shfl_xor_sync(kAll, top.b, o));
            const uint32_t mine = top.score(a.group_top);
            const int g = lane / lanes;
            int better = 0;
            for (int q = 0; q < a.n_groups; ++q) {
                const uint32_t other = __shfl_sync(kAll, mine, q * lanes);
                better += other > mine || (other == mine && q < g);
            }
            if (better >= a.top_groups) {
#pragma unroll
                for (int i = 0; i < E; ++i) r[i] = minus_inf();
            }
        } else {
            float* value = staged + (size_t)warp * (n + a.n_groups);
            uint32_t* scores = reinterpret_cast<uint32_t*>(value + n);
#pragma unroll
            for (int i = 0; i < E; ++i)
                if (j0 + i < n) value[j0 + i] = sums ? (r[i] == minus_inf() ? minus_inf() : exp_below(x[i], m)) : r[i];
            __syncwarp();
            for (int g = lane; g < a.n_groups; g += 32) {
                Top2 top;
                int at = lane % per;  // lanes start apart, since groups are often a multiple of the banks
                for (int i = 0; i < per; ++i) {
                    top.add(value[g * per + at]);
                    at = at + 1 == per ? 0 : at + 1;
                }
                scores[g] = top.score(a.group_top);
            }
            __syncwarp();
            uint32_t stays[kMaxGroups / 32];  // bit `lane` of word i: group 32 i + lane
#pragma unroll
            for (int i = 0; i < kMaxGroups / 32; ++i) {
                const int g = 32 * i + lane;
                if (32 * i < a.n_groups)
                    stays[i] = __ballot_sync(kAll, g < a.n_groups && group_stays(scores, a.n_groups, a.top_groups, g));
            }
            __syncwarp();
            if (lane == 0) {
#pragma unroll
                for (int i = 0; i < kMaxGroups / 32; ++i)
                    if (32 * i < a.n_groups) scores[i] = stays[i];
            }
            __syncwarp();
            int g = j0 / per, left = per - j0 % per;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                if (j0 + i < n && !((scores[g >> 5] >> (g & 31)) & 1u)) r[i] = minus_inf();
                if (--left == 0) {
                    ++g;
                    left = per;
                }
            }
        }
    }

    // the entries that reach the k-th largest of the lanes' maxima
    float best = r[0];
#pragma unroll
    for (int i = 1; i < E; ++i) best = fmaxf(best, r[i]);
    float most;
    const float bound = kth_of_lanes(best, k, &most);
    if (softmax && !biased && a.renorm) m = most;  // any reference does: it cancels in the weights
    int own = 0, count;
#pragma unroll
    for (int i = 0; i < E; ++i) own += r[i] >= bound && r[i] > minus_inf();
    int at = lanes_before(own, &count);
    uint64_t* cand = found[warp];
    const bool many = count > kWarpCandidates;
    if (!many) {
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (r[i] >= bound && r[i] > minus_inf()) cand[at++] = candidate(ordered(r[i]), j0 + i);
    } else {
        // too many alike: k rounds of a maximum over the warp, the lowest index first
        for (int round = 0; round < k; ++round) {
            const uint32_t top = __reduce_max_sync(kAll, ordered(best));
            const int src = __ffs(__ballot_sync(kAll, ordered(best) == top)) - 1;  // there are more than k live ones
            if (lane == src) {
                int hit = 0;
#pragma unroll
                for (int i = E - 1; i >= 0; --i)
                    if (ordered(r[i]) == top) hit = i;
                best = minus_inf();
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    if (i == hit) r[i] = minus_inf();
                    best = fmaxf(best, r[i]);
                }
                cand[round] = candidate(top, j0 + hit);
            }
        }
        count = k;
    }
    __syncwarp();
    uint64_t mine[kWarpCandidates / 32];
    int rank[kWarpCandidates / 32];
    float score[kWarpCandidates / 32], sum = 0.0f;
#pragma unroll
    for (int q = 0; q < kWarpCandidates / 32; ++q) {
        rank[q] = k;
        score[q] = 0.0f;
        if (lane + 32 * q < count) {
            mine[q] = cand[lane + 32 * q];
            rank[q] = 0;
            for (int o = 0; o < count; ++o) rank[q] += cand[o] > mine[q];
            if (rank[q] < k) {
                const float y = to_f32(__ldg(row + candidate_index(mine[q])));
                score[q] = softmax ? exp_below(y, m) : sigmoid(y);
                sum += score[q];
            }
        }
    }
    if (a.renorm) total = warp_sum(sum);
#pragma unroll
    for (int q = 0; q < kWarpCandidates / 32; ++q) {
        if (rank[q] < k) {
            put_index(a, t, rank[q], candidate_index(mine[q]));
            a.w[t * k + rank[q]] = total > 0.0f && (softmax || a.renorm) ? __fdiv_rn(score[q], total) * a.scale : score[q] * a.scale;
        }
    }
    if (count < k) {  // fill up with masked entries, in index order
        own = 0;
#pragma unroll
        for (int i = 0; i < E; ++i) own += j0 + i < n && r[i] == minus_inf();
        int all;
        at = count + lanes_before(own, &all);
#pragma unroll
        for (int i = 0; i < E; ++i) {
            if (j0 + i < n && r[i] == minus_inf()) {
                if (at < k) {
                    put_index(a, t, at, j0 + i);
                    a.w[t * k + at] = 0.0f;
                }
                ++at;
            }
        }
    }
}

// ---------------------------------------------------------------- a block for each token

constexpr int kBins = 2048;

__device__ __forceinline__ float block_reduce(float x, bool sum, float* tmp, int warps) {
    x = sum ? warp_sum(x) : warp_max(x);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) tmp[threadIdx.x >> 5] = x;
    __syncthreads();
    float r = tmp[0];
    for (int i = 1; i < warps; ++i) r = sum ? r + tmp[i] : fmaxf(r, tmp[i]);
    return r;
}

template <int NT, typename L>
__global__ void __launch_bounds__(NT, NT == 512 ? 2 : 4) route_block_kernel(const RouteArgs a, int staged) {
    constexpr int WARPS = NT / 32;
    extern __shared__ __align__(16) uint32_t keys[];  // [n] when staged
    __shared__ int hist[kBins];
    __shared__ uint64_t cand[kCandidates];
    __shared__ uint32_t scores[kMaxGroups];
    __shared__ uint32_t stays[kMaxGroups / 32];
    __shared__ float tmp[WARPS];
    __shared__ int counts[WARPS];
    __shared__ int sel_j[kMaxK];
    __shared__ float sel_s[kMaxK];
    __shared__ int found_bin, found_above, n_cand;
    grid_dependency_wait();
    grid_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t t = blockIdx.x;
    const int n = a.n, k = a.k;
    const bool softmax = a.score == SDM_SOFTMAX, biased = a.bias != nullptr;
    const bool grouped = a.n_groups > 1 && a.top_groups < a.n_groups;
    const int per = n / a.n_groups;
    const L* row = static_cast<const L*>(a.logits) + t * a.row_stride;
    const bool vec = (reinterpret_cast<uintptr_t>(row) & 15u) == 0;
    constexpr int V = 16 / sizeof(L);  // logits of a 16-byte load

    // f(j, x) for every logit: whole 16 bytes where the row is aligned
    const auto each = [&](const auto& f) {
        int first = 0;
        if (vec) {
            first = n / V * V;
            int j = tid * V;
            for (; j + 3 * NT * V < first; j += 4 * NT * V) {  // four loads on their way together
                uint4 v[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) v[u] = __ldg(reinterpret_cast<const uint4*>(row + j + u * NT * V));
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    float x[V];
                    if constexpr (sizeof(L) == 2)
                        unpack<Bf16>(v[u], x);
                    else
                        unpack<F32>(v[u], x);
#pragma unroll
                    for (int i = 0; i < V; ++i) f(j + u * NT * V + i, x[i]);
                }
            }
            for (; j < first; j += NT * V) {
                const uint4 v = __ldg(reinterpret_cast<const uint4*>(row + j));
                float x[V];
                if constexpr (sizeof(L) == 2)
                    unpack<Bf16>(v, x);
                else
                    unpack<F32>(v, x);
#pragma unroll
                for (int i = 0; i < V; ++i) f(j + i, x[i]);
            }
        }
        for (int j = first + tid; j < n; j += NT) f(j, to_f32(__ldg(row + j)));
    };

    float m = minus_inf(), total = 1.0f;
    if (softmax && (biased || !a.renorm || (grouped && a.group_top == 2))) {
        each([&](int, float x) { m = fmaxf(m, x); });
        m = block_reduce(m, false, tmp, WARPS);
        if (biased || !a.renorm) {
            total = 0.0f;
            each([&](int, float x) { total += exp_below(x, m); });
            total = block_reduce(total, true, tmp, WARPS);
        }
    }
    const auto rank_of = [&](int j, float x) {
        if (masked(x)) return x;
        float r = x;
        if (!softmax)
            r = sigmoid(x);
        else if (biased)
            r = __fdiv_rn(exp_below(x, m), total);
        return biased ? r + __ldg(a.bias + j) : r;
    };

    if (grouped) {
        for (int g = warp; g < a.n_groups; g += WARPS) {
            Top2 top;
            for (int i = lane; i < per; i += 32) {
                const int j = g * per + i;
                const float x = to_f32(__ldg(row + j)), r = rank_of(j, x);
                top.add(masked(r) ? minus_inf() : softmax && !biased && a.group_top == 2 ? exp_below(x, m) : r);
            }
            for (int o = 16; o; o >>= 1) top.join(__shfl_xor_sync(kAll, top.a, o), __shfl_xor_sync(kAll, top.b, o));
            if (lane == 0) scores[g] = top.score(a.group_top);
        }
        __syncthreads();
        for (int g0 = warp * 32; g0 < a.n_groups; g0 += NT) {
            const int g = g0 + lane;
            const uint32_t b = __ballot_sync(kAll, g < a.n_groups && group_stays(scores, a.n_groups, a.top_groups, g));
            if (lane == 0) stays[g0 / 32] = b;
        }
        __syncthreads();
    }
    const auto make_key = [&](int j, float x) -> uint32_t {
        if (grouped) {
            const int g = j / per;
            if (!((stays[g >> 5] >> (g & 31)) & 1u)) return kMasked;
        }
        return ordered(rank_of(j, x));
    };
    uint32_t best = 0;  // the largest rank of this thread's entries
    each([&](int j, float x) {
        const uint32_t key = make_key(j, x);
        best = max(best, key);
        if (staged) keys[j] = key;
    });
    const auto key_at = [&](int j) -> uint32_t { return staged ? keys[j] : make_key(j, to_f32(__ldg(row + j))); };

    // the bin of the need-th largest of the values counted in hist, from the top: found_bin (-1: there
    // are fewer), and found_above, those in higher bins; counts holds the warps' shares of all of them
    const auto find_bin = [&](int need) {
        constexpr int PER = kBins / NT;  // thread i owns the PER bins from i * PER on, counted from the top
        int own = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) own += hist[kBins - 1 - (tid * PER + i)];
        int all;
        int before = lanes_before(own, &all);
        if (lane == 31) counts[warp] = all;
        if (tid == 0) found_bin = -1;
        __syncthreads();
        for (int i = 0; i < warp; ++i) before += counts[i];
        if (before < need && before + own >= need) {
            for (int i = 0; i < PER; ++i) {
                const int b = kBins - 1 - (tid * PER + i), c = hist[b];
                if (before + c >= need) {
                    found_bin = b;
                    found_above = before;
                    break;
                }
                before += c;
            }
        }
        __syncthreads();
    };
    const auto clear_bins = [&]() {
        for (int b = tid; b < kBins; b += NT) hist[b] = 0;
        __syncthreads();
    };
    // candidates: the live entries with key >= lowest; those that fit are kept
    const auto collect = [&](uint32_t lowest) {
        if (tid == 0) n_cand = 0;
        __syncthreads();
        const auto test = [&](uint32_t key, int j) {
            if (key > kMasked && key >= lowest) {
                const int c = atomicAdd(&n_cand, 1);
                if (c < kCandidates) cand[c] = candidate(key, j);
            }
        };
        if (staged) {
            const int whole = n / 4 * 4;
            for (int j = tid * 4; j < whole; j += NT * 4) {
                const uint4 v = *reinterpret_cast<const uint4*>(keys + j);
                test(v.x, j), test(v.y, j + 1), test(v.z, j + 2), test(v.w, j + 3);
            }
            for (int j = whole + tid; j < n; j += NT) test(keys[j], j);
        } else {
            for (int j = tid; j < n; j += NT) test(key_at(j), j);
        }
        __syncthreads();
    };

    // a lower bound by the threads' maxima
    clear_bins();
    if (best > kMasked) atomicAdd(&hist[best >> 21], 1);
    __syncthreads();
    find_bin(k);
    bool done = false, few = false, ties = false;
    uint32_t lowest = 0;
    int C = 0;
    if (found_bin >= 0) {
        collect((uint32_t)found_bin << 21);
        C = n_cand;
        done = C <= kCandidates;
    }
    if (!done) {
        // narrow the k-th rank down: `above` live entries lie above the prefix, and those of the prefix
        // and above are at most kCandidates, or all their bits are fixed
        int above = 0, need = k, inside = 0;
        bool exact = false;  // the prefix is a whole key
        uint32_t prefix = 0;
        for (int level = 0; level < 3; ++level) {
            const int shift = level == 0 ? 21 : level == 1 ? 10 : 0, bits = level == 2 ? 10 : 11;
            __syncthreads();
            clear_bins();
            for (int j = tid; j < n; j += NT) {
                const uint32_t key = key_at(j);
                if (key > kMasked && (level == 0 || key >> (shift + bits) == prefix))
                    atomicAdd(&hist[(key >> shift) & ((1u << bits) - 1u)], 1);
            }
            __syncthreads();
            find_bin(need);
            if (found_bin < 0) {  // level 0 only: all live entries are taken
                few = true;
                lowest = kMasked + 1;
                break;
            }
            above += found_above;
            need -= found_above;
            prefix = (prefix << bits) | (uint32_t)found_bin;
            inside = hist[found_bin];
            lowest = prefix << shift;
            exact = level == 2;
            if (above + inside <= kCandidates) break;
        }
        // only what lies above the last rank when too many share it
        ties = !few && exact && above + inside > kCandidates;
        collect(ties ? lowest + 1 : lowest);
        C = n_cand;
    }
    // rank the candidates by counting, four threads for each
    for (int c0 = 0; c0 < C; c0 += NT / 4) {
        const int c = c0 + tid / 4;
        const uint64_t mine = c < C ? cand[c] : 0;
        int better = 0;
        for (int o = tid % 4; o < C; o += 4) better += cand[o] > mine;
        better += __shfl_xor_sync(kAll, better, 1);
        better += __shfl_xor_sync(kAll, better, 2);
        if (c < C && better < k && tid % 4 == 0) sel_j[better] = candidate_index(mine);
    }
    __syncthreads();
    if (softmax && !biased && a.renorm && C > 0) m = to_f32(__ldg(row + sel_j[0]));  // any reference does: it cancels
    for (int i = tid; i < min(C, k); i += NT) {
        const float x = to_f32(__ldg(row + sel_j[i]));
        sel_s[i] = softmax ? exp_below(x, m) : sigmoid(x);
    }
    // fill up, in index order, with entries of the shared last rank, or with masked ones of weight 0
    if (few || ties) {
        const uint32_t want = few ? kMasked : lowest;
        int have = C;
        for (int j0 = 0; j0 < n && have < k; j0 += NT) {
            const int j = j0 + tid;
            const bool hit = j < n && key_at(j) == want;
            const uint32_t ballot = __ballot_sync(kAll, hit);
            if (lane == 0) counts[warp] = __popc(ballot);
            __syncthreads();
            int at = have + __popc(ballot & ((1u << lane) - 1u));
            for (int i = 0; i < WARPS; ++i) {
                if (i < warp) at += counts[i];
                have += counts[i];
            }
            if (hit && at < k) {
                sel_j[at] = j;
                const float x = to_f32(__ldg(row + j));
                if (softmax && !biased && a.renorm && C == 0) m = x;  // all that are taken share this logit
                sel_s[at] = few ? 0.0f : softmax ? exp_below(x, m) : sigmoid(x);
            }
            __syncthreads();
        }
    }
    __syncthreads();
    if (a.renorm) {
        float sum = 0.0f;
        for (int i = lane; i < k; i += 32) sum += sel_s[i];
        total = warp_sum(sum);  // every warp sums alike
    }
    for (int i = tid; i < k; i += NT) {
        put_index(a, t, i, sel_j[i]);
        const float s = sel_s[i];
        a.w[t * k + i] = total > 0.0f && (softmax || a.renorm) ? __fdiv_rn(s, total) * a.scale : s * a.scale;
    }
}

// ---------------------------------------------------------------- the gradient

// A team of TEAM threads (a warp, or a block) for each token. Only a softmax that is not
// renormalised has gradients outside the chosen entries; all others just get zeros there.
template <int TEAM, typename L>
__global__ void __launch_bounds__(TEAM == 32 ? 128 : TEAM) route_backward_kernel(const RouteArgs a) {
    constexpr int NT = TEAM == 32 ? 128 : TEAM, TEAMS = NT / TEAM, WARPS = TEAM / 32;
    __shared__ float u_of[TEAMS][kMaxK];  // gradients of the chosen scores
    __shared__ float s_of[TEAMS][kMaxK];
    __shared__ int j_of[TEAMS][kMaxK];
    __shared__ float tmp[NT / 32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int team = threadIdx.x / TEAM, tid = threadIdx.x % TEAM, lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * TEAMS + team;
    if (t >= a.tokens) return;  // a whole team
    const int n = a.n, k = a.k;
    const L* row = static_cast<const L*>(a.logits) + t * a.row_stride;
    L* out = static_cast<L*>(a.dlogits) + t * a.dlogits_stride;
    float *u = u_of[team], *s = s_of[team];
    int* at = j_of[team];
    const bool softmax = a.score == SDM_SOFTMAX, dense = softmax && !a.renorm;

    const auto sync = [] {
        if constexpr (TEAM == 32)
            __syncwarp();
        else
            __syncthreads();
    };
    const auto team_sum = [&](float v) {
        if constexpr (TEAM == 32)
            return warp_sum(v);
        else
            return block_reduce(v, true, tmp, WARPS);
    };
    const auto team_max = [&](float v) {
        if constexpr (TEAM == 32)
            return warp_max(v);
        else
            return block_reduce(v, false, tmp, WARPS);
    };

    float m = minus_inf(), total = 1.0f;
    if (dense) {
        for (int j = tid; j < n; j += TEAM) m = fmaxf(m, to_f32(__ldg(row + j)));
        m = team_max(m);
        total = 0.0f;
        for (int j = tid; j < n; j += TEAM) total += exp_below(to_f32(__ldg(row + j)), m);
        total = team_sum(total);
    }
    for (int i = tid; i < k; i += TEAM) {
        const int64_t e = t * k + i;
        const int64_t j = (a.idx64 ? __ldg(static_cast<const int64_t*>(a.idx) + e) : __ldg(static_cast<const int32_t*>(a.idx) + e)) -
                          (a.base == nullptr ? 0 : a.idx64 ? __ldg(static_cast<const int64_t*>(a.base) + t) : __ldg(static_cast<const int32_t*>(a.base) + t));
        const bool in = j >= 0 && j < n;
        if (!in) atomicOr(&g_route_status, SDM_DEV_BAD_INDEX);
        at[i] = in ? (int)j : -1;
        s[i] = in ? to_f32(__ldg(row + j)) : minus_inf();
        u[i] = __ldg(a.dw + e) * a.scale;
    }
    if (softmax && a.renorm) {
        for (int i = tid; i < k; i += TEAM) m = fmaxf(m, s[i]);  // each thread's own entries
        m = team_max(m);
    }
    float own = 0.0f;
    for (int i = tid; i < k; i += TEAM) {
        s[i] = !softmax ? sigmoid(s[i]) : dense ? (total > 0.0f ? __fdiv_rn(exp_below(s[i], m), total) : 0.0f) : exp_below(s[i], m);
        own += s[i];
    }
    // u: the gradients of the scores (of exp(x - m) when a softmax is renormalised, which is as good:
    // the factor between them cancels in u * s)
    if (a.renorm) {
        const float all = team_sum(own);
        float dot = 0.0f;
        for (int i = tid; i < k; i += TEAM) dot += all > 0.0f ? u[i] * __fdiv_rn(s[i], all) : 0.0f;
        dot = team_sum(dot);
        for (int i = tid; i < k; i += TEAM) u[i] = all > 0.0f ? __fdiv_rn(u[i] - dot, all) : 0.0f;
    }
    float mean = 0.0f;
    if (dense) {
        for (int i = tid; i < k; i += TEAM) mean += u[i] * s[i];
        mean = team_sum(mean);
    }
    for (int j = tid; j < n; j += TEAM) {
        float d = 0.0f;
        if (dense && total > 0.0f) d = -mean * __fdiv_rn(exp_below(to_f32(__ldg(row + j)), m), total);
        out[j] = from_f32<L>(d);
    }
    sync();  // the chosen entries are written again, over what is there
    for (int i = tid; i < k; i += TEAM) {
        if (at[i] < 0) continue;
        out[at[i]] = from_f32<L>(!softmax ? u[i] * s[i] * (1.0f - s[i]) : dense ? s[i] * (u[i] - mean) : s[i] * u[i]);
    }
    (void)lane;
}

template <typename L>
const void* warp_kernel(int n) {
    return n <= 256   ? (const void*)route_warp_kernel<8, L>
           : n <= 512 ? (const void*)route_warp_kernel<16, L>
                      : (const void*)route_warp_kernel<32, L>;
}

}  // namespace

int launch_route(const RouteArgs& a0, cudaStream_t stream) {
    RouteArgs a = a0;
    if (a.n <= 1024 && a.k <= 32) {
        constexpr int WARPS = kWarpThreads / 32;
        const int64_t blocks = (a.tokens + WARPS - 1) / WARPS;
        if (blocks > INT_MAX) return SDM_ECOUNT;
        const bool grouped = a.n_groups > 1 && a.top_groups < a.n_groups;
        const size_t smem = grouped ? (size_t)WARPS * (a.n + a.n_groups) * 4 : 0;
        void* args[] = {&a};
        return launch_pdl_raw(a.logit_bf16 ? warp_kernel<uint16_t>(a.n) : warp_kernel<float>(a.n), dim3((unsigned)blocks),
                              dim3(kWarpThreads), smem, stream, args);
    }
    if (a.tokens > INT_MAX) return SDM_ECOUNT;
    int staged = (size_t)a.n * 4 <= kStagedBytes ? 1 : 0;
    const size_t smem = staged ? (size_t)a.n * 4 : 0;
    const bool large = a.n > 4096;
    const void* fn = a.logit_bf16 ? (large ? (const void*)route_block_kernel<512, uint16_t> : (const void*)route_block_kernel<128, uint16_t>)
                                  : (large ? (const void*)route_block_kernel<512, float> : (const void*)route_block_kernel<128, float>);
    // the limit without a request counts the kernel's static arrays (16 KB) too
    const int rc = allow_smem(fn, smem > 32 * 1024 ? std::max(smem, (size_t)48 * 1024 + 16) : smem);
    if (rc != 0) return rc;
    void* args[] = {&a, &staged};
    return launch_pdl_raw(fn, dim3((unsigned)a.tokens), dim3(large ? 512 : 128), smem, stream, args);
}

int launch_route_backward(const RouteArgs& a0, cudaStream_t stream) {
    RouteArgs a = a0;
    const bool warp = a.n <= 1024;
    const int64_t blocks = warp ? (a.tokens + 3) / 4 : a.tokens;
    if (blocks > INT_MAX) return SDM_ECOUNT;
    const void* fn = warp ? (a.logit_bf16 ? (const void*)route_backward_kernel<32, uint16_t> : (const void*)route_backward_kernel<32, float>)
                          : (a.logit_bf16 ? (const void*)route_backward_kernel<256, uint16_t> : (const void*)route_backward_kernel<256, float>);
    void* args[] = {&a};
    return launch_pdl_raw(fn, dim3((unsigned)blocks), dim3(warp ? 128 : 256), 0, stream, args);
}

int route_status(unsigned int* word, bool clear) {
    cudaError_t e = cudaMemcpyFromSymbol(word, g_route_status, sizeof(unsigned int));
    if (e == cudaSuccess && clear) {
        const unsigned int zero = 0;
        e = cudaMemcpyToSymbol(g_route_status, &zero, sizeof(unsigned int));
    }
    return (int)e;
}

}  // namespace sdm
