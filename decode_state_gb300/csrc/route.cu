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
// that reach it are few more than k; they are collected in shared memory and ranked by counting. With
// too few lanes for that, a warp halves the range of the ranks until few enough reach its lower end.
// Where they are too many (equal ranks), or fewer than k entries are not masked, a slower path
// follows that takes any ranks.
//
// route_warp_kernel (n <= 1024, k <= 64): a warp for each token, its ranks in registers, lane l the
// consecutive entries from l * E on, so that lane order is index order. Bound by instructions (an
// exponential and a reciprocal for every entry of a biased sigmoid), not by its 2 or 4 bytes; small
// rows get half a warp, which halves what is spent on a token rather than on its entries.
// route_block_kernel: a block for each token, its ranks staged in shared memory. The slower path
// narrows the k-th rank down by histograms of its leading 11, then 11, then 10 bits.
#include <algorithm>
#include <climits>
#include <type_traits>

#include "quant_device.cuh"
#include "score_device.cuh"
#include "sdm_internal.h"

namespace sdm {
namespace {

__device__ unsigned int g_route_status;

constexpr uint32_t kMasked = 1;
constexpr int kMaxGroups = 256, kMaxK = 256;
constexpr int kCandidates = 512;
constexpr size_t kStagedBytes = 192 * 1024;  // ranks a block keeps in shared memory

__device__ __forceinline__ float sigmoid(float x) { return masked(x) ? 0.0f : __frcp_rn(__fadd_rn(1.0f, expf(-x))); }

// Scores of N logits: sigmoid() bit by bit (any value for masked ones), but without a branch for each,
// so that they overlap. A reciprocal of a float in [1, 2^126] is correctly rounded by one Newton step from the
// hardware's approximation (the tests compare ranks with weights over [1, 2]); the rare others are done again.
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
    // a group's score: -inf for a group of masked entries
    __device__ __forceinline__ float value(int group_top) const {
        return group_top == 1 || b == minus_inf() ? a : a + b;
    }
};

// Whether group g is among the `top` best of scores[0 .. groups), ties to the lower index.
__device__ __forceinline__ bool group_stays(const float* scores, int groups, int top, int g) {
    const float mine = scores[g];
    int better = 0;
    for (int o = 0; o < groups; ++o) better += scores[o] > mine || (scores[o] == mine && o < g);
    return better < top;
}

// The float of an ordered integer from that of -inf to that of +inf; a NaN outside them.
__device__ __forceinline__ float unordered(uint32_t u) { return __uint_as_float(u & 0x80000000u ? u ^ 0x80000000u : ~u); }

// A candidate as 64 bits that order first by rank, then by the lower index.
__device__ __forceinline__ uint64_t candidate(uint32_t rank, int j) { return (uint64_t)rank << 32 | (uint32_t)~j; }
__device__ __forceinline__ int candidate_index(uint64_t c) { return (int)~(uint32_t)c; }

// The sum of `own` over the lanes of this lane's LANES before it, and over all of them.
template <int LANES>
__device__ __forceinline__ int lanes_before(int own, int* all) {
    const int l = threadIdx.x % LANES;
    int sum = own;
#pragma unroll
    for (int o = 1; o < LANES; o <<= 1) {
        const int y = __shfl_up_sync(kAll, sum, o, LANES);
        if (l >= o) sum += y;
    }
    *all = __shfl_sync(kAll, sum, LANES - 1, LANES);
    return sum - own;
}

// ---------------------------------------------------------------- a warp, or half of one, for each token

constexpr int kWarpThreads = 256;

// The k-th largest of V values on each of LANES lanes, on every lane: a bitonic sort, in falling order,
// value s of lane l at place l * V + s. Where a stage sorts in rising order the signs are turned, so
// that a step asks for one bit of the lane only.
template <int LANES, int V>
__device__ __forceinline__ float kth_of_lanes(float* x, int k) {
    static_assert(V == 1 || V == 2, "one or two values");
    const uint32_t l = threadIdx.x % LANES;
    uint32_t turned = 0;
#pragma unroll
    for (int size = 2; size <= LANES * V; size *= 2) {
        const uint32_t turn = size < LANES * V && (l & size / V) ? 0x80000000u : 0u;
#pragma unroll
        for (int v = 0; v < V; ++v) x[v] = __uint_as_float(__float_as_uint(x[v]) ^ turn ^ turned);
        turned = turn;
#pragma unroll
        for (int o = size / 2; o >= V; o /= 2) {
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float y = __shfl_xor_sync(kAll, x[v], o / V);
                x[v] = l & o / V ? fminf(x[v], y) : fmaxf(x[v], y);
            }
        }
        if (V == 2) {
            const float high = fmaxf(x[0], x[V - 1]);
            x[V - 1] = fminf(x[0], x[V - 1]);
            x[0] = high;
        }
    }
    return __shfl_sync(kAll, V == 2 && !(k & 1) ? x[V - 1] : x[0], (k - 1) / V, LANES);
}

template <int LANES>
__device__ __forceinline__ float lanes_max(float x) {
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(kAll, x, o));
    return x;
}

// A bound that at least k of a warp's ranks reach (E on each lane, -inf for masked ones; k <= 64), and at
// most `most` unless too many are equal; that of all ranks where no more are live. Halves the range
// between a bound that k reach and one that fewer do, by value and by the order of the floats in turn: the
// first is quick for ranks of one size, the second needs no more than 32 steps for any. At most a rank of
// each lane lies above all lanes' second largest, and at least two of each reach the least of those.
template <int E>
__device__ __forceinline__ float reached_by(const float* r, int k, int most) {
    Top2 top;
#pragma unroll
    for (int i = 0; i < E; ++i) top.add(r[i]);
    float low = k <= 32 ? top.a : top.b, high = low;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        low = fminf(low, __shfl_xor_sync(kAll, low, o));
        high = fmaxf(high, __shfl_xor_sync(kAll, high, o));
    }
    if (low == minus_inf()) {  // some lanes have too few: the least live rank
        low = 3.402823466e38f;
#pragma unroll
        for (int i = 0; i < E; ++i) low = fminf(low, r[i] == minus_inf() ? low : r[i]);
#pragma unroll
        for (int o = 16; o; o >>= 1) low = fminf(low, __shfl_xor_sync(kAll, low, o));
        high = lanes_max<32>(top.a);
    }
    const auto reaching = [&](float bound) {
        float c = 0.0f;  // a comparison gives 1 or 0 as a float in one instruction
#pragma unroll
        for (int i = 0; i < E; ++i) c += r[i] >= bound ? 1.0f : 0.0f;
        return __reduce_add_sync(kAll, (int)c);
    };
    int reach = reaching(low);
    for (int step = 0; reach > most; ++step) {
        float mid = 0.5f * low + 0.5f * high;
        if (step & 1 || !(mid > low && mid < high)) {
            const uint32_t a = ordered(low), b = ordered(high);
            if (b <= a + 1) break;  // neighbours
            mid = unordered(a + (b - a) / 2);
        }
        const int c = reaching(mid);
        if (c >= k) {
            low = mid;
            reach = c;
        } else {
            high = mid;
        }
    }
    return low;
}

template <int LANES>
__device__ __forceinline__ float lanes_sum(float x) {
#pragma unroll
    for (int o = LANES / 2; o; o >>= 1) x += __shfl_xor_sync(kAll, x, o);
    return x;
}

// A sigmoid from the hardware's approximations: within 2^-21 of the score (ex2 to 2^-22, its argument
// rounded once, rcp to 2^-23, and the score's own roundings).
__device__ __forceinline__ float rough_sigmoid(float x) {
    float e, r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.44269504f));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
    return r;
}

// LANES lanes work on a token, E entries each, the consecutive ones from l * E on, so that the order of
// the lanes is the order of the indices. V: maxima of a lane's entries that the bound is taken from. L: uint16_t (bf16) or float logits.
//
// The ranks of a sigmoid are first computed roughly, with a margin, at a third of the instructions;
// what is near enough to matter is computed exactly: the candidates, and all entries where two groups
// are too close to call.
//
// Bound by instructions and the latencies between them: 65536 rows of 256 by sigmoid, bias and groups, k = 8, take
// some 1070 instructions for two tokens, 0.74 a cycle and scheduler, at a tenth of the DRAM's rate. So the registers are
// bounded for 4 to 6 blocks an SM: 45 -> 39 us; 32768 rows of 1000 float32, k = 64, 221 -> 140 (4 blocks; 6: 158).
template <int LANES, int E, int V, bool SOFTMAX, typename L>
__global__ void __launch_bounds__(kWarpThreads, E == 32 ? 4 : E == 16 ? 5 : 6) route_warp_kernel(const RouteArgs a) {
    constexpr int TEAMS = kWarpThreads / LANES, Q = V == 0 ? 3 : 2, CANDS = Q * LANES;  // Q: candidates of a lane at most
    extern __shared__ float staged[];  // groups that are no whole lanes: every team's group values [n] and scores [n_groups]
    __shared__ uint16_t found[TEAMS][CANDS];
    grid_dependency_wait();
    grid_launch_dependents();
    const int l = threadIdx.x % LANES, team = threadIdx.x / LANES, first_lane = threadIdx.x % 32 / LANES * LANES;
    const int64_t token = (int64_t)blockIdx.x * TEAMS + team;
    if (token - (threadIdx.x % 32) / LANES >= a.tokens) return;  // a whole warp
    const bool there = token < a.tokens;
    const int64_t t = there ? token : a.tokens - 1;  // spare teams work along on the last token, and write nothing
    const int n = a.n, k = a.k, j0 = l * E;
    const uint32_t team_bits = LANES == 32 ? kAll : (1u << LANES % 32) - 1u;
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

    constexpr bool softmax = SOFTMAX;
    const bool biased = a.bias != nullptr;
    const bool grouped = a.n_groups > 1 && a.top_groups < a.n_groups, by_sum = grouped && a.group_top == 2;
    const bool by_exp = by_sum && softmax && !biased;  // groups judged by exp(x - m), not by the ranks
    float m = minus_inf(), total = 1.0f;
    if (softmax) {
#pragma unroll
        for (int i = 0; i < E; ++i) m = fmaxf(m, x[i]);  // NaN takes no part
        m = lanes_max<LANES>(m);
        if (biased || !a.renorm) {
            total = 0.0f;
#pragma unroll
            for (int i = 0; i < E; ++i) total += exp_below(x[i], m);
            total = lanes_sum<LANES>(total);
        }
    }
    const int per = n / a.n_groups, group_lanes = per / E;
    const bool by_lanes = per % E == 0 && group_lanes <= LANES && (group_lanes & (group_lanes - 1)) == 0;
    bool rough = !softmax && (!grouped || by_lanes);

    // ranks, -inf where masked
    float r[E];
    const auto add_bias = [&]() {
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
    };
    const auto exact_ranks = [&]() {
        if (!softmax) {
            sigmoids<E>(x, r);
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) r[i] = biased ? __fdiv_rn(exp_below(x[i], m), total) : x[i];
        }
        if (biased) add_bias();
#pragma unroll
        for (int i = 0; i < E; ++i) r[i] = masked(x[i]) ? minus_inf() : fmaxf(r[i], minus_inf());  // the number of the two
    };
    if (rough) {
#pragma unroll
        for (int i = 0; i < E; ++i) r[i] = rough_sigmoid(x[i]);
        if (biased) add_bias();
#pragma unroll
        for (int i = 0; i < E; ++i) r[i] = masked(x[i]) ? minus_inf() : fmaxf(r[i], minus_inf());
    } else {
        exact_ranks();
    }
    const auto margin = [](float at) { return fmaf(fabsf(at), 0x1p-20f, 0x1p-18f); };  // eight errors, for differences of sums of two

    if (grouped && by_lanes) {
        // groups of whole lanes, a power of two of them
        const auto judge = [&]() {
            Top2 top;
#pragma unroll
            for (int i = 0; i < E; ++i) top.add(by_exp ? (r[i] == minus_inf() ? minus_inf() : exp_below(x[i], m)) : r[i]);
            for (int o = 1; o < group_lanes; o <<= 1) top.join(__shfl_xor_sync(kAll, top.a, o), __shfl_xor_sync(kAll, top.b, o));
            return top.value(a.group_top);
        };
        const int g = l / group_lanes;
        float mine = judge();
        int better = 0, near = 0;  // groups that are surely better; and those that may be
        if (rough) {
            // an infinite score (a bias) is exact: no margin, so that equal ones are near
            const float d = fabsf(mine) <= 3.402823466e38f ? margin(mine) : 0.0f, high = mine + d, low = mine - d;
            for (int q = 0, from = 0; q < a.n_groups; ++q, from += group_lanes) {
                const float other = __shfl_sync(kAll, mine, from, LANES);
                better += other > high;
                near += other >= low;
            }
            --near;  // the group itself
        }
        if (!rough || __any_sync(kAll, better < a.top_groups && near >= a.top_groups)) {
            if (rough) {
                exact_ranks();
                mine = judge();
                rough = false;
            }
            better = 0;
            for (int q = 0; q < a.n_groups; ++q) {
                const float other = __shfl_sync(kAll, mine, q * group_lanes, LANES);
                better += other > mine || (other == mine && q < g);
            }
        }
        if (better >= a.top_groups) {
#pragma unroll
            for (int i = 0; i < E; ++i) r[i] = minus_inf();
        }
    } else if (grouped) {
        float* value = staged + (size_t)team * (n + LANES + a.n_groups);
        float* scores = value + n + LANES;
        const auto place = [](int j) { return j + j / E; };  // lanes' entries are one bank apart
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (j0 + i < n) value[place(j0 + i)] = by_exp ? (r[i] == minus_inf() ? minus_inf() : exp_below(x[i], m)) : r[i];
        __syncwarp();
        int share = 1;  // lanes of a group
        while (2 * share * a.n_groups <= LANES && 2 * share <= per) share *= 2;
        for (int g0 = 0; g0 < a.n_groups; g0 += LANES / share) {
            const int g = g0 + l / share, from = l % share;
            Top2 top;
            if (g < a.n_groups) {
                const int own = (per - from + share - 1) / share;
                int i = g % own;  // groups start apart, since they are often a multiple of the banks long
                for (int left = own; left > 0; --left) {
                    top.add(value[place(g * per + from + i * share)]);
                    i = i + 1 == own ? 0 : i + 1;
                }
            }
            for (int o = 1; o < share; o <<= 1) top.join(__shfl_xor_sync(kAll, top.a, o), __shfl_xor_sync(kAll, top.b, o));
            if (g < a.n_groups && from == 0) scores[g] = top.value(a.group_top);
        }
        __syncwarp();
        uint32_t* stays = reinterpret_cast<uint32_t*>(value);  // the values have been read
        for (int g = l; g < a.n_groups; g += LANES) stays[g] = group_stays(scores, a.n_groups, a.top_groups, g);
        __syncwarp();
        int g = j0 / per, left = per - j0 % per;
#pragma unroll
        for (int i = 0; i < E; ++i) {
            if (j0 + i < n && !stays[g]) r[i] = minus_inf();
            if (--left == 0) {
                ++g;
                left = per;
            }
        }
    }

    // a bound that k entries reach at least, and few more
    float bound;
    if constexpr (V == 0) {
        static_assert(LANES == 32, "a warp for each token");
        bound = reached_by<E>(r, k, CANDS);
    } else {
        // the k-th largest of the maxima of the lanes' entries (V 2: of both halves of them)
        float best[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            best[v] = r[v * (E / V)];
#pragma unroll
            for (int i = 1; i < E / V; ++i) best[v] = fmaxf(best[v], r[v * (E / V) + i]);
        }
        bound = kth_of_lanes<LANES, V>(best, k);
    }
    if (rough && bound > minus_inf()) bound -= margin(bound);
    bound = fmaxf(bound, -3.402823466e38f);  // masked entries never reach it
    uint32_t reach = 0;  // bit i: entry i does
#pragma unroll
    for (int i = 0; i < E; ++i) reach |= r[i] >= bound ? 1u << i : 0u;
    int count;
    int at = lanes_before<LANES>(__popc(reach), &count);
    uint16_t* cand = found[team];
    if (__any_sync(kAll, count > CANDS)) {
        // too many alike: k rounds of a maximum over the lanes, the lowest index first
        if (rough) {
            uint32_t gone = 0;
#pragma unroll
            for (int i = 0; i < E; ++i) gone |= r[i] == minus_inf() ? 1u << i : 0u;
            exact_ranks();
#pragma unroll
            for (int i = 0; i < E; ++i)
                if (gone >> i & 1u) r[i] = minus_inf();
        }
        uint32_t live = 0, taken = 0;
#pragma unroll
        for (int i = 0; i < E; ++i) live |= r[i] > minus_inf() ? 1u << i : 0u;
        int all;
        lanes_before<LANES>(__popc(live), &all);
        count = min(k, all);
        for (int round = 0; round < k; ++round) {
            float own = minus_inf();
#pragma unroll
            for (int i = 0; i < E; ++i) own = taken >> i & 1u ? own : fmaxf(own, r[i]);
            const float top = lanes_max<LANES>(own);
            const uint32_t holders = __ballot_sync(kAll, own == top) >> first_lane & team_bits;
            if (round < count && l == __ffs(holders) - 1) {
                uint32_t hit = 0;
#pragma unroll
                for (int i = 0; i < E; ++i) hit |= r[i] == top ? 1u << i : 0u;
                const int i = __ffs(hit & ~taken) - 1;
                taken |= 1u << i;
                cand[round] = (uint16_t)(j0 + i);
            }
        }
    } else {
        for (; reach; reach &= reach - 1) cand[at++] = (uint16_t)(j0 + __ffs(reach) - 1);
    }
    __syncwarp();
    // exact ranks of the candidates; where they were collected their order is that of the indices,
    // and where they were taken in rounds it is that of the ranks: equal ranks go by the place
    int j[Q], rank[Q];
    float score[Q], key[Q];
    bool some[Q];  // whether a lane has a candidate q
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        rank[q] = 0;
        score[q] = 0.0f;
        key[q] = minus_inf();
        some[q] = q == 0 || __any_sync(kAll, count > LANES * q);
        if (some[q] && l + LANES * q < count) {
            j[q] = cand[l + LANES * q];
            const float y = to_f32(__ldg(row + j[q]));
            score[q] = softmax ? exp_below(y, m) : sigmoid(y);
            key[q] = !softmax ? score[q] : biased ? __fdiv_rn(score[q], total) : y;
            if (biased) key[q] += __ldg(a.bias + j[q]);
        }
    }
    const int most = LANES == 32 ? count : max(count, __shfl_xor_sync(kAll, count, 16));
#pragma unroll
    for (int p = 0; p < Q; ++p) {
        const int end = min(LANES, most - LANES * p);
        for (int o0 = 0; o0 < end; o0 += 4) {
#pragma unroll
            for (int o = o0; o < o0 + 4; ++o) {
                const float other = __shfl_sync(kAll, key[p], o, LANES);  // -inf behind the last one: better than none
#pragma unroll
                for (int q = 0; q < Q; ++q)
                    if (some[q]) rank[q] += other > key[q] || (other == key[q] && (p == q ? o < l : p < q));
            }
        }
    }
    bool mine[Q];
    float chosen = 0.0f;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        mine[q] = some[q] && l + LANES * q < count && rank[q] < k;
        if (mine[q]) chosen += score[q];
    }
    if (a.renorm) total = lanes_sum<LANES>(chosen);
    // a share of the total first: scale / total overflows where all that are chosen have tiny scores
    const bool shares = (softmax || a.renorm) && total > 0.0f;
    if (!there) return;
    const int64_t to = t * k;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
        if (mine[q]) {
            put_index(a, t, rank[q], j[q]);
            a.w[to + rank[q]] = (shares ? __fdiv_rn(score[q], total) : score[q]) * a.scale;
        }
    }
    if (count < k) {  // fill up with masked entries, in index order
        uint32_t gone = 0;
#pragma unroll
        for (int i = 0; i < E; ++i) gone |= j0 + i < n && r[i] == minus_inf() ? 1u << i : 0u;
        const int own = __popc(gone);
        at = count;
        for (int o = 0; o < LANES; ++o) {
            const int y = __shfl_sync(team_bits << first_lane, own, o, LANES);
            if (o < l) at += y;
        }
        for (; gone && at < k; gone &= gone - 1, ++at) {
            put_index(a, t, at, j0 + __ffs(gone) - 1);
            a.w[to + at] = 0.0f;
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

// PLAIN: a softmax without bias and groups, whose ranks are the logits.
// The steps of a block wait for one another, so blocks are many: the registers are bounded for 12 of 128
// threads, 5 of 256, or 3 of 512 (16384 rows of 1500, k = 8: 78 us with 4 blocks as the bound, 45 with 12; 2048 of
// 8000 23 with 3, 18 with 5). What is left is latency and instructions, of the candidates' ranking by counting most.
template <int NT, bool PLAIN, typename L>
__global__ void __launch_bounds__(NT, NT == 512 ? 3 : NT == 256 ? 5 : 12) route_block_kernel(const RouteArgs a, int staged) {
    constexpr int WARPS = NT / 32;
    extern __shared__ __align__(16) float staging[];  // [n + 4] when staged
    __shared__ __align__(16) int hist[kBins];
    // the histogram has been read when candidates are collected and chosen
    uint64_t* cand = reinterpret_cast<uint64_t*>(hist);                     // [kCandidates]
    int* sel_j = hist + 2 * kCandidates;                                    // [kMaxK]
    float* sel_s = reinterpret_cast<float*>(hist + 2 * kCandidates + kMaxK);  // [kMaxK]
    static_assert(2 * kCandidates + 2 * kMaxK <= kBins, "they fit the histogram");
    __shared__ float scores[kMaxGroups];
    __shared__ uint32_t stays[kMaxGroups / 32];
    __shared__ float tmp[WARPS];
    __shared__ float ends[2 * WARPS];  // not in tmp: no barrier is behind the last reads of a sum there
    __shared__ int counts[WARPS];
    __shared__ int found_bin, found_above, n_cand;
    grid_dependency_wait();
    grid_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t t = blockIdx.x;
    const int n = a.n, k = a.k;
    const bool softmax = PLAIN || a.score == SDM_SOFTMAX, biased = !PLAIN && a.bias != nullptr;
    const bool grouped = !PLAIN && a.n_groups > 1 && a.top_groups < a.n_groups;
    const int per = n / a.n_groups;
    const L* row = static_cast<const L*>(a.logits) + t * a.row_stride;
    constexpr int V = 16 / sizeof(L);  // logits of a 16-byte load
    // the row's first logit at a 16-byte boundary; ranks + j is at one where row + j is
    const int head = min(n, (int)((16 - reinterpret_cast<uintptr_t>(row) % 16) % 16 / sizeof(L)));
    float* ranks = staging + (4 - head % 4) % 4;

    // f(j, x, count) for `count` logits x from j on, V or one, all in all every one
    const auto each = [&](const auto& f) {
        const auto piece = [&](int j, const uint4& v) {
            float x[V];
            if constexpr (sizeof(L) == 2)
                unpack<Bf16>(v, x);
            else
                unpack<F32>(v, x);
            f(j, x, V);
        };
        const int end = head + (n - head) / V * V;
        int j = head + tid * V;
        for (; j + 3 * NT * V < end; j += 4 * NT * V) {  // four loads on their way together
            uint4 v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) v[u] = __ldg(reinterpret_cast<const uint4*>(row + j + u * NT * V));
#pragma unroll
            for (int u = 0; u < 4; ++u) piece(j + u * NT * V, v[u]);
        }
        {  // and the up to four that are left
            uint4 v[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) v[u] = load16_if(row + j + u * NT * V, j + u * NT * V < end);
#pragma unroll
            for (int u = 0; u < 4; ++u)
                if (j + u * NT * V < end) piece(j + u * NT * V, v[u]);
        }
        // the few before the first boundary and behind the last one
        const int rest = head + n - end;
        if (tid < rest) {
            j = tid < head ? tid : end + tid - head;
            float x[V] = {to_f32(__ldg(row + j))};
            f(j, x, 1);
        }
    };

    float m = minus_inf(), total = 1.0f;
    if (!PLAIN && softmax && (biased || !a.renorm || (grouped && a.group_top == 2))) {
        each([&](int, const float* x, int count) {
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (i < count) m = fmaxf(m, x[i]);
        });
        m = block_reduce(m, false, tmp, WARPS);
        if (biased || !a.renorm) {
            total = 0.0f;
            for (int j = tid; j < n; j += NT) total += exp_below(to_f32(__ldg(row + j)), m);  // in one order, wherever the row starts
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
            if (lane == 0) scores[g] = top.value(a.group_top);
        }
        __syncthreads();
        for (int g0 = warp * 32; g0 < a.n_groups; g0 += NT) {
            const int g = g0 + lane;
            const uint32_t b = __ballot_sync(kAll, g < a.n_groups && group_stays(scores, a.n_groups, a.top_groups, g));
            if (lane == 0) stays[g0 / 32] = b;
        }
        __syncthreads();
    }
    const auto stays_at = [&](int j) {
        const int g = j / per;
        return ((stays[g >> 5] >> (g & 31)) & 1u) != 0;
    };
    // the ranks of V entries from j on, or of one, -inf where they are masked
    const auto final_ranks = [&](int j, const float* x, int count, float* r) {
        if (PLAIN || softmax) {
#pragma unroll
            for (int i = 0; i < V; ++i) r[i] = !biased ? x[i] : i < count ? rank_of(j + i, x[i]) : 0.0f;
        } else {
            sigmoids<V>(x, r);
#pragma unroll
            for (int i = 0; i < V; ++i) r[i] = masked(x[i]) ? minus_inf() : r[i];
            if (biased) {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (i < count) r[i] += __ldg(a.bias + j + i);
            }
        }
#pragma unroll
        for (int i = 0; i < V; ++i) r[i] = i < count ? fmaxf(r[i], minus_inf()) : minus_inf();  // the number of the two
        if (grouped) {
            if (per % V == 0 && head == 0) {  // a group, or none, for all of them
                const bool on = stays_at(j);
#pragma unroll
                for (int i = 0; i < V; ++i) r[i] = on ? r[i] : minus_inf();
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (i < count && !stays_at(j + i)) r[i] = minus_inf();
            }
        }
    };
    float best = minus_inf();  // the largest rank of this thread's entries
    each([&](int j, const float* x, int count) {
        float r[V];
        final_ranks(j, x, count, r);
#pragma unroll
        for (int i = 0; i < V; ++i) best = fmaxf(best, r[i]);
        if (!staged) return;
        if (count == V) {
#pragma unroll
            for (int i = 0; i < V; i += 4) *reinterpret_cast<float4*>(ranks + j + i) = make_float4(r[i], r[i + 1], r[i + 2], r[i + 3]);
        } else {
            ranks[j] = r[0];
        }
    });
    const auto rank_at = [&](int j) {
        if (staged) return ranks[j];
        float x[V] = {to_f32(__ldg(row + j))}, r[V];
        final_ranks(j, x, 1, r);
        return r[0];
    };
    if (PLAIN && !a.renorm) {  // the ranks are the logits
        m = block_reduce(best, false, tmp, WARPS);
        total = 0.0f;
        for (int j = tid; j < n; j += NT) total += exp_below(rank_at(j), m);
        total = block_reduce(total, true, tmp, WARPS);
    }
    const auto key_at = [&](int j) { return ordered(rank_at(j)); };

    // the bin of the need-th largest of the values counted in hist, from the top: found_bin (-1: there
    // are fewer), and found_above, those in higher bins; counts holds the warps' shares of all of them
    const auto find_bin = [&](int need, auto bins) {
        constexpr int BINS = decltype(bins)::value, PER = BINS / NT;  // thread i owns the PER bins from i * PER on, counted from the top
        int own = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) own += hist[BINS - 1 - (tid * PER + i)];
        int all;
        int before = lanes_before<32>(own, &all);
        if (lane == 31) counts[warp] = all;
        if (tid == 0) found_bin = -1;
        __syncthreads();
        for (int i = 0; i < warp; ++i) before += counts[i];
        if (before < need && before + own >= need) {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                const int b = BINS - 1 - (tid * PER + i), c = hist[b];
                if (before < need && before + c >= need) {
                    found_bin = b;
                    found_above = before;
                }
                before += c;
            }
        }
        __syncthreads();
    };
    const auto clear_bins = [&](int bins) {
        for (int b = tid; b < bins; b += NT) hist[b] = 0;
        __syncthreads();
    };
    constexpr int kFew = 2 * NT;  // bins for the threads' maxima
    // candidates: the live entries with a rank from `bound` on, or above it; those that fit are kept
    // (the key behind that of +inf is no rank's: what lies above a rank is asked of the rank itself)
    const auto collect = [&](float bound, bool above) {
        if (tid == 0) n_cand = 0;
        __syncthreads();
        bound = fmaxf(bound, -3.402823466e38f);  // -inf is no live entry's rank
        const auto keep = [&](float r, int j) {
            if (above ? r > bound : r >= bound) {
                const int c = atomicAdd(&n_cand, 1);
                if (c < kCandidates) cand[c] = candidate(ordered(r), j);
            }
        };
        if (staged) {
            const int first = head % 4, whole = first + (n - first) / 4 * 4;
            for (int j = first + tid * 4; j < whole; j += NT * 4) {
                const float4 v = *reinterpret_cast<const float4*>(ranks + j);
                if (fmaxf(fmaxf(v.x, v.y), fmaxf(v.z, v.w)) >= bound) keep(v.x, j), keep(v.y, j + 1), keep(v.z, j + 2), keep(v.w, j + 3);
            }
            const int rest = first + n - whole;
            if (tid < rest) {
                const int j = tid < first ? tid : whole + tid - first;
                keep(ranks[j], j);
            }
        } else {
            for (int j = tid; j < n; j += NT) keep(rank_at(j), j);
        }
        __syncthreads();
    };

    // a lower bound by the threads' maxima: the bin of the k-th largest of them among bins of equal width
    // from the least to the greatest
    float low = best > minus_inf() ? best : 3.402823466e38f, high = best;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        low = fminf(low, __shfl_xor_sync(kAll, low, o));
        high = fmaxf(high, __shfl_xor_sync(kAll, high, o));
    }
    if (lane == 0) {
        ends[warp] = low;
        ends[WARPS + warp] = high;
    }
    clear_bins(kFew);
    for (int i = 0; i < WARPS; ++i) {
        low = fminf(low, ends[i]);
        high = fmaxf(high, ends[WARPS + i]);
    }
    const float width = (high - low) * (1.0f / kFew);
    const bool spread = width > 0x1p-100f && width < 0x1p100f;
    if (best > minus_inf()) atomicAdd(&hist[spread ? min(kFew - 1, (int)__fdividef(best - low, width)) : 0], 1);
    __syncthreads();
    find_bin(k, std::integral_constant<int, kFew>{});
    bool done = false, few = false, ties = false;
    uint32_t lowest = 0;
    int C = 0;
    if (found_bin >= 0) {
        // one bin lower, for the roundings
        collect(spread && found_bin > 0 ? fmaf((float)(found_bin - 1), width, low) : low, false);
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
            clear_bins(kBins);
            for (int j = tid; j < n; j += NT) {
                const uint32_t key = key_at(j);
                if (key > kMasked && (level == 0 || key >> (shift + bits) == prefix))
                    atomicAdd(&hist[(key >> shift) & ((1u << bits) - 1u)], 1);
            }
            __syncthreads();
            find_bin(need, std::integral_constant<int, kBins>{});
            if (found_bin < 0) {  // level 0 only: all live entries are taken
                few = true;
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
        collect(few ? minus_inf() : unordered(lowest), ties);
        C = min(n_cand, kCandidates);
    }
    // rank the candidates by counting, four threads for each
    for (int c0 = 0; c0 < C; c0 += NT / 4) {
        const int c = c0 + tid / 4;
        const uint64_t mine = c < C ? cand[c] : 0;
        int better = 0;
#pragma unroll 4
        for (int o = tid % 4; o < C; o += 4) better += cand[o] > mine;
        better += __shfl_xor_sync(kAll, better, 1);
        better += __shfl_xor_sync(kAll, better, 2);
        if (c < C && better < k && tid % 4 == 0) {
            sel_j[better] = candidate_index(mine);
            sel_s[better] = PLAIN ? unordered((uint32_t)(mine >> 32)) : to_f32(__ldg(row + candidate_index(mine)));
        }
    }
    __syncthreads();
    if (softmax && !biased && a.renorm && C > 0) m = sel_s[0];  // any reference does: it cancels
    __syncthreads();
    for (int i = tid; i < min(C, k); i += NT) sel_s[i] = softmax ? exp_below(sel_s[i], m) : sigmoid(sel_s[i]);
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

// Blocks an SM that the registers are bounded for: a token's steps wait for memory and for one another, so
// tokens have to be many, as long as their rows fit the registers. Softmax without renormalisation, k = 8:
// 65536 rows of 256 float32 39 us with 12 blocks, 47 with 8, 52 unbounded; 32768 of 500 29, 32, 42; 16384 of 1000 34, 25, 33
// (it spills with 12); 2048 of 8000 28 with 4 blocks, 32 with 3, 40 unbounded; 1024 of 16384 33 with 2, 48 unbounded.
// Teams of 128 threads for rows up to 6144: 8192 rows of 1500 26 us, on 256 threads 52; 4097 of 4099 29 and 40.
constexpr int backward_blocks(int team, int e) {
    return team <= 128 ? (e <= 16 ? 12 : 8) : team == 256 ? (e == 0 ? 6 : 4) : 2;
}

// A team of TEAM threads (a warp, or a block) for each token. Only a softmax that is not
// renormalised has gradients outside the chosen entries: its row is read once, E logits a thread, and
// its exponentials stay in registers until the gradients are written (E 0: rows too long for that are
// read three times). All others get zeros there. The chosen entries are written over that.
template <int TEAM, int E, typename L>
__global__ void __launch_bounds__(TEAM == 32 ? 128 : TEAM, backward_blocks(TEAM, E)) route_backward_kernel(const RouteArgs a) {
    constexpr int NT = TEAM == 32 ? 128 : TEAM, TEAMS = NT / TEAM, WARPS = TEAM / 32, U = 4 / sizeof(L);
    __shared__ float largest[NT / 32], sums[NT / 32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int team = threadIdx.x / TEAM, tid = threadIdx.x % TEAM, lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * TEAMS + team;
    if (t >= a.tokens) return;  // a whole team
    const int n = a.n, k = a.k;
    const L* row = static_cast<const L*>(a.logits) + t * a.row_stride;
    L* out = static_cast<L*>(a.dlogits) + t * a.dlogits_stride;
    const bool softmax = a.score == SDM_SOFTMAX, dense = softmax && !a.renorm;
    // Thread tid works on the U logits of 4 bytes from (p * TEAM + tid) * U on, p = 0, 1, ...: runs of 128
    // bytes for a warp, and one order of the sums wherever the row starts.
    const bool words = U == 1 || ((reinterpret_cast<uintptr_t>(row) | reinterpret_cast<uintptr_t>(out)) & 3u) == 0;

    const auto sync = [] {
        if constexpr (TEAM == 32)
            __syncwarp();
        else
            __syncthreads();
    };
    // the largest value m of the team's threads, with the sum of their `own` sums of exp(x - their m)
    const auto join = [&](float& m, float& own) {
        const float mine = m;
        m = warp_max(m);
        own = warp_sum(mine == m ? own : own * exp_below(mine, m));
        if constexpr (TEAM > 32) {
            if (lane == 0) {
                largest[tid >> 5] = m;
                sums[tid >> 5] = own;
            }
            __syncthreads();
            own = 0.0f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) m = fmaxf(m, largest[w]);
#pragma unroll
            for (int w = 0; w < WARPS; ++w) own += sums[w] * exp_below(largest[w], m);
        }
    };
    // chosen entry i: its column (-1: outside the row), its logit and the gradient of its weight. A weight that
    // is 0 whatever the logits are has no gradient, and its dw, which may be anything, takes no part: that of a
    // masked entry, of an index outside the row and, with the forward's weights, of an entry of weight 0. All of
    // them get a masked logit here.
    const auto chosen = [&](int i, float& x, float& dw) {
        const int64_t e = t * k + i;
        const float given = __ldg(a.dw + e) * a.scale;  // on its way beside the index
        const int64_t j = (a.idx64 ? __ldg(static_cast<const int64_t*>(a.idx) + e) : __ldg(static_cast<const int32_t*>(a.idx) + e)) -
                          (a.base == nullptr ? 0 : a.idx64 ? __ldg(static_cast<const int64_t*>(a.base) + t) : __ldg(static_cast<const int32_t*>(a.base) + t));
        const bool in = j >= 0 && j < n;
        const bool filled = a.w != nullptr && __ldg(a.w + e) == 0.0f;
        x = in && !filled ? to_f32(__ldg(row + j)) : minus_inf();
        dw = masked(x) ? 0.0f : given;
        return in ? (int)j : -1;
    };
    const auto get = [&](int j, float* x) {  // U logits from j on; masked ones behind the end
        if (U == 2 && words && j + U <= n) {
            const uint32_t w = __ldg(reinterpret_cast<const uint32_t*>(row + j));
            x[0] = __uint_as_float(w << 16);
            x[U - 1] = __uint_as_float(w & 0xffff0000u);
        } else {
#pragma unroll
            for (int c = 0; c < U; ++c) x[c] = j + c < n ? to_f32(__ldg(row + j + c)) : minus_inf();
        }
    };
    const auto put = [&](int j, const float* d) {  // U gradients from j on
        if (U == 2 && words && j + U <= n) {
            const __nv_bfloat162 b = __floats2bfloat162_rn(d[0], d[U - 1]);
            *reinterpret_cast<uint32_t*>(out + j) = *reinterpret_cast<const uint32_t*>(&b);
        } else {
#pragma unroll
            for (int c = 0; c < U; ++c)
                if (j + c < n) out[j + c] = from_f32<L>(d[c]);
        }
    };

    // every warp has the first chosen entries at hand, loaded while the row is on its way
    constexpr int KEPT = 1;
    int kept_j[KEPT];
    float kept_x[KEPT], kept_dw[KEPT];
#pragma unroll
    for (int q = 0; q < KEPT; ++q) {
        kept_j[q] = -1;
        kept_x[q] = minus_inf();
        kept_dw[q] = 0.0f;
        if (lane + 32 * q < k && (dense || tid < 32)) kept_j[q] = chosen(lane + 32 * q, kept_x[q], kept_dw[q]);
    }
    // f(j, x, dw) for this lane's chosen entries
    const auto each_chosen = [&](const auto& f) {
#pragma unroll
        for (int q = 0; q < KEPT; ++q)
            if (lane + 32 * q < k) f(kept_j[q], kept_x[q], kept_dw[q]);
        for (int i = lane + 32 * KEPT; i < k; i += 32) {
            float y, dw;
            const int j = chosen(i, y, dw);
            f(j, y, dw);
        }
    };

    float m = minus_inf(), total = 0.0f, mean = 0.0f, factor = 0.0f;
    float x[E > 0 ? E : 1];
    if (dense) {
        float own = 0.0f, rescale = 1.0f;
        if constexpr (E > 0) {
#pragma unroll
            for (int i = 0; i < E; i += U) get((i / U * TEAM + tid) * U, x + i);
#pragma unroll
            for (int i = 0; i < E; ++i) {
                x[i] = fmaxf(x[i], minus_inf());  // NaN is masked
                m = fmaxf(m, x[i]);
            }
            const bool plain = fabsf(m) <= 3.402823466e38f;  // neither +inf nor masked throughout
            if (plain) {
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    x[i] = expf(x[i] - m);
                    own += x[i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < E; ++i) {
                    x[i] = exp_below(x[i], m);
                    own += x[i];
                }
            }
            const float mine = m;
            join(m, own);
            rescale = exp_below(mine, m);  // x holds exp(logit - mine)
        } else {
            for (int j = tid; j < n; j += TEAM) m = fmaxf(m, to_f32(__ldg(row + j)));
            for (int j = tid; j < n; j += TEAM) own += exp_below(to_f32(__ldg(row + j)), m);
            join(m, own);
        }
        total = own;
        // every warp for itself: a barrier would cost more
        each_chosen([&](int, float y, float dw) { mean += dw * exp_below(y, m); });
        mean = total > 0.0f ? __fdiv_rn(warp_sum(mean), total) : 0.0f;
        factor = total > 0.0f ? __fdiv_rn(-mean, total) : 0.0f;
        if constexpr (E > 0) {
            rescale *= factor;
#pragma unroll
            for (int i = 0; i < E; ++i) x[i] *= rescale;
#pragma unroll
            for (int i = 0; i < E; i += U) put((i / U * TEAM + tid) * U, x + i);
        } else {
            for (int j = tid; j < n; j += TEAM) out[j] = from_f32<L>(factor * exp_below(to_f32(__ldg(row + j)), m));
        }
    } else {
        // zeros, 16 bytes at a time between the boundaries in the row
        constexpr int V = 16 / sizeof(L);
        const int head = min(n, (int)((16 - reinterpret_cast<uintptr_t>(out) % 16) % 16 / sizeof(L)));
        const int end = head + (n - head) / V * V, rest = head + n - end;
        for (int j = head + tid * V; j < end; j += TEAM * V) *reinterpret_cast<uint4*>(out + j) = make_uint4(0u, 0u, 0u, 0u);
        if (tid < rest) out[tid < head ? tid : end + tid - head] = L(0);
    }
    // the chosen entries are written again, over what is there, by the team's first warp
    float all = 1.0f, dot = 0.0f;
    const auto score_of = [&](float y) { return softmax ? exp_below(y, m) : sigmoid(y); };
    // shares of the sum, not its reciprocal, which overflows where all that are chosen have tiny scores
    const auto share_of = [&](float s) { return all > 0.0f ? __fdiv_rn(s, all) : 0.0f; };
    if (a.renorm && tid < 32) {
        // scores, or exp(x - m) for a softmax, which is as good: the factor between them cancels
        if (softmax) {
            each_chosen([&](int, float y, float) { m = fmaxf(m, y); });
            m = warp_max(m);
        }
        all = 0.0f;
        each_chosen([&](int, float y, float dw) {
            const float s = score_of(y);
            all += s;
            dot = fmaf(dw, s * 0x1p32f, dot);  // products of tiny scores keep their bits
        });
        all = warp_sum(all);
        dot = all > 0.0f ? __fdiv_rn(warp_sum(dot), all * 0x1p32f) : 0.0f;
    }
    sync();
    if (tid >= 32) return;
    each_chosen([&](int j, float y, float dw) {
        if (masked(y)) {  // what is there stays: 0, or in a dense row that of an entry not chosen
            if (j < 0) atomicOr(&g_route_status, SDM_DEV_BAD_INDEX);
            return;
        }
        const float s = score_of(y);
        float d;
        if (dense)
            d = total > 0.0f ? __fdiv_rn(s, total) * (dw - mean) : 0.0f;
        else
            d = (a.renorm ? (dw - dot) * share_of(s) : dw * s) * (softmax ? 1.0f : 1.0f - s);
        out[j] = from_f32<L>(d);
    });
}

struct Team {
    const void* fn;
    int threads, teams;
};

// Teams with 8 to 48 logits a thread where the row is kept; without a row to keep, and beyond 1024 entries, of 128 or 256 threads.
template <typename L>
Team backward_kernel(int n, bool dense) {
    if (n <= 256) return {(const void*)route_backward_kernel<32, 8, L>, 128, 4};
    if (n <= 512) return {(const void*)route_backward_kernel<32, 16, L>, 128, 4};
    if (n <= 1024) return {(const void*)route_backward_kernel<32, 32, L>, 128, 4};
    if (!dense && n <= 4096) return {(const void*)route_backward_kernel<128, 0, L>, 128, 1};
    if (!dense) return {(const void*)route_backward_kernel<256, 0, L>, 256, 1};
    if (n <= 2048) return {(const void*)route_backward_kernel<128, 16, L>, 128, 1};
    if (n <= 4096) return {(const void*)route_backward_kernel<128, 32, L>, 128, 1};
    if (n <= 5120) return {(const void*)route_backward_kernel<128, 40, L>, 128, 1};
    if (n <= 6144) return {(const void*)route_backward_kernel<128, 48, L>, 128, 1};
    if (n <= 8192) return {(const void*)route_backward_kernel<256, 32, L>, 256, 1};
    if (n <= 16384) return {(const void*)route_backward_kernel<512, 32, L>, 512, 1};
    return {(const void*)route_backward_kernel<512, 0, L>, 512, 1};
}

template <typename L, bool SOFTMAX>
const void* warp_kernel(int lanes, int e, int v) {
    if (lanes == 16) return e == 8 ? (const void*)route_warp_kernel<16, 8, 2, SOFTMAX, L> : (const void*)route_warp_kernel<16, 16, 2, SOFTMAX, L>;
    if (v == 0)
        return e == 8    ? (const void*)route_warp_kernel<32, 8, 0, SOFTMAX, L>
               : e == 16 ? (const void*)route_warp_kernel<32, 16, 0, SOFTMAX, L>
                         : (const void*)route_warp_kernel<32, 32, 0, SOFTMAX, L>;
    if (v == 1)
        return e == 8    ? (const void*)route_warp_kernel<32, 8, 1, SOFTMAX, L>
               : e == 16 ? (const void*)route_warp_kernel<32, 16, 1, SOFTMAX, L>
                         : (const void*)route_warp_kernel<32, 32, 1, SOFTMAX, L>;
    return e == 8    ? (const void*)route_warp_kernel<32, 8, 2, SOFTMAX, L>
           : e == 16 ? (const void*)route_warp_kernel<32, 16, 2, SOFTMAX, L>
                     : (const void*)route_warp_kernel<32, 32, 2, SOFTMAX, L>;
}

template <typename L, bool PLAIN>
const void* block_kernel(int threads) {
    return threads == 512   ? (const void*)route_block_kernel<512, PLAIN, L>
           : threads == 256 ? (const void*)route_block_kernel<256, PLAIN, L>
                            : (const void*)route_block_kernel<128, PLAIN, L>;
}

template <typename L>
const void* block_kernel(int threads, bool plain) {
    return plain ? block_kernel<L, true>(threads) : block_kernel<L, false>(threads);
}

}  // namespace

int launch_route(const RouteArgs& a0, cudaStream_t stream) {
    RouteArgs a = a0;
    // The warp kernel, with as few lanes and maxima as leave twice k maxima among the entries whose groups
    // stay: the k-th largest of them is then a close bound. Half a warp and two maxima a lane for 65536 rows
    // of 256, k = 8, 4 of 8 groups of 32: 39 us, a whole one and one each: 51. Where no such choice is left, and
    // for more than 32 entries, a bound by halving: 32768 float32 rows of 200, 500, 1000 with k = 64 take 98, 106,
    // 140 us, the block kernel 180, 139, 162; of 500 with k = 8 the maxima take 28 us, halving 69.
    const bool grouped = a.n_groups > 1 && a.top_groups < a.n_groups;
    const int live = grouped ? a.n / a.n_groups * a.top_groups : a.n;
    if (a.n <= 1024 && a.k <= 64) {
        const int e32 = a.n <= 256 ? 8 : a.n <= 512 ? 16 : 32, e16 = a.n <= 128 ? 8 : 16;
        int lanes = 0, e = 0, v = 0;
        if (a.n <= 256 && 2 * a.k <= live / (e16 / 2))
            lanes = 16, e = e16, v = 2;
        else if (2 * a.k <= live / e32)
            lanes = 32, e = e32, v = 1;
        else if (a.k <= 32 && (a.n <= 256 ? a.k <= live / (e32 / 2) : 3 * a.k <= 2 * (live / (e32 / 2))))
            lanes = 32, e = e32, v = 2;
        else
            lanes = 32, e = e32, v = 0;
        const int teams = kWarpThreads / lanes;
        const int64_t blocks = (a.tokens + teams - 1) / teams;
        if (blocks > INT_MAX) return SDM_ECOUNT;
        const size_t smem = grouped ? (size_t)teams * (a.n + lanes + a.n_groups) * 4 : 0;
        const bool softmax = a.score == SDM_SOFTMAX;
        const void* fn = a.logit_bf16 ? (softmax ? warp_kernel<uint16_t, true>(lanes, e, v) : warp_kernel<uint16_t, false>(lanes, e, v))
                                      : (softmax ? warp_kernel<float, true>(lanes, e, v) : warp_kernel<float, false>(lanes, e, v));
        void* args[] = {&a};
        return launch_pdl_raw(fn, dim3((unsigned)blocks), dim3(kWarpThreads), smem, stream, args);
    }
    if (a.tokens > INT_MAX) return SDM_ECOUNT;
    // Ranks that are the logits themselves are read again, out of L2, when a row of them is long, since the
    // shared memory to keep them is room for blocks: 1024 rows of 16384 bf16 logits, k = 64, 21 us and staged 26, 512
    // of 32768 19 and 28. Sigmoid ranks would be computed again: 58 us and staged 34.
    const bool plain = a.score == SDM_SOFTMAX && a.bias == nullptr && !grouped;
    int staged = (size_t)a.n * 4 <= kStagedBytes && !(plain && a.n > 8192) ? 1 : 0;
    const size_t smem = staged ? (size_t)(a.n + 4) * 4 : 0;
    // Threads for 16 to 64 ranks each. 16384 rows of 1500, k = 64: 128 threads 92 us, 256 132, 512 188; 4096 of 4096
    // 36, 41, 53; 1024 of 16384 29, 23, 23 (by sigmoid 59, 36, 34); 256 of 65536 45, 26, 22. For k up to half the threads: nearer
    // to them the k-th largest of their maxima is a poor bound, and above them there is none, so that the histograms follow:
    // 16384 rows of 1500 with k = 128, 129, 256 take 425, 208, 386 us.
    const int threads = a.n > 16384 ? 512 : a.n > 4096 ? 256 : 128;
    const void* fn = a.logit_bf16 ? block_kernel<uint16_t>(threads, plain) : block_kernel<float>(threads, plain);
    // the limit without a request counts the kernel's static arrays (10 KB) too
    const int rc = allow_smem(fn, smem > 32 * 1024 ? std::max(smem, (size_t)48 * 1024 + 16) : smem);
    if (rc != 0) return rc;
    void* args[] = {&a, &staged};
    return launch_pdl_raw(fn, dim3((unsigned)a.tokens), dim3(threads), smem, stream, args);
}

int launch_route_backward(const RouteArgs& a0, cudaStream_t stream) {
    RouteArgs a = a0;
    const bool dense = a.score == SDM_SOFTMAX && !a.renorm;
    const Team team = a.logit_bf16 ? backward_kernel<uint16_t>(a.n, dense) : backward_kernel<float>(a.n, dense);
    const int64_t blocks = (a.tokens + team.teams - 1) / team.teams;
    if (blocks > INT_MAX) return SDM_ECOUNT;
    void* args[] = {&a};
    return launch_pdl_raw(team.fn, dim3((unsigned)blocks), dim3(team.threads), 0, stream, args);
}

cudaError_t route_status(void** word) { return cudaGetSymbolAddress(word, g_route_status); }

}  // namespace sdm
