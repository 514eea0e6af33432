// Routing: the k best of n entries a token, with their weights, and the gradient of the logits.
//
// Math (include/sdm.h): scores s = softmax(x) or 1 / (1 + exp(-x)); entries ranked by x, s or
// s + bias; best groups, then best entries, ties to the lower index; weights s, renormalised.
//
// Ranks are compared as 32-bit integers in the order of the floats: 0 for entries already taken (or
// behind the end of a row), 1 for masked entries, and more for all others.
//
// Two kernels. route_warp_kernel (n <= 1024, k <= 32): a warp keeps a token's ranks in registers,
// lane l the consecutive entries from l * E on, so that the lowest lane that holds the maximum also
// holds the lowest index; k rounds of a warp-wide maximum take the entries in order. route_block_kernel:
// a block narrows the k-th rank down by histograms of its leading 11, then 11, then 10 bits, until at
// most kCandidates entries can still be chosen (one or two passes over ranks kept in shared memory),
// and sorts those by counting.
#include <algorithm>
#include <climits>
#include <cmath>

#include "quant_device.cuh"
#include "sdm_internal.h"

namespace sdm {
namespace {

__device__ unsigned int g_route_status;

constexpr unsigned kAll = 0xffffffffu;
constexpr uint32_t kTaken = 0, kMasked = 1;
constexpr int kMaxGroups = 256, kMaxK = 256;
constexpr int kCandidates = 512;
constexpr size_t kStagedBytes = 192 * 1024;  // ranks a block keeps in shared memory

__device__ __forceinline__ float minus_inf() { return __uint_as_float(0xff800000u); }
__device__ __forceinline__ bool masked(float x) { return !(x > minus_inf()); }  // NaN too

// exp(x - m) with m the largest of the logits; several +inf are the largest together
__device__ __forceinline__ float exp_below(float x, float m) {
    return masked(x) ? 0.0f : x == m ? 1.0f : expf(x - m);
}
__device__ __forceinline__ float sigmoid(float x) { return masked(x) ? 0.0f : __fdiv_rn(1.0f, __fadd_rn(1.0f, expf(-x))); }

// A float as an unsigned integer in the same order (-0 and +0 alike); masked ranks become kMasked.
__device__ __forceinline__ uint32_t ordered(float r) {
    if (masked(r)) return kMasked;
    const uint32_t b = __float_as_uint(r + 0.0f);
    return b ^ ((b >> 31) ? 0xffffffffu : 0x80000000u);
}

__device__ __forceinline__ float logit(const RouteArgs& a, int64_t t, int j) {
    const int64_t i = t * a.row_stride + j;
    return a.logit_bf16 ? to_f32(__ldg(static_cast<const uint16_t*>(a.logits) + i)) : __ldg(static_cast<const float*>(a.logits) + i);
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

// ---------------------------------------------------------------- a warp for each token

constexpr int kWarpThreads = 128;

// E: entries of a lane. L: uint16_t (bf16) or float logits.
template <int E, typename L>
__global__ void __launch_bounds__(kWarpThreads) route_warp_kernel(const RouteArgs a) {
    extern __shared__ float staged[];  // with groups: every warp's group values [n] and scores [n_groups]
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t = (int64_t)blockIdx.x * (kWarpThreads / 32) + warp;
    if (t >= a.tokens) return;
    const int n = a.n, j0 = lane * E;
    const L* row = static_cast<const L*>(a.logits) + t * a.row_stride;

    float x[E];
    const bool vec = (reinterpret_cast<uintptr_t>(row) & 15u) == 0 && j0 + E <= n;
    if (vec) {
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

    const bool softmax = a.score == SDM_SOFTMAX;
    const bool by_sum = a.n_groups > 1 && a.group_top == 2;
    float m = 0.0f, total = 1.0f;
    if (softmax) {
        m = minus_inf();
#pragma unroll
        for (int i = 0; i < E; ++i) m = fmaxf(m, x[i]);  // NaN takes no part
        m = warp_max(m);
        if (a.bias != nullptr || !a.renorm) {
            total = 0.0f;
#pragma unroll
            for (int i = 0; i < E; ++i) total += exp_below(x[i], m);
            total = warp_sum(total);
        }
    }
    uint32_t key[E];
#pragma unroll
    for (int i = 0; i < E; ++i) {
        float r = x[i];
        if (!masked(x[i])) {
            if (!softmax)
                r = sigmoid(x[i]);
            else if (a.bias != nullptr)
                r = __fdiv_rn(exp_below(x[i], m), total);
            if (a.bias != nullptr) r += __ldg(a.bias + j0 + i);
        }
        key[i] = j0 + i < n ? ordered(r) : kTaken;
        // what the groups are judged by, from here on in x
        x[i] = masked(r) ? minus_inf() : softmax && a.bias == nullptr && by_sum ? exp_below(x[i], m) : r;
    }

    if (a.n_groups > 1 && a.top_groups < a.n_groups) {
        float* value = staged + (size_t)warp * (n + a.n_groups);
        uint32_t* scores = reinterpret_cast<uint32_t*>(value + n);
        const int per = n / a.n_groups;
#pragma unroll
        for (int i = 0; i < E; ++i)
            if (j0 + i < n) value[j0 + i] = x[i];
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
            if (j0 + i < n && !((scores[g >> 5] >> (g & 31)) & 1u)) key[i] = kMasked;
            if (--left == 0) {
                ++g;
                left = per;
            }
        }
    }

    uint32_t best = 0;
#pragma unroll
    for (int i = 0; i < E; ++i) best = max(best, key[i]);
    int mine = 0;  // lane r: the entry taken in round r, and whether it is a live one
    bool live = false;
    for (int r = 0; r < a.k; ++r) {
        const uint32_t top = __reduce_max_sync(kAll, best);
        const int src = __ffs(__ballot_sync(kAll, best == top)) - 1;
        int at = 0;
        if (lane == src) {
#pragma unroll
            for (int i = E - 1; i >= 0; --i)
                if (key[i] == top) at = i;
            best = 0;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                if (i == at) key[i] = kTaken;
                best = max(best, key[i]);
            }
        }
        const int j = __shfl_sync(kAll, j0 + at, src);
        if (lane == r) {
            mine = j;
            live = top != kMasked;
        }
    }
    float s = 0.0f;
    if (lane < a.k && live) {
        const float y = to_f32(__ldg(row + mine));
        s = softmax ? exp_below(y, m) : sigmoid(y);
    }
    if (a.renorm) total = warp_sum(s);
    if (lane < a.k) {
        put_index(a, t, lane, mine);
        a.w[t * a.k + lane] = total > 0.0f && (softmax || a.renorm) ? __fdiv_rn(s, total) * a.scale : s * a.scale;
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

template <int NT>
__global__ void __launch_bounds__(NT) route_block_kernel(const RouteArgs a, int staged) {
    constexpr int WARPS = NT / 32;
    extern __shared__ uint32_t keys[];  // [n] when staged
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

    float m = 0.0f, total = 1.0f;
    if (softmax) {
        m = minus_inf();
        for (int j = tid; j < n; j += NT) m = fmaxf(m, logit(a, t, j));
        m = block_reduce(m, false, tmp, WARPS);
        if (biased || !a.renorm) {
            total = 0.0f;
            for (int j = tid; j < n; j += NT) total += exp_below(logit(a, t, j), m);
            total = block_reduce(total, true, tmp, WARPS);
        }
    }
    const auto rank_of = [&](int j) {
        const float x = logit(a, t, j);
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
                const float r = rank_of(j);
                top.add(masked(r) ? minus_inf() : softmax && !biased && a.group_top == 2 ? exp_below(logit(a, t, j), m) : r);
            }
            for (int o = 16; o; o >>= 1) {
                const float oa = __shfl_xor_sync(kAll, top.a, o), ob = __shfl_xor_sync(kAll, top.b, o);
                top.add(oa);
                top.b = fmaxf(top.b, ob);  // ob <= oa: it is second at best
            }
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
    const auto make_key = [&](int j) -> uint32_t {
        if (grouped) {
            const int g = j / per;
            if (!((stays[g >> 5] >> (g & 31)) & 1u)) return kMasked;
        }
        return ordered(rank_of(j));
    };
    if (staged) {
        for (int j = tid; j < n; j += NT) keys[j] = make_key(j);
    }
    const auto key_at = [&](int j) -> uint32_t { return staged ? keys[j] : make_key(j); };

    // narrow the k-th rank down: `above` live entries lie above the prefix, and those of the prefix
    // and above are at most kCandidates, or all their bits are fixed
    uint32_t lowest = 0;  // candidates are the live entries with key >= lowest
    int above = 0, need = k, inside = 0;
    bool few = false, exact = false;  // fewer than k live entries; the prefix is a whole key
    uint32_t prefix = 0;
    for (int level = 0; level < 3; ++level) {
        const int shift = level == 0 ? 21 : level == 1 ? 10 : 0, bits = level == 2 ? 10 : 11;
        for (int b = tid; b < kBins; b += NT) hist[b] = 0;
        __syncthreads();
        for (int j = tid; j < n; j += NT) {
            const uint32_t key = key_at(j);
            if (key > kMasked && (level == 0 || key >> (shift + bits) == prefix))
                atomicAdd(&hist[(key >> shift) & ((1u << bits) - 1u)], 1);
        }
        __syncthreads();
        // the bin of the need-th largest: thread i owns the PER bins from the top, i * PER on
        constexpr int PER = kBins / NT;
        int own = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) own += hist[kBins - 1 - (tid * PER + i)];
        int sum = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kAll, sum, o);
            if (lane >= o) sum += y;
        }
        if (lane == 31) counts[warp] = sum;
        if (tid == 0) found_bin = -1;
        __syncthreads();
        int before = sum - own;
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
        if (found_bin < 0) {  // level 0 only: all live entries are taken
            few = true;
            int all = 0;
            for (int i = 0; i < WARPS; ++i) all += counts[i];
            above = all;
            lowest = kMasked + 1;
            break;
        }
        above += found_above;
        need -= found_above;
        prefix = (prefix << bits) | (uint32_t)found_bin;
        inside = hist[found_bin];
        lowest = prefix << shift;
        exact = level == 2;
        __syncthreads();
        if (above + inside <= kCandidates) break;
    }
    // candidates: everything from `lowest` on, or only what lies above when too many share the last rank
    const bool ties = !few && exact && above + inside > kCandidates;
    if (tid == 0) n_cand = 0;
    __syncthreads();
    for (int j = tid; j < n; j += NT) {
        const uint32_t key = key_at(j);
        if (key > kMasked && (ties ? key > lowest : key >= lowest))
            cand[atomicAdd(&n_cand, 1)] = ((uint64_t)key << 32) | (uint32_t)~j;
    }
    __syncthreads();
    const int C = n_cand;
    for (int c = tid; c < C; c += NT) {
        const uint64_t mine = cand[c];
        int better = 0;
        for (int o = 0; o < C; ++o) better += cand[o] > mine;
        if (better < k) {
            const int j = (int)~(uint32_t)mine;
            sel_j[better] = j;
            const float x = logit(a, t, j);
            sel_s[better] = softmax ? exp_below(x, m) : sigmoid(x);
        }
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
                const float x = logit(a, t, j);
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
    const void* fn = a.n > 4096 ? (const void*)route_block_kernel<512> : (const void*)route_block_kernel<128>;
    // the limit without a request counts the kernel's static arrays (16 KB) too
    const int rc = allow_smem(fn, smem > 32 * 1024 ? std::max(smem, (size_t)48 * 1024 + 16) : smem);
    if (rc != 0) return rc;
    void* args[] = {&a, &staged};
    return launch_pdl_raw(fn, dim3((unsigned)a.tokens), dim3(a.n > 4096 ? 512 : 128), smem, stream, args);
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
