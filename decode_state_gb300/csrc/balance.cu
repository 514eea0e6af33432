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

#include "balance_internal.h"
#include "balance_rows.cuh"
#include "sdm_internal.h"

namespace sdm {
namespace {

constexpr int kCountThreads = 256;
constexpr int kCountBins = 4096;  // entries of a row that a block counts in shared memory

__global__ void __launch_bounds__(kCountThreads) balance_zero_kernel(const BalanceArgs a) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t all = (int64_t)a.sequences * a.n, step = (int64_t)gridDim.x * kCountThreads;
    for (int64_t i = (int64_t)blockIdx.x * kCountThreads + threadIdx.x; i < all; i += step) a.counts[i] = 0;
    for (int64_t i = (int64_t)blockIdx.x * kCountThreads + threadIdx.x; i < a.sequences; i += step) a.totals[i] = 0;
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
    const int first = blockIdx.x * run, last = first + min(run, a.tokens - first), tid = threadIdx.x;  // tokens may be near 2^31
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

// A sequence's loss out of its parts: those of the teams that met it lie side by side. LANES threads a sequence: a block, or a
// warp where there are many.
template <int LANES>
__global__ void __launch_bounds__(kCountThreads) balance_loss_kernel(const BalanceArgs a) {
    __shared__ double sums[kCountThreads / 32];
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x % LANES;
    const int64_t s = (int64_t)blockIdx.x * (kCountThreads / LANES) + threadIdx.x / LANES;
    if (s >= a.sequences) return;  // whole warps
    int begin = 0, end = a.tokens;
    if (a.offsets != nullptr) {
        begin = max(__ldg(a.offsets + s), 0);
        end = min(__ldg(a.offsets + s + 1), a.tokens);
    }
    const bool any = end > begin && a.totals[s] > 0;
    double sum = 0.0;
    if (any)
        for (int64_t p = begin / a.rows + s + lane; p <= (end - 1) / a.rows + s; p += LANES) sum += a.parts[p];
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(kAll, sum, o);
    if constexpr (LANES > 32) {
        if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = sum;
        __syncthreads();
        if (threadIdx.x == 0) {
            sum = 0.0;
            for (int w = 0; w < kCountThreads / 32; ++w) sum += sums[w];
        }
    }
    if (lane == 0) a.loss[s] = any ? (float)(a.scale * sum / (double)(end - begin)) : 0.0f;
}

// Calls that one launch takes, a cluster for each sequence. Blocks of up to 32 of them, and of one for the tokens outside all,
// are on the chip together: 1024 rows of 64 with the gradient take 9.2 us in 32 sequences and 14.0 in four launches, in
// 64 18 and 13, and each further 19 clusters take as long again. A cluster's blocks each count all of its entries, and
// 64 rows of 16 go through a block at a time: one sequence of 512 rows (64 columns, 8 chosen) 9.2 us for 10.8 in four launches,
// of 1024 12.9 for 10.0; of 1024 rows of 16 (one chosen) 8.5 for 9.9, of 2048 11.5 for 10.5. Offsets may give
// all tokens to one sequence, so that the whole call is bounded too.
bool small(const BalanceArgs& a) {
    const int64_t entries = (int64_t)a.tokens * a.k;
    return a.sequences > 0 && a.sequences <= 32 && a.n <= kSmallBins && (int64_t)a.tokens * a.n <= 65536 && entries <= 8192 &&
           entries <= (int64_t)4096 * a.sequences && a.tokens <= 1024 * a.sequences;
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
    if (small(a)) {
        const void* fn = a.logit_bf16 ? (grad ? small_kernel<true, uint16_t>(a.n) : small_kernel<false, uint16_t>(a.n))
                                      : (grad ? small_kernel<true, float>(a.n) : small_kernel<false, float>(a.n));
        const unsigned clusters = (unsigned)a.sequences + (grad && a.offsets != nullptr ? 1 : 0);
        void* args[] = {&a};
        return launch_cluster_raw(fn, kSmallCluster, dim3(clusters * kSmallCluster), dim3(kSmallThreads), 0, stream, args);
    }
    const BalanceTeam team = a.logit_bf16 ? balance_team_bf16(a.n, vec, grad) : balance_team_f32(a.n, vec, grad);
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
        int run = (a.tokens - 1) / blocks + 1;
        blocks = (a.tokens - 1) / run + 1;
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
    if (a.sequences <= 1024)
        return launch_pdl_raw((const void*)balance_loss_kernel<kCountThreads>, dim3(a.sequences), dim3(kCountThreads), 0, stream, args);
    constexpr int each = kCountThreads / 32;
    return launch_pdl_raw((const void*)balance_loss_kernel<32>, dim3((a.sequences + each - 1) / each), dim3(kCountThreads), 0, stream, args);
}

cudaError_t balance_status(void** word) { return cudaGetSymbolAddress(word, g_balance_status); }

}  // namespace sdm
