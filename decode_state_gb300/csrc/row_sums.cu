// Sums of weighted rows by slot: the gradient of an embedding table by token, or of a gather's bank by slot.
//
// Math (include/sdm.h): out[r] (+)= scale * sum over the entries e with idx[e] = r of w[e] * dout[token(e)].
//
// Design. The entries are sorted by slot, in their own order within a slot, so that a slot's sum is taken in one
// order whatever the launch, without atomics. The sorted entries are then cut into pieces of equal length, one for
// each warp and column slice, however unevenly the slots share them: a run of equal slots that crosses the ends of
// pieces leaves one float32 sum for each of them, which a last launch adds up in order.
//   up to 512 entries    one launch: the warp of a slot's first entry finds the others by scanning all of them
//   up to 8192           ranks by counting: an entry's place is the number of entries that come before it
//   more                 a stable radix sort with digits of at most 11 bits: counts, their running sums, places
// Rows without entries are set to zero by blocks of the same launch as the sums, which search the sorted slots.
#include <algorithm>
#include <climits>

#include "score_device.cuh"
#include "sdm_internal.h"

namespace sdm {
namespace {

__device__ unsigned int g_row_sums_status;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr uint32_t kDirect = 512;    // entries that one launch sums
constexpr uint32_t kRanked = 8192;   // entries ranked by counting
constexpr int kItems = 16, kTile = kThreads * kItems;
constexpr int kMostBits = 11;
constexpr int kZeroRows = 256;       // rows that a block sets to zero, at most

struct Place {
    int op;
    uint32_t token, at;  // at: the entry's number within its operand
};
__device__ __forceinline__ Place place_of(const RowSumArgs& a, uint32_t e) {
    const int op = e >= a.split;
    const uint32_t at = op ? e - a.split : e;
    return {op, at / (uint32_t)(op ? a.width[1] : a.width[0]), at};
}
__device__ __forceinline__ float weight_of(const RowSumArgs& a, int op, uint32_t at) {
    const void* w = op ? a.w[1] : a.w[0];
    if (w == nullptr) return 1.0f;
    return a.w_bf16 ? to_f32(__ldg(static_cast<const uint16_t*>(w) + at)) : __ldg(static_cast<const float*>(w) + at);
}

// The slot of entry e, or n_slots where it takes no part: padding, a weight of zero, an index outside the bank (flagged).
__device__ __forceinline__ uint32_t key_of(const RowSumArgs& a, uint32_t e) {
    const Place p = place_of(a, e);
    const int chunk = a.chunk;
    const int valid = a.chunk_valid != nullptr ? __ldg(a.chunk_valid + p.token / chunk) : a.valid;
    if ((int)(p.token % chunk) >= valid) return (uint32_t)a.n_slots;
    const void* idx = p.op ? a.idx[1] : a.idx[0];
    const int64_t j = a.idx64 ? __ldg(static_cast<const int64_t*>(idx) + p.at) : __ldg(static_cast<const int32_t*>(idx) + p.at);
    if (j == a.padding) return (uint32_t)a.n_slots;
    if (j < 0 || j >= a.n_slots) {
        atomicOr(&g_row_sums_status, SDM_DEV_BAD_INDEX);
        return (uint32_t)a.n_slots;
    }
    return weight_of(a, p.op, p.at) == 0.0f ? (uint32_t)a.n_slots : (uint32_t)j;
}

// ---------------------------------------------------------------- columns

// V columns of type T moved together.
template <typename T, int V>
struct alignas(sizeof(T) * V < 16 ? sizeof(T) * V : 16) Pack {
    T v[V];
};

template <typename D, int V>
__device__ __forceinline__ Pack<D, V> load_pack(const D* p) {
    return *reinterpret_cast<const Pack<D, V>*>(p);
}

template <typename O, int V>
__device__ __forceinline__ void put_row(const RowSumArgs& a, int64_t row, int col, const float* sum) {
    Pack<O, V>* to = reinterpret_cast<Pack<O, V>*>(static_cast<O*>(a.out) + row * a.hd + col);
    Pack<O, V> y;
    if (a.accumulate) {
        y = *to;
#pragma unroll
        for (int c = 0; c < V; ++c) y.v[c] = from_f32<O>(fmaf(sum[c], a.scale, to_f32(y.v[c])));
    } else {
#pragma unroll
        for (int c = 0; c < V; ++c) y.v[c] = from_f32<O>(sum[c] * a.scale);
    }
    *to = y;
}

// Rows [first, first + count) of the output whose flag is not set become zero, by a block.
template <typename O, int V>
__device__ __forceinline__ void zero_rows(const RowSumArgs& a, int64_t first, int count, const uint8_t* touched) {
    Pack<O, V> none;
#pragma unroll
    for (int c = 0; c < V; ++c) none.v[c] = O(0);
    for (int r = threadIdx.x >> 5; r < count; r += kWarps) {
        if (touched[r]) continue;
        O* row = static_cast<O*>(a.out) + (first + r) * a.hd;
        for (int c = (threadIdx.x & 31) * V; c < a.hd; c += 32 * V) *reinterpret_cast<Pack<O, V>*>(row + c) = none;
    }
}

// ---------------------------------------------------------------- few entries

template <typename D, typename O, int V>
__global__ void __launch_bounds__(kThreads) direct_kernel(const RowSumArgs a, int zero_span) {
    __shared__ uint32_t keys[kDirect];
    __shared__ uint16_t list[kWarps][kDirect];
    __shared__ uint8_t touched[kZeroRows];
    grid_dependency_wait();
    grid_launch_dependents();
    const int n = (int)a.entries, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int e = threadIdx.x; e < n; e += kThreads) keys[e] = key_of(a, e);
    if ((int64_t)blockIdx.x < a.zero_blocks) {
        const int64_t first = (int64_t)blockIdx.x * zero_span;
        const int count = (int)min((int64_t)zero_span, a.n_slots - first);
        for (int r = threadIdx.x; r < count; r += kThreads) touched[r] = 0;
        __syncthreads();
        for (int e = threadIdx.x; e < n; e += kThreads)
            if (keys[e] >= first && keys[e] < first + count) touched[keys[e] - first] = 1;
        __syncthreads();
        zero_rows<O, V>(a, first, count, touched);
        return;
    }
    __syncthreads();
    const int64_t unit = ((int64_t)blockIdx.x - a.zero_blocks) * kWarps + warp;
    const int e = (int)(unit / a.slices);
    if (e >= n) return;
    const uint32_t key = keys[e];
    if (key >= a.n_slots) return;
    bool earlier = false;
    for (int i = lane; i < e; i += 32) earlier |= keys[i] == key;
    if (__any_sync(kAll, earlier)) return;
    int found = 0;  // the entries of the slot, in order
    for (int base = e & ~31; base < n; base += 32) {
        const int i = base + lane;
        const bool same = i >= e && i < n && keys[i] == key;
        const unsigned mask = __ballot_sync(kAll, same);
        if (same) list[warp][found + __popc(mask & ((1u << lane) - 1))] = (uint16_t)i;
        found += __popc(mask);
    }
    __syncwarp();
    const int col = (int)(unit % a.slices) * a.slice_cols + lane * V;
    if (lane * V >= a.slice_cols || col >= a.hd) return;
    float sum[V];
#pragma unroll
    for (int c = 0; c < V; ++c) sum[c] = 0.0f;
    constexpr int U = 8;
    for (int i0 = 0; i0 < found; i0 += U) {
        Pack<D, V> x[U];
        float w[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i0 + u < found) {
                const Place p = place_of(a, list[warp][i0 + u]);
                w[u] = weight_of(a, p.op, p.at);
                x[u] = load_pack<D, V>(static_cast<const D*>(p.op ? a.dout[1] : a.dout[0]) + (int64_t)p.token * a.hd + col);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i0 + u < found) {
#pragma unroll
                for (int c = 0; c < V; ++c) sum[c] = fmaf(w[u], to_f32(x[u].v[c]), sum[c]);
            }
        }
    }
    put_row<O, V>(a, key, col, sum);
}

// ---------------------------------------------------------------- the sort

// Places by counting. A block takes 32 entries, a warp four of them, and compares with all.
__global__ void __launch_bounds__(kThreads) rank_kernel(const RowSumArgs a, uint32_t* keys_out, uint32_t* ents_out) {
    extern __shared__ uint32_t all[];
    grid_dependency_wait();
    grid_launch_dependents();
    const int n = (int)a.entries, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int e = threadIdx.x; e < n; e += kThreads) all[e] = key_of(a, e);
    __syncthreads();
    const int e0 = blockIdx.x * 32 + warp * 4;
    uint32_t key[4];
    int before[4] = {0, 0, 0, 0};
#pragma unroll
    for (int q = 0; q < 4; ++q) key[q] = e0 + q < n ? all[e0 + q] : 0u;
    for (int i = lane; i < n; i += 32) {
        const uint32_t k = all[i];
#pragma unroll
        for (int q = 0; q < 4; ++q) before[q] += k < key[q] || (k == key[q] && i < e0 + q);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        before[q] = __reduce_add_sync(kAll, before[q]);
        if (lane == q && e0 + q < n) {
            keys_out[before[q]] = key[q];
            ents_out[before[q]] = e0 + q;
        }
    }
}

// The counts of a tile's digits, counts[digit * tiles + tile]. FIRST: the keys are made here and kept.
template <bool FIRST>
__global__ void __launch_bounds__(kThreads) digit_count_kernel(const RowSumArgs a, uint32_t* keys, uint32_t* counts, int shift, int bits) {
    __shared__ uint32_t bins[1 << kMostBits];
    grid_dependency_wait();
    grid_launch_dependents();
    const int all = 1 << bits;
    for (int b = threadIdx.x; b < all; b += kThreads) bins[b] = 0;
    __syncthreads();
    const uint32_t from = blockIdx.x * (uint32_t)kTile;
#pragma unroll 4
    for (int i = 0; i < kItems; ++i) {
        const uint32_t e = from + i * kThreads + threadIdx.x;
        if (e < a.entries) {
            const uint32_t key = FIRST ? key_of(a, e) : keys[e];
            if (FIRST) keys[e] = key;
            atomicAdd(&bins[key >> shift & (all - 1)], 1u);
        }
    }
    __syncthreads();
    for (int b = threadIdx.x; b < all; b += kThreads) counts[(int64_t)b * gridDim.x + blockIdx.x] = bins[b];
}

// Each digit's counts become their running sums over the tiles, and their total.
__global__ void __launch_bounds__(kThreads) digit_scan_kernel(uint32_t* counts, uint32_t* totals, int tiles) {
    __shared__ uint32_t sums[kWarps];
    grid_dependency_wait();
    grid_launch_dependents();
    uint32_t* row = counts + (int64_t)blockIdx.x * tiles;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t carry = 0;
    for (int base = 0; base < tiles; base += kThreads) {
        const int i = base + threadIdx.x;
        const uint32_t own = i < tiles ? row[i] : 0u;
        uint32_t sum = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(kAll, sum, o);
            if (lane >= o) sum += y;
        }
        if (lane == 31) sums[warp] = sum;
        __syncthreads();
        uint32_t before = carry;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp) before += sums[w];
            carry += sums[w];
        }
        if (i < tiles) row[i] = before + sum - own;
        __syncthreads();
    }
    if (threadIdx.x == 0) totals[blockIdx.x] = carry;
}

// A tile's keys go to their places: behind all smaller digits, behind the same digit of earlier tiles, in order.
__global__ void __launch_bounds__(kThreads) digit_place_kernel(uint32_t entries, const uint32_t* keys_in, const uint32_t* ents_in,
                                                               uint32_t* keys_out, uint32_t* ents_out, const uint32_t* counts,
                                                               const uint32_t* totals, int shift, int bits) {
    __shared__ uint16_t own[kWarps][1 << kMostBits];
    __shared__ uint32_t start[1 << kMostBits];
    __shared__ uint32_t sums[kWarps];
    grid_dependency_wait();
    grid_launch_dependents();
    const int all = 1 << bits, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int b = lane; b < all; b += 32) own[warp][b] = 0;
    __syncwarp();
    // a warp's keys are consecutive, 32 at a time
    const uint32_t from = blockIdx.x * (uint32_t)kTile + warp * (32 * kItems);
    uint32_t key[kItems];
    uint16_t rank[kItems];
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const uint32_t e = from + i * 32 + lane;
        key[i] = e < entries ? keys_in[e] : 0u;
    }
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const bool on = from + i * 32 + lane < entries;
        const uint32_t d = key[i] >> shift & (all - 1);
        unsigned same = __ballot_sync(kAll, on);  // lanes with the same digit
        for (int b = 0; b < bits; ++b) {
            const bool set = d >> b & 1;
            const unsigned with = __ballot_sync(kAll, set);
            same &= set ? with : ~with;
        }
        const uint32_t before = own[warp][d];
        __syncwarp();
        if (on && lane == 31 - __clz(same)) own[warp][d] = (uint16_t)(before + __popc(same));
        __syncwarp();
        rank[i] = (uint16_t)(before + __popc(same & ((1u << lane) - 1)));
    }
    __syncthreads();
    // where each digit starts: running sums of the totals, eight consecutive digits a thread at most
    const int per = (all + kThreads - 1) / kThreads, b0 = threadIdx.x * per;
    uint32_t mine = 0;
    for (int b = b0; b < b0 + per && b < all; ++b) mine += __ldg(totals + b);
    uint32_t sum = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(kAll, sum, o);
        if (lane >= o) sum += y;
    }
    if (lane == 31) sums[warp] = sum;
    __syncthreads();
    uint32_t before = sum - mine;
    for (int w = 0; w < warp; ++w) before += sums[w];
    for (int b = b0; b < b0 + per && b < all; ++b) {
        start[b] = before + __ldg(counts + (int64_t)b * gridDim.x + blockIdx.x);
        before += __ldg(totals + b);
        uint32_t run = 0;
        for (int w = 0; w < kWarps; ++w) {
            const uint32_t c = own[w][b];
            own[w][b] = (uint16_t)run;
            run += c;
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kItems; ++i) {
        const uint32_t e = from + i * 32 + lane;
        if (e < entries) {
            const uint32_t d = key[i] >> shift & (all - 1), to = start[d] + own[warp][d] + rank[i];
            keys_out[to] = key[i];
            ents_out[to] = ents_in != nullptr ? ents_in[e] : e;
        }
    }
}

// ---------------------------------------------------------------- the sums

// The first place whose key is not below `key`, in keys[lo, hi).
__device__ __forceinline__ uint32_t lower_bound(const uint32_t* keys, uint32_t lo, uint32_t hi, uint32_t key) {
    while (lo < hi) {
        const uint32_t mid = lo + (hi - lo) / 2;
        if (__ldg(keys + mid) < key)
            lo = mid + 1;
        else
            hi = mid;
    }
    return lo;
}

template <typename D, typename O, int V>
__global__ void __launch_bounds__(kThreads) sums_kernel(const RowSumArgs a, int zero_span) {
    __shared__ uint8_t touched[kZeroRows];
    __shared__ uint32_t range[2];
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    if ((int64_t)blockIdx.x < a.zero_blocks) {
        const int64_t first = (int64_t)blockIdx.x * zero_span;
        const int count = (int)min((int64_t)zero_span, a.n_slots - first);
        if (threadIdx.x < 2) range[threadIdx.x] = lower_bound(a.keys, 0, a.entries, (uint32_t)(first + threadIdx.x * count));
        __syncthreads();
        for (int r = threadIdx.x; r < count; r += kThreads) {
            const uint32_t at = lower_bound(a.keys, range[0], range[1], (uint32_t)(first + r));
            touched[r] = at < range[1] && __ldg(a.keys + at) == (uint32_t)(first + r);
        }
        __syncthreads();
        zero_rows<O, V>(a, first, count, touched);
        return;
    }
    const int64_t unit = ((int64_t)blockIdx.x - a.zero_blocks) * kWarps + (threadIdx.x >> 5);
    const uint32_t piece = (uint32_t)(unit / a.slices);
    if (piece >= a.pieces) return;
    const uint32_t from = piece * a.piece, to = min(from + a.piece, a.entries);
    const int in_slice = lane * V, col = (int)(unit % a.slices) * a.slice_cols + in_slice;
    const bool on = in_slice < a.slice_cols && col < a.hd;
    uint32_t current = __ldg(a.keys + from);
    if (current >= a.n_slots) return;
    bool continues = from > 0 && __ldg(a.keys + from - 1) == current;
    const uint32_t next = to < a.entries ? __ldg(a.keys + to) : 0xffffffffu;
    float sum[V];
#pragma unroll
    for (int c = 0; c < V; ++c) sum[c] = 0.0f;
    const auto flush = [&](bool ends) {
        if (on) {
            if (continues || !ends) {
                float* part = (continues ? a.heads : a.tails) + (int64_t)piece * a.hd + col;
#pragma unroll
                for (int c = 0; c < V; ++c) part[c] = sum[c];
            } else {
                put_row<O, V>(a, current, col, sum);
            }
        }
        continues = false;
#pragma unroll
        for (int c = 0; c < V; ++c) sum[c] = 0.0f;
    };
    constexpr int U = 8;
    for (uint32_t base = from; base < to; base += 32) {
        uint32_t key = 0xffffffffu;
        float w = 0.0f;
        const D* row = nullptr;
        if (base + lane < to) {
            key = __ldg(a.keys + base + lane);
            if (key < a.n_slots) {
                const Place p = place_of(a, __ldg(a.ents + base + lane));
                w = weight_of(a, p.op, p.at);
                row = static_cast<const D*>(p.op ? a.dout[1] : a.dout[0]) + (int64_t)p.token * a.hd;
            }
        }
        for (int j0 = 0; j0 < 32 && base + j0 < to; j0 += U) {  // U divides a piece: only the last one ends within
            Pack<D, V> x[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const D* r = reinterpret_cast<const D*>(__shfl_sync(kAll, reinterpret_cast<unsigned long long>(row), j0 + u));
                if (r != nullptr && on) x[u] = load_pack<D, V>(r + col);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t k = __shfl_sync(kAll, key, j0 + u);
                const float f = __shfl_sync(kAll, w, j0 + u);
                if (k != current) {
                    if (current < a.n_slots) flush(true);
                    current = k;
                }
                if (k < a.n_slots) {
#pragma unroll
                    for (int c = 0; c < V; ++c) sum[c] = fmaf(f, to_f32(x[u].v[c]), sum[c]);
                }
            }
            if (current >= a.n_slots) return;  // nothing but dropped entries, or the end of the last piece
        }
    }
    flush(next != current);
}

// The runs that cross the ends of pieces: the sum in the piece where a run begins, then those that continue it. A
// block for each piece and slice; its warps share out the pieces of a long run.
template <typename O, int V>
__global__ void __launch_bounds__(kThreads) join_kernel(const RowSumArgs a) {
    __shared__ float parts[kWarps][32 * V];
    grid_dependency_wait();
    grid_launch_dependents();
    const uint32_t piece = blockIdx.x / a.slices, from = piece * a.piece, to = from + a.piece;
    if (to >= a.entries) return;
    const uint32_t key = __ldg(a.keys + to - 1);
    if (key >= a.n_slots || __ldg(a.keys + to) != key) return;
    if (from > 0 && __ldg(a.keys + from - 1) == key) return;  // it began earlier
    // the pieces that begin with this slot: piece + 1 .. piece + more
    uint32_t lo = piece + 1, hi = a.pieces;
    while (lo < hi) {
        const uint32_t mid = lo + (hi - lo) / 2;
        if (__ldg(a.keys + (int64_t)mid * a.piece) <= key)
            lo = mid + 1;
        else
            hi = mid;
    }
    const uint32_t more = lo - piece - 1, share = (more + kWarps - 1) / kWarps;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int in_slice = lane * V, col = (int)(blockIdx.x % a.slices) * a.slice_cols + in_slice;
    const bool on = in_slice < a.slice_cols && col < a.hd;
    float sum[V];
#pragma unroll
    for (int c = 0; c < V; ++c) sum[c] = 0.0f;
    if (on) {
        const uint32_t last = min((uint32_t)(warp + 1) * share, more);
#pragma unroll 8
        for (uint32_t q = warp * share; q < last; ++q) {
            const float* part = a.heads + (int64_t)(piece + 1 + q) * a.hd + col;
#pragma unroll
            for (int c = 0; c < V; ++c) sum[c] += part[c];
        }
#pragma unroll
        for (int c = 0; c < V; ++c) parts[warp][in_slice + c] = sum[c];
    }
    __syncthreads();
    if (warp != 0 || !on) return;
    const float* tail = a.tails + (int64_t)piece * a.hd + col;
#pragma unroll
    for (int c = 0; c < V; ++c) {
        sum[c] = tail[c];
        for (int w = 0; w < kWarps; ++w) sum[c] += parts[w][in_slice + c];
    }
    put_row<O, V>(a, key, col, sum);
}

struct Kernels {
    const void *direct, *sums, *join;
};
template <typename D, typename O, int V>
Kernels kernels() {
    return {(const void*)direct_kernel<D, O, V>, (const void*)sums_kernel<D, O, V>, (const void*)join_kernel<O, V>};
}
template <typename D, typename O>
Kernels kernels(int v) {
    return v == 8 ? kernels<D, O, 8>() : v == 4 ? kernels<D, O, 4>() : v == 2 ? kernels<D, O, 2>() : kernels<D, O, 1>();
}

// Entries of a piece: as many as leave 8192 pieces and slices of 256 columns, so that all warps have work, from 16,
// below which the sums at the ends are most of the work, to 256.
uint32_t piece_of(int64_t entries, int hd) {
    const int64_t want = (entries * ((hd + 255) / 256) + 8191) / 8192;
    uint32_t piece = 16;
    while (piece < want && piece < 256) piece *= 2;
    return piece;
}
int64_t round_up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

}  // namespace

int64_t row_sums_workspace(int64_t entries, int64_t n_slots, int hd) {
    (void)n_slots;
    if (entries <= kDirect) return 0;
    const int64_t e = round_up(entries, 64), tiles = (entries + kTile - 1) / kTile, piece = piece_of(entries, hd);
    const int64_t pieces = (entries + piece - 1) / piece;
    const int64_t sort = entries <= kRanked ? 2 * e : 4 * e + round_up((tiles + 1) << kMostBits, 64);
    return 4 * (sort + 2 * round_up(pieces * hd, 64));
}

int launch_row_sums(const RowSumArgs& a0, cudaStream_t stream) {
    RowSumArgs a = a0;
    const auto whole = [&](int v) {  // accesses of v columns are aligned everywhere
        if (a.hd % v != 0) return false;
        const uintptr_t in = std::min(16, v * (a.dout_bf16 ? 2 : 4)), out = std::min(16, v * (a.out_bf16 ? 2 : 4));
        for (int o = 0; o < a.n_ops; ++o)
            if (reinterpret_cast<uintptr_t>(a.dout[o]) % in != 0) return false;
        return reinterpret_cast<uintptr_t>(a.out) % out == 0;
    };
    // columns of a lane: as many as 16 bytes of dout hold, fewer where that leaves lanes of a short row without work
    int v = a.dout_bf16 ? 8 : 4;
    while (v > 1 && (!whole(v) || a.hd < 32 * v)) v /= 2;
    const int packs = (a.hd + v - 1) / v;
    a.slices = (packs + 31) / 32;
    a.slice_cols = (packs + a.slices - 1) / a.slices * v;
    const Kernels fn = a.dout_bf16 ? (a.out_bf16 ? kernels<uint16_t, uint16_t>(v) : kernels<uint16_t, float>(v))
                                   : (a.out_bf16 ? kernels<float, uint16_t>(v) : kernels<float, float>(v));
    // rows that a block sets to zero: 128 KB of them
    int zero_span = (int)std::clamp<int64_t>((int64_t)128 * 1024 / ((int64_t)a.hd * (a.out_bf16 ? 2 : 4)), 8, kZeroRows);
    a.zero_blocks = a.accumulate ? 0 : (a.n_slots + zero_span - 1) / zero_span;
    int rc;
    if (a.entries <= kDirect) {
        const int64_t blocks = a.zero_blocks + ((int64_t)a.entries * a.slices + kWarps - 1) / kWarps;
        if (blocks == 0) return 0;
        void* args[] = {&a, &zero_span};
        return launch_pdl_raw(fn.direct, dim3((unsigned)blocks), dim3(kThreads), 0, stream, args);
    }
    const int64_t e = round_up(a.entries, 64);
    uint32_t* words = static_cast<uint32_t*>(a.workspace);
    if (a.entries <= kRanked) {
        uint32_t *keys = words, *ents = words + e;
        void* args[] = {&a, &keys, &ents};
        rc = launch_pdl_raw((const void*)rank_kernel, dim3((a.entries + 31) / 32), dim3(kThreads), a.entries * 4, stream, args);
        if (rc != 0) return rc;
        a.keys = keys;
        a.ents = ents;
        words += 2 * e;
    } else {
        int tiles = (int)((a.entries + (int64_t)kTile - 1) / kTile);
        uint32_t *keys[2] = {words, words + e}, *ents[2] = {words + 2 * e, words + 3 * e};
        uint32_t *totals = words + 4 * e, *counts = totals + (1 << kMostBits);
        int significant = 1;
        while ((a.n_slots >> significant) != 0) ++significant;  // n_slots itself is a key
        const int passes = (significant + kMostBits - 1) / kMostBits;
        int bits = (significant + passes - 1) / passes;
        for (int p = 0; p < passes; ++p) {
            int shift = p * bits;
            uint32_t *in = keys[p & 1], *out = keys[~p & 1], *ents_in = p ? ents[p & 1] : nullptr, *ents_out = ents[~p & 1];
            void* count_args[] = {&a, &in, &counts, &shift, &bits};
            rc = launch_pdl_raw(p ? (const void*)digit_count_kernel<false> : (const void*)digit_count_kernel<true>, dim3(tiles),
                                dim3(kThreads), 0, stream, count_args);
            if (rc != 0) return rc;
            void* scan_args[] = {&counts, &totals, &tiles};
            rc = launch_pdl_raw((const void*)digit_scan_kernel, dim3(1u << bits), dim3(kThreads), 0, stream, scan_args);
            if (rc != 0) return rc;
            uint32_t entries = a.entries;
            void* place_args[] = {&entries, &in, &ents_in, &out, &ents_out, &counts, &totals, &shift, &bits};
            rc = launch_pdl_raw((const void*)digit_place_kernel, dim3(tiles), dim3(kThreads), 0, stream, place_args);
            if (rc != 0) return rc;
        }
        a.keys = keys[passes & 1];
        a.ents = ents[passes & 1];
        words += 4 * e + round_up((int64_t)(tiles + 1) << kMostBits, 64);
    }
    a.piece = piece_of(a.entries, a.hd);
    a.pieces = (a.entries + a.piece - 1) / a.piece;
    a.heads = reinterpret_cast<float*>(words);
    a.tails = a.heads + round_up((int64_t)a.pieces * a.hd, 64);
    const int64_t blocks = a.zero_blocks + ((int64_t)a.pieces * a.slices + kWarps - 1) / kWarps;
    if (blocks > INT_MAX || (int64_t)a.pieces * a.slices > INT_MAX) return SDM_ECOUNT;
    void* args[] = {&a, &zero_span};
    rc = launch_pdl_raw(fn.sums, dim3((unsigned)blocks), dim3(kThreads), 0, stream, args);
    if (rc != 0) return rc;
    void* join_args[] = {&a};
    return launch_pdl_raw(fn.join, dim3(a.pieces * (uint32_t)a.slices), dim3(kThreads), 0, stream, join_args);
}

cudaError_t row_sums_status(void** word) { return cudaGetSymbolAddress(word, g_row_sums_status); }

}  // namespace sdm
