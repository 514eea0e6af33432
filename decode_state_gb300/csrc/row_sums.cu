// Sums of weighted rows by slot: the gradient of an embedding table by token, or of a gather's bank by slot.
//
// Math (include/sdm.h): out[r] (+)= scale * sum over the entries e with idx[e] = r of w[e] * dout[token(e)].
//
// Design. The entries are sorted by slot, in their own order within a slot, so that a slot's sum is taken in one
// order whatever the launch, without atomics. The sorted entries are then cut into pieces of equal length, one for
// each warp and column slice, however unevenly the slots share them: a run of equal slots that crosses the ends of
// pieces leaves one float32 sum for each of them, which a last launch adds up in order.
//   up to 512 entries    one launch: the warp of a slot's first entry finds the others by scanning all of them
//   up to 32768          a stable radix sort in the shared memory of a cluster of blocks
//   more                 the same in launches, with digits of at most 11 bits: counts, their running sums, places
// Rows without entries are set to zero by blocks of the same launch as the sums, which search the sorted slots.
#include <algorithm>
#include <climits>

#include "cluster_device.cuh"
#include "score_device.cuh"
#include "sdm_internal.h"

namespace sdm {
namespace {

__device__ unsigned int g_row_sums_status;

constexpr int kThreads = 256, kWarps = kThreads / 32;
// Entries that one launch sums. 512 of them, spread over 32768 rows of 1024: 4.8 us, by the cluster 15.9; all of one row of 128: 42
// and 16.5, which 1024 entries would make 84 and 18 (spread 13.3 and 16.3).
constexpr uint32_t kDirect = 512;
constexpr int kMostBits = 11;
constexpr int kZeroRows = 256;       // rows that a block sets to zero, at most

// x / d for x < 2^31 as a product (Granlund and Montgomery): m = ceil(2^(31 + l) / d), l = ceil(log2 d).
__device__ __forceinline__ uint32_t divided(uint32_t x, const Divisor& d) { return d.m == 0 ? x : __umulhi(x, d.m) >> d.shift; }

struct Place {
    int op;
    uint32_t token, at;  // at: the entry's number within its operand
};
__device__ __forceinline__ Place place_of(const RowSumArgs& a, uint32_t e) {
    const int op = e >= a.split;
    const uint32_t at = op ? e - a.split : e;
    return {op, divided(at, op ? a.by_width[1] : a.by_width[0]), at};
}
__device__ __forceinline__ float weight_of(const RowSumArgs& a, int op, uint32_t at) {
    const void* w = op ? a.w[1] : a.w[0];
    if (w == nullptr) return 1.0f;
    return a.w_bf16 ? to_f32(__ldg(static_cast<const uint16_t*>(w) + at)) : __ldg(static_cast<const float*>(w) + at);
}

// The slots of entries e, e + step, ..., or n_slots where one takes no part: padding, a weight of zero, an index
// outside the bank (flagged), nothing behind the last. The loads of all are on their way together.
template <int N>
__device__ __forceinline__ void keys_of(const RowSumArgs& a, uint32_t e, uint32_t step, uint32_t* key) {
    int64_t j[N];
    float w[N];
    uint32_t read = 0;  // which entries have an index
    const bool padded = a.chunk_valid != nullptr || a.valid < a.chunk;
    const auto load = [&](int i, int op, uint32_t at) {
        bool live = true;
        if (padded) {
            const uint32_t token = divided(at, op ? a.by_width[1] : a.by_width[0]), chunk = divided(token, a.by_chunk);
            const int valid = a.chunk_valid != nullptr ? __ldg(a.chunk_valid + chunk) : a.valid;
            live = (int)(token - chunk * a.chunk) < valid;
        }
        if (live) {
            const void* idx = op ? a.idx[1] : a.idx[0];
            j[i] = a.idx64 ? __ldg(static_cast<const int64_t*>(idx) + at) : __ldg(static_cast<const int32_t*>(idx) + at);
            w[i] = weight_of(a, op, at);
            read |= 1u << i;
        }
    };
#pragma unroll
    for (int i = 0; i < N; ++i) {
        j[i] = -1;
        w[i] = 0.0f;
    }
    // entries of one operand, as nearly all warps have them, choose between its arrays once
    if (__all_sync(kAll, e + (N - 1) * step < a.split)) {
#pragma unroll
        for (int i = 0; i < N; ++i) load(i, 0, e + i * step);
    } else if (__all_sync(kAll, e >= a.split && e + (N - 1) * step < a.entries)) {
#pragma unroll
        for (int i = 0; i < N; ++i) load(i, 1, e + i * step - a.split);
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const uint32_t at = e + i * step;
            if (at < a.entries) load(i, at >= a.split, at >= a.split ? at - a.split : at);
        }
    }
    bool outside = false;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const bool in = j[i] >= 0 && j[i] < a.n_slots, none = j[i] == a.padding && a.padding != SDM_NO_PADDING;
        outside |= (read >> i & 1) && !in && !none;
        key[i] = in && !none && w[i] != 0.0f ? (uint32_t)j[i] : (uint32_t)a.n_slots;
    }
    if (outside) atomicOr(&g_row_sums_status, SDM_DEV_BAD_INDEX);
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

template <typename O>
__device__ __forceinline__ O* place_in(const RowSumArgs& a, uint32_t row, int col) {
    return static_cast<O*>(a.out) + (uint64_t)row * (uint32_t)a.hd + col;
}
// A row's sum goes to its place, `there` being what is there where sums are added to it.
template <typename O, int V>
__device__ __forceinline__ void put_row(const RowSumArgs& a, bool accumulate, uint32_t row, int col, const float* sum, const Pack<O, V>& there) {
    Pack<O, V> y;
    if (accumulate) {
#pragma unroll
        for (int c = 0; c < V; ++c) y.v[c] = from_f32<O>(fmaf(sum[c], a.scale, to_f32(there.v[c])));
    } else {
#pragma unroll
        for (int c = 0; c < V; ++c) y.v[c] = from_f32<O>(sum[c] * a.scale);
    }
    // streaming: rows of dout that other warps will read stay in L2
    if constexpr (sizeof(y) == 16)
        __stcs(reinterpret_cast<uint4*>(place_in<O>(a, row, col)), *reinterpret_cast<const uint4*>(&y));
    else
        *reinterpret_cast<Pack<O, V>*>(place_in<O>(a, row, col)) = y;
}

// Rows [first, first + count) of the output whose flag is not set become zero, by a block: copies of `zeros` in shared
// memory where rows are whole 16-byte pieces, which cost a thread one instruction a row, else stores.
constexpr int kZeroBytes = 4096;
template <typename O, int V>
__device__ __forceinline__ void zero_rows(const RowSumArgs& a, int64_t first, int count, const uint8_t* touched, uint4* zeros) {
    const int64_t bytes = (int64_t)a.hd * sizeof(O);
    if ((reinterpret_cast<uintptr_t>(a.out) | (uintptr_t)bytes) % 16 == 0) {
        for (int i = threadIdx.x; i < kZeroBytes / 16; i += kThreads) zeros[i] = make_uint4(0u, 0u, 0u, 0u);
        fence_proxy_async_shared();
        __syncthreads();
        char* rows = static_cast<char*>(a.out) + first * bytes;
        const int parts = (int)((bytes + kZeroBytes - 1) / kZeroBytes);
        for (int u = threadIdx.x; u < count * parts; u += kThreads) {
            const int r = u / parts;
            const int64_t at = (int64_t)(u - r * parts) * kZeroBytes;
            if (!touched[r]) bulk_s2g(rows + r * bytes + at, zeros, (uint32_t)min((int64_t)kZeroBytes, bytes - at));
        }
        bulk_commit();
        bulk_wait_read_all();  // the block's shared memory is given back with its end
        return;
    }
    Pack<O, V> none;
#pragma unroll
    for (int c = 0; c < V; ++c) none.v[c] = O(0);
    for (int r = threadIdx.x >> 5; r < count; r += kWarps) {
        if (touched[r]) continue;
        O* row = static_cast<O*>(a.out) + (first + r) * a.hd;
        for (int c = (threadIdx.x & 31) * V; c < a.hd; c += 32 * V) *reinterpret_cast<Pack<O, V>*>(row + c) = none;
    }
}

// Which of the launch's blocks sets rows to zero, the `zero_blocks` of them spread evenly among the others: its number, or
// -1 less that of another.
__device__ __forceinline__ int64_t zero_block(const RowSumArgs& a) {
    const uint64_t b = blockIdx.x, z = (uint64_t)a.zero_blocks, before = b * z / gridDim.x;
    return (b + 1) * z / gridDim.x > before ? (int64_t)before : -1 - (int64_t)(b - before);
}

// An entry as its warp sums it.
template <typename D>
struct alignas(16) Entry {
    const D* row;
    float w;
    uint32_t key;
};

// ---------------------------------------------------------------- few entries

template <typename D, typename O, int V>
__global__ void __launch_bounds__(kThreads) direct_kernel(const RowSumArgs a, int zero_span) {
    __shared__ uint32_t keys[kDirect];
    __shared__ uint16_t list[kWarps][kDirect];
    __shared__ Entry<D> batch[kWarps][32];
    __shared__ uint8_t touched[kZeroRows];
    __shared__ uint4 zeros[kZeroBytes / 16];
    grid_dependency_wait();
    grid_launch_dependents();
    const int n = (int)a.entries, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t zero = zero_block(a);
    uint32_t own[kDirect / kThreads];
    keys_of<kDirect / kThreads>(a, threadIdx.x, kThreads, own);
    for (int i = 0; i < kDirect / kThreads; ++i) keys[i * kThreads + threadIdx.x] = own[i];
    if (zero >= 0) {
        const int64_t first = zero * zero_span;
        const int count = (int)min((int64_t)zero_span, a.n_slots - first);
        for (int r = threadIdx.x; r < count; r += kThreads) touched[r] = 0;
        __syncthreads();
        for (int e = threadIdx.x; e < n; e += kThreads)
            if (keys[e] >= first && keys[e] < first + count) touched[keys[e] - first] = 1;
        __syncthreads();
        zero_rows<O, V>(a, first, count, touched, zeros);
        return;
    }
    __syncthreads();
    const int64_t unit = (-1 - zero) * kWarps + warp;
    const int e = (int)(unit / a.slices);
    if (e >= n) return;
    const uint32_t key = keys[e];
    if (key >= a.n_slots) return;
    int found = 0;  // the entries of the slot, in order
    for (int base = 0; base < n; base += 32) {
        const int i = base + lane;
        const bool same = i < n && keys[i] == key;
        const unsigned mask = __ballot_sync(kAll, same);
        if (found == 0 && mask != 0 && base + __ffs(mask) - 1 < e) return;  // another warp's
        if (same) list[warp][found + __popc(mask & ((1u << lane) - 1))] = (uint16_t)i;
        found += __popc(mask);
    }
    __syncwarp();
    const int in_slice = lane * V, col = (int)(unit % a.slices) * a.slice_cols + in_slice;
    const bool on = in_slice < a.slice_cols && col < a.hd;
    float sum[V];
#pragma unroll
    for (int c = 0; c < V; ++c) sum[c] = 0.0f;
    Pack<O, V> there;
    if (a.accumulate && on) there = load_pack<O, V>(place_in<O>(a, key, col));  // on its way meanwhile
    Entry<D>* mine = batch[warp];
    for (int base = 0; base < found; base += 32) {
        if (base + lane < found) {
            const Place p = place_of(a, list[warp][base + lane]);
            mine[lane] = {static_cast<const D*>(p.op ? a.dout[1] : a.dout[0]) + (uint64_t)p.token * (uint32_t)a.hd, weight_of(a, p.op, p.at), key};
        }
        __syncwarp();
        const int left = min(found - base, 32);
        constexpr int U = 16;
        for (int j0 = 0; j0 < left; j0 += U) {
            Pack<D, V> x[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (j0 + u < left && on) x[u] = load_pack<D, V>(mine[j0 + u].row + col);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (j0 + u < left) {
                    const float w = mine[j0 + u].w;
#pragma unroll
                    for (int c = 0; c < V; ++c) sum[c] = fmaf(w, to_f32(x[u].v[c]), sum[c]);
                }
            }
        }
        __syncwarp();
    }
    if (!on) return;
    put_row<O, V>(a, a.accumulate, key, col, sum, there);
}

// ---------------------------------------------------------------- the sort

// The digits of a pass.
struct Digit {
    int shift, bits;
    __device__ __forceinline__ uint32_t of(uint32_t key) const { return key >> shift & ((1u << bits) - 1); }
    __device__ __forceinline__ int end() const { return min(shift + bits, 32); }  // the last digit may be short
};

// The counts of a tile's digits, counts[tile][digit]. FIRST: the keys are made here and kept, and entries
// that take no part are not counted; later passes have the others only.
template <bool FIRST, int ITEMS>
__global__ void __launch_bounds__(kThreads) digit_count_kernel(const RowSumArgs a, uint32_t* keys, const uint2* in, uint32_t* counts, Digit digit) {
    __shared__ uint32_t bins[1 << kMostBits];
    grid_dependency_wait();
    grid_launch_dependents();
    const uint32_t entries = FIRST ? a.entries : a.counters[0], from = blockIdx.x * (uint32_t)(kThreads * ITEMS);
    if (FIRST && blockIdx.x == 0 && threadIdx.x < 2) a.counters[threadIdx.x] = 0;
    const int all = 1 << digit.bits;
    for (int b = threadIdx.x; b < all; b += kThreads) bins[b] = 0;
    __syncthreads();
    constexpr int BATCH = ITEMS < 8 ? ITEMS : 8;
    for (int i0 = 0; i0 < ITEMS; i0 += BATCH) {
        const uint32_t first = from + i0 * kThreads + threadIdx.x;
        uint32_t key[BATCH];
        if constexpr (FIRST) {
            keys_of<BATCH>(a, first, kThreads, key);
        } else {
#pragma unroll
            for (int i = 0; i < BATCH; ++i) {
                const uint32_t e = first + i * kThreads;
                key[i] = e < entries ? in[e].x : (uint32_t)a.n_slots;
            }
        }
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
            const uint32_t e = first + i * kThreads;
            if (FIRST && e < entries) keys[e] = key[i];
            if (key[i] < a.n_slots) atomicAdd(&bins[digit.of(key[i])], 1u);
        }
    }
    __syncthreads();
    for (int b = threadIdx.x; b < all; b += kThreads) counts[((int64_t)blockIdx.x << digit.bits) + b] = bins[b];
}

// The sum of `own` over the block's threads before this one, and over all of them.
template <int WARPS>
__device__ __forceinline__ uint32_t sum_before(uint32_t own, uint32_t* sums, uint32_t* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t sum = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(kAll, sum, o);
        if (lane >= o) sum += y;
    }
    if (lane == 31) sums[warp] = sum;
    __syncthreads();
    uint32_t before = 0, every = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        if (w < warp) before += sums[w];
        every += sums[w];
    }
    *total = every;
    return before + sum - own;
}

// Each digit's counts become their running sums over the tiles, and their total. A block takes 8 digits, whose
// counts of a tile are one 32-byte sector; 128 threads a digit share out the tiles.
constexpr int kScanThreads = 1024, kScanDigits = 8, kScanShares = kScanThreads / kScanDigits;
__global__ void __launch_bounds__(kScanThreads) digit_scan_kernel(uint32_t* counts, uint32_t* totals, int tiles, int bits) {
    __shared__ uint32_t sums[kScanShares][kScanDigits + 1];
    grid_dependency_wait();
    grid_launch_dependents();
    const int in = threadIdx.x % kScanDigits, share = threadIdx.x / kScanDigits, digit = blockIdx.x * kScanDigits + in;
    const int each = (tiles + kScanShares - 1) / kScanShares, first = share * each, last = min(first + each, tiles);
    const bool on = digit < 1 << bits;
    uint32_t* column = counts + (on ? digit : 0);
    constexpr int U = 16;
    uint32_t own[U], sum = 0;  // of as many tiles as a thread has, up to 2048 of them; of more they are read again
    for (int t0 = first; t0 < last; t0 += U) {
#pragma unroll
        for (int i = 0; i < U; ++i) own[i] = t0 + i < last ? column[(int64_t)(t0 + i) << bits] : 0u;
#pragma unroll
        for (int i = 0; i < U; ++i) sum += own[i];
    }
    sums[share][in] = sum;
    __syncthreads();
    if (threadIdx.x < 32 * kScanDigits) {  // a warp for each digit, four shares a lane
        const int d = threadIdx.x >> 5, lane = threadIdx.x & 31;
        uint32_t part[kScanShares / 32], mine = 0;
#pragma unroll
        for (int i = 0; i < kScanShares / 32; ++i) mine += part[i] = sums[lane * (kScanShares / 32) + i][d];
        uint32_t before = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t y = __shfl_up_sync(kAll, before, o);
            if (lane >= o) before += y;
        }
        if (lane == 31 && blockIdx.x * kScanDigits + d < 1 << bits) totals[blockIdx.x * kScanDigits + d] = before;
        before -= mine;
#pragma unroll
        for (int i = 0; i < kScanShares / 32; ++i) {
            sums[lane * (kScanShares / 32) + i][d] = before;
            before += part[i];
        }
    }
    __syncthreads();
    if (!on) return;
    uint32_t before = sums[share][in];
    for (int t0 = first; t0 < last; t0 += U) {
        if (each > U) {
#pragma unroll
            for (int i = 0; i < U; ++i) own[i] = t0 + i < last ? column[(int64_t)(t0 + i) << bits] : 0u;
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (t0 + i < last) column[(int64_t)(t0 + i) << bits] = before;
            before += own[i];
        }
    }
}

// ---------------------------------------------------------------- up to 32768 entries: one cluster

// The blocks of a cluster hold the entries in shared memory and each other's within reach, so that a pass of the sort
// costs two barriers of the cluster and not three launches. What goes to other blocks goes there in pieces of 8 bytes,
// though: with four entries a thread launches are faster again (65536 entries: 21 us and launches 18, both alone).
constexpr int kCluster = 16, kClusterThreads = 1024, kClusterWarps = kClusterThreads / 32, kClusterBits = 10;
constexpr uint32_t kClustered = kCluster * kClusterThreads * 2;

// Block r holds places r * size .. of the entries, `size` a power of two, ITEMS entries a thread.
template <int ITEMS>
__global__ void __launch_bounds__(kClusterThreads, 1) cluster_sort_kernel(const RowSumArgs a, uint2* sorted, int passes, int bits) {
    constexpr uint32_t size = kClusterThreads * ITEMS;
    extern __shared__ uint2 cluster_smem[];
    __shared__ uint32_t sums[kClusterWarps];
    const int all = 1 << bits, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint2* buffers = cluster_smem;  // two of `size` pairs, the second for a third pass on
    uint32_t* hist = reinterpret_cast<uint32_t*>(buffers + (passes > 2 ? 2 : 1) * size);  // this block's count of each digit
    uint32_t* offset = hist + all;                                                        // where it puts the first of them
    uint16_t* own = reinterpret_cast<uint16_t*>(offset + all) + warp * all;               // a warp's counts, then their sums
    const uint16_t* owns = reinterpret_cast<uint16_t*>(offset + all);
    grid_dependency_wait();
    grid_launch_dependents();
    const uint32_t rank = cluster_rank(), first = rank * size;
    uint32_t entries = a.entries;  // those left
    for (int p = 0; p < passes; ++p) {
        const Digit digit{p * bits, bits};
        const uint2* in = buffers + ((p - 1) & 1) * size;
        for (int b = lane; b < all; b += 32) own[b] = 0;
        __syncwarp();
        // a warp's entries are consecutive, 32 at a time
        const uint32_t local = warp * (32 * ITEMS) + lane;
        uint32_t key[ITEMS], place[ITEMS];
        if (p == 0) {
            keys_of<ITEMS>(a, first + local, 32, key);
        } else {
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) key[i] = first + local + i * 32 < entries ? in[local + i * 32].x : (uint32_t)a.n_slots;
        }
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) place[i] = __ballot_sync(kAll, key[i] < a.n_slots);
        for (int b = digit.shift; b < digit.end(); ++b) {
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) {
                const uint32_t bit = key[i] >> b & 1;
                place[i] &= ~(__ballot_sync(kAll, bit) ^ (0u - bit));
            }
        }
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const unsigned same = place[i];
            const uint32_t d = digit.of(key[i]), before = own[d];
            __syncwarp();
            if (key[i] < a.n_slots && lane == 31 - __clz(same)) own[d] = (uint16_t)(before + __popc(same));
            __syncwarp();
            place[i] = before + __popc(same & ((1u << lane) - 1));
        }
        __syncthreads();
        // a thread for each digit: its sums over the warps, and then over the blocks
        if (tid < all) {
            uint32_t run = 0;
#pragma unroll 8
            for (int w = 0; w < kClusterWarps; ++w) {
                uint16_t* at = const_cast<uint16_t*>(owns) + w * all + tid;
                const uint32_t c = *at;
                *at = (uint16_t)run;
                run += c;
            }
            hist[tid] = run;
        }
        cluster_sync();
        uint32_t total = 0, earlier = 0, live;
        if (tid < all) {
#pragma unroll
            for (uint32_t q = 0; q < kCluster; ++q) {
                const uint32_t c = cluster_load(cluster_address(hist + tid, q));
                total += c;
                if (q < rank) earlier += c;
            }
        }
        const uint32_t start = sum_before<kClusterWarps>(total, sums, &live);
        if (tid < all) offset[tid] = start + earlier;
        if (p == 0 && rank == 0 && tid == 0) {
            a.counters[0] = live;
            a.counters[1] = 0;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            if (key[i] < a.n_slots) {
                const uint32_t d = digit.of(key[i]), to = offset[d] + own[d] + place[i];
                const uint2 pair = make_uint2(key[i], p == 0 ? first + local + i * 32 : in[local + i * 32].y);
                if (p + 1 == passes)
                    sorted[to] = pair;
                else
                    cluster_store(cluster_address(buffers + (p & 1) * size + to % size, to / size), pair);
            }
        }
        entries = live;
        cluster_sync();  // what others wrote here is here, and nobody reads here any more
    }
}

// ---------------------------------------------------------------- more: a launch for each step

// A tile's entries go to their places: behind all smaller digits, behind the same digit of earlier tiles, in order. They
// are put in order in shared memory first, so that what goes to one place is written side by side. (Later passes over
// tiles of 4096 spill 32 bytes a thread, for a third block an SM.)
template <bool FIRST, int ITEMS>
__global__ void __launch_bounds__(kThreads, 3) digit_place_kernel(const RowSumArgs a, const uint32_t* keys, const uint2* in, uint2* out,
                                                                  const uint32_t* counts, const uint32_t* totals, Digit digit) {
    constexpr int TILE = kThreads * ITEMS;
    // a warp's counts of each digit; then the tile's entries
    __shared__ union {
        uint16_t own[kWarps][1 << kMostBits];
        uint2 staged[TILE];
    } m;
    __shared__ uint32_t shift_of[1 << kMostBits];  // from an entry's place in the tile to its place in the output
    __shared__ uint32_t sums[kWarps];
    grid_dependency_wait();
    grid_launch_dependents();
    const int all = 1 << digit.bits, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t entries = FIRST ? a.entries : a.counters[0], tile = blockIdx.x;
    if (tile * (uint32_t)TILE >= entries && !(FIRST && tile == 0)) return;
    for (int b = lane * 2; b < all; b += 64) *reinterpret_cast<uint32_t*>(&m.own[warp][b]) = 0;
    __syncwarp();
    // a warp's entries are consecutive, 32 at a time
    const uint32_t from = tile * (uint32_t)TILE + warp * (32 * ITEMS);
    uint32_t key[ITEMS], rank[ITEMS];
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const uint32_t e = from + i * 32 + lane;
        key[i] = (uint32_t)a.n_slots;
        if (e < entries) key[i] = FIRST ? keys[e] : in[e].x;
    }
    // lanes with the same digit, bit by bit (a match over all bits at once took half as long again)
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) rank[i] = __ballot_sync(kAll, key[i] < a.n_slots);
    for (int b = digit.shift; b < digit.end(); ++b) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            const uint32_t bit = key[i] >> b & 1;
            rank[i] &= ~(__ballot_sync(kAll, bit) ^ (0u - bit));
        }
    }
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const unsigned same = rank[i];
        if (FIRST && !__any_sync(kAll, same)) continue;  // padding comes in runs
        const uint32_t d = digit.of(key[i]), before = m.own[warp][d];
        __syncwarp();
        if (key[i] < a.n_slots && lane == 31 - __clz(same)) m.own[warp][d] = (uint16_t)(before + __popc(same));
        __syncwarp();
        rank[i] = before + __popc(same & ((1u << lane) - 1));
    }
    __syncthreads();
    // Where each digit starts, among all entries and in the tile: running sums over the digits, up to eight consecutive
    // ones a thread.
    constexpr int PER = (1 << kMostBits) / kThreads;
    const int per = (all + kThreads - 1) / kThreads, b0 = threadIdx.x * per;
    uint32_t total[PER], earlier[PER], of_all = 0, of_tile = 0, unused;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        total[i] = earlier[i] = 0;
        const int b = b0 + i;
        if (i < per && b < all) {
            total[i] = __ldg(totals + b);
            earlier[i] = __ldg(counts + ((int64_t)tile << digit.bits) + b);
            of_all += total[i];
            uint32_t run = 0;
            for (int w = 0; w < kWarps; ++w) run += m.own[w][b];
            of_tile += run;
        }
    }
    uint32_t start = sum_before<kWarps>(of_all, sums, &unused), live;
    if (FIRST && tile == 0 && threadIdx.x == 0) a.counters[0] = unused;
    __syncthreads();
    uint32_t local = sum_before<kWarps>(of_tile, sums, &live);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int b = b0 + i;
        if (i < per && b < all) {
            shift_of[b] = start + earlier[i] - local;
            start += total[i];
            for (int w = 0; w < kWarps; ++w) {
                const uint32_t c = m.own[w][b];
                m.own[w][b] = (uint16_t)local;
                local += c;
            }
        }
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ITEMS; ++i)
        if (key[i] < a.n_slots) rank[i] += m.own[warp][digit.of(key[i])];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ITEMS; ++i) {
        const uint32_t e = from + i * 32 + lane;
        if (key[i] < a.n_slots) m.staged[rank[i]] = make_uint2(key[i], FIRST ? e : in[e].y);
    }
    __syncthreads();
#pragma unroll 4
    for (uint32_t p = threadIdx.x; p < live; p += kThreads) {
        const uint2 pair = m.staged[p];
        out[p + shift_of[digit.of(pair.x)]] = pair;
    }
}

// ---------------------------------------------------------------- the sums

// The first place whose key is not below `key`, in sorted[lo, hi).
__device__ __forceinline__ uint32_t lower_bound(const uint2* sorted, uint32_t lo, uint32_t hi, uint32_t key) {
    while (lo < hi) {
        const uint32_t mid = lo + (hi - lo) / 2;
        if (__ldg(&sorted[mid].x) < key)
            lo = mid + 1;
        else
            hi = mid;
    }
    return lo;
}

// The same by a warp, 32 places at a time.
__device__ __forceinline__ uint32_t warp_lower_bound(const uint2* sorted, uint32_t n, uint32_t key) {
    const int lane = threadIdx.x & 31;
    uint32_t lo = 0, len = n;  // the answer is in [lo, lo + len]
    while (len > 0) {
        const uint32_t step = (len + 31) / 32, at = min((uint32_t)lane * step + step, len) - 1;  // the last of each of 32 shares
        const bool below = __ldg(&sorted[lo + at].x) < key;
        const int shares = __popc(__ballot_sync(kAll, below));
        const uint32_t skip = min(shares * step, len);
        lo += skip;
        len = shares == 32 ? 0 : min(step, len - skip) - 1;  // the last of the share is not below
    }
    return lo;
}

constexpr uint32_t kShort = 32;  // entries of a run beyond the end of a piece that its warp sums as well

// A warp loads U rows of dout together, and the entries of the next batch meanwhile. Bound by latency and by what L2 gives:
// 65536 tokens of 64 and 32 entries over 2^20 rows of 128 read 1.6 GB of dout out of L2, and a call with 4 rows together and
// registers for 5 blocks an SM takes 292 us; 8 and 4 323, 2 and 6 298, 4 and 6 (spilled) 340; rows that wait in shared memory
// instead, 16 of them by cp.async, 381.
// ACC: sums are added to what is there, which is loaded beside the entries, so that it is at hand when a run ends.
template <typename D, typename O, int V, bool ACC>
__global__ void __launch_bounds__(kThreads, V <= 4 ? (ACC ? 3 : 5) : (ACC ? 2 : 3)) sums_kernel(const RowSumArgs a, int zero_span) {
    __shared__ union {
        uint4 zeros[kZeroBytes / 16];
        Entry<D> batch[kWarps][32];
    } m;
    __shared__ uint8_t touched[kZeroRows];
    __shared__ uint32_t range[2];
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x & 31;
    const uint32_t entries = a.counters[0];
    const int64_t zero = zero_block(a);
    if (zero >= 0) {
        const int64_t first = zero * zero_span;
        const int count = (int)min((int64_t)zero_span, a.n_slots - first), warp = threadIdx.x >> 5;
        if (warp < 2) range[warp] = warp_lower_bound(a.sorted, entries, (uint32_t)(first + warp * count));
        for (int r = threadIdx.x; r < count; r += kThreads) touched[r] = 0;
        __syncthreads();
        const uint32_t lo = range[0], hi = range[1];
        if (hi - lo <= 8 * kThreads) {
            for (uint32_t i = lo + threadIdx.x; i < hi; i += kThreads) touched[__ldg(&a.sorted[i].x) - first] = 1;
        } else {  // long runs: a search for each row
            for (int r = threadIdx.x; r < count; r += kThreads) {
                const uint32_t at = lower_bound(a.sorted, lo, hi, (uint32_t)(first + r));
                touched[r] = at < hi && __ldg(&a.sorted[at].x) == (uint32_t)(first + r);
            }
        }
        __syncthreads();
        zero_rows<O, V>(a, first, count, touched, m.zeros);
        return;
    }
    const int64_t unit = (-1 - zero) * kWarps + (threadIdx.x >> 5);
    const int64_t piece = unit / a.slices;
    uint32_t from = (uint32_t)min(piece * a.piece, (int64_t)entries), to = (uint32_t)min((piece + 1) * a.piece, (int64_t)entries);
    if (from >= to) return;
    const int slice = (int)(unit % a.slices), in_slice = lane * V, col = slice * a.slice_cols + in_slice;
    const bool on = in_slice < a.slice_cols && col < a.hd;
    // A run that began before this piece is summed by the warp before, if few of its entries are left here; else
    // its part here goes to `heads`, to be joined.
    bool continues = false;
    if (from > 0) {
        const uint32_t before = __ldg(&a.sorted[from - 1].x);
        const bool same = from + lane < entries && __ldg(&a.sorted[from + lane].x) == before;
        const unsigned rest = __ballot_sync(kAll, same);
        if (rest == kAll)
            continues = true;
        else
            from += __popc(rest);
    }
    bool goes_on = false;
    if (to < entries) {
        const uint32_t last = __ldg(&a.sorted[to - 1].x);
        const bool same = to + lane < entries && __ldg(&a.sorted[to + lane].x) == last;
        const unsigned rest = __ballot_sync(kAll, same);
        if (rest == kAll)
            goes_on = true;
        else if (from < to)  // not all of the piece was the end of another's run
            to += __popc(rest);
    }
    if (from >= to) return;
    uint32_t current = __ldg(&a.sorted[from].x);
    float sum[V];
#pragma unroll
    for (int c = 0; c < V; ++c) sum[c] = 0.0f;
    const auto flush = [&](bool ends, const Pack<O, V>& there) {
        if (continues || !ends) {
            if (on) {
                Pack<float, V> part;
#pragma unroll
                for (int c = 0; c < V; ++c) part.v[c] = sum[c];
                *reinterpret_cast<Pack<float, V>*>((continues ? a.heads : a.tails) + piece * a.hd + col) = part;
            }
            if (!continues && slice == 0 && lane == 0) a.list[atomicAdd(a.counters + 1, 1u)] = (uint32_t)piece;
        } else if (on) {
            put_row<O, V>(a, ACC, current, col, sum, there);
        }
        continues = false;
#pragma unroll
        for (int c = 0; c < V; ++c) sum[c] = 0.0f;
    };
    Entry<D>* mine = m.batch[threadIdx.x >> 5];
    const auto fetch = [&](uint32_t at) -> Entry<D> {
        if (at + lane >= to) return {nullptr, 0.0f, 0u};
        const uint2 pair = __ldg(a.sorted + at + lane);
        const Place p = place_of(a, pair.y);
        return {static_cast<const D*>(p.op ? a.dout[1] : a.dout[0]) + (uint64_t)p.token * (uint32_t)a.hd, weight_of(a, p.op, p.at), pair.x};
    };
    Entry<D> next = fetch(from);  // 32 entries ahead
    for (uint32_t base = from; base < to; base += 32) {
        // these 32 entries go through shared memory, where each of them is one load for the whole warp
        const int left = (int)min(to - base, 32u);
        const uint32_t key = next.key;
        mine[lane] = next;
        next = fetch(base + 32);
        uint32_t before = __shfl_up_sync(kAll, key, 1);
        if (lane == 0) before = current;
        __syncwarp();
        const unsigned begins = __ballot_sync(kAll, lane < left && key != before);  // entries that begin another run
        constexpr int U = 4;
        for (int j0 = 0; j0 < left; j0 += U) {
            const int count = left - j0;
            const unsigned first = begins >> j0;
            Pack<D, V> x[U];
            Pack<O, V> there[ACC ? U : 1];  // of the run before the entry
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (u < count && on) x[u] = load_pack<D, V>(mine[j0 + u].row + col);
                if (ACC && u < count && on) {
                    const uint32_t row = u > 0 ? mine[j0 + u - 1].key : current;
                    there[u] = load_pack<O, V>(place_in<O>(a, row, col));
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (u < count) {
                    if (first >> u & 1) {
                        flush(true, there[ACC ? u : 0]);
                        current = mine[j0 + u].key;
                    }
                    const float w = mine[j0 + u].w;
#pragma unroll
                    for (int c = 0; c < V; ++c) sum[c] = fmaf(w, to_f32(x[u].v[c]), sum[c]);
                }
            }
        }
        __syncwarp();
    }
    Pack<O, V> there;
    if (ACC && on) there = load_pack<O, V>(place_in<O>(a, current, col));
    flush(!goes_on, there);
}

// The listed runs, which go on far beyond the piece they begin in: the sum in that piece, then those in the pieces that
// continue it. A block for each run and slice; its warps share out the pieces of a long run.
template <typename O, int V>
__global__ void __launch_bounds__(kThreads) join_kernel(const RowSumArgs a) {
    __shared__ float parts[kWarps][32 * V];
    grid_dependency_wait();
    grid_launch_dependents();
    const uint32_t entries = a.counters[0];
    const int64_t units = (int64_t)a.counters[1] * a.slices;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const int64_t piece = a.list[unit / a.slices];
        const uint32_t key = __ldg(&a.sorted[(piece + 1) * a.piece].x);
        // the pieces that begin with this slot and go on with it for more than kShort entries
        const uint32_t from = (uint32_t)((piece + 1) * a.piece), end = from + warp_lower_bound(a.sorted + from, entries - from, key + 1);
        const int64_t more = ((int64_t)end - kShort) / a.piece - piece, share = (more + kWarps - 1) / kWarps;
        const int in_slice = lane * V, col = (int)(unit % a.slices) * a.slice_cols + in_slice;
        const bool on = in_slice < a.slice_cols && col < a.hd;
        float sum[V];
#pragma unroll
        for (int c = 0; c < V; ++c) sum[c] = 0.0f;
        if (on) {
            const int64_t last = min((warp + 1) * share, more);
#pragma unroll 8
            for (int64_t q = warp * share; q < last; ++q) {
                const Pack<float, V> part = load_pack<float, V>(a.heads + (piece + 1 + q) * a.hd + col);
#pragma unroll
                for (int c = 0; c < V; ++c) sum[c] += part.v[c];
            }
#pragma unroll
            for (int c = 0; c < V; ++c) parts[warp][in_slice + c] = sum[c];
        }
        __syncthreads();
        if (warp == 0 && on) {
            const Pack<float, V> tail = load_pack<float, V>(a.tails + piece * a.hd + col);
#pragma unroll
            for (int c = 0; c < V; ++c) {
                sum[c] = tail.v[c];
                for (int w = 0; w < kWarps; ++w) sum[c] += parts[w][in_slice + c];
            }
            Pack<O, V> there;
            if (a.accumulate) there = load_pack<O, V>(place_in<O>(a, key, col));
            put_row<O, V>(a, a.accumulate, key, col, sum, there);
        }
        __syncthreads();
    }
}

struct Kernels {
    const void *direct, *sums, *join;
};
template <typename D, typename O, int V>
Kernels kernels(bool accumulate) {
    return {(const void*)direct_kernel<D, O, V>, accumulate ? (const void*)sums_kernel<D, O, V, true> : (const void*)sums_kernel<D, O, V, false>,
            (const void*)join_kernel<O, V>};
}
template <typename D, typename O>
Kernels kernels(int v, bool accumulate) {
    constexpr int MOST = 16 / sizeof(D);
    return v == MOST       ? kernels<D, O, MOST>(accumulate)
           : v == MOST / 2 ? kernels<D, O, MOST / 2>(accumulate)
           : v == MOST / 4 ? kernels<D, O, MOST / 4>(accumulate)
                           : kernels<D, O, 1>(accumulate);
}

// Entries of a piece: as many as leave 8192 pieces and slices of 256 columns, so that all warps have work, from 16,
// below which the sums at the ends are most of the work, to 128.
uint32_t piece_of(int64_t entries, int hd) {
    const int64_t want = (entries * ((hd + 255) / 256) + 8191) / 8192;
    uint32_t piece = 16;
    while (piece < want && piece < 128) piece *= 2;
    return piece;
}
int64_t round_up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

Divisor divisor(int d) {
    int l = 0;
    while (((int64_t)1 << l) < d) ++l;
    if (l == 0) return {0u, 0};
    return {(uint32_t)((((uint64_t)1 << (31 + l)) + d - 1) / d), l - 1};
}

// The passes of the sort over slots below n_slots, with digits of `most` bits at most.
struct Radix {
    int passes, bits;
};
Radix radix_of(int64_t n_slots, int most) {
    int significant = 1;
    while ((n_slots - 1) >> significant != 0) ++significant;
    const int passes = (significant + most - 1) / most;
    return {passes, (significant + passes - 1) / passes};
}

// Entries of a thread of the sort by launches: tiles of 1024 entries, of which few entries make more blocks, up to 2^20 of
// them, else of 4096, whose digits come in longer runs. Whole calls over 2^20 and over 2^17 rows of 8, us, with tiles of 1024 and of
// 4096: 131072 entries 39, 48 and 31, 36; 262144 46, 60 and 39, 42; 2^20 115, 119 and 81, 88; 2^21 207, 186 and 169, 162;
// 6.3 million 572, 481 and 736, 691.
int items_of(int64_t entries) { return entries <= 1 << 20 ? 4 : 16; }
int64_t tiles_of(int64_t entries) { return (entries + kThreads * items_of(entries) - 1) / (kThreads * items_of(entries)); }

// Where everything lies in the workspace, in words.
struct Layout {
    int64_t counters, pairs, keys, counts, totals, heads, tails, list, words;
};
Layout layout_of(int64_t entries, int64_t n_slots, int hd) {
    const bool launches = entries > kClustered;
    const int64_t e = round_up(entries, 64), piece = piece_of(entries, hd), pieces = (entries + piece - 1) / piece;
    const int64_t tiles = tiles_of(entries);
    Layout l{};
    l.pairs = l.counters + 64;
    l.keys = l.pairs + (launches ? 4 : 2) * e;
    l.counts = l.keys + (launches ? e : 0);
    l.totals = l.counts + (launches ? round_up(tiles << radix_of(n_slots, kMostBits).bits, 64) : 0);
    l.heads = l.totals + (launches ? 1 << kMostBits : 0);
    l.tails = l.heads + round_up(pieces * hd, 64);
    l.list = l.tails + round_up(pieces * hd, 64);
    l.words = l.list + round_up(pieces, 64);
    return l;
}

// The sort by a cluster.
int launch_cluster_sort(const RowSumArgs& a, uint2* sorted, cudaStream_t stream) {
    const Radix r = radix_of(a.n_slots, kClusterBits);
    const uint32_t each = (a.entries + kCluster * kClusterThreads - 1) / (kCluster * kClusterThreads);  // entries of a thread
    const int items = each <= 1 ? 1 : 2;
    const void* fn = items == 1 ? (const void*)cluster_sort_kernel<1> : (const void*)cluster_sort_kernel<2>;
    const size_t smem = (size_t)(r.passes > 2 ? 2 : 1) * kClusterThreads * items * sizeof(uint2) + ((size_t)8 << r.bits) +
                        ((size_t)kClusterWarps * 2 << r.bits);
    int rc = allow_smem(fn, smem + 1024);  // and what the kernel has besides
    if (rc == 0) rc = (int)cudaFuncSetAttribute(fn, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (rc != 0) return rc;
    RowSumArgs args_a = a;
    int passes = r.passes, bits = r.bits;
    void* args[] = {&args_a, &sorted, &passes, &bits};
    return launch_cluster_raw(fn, kCluster, dim3(kCluster), dim3(kClusterThreads), smem, stream, args);
}

// Sorts the entries; `sorted` becomes where they are.
int launch_sort(const RowSumArgs& a, const Layout& l, uint32_t* words, const uint2** sorted, cudaStream_t stream) {
    Radix r = radix_of(a.n_slots, kMostBits);
    int tiles = (int)tiles_of(a.entries);
    const bool few = items_of(a.entries) == 4;
    uint32_t *keys = words + l.keys, *counts = words + l.counts, *totals = words + l.totals;
    uint2* pairs[2] = {reinterpret_cast<uint2*>(words + l.pairs), reinterpret_cast<uint2*>(words + l.pairs) + round_up(a.entries, 64)};
    RowSumArgs args = a;
    for (int p = 0; p < r.passes; ++p) {
        Digit digit{p * r.bits, r.bits};
        uint2 *in = pairs[~p & 1], *out = pairs[p & 1];
        void* count_args[] = {&args, &keys, &in, &counts, &digit};
        const void* count = p == 0 ? (few ? (const void*)digit_count_kernel<true, 4> : (const void*)digit_count_kernel<true, 16>)
                                   : (few ? (const void*)digit_count_kernel<false, 4> : (const void*)digit_count_kernel<false, 16>);
        int rc = launch_pdl_raw(count, dim3(tiles), dim3(kThreads), 0, stream, count_args);
        if (rc != 0) return rc;
        void* scan_args[] = {&counts, &totals, &tiles, &r.bits};
        rc = launch_pdl_raw((const void*)digit_scan_kernel, dim3(((1u << r.bits) + kScanDigits - 1) / kScanDigits), dim3(kScanThreads), 0,
                            stream, scan_args);
        if (rc != 0) return rc;
        void* place_args[] = {&args, &keys, &in, &out, &counts, &totals, &digit};
        const void* place = p == 0 ? (few ? (const void*)digit_place_kernel<true, 4> : (const void*)digit_place_kernel<true, 16>)
                                   : (few ? (const void*)digit_place_kernel<false, 4> : (const void*)digit_place_kernel<false, 16>);
        rc = launch_pdl_raw(place, dim3(tiles), dim3(kThreads), 0, stream, place_args);
        if (rc != 0) return rc;
        *sorted = out;
    }
    return 0;
}

}  // namespace

int64_t row_sums_workspace(int64_t entries, int64_t n_slots, int hd) {
    return entries <= kDirect ? 0 : 4 * layout_of(entries, n_slots, hd).words;
}

int launch_row_sums(const RowSumArgs& a0, cudaStream_t stream) {
    RowSumArgs a = a0;
    for (int o = 0; o < 2; ++o) a.by_width[o] = divisor(a.width[o]);
    a.by_chunk = divisor(a.chunk);
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
    const bool acc = a.accumulate != 0;
    const Kernels fn = a.dout_bf16 ? (a.out_bf16 ? kernels<uint16_t, uint16_t>(v, acc) : kernels<uint16_t, float>(v, acc))
                                   : (a.out_bf16 ? kernels<float, uint16_t>(v, acc) : kernels<float, float>(v, acc));
    // rows that a block sets to zero: 128 KB of them
    int zero_span = (int)std::clamp<int64_t>((int64_t)128 * 1024 / ((int64_t)a.hd * (a.out_bf16 ? 2 : 4)), 8, kZeroRows);
    a.zero_blocks = a.accumulate ? 0 : (a.n_slots + zero_span - 1) / zero_span;
    if (a.entries <= kDirect) {
        const int64_t blocks = a.zero_blocks + ((int64_t)a.entries * a.slices + kWarps - 1) / kWarps;
        if (blocks == 0) return 0;
        void* args[] = {&a, &zero_span};
        return launch_pdl_raw(fn.direct, dim3((unsigned)blocks), dim3(kThreads), 0, stream, args);
    }
    const Layout l = layout_of(a.entries, a.n_slots, a.hd);
    uint32_t* words = static_cast<uint32_t*>(a.workspace);
    a.counters = words + l.counters;
    a.heads = reinterpret_cast<float*>(words + l.heads);
    a.tails = reinterpret_cast<float*>(words + l.tails);
    a.list = words + l.list;
    a.piece = piece_of(a.entries, a.hd);
    const int64_t pieces = ((int64_t)a.entries + a.piece - 1) / a.piece, blocks = a.zero_blocks + (pieces * a.slices + kWarps - 1) / kWarps;
    if (blocks > INT_MAX) return SDM_ECOUNT;
    int rc;
    if (a.entries <= kClustered) {
        uint2* sorted = reinterpret_cast<uint2*>(words + l.pairs);
        rc = launch_cluster_sort(a, sorted, stream);
        a.sorted = sorted;
    } else {
        rc = launch_sort(a, l, words, &a.sorted, stream);
    }
    if (rc != 0) return rc;
    void* args[] = {&a, &zero_span};
    rc = launch_pdl_raw(fn.sums, dim3((unsigned)blocks), dim3(kThreads), 0, stream, args);
    if (rc != 0) return rc;
    const int64_t joins = std::min<int64_t>(pieces * a.slices, 2 * sm_count());
    return launch_pdl_raw(fn.join, dim3((unsigned)joins), dim3(kThreads), 0, stream, args);
}

cudaError_t row_sums_status(void** word) { return cudaGetSymbolAddress(word, g_row_sums_status); }

}  // namespace sdm
