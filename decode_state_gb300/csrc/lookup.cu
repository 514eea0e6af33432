// Scaled rows of a table by token.
//
// Math (include/sdm.h): out[t] = round(scale * row(token[t])), zeros for a padding token.
//
// Design. A copy, bound by memory: a team of lanes moves 16 bytes of the table each, of ROWS rows at once, whose tokens
// and then rows are loaded together before any is stored. Rows longer than 256 such accesses are shared by blocks.
#include <algorithm>
#include <climits>
#include <cstring>

#include "sdm.h"
#include "sdm_device.cuh"
#include "sdm_internal.h"

namespace sdm {
namespace {

__device__ unsigned int g_lookup_status;

constexpr int kThreads = 256;

// V elements of type T moved together.
template <typename T, int V>
struct alignas(sizeof(T) * V < 16 ? sizeof(T) * V : 16) Pack {
    T v[V];
};

template <typename T, typename O, int V, int ROWS>
__global__ void __launch_bounds__(kThreads) lookup_kernel(const LookupArgs a) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int lanes = 1 << a.lane_bits, teams = kThreads >> a.lane_bits, lane = threadIdx.x & (lanes - 1);
    const int64_t group = blockIdx.x / a.column_blocks;
    const int col = ((int)(blockIdx.x - group * a.column_blocks) * lanes + lane) * V;
    const int64_t first = group * (teams * ROWS) + (threadIdx.x >> a.lane_bits);
    if (col >= a.hd) return;
    int64_t slot[ROWS];
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const int64_t t = first + r * teams;
        slot[r] = 0;
        if (t < a.n_tokens) slot[r] = a.idx64 ? __ldg(static_cast<const int64_t*>(a.tokens) + t) : __ldg(static_cast<const int32_t*>(a.tokens) + t);
    }
    Pack<T, V> x[ROWS];
    bool outside = false;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        const bool in = slot[r] >= 0 && slot[r] < a.n_rows, none = slot[r] == a.padding && a.padding != SDM_NO_PADDING;
        outside |= !in && !none;
        if (!in || none) slot[r] = -1;
        if (slot[r] >= 0) x[r] = *reinterpret_cast<const Pack<T, V>*>(static_cast<const T*>(a.table) + slot[r] * a.hd + col);
    }
    if (outside) atomicOr(&g_lookup_status, SDM_DEV_BAD_INDEX);
    O* to = static_cast<O*>(a.out) + first * a.hd + col;
#pragma unroll
    for (int r = 0; r < ROWS; ++r) {
        if (first + r * teams >= a.n_tokens) break;
        Pack<O, V> y;
        if (slot[r] < 0) {
#pragma unroll
            for (int c = 0; c < V; ++c) y.v[c] = O(0);
        } else if constexpr (sizeof(T) == 2 && V > 1) {
            uint32_t w[V / 2];
            memcpy(w, &x[r], sizeof(w));
#pragma unroll
            for (int c = 0; c < V / 2; ++c) {
                const float low = __uint_as_float(w[c] << 16) * a.scale, high = __uint_as_float(w[c] & 0xffff0000u) * a.scale;
                if constexpr (sizeof(O) == 2) {
                    const __nv_bfloat162 b = __floats2bfloat162_rn(low, high);
                    memcpy(&w[c], &b, 4);
                } else {
                    y.v[2 * c] = low;
                    y.v[2 * c + 1] = high;
                }
            }
            if constexpr (sizeof(O) == 2) memcpy(&y, w, sizeof(w));
        } else {
#pragma unroll
            for (int c = 0; c < V; ++c) y.v[c] = from_f32<O>(to_f32(x[r].v[c]) * a.scale);
        }
        *reinterpret_cast<Pack<O, V>*>(to) = y;
        to += (int64_t)teams * a.hd;
    }
}

template <typename T, typename O>
const void* kernel(bool vec, bool many) {
    constexpr int V = 16 / sizeof(T);
    return vec ? (many ? (const void*)lookup_kernel<T, O, V, 4> : (const void*)lookup_kernel<T, O, V, 1>) : (const void*)lookup_kernel<T, O, 1, 4>;
}

}  // namespace

int launch_lookup(const LookupArgs& a0, cudaStream_t stream) {
    LookupArgs a = a0;
    const int v = a.table_bf16 ? 8 : 4;
    const bool vec = a.hd % v == 0 && reinterpret_cast<uintptr_t>(a.table) % 16 == 0 &&
                     reinterpret_cast<uintptr_t>(a.out) % std::min(16, v * (a.out_bf16 ? 2 : 4)) == 0;
    const int accesses = vec ? a.hd / v : a.hd;
    // of 8 to 256 lanes, the most that leave the fewest without work in a row's last access
    a.lane_bits = 3;
    for (int bits = 4, least = (accesses + 7) / 8 * 8; bits <= 8; ++bits) {
        const int taken = (accesses + (1 << bits) - 1 >> bits) << bits;
        if (taken <= least) {
            least = taken;
            a.lane_bits = bits;
        }
    }
    a.column_blocks = (accesses + (1 << a.lane_bits) - 1) >> a.lane_bits;
    const int teams = kThreads >> a.lane_bits;
    const bool many = !vec || a.n_tokens * a.column_blocks >= (int64_t)8 * 4 * teams * sm_count();
    const int64_t blocks = (a.n_tokens + teams * (many ? 4 : 1) - 1) / (teams * (many ? 4 : 1)) * a.column_blocks;
    if (blocks > INT_MAX) return SDM_ECOUNT;
    const void* fn = a.table_bf16 ? (a.out_bf16 ? kernel<uint16_t, uint16_t>(vec, many) : kernel<uint16_t, float>(vec, many))
                                  : (a.out_bf16 ? kernel<float, uint16_t>(vec, many) : kernel<float, float>(vec, many));
    void* args[] = {&a};
    return launch_pdl_raw(fn, dim3((unsigned)blocks), dim3(kThreads), 0, stream, args);
}

cudaError_t lookup_status(void** word) { return cudaGetSymbolAddress(word, g_lookup_status); }

}  // namespace sdm
