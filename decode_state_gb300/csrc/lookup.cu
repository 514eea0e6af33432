// Scaled rows of a table by token.
//
// Math (include/sdm.h): out[t] = round(scale * row(token[t])), zeros for a padding token.
//
// Design. A copy, bound by memory: a thread moves kUnits accesses of 16 bytes of the table, whose tokens and then
// rows it loads together before it stores any. Consecutive threads take consecutive accesses of a row and then the
// next row's, so that rows of any length leave no thread without work.
#include <algorithm>
#include <climits>

#include "sdm.h"
#include "sdm_device.cuh"
#include "sdm_internal.h"

namespace sdm {
namespace {

__device__ unsigned int g_lookup_status;

constexpr int kThreads = 256, kUnits = 4;

// V elements of type T moved together.
template <typename T, int V>
struct alignas(sizeof(T) * V < 16 ? sizeof(T) * V : 16) Pack {
    T v[V];
};

template <typename T, typename O, int V>
__global__ void __launch_bounds__(kThreads) lookup_kernel(const LookupArgs a) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int64_t from = (int64_t)blockIdx.x * (kThreads * kUnits);
    const int64_t t0 = from / a.per_row;  // the block's first token, and the access of its row
    const uint32_t first = (uint32_t)(from - t0 * a.per_row);
    Pack<T, V> x[kUnits];
    int64_t to[kUnits];
    int64_t slot[kUnits];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        const uint32_t at = first + threadIdx.x + u * kThreads;
        const uint32_t row = a.magic ? __umulhi(at, a.magic) : at / a.per_row;
        const int64_t t = t0 + row;
        to[u] = t < a.n_tokens ? t * a.hd + (int64_t)(at - row * a.per_row) * V : -1;
        slot[u] = -1;
        if (to[u] >= 0) {
            slot[u] = a.idx64 ? __ldg(static_cast<const int64_t*>(a.tokens) + t) : __ldg(static_cast<const int32_t*>(a.tokens) + t);
            if (slot[u] == a.padding) {
                slot[u] = -1;
            } else if (slot[u] < 0 || slot[u] >= a.n_rows) {
                slot[u] = -1;
                atomicOr(&g_lookup_status, SDM_DEV_BAD_INDEX);
            }
            if (slot[u] >= 0) slot[u] = slot[u] * a.hd + (int64_t)(at - row * a.per_row) * V;
        }
    }
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        if (slot[u] >= 0)
            x[u] = *reinterpret_cast<const Pack<T, V>*>(static_cast<const T*>(a.table) + slot[u]);
        else
#pragma unroll
            for (int c = 0; c < V; ++c) x[u].v[c] = T(0);
    }
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
        if (to[u] < 0) continue;
        Pack<O, V> y;
#pragma unroll
        for (int c = 0; c < V; ++c) y.v[c] = from_f32<O>(slot[u] >= 0 ? to_f32(x[u].v[c]) * a.scale : 0.0f);
        *reinterpret_cast<Pack<O, V>*>(static_cast<O*>(a.out) + to[u]) = y;
    }
}

template <typename T, typename O>
const void* kernel(bool vec) {
    return vec ? (const void*)lookup_kernel<T, O, 16 / sizeof(T)> : (const void*)lookup_kernel<T, O, 1>;
}

}  // namespace

int launch_lookup(const LookupArgs& a0, cudaStream_t stream) {
    LookupArgs a = a0;
    const int v = a.table_bf16 ? 8 : 4;
    const bool vec = a.hd % v == 0 && reinterpret_cast<uintptr_t>(a.table) % 16 == 0 &&
                     reinterpret_cast<uintptr_t>(a.out) % std::min(16, v * (a.out_bf16 ? 2 : 4)) == 0;
    a.per_row = vec ? a.hd / v : a.hd;
    // x * magic >> 32 is x / per_row for x < 2^32 / per_row, and x < per_row + 1024 here
    a.magic = a.per_row > 1 && a.per_row <= 32768 ? (uint32_t)(((uint64_t)1 << 32) / a.per_row + 1) : 0;
    const int64_t units = a.n_tokens * a.per_row, blocks = (units + kThreads * kUnits - 1) / (kThreads * kUnits);
    if (blocks > INT_MAX) return SDM_ECOUNT;
    const void* fn = a.table_bf16 ? (a.out_bf16 ? kernel<uint16_t, uint16_t>(vec) : kernel<uint16_t, float>(vec))
                                  : (a.out_bf16 ? kernel<float, uint16_t>(vec) : kernel<float, float>(vec));
    void* args[] = {&a};
    return launch_pdl_raw(fn, dim3((unsigned)blocks), dim3(kThreads), 0, stream, args);
}

cudaError_t lookup_status(void** word) { return cudaGetSymbolAddress(word, g_lookup_status); }

}  // namespace sdm
