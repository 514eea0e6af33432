// Write-then-read tokens on a quantised bank.
//
// Math (include/sdm.h), per stream and token, row = scale * code, d_w = exp(g_w):
//     retrieved = sum_w k_w d_w row_w,  delta = beta (v - retrieved)
//     row_w <- quantised(d_w row_w + k_w delta),  out = sum_r q_r row_r  (after the write)
//
// Design. Everything but a group's scale is independent by columns, so one block owns a (stream,
// slice of 8 pieces = 128 columns, a whole number of scale groups) for all T tokens, and a block
// barrier orders a token's writes before its reads: no other block touches those bytes. LR lanes
// hold a row's slice, 16 bytes each, so a thread keeps its few rows' codes in registers from the
// retrieval to the write-back: each row is read once and written once, and the group's maximum is
// a shuffle among neighbouring lanes. The sums over rows go through shuffles within a warp and
// shared memory across warps, in a fixed order.
//
// A token is a chain of dependent steps, so the waits for memory are taken off the chain. One thread
// for each entry loads its slot, weight and gate two tokens ahead into registers, turns them into a
// record in shared memory and warms the row in L2; a value column's thread does the same with v. And
// behind the barrier that ends a token's writes its read rows and the next token's write rows are
// requested together, without branches between the requests, so a token waits once, for L2.
//
// What bounds it: instructions. 512 streams of 64 and 64 rows of 128 columns take 4.6 us a token (3.1 TB/s
// through L2, where the state of a chunk of tokens stays); a warp spends 1326 instructions on its 16 and 16
// rows, at 0.55 a cycle and scheduler, 876 of them on the rows written: their 8-bit codes are unpacked for the
// retrieval, for the scale and for the new codes, since the columns of four rows do not fit the registers.
// Keeping them two rows at a time spills (4.8 us). So 8-bit rows halve the bytes of a bf16 bank, not its time: 1024
// streams of 16384 rows, from HBM, 64 and 64 a token, 32 tokens take 10.2 us a token (int8) or 9.6 (fp8) and 8.7 on bf16 rows.
#include <algorithm>
#include <climits>

#include "quant_device.cuh"
#include "sdm_internal.h"

namespace sdm {
namespace {

__device__ unsigned int g_qdecode_status;

constexpr unsigned kAll = 0xffffffffu;

// One entry of a token: where its row is, its weight, and for a write its decay.
struct __align__(16) Entry {
    int slot;  // -1: none
    float weight, decay, unused;
};
constexpr int kRing = 3;  // tokens whose entries are kept

// Sum x[0..16) over the row slots of a warp (lanes LR apart); x[0 .. 16 * LR / 32) then holds the
// columns from the returned one on.
template <int LR>
__device__ __forceinline__ int reduce_rows(float* x, int lane) {
    int first = 0, half = 8;
#pragma unroll
    for (int o = 16; o >= LR; o >>= 1) {
        const bool up = lane & o;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i < half) {
                const float keep = up ? x[i + half] : x[i], give = up ? x[i] : x[i + half];
                x[i] = keep + __shfl_xor_sync(kAll, give, o);
            }
        }
        first += up ? half : 0;
        half /= 2;
    }
    return first;
}

// F: Int8 or Fp8. LR: lanes of a row slice (its columns: 16 * LR). NT: threads. RPT: rows a thread
// holds. ITEMS: entries (W + R of them) that a thread prepares.
// The registers are bounded for four blocks of 128 threads an SM, or two of 256: 512 streams of 64 rows take
// 4.6 us a token with 128 registers, 12 with the 153 it would use, in two waves.
template <typename F, int LR, int NT, int RPT, int ITEMS>
__global__ void __launch_bounds__(NT, NT == 512 ? 1 : NT == 256 ? 2 : 4) qdecode_kernel(const QDecodeArgs a) {
    static_assert(F::C == 16, "pieces of 16 columns");
    constexpr int COLS = 16 * LR, RS = NT / LR, WARPS = NT / 32, KEEP = 16 * LR / 32;
    static_assert(COLS <= NT, "a thread for every column");
    extern __shared__ __align__(16) Entry entries[];  // [kRing][W + R]
    __shared__ __align__(16) float part_k[WARPS][COLS];
    __shared__ __align__(16) float part_q[WARPS][COLS];
    __shared__ __align__(16) float delta[COLS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rs = tid / LR, lp = tid % LR;
    const int64_t s = blockIdx.x / a.slices;
    const int slice = (int)(blockIdx.x % a.slices);
    const int p = slice * LR + lp, c0 = slice * COLS, hd = a.hd, W = a.W, R = a.R;
    const bool active = p < a.pieces;
    const int gl = min(a.group / 16, LR);  // lanes of a scale group
    uint4* codes = reinterpret_cast<uint4*>(a.codes) + p;
    float* scales = a.scales + p * 16 / a.group;
    const bool column = tid < COLS && c0 + tid < hd;  // this thread has a value column
    grid_dependency_wait();
    grid_launch_dependents();

    // this thread's entries of a token as they are loaded, and as they are kept
    // (an index waits as it was loaded: widening it would wait for it)
    uint32_t raw_lo[ITEMS], raw_hi[ITEMS];
    float raw_weight[ITEMS], raw_gate[ITEMS], v_next = 0.0f, beta_next = 0.0f;
    const auto load_entries = [&](int t) {
        if (t >= a.T) return;
        const int64_t ts = t * a.tstride + s * a.sstride;
#pragma unroll
        for (int n = 0; n < ITEMS; ++n) {
            const int i = tid + n * NT;
            if (i < W + R) {
                const bool write = i < W;
                const int64_t e = write ? ts * W + i : ts * R + (i - W);
                const void* idx = write ? a.k_idx : a.q_idx;
                const uint32_t* word = static_cast<const uint32_t*>(idx) + (a.idx64 ? 2 * e : e);
                raw_lo[n] = __ldg(word);
                if (a.idx64) raw_hi[n] = __ldg(word + 1);
                raw_weight[n] = __ldg((write ? a.k_val : a.q_val) + e);
                raw_gate[n] = write ? __ldg(a.g + ts * a.G + (a.G == 1 ? 0 : i)) : 0.0f;
            }
        }
    };
    const auto load_value = [&](int t) {
        if (t >= a.T) return;
        const int64_t ts = t * a.tstride + s * a.sstride;
        beta_next = __ldg(a.beta + ts);
        if (column) v_next = __ldg(a.v + ts * hd + c0 + tid);
    };
    const auto keep_entries = [&](int t) {
        if (t >= a.T) return;
        Entry* to = entries + (t % kRing) * (W + R);
#pragma unroll
        for (int n = 0; n < ITEMS; ++n) {
            const int i = tid + n * NT;
            if (i < W + R) {
                const int64_t x = a.idx64 ? (int64_t)((uint64_t)raw_hi[n] << 32 | raw_lo[n]) : (int64_t)(int32_t)raw_lo[n];
                const bool in = x >= 0 && x < a.n_slots;
                if (in) {
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(a.codes + (x * a.pieces + slice * LR) * 16));
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(a.scales + x * a.groups + c0 / a.group));
                } else {
                    atomicOr(&g_qdecode_status, SDM_DEV_BAD_INDEX);
                }
                to[i] = Entry{in ? (int)x : -1, raw_weight[n], expf(raw_gate[n]), 0.0f};
            }
        }
    };
    int slot[RPT];
    uint4 code[RPT];
    float ds[RPT], kv[RPT];  // scale * decay, and the weight, of the write rows
    // request the write rows of token t; ds holds the decay until scale_writes()
    float row_scale[RPT];
    const auto load_writes = [&](int t) {
        const Entry* from = entries + (t % kRing) * (W + R);
#pragma unroll
        for (int j = 0; j < RPT; ++j) {
            const int w = rs + j * RS;
            const Entry e = from[min(w, W - 1)];
            slot[j] = w < W && active ? e.slot : -1;
            kv[j] = w < W ? e.weight : 0.0f;
            ds[j] = e.decay;
        }
#pragma unroll
        for (int j = 0; j < RPT; ++j) {
            code[j] = load16_if(codes + (int64_t)slot[j] * a.pieces, slot[j] >= 0);
            row_scale[j] = load4_if(scales + (int64_t)slot[j] * a.groups, slot[j] >= 0);
        }
    };

    load_entries(0);
    load_value(0);
    keep_entries(0);
    load_entries(1);
    keep_entries(1);
    load_entries(2);
    __syncthreads();
    load_writes(0);

    for (int t = 0; t < a.T; ++t) {
        // the decayed sum of the write rows
        f32x2 x[8], acc2[8];
        float acc[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) acc2[i] = 0;
#pragma unroll
        for (int j = 0; j < RPT; ++j) {
            ds[j] *= row_scale[j];
            F::unpack2(code[j], x);
            const f32x2 f = pair(kv[j] * ds[j], kv[j] * ds[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc2[i] = fma2(f, x[i], acc2[i]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) split(acc2[i], acc[2 * i], acc[2 * i + 1]);
        int first = reduce_rows<LR>(acc, lane);
#pragma unroll
        for (int i = 0; i < KEEP; ++i) part_k[warp][lp * 16 + first + i] = acc[i];
        __syncthreads();  // 1: the sums of this token's writes and of the last one's reads
        const auto put_out = [&](int of) {
            float r = part_q[0][tid];
#pragma unroll
            for (int q = 1; q < WARPS; ++q) r += part_q[q][tid];
            const int64_t o = (of * a.tstride + s * a.sstride) * hd + c0 + tid;
            if (a.out_bf16)
                static_cast<uint16_t*>(a.out)[o] = from_f32<uint16_t>(r);
            else
                static_cast<float*>(a.out)[o] = r;
        };
        if (tid < COLS) {
            float r = part_k[0][tid];
#pragma unroll
            for (int q = 1; q < WARPS; ++q) r += part_k[q][tid];
            delta[tid] = column ? beta_next * (v_next - r) : 0.0f;
        }
        __syncthreads();  // 2: delta
        if (column && t > 0) put_out(t - 1);
        load_value(t + 1);
        keep_entries(t + 2);
        load_entries(t + 3);
        // the new rows
        f32x2 dl[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 f = *reinterpret_cast<const float4*>(&delta[lp * 16 + 4 * i]);
            dl[2 * i] = pair(f.x, f.y);
            dl[2 * i + 1] = pair(f.z, f.w);
        }
        // first every row's scale, then every row's codes from the columns computed again: the rows'
        // chains of shuffles and divisions overlap, where all the columns would not fit the registers
        const auto new_row = [&](int j, f32x2* y) {
            F::unpack2(code[j], y);
            const f32x2 k2 = pair(kv[j], kv[j]), d2 = pair(ds[j], ds[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = fma2(k2, dl[i], mul2(d2, y[i]));
        };
        float top[RPT], new_scale[RPT], inv[RPT];
#pragma unroll
        for (int j = 0; j < RPT; ++j) {
            new_row(j, x);
            top[j] = piece_top<16>(x);
        }
        group_scales<F, RPT>(top, gl, new_scale, inv);
#pragma unroll
        for (int j = 0; j < RPT; ++j) {
            new_row(j, x);
            store16_if(codes + (int64_t)slot[j] * a.pieces, pack_piece<F>(x, inv[j]), slot[j] >= 0);
            store4_if(scales + (int64_t)slot[j] * a.groups, new_scale[j], slot[j] >= 0 && lp % gl == 0);
        }
        __syncthreads();  // 3: the rows are written, and may be read by this token and the next
        uint4 v[RPT];
        float qs[RPT], q_scale[RPT];
        const Entry* reads = entries + (t % kRing) * (W + R) + W;
        const auto load_reads = [&](int r0) {
            int sl[RPT];
#pragma unroll
            for (int j = 0; j < RPT; ++j) {
                const int r = r0 + j * RS;
                const Entry e = reads[min(r, R - 1)];
                sl[j] = r < R && active ? e.slot : -1;
                qs[j] = e.weight;
            }
#pragma unroll
            for (int j = 0; j < RPT; ++j) {
                v[j] = load16_if(codes + (int64_t)sl[j] * a.pieces, sl[j] >= 0);
                q_scale[j] = load4_if(scales + (int64_t)sl[j] * a.groups, sl[j] >= 0);
            }
        };
        load_reads(rs);
        if (t + 1 < a.T) load_writes(t + 1);
        // the readings
#pragma unroll
        for (int i = 0; i < 8; ++i) acc2[i] = 0;
        for (int r0 = 0;;) {  // alike for all threads: rows behind the end are zeros
#pragma unroll
            for (int j = 0; j < RPT; ++j) {
                F::unpack2(v[j], x);
                const float q = qs[j] * q_scale[j];
                const f32x2 f = pair(q, q);
#pragma unroll
                for (int i = 0; i < 8; ++i) acc2[i] = fma2(f, x[i], acc2[i]);
            }
            r0 += RPT * RS;
            if (r0 >= R) break;
            load_reads(r0 + rs);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) split(acc2[i], acc[2 * i], acc[2 * i + 1]);
        first = reduce_rows<LR>(acc, lane);
#pragma unroll
        for (int i = 0; i < KEEP; ++i) part_q[warp][lp * 16 + first + i] = acc[i];
        if (t + 1 == a.T) {
            __syncthreads();
            if (column) put_out(t);
        }
    }
}

struct Chosen {
    const void* fn;
    int threads;
};

template <typename F, int LR, int NT, int RPT>
Chosen with_items(int entries) {
    if constexpr (NT < 512) {  // of the 512 entries at most
        if (entries > NT) return {(const void*)qdecode_kernel<F, LR, NT, RPT, 512 / NT>, NT};
    }
    return {(const void*)qdecode_kernel<F, LR, NT, RPT, 1>, NT};
}

// Blocks that fit the GPU at once as two of 256 threads on each of 152 SMs. A constant, since the threads
// settle the order of the sums, and results do not depend on the GPU that is there.
constexpr int64_t kFewBlocks = 304;

// Threads and rows of each. Few blocks get 256 threads, since a token's chain of steps is then all the
// time there is, and more blocks 128, whose warps spend fewer instructions on a token. us a token, 128
// / 256 threads: 64 streams of 64 rows 3.00 / 2.51, 304 streams 3.37 / 3.08, 512 streams 4.59 / 5.91;
// of 32 rows 2.19 / 1.81, 2.36 / 2.23, 2.99 / 4.12. Eight rows a thread lose even to that: 128 rows a
// stream 5.28 / 3.80 for 64 streams and 10.9 / 9.5 for 512; 256 rows on 256 / 512 threads 6.12 / 5.78 and 22.0 / 20.4.
template <typename F, int LR>
Chosen choose(int W, int R, bool few) {
    constexpr int S = 128 / LR;  // row slots of 128 threads
    if (W <= 2 * S) return few ? with_items<F, LR, 256, 1>(W + R) : with_items<F, LR, 128, 2>(W + R);
    if (W <= 4 * S) return few ? with_items<F, LR, 256, 2>(W + R) : with_items<F, LR, 128, 4>(W + R);
    if constexpr (LR == 8) {  // the 256 rows of a token at most fit 256 threads of 4 lanes a row
        if (W > 8 * S) return with_items<F, LR, 512, 4>(W + R);
    }
    return with_items<F, LR, 256, 4>(W + R);
}

}  // namespace

int launch_qdecode(const QDecodeArgs& a0, int format, cudaStream_t stream) {
    QDecodeArgs a = a0;
    a.pieces = (a.hd + 15) / 16;
    a.groups = (a.hd + a.group - 1) / a.group;
    const bool narrow = a.pieces <= 4;
    a.slices = narrow ? 1 : (a.pieces + 7) / 8;
    const int64_t blocks = a.n_streams * a.slices;
    if (blocks > INT_MAX) return SDM_ECOUNT;
    const bool few = blocks <= kFewBlocks;
    const Chosen c = format == SDM_INT8 ? (narrow ? choose<Int8, 4>(a.W, a.R, few) : choose<Int8, 8>(a.W, a.R, few))
                                        : (narrow ? choose<Fp8, 4>(a.W, a.R, few) : choose<Fp8, 8>(a.W, a.R, few));
    const size_t smem = (size_t)kRing * (a.W + a.R) * sizeof(Entry);
    void* args[] = {&a};
    return launch_pdl_raw(c.fn, dim3((unsigned)blocks), dim3((unsigned)c.threads), smem, stream, args);
}

cudaError_t qdecode_status(void** word) { return cudaGetSymbolAddress(word, g_qdecode_status); }

}  // namespace sdm
