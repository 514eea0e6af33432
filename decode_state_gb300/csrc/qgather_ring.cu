// Gather over a quantised bank, and the gradient of a gather's weights, for many tokens.
//
// Math (include/sdm.h): out[t] = sum_n w[t, n] * row(idx[t, n]) and
// dw[t, n] = <dout[t], row(idx[t, n])>, row = scale * code (or the row of a bf16 / float32 bank).
//
// Design. Rows of 128 bytes at random places are what bounds both: at 7 TB/s every SM has to have
// some 50 KB of them on their way all the time. One block an SM; its persistent warps walk over the live
// tokens in steps of up to 32 entries. While a step is summed from shared memory, the rows of the next are
// on their way by cp.async, and the indices of the one behind it by plain loads. LR lanes copy
// one row (or a slice of it), 16 bytes each. A block finds the live tokens by the prefix sums of
// chunk_valid, so that every warp gets as many of them: by token number, warps whose tokens mostly lay at
// the end of their chunks were done long before the others.
//
// The sums are matrix products of codes, which are exact as f16, with the float32 factors as three f16
// limbs: columns x entries times entries x limbs for the gather, entries x columns times columns x limbs
// for the gradient; the accumulators are float32. A product of a row with a vector leaves most of the
// tensor core idle, and still it is what makes the kernel keep up with memory: unpacking to float32 and
// multiplying there took 773 instructions a step, half of them on pipes of half rate (HADD2, FFMA2).
// The products are mma.sync: their accumulators stay in registers across steps, 16 columns or entries
// high, where a tcgen05 product is 128 rows high and would need 8 tokens' rows in one tile.
// float32 rows are multiplied in float32.
//
// What bounds it: 65536 tokens, 64 and 64 fp8 rows of 128 bytes with a scale each, half of the tokens padding, take
// 130 us (5.1 TB/s; the gradient of 64 int8 rows 73). Loads of the same rows and scales alone take 107,
// since a scale's 4 bytes cost a sector of 32. The rest is latency: 640 instructions a step on 4 warps a scheduler at
// 0.64 a cycle; 50 instructions fewer (sums in a running exponent), more warps or more steps ahead gained nothing.
#include <cuda_fp16.h>

#include <algorithm>
#include <climits>
#include <type_traits>

#include "qgather_device.cuh"

namespace sdm {
namespace {

__device__ unsigned int g_ring_status;

constexpr unsigned kAll = 0xffffffffu;

// Warps of a block at most, and the steps whose rows are on their way while one is summed. More of
// either is slower: the stages take shared memory from L1, whose lines the requests on their way need.
// 65536 tokens, half of them padding, a gather of 64 and 64 rows of 128 bytes / the gradient of 64 rows, single calls: 16
// warps 1 ahead 138 / 82 us, 2 ahead 173 / 101; 12 warps 1 ahead 146 / 93, 2 ahead 150 / 95; 20 warps 1 ahead 143 / 100.
constexpr int kRingWarps = 16;
constexpr int kAhead = 1;

__device__ __forceinline__ void copy16_if(void* dst, const void* src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy8_if(void* dst, const void* src, bool on) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(on ? 8 : 0) : "memory");
}
__device__ __forceinline__ void copy4_if(void* dst, const void* src, bool on) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_u32(dst)), "l"(src), "r"(on ? 4 : 0) : "memory");
}

// Rows in shared memory: piece lp of row r lies at piece lp ^ turn(r) of the row, so that the same piece of
// eight neighbouring rows, which a matrix load asks for, is spread over all banks.
template <int LR>
__device__ __forceinline__ int turn(int r) {
    return LR == 4 ? (r >> 1) & 3 : r & 7;
}

// One step's share of shared memory: the rows' slices by 16-byte pieces, for the gradient the slice of
// dout, and the entries' scales, unless (ONE) a row's slice has a single one.
template <typename F, int LR, bool GRAD, bool ONE>
struct RingStage {
    static constexpr int ENTRIES = LR <= 8 ? 32 : 256 / LR;  // of a step, so that its rows are 4 KB
    static constexpr int STEPS = ENTRIES * LR / 32;          // rows of a row slot
    static constexpr int COLS = LR * F::C;
    static constexpr int GROUPS = !F::kQuantised || ONE ? 0 : (COLS + 31) / 32;  // scales of a row's slice at most
    uint4 rows[ENTRIES * LR];
    float dout[GRAD ? COLS : 4];
    __align__(16) float scale[GROUPS > 0 ? ENTRIES * GROUPS : 4];
};

// What a warp keeps beside its stages: three 16-bit limbs of each weight, or of each column of dout.
template <typename F, int LR, bool GRAD>
struct RingScratch {
    __align__(16) uint16_t limb[3][GRAD ? LR * F::C : 32];
};

// ---------------------------------------------------------------- float32 factors as 16-bit limbs
// Codes are exact as 16-bit floats, and so are their products with 16-bit factors in a float32
// accumulator; a float32 factor is the sum of three limbs of 11 bits (or 8, as bfloat16), which are
// three columns of the tensor core's second operand.

constexpr float kLimb = 0x1p-11f;  // weight of the next f16 limb

// The power of two that brings magnitudes of at most `most` below 4, and (undo) back; any magnitudes
// where `most` is not finite.
__device__ __forceinline__ float limb_scale(float most, float* undo) {
    const uint32_t e = min(max(__float_as_uint(most) >> 23, 27u), 253u);
    *undo = __uint_as_float(e << 23);
    return __uint_as_float((254u - e) << 23);
}

// x as three f16 limbs, |x| < 4; an infinity or NaN is in the first alone
__device__ __forceinline__ void limbs_f16(float x, uint16_t* l) {
    const __half a = __float2half_rn(x);
    float rest = (x - __half2float(a)) * 2048.0f;
    const __half b = __float2half_rn(rest);
    float last = (rest - __half2float(b)) * 2048.0f;
    const bool finite = fabsf(x) <= 3.402823466e38f;
    l[0] = __half_as_ushort(a);
    l[1] = finite ? __half_as_ushort(b) : (uint16_t)0;
    l[2] = finite ? __half_as_ushort(__float2half_rn(last)) : (uint16_t)0;
}

// x as three bf16 limbs, each of its own exponent
__device__ __forceinline__ void limbs_bf16(float x, uint16_t* l) {
    const uint16_t a = from_f32<uint16_t>(x);
    const float rest = x - to_f32(a);
    const uint16_t b = from_f32<uint16_t>(rest);
    const bool finite = fabsf(x) <= 3.38e38f;
    l[0] = a;
    l[1] = finite ? b : (uint16_t)0;
    l[2] = finite ? from_f32<uint16_t>(rest - to_f32(b)) : (uint16_t)0;
}

// Four 8 x 8 matrices of 16-bit elements; every eight lanes give the rows of one. Transposed, lane
// 4 q + i has rows 2 i and 2 i + 1 of column q; as they are, columns 2 i and 2 i + 1 of row q.
template <bool TRANS, int N>
__device__ __forceinline__ void load_matrices(uint32_t address, uint32_t* m) {
    if constexpr (N == 4 && TRANS)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(m[0]), "=r"(m[1]), "=r"(m[2]), "=r"(m[3])
                     : "r"(address)
                     : "memory");
    else if constexpr (N == 4)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(m[0]), "=r"(m[1]), "=r"(m[2]), "=r"(m[3])
                     : "r"(address)
                     : "memory");
    else if constexpr (TRANS)
        asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0, %1}, [%2];" : "=r"(m[0]), "=r"(m[1]) : "r"(address) : "memory");
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0, %1}, [%2];" : "=r"(m[0]), "=r"(m[1]) : "r"(address) : "memory");
}

template <bool BF16>
__device__ __forceinline__ void mma(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
    if constexpr (BF16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Bytes (LO, HI) of r as two f16.
template <int LO, int HI>
__device__ __forceinline__ uint32_t bytes_f16(Int8, uint32_t r) {
    const uint32_t h = __byte_perm(r ^ 0x80808080u, 0x64646464u, LO | 0x40 | HI << 8 | 0x4000);  // 1024 + 128 + code
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&h), __floats2half2_rn(1152.0f, 1152.0f));
    return *reinterpret_cast<const uint32_t*>(&x);
}
template <int LO, int HI>
__device__ __forceinline__ uint32_t bytes_f16(Fp8, uint32_t r) {
    const uint32_t two = LO == 0 && HI == 1 ? r : __byte_perm(r, 0u, LO | HI << 4);
    uint32_t h;
    asm("{ .reg .b16 lo, hi; mov.b32 {lo, hi}, %1; cvt.rn.f16x2.e4m3x2 %0, lo; }" : "=r"(h) : "r"(two));
    return h;
}
// The low (SHIFT 0) or high (4) halves of bytes (LO, HI) of r as two f16.
template <int LO, int HI, int SHIFT>
__device__ __forceinline__ uint32_t nibbles_f16(uint32_t r) {
    const uint32_t n = (r >> SHIFT & 0x0f0f0f0fu) ^ 0x08080808u;
    const uint32_t h = __byte_perm(n, 0x64646464u, LO | 0x40 | HI << 8 | 0x4000);  // 1024 + 8 + code
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&h), __floats2half2_rn(1032.0f, 1032.0f));
    return *reinterpret_cast<const uint32_t*>(&x);
}

// Where a step is: token, column slice, operand, its first entry; token -1: none.
struct Step {
    int t, slice, op, base;
};

// F: format. LR: lanes of a row. GRAD: the weights' gradient.
template <typename F, int LR, bool GRAD, bool ONE>
__global__ void __launch_bounds__(kRingWarps * 32, 1) gather_ring(const QGatherArgs a) {
    using S = RingStage<F, LR, GRAD, ONE>;
    using Scratch = RingScratch<F, LR, GRAD>;
    constexpr int C = F::C, SLOTS = 32 / LR, STEPS = S::STEPS, ENTRIES = S::ENTRIES, COLS = S::COLS;
    constexpr bool IS_BF16 = std::is_same<F, Bf16>::value, IS_F32 = std::is_same<F, F32>::value, IS_INT4 = std::is_same<F, Int4>::value;
    extern __shared__ __align__(16) unsigned char ring[];
    __shared__ int warp_sums[kRingWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    const int rs = lane / LR, lp = lane % LR, hd = a.hd;
    const int tokens = (int)a.tokens, chunks = tokens / a.chunk;
    int* prefix = reinterpret_cast<int*>(ring);  // [chunks + 1] live tokens ahead of a chunk, with chunk_valid
    unsigned char* mine = ring + (a.chunk_valid ? ((size_t)chunks + 4) / 4 * 16 : 0) + warp * ((kAhead + 1) * sizeof(S) + sizeof(Scratch));
    S* stages = reinterpret_cast<S*>(mine);
    Scratch& scratch = *reinterpret_cast<Scratch*>(stages + kAhead + 1);
    const int slices = (a.pieces + LR - 1) / LR;
    const int unit_slices = GRAD ? 1 : slices;  // the gradient's steps walk over the slices themselves
    grid_dependency_wait();
    grid_launch_dependents();

    int live = chunks * a.valid;  // live tokens
    if (a.chunk_valid != nullptr) {
        const int per = (chunks + blockDim.x - 1) / blockDim.x, c0 = min(chunks, tid * per), c1 = min(chunks, c0 + per);
        int own = 0;
        for (int c = c0; c < c1; ++c) own += min(max(__ldg(a.chunk_valid + c), 0), a.chunk);
        int sum = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(kAll, sum, o);
            if (lane >= o) sum += y;
        }
        if (lane == 31) warp_sums[warp] = sum;
        __syncthreads();
        sum -= own;
        live = 0;
        for (int w = 0; w < warps; ++w) {
            if (w < warp) sum += warp_sums[w];
            live += warp_sums[w];
        }
        for (int c = c0; c < c1; ++c) {
            prefix[c] = sum;
            sum += min(max(__ldg(a.chunk_valid + c), 0), a.chunk);
        }
        if (tid == 0) prefix[chunks] = live;
        __syncthreads();
    }
    // the k-th live token
    const auto live_token = [&](int k) {
        if (a.chunk_valid == nullptr) return a.valid == a.chunk ? k : k / a.valid * a.chunk + k % a.valid;
        int lo = 0, hi = chunks - 1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (prefix[mid] <= k)
                lo = mid;
            else
                hi = mid - 1;
        }
        return lo * a.chunk + k - prefix[lo];
    };

    const int me = blockIdx.x * warps + warp, stride = gridDim.x * warps;
    const int64_t units = (int64_t)live * unit_slices;
    int64_t next = me;  // the unit behind the 32 that the lanes hold
    int held_t = 0, held_slice = 0, held = 0, taken = 0;
    Step at{-1, 0, 0, 0};
    // the next step of this warp's walk
    const auto advance = [&]() {
        if (at.t >= 0) {
            if (GRAD && ++at.slice < slices) return;
            if (GRAD) at.slice = 0;
            at.base += ENTRIES;
            if (at.base < a.width[at.op]) return;
            at.base = 0;
            if (++at.op < a.n_ops) return;
        }
        at.op = at.base = 0;
        if (taken == held) {
            const int64_t u = next + (int64_t)lane * stride;
            held = __popc(__ballot_sync(kAll, u < units));
            taken = 0;
            next += 32 * (int64_t)stride;
            if (u < units) {
                const int k = (int)(unit_slices > 1 ? u / unit_slices : u);
                held_slice = unit_slices > 1 ? (int)(u - (int64_t)k * unit_slices) : 0;
                held_t = live_token(k);
            }
        }
        if (taken < held) {
            at.t = __shfl_sync(kAll, held_t, taken);
            at.slice = __shfl_sync(kAll, held_slice, taken);
            ++taken;
        } else {
            at.t = -1;
            held = taken = 0;
            next = units;
        }
    };
    // a step's indices and weights as they are in memory, an entry for each lane
    uint32_t raw_lo = 0, raw_hi = 0, raw_w = 0;
    const auto load_entries = [&]() {
        const int e = at.base + lane;
        if (at.t < 0 || lane >= ENTRIES || e >= a.width[at.op]) return;
        const int64_t i = (int64_t)at.t * a.width[at.op] + e;
        const uint32_t* word = static_cast<const uint32_t*>(a.idx[at.op]) + (a.idx64 ? 2 * i : i);
        raw_lo = __ldg(word);
        if (a.idx64) raw_hi = __ldg(word + 1);
        if (!GRAD) raw_w = a.w_bf16 ? __ldg(static_cast<const uint16_t*>(a.w[at.op]) + i) : __ldg(static_cast<const uint32_t*>(a.w[at.op]) + i);
    };
    // request the step's rows (one commit for every step, requested or not); gives the lane's weight (of the
    // gradient: whether the lane's entry is skipped) and, where a row's slice has one, its scale
    const auto request = [&](S& st, float& weight, float& scale) {
        weight = scale = 0.0f;
        if (at.t >= 0) {
            const int n = a.width[at.op] - at.base;
            int slot = -1;
            if (lane < min(n, ENTRIES)) {
                const int64_t x = a.idx64 ? (int64_t)((uint64_t)raw_hi << 32 | raw_lo) : (int64_t)(int32_t)raw_lo;
                if (x >= 0 && x < a.n_slots)
                    slot = (int)x;
                else
                    atomicOr(&g_ring_status, SDM_DEV_BAD_INDEX);
                if (GRAD)
                    weight = slot < 0 ? 1.0f : 0.0f;
                else if (slot >= 0)  // a skipped entry's may be anything
                    weight = a.w_bf16 ? __uint_as_float(raw_w << 16) : __uint_as_float(raw_w);
            }
            const int p = at.slice * LR + lp, g0 = ONE ? 0 : at.slice * LR * C / a.group;
            const unsigned char* bank = static_cast<const unsigned char*>(a.bank) + p * 16;
            const bool active = p < a.pieces;
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                const int sl = __shfl_sync(kAll, slot, s * SLOTS + rs);
                const int e = s * SLOTS + rs;
                copy16_if(&st.rows[e * LR + (lp ^ turn<LR>(e))], bank + sl * a.row_bytes, sl >= 0 && active);
            }
            if constexpr (F::kQuantised) {
                const float* scales = a.scales + (int64_t)slot * a.groups + g0;
                if (ONE) {
                    // to a register, past L1: copies of 32 scattered words would each take a line of the little L1
                    // that the stages leave
                    scale = load4_if(scales, slot >= 0);
                } else if (lane < ENTRIES) {
                    const int ng = min(a.groups - g0, (LR * C + a.group - 1) / a.group);
                    float* to = &st.scale[lane * S::GROUPS];
                    if (a.scale_words == 4) {
                        for (int g = 0; g < ng; g += 4) copy16_if(to + g, scales + g, slot >= 0);
                    } else if (a.scale_words == 2) {
                        for (int g = 0; g < ng; g += 2) copy8_if(to + g, scales + g, slot >= 0);
                    } else {
                        for (int g = 0; g < ng; ++g) copy4_if(to + g, scales + g, slot >= 0);
                    }
                }
            }
            if (GRAD) {
                const float* d = a.dout[at.op] + (int64_t)at.t * hd + at.slice * LR * C;
                const int left = hd - at.slice * LR * C;
                if (a.vec_out) {
                    for (int c = lane; c < LR * C / 4; c += 32) copy16_if(&st.dout[4 * c], d + 4 * c, 4 * c < left);
                } else {
                    for (int c = lane; c < LR * C; c += 32) copy4_if(&st.dout[c], d + c, c < left);
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };

    Step steps[kAhead + 1];  // the steps of the ring, the oldest first, and their weights
    float weights[kAhead + 1], one_scale[kAhead + 1];
    int head = 0;  // the stage of the oldest
    advance();
    load_entries();
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
        steps[i] = at;
        request(stages[i], weights[i], one_scale[i]);
        if (at.t >= 0) advance();
        load_entries();
    }
    // padding tokens get zeros, one for every step, while rows are on their way
    int64_t pad_at = live < tokens ? (int64_t)me * 32 : tokens;  // the 32 tokens that are looked at next
    uint32_t pads = 0;                                           // padding among the 32 before
    const auto zero_one = [&]() {
        if (pads == 0) {
            if (pad_at >= tokens) return;
            pads = __ballot_sync(kAll, pad_at + lane < tokens && padding(a, pad_at + lane));
            pad_at += (int64_t)stride * 32;
            if (pads == 0) return;
        }
        const int64_t t = pad_at - (int64_t)stride * 32 + __ffs(pads) - 1;
        pads &= pads - 1;
        for (int op = 0; op < a.n_ops; ++op) {
            if (GRAD) {
                for (int i = lane; i < a.width[op]; i += 32) store_dw(a, op, t * a.width[op] + i, 0.0f);
            } else if (a.vec_out) {
                for (int c = 4 * lane; c < hd; c += 128) *reinterpret_cast<float4*>(a.out[op] + t * hd + c) = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            } else {
                for (int c = lane; c < hd; c += 32) a.out[op][t * hd + c] = 0.0f;
            }
        }
    };
    const int q = lane >> 2, i4 = lane & 3;  // the lane's row (or column) and place in it of a matrix
    constexpr int MATS = ENTRIES / 8;         // matrices of a step's rows
    constexpr int TILES = IS_INT4 ? 2 * LR : LR;  // 16 columns of the sums each
    float acc[GRAD ? 1 : TILES][4];           // limb sums of the tile's columns
    float dots[MATS > 1 ? MATS / 2 : 1][4];   // limb sums of 16 entries each
    float dot[IS_F32 ? STEPS : 1];
    while (steps[0].t >= 0) {
        steps[kAhead] = at;
        request(stages[head == 0 ? kAhead : head - 1], weights[kAhead], one_scale[kAhead]);
        if (at.t >= 0) advance();
        load_entries();
        zero_one();
        asm volatile("cp.async.wait_group %0;" ::"n"(kAhead) : "memory");
        __syncwarp();
        const S& st = stages[head];
        const Step now = steps[0];
        const int width = a.width[now.op], n = width - now.base;  // entries from here on
        const int g0 = ONE || !F::kQuantised ? 0 : now.slice * COLS / a.group;
        if constexpr (IS_F32) {
            if (now.slice == 0) {
#pragma unroll
                for (int s = 0; s < STEPS; ++s) dot[s] = 0.0f;
            }
            const float4 d = *reinterpret_cast<const float4*>(&st.dout[lp * C]);
            const float dl[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                const int e = s * SLOTS + rs;
                dot[s] += dot_piece<F>(dl, st.rows[e * LR + (lp ^ turn<LR>(e))]);
            }
            if (now.slice + 1 == slices) {
                // the sums over the lanes of a row: halves of the steps are handed over while there are any
                int left = STEPS;
#pragma unroll
                for (int h = LR / 2; h >= 1; h /= 2) {
                    const bool up = lane & h;
                    if (left > 1) {
                        left /= 2;
#pragma unroll
                        for (int i = 0; i < STEPS / 2; ++i) {
                            if (i < left) {
                                const float keep = up ? dot[i + left] : dot[i], give = up ? dot[i] : dot[i + left];
                                dot[i] = keep + __shfl_xor_sync(kAll, give, h);
                            }
                        }
                    } else {
                        dot[0] += __shfl_xor_sync(kAll, dot[0], h);
                    }
                }
                constexpr int PER = LR / STEPS;  // lanes that hold the same step's sum
                const int e = lp / PER * SLOTS + rs;
                if (lp % PER == 0 && e < n) store_dw(a, now.op, (int64_t)now.t * width + now.base + e, dot[0]);
            }
        } else if constexpr (GRAD) {
            // dout's slice as limbs, by column
            float undo = 1.0f;
            {
                float d[COLS / 32], most = 0.0f, f = 1.0f;
#pragma unroll
                for (int c = 0; c < COLS / 32; ++c) {
                    d[c] = st.dout[lane * (COLS / 32) + c];
                    most = fmaxf(most, fabsf(d[c]));
                }
                if (!IS_BF16) f = limb_scale(__uint_as_float(__reduce_max_sync(kAll, __float_as_uint(most))), &undo);
#pragma unroll
                for (int c = 0; c < COLS / 32; ++c) {
                    uint16_t l[3];
                    if (IS_BF16)
                        limbs_bf16(d[c], l);
                    else
                        limbs_f16(d[c] * f, l);
#pragma unroll
                    for (int k = 0; k < 3; ++k) scratch.limb[k][lane * (COLS / 32) + c] = l[k];
                }
            }
            __syncwarp();
            if (now.slice == 0) {
#pragma unroll
                for (int m = 0; m < MATS / 2; ++m) dots[m][0] = dots[m][1] = dots[m][2] = dots[m][3] = 0.0f;
            }
            const int row = lane % (8 * MATS);  // the row whose address this lane gives
            const uint32_t rows = smem_u32(st.rows) + row * LR * 16, row_turn = turn<LR>(row);
            float part[MATS / 2][4];
            uint32_t held_v[MATS], held_b = 0;
#pragma unroll
            for (int p = 0; p < LR; ++p) {
                if (p == 0 || (F::kQuantised && !ONE && p * C % a.group == 0)) {
#pragma unroll
                    for (int m = 0; m < MATS / 2; ++m) part[m][0] = part[m][1] = part[m][2] = part[m][3] = 0.0f;
                }
                uint32_t v[MATS];
                load_matrices<false, MATS>(rows + ((p ^ row_turn) << 4), v);
                if constexpr (IS_BF16) {
                    uint32_t b = 0;
                    if (q < 3) b = *reinterpret_cast<const uint32_t*>(&scratch.limb[q][p * 8 + 2 * i4]);
                    if (p % 2 == 0) {  // 8 columns a piece: two pieces fill a product
                        held_b = b;
#pragma unroll
                        for (int m = 0; m < MATS; ++m) held_v[m] = v[m];
                    } else {
#pragma unroll
                        for (int m = 0; m < MATS / 2; ++m) {
                            const uint32_t frag[4] = {held_v[2 * m], held_v[2 * m + 1], v[2 * m], v[2 * m + 1]};
                            mma<true>(part[m], frag, held_b, b);
                        }
                    }
                } else if constexpr (IS_INT4) {
                    uint4 w = make_uint4(0u, 0u, 0u, 0u);  // columns 8 i4 .. + 7 of the piece
                    if (q < 3) w = *reinterpret_cast<const uint4*>(&scratch.limb[q][p * 32 + 8 * i4]);
                    const uint32_t even0 = __byte_perm(w.x, w.y, 0x5410), even1 = __byte_perm(w.z, w.w, 0x5410),
                                   odd0 = __byte_perm(w.x, w.y, 0x7632), odd1 = __byte_perm(w.z, w.w, 0x7632);
#pragma unroll
                    for (int m = 0; m < MATS / 2; ++m) {
                        const uint32_t lo[4] = {nibbles_f16<0, 1, 0>(v[2 * m]), nibbles_f16<0, 1, 0>(v[2 * m + 1]),
                                                nibbles_f16<2, 3, 0>(v[2 * m]), nibbles_f16<2, 3, 0>(v[2 * m + 1])};
                        mma<false>(part[m], lo, even0, even1);
                        const uint32_t hi[4] = {nibbles_f16<0, 1, 4>(v[2 * m]), nibbles_f16<0, 1, 4>(v[2 * m + 1]),
                                                nibbles_f16<2, 3, 4>(v[2 * m]), nibbles_f16<2, 3, 4>(v[2 * m + 1])};
                        mma<false>(part[m], hi, odd0, odd1);
                    }
                } else {
                    uint2 w = make_uint2(0u, 0u);  // columns 4 i4 .. + 3 of the piece
                    if (q < 3) w = *reinterpret_cast<const uint2*>(&scratch.limb[q][p * 16 + 4 * i4]);
#pragma unroll
                    for (int m = 0; m < MATS / 2; ++m) {
                        const uint32_t frag[4] = {bytes_f16<0, 1>(F{}, v[2 * m]), bytes_f16<0, 1>(F{}, v[2 * m + 1]),
                                                  bytes_f16<2, 3>(F{}, v[2 * m]), bytes_f16<2, 3>(F{}, v[2 * m + 1])};
                        mma<false>(part[m], frag, w.x, w.y);
                    }
                }
                // a scale's columns are done: its share of the dots
                if (p + 1 == LR || (F::kQuantised && !ONE && (p + 1) * C % a.group == 0)) {
                    const int g = ONE || !F::kQuantised ? 0 : p * C / a.group;
#pragma unroll
                    for (int m = 0; m < MATS / 2; ++m) {
                        float low = 1.0f, high = 1.0f;
                        if constexpr (F::kQuantised) {
                            if (ONE) {
                                low *= __shfl_sync(kAll, one_scale[0], 16 * m + q);
                                high *= __shfl_sync(kAll, one_scale[0], 16 * m + 8 + q);
                            } else {
                                const bool there = g0 + g < a.groups;  // behind the row's end there are no scales
                                low *= there ? st.scale[(16 * m + q) * S::GROUPS + g] : 0.0f;
                                high *= there ? st.scale[(16 * m + 8 + q) * S::GROUPS + g] : 0.0f;
                            }
                        }
                        dots[m][0] = fmaf(part[m][0] * low, undo, dots[m][0]);
                        dots[m][1] = fmaf(part[m][1] * low, undo, dots[m][1]);
                        dots[m][2] = fmaf(part[m][2] * high, undo, dots[m][2]);
                        dots[m][3] = fmaf(part[m][3] * high, undo, dots[m][3]);
                    }
                }
            }
            if (now.slice + 1 == slices) {
                constexpr float next = IS_BF16 ? 1.0f : kLimb;
#pragma unroll
                for (int m = 0; m < MATS / 2; ++m) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        // lanes 4 q have limbs 0 and 1, lanes 4 q + 1 limb 2
                        const float third = __shfl_down_sync(kAll, dots[m][2 * h], 1);
                        const float sum = fmaf(fmaf(third, next, dots[m][2 * h + 1]), next, dots[m][2 * h]);
                        const int e = 16 * m + 8 * h + q;
                        if (i4 == 0 && e < n) store_dw(a, now.op, (int64_t)now.t * width + now.base + e, sum);
                    }
                }
            }
        } else {
            if (now.base == 0) {
#pragma unroll
                for (int m = 0; m < TILES; ++m) acc[m][0] = acc[m][1] = acc[m][2] = acc[m][3] = 0.0f;
            }
            const int row = lane % (8 * MATS);
            const uint32_t rows = smem_u32(st.rows) + row * LR * 16, row_turn = turn<LR>(row);
            uint32_t b[MATS];
            float undo = 1.0f;
#pragma unroll
            for (int p = 0; p < LR; ++p) {
                if (p == 0 || (!ONE && p * C % a.group == 0)) {
                    // the entries' weights, with the scales of the columns that follow, as limbs
                    const int g = ONE ? 0 : p * C / a.group;
                    const bool there = lane < ENTRIES && (ONE || g0 + g < a.groups);
                    const float w = there ? weights[0] * (ONE ? one_scale[0] : st.scale[lane * S::GROUPS + g]) : 0.0f;
                    const float f = limb_scale(__uint_as_float(__reduce_max_sync(kAll, __float_as_uint(fabsf(w)))), &undo);
                    uint16_t l[3];
                    limbs_f16(w * f, l);
                    __syncwarp();  // the limbs before have been read
#pragma unroll
                    for (int k = 0; k < 3; ++k) scratch.limb[k][lane] = l[k];
                    __syncwarp();
#pragma unroll
                    for (int m = 0; m < MATS; ++m) b[m] = q < 3 ? *reinterpret_cast<const uint32_t*>(&scratch.limb[q][8 * m + 2 * i4]) : 0u;
                }
                uint32_t v[MATS];
                load_matrices<true, MATS>(rows + ((p ^ row_turn) << 4), v);
                // lane 4 q + i has bytes 2 q and 2 q + 1 of entries 2 i and 2 i + 1
                const auto product = [&](int tile, const auto& first, const auto& second) {
                    float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int m = 0; m < MATS; m += 2) {
                        const uint32_t frag[4] = {first(v[m]), second(v[m]), first(v[m + 1]), second(v[m + 1])};
                        mma<false>(c, frag, b[m], b[m + 1]);
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) acc[tile][k] = fmaf(c[k], undo, acc[tile][k]);
                };
                if constexpr (IS_INT4) {
                    product(2 * p, [](uint32_t x) { return nibbles_f16<0, 2, 0>(x); }, [](uint32_t x) { return nibbles_f16<0, 2, 4>(x); });
                    product(2 * p + 1, [](uint32_t x) { return nibbles_f16<1, 3, 0>(x); }, [](uint32_t x) { return nibbles_f16<1, 3, 4>(x); });
                } else {
                    product(p, [](uint32_t x) { return bytes_f16<0, 2>(F{}, x); }, [](uint32_t x) { return bytes_f16<1, 3>(F{}, x); });
                }
            }
            if (n <= ENTRIES) {
                // lanes 4 q have limbs 0 and 1 of a tile's columns, lanes 4 q + 1 limb 2
                float* out = a.out[now.op] + (int64_t)now.t * hd;
#pragma unroll
                for (int m = 0; m < TILES; ++m) {
                    float y[2];
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float third = __shfl_down_sync(kAll, acc[m][2 * h], 1);
                        y[h] = fmaf(fmaf(third, kLimb, acc[m][2 * h + 1]), kLimb, acc[m][2 * h]);
                    }
                    // columns 2 q and 2 q + 1 of a piece; of 4 bits, 4 q and 4 q + 1, and the two behind them
                    const int c = now.slice * COLS + (IS_INT4 ? m / 2 * 32 + 4 * q + m % 2 * 2 : m * 16 + 2 * q);
                    if (i4 == 0) {
                        if (a.vec_out && c + 2 <= hd) {
                            *reinterpret_cast<float2*>(out + c) = make_float2(y[0], y[1]);
                        } else {
                            if (c < hd) out[c] = y[0];
                            if (c + 1 < hd) out[c + 1] = y[1];
                        }
                    }
                }
            }
        }
        __syncwarp();  // the stage may be filled again
        if (GRAD && weights[0] != 0.0f && now.slice + 1 == slices)  // over what is there: 0 whatever dout holds
            store_dw(a, now.op, (int64_t)now.t * width + now.base + lane, 0.0f);
        head = head == kAhead ? 0 : head + 1;
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            steps[i] = steps[i + 1];
            weights[i] = weights[i + 1];
            one_scale[i] = one_scale[i + 1];
        }
    }
    while (pads != 0 || pad_at < tokens) zero_one();
}

struct Kernel {
    const void* fn;
    size_t per_warp;
};

template <typename F, int LR, bool GRAD>
Kernel kernel_lr(bool one) {
    if constexpr (F::kQuantised) {
        if (!one)
            return {(const void*)gather_ring<F, LR, GRAD, false>,
                    sizeof(RingStage<F, LR, GRAD, false>) * (kAhead + 1) + sizeof(RingScratch<F, LR, GRAD>)};
    }
    return {(const void*)gather_ring<F, LR, GRAD, true>, sizeof(RingStage<F, LR, GRAD, true>) * (kAhead + 1) + sizeof(RingScratch<F, LR, GRAD>)};
}

// MOST: lanes of a row at most
template <typename F, bool GRAD, int MOST>
Kernel kernel_of(int lr, bool one) {
    if constexpr (MOST == 32) {
        if (lr == 32) return kernel_lr<F, 32, GRAD>(one);
    }
    if constexpr (MOST >= 16) {
        if (lr == 16) return kernel_lr<F, 16, GRAD>(one);
    }
    return lr == 8 ? kernel_lr<F, 8, GRAD>(one) : kernel_lr<F, 4, GRAD>(one);
}

}  // namespace

int launch_gather_ring(const QGatherArgs& a0, int format, bool grad, cudaStream_t stream) {
    QGatherArgs a = a0;
    // Slices of codes have at most 128 bytes: 65536 tokens, half of them padding, with 64 and 64 rows of 256 bytes take 311
    // us (the gradient of 64 rows 171) in two slices and 392 (227) in one, whose 256 sums fill the registers. bf16 has
    // half the columns in as many bytes: the gradient of 64 rows 107 us in one slice of 256 bytes, 125 in two.
    const int lr = row_lanes(a.pieces, format == SDM_F32 ? 32 : format == SDM_BF16 ? 16 : 8);
    a.slices = (a.pieces + lr - 1) / lr;
    const bool one = a.groups <= 1;
    const Kernel k = grad ? (format == SDM_INT8   ? kernel_of<Int8, true, 8>(lr, one)
                             : format == SDM_FP8  ? kernel_of<Fp8, true, 8>(lr, one)
                             : format == SDM_INT4 ? kernel_of<Int4, true, 8>(lr, one)
                             : format == SDM_BF16 ? kernel_of<Bf16, true, 16>(lr, one)
                                                  : kernel_of<F32, true, 32>(lr, one))
                          : (format == SDM_INT8  ? kernel_of<Int8, false, 8>(lr, one)
                             : format == SDM_FP8 ? kernel_of<Fp8, false, 8>(lr, one)
                                                 : kernel_of<Int4, false, 8>(lr, one));
    // a slice starts at a multiple of them, and so does every row; the same tokens with 64 and 64 rows of 128 columns
    // in groups of 32: 191 us (the gradient of 64 rows 108) by four, 199 (111) one by one
    const int slice_groups = std::max(1, lr * (format == SDM_INT4 ? 32 : 16) / a.group);
    a.scale_words = 1;
    for (int words = 2; words <= 4; words *= 2)
        if (a.groups % words == 0 && (a.slices == 1 || slice_groups % words == 0) && reinterpret_cast<uintptr_t>(a.scales) % (4 * words) == 0)
            a.scale_words = words;
    // one block for every SM, of as many warps as find room for their stages
    const size_t prefix = a.chunk_valid ? ((size_t)(a.tokens / a.chunk) + 4) / 4 * 16 : 0;
    const size_t room = smem_per_sm() - smem_reserved_per_block() - kRingWarps * 4 - prefix;
    const int warps = (int)std::min<size_t>(kRingWarps, room / k.per_warp);
    const size_t smem = prefix + k.per_warp * warps;
    const int rc = allow_smem(k.fn, smem);
    if (rc != 0) return rc;
    const int64_t units = a.tokens * (grad ? 1 : a.slices);
    const int64_t blocks = std::min((int64_t)sm_count(), (units + warps - 1) / warps);
    void* args[] = {&a};
    return launch_pdl_raw(k.fn, dim3((unsigned)blocks), dim3(warps * 32), smem, stream, args);
}

cudaError_t gather_ring_status(void** word) { return cudaGetSymbolAddress(word, g_ring_status); }

}  // namespace sdm
