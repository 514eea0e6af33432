/*
 * sdm.h - C ABI of the GB300 (sm_103a) sparse delta-memory (SDM) decode-state library.
 *
 * Three operations, each one kernel launch on the caller's stream:
 *   sdm_decode_step  one write-then-read token for every stream (sdm_decode_step_ex: with flags)
 *   sdm_decode_seq   T tokens for every stream in one persistent launch (sdm_decode_seq_ex: with
 *                    flags, e.g. the stream-major [n_streams, T, .] layout of a prompt)
 *   sdm_gather       per-token weighted sums of bank rows (one or two operands), optional stash
 *                    (sdm_gather_kpos: with a compact snapshot instead; sdm_gather_plan_*: a
 *                    checked launch, replayed per slab of an index tensor; _launch_ex: with
 *                    flags)
 *
 *
 * and the operators around them (routing and quantised banks, at the end of this file):
 *   sdm_route          scores to slots and weights (top-k), sdm_route_backward its gradient (_ex: with
 *                      the weights, by which entries that filled up are known)
 *   sdm_quantize_rows  rows into a quantised bank, sdm_dequantize_rows back out of it
 *   sdm_qgather        weighted sums of quantised rows, sdm_gather_dw the weights' gradient
 *   sdm_qdecode_step   write-then-read tokens on a quantised bank (sdm_qdecode_seq: T tokens)
 *   sdm_balance        a router's balance loss and counts, with the gradient of its logits
 *   sdm_lookup         scaled rows of a table by token, sdm_lookup_backward the table's gradient
 *   sdm_gather_drows   the gradient of the bank's rows in a gather
 *
 * Common rules
 *   - Every pointer argument except `stream` (and the host records and arrays named as such) is a
 *     DEVICE pointer the caller owns; the library keeps no pointer after the call returns (apart
 *     from the work it enqueued, and from a gather plan record, which the caller owns and which
 *     holds the pointers it was made with) and frees nothing.
 *   - Calls allocate no memory, synchronise nothing and only enqueue work on `stream` (NULL = the
 *     legacy default stream), so they may be captured in a CUDA graph.
 *   - Return value: 0 = launched (or nothing to do); < 0 = argument error (an SDM_E* code below,
 *     nothing launched); > 0 = the cudaError_t of a failed launch (the error state is consumed).
 *   - Index ranges are the caller's contract: decode slots must lie in the bank, every stream's
 *     slots must be private to it and its W write slots distinct (none of this is checked, as in
 *     the reference). A float32 bank of 64 or more columns is taken to hold fewer than 2^32 rows
 *     (it would exceed 1 TiB otherwise): its streaming kernel keeps slots as 32-bit row indices. The gather knows the bank's row count and skips out-of-range rows, raising
 *     SDM_DEV_BAD_INDEX in the device status word (sdm_device_status).
 *   - Launches use programmatic stream serialization: a kernel may be scheduled while the previous
 *     kernel on the stream is still finishing, but it reads and writes no memory before that kernel
 *     has completed (griddepcontrol.wait), so stream order is kept. The one exception is opt-in:
 *     with SDM_INPUTS_READY an _ex call may read its inputs (never the bank, never its outputs)
 *     and warm L2 before that wait, on the caller's promise that those inputs are already final.
 *   - bfloat16 data is raw 16-bit patterns (the high half of an IEEE float32).
 *   - Results are deterministic: every sum is accumulated in a fixed order independent of the GPU.
 *
 * Reference: the "sparse-delta-memory 2.0.0" wheel, files sparse_delta_memory/decode.py
 * (sdm_decode_step, _decode_launch, _sdm_decode_kernel) and sparse_delta_memory/cuda/gather_cuda.py
 * (module docstring, token_gather).
 */
#ifndef SDM_H
#define SDM_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* A CUDA stream handle; layout-compatible with cudaStream_t / CUstream. */
typedef struct CUstream_st* sdm_stream_t;

/* bank / weight element types */
#define SDM_BF16 0
#define SDM_F32 1
/* index element types */
#define SDM_I32 0
#define SDM_I64 1

/* argument errors (negative return values; nothing was launched) */
#define SDM_OK 0
#define SDM_ENULL (-1)      /* a required pointer is NULL */
#define SDM_EDTYPE (-2)     /* bank or weight dtype is not SDM_BF16 / SDM_F32 */
#define SDM_EIDX (-3)       /* index dtype is not SDM_I32 / SDM_I64 */
#define SDM_EHD (-4)        /* head_dim < 1 or > 65536 */
#define SDM_EWIDTH (-5)     /* W, R or a gather width outside 1..256 */
#define SDM_EGATES (-6)     /* G is neither 1 nor W */
#define SDM_ECOUNT (-7)     /* negative count, n_slots < 1 or >= 2^31, or more units than one launch holds */
#define SDM_ECHUNK (-8)     /* chunk < 1, tokens not a multiple of chunk, or valid outside 0..chunk */
#define SDM_EALIGN (-9)     /* a pointer is not aligned to its element size */
#define SDM_EOVERLAP (-10)  /* an output overlaps memory that the call reads (a gather's: its bank), or another output */
#define SDM_ENOPS (-11)     /* gather operand count is not 1 or 2 */
#define SDM_EPLAN (-12)     /* not an initialised gather or decode plan (wrong tag or record size) */
#define SDM_EROW (-13)      /* row0 outside 0..row0_max, row0_max + tokens beyond the index rows, or a plan step outside 0..T-1 */
#define SDM_EDEVICE (-14)   /* the current device is not the one the plan was made on */
#define SDM_EFLAGS (-15)    /* unknown bits in the flags of an _ex entry point */

#define SDM_EFORMAT (-16)   /* the format is not one that this operation takes */
#define SDM_EGROUP (-17)    /* a scale's group is not 32, 64 or 128 columns */
#define SDM_EROUTE (-18)    /* routing sizes, score kind or groups out of range */
#define SDM_ESTRIDE (-19)   /* a row stride is smaller than the row */
#define SDM_EWORKSPACE (-20) /* the workspace is smaller than the call's _workspace function says */

/* bits of the device status word */
#define SDM_DEV_TIMEOUT 1u   /* reserved: a kernel gave up a bounded wait (no current kernel waits) */
#define SDM_DEV_BAD_INDEX 2u /* the gather met a row index outside [0, n_slots) and skipped it */

/*
 * sdm_decode_step - advance every stream by one token: write, then read.
 *
 * Defined by sdm_decode_step (decode.py): per stream s, with d_w = exp(g[s, G == 1 ? 0 : w]),
 *     retrieved      = sum_w k_val[s,w] * d_w * bank[k_idx[s,w]]
 *     delta_v        = beta[s] * (v[s] - retrieved)
 *     bank[k_idx[w]] = d_w * bank[k_idx[w]] + k_val[s,w] * delta_v        (all w)
 *     out[s]         = sum_r q_val[s,r] * bank[q_idx[s,r]]                (after the write)
 * k_val, v and q_val are rounded to the bank dtype (round to nearest even) before use; beta and
 * g are used in float32; d_w is the float32 nearest to e^g; all arithmetic is float32 and the
 * new rows and the readings are rounded to the bank dtype.
 *
 *   bank      [n_slots, hd] bank dtype, row-major, updated in place
 *   k_idx     [n_streams, W] idx dtype: write slots (distinct within a stream)
 *   k_val     [n_streams, W] float32: write weights
 *   v         [n_streams, hd] float32: values
 *   beta      [n_streams] float32: write strengths
 *   g         [n_streams, G] float32: log-decay per token (G == 1) or per write (G == W)
 *   q_idx     [n_streams, R] idx dtype: read slots (repeats allowed)
 *   q_val     [n_streams, R] float32: read weights
 *   out       [n_streams, hd] bank dtype: readings
 *   n_streams >= 0 (0: nothing launched); hd >= 1; 1 <= W, R <= 256; G in {1, W}
 *   bank_dtype SDM_BF16 | SDM_F32; idx_dtype SDM_I32 | SDM_I64 (both index arrays)
 */
int sdm_decode_step(void* bank, const void* k_idx, const float* k_val, const float* v, const float* beta,
                    const float* g, const void* q_idx, const float* q_val, void* out, int64_t n_streams, int hd,
                    int W, int R, int G, int bank_dtype, int idx_dtype, sdm_stream_t stream);

/*
 * sdm_decode_step_ex - sdm_decode_step with flags; flags == 0 is sdm_decode_step.
 *
 * SDM_INPUTS_READY promises that every input but the bank (k_idx, k_val, v, beta, g, q_idx,
 * q_val) was complete before the kernel enqueued just ahead of this launch on the stream began.
 * The launch may then read them, derive the token's weights and gates and warm L2 with the
 * token's bank rows before it waits for that kernel (the launches of this library chain by
 * programmatic dependent launch); it reads and writes the bank, and writes `out`, only after the
 * wait. Results are the same bits as without the flag. Use it for steps whose inputs are staged
 * ahead (e.g. one CUDA graph of many steps over inputs filled before the replay); without the
 * promise the flag may read stale inputs. Unknown bits return SDM_EFLAGS.
 */
#define SDM_INPUTS_READY 1u
int sdm_decode_step_ex(void* bank, const void* k_idx, const float* k_val, const float* v, const float* beta,
                       const float* g, const void* q_idx, const float* q_val, void* out, int64_t n_streams, int hd,
                       int W, int R, int G, int bank_dtype, int idx_dtype, unsigned flags, sdm_stream_t stream);

/*
 * sdm_decode_seq - T tokens for every stream in one launch, equal to T sdm_decode_step calls.
 *
 * One block owns one (stream, column slice) for all T tokens; the reads of token t and the
 * retrieve of token t+1 are ordered after token t's writes by a block barrier, which is valid
 * because no other block touches those slots and columns (the barrier argument of
 * _sdm_decode_kernel in decode.py).
 *
 * Every per-token array gains a leading time axis (time-major): k_idx, k_val [T, n_streams, W];
 * v [T, n_streams, hd]; beta [T, n_streams]; g [T, n_streams, G]; q_idx, q_val [T, n_streams, R];
 * out [T, n_streams, hd]. T >= 0 (0: nothing launched). Other arguments as sdm_decode_step.
 */
int sdm_decode_seq(void* bank, const void* k_idx, const float* k_val, const float* v, const float* beta,
                   const float* g, const void* q_idx, const float* q_val, void* out, int64_t n_streams, int hd,
                   int W, int R, int G, int T, int bank_dtype, int idx_dtype, sdm_stream_t stream);

/*
 * sdm_decode_seq_ex - sdm_decode_seq with flags; flags == 0 is sdm_decode_seq.
 *
 * SDM_STREAM_MAJOR: every per-token array is in the layer's own stream-major layout, each
 * stream's T tokens contiguous: k_idx, k_val [n_streams, T, W]; v [n_streams, T, hd]; beta
 * [n_streams, T]; g [n_streams, T, G]; q_idx, q_val [n_streams, T, R]; and the readings go to
 * out [n_streams, T, hd]. This is the [P, T, .] layout of a prompt that forward_steps
 * (forward.py) stages to time-major with stage_time_major before its steps and whose readings it
 * takes back with unstage_time_major; here the kernel reads and writes that layout by stride, so
 * neither staging copy is made. Results are the bits of sdm_decode_seq on the staged arrays.
 * SDM_INPUTS_READY: as for sdm_decode_step_ex (token 0's inputs are read before the wait).
 * Unknown bits return SDM_EFLAGS. Other arguments as sdm_decode_seq.
 */
#define SDM_STREAM_MAJOR 2u
int sdm_decode_seq_ex(void* bank, const void* k_idx, const float* k_val, const float* v, const float* beta,
                      const float* g, const void* q_idx, const float* q_val, void* out, int64_t n_streams, int hd,
                      int W, int R, int G, int T, int bank_dtype, int idx_dtype, unsigned flags, sdm_stream_t stream);

/*
 * Decode-step plan: T single-token steps over time-major inputs, checked once (the decode-side
 * counterpart of the gather launch plan below, for a loop that launches one token at a time, e.g.
 * while serving; the pages drive their decode step from such a loop, forward.py, and check each
 * launch in decode.py's sdm_decode_step). sdm_decode_plan_init checks the arguments of sdm_decode_seq(..., T, ...) once
 * and records the launch of one token; sdm_decode_plan_launch(t) then launches exactly
 * sdm_decode_step on the rows of token t (k_idx + t * n_streams * W, ..., out + t * n_streams * hd),
 * and sdm_decode_plan_walk launches tokens t0 .. t0 + n - 1 in order from one call. The record is
 * caller-owned, valid on the device current at init, in this process, until the library is
 * unloaded; it keeps the pointers given at init (their memory must stay allocated). Every step
 * returns 0, an SDM_E* code (nothing launched) or the cudaError_t of a failed launch.
 */
#define SDM_DECODE_PLAN_BYTES 512
typedef struct sdm_decode_plan {
    uint64_t opaque[SDM_DECODE_PLAN_BYTES / 8];
} sdm_decode_plan;

/*
 * sdm_decode_plan_init - check a time-major T-token decode once and record a one-token launch in
 * *plan (nothing is launched). Arguments as sdm_decode_seq; T >= 0. Returns 0, an SDM_E* code
 * (the record untouched) or a cudaError_t from the device queries and settings.
 */
int sdm_decode_plan_init(sdm_decode_plan* plan, void* bank, const void* k_idx, const float* k_val, const float* v,
                         const float* beta, const float* g, const void* q_idx, const float* q_val, void* out,
                         int64_t n_streams, int hd, int W, int R, int G, int T, int bank_dtype, int idx_dtype);

/*
 * sdm_decode_plan_launch - step t of a plan (0 <= t < T, else SDM_EROW); flags 0 or
 * SDM_INPUTS_READY (as for sdm_decode_step_ex). Checks, in order: the flags (SDM_EFLAGS), the
 * record (SDM_EPLAN), t (SDM_EROW), the current device (SDM_EDEVICE).
 */
int sdm_decode_plan_launch(const sdm_decode_plan* plan, int t, unsigned flags, sdm_stream_t stream);

/*
 * sdm_decode_plan_walk - steps t0, t0 + 1, ..., t0 + n - 1 of a plan, enqueued in order from one
 * call (n >= 0, else SDM_ECOUNT; every step inside 0..T-1, else SDM_EROW). All checks come before
 * the first launch; a positive return is the cudaError_t of the first failed launch (the steps
 * before it were launched, none after it).
 */
int sdm_decode_plan_walk(const sdm_decode_plan* plan, int t0, int n, unsigned flags, sdm_stream_t stream);

/*
 * sdm_gather - token gather (gather_cuda.py, module docstring and token_gather).
 *
 * For every token t in [0, tokens) and operand o in [0, n_ops):
 *     out[o][t, :] = sum_n w[o][t, n] * bank[idx[o][t, n], :]    (float32, ascending n, fmaf)
 *     stash[t, n, :] = bank[idx[0][t, n], :]                      (raw rows of operand 0)
 * Token t is padding when t % chunk >= valid_t, where valid_t = chunk_valid[t / chunk] if
 * chunk_valid is not NULL, else `valid`. Padding tokens read nothing and get zero outputs and
 * all-zero stash rows. The bank must not be written while the gather runs.
 *
 *   bank       [n_slots, hd] bank dtype (read only); 1 <= n_slots < 2^31
 *   n_ops      1 or 2; idx[1], w[1], out[1], width[1] are ignored when n_ops == 1
 *   idx[o]     [tokens, width[o]] idx dtype (same dtype for both operands)
 *   w[o]       [tokens, width[o]] w dtype: SDM_BF16 or SDM_F32 (same for both operands)
 *   out[o]     [tokens, hd] float32
 *   width[o]   1..256
 *   stash      [tokens, width[0], hd] bank dtype, or NULL for no stash
 *   tokens     >= 0, a multiple of chunk; chunk >= 1; 0 <= valid <= chunk (ignored when
 *              chunk_valid is given)
 *   chunk_valid [tokens / chunk] int32 per-chunk valid counts in 0..chunk, or NULL
 * The arrays idx, w, out and width are HOST arrays of two entries holding device pointers.
 * Outputs and the stash must not overlap the bank.
 */
int sdm_gather(const void* bank, int64_t n_slots, int hd, int bank_dtype, int n_ops, const void* const idx[2],
               const void* const w[2], float* const out[2], const int width[2], int idx_dtype, int w_dtype,
               void* stash, int64_t tokens, int chunk, int valid, const int32_t* chunk_valid, sdm_stream_t stream);

/*
 * sdm_gather_kpos - token gather with a compact snapshot of operand 0 instead of the stash
 * (gather_cuda.py, the compact-snapshot form of the kernel: `kpos`, `crow`).
 *
 * Outputs as sdm_gather. Operand 0's rows go to a snapshot of chunk * width[0] rows per chunk:
 * for every live token t and entry n with kpos[t, n] >= 0,
 *     compact[t / chunk, kpos[t, n], :] = bank[idx[0][t, n], :]
 * (kpos names the entry's first position among the chunk's sorted rows, so each distinct row is
 * stored once per chunk). Entries with kpos = -1 and padding tokens store nothing, and no other
 * snapshot row is written. An entry whose kpos is >= chunk * width[0] or whose row index is outside
 * [0, n_slots) stores nothing and raises SDM_DEV_BAD_INDEX.
 *
 *   compact    [tokens / chunk, chunk * width[0], hd] bank dtype (device), must not overlap the bank
 *   kpos       [tokens, width[0]] int32 (device)
 * Other arguments as sdm_gather (there is no stash argument).
 */
int sdm_gather_kpos(const void* bank, int64_t n_slots, int hd, int bank_dtype, int n_ops, const void* const idx[2],
                    const void* const w[2], float* const out[2], const int width[2], int idx_dtype, int w_dtype,
                    void* compact, const int32_t* kpos, int64_t tokens, int chunk, int valid,
                    const int32_t* chunk_valid, sdm_stream_t stream);

/*
 * Gather launch plan (gather_cuda.py, token_gather_dc_plan / token_gather_dc_step): the checks
 * and the launch geometry of a no-stash gather, done once; each step then only checks row0 and
 * valid and relaunches the same kernel. Meant for a loop over the slabs of one index tensor:
 * launch k reads index and weight rows [row0, row0 + tokens) and writes out[o][0 .. tokens).
 *
 * The plan is a caller-owned record (any memory the caller likes, usually a host stack or struct
 * field); the library writes it in sdm_gather_plan_init and only reads it afterwards. It holds the
 * device pointers it was given: they must stay valid (and the arrays unresized) while the plan is
 * used. It is valid on the device that was current at init, in this process, until the library is
 * unloaded. Copying the record copies the plan.
 */
#define SDM_GATHER_PLAN_BYTES 512
typedef struct sdm_gather_plan {
    uint64_t opaque[SDM_GATHER_PLAN_BYTES / 8];
} sdm_gather_plan;

/*
 * sdm_gather_plan_init - check a no-stash sdm_gather once, at the largest row0 it will be used
 * with, and record its launch in *plan. Nothing is launched.
 *
 *   plan       host pointer to the record to fill (written only when 0 is returned)
 *   idx[o], w[o] [rows, width[o]]: the whole index / weight arrays of operand o (device)
 *   out[o]     [tokens, hd] float32, written by every launch (device)
 *   rows       index rows the arrays hold; row0_max >= 0 with row0_max + tokens <= rows
 *   tokens, chunk  tokens per launch (>= 0, a multiple of chunk), chunk >= 1
 * Other arguments as sdm_gather. Returns 0, an SDM_E* code, or a cudaError_t from the device
 * queries and settings (current device, multiprocessor count, the kernel's shared-memory limit,
 * occupancy).
 */
int sdm_gather_plan_init(sdm_gather_plan* plan, const void* bank, int64_t n_slots, int hd, int bank_dtype, int n_ops,
                         const void* const idx[2], const void* const w[2], float* const out[2], const int width[2],
                         int idx_dtype, int w_dtype, int64_t rows, int64_t row0_max, int64_t tokens, int chunk);

/*
 * sdm_gather_plan_launch - one step of a plan: the planned gather over index rows
 * [row0, row0 + tokens) with `valid` live tokens per chunk (the tokens at t % chunk >= valid are
 * padding, as in sdm_gather). Checks, in order: the record (SDM_EPLAN), 0 <= row0 <= row0_max
 * (SDM_EROW), 0 <= valid <= chunk (SDM_ECHUNK), the current device (SDM_EDEVICE); then launches
 * on `stream` exactly what sdm_gather would launch for the same rows. Returns 0, an SDM_E* code
 * (nothing launched) or the cudaError_t of a failed launch.
 */
int sdm_gather_plan_launch(const sdm_gather_plan* plan, int64_t row0, int valid, sdm_stream_t stream);

/*
 * sdm_gather_plan_launch_ex - sdm_gather_plan_launch with flags; flags == 0 is
 * sdm_gather_plan_launch. SDM_INPUTS_READY promises that the launch's index and weight rows
 * [row0, row0 + tokens) were complete before the kernel enqueued just ahead of it on the stream
 * began: the launch may then read them and warm L2 with the rows they name before it waits for
 * that kernel (which may still be writing the bank). The bank is read, and the outputs written,
 * only after the wait; results are the same bits as without the flag. Unknown bits return
 * SDM_EFLAGS before any other check.
 */
int sdm_gather_plan_launch_ex(const sdm_gather_plan* plan, int64_t row0, int valid, unsigned flags,
                              sdm_stream_t stream);

/*
 * sdm_gather_plan_walk - n steps of a plan from one call: the native step loop over a walk of
 * slabs (sparse-delta-memory 2.0.0, cuda/gather_cuda.py: `token_gather_dc_step` driven from a
 * native loop), without a host-language call per slab.
 *
 *   row0[i]    host array of n slab offsets (each 0 <= row0[i] <= row0_max)
 *   valid[i]   host array of n live-token counts per chunk (0..chunk), or NULL: chunk for every slab
 *   n          slabs, >= 0
 *   flags      0 or SDM_INPUTS_READY (applies to every slab; see sdm_gather_plan_launch_ex)
 * Slab i is exactly sdm_gather_plan_launch_ex(plan, row0[i], valid[i], flags, stream), enqueued in
 * order on `stream`. Every argument is checked before the first launch: an SDM_E* code means
 * nothing was launched. A positive return is the cudaError_t of the first failed launch; the
 * slabs before it were launched, none after it.
 */
int sdm_gather_plan_walk(const sdm_gather_plan* plan, const int64_t* row0, const int32_t* valid, int n,
                         unsigned flags, sdm_stream_t stream);

/*
 * Quantised banks
 *
 * A quantised bank holds n_slots rows of hd columns as two device arrays:
 *   codes   [n_slots, row_bytes] bytes, 16-byte aligned; row_bytes = sdm_quant_row_bytes(hd, format):
 *           one byte a column (SDM_INT8, SDM_FP8) or two columns a byte, the even one in the low half
 *           (SDM_INT4), padded with zero bytes to a multiple of 16
 *   scales  [n_slots, ceil(hd / group)] float32; group = 32, 64 or 128 columns share a scale
 * and stands for scale * code, with code a two's complement integer (SDM_INT8, SDM_INT4) or a float
 * with 4 exponent and 3 mantissa bits (SDM_FP8, e4m3 without infinities).
 *
 * A group of values x is stored as
 *     scale = max|x| / L,  code = round(x * (L / max|x|)),  L = 127 (INT8), 448 (FP8), 7 (INT4)
 * in float32, rounding codes to nearest even. A group whose max|x| is below 2^-100 is stored as
 * zeros with scale 0; one that holds an infinity or NaN gets the scale NaN, so that it reads back
 * as NaN rather than as something plausible.
 *
 * In the calls from here on, outputs must not overlap what the call reads, nor one another (SDM_EOVERLAP;
 * the gathers look at the bank only). Rows by a stride may lie beside others in a wider matrix of that
 * stride. One output may take its input's place: float32 readings that of v in the decode.
 */
#define SDM_INT8 2
#define SDM_FP8 3
#define SDM_INT4 4

/* Bytes from one row of codes to the next, or 0 for an unknown format or hd outside 1..65536. */
int sdm_quant_row_bytes(int hd, int format);

/*
 * sdm_quantize_rows - write rows into a quantised bank: row i goes to slot slots[i], or to slot i
 * when slots is NULL (then n_rows <= n_slots, else SDM_EROW). The slots of one call must be
 * distinct. A slot outside [0, n_slots) is skipped and raises SDM_DEV_BAD_INDEX.
 *
 *   rows       n_rows rows of hd columns, row_dtype SDM_BF16 | SDM_F32, row i at rows + i * row_stride
 *              elements (row_stride >= hd)
 *   slots      [n_rows] idx dtype, or NULL
 */
int sdm_quantize_rows(void* codes, float* scales, int64_t n_slots, int hd, int group, int format, const void* rows,
                      int64_t row_stride, int row_dtype, const void* slots, int idx_dtype, int64_t n_rows,
                      sdm_stream_t stream);

/*
 * sdm_dequantize_rows - read rows of a quantised bank back: row i is scale * code of slot slots[i]
 * (slot i when slots is NULL; repeats allowed), computed in float32 and rounded to row_dtype once.
 * A slot outside [0, n_slots) gives a zero row and raises SDM_DEV_BAD_INDEX. Arguments as
 * sdm_quantize_rows, with `rows` written.
 */
int sdm_dequantize_rows(const void* codes, const float* scales, int64_t n_slots, int hd, int group, int format,
                        void* rows, int64_t row_stride, int row_dtype, const void* slots, int idx_dtype,
                        int64_t n_rows, sdm_stream_t stream);

/*
 * sdm_qgather - sdm_gather (no stash) over a quantised bank:
 *     out[o][t, :] = sum_n w[o][t, n] * row(idx[o][t, n])
 * with the sum in float32 in an order that depends on the sizes alone. Padding tokens
 * (t % chunk >= valid) read nothing and get zeros. An entry whose index is outside [0, n_slots) is
 * skipped, whatever its weight, and raises SDM_DEV_BAD_INDEX. Arguments as sdm_gather and above.
 * From 4096 tokens and operands on (of a call with chunk_valid: in at most 16384 chunks), the product
 * of a weight with a scale enters in three parts of 11 bits, relative to the largest of up to 32
 * neighbouring entries: it keeps all its bits down to 2^-22 of that, and what lies below 2^-46 of it is
 * lost. (The same holds for dout in sdm_gather_dw, among the columns of a row's slice; over a bf16 bank
 * with an infinite row the gradients it enters may be NaN.) More chunks, or fewer tokens, are summed in
 * float32 throughout, by a kernel that is two to three times slower on many tokens.
 */
int sdm_qgather(const void* codes, const float* scales, int64_t n_slots, int hd, int group, int format, int n_ops,
                const void* const idx[2], const void* const w[2], float* const out[2], const int width[2],
                int idx_dtype, int w_dtype, int64_t tokens, int chunk, int valid, const int32_t* chunk_valid,
                sdm_stream_t stream);

/*
 * sdm_gather_dw - gradient of the weights of sdm_gather or sdm_qgather:
 *     dw[o][t, n] = sum_c dout[o][t, c] * row(idx[o][t, n])[c]
 * summed in float32 and rounded to dw_dtype once. Padding tokens read nothing and get zeros; an
 * entry whose index is outside [0, n_slots) gets zero, whatever dout holds, and raises SDM_DEV_BAD_INDEX.
 *
 *   bank       format SDM_BF16 | SDM_F32: the [n_slots, hd] bank (scales and group are ignored);
 *              SDM_INT8 | SDM_FP8 | SDM_INT4: the codes of a quantised bank
 *   dout[o]    [tokens, hd] float32
 *   dw[o]      [tokens, width[o]] dw_dtype SDM_BF16 | SDM_F32
 */
int sdm_gather_dw(const void* bank, const float* scales, int64_t n_slots, int hd, int group, int format, int n_ops,
                  const void* const idx[2], const float* const dout[2], void* const dw[2], const int width[2],
                  int idx_dtype, int dw_dtype, int64_t tokens, int chunk, int valid, const int32_t* chunk_valid,
                  sdm_stream_t stream);

/*
 * sdm_qdecode_step / sdm_qdecode_seq - sdm_decode_step / sdm_decode_seq on a quantised bank
 * (SDM_INT8 or SDM_FP8; 4 bits are too few for rows that are written again and again):
 *     retrieved      = sum_w k_val[w] * d_w * row(k_idx[w]),  d_w = exp(g[G == 1 ? 0 : w])
 *     delta_v        = beta * (v - retrieved)
 *     row(k_idx[w]) <- quantised(d_w * row(k_idx[w]) + k_val[w] * delta_v)
 *     out            = sum_r q_val[r] * row(q_idx[r])       (after the write)
 * All arithmetic is float32; k_val, v and q_val are used as given; the readings are rounded to
 * out_dtype once. A decay alone (k_val = 0) goes into the scales and leaves the codes as they are.
 * The slots of a stream are private to it and its W write slots distinct, as in sdm_decode_step; a
 * slot outside [0, n_slots) reads as zeros, is not written, and raises SDM_DEV_BAD_INDEX.
 * sdm_qdecode_seq takes time-major arrays, or with SDM_STREAM_MAJOR stream-major ones
 * (sdm_decode_seq_ex); other flags return SDM_EFLAGS.
 */
int sdm_qdecode_step(void* codes, float* scales, int64_t n_slots, const void* k_idx, const float* k_val,
                     const float* v, const float* beta, const float* g, const void* q_idx, const float* q_val,
                     void* out, int64_t n_streams, int hd, int group, int format, int W, int R, int G, int idx_dtype,
                     int out_dtype, sdm_stream_t stream);
int sdm_qdecode_seq(void* codes, float* scales, int64_t n_slots, const void* k_idx, const float* k_val,
                    const float* v, const float* beta, const float* g, const void* q_idx, const float* q_val,
                    void* out, int64_t n_streams, int hd, int group, int format, int W, int R, int G, int T,
                    int idx_dtype, int out_dtype, unsigned flags, sdm_stream_t stream);

/*
 * Routing: which k of n entries a token takes, and with which weights. The entries are a stream's
 * memory slots (the results are then k_idx / k_val or q_idx / q_val of the decode, or idx / w of a
 * gather) or experts (whose output rows a gather joins).
 *
 * sdm_route - for every token t with logits x = logits[t, :]:
 *     s_j = exp(x_j - max x) / sum_i exp(x_i - max x)     (SDM_SOFTMAX)
 *     s_j = 1 / (1 + exp(-x_j))                           (SDM_SIGMOID)
 *   Entries are ranked by s_j + bias_j when bias is given, else by s_j (SDM_SIGMOID) or x_j
 *   (SDM_SOFTMAX: the same order, without the rounding of s). Entries whose x is -inf or NaN, or
 *   whose rank is -inf or NaN, are masked: they rank last and have weight 0. Several +inf under a
 *   softmax share it evenly.
 *   With n_groups > 1 the entries form n_groups consecutive groups of n / n_groups; the
 *   top_groups best groups stay and the entries of the others are masked. A group's score is its
 *   largest rank (group_top 1) or the sum of its two largest (group_top 2; for a softmax without a
 *   bias the sum of the two largest exp(x_j - max x)); masked entries take no part, and a group
 *   without others comes last.
 *   The k best entries are taken, best first; equal ranks, of groups too, go by the lower index.
 *   idx[t, i] is the entry's number j (plus base[t] when base is given), and
 *     w[t, i] = scale * s_j, or with SDM_RENORM  scale * s_j / sum of the chosen s
 *   (0 where that sum is 0). When fewer than k entries are not masked, masked ones fill up in
 *   index order with weight 0, so the k indices are always distinct.
 *
 *   logits      row t at logits + t * row_stride elements (row_stride >= n), SDM_BF16 | SDM_F32
 *   bias        [n] float32, or NULL; moves the choice only, never the weights
 *   base        [tokens] idx dtype, or NULL: e.g. the first slot of the token's stream
 *   idx, w      [tokens, k] idx dtype and float32
 *   1 <= n <= 65536, 1 <= k <= min(n, 256); n_groups divides n, at most 256; 1 <= top_groups <=
 *   n_groups; group_top 1 or 2 (else SDM_EROUTE); flags 0 or SDM_RENORM
 */
#define SDM_SOFTMAX 0
#define SDM_SIGMOID 1
#define SDM_RENORM 4u
int sdm_route(const void* logits, int64_t row_stride, int logit_dtype, const float* bias, const void* base, void* idx,
              float* w, int64_t tokens, int n, int k, int score, int n_groups, int top_groups, int group_top,
              float scale, unsigned flags, int idx_dtype, sdm_stream_t stream);

/*
 * sdm_route_backward - gradient of the logits: with u_i = scale * dw[t, i], or with SDM_RENORM
 * u_i = scale / S * (dw[t, i] - sum_m dw[t, m] * s_m / S), S the sum of the chosen s,
 *     dlogits_j = u_j * s_j * (1 - s_j)                        (SDM_SIGMOID; 0 for entries not chosen)
 *     dlogits_j = s_j * (u_j [chosen] - sum_i u_i * s_i)       (SDM_SOFTMAX)
 * The choice itself, and the bias, have no gradient. idx is what sdm_route returned (base added);
 * an index outside the row is skipped and raises SDM_DEV_BAD_INDEX; the k indices of a token are
 * distinct. Masked logits get 0, and the dw of masked entries, which may be anything, takes no part.
 *
 * Where sdm_route filled up with masked entries whose logits are live (of groups that did not stay, or
 * with a rank of -inf by their bias) it has to be known which these are: sdm_route_backward_ex takes
 * the weights that sdm_route returned, and an entry of weight 0 counts as not chosen. sdm_route_backward
 * is the call without them (w NULL): it takes every entry with a live logit as chosen, which is so
 * wherever k entries at least are not masked, and without groups and biases always.
 *
 *   w           [tokens, k] float32, or NULL
 *   dlogits     row t at dlogits + t * dlogits_stride elements, logit dtype; all n columns written
 */
int sdm_route_backward(const void* logits, int64_t row_stride, int logit_dtype, const void* base, const void* idx,
                       const float* dw, void* dlogits, int64_t dlogits_stride, int64_t tokens, int n, int k, int score,
                       float scale, unsigned flags, int idx_dtype, sdm_stream_t stream);
int sdm_route_backward_ex(const void* logits, int64_t row_stride, int logit_dtype, const void* base, const void* idx,
                          const float* w, const float* dw, void* dlogits, int64_t dlogits_stride, int64_t tokens, int n,
                          int k, int score, float scale, unsigned flags, int idx_dtype, sdm_stream_t stream);

/*
 * Training: the loss that keeps a router's choices spread over its entries, and the gradients of rows
 * that are read by index.
 *
 * Some of these calls work in memory that the caller lends them: `workspace`, 256-byte aligned device
 * memory of at least the bytes that the call's _workspace function stores in *bytes (0: none is needed,
 * and it may be NULL). It holds nothing before the call or after it; calls that may run at the same time
 * need one each, and so do captured graphs that may be replayed at the same time.
 *
 * sdm_balance - for every sequence s of tokens offsets[s] <= t < offsets[s + 1] (all tokens, and one
 * sequence, when offsets is NULL), with T their number:
 *     p_tj      = s_tj / sum_i s_ti          the shares of a token's scores (those of sdm_route; masked
 *                                            entries, and all of a row that is masked throughout, have 0)
 *                                            in float32: a share below 2^-96 may be 0, and one is off by up
 *                                            to 50 steps of 2^-24 and 2.5 more for each unit that its logit
 *                                            lies below the row's largest (softmax) or below 0 (sigmoid)
 *     counts[s, j] = how often the sequence's tokens chose entry j
 *     loss[s]   = scale * n / (T * C) * sum_t sum_j counts[s, j] * p_tj,   C = sum_j counts[s, j]
 * (0 where T or C is 0): scale where choices or scores are spread evenly, up to scale * n where both are on
 * one entry. The counts have no gradient. With dlogits, the logits' gradient too:
 *     dlogits[t, j] = add[t, j] + dloss[s] * scale * n / (T * C) * p_tj * (counts[s, j] - sum_i counts[s, i] * p_ti)
 * for a softmax, and that second term times 1 - s_tj for a sigmoid. A token outside every sequence takes
 * no part; its row of dlogits is that of add, or zeros. Masked logits too have a gradient of 0 here.
 * idx is what sdm_route returned (base added). An entry whose w is 0 is not counted (one that
 * only filled up); without w every entry is. An index outside the row is not counted and raises
 * SDM_DEV_BAD_INDEX.
 *
 *   offsets    [sequences + 1] int32, not decreasing, within 0..tokens; NULL with sequences 1
 *   loss       [sequences] float32; counts [sequences, n] int32
 *   dloss      [sequences] float32, or NULL for ones: the gradient that comes for each loss
 *   add        tokens rows of logit dtype, or NULL; may be dlogits itself with the same stride
 *   dlogits    tokens rows of logit dtype, all n columns written; or NULL (then add and dloss are not read)
 *   tokens and tokens * k below 2^31, sequences below 2^24
 * Other arguments as sdm_route.
 */
int sdm_balance_workspace(int64_t sequences, int64_t* bytes);
int sdm_balance(const void* logits, int64_t row_stride, int logit_dtype, const void* base, const void* idx, const float* w,
                const int32_t* offsets, int64_t sequences, float* loss, int32_t* counts, const float* dloss,
                const void* add, int64_t add_stride, void* dlogits, int64_t dlogits_stride, int64_t tokens, int n, int k,
                int score, float scale, int idx_dtype, void* workspace, int64_t workspace_bytes, sdm_stream_t stream);

/*
 * sdm_lookup - scaled rows by token: out[t, :] = scale * table[tokens[t], :], computed in float32 and
 * rounded to out_dtype once. The token `padding` gives zeros; so does one outside [0, n_rows), which raises
 * SDM_DEV_BAD_INDEX.
 *
 *   table      [n_rows, hd] table_dtype; 1 <= n_rows < 2^31
 *   tokens     [n_tokens] idx dtype (repeats allowed)
 *   padding    a token that stands for nothing, inside the table or not; SDM_NO_PADDING: none does
 *   out        [n_tokens, hd] out_dtype
 */
#define SDM_NO_PADDING INT64_MIN
int sdm_lookup(const void* table, int64_t n_rows, int hd, int table_dtype, const void* tokens, int idx_dtype,
               int64_t n_tokens, int64_t padding, float scale, void* out, int out_dtype, sdm_stream_t stream);

/*
 * sdm_lookup_backward - gradient of the table of sdm_lookup:
 *     grad[r, :] = scale * sum over t with tokens[t] = r of dout[t, :]
 * summed in float32 in an order that depends on the sizes and the tokens alone, and rounded to grad_dtype
 * once. Padding tokens and those outside the table (which raise SDM_DEV_BAD_INDEX) take no part; what is
 * in their dout is not looked at. Rows without tokens become zero; with SDM_ACCUMULATE the sums are added
 * to what grad holds, and only rows that have tokens are read or written.
 *
 *   dout       [n_tokens, hd] dout_dtype; n_tokens below 2^31
 *   grad       [n_rows, hd] grad_dtype
 */
#define SDM_ACCUMULATE 8u
int sdm_lookup_backward_workspace(int64_t n_tokens, int64_t n_rows, int hd, int64_t* bytes);
int sdm_lookup_backward(const void* dout, int dout_dtype, const void* tokens, int idx_dtype, int64_t n_tokens,
                        int64_t padding, float scale, void* grad, int64_t n_rows, int hd, int grad_dtype, unsigned flags,
                        void* workspace, int64_t workspace_bytes, sdm_stream_t stream);

/*
 * sdm_gather_drows - gradient of the bank's rows in sdm_gather (or, of the values that its codes stand for,
 * in sdm_qgather):
 *     drows[r, :] = sum over operands o, live tokens t and entries n with idx[o][t, n] = r of w[o][t, n] * dout[o][t, :]
 * summed, rounded and accumulated as in sdm_lookup_backward. Padding tokens (t % chunk >= valid) and entries of
 * weight 0 take no part, whatever their dout holds; nor do indices outside [0, n_slots), which raise
 * SDM_DEV_BAD_INDEX.
 *
 *   idx[o], w[o]  [tokens, width[o]], w dtype SDM_BF16 | SDM_F32; width[o] 1..256
 *   dout[o]       [tokens, hd] float32
 *   drows         [n_slots, hd] drows_dtype
 *   tokens * (width[0] + width[1]) below 2^31, which is also the `entries` of the workspace
 * Other arguments as sdm_gather.
 */
int sdm_gather_drows_workspace(int64_t entries, int64_t n_slots, int hd, int64_t* bytes);
int sdm_gather_drows(int n_ops, const void* const idx[2], const void* const w[2], const float* const dout[2],
                     const int width[2], int idx_dtype, int w_dtype, void* drows, int64_t n_slots, int hd, int drows_dtype,
                     unsigned flags, int64_t tokens, int chunk, int valid, const int32_t* chunk_valid, void* workspace,
                     int64_t workspace_bytes, sdm_stream_t stream);

/* A static string naming a return code of the calls above. */
const char* sdm_status_string(int status);

/*
 * sdm_device_status - read (and, if clear != 0, reset) the device status word of the current
 * device: an OR of SDM_DEV_* bits raised by kernels since the last reset. Synchronises the whole
 * device first (cudaDeviceSynchronize), so that the kernels of every stream, non-blocking streams
 * included, have finished before the word is read or cleared; not for use inside graph capture.
 * Returns 0 or a cudaError_t (then *status is 0); *status receives the word.
 */
int sdm_device_status(unsigned int* status, int clear);

/* Library version, major * 10000 + minor * 100 + patch. */
int sdm_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SDM_H */
