// C ABI of the quantised banks and the routing: argument validation (host only, before any CUDA
// call) and dispatch to the kernel files. Every entry point follows include/sdm.h: 0 = launched,
// < 0 = argument error, > 0 = cudaError_t.
#include <climits>

#include "sdm.h"
#include "sdm_checks.h"
#include "sdm_internal.h"

namespace {

using namespace sdm::checks;

bool quantised(int format) { return format == SDM_INT8 || format == SDM_FP8 || format == SDM_INT4; }

// The sizes of a quantised bank.
int check_bank(int64_t n_slots, int hd, int group, int format) {
    if (!quantised(format)) return SDM_EFORMAT;
    if (hd < 1 || hd > 65536) return SDM_EHD;
    if (group != 32 && group != 64 && group != 128) return SDM_EGROUP;
    if (n_slots < 1 || n_slots > (int64_t)INT_MAX) return SDM_ECOUNT;
    return SDM_OK;
}

int quant_rows(uint8_t* codes, float* scales, int64_t n_slots, int hd, int group, int format, void* rows,
               int64_t row_stride, int row_dtype, const void* slots, int idx_dtype, int64_t n_rows, bool write,
               sdm_stream_t stream) {
    const int rc = check_bank(n_slots, hd, group, format);
    if (rc != SDM_OK) return rc;
    if (!float_type(row_dtype)) return SDM_EDTYPE;
    if (slots && !index_type(idx_dtype)) return SDM_EIDX;
    if (n_rows < 0 || n_rows > (int64_t)1 << 40) return SDM_ECOUNT;
    if (!slots && n_rows > n_slots) return SDM_EROW;
    if (n_rows == 0) return SDM_OK;
    if (!codes || !scales || !rows) return SDM_ENULL;
    if (row_stride < hd) return SDM_ESTRIDE;
    if (!aligned(codes, 16) || !aligned(scales, 4) || !aligned(rows, float_size(row_dtype)) ||
        (slots && !aligned(slots, index_size(idx_dtype))))
        return SDM_EALIGN;
    const Rows r{rows, n_rows, row_stride, hd, float_size(row_dtype)};
    const Rows c = array(codes, n_slots, sdm_quant_row_bytes(hd, format), 1), sc = array(scales, n_slots, (hd + group - 1) / group, 4);
    const Rows sl = array(slots, n_rows, 1, index_size(idx_dtype));
    if (overlaps(c, sc) || overlaps(r, c) || overlaps(r, sc)) return SDM_EOVERLAP;
    if (write ? overlaps(c, sl) || overlaps(sc, sl) : overlaps(r, sl)) return SDM_EOVERLAP;
    sdm::QuantRowsArgs a{};
    a.codes = codes;
    a.scales = scales;
    a.rows = rows;
    a.slots = slots;
    a.n_slots = n_slots;
    a.row_stride = row_stride;
    a.n_rows = n_rows;
    a.hd = hd;
    a.group = group;
    a.idx64 = idx_dtype == SDM_I64;
    return sdm::launch_quant_rows(a, format, row_dtype, write, reinterpret_cast<cudaStream_t>(stream));
}

// Shared by the gather over a quantised bank and the weights' gradient: operands and padding.
int check_operands(int n_ops, const void* const idx[2], const void* const a0[2], const void* const a1[2],
                   const int width[2], int idx_dtype, int w_dtype, int64_t tokens, int chunk, int valid,
                   const int32_t* chunk_valid) {
    if (!float_type(w_dtype)) return SDM_EDTYPE;
    if (!index_type(idx_dtype)) return SDM_EIDX;
    if (n_ops != 1 && n_ops != 2) return SDM_ENOPS;
    if (!idx || !a0 || !a1 || !width) return SDM_ENULL;
    for (int o = 0; o < n_ops; ++o)
        if (width[o] < 1 || width[o] > 256) return SDM_EWIDTH;
    if (tokens < 0 || tokens > (int64_t)1 << 40) return SDM_ECOUNT;
    if (chunk < 1 || tokens % chunk != 0 || (!chunk_valid && (valid < 0 || valid > chunk))) return SDM_ECHUNK;
    return SDM_OK;
}

}  // namespace

extern "C" {

int sdm_quant_row_bytes(int hd, int format) {
    if (hd < 1 || hd > 65536 || !quantised(format)) return 0;
    return ((format == SDM_INT4 ? (hd + 1) / 2 : hd) + 15) / 16 * 16;
}

int sdm_quantize_rows(void* codes, float* scales, int64_t n_slots, int hd, int group, int format, const void* rows,
                      int64_t row_stride, int row_dtype, const void* slots, int idx_dtype, int64_t n_rows,
                      sdm_stream_t stream) {
    return quant_rows(static_cast<uint8_t*>(codes), scales, n_slots, hd, group, format, const_cast<void*>(rows),
                      row_stride, row_dtype, slots, idx_dtype, n_rows, true, stream);
}

int sdm_dequantize_rows(const void* codes, const float* scales, int64_t n_slots, int hd, int group, int format,
                        void* rows, int64_t row_stride, int row_dtype, const void* slots, int idx_dtype,
                        int64_t n_rows, sdm_stream_t stream) {
    return quant_rows(static_cast<uint8_t*>(const_cast<void*>(codes)), const_cast<float*>(scales), n_slots, hd, group,
                      format, rows, row_stride, row_dtype, slots, idx_dtype, n_rows, false, stream);
}

int sdm_qgather(const void* codes, const float* scales, int64_t n_slots, int hd, int group, int format, int n_ops,
                const void* const idx[2], const void* const w[2], float* const out[2], const int width[2],
                int idx_dtype, int w_dtype, int64_t tokens, int chunk, int valid, const int32_t* chunk_valid,
                sdm_stream_t stream) {
    int rc = check_bank(n_slots, hd, group, format);
    if (rc != SDM_OK) return rc;
    rc = check_operands(n_ops, idx, w, reinterpret_cast<const void* const*>(out), width, idx_dtype, w_dtype, tokens,
                        chunk, valid, chunk_valid);
    if (rc != SDM_OK || tokens == 0) return rc;
    if (!codes || !scales) return SDM_ENULL;
    if (!aligned(codes, 16) || !aligned(scales, 4) || !aligned(chunk_valid, 4)) return SDM_EALIGN;
    const size_t code_bytes = (size_t)n_slots * sdm_quant_row_bytes(hd, format);
    const size_t scale_bytes = (size_t)n_slots * ((hd + group - 1) / group) * 4;
    sdm::QGatherArgs a{};
    for (int o = 0; o < n_ops; ++o) {
        if (!idx[o] || !w[o] || !out[o]) return SDM_ENULL;
        if (!aligned(idx[o], index_size(idx_dtype)) || !aligned(w[o], float_size(w_dtype)) || !aligned(out[o], 4))
            return SDM_EALIGN;
        const size_t out_bytes = (size_t)tokens * hd * 4;
        if (overlaps(out[o], out_bytes, codes, code_bytes) || overlaps(out[o], out_bytes, scales, scale_bytes))
            return SDM_EOVERLAP;
        a.idx[o] = idx[o];
        a.w[o] = w[o];
        a.out[o] = out[o];
        a.width[o] = width[o];
    }
    a.bank = codes;
    a.scales = scales;
    a.n_slots = n_slots;
    a.hd = hd;
    a.group = group;
    a.n_ops = n_ops;
    a.idx64 = idx_dtype == SDM_I64;
    a.w_bf16 = w_dtype == SDM_BF16;
    a.tokens = tokens;
    a.chunk = chunk;
    a.valid = valid;
    a.chunk_valid = chunk_valid;
    return sdm::launch_qgather(a, format, reinterpret_cast<cudaStream_t>(stream));
}

int sdm_gather_dw(const void* bank, const float* scales, int64_t n_slots, int hd, int group, int format, int n_ops,
                  const void* const idx[2], const float* const dout[2], void* const dw[2], const int width[2],
                  int idx_dtype, int dw_dtype, int64_t tokens, int chunk, int valid, const int32_t* chunk_valid,
                  sdm_stream_t stream) {
    const bool plain = float_type(format);
    int rc = plain ? check_bank(n_slots, hd, 32, SDM_INT8) : check_bank(n_slots, hd, group, format);
    if (rc != SDM_OK) return rc;
    rc = check_operands(n_ops, idx, reinterpret_cast<const void* const*>(dout), dw, width, idx_dtype, dw_dtype,
                        tokens, chunk, valid, chunk_valid);
    if (rc != SDM_OK || tokens == 0) return rc;
    if (!bank || (!plain && !scales)) return SDM_ENULL;
    if (!aligned(bank, plain ? float_size(format) : 16) || !aligned(scales, 4) || !aligned(chunk_valid, 4))
        return SDM_EALIGN;
    const size_t bank_bytes = (size_t)n_slots * (plain ? hd * float_size(format) : (size_t)sdm_quant_row_bytes(hd, format));
    const size_t scale_bytes = plain ? 0 : (size_t)n_slots * ((hd + group - 1) / group) * 4;
    sdm::QGatherArgs a{};
    for (int o = 0; o < n_ops; ++o) {
        if (!idx[o] || !dout[o] || !dw[o]) return SDM_ENULL;
        if (!aligned(idx[o], index_size(idx_dtype)) || !aligned(dw[o], float_size(dw_dtype)) || !aligned(dout[o], 4))
            return SDM_EALIGN;
        const size_t dw_bytes = (size_t)tokens * width[o] * float_size(dw_dtype);
        if (overlaps(dw[o], dw_bytes, bank, bank_bytes) || (!plain && overlaps(dw[o], dw_bytes, scales, scale_bytes)))
            return SDM_EOVERLAP;
        a.idx[o] = idx[o];
        a.dout[o] = dout[o];
        a.dw[o] = dw[o];
        a.width[o] = width[o];
    }
    a.bank = bank;
    a.scales = scales;
    a.n_slots = n_slots;
    a.hd = hd;
    a.group = plain ? 32 : group;
    a.n_ops = n_ops;
    a.idx64 = idx_dtype == SDM_I64;
    a.w_bf16 = dw_dtype == SDM_BF16;
    a.tokens = tokens;
    a.chunk = chunk;
    a.valid = valid;
    a.chunk_valid = chunk_valid;
    return sdm::launch_gather_dw(a, format, reinterpret_cast<cudaStream_t>(stream));
}

int sdm_qdecode_seq(void* codes, float* scales, int64_t n_slots, const void* k_idx, const float* k_val,
                    const float* v, const float* beta, const float* g, const void* q_idx, const float* q_val,
                    void* out, int64_t n_streams, int hd, int group, int format, int W, int R, int G, int T,
                    int idx_dtype, int out_dtype, unsigned flags, sdm_stream_t stream) {
    if (flags & ~SDM_STREAM_MAJOR) return SDM_EFLAGS;
    if (format == SDM_INT4) return SDM_EFORMAT;
    const int rc = check_bank(n_slots, hd, group, format);
    if (rc != SDM_OK) return rc;
    if (!float_type(out_dtype)) return SDM_EDTYPE;
    if (!index_type(idx_dtype)) return SDM_EIDX;
    if (W < 1 || W > 256 || R < 1 || R > 256) return SDM_EWIDTH;
    if (G != 1 && G != W) return SDM_EGATES;
    if (n_streams < 0 || T < 0 || n_streams > (int64_t)INT_MAX) return SDM_ECOUNT;
    if (n_streams == 0 || T == 0) return SDM_OK;
    if (!codes || !scales || !k_idx || !k_val || !v || !beta || !g || !q_idx || !q_val || !out) return SDM_ENULL;
    const size_t is = index_size(idx_dtype);
    if (!aligned(codes, 16) || !aligned(scales, 4) || !aligned(out, float_size(out_dtype)) || !aligned(k_idx, is) ||
        !aligned(q_idx, is) || !aligned(k_val, 4) || !aligned(v, 4) || !aligned(beta, 4) || !aligned(g, 4) ||
        !aligned(q_val, 4))
        return SDM_EALIGN;
    const int64_t tokens = n_streams * T;
    if (tokens > (int64_t)1 << 40) return SDM_ECOUNT;
    const Rows c = array(codes, n_slots, sdm_quant_row_bytes(hd, format), 1), sc = array(scales, n_slots, (hd + group - 1) / group, 4);
    const Rows o = array(out, tokens, hd, float_size(out_dtype));
    for (const Rows& in : {array(k_idx, tokens, W, is), array(q_idx, tokens, R, is), array(k_val, tokens, W, 4), array(q_val, tokens, R, 4),
                           array(v, tokens, hd, 4), array(beta, tokens, 1, 4), array(g, tokens, G, 4)}) {
        // a column of v has been read when its reading is written, so float32 readings may take its place
        if (overlaps(in, c) || overlaps(in, sc) || (overlaps(in, o) && !(in.p == v && out == v && out_dtype == SDM_F32))) return SDM_EOVERLAP;
    }
    if (overlaps(c, sc) || overlaps(o, c) || overlaps(o, sc)) return SDM_EOVERLAP;
    sdm::QDecodeArgs a{};
    a.codes = static_cast<uint8_t*>(codes);
    a.scales = scales;
    a.n_slots = n_slots;
    a.k_idx = k_idx;
    a.k_val = k_val;
    a.v = v;
    a.beta = beta;
    a.g = g;
    a.q_idx = q_idx;
    a.q_val = q_val;
    a.out = out;
    a.n_streams = n_streams;
    a.hd = hd;
    a.group = group;
    a.W = W;
    a.R = R;
    a.G = G;
    a.T = T;
    a.idx64 = idx_dtype == SDM_I64;
    a.out_bf16 = out_dtype == SDM_BF16;
    a.tstride = flags & SDM_STREAM_MAJOR ? 1 : n_streams;
    a.sstride = flags & SDM_STREAM_MAJOR ? T : 1;
    return sdm::launch_qdecode(a, format, reinterpret_cast<cudaStream_t>(stream));
}

int sdm_qdecode_step(void* codes, float* scales, int64_t n_slots, const void* k_idx, const float* k_val,
                     const float* v, const float* beta, const float* g, const void* q_idx, const float* q_val,
                     void* out, int64_t n_streams, int hd, int group, int format, int W, int R, int G, int idx_dtype,
                     int out_dtype, sdm_stream_t stream) {
    return sdm_qdecode_seq(codes, scales, n_slots, k_idx, k_val, v, beta, g, q_idx, q_val, out, n_streams, hd, group,
                           format, W, R, G, 1, idx_dtype, out_dtype, 0u, stream);
}

// Shared checks of the two directions; which of them applies is said by the pointers.
static int check_route(const void* logits, int64_t row_stride, int logit_dtype, const void* base, const void* idx,
                       int64_t tokens, int n, int k, int score, unsigned flags, int idx_dtype) {
    if (flags & ~SDM_RENORM) return SDM_EFLAGS;
    if (!float_type(logit_dtype)) return SDM_EDTYPE;
    if (!index_type(idx_dtype)) return SDM_EIDX;
    if (n < 1 || n > 65536 || k < 1 || k > 256 || k > n || (score != SDM_SOFTMAX && score != SDM_SIGMOID))
        return SDM_EROUTE;
    if (tokens < 0 || tokens > (int64_t)1 << 40) return SDM_ECOUNT;
    if (tokens == 0) return SDM_OK;
    if (!logits || !idx) return SDM_ENULL;
    if (row_stride < n) return SDM_ESTRIDE;
    if (!aligned(logits, float_size(logit_dtype)) || !aligned(idx, index_size(idx_dtype)) ||
        !aligned(base, index_size(idx_dtype)))
        return SDM_EALIGN;
    return SDM_OK;
}

int sdm_route(const void* logits, int64_t row_stride, int logit_dtype, const float* bias, const void* base, void* idx,
              float* w, int64_t tokens, int n, int k, int score, int n_groups, int top_groups, int group_top,
              float scale, unsigned flags, int idx_dtype, sdm_stream_t stream) {
    const int rc = check_route(logits, row_stride, logit_dtype, base, idx, tokens, n, k, score, flags, idx_dtype);
    if (rc != SDM_OK) return rc;
    if (n_groups < 1 || n_groups > 256 || n % n_groups != 0 || top_groups < 1 || top_groups > n_groups ||
        (group_top != 1 && group_top != 2))
        return SDM_EROUTE;
    if (tokens == 0) return SDM_OK;
    if (!w) return SDM_ENULL;
    if (!aligned(w, 4) || !aligned(bias, 4)) return SDM_EALIGN;
    const Rows oi = array(idx, tokens, k, index_size(idx_dtype)), ow = array(w, tokens, k, 4);
    for (const Rows& in : {Rows{logits, tokens, row_stride, n, float_size(logit_dtype)}, array(bias, 1, n, 4),
                           array(base, tokens, 1, index_size(idx_dtype))})
        if (overlaps(in, oi) || overlaps(in, ow)) return SDM_EOVERLAP;
    if (overlaps(oi, ow)) return SDM_EOVERLAP;
    sdm::RouteArgs a{};
    a.logits = logits;
    a.row_stride = row_stride;
    a.bias = bias;
    a.base = base;
    a.idx = idx;
    a.w = w;
    a.tokens = tokens;
    a.n = n;
    a.k = k;
    a.score = score;
    a.n_groups = n_groups;
    a.top_groups = top_groups;
    a.group_top = group_top;
    a.scale = scale;
    a.renorm = (flags & SDM_RENORM) != 0;
    a.idx64 = idx_dtype == SDM_I64;
    a.logit_bf16 = logit_dtype == SDM_BF16;
    return sdm::launch_route(a, reinterpret_cast<cudaStream_t>(stream));
}

int sdm_route_backward_ex(const void* logits, int64_t row_stride, int logit_dtype, const void* base, const void* idx,
                          const float* w, const float* dw, void* dlogits, int64_t dlogits_stride, int64_t tokens, int n,
                          int k, int score, float scale, unsigned flags, int idx_dtype, sdm_stream_t stream) {
    const int rc = check_route(logits, row_stride, logit_dtype, base, idx, tokens, n, k, score, flags, idx_dtype);
    if (rc != SDM_OK || tokens == 0) return rc;
    if (!dw || !dlogits) return SDM_ENULL;
    if (dlogits_stride < n) return SDM_ESTRIDE;
    if (!aligned(w, 4) || !aligned(dw, 4) || !aligned(dlogits, float_size(logit_dtype))) return SDM_EALIGN;
    const size_t es = float_size(logit_dtype), is = index_size(idx_dtype);
    const Rows out{dlogits, tokens, dlogits_stride, n, es};
    for (const Rows& in : {Rows{logits, tokens, row_stride, n, es}, array(idx, tokens, k, is), array(base, tokens, 1, is),
                           array(w, tokens, k, 4), array(dw, tokens, k, 4)})
        if (overlaps(in, out)) return SDM_EOVERLAP;
    sdm::RouteArgs a{};
    a.logits = logits;
    a.row_stride = row_stride;
    a.base = base;
    a.idx = const_cast<void*>(idx);
    a.tokens = tokens;
    a.n = n;
    a.k = k;
    a.score = score;
    a.scale = scale;
    a.renorm = (flags & SDM_RENORM) != 0;
    a.idx64 = idx_dtype == SDM_I64;
    a.logit_bf16 = logit_dtype == SDM_BF16;
    a.w = const_cast<float*>(w);
    a.dw = dw;
    a.dlogits = dlogits;
    a.dlogits_stride = dlogits_stride;
    return sdm::launch_route_backward(a, reinterpret_cast<cudaStream_t>(stream));
}

int sdm_route_backward(const void* logits, int64_t row_stride, int logit_dtype, const void* base, const void* idx,
                       const float* dw, void* dlogits, int64_t dlogits_stride, int64_t tokens, int n, int k, int score,
                       float scale, unsigned flags, int idx_dtype, sdm_stream_t stream) {
    return sdm_route_backward_ex(logits, row_stride, logit_dtype, base, idx, nullptr, dw, dlogits, dlogits_stride, tokens,
                                 n, k, score, scale, flags, idx_dtype, stream);
}

}  // extern "C"
