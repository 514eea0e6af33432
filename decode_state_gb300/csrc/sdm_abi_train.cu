// C ABI of the balance loss, the embedding lookup and the gradients of rows: argument validation (host only,
// before any CUDA call) and dispatch to the kernel files.
#include <climits>

#include "sdm.h"
#include "sdm_checks.h"
#include "sdm_internal.h"

namespace {

using namespace sdm::checks;

constexpr int64_t kMostSequences = (int64_t)1 << 24;

// An array as Rows; one without elements overlaps nothing.
Rows any(const void* p, int64_t n, int64_t per, size_t es) { return array(n * per == 0 ? nullptr : p, n, per, es); }

int check_sums(int64_t entries, int64_t n_slots, int hd) {
    if (hd < 1 || hd > 65536) return SDM_EHD;
    if (n_slots < 1 || n_slots > (int64_t)INT_MAX || entries < 0 || entries > (int64_t)INT_MAX) return SDM_ECOUNT;
    return SDM_OK;
}

int check_workspace(const void* workspace, int64_t bytes, int64_t need) {
    if (need == 0) return SDM_OK;
    if (!workspace) return SDM_ENULL;
    if (!aligned(workspace, 256)) return SDM_EALIGN;
    return bytes < need ? SDM_EWORKSPACE : SDM_OK;
}

int sums_workspace(int64_t entries, int64_t n_slots, int hd, int64_t* bytes) {
    if (!bytes) return SDM_ENULL;
    const int rc = check_sums(entries, n_slots, hd);
    *bytes = rc == SDM_OK ? sdm::row_sums_workspace(entries, n_slots, hd) : 0;
    return rc;
}

}  // namespace

extern "C" {

int sdm_balance_workspace(int64_t sequences, int64_t* bytes) {
    if (!bytes) return SDM_ENULL;
    *bytes = 0;
    if (sequences < 0 || sequences >= kMostSequences) return SDM_ECOUNT;
    *bytes = sdm::balance_workspace(sequences);
    return SDM_OK;
}

int sdm_balance(const void* logits, int64_t row_stride, int logit_dtype, const void* base, const void* idx, const float* w,
                const int32_t* offsets, int64_t sequences, float* loss, int32_t* counts, const float* dloss,
                const void* add, int64_t add_stride, void* dlogits, int64_t dlogits_stride, int64_t tokens, int n, int k,
                int score, float scale, int idx_dtype, void* workspace, int64_t workspace_bytes, sdm_stream_t stream) {
    if (!float_type(logit_dtype)) return SDM_EDTYPE;
    if (!index_type(idx_dtype)) return SDM_EIDX;
    if (n < 1 || n > 65536 || k < 1 || k > 256 || k > n || (score != SDM_SOFTMAX && score != SDM_SIGMOID)) return SDM_EROUTE;
    if (tokens < 0 || tokens > (int64_t)INT_MAX || tokens * k > (int64_t)INT_MAX || sequences < 0 || sequences >= kMostSequences ||
        (!offsets && sequences != 1))
        return SDM_ECOUNT;
    if (tokens == 0 && sequences == 0) return SDM_OK;
    if (sequences > 0 && (!loss || !counts)) return SDM_ENULL;
    if (tokens > 0 && (!logits || !idx)) return SDM_ENULL;
    if (!dlogits) {
        add = nullptr;
        dloss = nullptr;
    }
    if (tokens > 0 && (row_stride < n || (add && add_stride < n) || (dlogits && dlogits_stride < n))) return SDM_ESTRIDE;
    const size_t es = float_size(logit_dtype), is = index_size(idx_dtype);
    if (!aligned(logits, es) || !aligned(add, es) || !aligned(dlogits, es) || !aligned(idx, is) || !aligned(base, is) || !aligned(w, 4) ||
        !aligned(offsets, 4) || !aligned(loss, 4) || !aligned(counts, 4) || !aligned(dloss, 4))
        return SDM_EALIGN;
    const int64_t need = sdm::balance_workspace(sequences);
    const int rc = check_workspace(workspace, workspace_bytes, need);
    if (rc != SDM_OK) return rc;
    const Rows to{tokens == 0 ? nullptr : dlogits, tokens, dlogits_stride, n, es}, from{tokens == 0 ? nullptr : add, tokens, add_stride, n, es};
    const Rows outs[4] = {any(loss, sequences, 1, 4), any(counts, sequences, n, 4), to, array(workspace, need, 1, 1)};
    for (int o = 0; o < 4; ++o) {
        for (const Rows& in : {Rows{tokens == 0 ? nullptr : logits, tokens, row_stride, n, es}, any(idx, tokens, k, is), any(base, tokens, 1, is),
                               any(w, tokens, k, 4), array(offsets, sequences + 1, 1, 4), any(dloss, sequences, 1, 4)})
            if (overlaps(in, outs[o])) return SDM_EOVERLAP;
        // an element of add is read by the thread that writes its place
        if (overlaps(from, outs[o]) && !(o == 2 && add == dlogits && add_stride == dlogits_stride)) return SDM_EOVERLAP;
        for (int p = 0; p < o; ++p)
            if (overlaps(outs[p], outs[o])) return SDM_EOVERLAP;
    }
    sdm::BalanceArgs a{};
    a.logits = logits;
    a.row_stride = row_stride;
    a.base = base;
    a.idx = idx;
    a.w = w;
    a.offsets = offsets;
    a.sequences = static_cast<int>(sequences);
    a.loss = loss;
    a.counts = counts;
    a.dloss = dloss;
    a.add = add;
    a.add_stride = add_stride;
    a.dlogits = dlogits;
    a.dlogits_stride = dlogits_stride;
    a.tokens = static_cast<int>(tokens);
    a.n = n;
    a.k = k;
    a.score = score;
    a.scale = scale;
    a.idx64 = idx_dtype == SDM_I64;
    a.logit_bf16 = logit_dtype == SDM_BF16;
    a.workspace = workspace;
    return sdm::launch_balance(a, reinterpret_cast<cudaStream_t>(stream));
}

int sdm_lookup(const void* table, int64_t n_rows, int hd, int table_dtype, const void* tokens, int idx_dtype,
               int64_t n_tokens, int64_t padding, float scale, void* out, int out_dtype, sdm_stream_t stream) {
    if (!float_type(table_dtype) || !float_type(out_dtype)) return SDM_EDTYPE;
    if (!index_type(idx_dtype)) return SDM_EIDX;
    if (hd < 1 || hd > 65536) return SDM_EHD;
    if (n_rows < 1 || n_rows > (int64_t)INT_MAX || n_tokens < 0 || n_tokens > (int64_t)1 << 40) return SDM_ECOUNT;
    if (n_tokens == 0) return SDM_OK;
    if (!table || !tokens || !out) return SDM_ENULL;
    if (!aligned(table, float_size(table_dtype)) || !aligned(tokens, index_size(idx_dtype)) || !aligned(out, float_size(out_dtype)))
        return SDM_EALIGN;
    const Rows to = array(out, n_tokens, hd, float_size(out_dtype));
    if (overlaps(array(table, n_rows, hd, float_size(table_dtype)), to) || overlaps(array(tokens, n_tokens, 1, index_size(idx_dtype)), to))
        return SDM_EOVERLAP;
    sdm::LookupArgs a{};
    a.table = table;
    a.n_rows = n_rows;
    a.tokens = tokens;
    a.n_tokens = n_tokens;
    a.padding = padding;
    a.out = out;
    a.hd = hd;
    a.scale = scale;
    a.table_bf16 = table_dtype == SDM_BF16;
    a.out_bf16 = out_dtype == SDM_BF16;
    a.idx64 = idx_dtype == SDM_I64;
    return sdm::launch_lookup(a, reinterpret_cast<cudaStream_t>(stream));
}

int sdm_lookup_backward_workspace(int64_t n_tokens, int64_t n_rows, int hd, int64_t* bytes) {
    return sums_workspace(n_tokens, n_rows, hd, bytes);
}

int sdm_lookup_backward(const void* dout, int dout_dtype, const void* tokens, int idx_dtype, int64_t n_tokens,
                        int64_t padding, float scale, void* grad, int64_t n_rows, int hd, int grad_dtype, unsigned flags,
                        void* workspace, int64_t workspace_bytes, sdm_stream_t stream) {
    if (flags & ~SDM_ACCUMULATE) return SDM_EFLAGS;
    if (!float_type(dout_dtype) || !float_type(grad_dtype)) return SDM_EDTYPE;
    if (!index_type(idx_dtype)) return SDM_EIDX;
    int rc = check_sums(n_tokens, n_rows, hd);
    if (rc != SDM_OK) return rc;
    if (n_tokens == 0 && (flags & SDM_ACCUMULATE)) return SDM_OK;
    if (!grad || (n_tokens > 0 && (!dout || !tokens))) return SDM_ENULL;
    const size_t ds = float_size(dout_dtype), is = index_size(idx_dtype), gs = float_size(grad_dtype);
    if (!aligned(dout, ds) || !aligned(tokens, is) || !aligned(grad, gs)) return SDM_EALIGN;
    const int64_t need = sdm::row_sums_workspace(n_tokens, n_rows, hd);
    rc = check_workspace(workspace, workspace_bytes, need);
    if (rc != SDM_OK) return rc;
    const Rows out = array(grad, n_rows, hd, gs), scratch = any(workspace, need, 1, 1);
    for (const Rows& in : {any(dout, n_tokens, hd, ds), any(tokens, n_tokens, 1, is)})
        if (overlaps(in, out) || overlaps(in, scratch)) return SDM_EOVERLAP;
    if (overlaps(out, scratch)) return SDM_EOVERLAP;
    sdm::RowSumArgs a{};
    a.n_ops = 1;
    a.idx[0] = tokens;
    a.dout[0] = dout;
    a.width[0] = a.width[1] = 1;
    a.idx64 = idx_dtype == SDM_I64;
    a.dout_bf16 = dout_dtype == SDM_BF16;
    a.out_bf16 = grad_dtype == SDM_BF16;
    a.accumulate = (flags & SDM_ACCUMULATE) != 0;
    a.tokens = n_tokens;
    a.chunk = a.valid = 1;
    a.padding = padding;
    a.n_slots = n_rows;
    a.hd = hd;
    a.scale = scale;
    a.out = grad;
    a.workspace = workspace;
    a.entries = a.split = (uint32_t)n_tokens;
    return sdm::launch_row_sums(a, reinterpret_cast<cudaStream_t>(stream));
}

int sdm_gather_drows_workspace(int64_t entries, int64_t n_slots, int hd, int64_t* bytes) {
    return sums_workspace(entries, n_slots, hd, bytes);
}

int sdm_gather_drows(int n_ops, const void* const idx[2], const void* const w[2], const float* const dout[2],
                     const int width[2], int idx_dtype, int w_dtype, void* drows, int64_t n_slots, int hd, int drows_dtype,
                     unsigned flags, int64_t tokens, int chunk, int valid, const int32_t* chunk_valid, void* workspace,
                     int64_t workspace_bytes, sdm_stream_t stream) {
    if (flags & ~SDM_ACCUMULATE) return SDM_EFLAGS;
    if (!float_type(w_dtype) || !float_type(drows_dtype)) return SDM_EDTYPE;
    if (!index_type(idx_dtype)) return SDM_EIDX;
    if (n_ops != 1 && n_ops != 2) return SDM_ENOPS;
    if (!idx || !w || !dout || !width) return SDM_ENULL;
    for (int o = 0; o < n_ops; ++o)
        if (width[o] < 1 || width[o] > 256) return SDM_EWIDTH;
    if (tokens < 0 || tokens > (int64_t)INT_MAX) return SDM_ECOUNT;
    const int64_t entries = tokens * (width[0] + (n_ops == 2 ? width[1] : 0));
    int rc = check_sums(entries, n_slots, hd);
    if (rc != SDM_OK) return rc;
    if (chunk < 1 || tokens % chunk != 0 || (!chunk_valid && (valid < 0 || valid > chunk))) return SDM_ECHUNK;
    if (tokens == 0 && (flags & SDM_ACCUMULATE)) return SDM_OK;
    if (!drows) return SDM_ENULL;
    const size_t is = index_size(idx_dtype), ws = float_size(w_dtype), rs = float_size(drows_dtype);
    if (!aligned(drows, rs) || !aligned(chunk_valid, 4)) return SDM_EALIGN;
    const int64_t need = sdm::row_sums_workspace(entries, n_slots, hd);
    rc = check_workspace(workspace, workspace_bytes, need);
    if (rc != SDM_OK) return rc;
    const Rows out = array(drows, n_slots, hd, rs), scratch = any(workspace, need, 1, 1);
    if (overlaps(out, scratch)) return SDM_EOVERLAP;
    const Rows cv = any(chunk_valid, tokens / chunk, 1, 4);
    if (overlaps(cv, out) || overlaps(cv, scratch)) return SDM_EOVERLAP;
    sdm::RowSumArgs a{};
    for (int o = 0; o < n_ops; ++o) {
        if (tokens > 0 && (!idx[o] || !w[o] || !dout[o])) return SDM_ENULL;
        if (!aligned(idx[o], is) || !aligned(w[o], ws) || !aligned(dout[o], 4)) return SDM_EALIGN;
        for (const Rows& in : {any(idx[o], tokens, width[o], is), any(w[o], tokens, width[o], ws), any(dout[o], tokens, hd, 4)})
            if (overlaps(in, out) || overlaps(in, scratch)) return SDM_EOVERLAP;
        a.idx[o] = idx[o];
        a.w[o] = w[o];
        a.dout[o] = dout[o];
        a.width[o] = width[o];
    }
    if (n_ops == 1) a.width[1] = 1;
    a.n_ops = n_ops;
    a.idx64 = idx_dtype == SDM_I64;
    a.w_bf16 = w_dtype == SDM_BF16;
    a.out_bf16 = drows_dtype == SDM_BF16;
    a.accumulate = (flags & SDM_ACCUMULATE) != 0;
    a.tokens = tokens;
    a.chunk = chunk;
    a.valid = valid;
    a.chunk_valid = chunk_valid;
    a.padding = SDM_NO_PADDING;
    a.n_slots = n_slots;
    a.hd = hd;
    a.scale = 1.0f;
    a.out = drows;
    a.workspace = workspace;
    a.entries = (uint32_t)entries;
    a.split = (uint32_t)(tokens * width[0]);
    return sdm::launch_row_sums(a, reinterpret_cast<cudaStream_t>(stream));
}

}  // extern "C"
