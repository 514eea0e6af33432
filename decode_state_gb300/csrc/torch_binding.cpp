// Python functions over the C ABI of the quantised banks, the routing and their training, for PyTorch tensors.
//
// Marshalling only: shapes, types and devices are checked, outputs allocated and pointers passed to
// the entry points of include/sdm.h, which do the rest. These operators are called once a token, and
// their checks take longer in Python than their kernels run: a decode step of 64 streams and the
// read-back of the rows it wrote took 59 us a call through ctypes wrappers, most of it in the checks.
// Shape errors raise ValueError, types TypeError, and status codes of the library SDMError.
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>
#include <torch/csrc/utils/object_ptr.h>

#include <climits>
#include <optional>
#include <vector>

#include "sdm.h"

namespace {

using at::Tensor;

PyObject* g_raise_status = nullptr;  // raises SDMError(function, status)

struct Args {
    PyObject* const* a;
    Py_ssize_t n;

    bool none(int i) const { return a[i] == Py_None; }
    const Tensor& tensor(int i, const char* name) const { return unpack(a[i], name); }
    int64_t integer(int i) const {
        const long long v = PyLong_AsLongLong(a[i]);
        if (v == -1 && PyErr_Occurred()) throw python_error();
        return v;
    }
    int small(int i) const {
        const int64_t v = integer(i);
        // out of range for an int: a value that no entry point takes either
        return v < INT_MIN || v > INT_MAX ? INT_MIN : static_cast<int>(v);
    }
    bool truth(int i) const {
        const int v = PyObject_IsTrue(a[i]);
        if (v < 0) throw python_error();
        return v != 0;
    }
    float real(int i) const {
        const double v = PyFloat_AsDouble(a[i]);
        if (v == -1.0 && PyErr_Occurred()) throw python_error();
        return static_cast<float>(v);
    }
    at::ScalarType dtype(int i, const char* name) const {
        TORCH_CHECK_TYPE(THPDtype_Check(a[i]), name, " must be a torch.dtype");
        return reinterpret_cast<THPDtype*>(a[i])->scalar_type;
    }

    static const Tensor& unpack(PyObject* o, const char* name) {
        TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a torch.Tensor");
        return THPVariable_Unpack(o);
    }
};

void expect(const Args& a, Py_ssize_t n, const char* fn) {
    TORCH_CHECK_TYPE(a.n == n, fn, " takes ", n, " arguments, got ", a.n);
}

THPObjectPtr attribute(PyObject* o, PyObject* name) {
    THPObjectPtr v(PyObject_GetAttr(o, name));
    if (!v) throw python_error();
    return v;
}

int64_t attribute_int(PyObject* o, PyObject* name) {
    THPObjectPtr p = attribute(o, name);
    const long long v = PyLong_AsLongLong(p.get());
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}

int float_code(at::ScalarType t, const char* name) {
    TORCH_CHECK_TYPE(t == at::kBFloat16 || t == at::kFloat, name, " must be bfloat16 or float32, got ", t);
    return t == at::kBFloat16 ? SDM_BF16 : SDM_F32;
}

int index_code(at::ScalarType t, const char* name) {
    TORCH_CHECK_TYPE(t == at::kInt || t == at::kLong, name, " must be int32 or int64, got ", t);
    return t == at::kLong ? SDM_I64 : SDM_I32;
}

void need_device(const Tensor& t, const char* name, const at::Device& dev) {
    TORCH_CHECK_VALUE(t.is_cuda() && t.device() == dev, name, " must be a CUDA tensor on ", dev, ", got ", t.device());
}

void need(const Tensor& t, const char* name, const at::Device& dev, at::IntArrayRef shape) {
    need_device(t, name, dev);
    TORCH_CHECK_VALUE(t.sizes() == shape, name, " has shape ", t.sizes(), ", expected ", shape);
    TORCH_CHECK_VALUE(t.is_contiguous(), name, " must be contiguous");
}

void need_f32(const Tensor& t, const char* name, const at::Device& dev, at::IntArrayRef shape) {
    TORCH_CHECK_TYPE(t.scalar_type() == at::kFloat, name, " must be float32, got ", t.scalar_type());
    need(t, name, dev, shape);
}

void check_cuda(cudaError_t e) {
    if (e == cudaSuccess) return;
    (void)cudaGetLastError();
    TORCH_CHECK(false, "CUDA error: ", cudaGetErrorString(e));
}

// The thread's stream waits for the work of the current one, `current`. The legacy default stream has this from itself. Where
// one of the two is being captured and the other is not, or in another graph, no event joins them.
void thread_stream_waits(cudaStream_t current) {
    if (current == nullptr || current == cudaStreamLegacy || current == cudaStreamPerThread) return;
    cudaStreamCaptureStatus status[2];
    unsigned long long graph[2] = {0, 0};
    check_cuda(cudaStreamGetCaptureInfo(current, &status[0], &graph[0]));
    check_cuda(cudaStreamGetCaptureInfo(cudaStreamPerThread, &status[1], &graph[1]));
    if (status[0] != status[1] || (status[0] != cudaStreamCaptureStatusNone && graph[0] != graph[1])) return;
    cudaEvent_t event = nullptr;
    check_cuda(cudaEventCreateWithFlags(&event, cudaEventDisableTiming));
    cudaError_t e = cudaEventRecord(event, current);
    if (e == cudaSuccess) e = cudaStreamWaitEvent(cudaStreamPerThread, event, 0);
    (void)cudaEventDestroy(event);  // when it has been reached
    check_cuda(e);
}

// The device of the work made current, and the stream it goes to. Outputs and workspaces made while a given stream is
// current come from that stream's memory: what else is free may still be in use by the current stream,
// whose work the given one does not wait for. The stream of the thread (handle 2) is another one in each thread, and has no
// memory of its own: it waits for the current stream, whose memory it takes, and what it took is not given to others before
// it is done with it.
struct Launch {
    c10::cuda::OptionalCUDAGuard guard;
    c10::cuda::OptionalCUDAStreamGuard stream_guard;
    sdm_stream_t stream;

    Launch(const at::Device& dev, PyObject* s) {
        if (c10::cuda::current_device() != dev.index()) guard.set_device(dev);
        if (s == Py_None) {
            stream = reinterpret_cast<sdm_stream_t>(c10::cuda::getCurrentCUDAStream(dev.index()).stream());
            return;
        }
        static PyObject* name = PyUnicode_InternFromString("cuda_stream");
        THPObjectPtr handle = PyLong_Check(s) ? THPObjectPtr(Py_NewRef(s)) : attribute(s, name);
        stream = static_cast<sdm_stream_t>(PyLong_AsVoidPtr(handle.get()));
        if (stream == nullptr && PyErr_Occurred()) throw python_error();
        // the handles 1 (the legacy default stream) and 2 (a thread's) are names, not streams of their own
        const cudaStream_t own = stream == reinterpret_cast<sdm_stream_t>(cudaStreamLegacy) ? nullptr : reinterpret_cast<cudaStream_t>(stream);
        per_thread = own == cudaStreamPerThread;
        if (!per_thread) stream_guard.reset_stream(c10::cuda::getStreamFromExternal(own, dev.index()));
    }

    bool per_thread = false;
    mutable bool waits = false;  // the thread's stream, for the current one

    Tensor empty(at::IntArrayRef shape, at::ScalarType t, const at::Device& dev) const {
        Tensor made(at::detail::empty_cuda(shape, t, dev, std::nullopt));
        if (per_thread && made.numel() > 0) {
            if (!waits) thread_stream_waits(c10::cuda::getCurrentCUDAStream(dev.index()).stream());
            waits = true;
            c10::cuda::CUDACachingAllocator::recordStream(made.storage().data_ptr(), c10::cuda::getStreamFromExternal(cudaStreamPerThread, dev.index()));
        }
        return made;
    }

    // Memory for the call to work in, given back when the caller lets go of it: free for what the stream does next.
    Tensor workspace(int64_t bytes, const at::Device& dev) const { return empty({bytes}, at::kByte, dev); }
};

// Raise SDMError for a status that is not 0.
void check(const char* fn, int status) {
    if (status == SDM_OK) return;
    PyObject* r = g_raise_status ? PyObject_CallFunction(g_raise_status, "si", fn, status) : nullptr;
    Py_XDECREF(r);
    if (!PyErr_Occurred()) PyErr_Format(PyExc_RuntimeError, "%s failed with status %d", fn, status);
    throw python_error();
}

PyObject* give(PyObject* given, const Tensor& made) {
    if (given == Py_None) return THPVariable_Wrap(made);
    Py_INCREF(given);
    return given;
}

// ---------------------------------------------------------------- quantised banks

struct Bank {
    void* codes = nullptr;
    float* scales = nullptr;
    int64_t n_slots = 0;
    int hd = 0, group = 0, format = 0;
    at::Device dev{at::kCPU};

    // a quant.QuantBank: codes, scales, hd, group and the format's code
    explicit Bank(PyObject* o) {
        static PyObject *n_codes = PyUnicode_InternFromString("codes"), *n_scales = PyUnicode_InternFromString("scales"),
                        *n_hd = PyUnicode_InternFromString("hd"), *n_group = PyUnicode_InternFromString("group"),
                        *n_format = PyUnicode_InternFromString("_code");
        THPObjectPtr po = attribute(o, n_codes), ps = attribute(o, n_scales);
        const Tensor& c = Args::unpack(po.get(), "codes");
        const Tensor& s = Args::unpack(ps.get(), "scales");
        hd = static_cast<int>(attribute_int(o, n_hd));
        group = static_cast<int>(attribute_int(o, n_group));
        format = static_cast<int>(attribute_int(o, n_format));
        TORCH_CHECK_TYPE(c.scalar_type() == at::kByte && s.scalar_type() == at::kFloat, "codes must be uint8 and scales float32, got ",
                         c.scalar_type(), ", ", s.scalar_type());
        const int row = sdm_quant_row_bytes(hd, format);
        TORCH_CHECK_VALUE(row > 0 && group > 0, "no such bank: hd ", hd, ", group ", group);
        n_slots = c.dim() == 2 ? c.size(0) : 0;
        dev = c.device();
        TORCH_CHECK_VALUE(c.is_cuda(), "codes must be a CUDA tensor, got ", dev);
        need(c, "codes", dev, {n_slots, row});
        need(s, "scales", dev, {n_slots, (hd + group - 1) / group});
        codes = c.data_ptr();
        scales = static_cast<float*>(s.data_ptr());
    }

    // a plain [n_slots, hd] bank, or a table of rows
    explicit Bank(const Tensor& t, const char* name = "bank") {
        format = float_code(t.scalar_type(), name);
        TORCH_CHECK_TYPE(t.dim() == 2, name, name[0] == 'b' ? " must be a QuantBank or a [n_slots, head_dim] bfloat16 or float32 tensor"
                                                            : " must be a [rows, hd] bfloat16 or float32 tensor");
        TORCH_CHECK_VALUE(t.size(1) >= 1 && t.size(1) <= 65536, "head_dim must be in 1..65536, got ", t.size(1));
        n_slots = t.size(0);
        hd = static_cast<int>(t.size(1));
        dev = t.device();
        TORCH_CHECK_VALUE(t.is_cuda(), name, " must be a CUDA tensor, got ", dev);
        need(t, name, dev, t.sizes());
        codes = t.data_ptr();
    }
};

// check_bank(bank)
PyObject* check_bank(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const Args a{args, n};
    expect(a, 1, "check_bank");
    Bank b(a.a[0]);
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// room(rows, columns, dtype, stream): an uninitialised [len(rows), columns] on the device of `rows`, for the stream to write
PyObject* room(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const Args a{args, n};
    expect(a, 4, "room");
    const Tensor& r = a.tensor(0, "rows");
    TORCH_CHECK_VALUE(r.is_cuda(), "rows must be a CUDA tensor, got ", r.device());
    Launch l(r.device(), a.a[3]);
    return THPVariable_Wrap(l.empty({r.size(0), a.integer(1)}, a.dtype(2, "dtype"), r.device()));
    END_HANDLE_TH_ERRORS
}

// rows(write, bank, rows or None, slots or None, dtype, stream): rows into the bank, or out of it
PyObject* rows(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const Args a{args, n};
    expect(a, 6, "rows");
    const bool write = a.truth(0);
    const Bank b(a.a[1]);
    const char* name = write ? "rows" : "out";
    const void* slot_ptr = nullptr;
    int it = SDM_I32;
    int64_t count = -1;
    if (!a.none(3)) {
        const Tensor& s = a.tensor(3, "slots");
        it = index_code(s.scalar_type(), "slots");
        count = s.numel();
        need(s, "slots", b.dev, {count});
        slot_ptr = s.data_ptr();
    }
    Launch l(b.dev, a.a[5]);
    Tensor made;
    if (a.none(2)) {
        const auto t = a.dtype(4, "dtype");
        float_code(t, "dtype");
        made = l.empty({count < 0 ? b.n_slots : count, b.hd}, t, b.dev);
    }
    const Tensor& r = a.none(2) ? made : a.tensor(2, name);
    const int rt = float_code(r.scalar_type(), name);
    TORCH_CHECK_VALUE(r.dim() == 2 && r.size(1) == b.hd, name, " must be [n, ", b.hd, "], got ", r.sizes());
    need_device(r, name, b.dev);
    const int64_t m = r.size(0);
    TORCH_CHECK_VALUE(count < 0 || count == m, "slots has shape [", count, "], expected [", m, "]");
    TORCH_CHECK_VALUE(count >= 0 || m <= b.n_slots, m, " rows do not fit a bank of ", b.n_slots, " slots");
    TORCH_CHECK_VALUE((b.hd == 1 || r.stride(1) == 1) && (m <= 1 || r.stride(0) >= b.hd), name,
                      " must have contiguous columns and rows that do not overlap");
    const int64_t stride = m <= 1 ? b.hd : r.stride(0);
    if (write)
        check("sdm_quantize_rows", sdm_quantize_rows(b.codes, b.scales, b.n_slots, b.hd, b.group, b.format, r.data_ptr(), stride, rt,
                                                     slot_ptr, it, m, l.stream));
    else
        check("sdm_dequantize_rows", sdm_dequantize_rows(b.codes, b.scales, b.n_slots, b.hd, b.group, b.format, r.data_ptr(), stride,
                                                         rt, slot_ptr, it, m, l.stream));
    return give(write ? a.a[1] : a.a[2], made);
    END_HANDLE_TH_ERRORS
}

// gather(bank, ops, chunk, valid or None, chunk_valid or None, dtype, outs or None, stream, gradient):
// weighted sums, or with `gradient` the gradient of the weights (bank: a QuantBank or a tensor)
PyObject* gather(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const Args a{args, n};
    expect(a, 9, "gather");
    const bool grad = a.truth(8);
    const Bank b = THPVariable_Check(a.a[0]) ? Bank(THPVariable_Unpack(a.a[0])) : Bank(a.a[0]);
    TORCH_CHECK_TYPE(grad || b.scales != nullptr, "bank must be a QuantBank (sdm.gather takes tensors)");
    const auto sequence = [](PyObject* o, const char* what) {
        TORCH_CHECK_TYPE(PyList_Check(o) || PyTuple_Check(o), what, " must be a list or tuple");
        return o;
    };
    PyObject* ops = sequence(a.a[1], "ops");
    const Py_ssize_t k = PySequence_Fast_GET_SIZE(ops);
    TORCH_CHECK_VALUE(k == 1 || k == 2, "gather takes one or two operands");
    PyObject* given = a.none(6) ? nullptr : sequence(a.a[6], "outputs");
    TORCH_CHECK_VALUE(!given || PySequence_Fast_GET_SIZE(given) == k, "there must be an output for each operand");
    const char *second = grad ? "dout" : "w", *third = grad ? "dw" : "out";

    const void* idx[2] = {nullptr, nullptr};
    const void* in[2] = {nullptr, nullptr};
    void* out[2] = {nullptr, nullptr};
    int width[2] = {0, 0}, it = SDM_I32, wt = SDM_F32;
    int64_t tokens = 0;
    Tensor made[2];
    Launch l(b.dev, a.a[7]);
    for (Py_ssize_t o = 0; o < k; ++o) {
        PyObject* pair = sequence(PySequence_Fast_GET_ITEM(ops, o), "an operand");
        TORCH_CHECK_VALUE(PySequence_Fast_GET_SIZE(pair) == 2, "an operand is a pair of tensors");
        const Tensor& i = Args::unpack(PySequence_Fast_GET_ITEM(pair, 0), "idx");
        const Tensor& x = Args::unpack(PySequence_Fast_GET_ITEM(pair, 1), second);
        const int t = index_code(i.scalar_type(), "idx");
        TORCH_CHECK_VALUE(i.dim() == 2, "idx must be [tokens, width]");
        if (o == 0) {
            tokens = i.size(0);
            it = t;
        }
        TORCH_CHECK_TYPE(t == it, "both operands must share the index dtype");
        need(i, "idx", b.dev, {tokens, i.size(1)});
        if (grad) {
            need_f32(x, second, b.dev, {tokens, b.hd});
        } else {
            const int xt = float_code(x.scalar_type(), "weights");
            if (o == 0) wt = xt;
            TORCH_CHECK_TYPE(xt == wt, "both operands must share the dtype of w");
            need(x, second, b.dev, i.sizes());
        }
        const int64_t cols = grad ? i.size(1) : b.hd;
        if (!given) made[o] = l.empty({tokens, cols}, grad ? a.dtype(5, "dtype") : at::kFloat, b.dev);
        const Tensor& r = given ? Args::unpack(PySequence_Fast_GET_ITEM(given, o), third) : made[o];
        if (grad) {
            const int rt = float_code(r.scalar_type(), "the gradients");
            if (o == 0) wt = rt;
            TORCH_CHECK_TYPE(rt == wt, "both gradients must share a dtype");
            need(r, third, b.dev, {tokens, cols});
        } else {
            need_f32(r, third, b.dev, {tokens, cols});
        }
        idx[o] = i.data_ptr();
        in[o] = x.data_ptr();
        out[o] = r.data_ptr();
        width[o] = i.size(1) > 256 ? 257 : static_cast<int>(i.size(1));
    }
    const int chunk = a.small(2);
    int valid = a.none(3) ? chunk : a.small(3);
    const int32_t* cv = nullptr;
    if (!a.none(4)) {
        const Tensor& c = a.tensor(4, "chunk_valid");
        TORCH_CHECK_TYPE(c.scalar_type() == at::kInt, "chunk_valid must be int32");
        TORCH_CHECK_VALUE(chunk >= 1 && tokens % chunk == 0, "tokens must be a multiple of chunk");
        need(c, "chunk_valid", b.dev, {tokens / chunk});
        cv = static_cast<const int32_t*>(c.data_ptr());
        valid = 0;
    }
    if (grad)
        check("sdm_gather_dw",
              sdm_gather_dw(b.codes, b.scales, b.n_slots, b.hd, b.group, b.format, static_cast<int>(k), idx,
                            reinterpret_cast<const float* const*>(in), out, width, it, wt, tokens, chunk, valid, cv, l.stream));
    else
        check("sdm_qgather", sdm_qgather(b.codes, b.scales, b.n_slots, b.hd, b.group, b.format, static_cast<int>(k), idx, in,
                                         reinterpret_cast<float* const*>(out), width, it, wt, tokens, chunk, valid, cv, l.stream));
    PyObject* list = PyList_New(k);
    if (list == nullptr) throw python_error();
    for (Py_ssize_t o = 0; o < k; ++o)
        PyList_SET_ITEM(list, o, give(given ? PySequence_Fast_GET_ITEM(given, o) : Py_None, made[o]));
    return list;
    END_HANDLE_TH_ERRORS
}

// decode(bank, k_idx, k_val, v, beta, g, q_idx, q_val, out or None, out dtype, leading dims, stream_major, stream)
PyObject* decode(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const Args a{args, n};
    expect(a, 13, "decode");
    const Bank b(a.a[0]);
    TORCH_CHECK_VALUE(b.format != SDM_INT4, "the decode takes int8 and fp8 banks");
    const int lead = a.small(10);
    const bool major = a.truth(11);
    const Tensor &k_idx = a.tensor(1, "k_idx"), &q_idx = a.tensor(6, "q_idx"), &g = a.tensor(5, "g");
    const int it = index_code(k_idx.scalar_type(), "k_idx");
    TORCH_CHECK_TYPE(q_idx.scalar_type() == k_idx.scalar_type(), "k_idx and q_idx must share one dtype, int32 or int64; got ",
                     k_idx.scalar_type(), ", ", q_idx.scalar_type());
    TORCH_CHECK_VALUE(k_idx.dim() == lead + 1 && q_idx.dim() == lead + 1 && g.dim() == lead + 1, "k_idx, q_idx and g must have ",
                      lead + 1, " dimensions");
    const int64_t A = k_idx.size(0), B = lead == 2 ? k_idx.size(1) : 1;
    const int64_t W = k_idx.size(lead), R = q_idx.size(lead), G = g.size(lead);
    int64_t shape[3] = {A, B, 0};
    const auto with = [&](int64_t last) {
        shape[lead] = last;
        return at::IntArrayRef(shape, lead + 1);
    };
    need(k_idx, "k_idx", b.dev, with(W));
    need(q_idx, "q_idx", b.dev, with(R));
    need_f32(g, "g", b.dev, with(G));
    const Tensor &k_val = a.tensor(2, "k_val"), &v = a.tensor(3, "v"), &beta = a.tensor(4, "beta"), &q_val = a.tensor(7, "q_val");
    need_f32(k_val, "k_val", b.dev, with(W));
    need_f32(q_val, "q_val", b.dev, with(R));
    need_f32(v, "v", b.dev, with(b.hd));
    if (lead == 2)
        need_f32(beta, "beta", b.dev, {A, B});
    else
        need_f32(beta, "beta", b.dev, {A});
    Launch l(b.dev, a.a[12]);
    Tensor made;
    if (a.none(8)) made = l.empty(with(b.hd), a.dtype(9, "out_dtype"), b.dev);
    const Tensor& out = a.none(8) ? made : a.tensor(8, "out");
    const int ot = float_code(out.scalar_type(), "readings");
    need(out, "out", b.dev, with(b.hd));
    const int64_t S = lead == 2 ? (major ? A : B) : A, T = lead == 2 ? (major ? B : A) : 1;
    const auto cap = [](int64_t x) { return x > 257 ? 257 : static_cast<int>(x); };  // 257: refused by the library
    TORCH_CHECK_VALUE(T <= INT_MAX, "too many tokens");
    check("sdm_qdecode_seq",
          sdm_qdecode_seq(b.codes, b.scales, b.n_slots, k_idx.data_ptr(), static_cast<const float*>(k_val.data_ptr()),
                          static_cast<const float*>(v.data_ptr()), static_cast<const float*>(beta.data_ptr()),
                          static_cast<const float*>(g.data_ptr()), q_idx.data_ptr(), static_cast<const float*>(q_val.data_ptr()),
                          out.data_ptr(), S, b.hd, b.group, b.format, cap(W), cap(R), cap(G), static_cast<int>(T), it, ot,
                          major ? SDM_STREAM_MAJOR : 0u, l.stream));
    return give(a.a[8], made);
    END_HANDLE_TH_ERRORS
}

// ---------------------------------------------------------------- routing

struct Logits {
    const Tensor& t;
    int64_t tokens, n, stride;
    int type;

    Logits(const Tensor& x, const char* name) : t(x) {
        type = float_code(x.scalar_type(), name);
        TORCH_CHECK_VALUE(x.dim() == 2, name, " must be [tokens, n]");
        TORCH_CHECK_VALUE(x.is_cuda(), name, " must be a CUDA tensor, got ", x.device());
        tokens = x.size(0);
        n = x.size(1);
        TORCH_CHECK_VALUE((n <= 1 || x.stride(1) == 1) && (tokens <= 1 || x.stride(0) >= n), name,
                          " must have contiguous columns and rows that do not overlap");
        stride = tokens <= 1 ? n : x.stride(0);
        if (n > 65536) n = 65537;  // refused by the library
    }
};

const void* base_of(const Args& a, int i, int64_t tokens, at::ScalarType it, const at::Device& dev) {
    if (a.none(i)) return nullptr;
    const Tensor& b = a.tensor(i, "base");
    TORCH_CHECK_TYPE(b.scalar_type() == it, "base must have the index dtype ", it, ", got ", b.scalar_type());
    need(b, "base", dev, {tokens});
    return b.data_ptr();
}

// route(logits, k, score, bias or None, groups, top_groups, group_top, renorm, scale, base or None,
//       index dtype, idx or None, w or None, stream)
PyObject* route(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const Args a{args, n};
    expect(a, 14, "route");
    const Logits x(a.tensor(0, "logits"), "logits");
    const at::Device dev = x.t.device();
    const int64_t k = a.integer(1);
    TORCH_CHECK_VALUE(k >= 1 && k <= 256, "k must be in 1..256, got ", k);
    const float* bias = nullptr;
    if (!a.none(3)) {
        const Tensor& b = a.tensor(3, "bias");
        need_f32(b, "bias", dev, {x.t.size(1)});
        bias = static_cast<const float*>(b.data_ptr());
    }
    Launch l(dev, a.a[13]);
    Tensor made_idx, made_w;
    if (a.none(11)) {
        const auto t = a.dtype(10, "idx_dtype");
        index_code(t, "idx_dtype");
        made_idx = l.empty({x.tokens, k}, t, dev);
    }
    if (a.none(12)) made_w = l.empty({x.tokens, k}, at::kFloat, dev);
    const Tensor& idx = a.none(11) ? made_idx : a.tensor(11, "idx");
    const Tensor& w = a.none(12) ? made_w : a.tensor(12, "w");
    const int it = index_code(idx.scalar_type(), "idx");
    need(idx, "idx", dev, {x.tokens, k});
    need_f32(w, "w", dev, {x.tokens, k});
    const void* base = base_of(a, 9, x.tokens, idx.scalar_type(), dev);
    check("sdm_route", sdm_route(x.t.data_ptr(), x.stride, x.type, bias, base, idx.data_ptr(), static_cast<float*>(w.data_ptr()),
                                 x.tokens, static_cast<int>(x.n), static_cast<int>(k), a.small(2), a.small(4), a.small(5), a.small(6),
                                 a.real(8), a.truth(7) ? SDM_RENORM : 0u, it, l.stream));
    PyObject* pair = PyTuple_New(2);
    if (pair == nullptr) throw python_error();
    PyTuple_SET_ITEM(pair, 0, give(a.a[11], made_idx));
    PyTuple_SET_ITEM(pair, 1, give(a.a[12], made_w));
    return pair;
    END_HANDLE_TH_ERRORS
}

// route_backward(logits, idx, dw, score, renorm, scale, base or None, w or None, out or None, stream)
PyObject* route_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const Args a{args, n};
    expect(a, 10, "route_backward");
    const Logits x(a.tensor(0, "logits"), "logits");
    const at::Device dev = x.t.device();
    const Tensor &idx = a.tensor(1, "idx"), &dw = a.tensor(2, "dw");
    const int it = index_code(idx.scalar_type(), "idx");
    TORCH_CHECK_VALUE(idx.dim() == 2, "idx must be [tokens, k]");
    const int64_t k = idx.size(1);
    need(idx, "idx", dev, {x.tokens, k});
    need_f32(dw, "dw", dev, {x.tokens, k});
    const void* base = base_of(a, 6, x.tokens, idx.scalar_type(), dev);
    const float* w = nullptr;
    if (!a.none(7)) {
        need_f32(a.tensor(7, "w"), "w", dev, {x.tokens, k});
        w = static_cast<const float*>(a.tensor(7, "w").data_ptr());
    }
    Launch l(dev, a.a[9]);
    Tensor made;
    if (a.none(8)) made = l.empty(x.t.sizes(), x.t.scalar_type(), dev);
    const Logits out(a.none(8) ? made : a.tensor(8, "out"), "out");
    TORCH_CHECK_TYPE(out.type == x.type && out.t.device() == dev, "out must have the dtype and the device of the logits");
    TORCH_CHECK_VALUE(out.t.sizes() == x.t.sizes(), "out has shape ", out.t.sizes(), ", expected ", x.t.sizes());
    check("sdm_route_backward_ex",
          sdm_route_backward_ex(x.t.data_ptr(), x.stride, x.type, base, idx.data_ptr(), w, static_cast<const float*>(dw.data_ptr()),
                                out.t.data_ptr(), out.stride, x.tokens, static_cast<int>(x.n), k > 256 ? 257 : static_cast<int>(k),
                                a.small(3), a.real(5), a.truth(4) ? SDM_RENORM : 0u, it, l.stream));
    return give(a.a[8], made);
    END_HANDLE_TH_ERRORS
}

// balance(logits, idx, score, w or None, base or None, offsets or None, scale, gradient, dloss or None, add or None,
//         loss or None, counts or None, out or None, stream)
PyObject* balance(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const Args a{args, n};
    expect(a, 14, "balance");
    const Logits x(a.tensor(0, "logits"), "logits");
    const at::Device dev = x.t.device();
    const Tensor& idx = a.tensor(1, "idx");
    const int it = index_code(idx.scalar_type(), "idx");
    TORCH_CHECK_VALUE(idx.dim() == 2, "idx must be [tokens, k]");
    const int64_t k = idx.size(1);
    need(idx, "idx", dev, {x.tokens, k});
    const float *w = nullptr, *dloss = nullptr;
    if (!a.none(3)) {
        need_f32(a.tensor(3, "w"), "w", dev, {x.tokens, k});
        w = static_cast<const float*>(a.tensor(3, "w").data_ptr());
    }
    const void* base = base_of(a, 4, x.tokens, idx.scalar_type(), dev);
    const int32_t* offsets = nullptr;
    int64_t sequences = 1;
    if (!a.none(5)) {
        const Tensor& o = a.tensor(5, "offsets");
        TORCH_CHECK_TYPE(o.scalar_type() == at::kInt, "offsets must be int32, got ", o.scalar_type());
        TORCH_CHECK_VALUE(o.dim() == 1 && o.size(0) >= 1, "offsets must be [sequences + 1], got ", o.sizes());
        sequences = o.size(0) - 1;
        need(o, "offsets", dev, {sequences + 1});
        offsets = static_cast<const int32_t*>(o.data_ptr());
    }
    const bool gradient = a.truth(7);
    TORCH_CHECK_VALUE(gradient || (a.none(8) && a.none(9) && a.none(12)), "dloss, add and out belong to the gradient");
    if (!a.none(8)) {
        need_f32(a.tensor(8, "dloss"), "dloss", dev, {sequences});
        dloss = static_cast<const float*>(a.tensor(8, "dloss").data_ptr());
    }
    Launch l(dev, a.a[13]);
    Tensor made_loss, made_counts, made_out;
    if (a.none(10)) made_loss = l.empty({sequences}, at::kFloat, dev);
    if (a.none(11)) made_counts = l.empty({sequences, x.t.size(1)}, at::kInt, dev);
    const Tensor& loss = a.none(10) ? made_loss : a.tensor(10, "loss");
    const Tensor& counts = a.none(11) ? made_counts : a.tensor(11, "counts");
    need_f32(loss, "loss", dev, {sequences});
    TORCH_CHECK_TYPE(counts.scalar_type() == at::kInt, "counts must be int32, got ", counts.scalar_type());
    need(counts, "counts", dev, {sequences, x.t.size(1)});
    const auto like_logits = [&](const Logits& g, const char* name) {
        TORCH_CHECK_TYPE(g.type == x.type && g.t.device() == dev, name, " must have the dtype and the device of the logits");
        TORCH_CHECK_VALUE(g.t.sizes() == x.t.sizes(), name, " has shape ", g.t.sizes(), ", expected ", x.t.sizes());
    };
    const void* add = nullptr;
    void* dlogits = nullptr;
    int64_t add_stride = 0, out_stride = 0;
    if (gradient) {
        if (!a.none(9)) {
            const Logits g(a.tensor(9, "add"), "add");
            like_logits(g, "add");
            add = g.t.data_ptr();
            add_stride = g.stride;
        }
        if (a.none(12)) made_out = l.empty(x.t.sizes(), x.t.scalar_type(), dev);
        const Logits g(a.none(12) ? made_out : a.tensor(12, "out"), "out");
        like_logits(g, "out");
        dlogits = g.t.data_ptr();
        out_stride = g.stride;
    }
    int64_t bytes = 0;
    check("sdm_balance_workspace", sdm_balance_workspace(sequences, &bytes));
    const Tensor scratch = l.workspace(bytes, dev);
    check("sdm_balance",
          sdm_balance(x.t.data_ptr(), x.stride, x.type, base, idx.data_ptr(), w, offsets, sequences, static_cast<float*>(loss.data_ptr()),
                      static_cast<int32_t*>(counts.data_ptr()), dloss, add, add_stride, dlogits, out_stride, x.tokens, static_cast<int>(x.n),
                      k > 256 ? 257 : static_cast<int>(k), a.small(2), a.real(6), it, scratch.data_ptr(), bytes, l.stream));
    PyObject* all = PyTuple_New(gradient ? 3 : 2);
    if (all == nullptr) throw python_error();
    PyTuple_SET_ITEM(all, 0, give(a.a[10], made_loss));
    PyTuple_SET_ITEM(all, 1, give(a.a[11], made_counts));
    if (gradient) PyTuple_SET_ITEM(all, 2, give(a.a[12], made_out));
    return all;
    END_HANDLE_TH_ERRORS
}

// ---------------------------------------------------------------- rows by token

int64_t padding_of(const Args& a, int i) {
    if (a.none(i)) return SDM_NO_PADDING;
    const int64_t p = a.integer(i);
    TORCH_CHECK_VALUE(p != SDM_NO_PADDING, "no such padding: ", p);
    return p;
}

// lookup(table, tokens, scale, padding or None, dtype or None, out or None, stream)
PyObject* lookup(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const Args a{args, n};
    expect(a, 7, "lookup");
    const Tensor &table = a.tensor(0, "table"), &tokens = a.tensor(1, "tokens");
    const int it = index_code(tokens.scalar_type(), "tokens");
    const Bank b(table, "table");
    need(tokens, "tokens", b.dev, tokens.sizes());
    std::vector<int64_t> shape(tokens.sizes().vec());
    shape.push_back(b.hd);
    Launch l(b.dev, a.a[6]);
    Tensor made;
    if (a.none(5)) {
        const auto t = a.none(4) ? table.scalar_type() : a.dtype(4, "dtype");
        float_code(t, "dtype");
        made = l.empty(shape, t, b.dev);
    }
    const Tensor& out = a.none(5) ? made : a.tensor(5, "out");
    const int ot = float_code(out.scalar_type(), "out");
    need(out, "out", b.dev, shape);
    check("sdm_lookup", sdm_lookup(b.codes, b.n_slots, b.hd, b.format, tokens.data_ptr(), it, tokens.numel(), padding_of(a, 3), a.real(2),
                                   out.data_ptr(), ot, l.stream));
    return give(a.a[5], made);
    END_HANDLE_TH_ERRORS
}

// The gradient of rows: made, or given to be written or added to.
struct RowsOut {
    Tensor made;
    const Tensor* t;
    int type;
    unsigned flags;

    RowsOut(const Args& a, const Launch& l, int dtype, int out, int accumulate, int64_t rows, int64_t hd, const at::Device& dev) {
        flags = a.truth(accumulate) ? SDM_ACCUMULATE : 0u;
        TORCH_CHECK_VALUE(!flags || !a.none(out), "there must be an out to add to");
        if (a.none(out)) {
            const auto ty = a.dtype(dtype, "dtype");
            float_code(ty, "dtype");
            made = l.empty({rows, hd}, ty, dev);
        }
        t = a.none(out) ? &made : &a.tensor(out, "out");
        type = float_code(t->scalar_type(), "the gradient");
        need(*t, "out", dev, {rows, hd});
    }
};

// lookup_backward(dout, tokens, rows, scale, padding or None, dtype, out or None, accumulate, stream)
PyObject* lookup_backward(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const Args a{args, n};
    expect(a, 9, "lookup_backward");
    const Tensor &dout = a.tensor(0, "dout"), &tokens = a.tensor(1, "tokens");
    const at::Device dev = dout.device();
    const int dt = float_code(dout.scalar_type(), "dout"), it = index_code(tokens.scalar_type(), "tokens");
    TORCH_CHECK_VALUE(dout.is_cuda(), "dout must be a CUDA tensor, got ", dev);
    TORCH_CHECK_VALUE(dout.dim() >= 1 && dout.dim() == tokens.dim() + 1, "dout must be [.., hd] for tokens [..], got ", dout.sizes(), " and ",
                      tokens.sizes());
    const int64_t hd = dout.size(-1);
    TORCH_CHECK_VALUE(hd >= 1 && hd <= 65536, "hd must be in 1..65536, got ", hd);
    need(tokens, "tokens", dev, dout.sizes().slice(0, dout.dim() - 1));
    need(dout, "dout", dev, dout.sizes());
    const int64_t count = tokens.numel(), rows = a.integer(2);
    int64_t bytes = 0;
    check("sdm_lookup_backward_workspace", sdm_lookup_backward_workspace(count, rows, static_cast<int>(hd), &bytes));
    Launch l(dev, a.a[8]);
    const RowsOut out(a, l, 5, 6, 7, rows, hd, dev);
    const Tensor scratch = l.workspace(bytes, dev);
    check("sdm_lookup_backward", sdm_lookup_backward(dout.data_ptr(), dt, tokens.data_ptr(), it, count, padding_of(a, 4), a.real(3),
                                                     out.t->data_ptr(), rows, static_cast<int>(hd), out.type, out.flags, scratch.data_ptr(),
                                                     bytes, l.stream));
    return give(a.a[6], out.made);
    END_HANDLE_TH_ERRORS
}

// gather_drows(ops, n_slots, chunk, valid or None, chunk_valid or None, dtype, out or None, accumulate, stream)
PyObject* gather_drows(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    const Args a{args, n};
    expect(a, 9, "gather_drows");
    const auto sequence = [](PyObject* o, const char* what) {
        TORCH_CHECK_TYPE(PyList_Check(o) || PyTuple_Check(o), what, " must be a list or tuple");
        return o;
    };
    PyObject* ops = sequence(a.a[0], "ops");
    const Py_ssize_t k = PySequence_Fast_GET_SIZE(ops);
    TORCH_CHECK_VALUE(k == 1 || k == 2, "gather_drows takes one or two operands");
    const void *idx[2] = {nullptr, nullptr}, *w[2] = {nullptr, nullptr};
    const float* dout[2] = {nullptr, nullptr};
    int width[2] = {0, 0}, it = SDM_I32, wt = SDM_F32;
    int64_t tokens = 0, entries = 0, hd = 0;
    at::Device dev(at::kCPU);
    for (Py_ssize_t o = 0; o < k; ++o) {
        PyObject* three = sequence(PySequence_Fast_GET_ITEM(ops, o), "an operand");
        TORCH_CHECK_VALUE(PySequence_Fast_GET_SIZE(three) == 3, "an operand is three tensors: idx, w and dout");
        const Tensor& i = Args::unpack(PySequence_Fast_GET_ITEM(three, 0), "idx");
        const Tensor& x = Args::unpack(PySequence_Fast_GET_ITEM(three, 1), "w");
        const Tensor& d = Args::unpack(PySequence_Fast_GET_ITEM(three, 2), "dout");
        const int t = index_code(i.scalar_type(), "idx"), xt = float_code(x.scalar_type(), "weights");
        TORCH_CHECK_VALUE(i.dim() == 2 && d.dim() == 2, "idx must be [tokens, width] and dout [tokens, hd]");
        if (o == 0) {
            dev = i.device();
            TORCH_CHECK_VALUE(i.is_cuda(), "idx must be a CUDA tensor, got ", dev);
            tokens = i.size(0);
            hd = d.size(1);
            it = t;
            wt = xt;
            TORCH_CHECK_VALUE(hd >= 1 && hd <= 65536, "hd must be in 1..65536, got ", hd);
        }
        TORCH_CHECK_TYPE(t == it, "both operands must share the index dtype");
        TORCH_CHECK_TYPE(xt == wt, "both operands must share the dtype of w");
        need(i, "idx", dev, {tokens, i.size(1)});
        need(x, "w", dev, i.sizes());
        need_f32(d, "dout", dev, {tokens, hd});
        idx[o] = i.data_ptr();
        w[o] = x.data_ptr();
        dout[o] = static_cast<const float*>(d.data_ptr());
        width[o] = i.size(1) > 256 ? 257 : static_cast<int>(i.size(1));
        entries += tokens * width[o];
    }
    const int chunk = a.small(2);
    int valid = a.none(3) ? chunk : a.small(3);
    const int32_t* cv = nullptr;
    if (!a.none(4)) {
        const Tensor& c = a.tensor(4, "chunk_valid");
        TORCH_CHECK_TYPE(c.scalar_type() == at::kInt, "chunk_valid must be int32");
        TORCH_CHECK_VALUE(chunk >= 1 && tokens % chunk == 0, "tokens must be a multiple of chunk");
        need(c, "chunk_valid", dev, {tokens / chunk});
        cv = static_cast<const int32_t*>(c.data_ptr());
        valid = 0;
    }
    const int64_t n_slots = a.integer(1);
    int64_t bytes = 0;
    check("sdm_gather_drows_workspace", sdm_gather_drows_workspace(entries, n_slots, static_cast<int>(hd), &bytes));
    Launch l(dev, a.a[8]);
    const RowsOut out(a, l, 5, 6, 7, n_slots, hd, dev);
    const Tensor scratch = l.workspace(bytes, dev);
    check("sdm_gather_drows", sdm_gather_drows(static_cast<int>(k), idx, w, dout, width, it, wt, out.t->data_ptr(), n_slots,
                                               static_cast<int>(hd), out.type, out.flags, tokens, chunk, valid, cv, scratch.data_ptr(), bytes,
                                               l.stream));
    return give(a.a[6], out.made);
    END_HANDLE_TH_ERRORS
}

// raise_with(f): f(function, status) is called to raise the error of a status code
PyObject* raise_with(PyObject*, PyObject* f) {
    Py_INCREF(f);
    Py_XSETREF(g_raise_status, f);
    Py_RETURN_NONE;
}

template <typename F>
PyCFunction fast(F f) {
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f));
}

PyMethodDef methods[] = {{"check_bank", fast(check_bank), METH_FASTCALL, nullptr},
                         {"room", fast(room), METH_FASTCALL, nullptr},
                         {"rows", fast(rows), METH_FASTCALL, nullptr},
                         {"gather", fast(gather), METH_FASTCALL, nullptr},
                         {"decode", fast(decode), METH_FASTCALL, nullptr},
                         {"route", fast(route), METH_FASTCALL, nullptr},
                         {"route_backward", fast(route_backward), METH_FASTCALL, nullptr},
                         {"balance", fast(balance), METH_FASTCALL, nullptr},
                         {"lookup", fast(lookup), METH_FASTCALL, nullptr},
                         {"lookup_backward", fast(lookup_backward), METH_FASTCALL, nullptr},
                         {"gather_drows", fast(gather_drows), METH_FASTCALL, nullptr},
                         {"raise_with", raise_with, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "sdm_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit_sdm_torch() { return PyModule_Create(&module_def); }
