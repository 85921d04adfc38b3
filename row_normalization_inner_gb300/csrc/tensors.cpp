// Tensor helpers of the token-side operators and of those on attention heads:
// checks, output allocation and the call, in one native step.
//
// A decode step's call takes 2 us on the GPU.  Checking its tensors,
// allocating its outputs through the interpreter and converting its
// arguments one by one took 9 to 19 us on the host; here it is a third to a half
// of that.  Python keeps the signatures and the documentation
// (row_normalization_inner_gb300/__init__.py); PyTorch provides device memory
// and streams only, and every step of the computation runs in libnf.so.
//
// Each function returns the helper's result, or the C call's status as an
// int where it is not NF_OK.  Wrong types raise TypeError, anything else that
// does not fit ValueError.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include "../../include/nf.h"

namespace {

using at::ScalarType;
using at::Tensor;

const Tensor& tensor(PyObject* o, const char* name) {
    TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
    return THPVariable_Unpack(o);
}

bool given(PyObject* o) { return o != Py_None; }

void need_type(const Tensor& t, const char* name, ScalarType type) {
    TORCH_CHECK_TYPE(t.scalar_type() == type, name, " must be ", type, ", got ", t.scalar_type());
}

// The tensor's device, which must be the current one: the call uses its
// context and stream.
int device_of(const Tensor& t, const char* name) {
    TORCH_CHECK_VALUE(t.is_cuda(), name, " must be a CUDA tensor");
    const int dev = t.get_device();
    TORCH_CHECK_VALUE(dev == c10::cuda::current_device(), name, " is on cuda:", dev, ", which is not the current device");
    return dev;
}

void need_on(const Tensor& t, const char* name, int dev, bool contiguous = true) {
    TORCH_CHECK_VALUE(t.is_cuda() && t.get_device() == dev, name, " must be a CUDA tensor on cuda:", dev);
    TORCH_CHECK_VALUE(!contiguous || t.is_contiguous(), name, " must be contiguous");
}

// Bytes per id.
int id_bytes(const Tensor& t, const char* name) {
    TORCH_CHECK_TYPE(t.scalar_type() == at::kLong || t.scalar_type() == at::kInt, name,
                     " must be torch.int32 or torch.int64, got ", t.scalar_type());
    return t.scalar_type() == at::kLong ? 8 : 4;
}

nf_stream stream_of(int dev) {
    return reinterpret_cast<nf_stream>(c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream());
}

Tensor empty(at::IntArrayRef shape, ScalarType type, int dev) {
    return Tensor(at::detail::empty_cuda(shape, type, at::Device(at::kCUDA, static_cast<c10::DeviceIndex>(dev)), std::nullopt));
}

double number(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    return v;
}

int64_t integer(PyObject* o) {
    const int64_t v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}

PyObject* status(nf_status st) { return PyLong_FromLong(st); }

// A tensor the caller gave is returned as the object it is.
PyObject* object(PyObject* was, const Tensor& t) {
    if (!given(was)) return THPVariable_Wrap(t);
    Py_INCREF(was);
    return was;
}

PyObject* pack(std::initializer_list<PyObject*> items) {
    PyObject* tuple = PyTuple_New(static_cast<Py_ssize_t>(items.size()));
    if (!tuple) throw python_error();
    Py_ssize_t i = 0;
    for (PyObject* o : items) PyTuple_SET_ITEM(tuple, i++, o);
    return tuple;
}

// The interpreter runs on while a helper allocates and launches: neither
// needs it, and both can wait (for memory, for room in the launch queue).
struct WithoutInterpreter {
    PyThreadState* state = PyEval_SaveThread();
    WithoutInterpreter() = default;
    WithoutInterpreter(const WithoutInterpreter&) = delete;
    WithoutInterpreter& operator=(const WithoutInterpreter&) = delete;
    ~WithoutInterpreter() { PyEval_RestoreThread(state); }
};

void count(Py_ssize_t n, Py_ssize_t want) { TORCH_CHECK_TYPE(n == want, "expected ", want, " arguments, got ", n); }

// (x, residual or None, weight, eps, fmt, group, out or None, scale or None) -> (q, scale)
PyObject* norm_q8(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 8);
    const Tensor& x = tensor(a[0], "x");
    need_type(x, "x", at::kBFloat16);
    const int dev = device_of(x, "x");
    need_on(x, "x", dev);
    const bool fused = given(a[1]);
    const int64_t hidden = x.dim() ? x.size(-1) : 0, rows = hidden ? x.numel() / hidden : 0;
    const Tensor& weight = tensor(a[2], "weight");
    need_type(weight, "weight", at::kBFloat16);
    need_on(weight, "weight", dev);
    TORCH_CHECK_VALUE(weight.dim() == 1 && weight.size(0) == hidden, "weight must be of shape [hidden]");
    if (fused) {
        const Tensor& residual = tensor(a[1], "residual");
        need_type(residual, "residual", at::kBFloat16);
        need_on(residual, "residual", dev);
        TORCH_CHECK_VALUE(residual.sizes() == x.sizes(), "residual must have x's shape");
    }
    const bool e4m3 = PyUnicode_Check(a[4]) && PyUnicode_CompareWithASCIIString(a[4], "e4m3") == 0;
    const bool int8 = PyUnicode_Check(a[4]) && PyUnicode_CompareWithASCIIString(a[4], "int8") == 0;
    TORCH_CHECK_VALUE(e4m3 || int8, "fmt must be 'e4m3' or 'int8'");
    const int64_t group = integer(a[5]);
    TORCH_CHECK_VALUE(group == 0 || group == 128, "group must be 0 (one scale per row) or 128, got ", group);
    const ScalarType type = int8 ? at::kChar : at::kFloat8_e4m3fn;
    c10::SmallVector<int64_t, 5> shape(x.sizes().begin(), x.sizes().end());
    if (!shape.empty()) shape.pop_back();
    if (group) shape.push_back((hidden + group - 1) / group);
    Tensor out, scale;
    if (given(a[6])) {
        out = tensor(a[6], "out");
        need_type(out, "out", type);
        need_on(out, "out", dev);
        TORCH_CHECK_VALUE(out.sizes() == x.sizes(), "out must have x's shape");
    }
    if (given(a[7])) {
        scale = tensor(a[7], "scale");
        need_type(scale, "scale", at::kFloat);
        need_on(scale, "scale", dev);
        TORCH_CHECK_VALUE(scale.sizes() == at::IntArrayRef(shape), "scale must be of shape ", at::IntArrayRef(shape));
    }
    const float eps = static_cast<float>(number(a[3]));
    nf_status st;
    {
        const WithoutInterpreter w;
        if (!out.defined()) out = empty(x.sizes(), type, dev);
        if (!scale.defined()) scale = empty(shape, at::kFloat, dev);
        const nf_q8_format format = int8 ? NF_Q8_INT8 : NF_Q8_E4M3;
        float* s = static_cast<float*>(scale.data_ptr());
        st =
            fused ? nf_fused_add_rmsnorm_q8(out.data_ptr(), s, x.const_data_ptr(), THPVariable_Unpack(a[1]).data_ptr(), weight.const_data_ptr(),
                                            rows, hidden, eps, format, group, stream_of(dev))
                  : nf_rmsnorm_q8(out.data_ptr(), s, x.const_data_ptr(), weight.const_data_ptr(), rows, hidden, eps, format, group, stream_of(dev));
    }
    if (st != NF_OK) return status(st);
    return pack({object(a[6], out), object(a[7], scale)});
    END_HANDLE_TH_ERRORS
}

// (ids, table, scale, out or None) -> out
PyObject* embedding_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 4);
    const Tensor& ids = tensor(a[0], "ids");
    const int bytes = id_bytes(ids, "ids");
    const Tensor& table = tensor(a[1], "table");
    need_type(table, "table", at::kBFloat16);
    const int dev = device_of(table, "table");
    need_on(ids, "ids", dev);
    TORCH_CHECK_VALUE(table.dim() == 2 && table.is_contiguous(), "table must be [vocab, hidden] and contiguous");
    c10::SmallVector<int64_t, 5> shape(ids.sizes().begin(), ids.sizes().end());
    shape.push_back(table.size(1));
    Tensor out;
    if (given(a[3])) {
        out = tensor(a[3], "out");
        need_type(out, "out", at::kBFloat16);
        need_on(out, "out", dev);
        TORCH_CHECK_VALUE(out.sizes() == at::IntArrayRef(shape), "out must be of shape ", at::IntArrayRef(shape));
    }
    const float scale = static_cast<float>(number(a[2]));
    nf_status st;
    {
        const WithoutInterpreter w;
        if (!out.defined()) out = empty(shape, at::kBFloat16, dev);
        st = nf_embedding_fwd(out.data_ptr(), ids.const_data_ptr(), bytes, table.const_data_ptr(), ids.numel(), table.size(0),
                                              table.size(1), scale, stream_of(dev));
    }
    return st != NF_OK ? status(st) : object(a[3], out);
    END_HANDLE_TH_ERRORS
}

// (dy, ids, vocab, scale, dtype or None, accumulate or None, out or None, workspace or None) -> gradient
PyObject* embedding_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 8);
    const Tensor& ids = tensor(a[1], "ids");
    const int bytes = id_bytes(ids, "ids");
    const Tensor& dy = tensor(a[0], "dy");
    need_type(dy, "dy", at::kBFloat16);
    const int dev = device_of(dy, "dy");
    need_on(ids, "ids", dev);
    TORCH_CHECK_VALUE(dy.dim() >= 1 && dy.sizes().slice(0, dy.dim() - 1) == ids.sizes() && dy.is_contiguous(),
                      "dy must be of shape [*ids.shape, hidden] and contiguous");
    const int64_t hidden = dy.size(-1), vocab = integer(a[2]), tokens = ids.numel();
    TORCH_CHECK_TYPE(!given(a[4]) || THPDtype_Check(a[4]), "dtype must be a torch.dtype");
    const ScalarType want = given(a[4]) ? reinterpret_cast<THPDtype*>(a[4])->scalar_type : at::kFloat;
    TORCH_CHECK_TYPE(want == at::kFloat || want == at::kBFloat16, "the gradient must be torch.float32 or torch.bfloat16, got ", want);
    const bool add = given(a[5]);
    TORCH_CHECK_VALUE(!add || !given(a[6]), "accumulate is written in place: out cannot be given too");
    PyObject* place = add ? a[5] : a[6];
    const std::array<int64_t, 2> shape = {vocab, hidden};
    Tensor grad;
    if (given(place)) {
        grad = tensor(place, "the gradient");
        TORCH_CHECK_TYPE(given(a[4]) ? grad.scalar_type() == want
                                     : grad.scalar_type() == at::kFloat || grad.scalar_type() == at::kBFloat16,
                         "the gradient must be torch.float32 or torch.bfloat16 and of the type asked for, got ", grad.scalar_type());
        need_on(grad, "the gradient", dev);
        TORCH_CHECK_VALUE(grad.sizes() == at::IntArrayRef(shape), "the gradient must be of shape ", at::IntArrayRef(shape));
    }
    Tensor ws;
    if (given(a[7])) {
        ws = tensor(a[7], "workspace");
        need_on(ws, "workspace", dev);
    }
    const float scale = static_cast<float>(number(a[3]));
    TORCH_CHECK_VALUE(vocab >= 0, "vocab must not be negative");
    nf_status st;
    {
        const WithoutInterpreter w;
        if (!grad.defined()) grad = empty(shape, want, dev);
        if (!ws.defined()) {
            // freed right after the launches: the allocator hands the block to
            // later work on the same stream only, which runs after these kernels
            const int64_t need = static_cast<int64_t>(nf_embedding_bwd_workspace_size(tokens, hidden));
            ws = empty({need > 16 ? need : 16}, at::kByte, dev);
        }
        st = nf_embedding_bwd(grad.data_ptr(), grad.scalar_type() == at::kFloat ? NF_F32 : NF_BF16, add, dy.const_data_ptr(),
                                              ids.const_data_ptr(), bytes, tokens, vocab, hidden, scale, ws.data_ptr(), ws.nbytes(),
                                              stream_of(dev));
    }
    return st != NF_OK ? status(st) : object(place, grad);
    END_HANDLE_TH_ERRORS
}

void need_logits(const Tensor& t) {
    TORCH_CHECK_TYPE(t.scalar_type() == at::kBFloat16 || t.scalar_type() == at::kFloat,
                     "logits must be torch.bfloat16 or torch.float32, got ", t.scalar_type());
}

nf_dtype type_of(const Tensor& t) { return t.scalar_type() == at::kFloat ? NF_F32 : NF_BF16; }

// Row stride of a [rows, vocab] tensor whose rows may be apart.
int64_t row_stride(const Tensor& t, const char* name) {
    TORCH_CHECK_VALUE(t.dim() == 2, name, " must be [rows, vocab]");
    const int64_t vocab = t.size(1), stride = t.size(0) <= 1 ? (vocab > 1 ? vocab : 1) : t.stride(0);
    TORCH_CHECK_VALUE((vocab <= 1 || t.stride(1) == 1) && stride >= vocab, name, "'s rows must be contiguous and apart");
    return stride;
}

void need_rows(const Tensor& t, const char* name, int dev, int64_t rows) {
    need_type(t, name, at::kFloat);
    need_on(t, name, dev);
    TORCH_CHECK_VALUE(t.dim() == 1 && t.size(0) == rows, name, " must be of shape [rows]");
}

// (logits, targets, temperature, top) -> (logprob, entropy, stats, top_logprob, top_ids)
PyObject* token_logprob_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 4);
    const Tensor& logits = tensor(a[0], "logits");
    need_logits(logits);
    const int dev = device_of(logits, "logits");
    const int64_t stride = row_stride(logits, "logits"), rows = logits.size(0), vocab = logits.size(1);
    const Tensor& targets = tensor(a[1], "targets");
    const int bytes = id_bytes(targets, "targets");
    need_on(targets, "targets", dev);
    TORCH_CHECK_VALUE(targets.dim() == 1 && targets.size(0) == rows, "targets must be of shape [rows]");
    const int64_t top = integer(a[3]);
    TORCH_CHECK_VALUE(top >= 0 && top <= NF_TOP_MAX, "top must be 0 to ", NF_TOP_MAX, ", got ", top);
    const float temperature = static_cast<float>(number(a[2]));
    Tensor logprob, entropy, stats, top_logprob, top_ids;
    nf_status st;
    {
        const WithoutInterpreter w;
        logprob = empty({rows}, at::kFloat, dev);
        entropy = empty({rows}, at::kFloat, dev);
        stats = empty({rows, 2}, at::kFloat, dev);
        if (top) {
            top_logprob = empty({rows, top}, at::kFloat, dev);
            top_ids = empty({rows, top}, at::kLong, dev);
        }
        const auto f32 = [](const Tensor& t) { return static_cast<float*>(t.data_ptr()); };
        st = nf_token_logprob_fwd(f32(logprob), f32(entropy), f32(stats), top ? f32(top_logprob) : nullptr,
                                                  top ? static_cast<int64_t*>(top_ids.data_ptr()) : nullptr, logits.const_data_ptr(),
                                                  type_of(logits), stride, targets.const_data_ptr(), bytes, rows, vocab, temperature,
                                                  static_cast<int32_t>(top), stream_of(dev));
    }
    if (st != NF_OK) return status(st);
    const auto wrap = [](const Tensor& t) {
        if (t.defined()) return THPVariable_Wrap(t);
        Py_INCREF(Py_None);
        return Py_None;
    };
    return pack({wrap(logprob), wrap(entropy), wrap(stats), wrap(top_logprob), wrap(top_ids)});
    END_HANDLE_TH_ERRORS
}

// (logits, targets, stats, entropy, d_logprob, d_entropy or None, temperature, out or None) -> out
PyObject* token_logprob_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 8);
    const Tensor& logits = tensor(a[0], "logits");
    need_logits(logits);
    const int dev = device_of(logits, "logits");
    const int64_t stride = row_stride(logits, "logits"), rows = logits.size(0), vocab = logits.size(1);
    const Tensor& targets = tensor(a[1], "targets");
    const int bytes = id_bytes(targets, "targets");
    need_on(targets, "targets", dev);
    TORCH_CHECK_VALUE(targets.dim() == 1 && targets.size(0) == rows, "targets must be of shape [rows]");
    const Tensor& stats = tensor(a[2], "stats");
    need_type(stats, "stats", at::kFloat);
    need_on(stats, "stats", dev);
    TORCH_CHECK_VALUE(stats.dim() == 2 && stats.size(0) == rows && stats.size(1) == 2, "stats must be of shape [rows, 2]");
    const Tensor& d_logprob = tensor(a[4], "d_logprob");
    need_rows(d_logprob, "d_logprob", dev, rows);
    const float *ent = nullptr, *d_ent = nullptr;
    if (given(a[5])) {
        const Tensor& d_entropy = tensor(a[5], "d_entropy");
        need_rows(d_entropy, "d_entropy", dev, rows);
        const Tensor& entropy = tensor(a[3], "entropy");
        need_rows(entropy, "entropy", dev, rows);
        ent = static_cast<const float*>(entropy.const_data_ptr());
        d_ent = static_cast<const float*>(d_entropy.const_data_ptr());
    }
    Tensor out;
    int64_t out_stride = vocab > 1 ? vocab : 1;
    if (given(a[7])) {
        out = tensor(a[7], "out");
        TORCH_CHECK_VALUE(out.scalar_type() == logits.scalar_type() && out.sizes() == logits.sizes(),
                          "out must have the logits' type and shape");
        need_on(out, "out", dev, false);
        out_stride = row_stride(out, "out");
    }
    const float temperature = static_cast<float>(number(a[6]));
    nf_status st;
    {
        const WithoutInterpreter w;
        if (!out.defined()) out = empty({rows, vocab}, logits.scalar_type(), dev);
        st = nf_token_logprob_bwd(out.data_ptr(), out_stride, logits.const_data_ptr(), type_of(logits), stride, targets.const_data_ptr(),
                                                  bytes, static_cast<const float*>(stats.const_data_ptr()), ent,
                                                  static_cast<const float*>(d_logprob.const_data_ptr()), d_ent, rows, vocab, temperature,
                                                  stream_of(dev));
    }
    return st != NF_OK ? status(st) : object(a[7], out);
    END_HANDLE_TH_ERRORS
}

// ---- attention heads

void need_head_type(const Tensor& t, const char* name) {
    TORCH_CHECK_TYPE(t.scalar_type() == at::kBFloat16 || t.scalar_type() == at::kFloat, name,
                     " must be torch.bfloat16 or torch.float32, got ", t.scalar_type());
}

// A [batch, tokens, heads, head_dim] or [tokens, heads, head_dim] tensor in any order.
struct Heads {
    Tensor t;
    nf_heads h{};
    int64_t batch = 1, tokens = 0, dim = 0;
};
Heads heads_of(const Tensor& t, const char* name, int dev) {
    need_on(t, name, dev, false);
    TORCH_CHECK_VALUE(t.dim() == 3 || t.dim() == 4, name, " must be [batch, tokens, heads, head_dim] or [tokens, heads, head_dim]");
    const int d = static_cast<int>(t.dim());
    Heads x;
    x.t = t;
    x.batch = d == 4 ? t.size(0) : 1;
    x.tokens = t.size(d - 3);
    x.dim = t.size(d - 1);
    TORCH_CHECK_VALUE(x.dim <= 1 || t.stride(d - 1) == 1, name, "'s heads must be contiguous");
    TORCH_CHECK_VALUE(t.size(d - 2) <= 0x7FFFFFFF, name, " has too many heads");
    x.h.data = t.numel() ? const_cast<void*>(t.const_data_ptr()) : nullptr;
    x.h.batch_stride = d == 4 ? t.stride(0) : 0;
    x.h.token_stride = t.stride(d - 3);
    x.h.head_stride = t.stride(d - 2);
    x.h.heads = static_cast<int32_t>(t.size(d - 2));
    return x;
}
// Another tensor of x's batch, tokens and head size, and of its heads too (`alike`).
Heads heads_like(PyObject* o, const char* name, const Heads& x, const char* x_name, bool alike) {
    const Tensor& t = tensor(o, name);
    need_type(t, name, x.t.scalar_type());
    Heads y = heads_of(t, name, x.t.get_device());
    TORCH_CHECK_VALUE(t.dim() == x.t.dim() && y.batch == x.batch && y.tokens == x.tokens && y.dim == x.dim && (!alike || y.h.heads == x.h.heads),
                      name, " of shape ", t.sizes(), " does not go with ", x_name, " of shape ", x.t.sizes());
    return y;
}
// Outputs of one call in one allocation, each from a 256-byte boundary: every
// further allocation and its release took 0.45 us of a decode step's 4.7.
class Together {
  public:
    explicit Together(int dev) : dev_(dev) {}
    // All are asked for, then taken in the same order.
    void want(at::IntArrayRef shape, ScalarType type) { bytes_ += room(shape, type); }
    Tensor take(at::IntArrayRef shape, ScalarType type) {
        if (!whole_.defined()) whole_ = empty({bytes_}, at::kByte, dev_);
        Tensor t = at::detail::make_tensor<at::TensorImpl>(c10::Storage(whole_.storage()), whole_.key_set(), c10::scalarTypeToTypeMeta(type));
        t.unsafeGetTensorImpl()->set_storage_offset(at_ / static_cast<int64_t>(c10::elementSize(type)));
        t.unsafeGetTensorImpl()->set_sizes_contiguous(shape);
        at_ += room(shape, type);
        return t;
    }
    void want(const Heads& x) { want(x.t.sizes(), x.t.scalar_type()); }
    Heads take(const Heads& x) { return heads_of(take(x.t.sizes(), x.t.scalar_type()), "out", dev_); }

  private:
    static int64_t room(at::IntArrayRef shape, ScalarType type) {
        int64_t n = static_cast<int64_t>(c10::elementSize(type));
        for (const int64_t s : shape) n *= s;
        return (n + 255) / 256 * 256;
    }
    const int dev_;
    int64_t bytes_ = 0, at_ = 0;
    Tensor whole_;
};
// The two outputs of a call that are not given.  Large ones, whose call takes longer on
// the GPU (10 us) than on the host, are apart: who keeps the keys alone does
// not keep the queries' memory, eight times as much, with them.
constexpr int64_t kMostTogether = 32 << 20;
void make_outputs(const Heads& q, Heads& q_out, bool two, const Heads& k, Heads& k_out) {
    const int dev = q.t.get_device();
    const bool make_q = !q_out.t.defined(), make_k = two && !k_out.t.defined();
    if (make_q && make_k && (q.t.numel() + k.t.numel()) * static_cast<int64_t>(q.t.element_size()) > kMostTogether) {
        q_out = heads_of(empty(q.t.sizes(), q.t.scalar_type(), dev), "out", dev);
        k_out = heads_of(empty(k.t.sizes(), k.t.scalar_type(), dev), "out", dev);
        return;
    }
    Together made(dev);
    if (make_q) made.want(q);
    if (make_k) made.want(k);
    if (make_q) q_out = made.take(q);
    if (make_k) k_out = made.take(k);
}

const void* head_weight(PyObject* o, const char* name, const Heads& x) {
    const Tensor& w = tensor(o, name);
    need_type(w, name, x.t.scalar_type());
    need_on(w, name, x.t.get_device());
    TORCH_CHECK_VALUE(w.dim() == 1 && w.size(0) == x.dim, name, " must be of shape [head_dim]");
    return w.const_data_ptr();
}

// The rotation of a call, from (positions or None, rates or None, layout, magnitude).
// The tensors it points to are the caller's.
nf_rope rope_of(PyObject* positions, PyObject* rates, PyObject* layout, PyObject* magnitude, const Heads& x, bool places) {
    nf_rope r{};
    const bool half = PyUnicode_Check(layout) && PyUnicode_CompareWithASCIIString(layout, "half") == 0;
    const bool inter = PyUnicode_Check(layout) && PyUnicode_CompareWithASCIIString(layout, "interleaved") == 0;
    TORCH_CHECK_VALUE(half || inter, "layout must be 'half' or 'interleaved'");
    r.layout = half ? NF_ROPE_HALF : NF_ROPE_INTERLEAVED;
    r.magnitude = static_cast<float>(number(magnitude));
    if (!given(rates)) {
        TORCH_CHECK_VALUE(!given(positions), "positions are given without rates");
        return r;
    }
    const int dev = x.t.get_device();
    const Tensor& f = tensor(rates, "rates");
    need_type(f, "rates", at::kLong);
    need_on(f, "rates", dev);
    TORCH_CHECK_VALUE(f.dim() == 1 && 2 * f.size(0) <= x.dim, "rates must be of shape [pairs], head_dim / 2 of them at most");
    r.rates = static_cast<const uint64_t*>(f.const_data_ptr());
    r.dim = static_cast<int32_t>(2 * f.size(0));
    TORCH_CHECK_VALUE(given(positions) || places || r.dim == 0, "positions must be given");
    if (!given(positions)) return r;
    const Tensor& p = tensor(positions, "positions");
    r.position_bytes = id_bytes(p, "positions");
    need_on(p, "positions", dev, false);
    const bool batched = p.dim() == 2 && x.t.dim() == 4;
    TORCH_CHECK_VALUE((batched && p.size(0) == x.batch) || p.dim() == 1, "positions must be of shape [batch, tokens] or [tokens]");
    TORCH_CHECK_VALUE(p.size(-1) == x.tokens && (x.tokens <= 1 || p.stride(-1) == 1),
                      "positions must be of shape [batch, tokens] or [tokens], contiguous within a batch");
    r.positions = p.const_data_ptr();
    r.position_stride = batched && x.batch > 1 ? p.stride(0) : 0;
    return r;
}

PyObject* none() {
    Py_INCREF(Py_None);
    return Py_None;
}

// (q, k or None, positions, rates, layout, magnitude, q_out or None, k_out or None, back) -> (q_out, k_out)
PyObject* rope(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 9);
    const Tensor& qt = tensor(a[0], "q");
    need_head_type(qt, "q");
    const Heads q = heads_of(qt, "q", device_of(qt, "q"));
    const bool two = given(a[1]);
    Heads k, qo, ko;
    if (two) k = heads_like(a[1], "k", q, "q", false);
    TORCH_CHECK_VALUE(two || !given(a[7]), "k_out is given without k");
    TORCH_CHECK_TYPE(given(a[3]), "rates must be a tensor");
    const nf_rope r = rope_of(a[2], a[3], a[4], a[5], q, false);
    if (given(a[6])) qo = heads_like(a[6], "q_out", q, "q", true);
    if (given(a[7])) ko = heads_like(a[7], "k_out", k, "k", true);
    const bool back = PyObject_IsTrue(a[8]);
    nf_status st;
    {
        const WithoutInterpreter w;
        make_outputs(q, qo, two, k, ko);
        st = (back ? nf_rope_bwd : nf_rope_fwd)(&qo.h, &q.h, two ? &ko.h : nullptr, two ? &k.h : nullptr, type_of(q.t), q.batch, q.tokens,
                                                q.dim, &r, stream_of(q.t.get_device()));
    }
    if (st != NF_OK) return status(st);
    return pack({object(a[6], qo.t), two ? object(a[7], ko.t) : none()});
    END_HANDLE_TH_ERRORS
}

// (q, k or None, q_weight, k_weight or None, positions or None, rates or None, eps, layout, magnitude, q_out or None,
//  k_out or None) -> (q_out, k_out)
PyObject* qk_rmsnorm_rope_fwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 11);
    const Tensor& qt = tensor(a[0], "q");
    need_head_type(qt, "q");
    const Heads q = heads_of(qt, "q", device_of(qt, "q"));
    const bool two = given(a[1]);
    Heads k, qo, ko;
    if (two) k = heads_like(a[1], "k", q, "q", false);
    TORCH_CHECK_VALUE(two || (!given(a[3]) && !given(a[10])), "k_weight or k_out is given without k");
    const void* qw = head_weight(a[2], "q_weight", q);
    const void* kw = two ? head_weight(a[3], "k_weight", k) : nullptr;
    const nf_rope r = rope_of(a[4], a[5], a[7], a[8], q, false);
    if (given(a[9])) qo = heads_like(a[9], "q_out", q, "q", true);
    if (given(a[10])) ko = heads_like(a[10], "k_out", k, "k", true);
    const float eps = static_cast<float>(number(a[6]));
    nf_status st;
    {
        const WithoutInterpreter w;
        make_outputs(q, qo, two, k, ko);
        st = nf_qk_rmsnorm_rope_fwd(&qo.h, &q.h, qw, two ? &ko.h : nullptr, two ? &k.h : nullptr, kw, type_of(q.t), q.batch, q.tokens, q.dim,
                                    eps, &r, stream_of(q.t.get_device()));
    }
    if (st != NF_OK) return status(st);
    return pack({object(a[9], qo.t), two ? object(a[10], ko.t) : none()});
    END_HANDLE_TH_ERRORS
}

// (dq_out, dk_out or None, q, k or None, q_weight, k_weight or None, positions or None, rates or None, eps, layout,
//  magnitude, dq or None, dk or None, workspace or None) -> (dq, dk, dq_weight, dk_weight)
PyObject* qk_rmsnorm_rope_bwd(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 14);
    const Tensor& qt = tensor(a[2], "q");
    need_head_type(qt, "q");
    const int dev = device_of(qt, "q");
    const Heads q = heads_of(qt, "q", dev), dqo = heads_like(a[0], "dq_out", q, "q", true);
    const bool two = given(a[3]);
    Heads k, dko, dq, dk;
    if (two) {
        k = heads_like(a[3], "k", q, "q", false);
        dko = heads_like(a[1], "dk_out", k, "k", true);
    }
    TORCH_CHECK_VALUE(two || (!given(a[1]) && !given(a[5]) && !given(a[12])), "dk_out, k_weight or dk is given without k");
    const void* qw = head_weight(a[4], "q_weight", q);
    const void* kw = two ? head_weight(a[5], "k_weight", k) : nullptr;
    const nf_rope r = rope_of(a[6], a[7], a[9], a[10], q, false);
    if (given(a[11])) dq = heads_like(a[11], "dq", q, "q", true);
    if (given(a[12])) dk = heads_like(a[12], "dk", k, "k", true);
    const float eps = static_cast<float>(number(a[8]));
    Tensor ws, dqw, dkw;
    if (given(a[13])) {
        ws = tensor(a[13], "workspace");
        need_on(ws, "workspace", dev);
    }
    nf_status st;
    {
        const WithoutInterpreter w;
        make_outputs(q, dq, two, k, dk);
        Together weights(dev);
        weights.want({q.dim}, at::kFloat);
        if (two) weights.want({q.dim}, at::kFloat);
        dqw = weights.take({q.dim}, at::kFloat);
        if (two) dkw = weights.take({q.dim}, at::kFloat);
        // freed right after the launches, as in embedding_bwd
        if (!ws.defined()) {
            const int64_t need = static_cast<int64_t>(nf_qk_rmsnorm_rope_bwd_workspace_size(q.dim));
            ws = empty({need > 16 ? need : 16}, at::kByte, dev);
        }
        st = nf_qk_rmsnorm_rope_bwd(&dq.h, static_cast<float*>(dqw.data_ptr()), &dqo.h, &q.h, qw, two ? &dk.h : nullptr,
                                    two ? static_cast<float*>(dkw.data_ptr()) : nullptr, two ? &dko.h : nullptr, two ? &k.h : nullptr, kw,
                                    type_of(q.t), q.batch, q.tokens, q.dim, eps, &r, ws.data_ptr(), ws.nbytes(), stream_of(dev));
    }
    if (st != NF_OK) return status(st);
    return pack({object(a[11], dq.t), two ? object(a[12], dk.t) : none(), THPVariable_Wrap(dqw), two ? THPVariable_Wrap(dkw) : none()});
    END_HANDLE_TH_ERRORS
}

const int32_t* int32s(PyObject* o, const char* name, int dev, int64_t size) {
    const Tensor& t = tensor(o, name);
    need_type(t, name, at::kInt);
    need_on(t, name, dev);
    TORCH_CHECK_VALUE(t.dim() == 1 && t.size(0) == size, name, " must be of shape [", size, "]");
    return static_cast<const int32_t*>(t.const_data_ptr());
}

// A cache [pages, page_size, heads, head_dim] in any order, and its scales.
nf_pages pages_of(PyObject* o, const char* name, PyObject* scale, const char* scale_name, bool scaled, int dev) {
    const Tensor& t = tensor(o, name);
    need_on(t, name, dev, false);
    TORCH_CHECK_VALUE(t.dim() == 4 && (t.size(3) <= 1 || t.stride(3) == 1), name,
                      " must be [pages, page_size, heads, head_dim] with contiguous heads");
    nf_pages c{};
    c.data = t.numel() ? t.data_ptr() : nullptr;
    c.page_stride = t.stride(0), c.slot_stride = t.stride(1), c.head_stride = t.stride(2);
    TORCH_CHECK_VALUE(scaled == given(scale), scale_name, scaled ? " must be given for an 8-bit cache" : " is for an 8-bit cache only");
    if (!scaled) return c;
    const Tensor& s = tensor(scale, scale_name);
    need_type(s, scale_name, at::kFloat);
    need_on(s, scale_name, dev, false);
    TORCH_CHECK_VALUE(s.sizes() == t.sizes().slice(0, 3), scale_name, " must be [pages, page_size, heads]");
    c.scale = s.numel() ? static_cast<float*>(s.data_ptr()) : nullptr;
    c.scale_page_stride = s.stride(0), c.scale_slot_stride = s.stride(1), c.scale_head_stride = s.stride(2);
    return c;
}

// (k, v, k_cache, v_cache, table, past, starts or None, rates or None, positions or None, q or None, q_weight or None,
//  k_weight or None, eps, layout, magnitude, k_scale or None, v_scale or None, q_out or None) -> q_out or None
PyObject* kv_append(PyObject*, PyObject* const* a, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    count(n, 18);
    const Tensor& kt = tensor(a[0], "k");
    need_head_type(kt, "k");
    const int dev = device_of(kt, "k");
    TORCH_CHECK_VALUE(kt.dim() == 3, "k must be [tokens, heads, head_dim]");
    const Heads k = heads_of(kt, "k", dev), v = heads_like(a[1], "v", k, "k", true);
    const Tensor &kc = tensor(a[2], "k_cache"), &vc = tensor(a[3], "v_cache");
    const ScalarType cell = kc.scalar_type();
    const bool scaled = cell == at::kFloat8_e4m3fn || cell == at::kChar;
    TORCH_CHECK_TYPE(scaled || cell == kt.scalar_type(), "k_cache must be of k's type, torch.float8_e4m3fn or torch.int8, got ", cell);
    need_type(vc, "v_cache", cell);
    const nf_pages kp = pages_of(a[2], "k_cache", a[15], "k_scale", scaled, dev), vp = pages_of(a[3], "v_cache", a[16], "v_scale", scaled, dev);
    TORCH_CHECK_VALUE(kc.sizes() == vc.sizes() && kc.size(2) == k.h.heads && kc.size(3) == k.dim, "caches of shapes ", kc.sizes(), " and ",
                      vc.sizes(), " do not go with k of shape ", kt.sizes());
    TORCH_CHECK_VALUE(kc.size(1) >= 1 && kc.size(1) <= 0x7FFFFFFF, "a page must have slots");
    const Tensor& table = tensor(a[4], "table");
    need_type(table, "table", at::kInt);
    need_on(table, "table", dev, false);
    TORCH_CHECK_VALUE(table.dim() == 2 && (table.size(1) <= 1 || table.stride(1) == 1) && table.size(1) <= 0x7FFFFFFF,
                      "table must be [seqs, max_pages] with contiguous rows");
    const int64_t seqs = table.size(0);
    const int32_t* past = int32s(a[5], "past", dev, seqs);
    const int32_t* starts = given(a[6]) ? int32s(a[6], "starts", dev, seqs + 1) : nullptr;
    const nf_rope r = rope_of(a[8], a[7], a[13], a[14], k, true);
    const bool queries = given(a[9]);
    Heads q, qo;
    const void *qw = nullptr, *kw = nullptr;
    if (queries) {
        q = heads_like(a[9], "q", k, "k", false);
        if (given(a[10])) qw = head_weight(a[10], "q_weight", q);
        if (given(a[17])) qo = heads_like(a[17], "q_out", q, "q", true);
    }
    TORCH_CHECK_VALUE(queries || (!given(a[10]) && !given(a[17])), "q_weight or q_out is given without q");
    if (given(a[11])) kw = head_weight(a[11], "k_weight", k);
    const float eps = static_cast<float>(number(a[12]));
    nf_status st;
    {
        const WithoutInterpreter w;
        if (queries) make_outputs(q, qo, false, q, qo);
        st = nf_kv_append(&kp, &vp, cell == at::kChar ? NF_CACHE_INT8 : scaled ? NF_CACHE_E4M3 : NF_CACHE_SAME, kc.size(0),
                          static_cast<int32_t>(kc.size(1)), &k.h, &v.h, kw, queries ? &qo.h : nullptr, queries ? &q.h : nullptr, qw, type_of(k.t),
                          k.tokens, seqs, k.dim, starts, past, static_cast<const int32_t*>(table.const_data_ptr()),
                          seqs > 1 ? table.stride(0) : table.size(1), static_cast<int32_t>(table.size(1)), eps, &r, stream_of(dev));
    }
    if (st != NF_OK) return status(st);
    return queries ? object(a[17], qo.t) : none();
    END_HANDLE_TH_ERRORS
}

#define NF_FUNCTION(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {NF_FUNCTION(norm_q8),           NF_FUNCTION(embedding_fwd),     NF_FUNCTION(embedding_bwd),
                         NF_FUNCTION(token_logprob_fwd), NF_FUNCTION(token_logprob_bwd), NF_FUNCTION(rope),
                         NF_FUNCTION(qk_rmsnorm_rope_fwd), NF_FUNCTION(qk_rmsnorm_rope_bwd), NF_FUNCTION(kv_append), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", "Tensor helpers of the token-side operators and of those on attention heads.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors() { return PyModule_Create(&module); }
