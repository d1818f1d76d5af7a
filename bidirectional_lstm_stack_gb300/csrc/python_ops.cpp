// The calls of binding.py's functions of lstm_ops.h and lstm_layers.h on torch tensors: what a call's
// sizes promise is checked here (the C entry points take sizes and strides on
// trust), outputs that are not given are allocated for the stream that the call
// runs on, and everything else is the library's.  Small calls last longer on the
// host than on the GPU, which is why these are not ctypes calls: a convolution step
// of one sequence takes 4.5 us (15.6 through ctypes), a scan step 5.7 (25), a norm
// with three outputs 8.7 (25), while their kernels take 2.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <optional>

#include "lstm_layers.h"

namespace {

using at::Tensor;

PyObject *g_error = nullptr;  // binding.LSTMError

// ---- arguments -----------------------------------------------------------------
// The functions take exactly their parameters, in the order of binding.py's, null
// here for those that are None.
template <int N>
struct Arguments {
    PyObject *at[N];

    Arguments(PyObject *const *args, Py_ssize_t count)
    {
        TORCH_CHECK_TYPE(count == N, count, " arguments, expected ", N);
        for (int i = 0; i < N; ++i)
            at[i] = args[i] == Py_None ? nullptr : args[i];
    }
    PyObject *operator[](int i) const { return at[i]; }
};

bool truth(PyObject *o, bool otherwise)
{
    if (!o)
        return otherwise;
    const int v = PyObject_IsTrue(o);
    if (v < 0)
        throw python_error();
    return v != 0;
}
int64_t number(PyObject *o, int64_t otherwise)
{
    if (!o)
        return otherwise;
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred())
        throw python_error();
    return v;
}
// A size as the C entry points take it.
int as_int(const char *name, int64_t v)
{
    TORCH_CHECK_VALUE(v >= INT_MIN && v <= INT_MAX, name, " is ", v, ", beyond 32 bits");
    return static_cast<int>(v);
}

const Tensor *optional_tensor(const char *name, PyObject *o)
{
    if (!o)
        return nullptr;
    TORCH_CHECK_TYPE(THPVariable_Check(o), name, " is no tensor");
    const Tensor &t = THPVariable_Unpack(o);
    // forward only: an output without a gradient would pass unnoticed
    TORCH_CHECK_VALUE(!t.requires_grad() || !c10::GradMode::is_enabled(), name,
                      " requires a gradient, which these operators do not have: detach it, or call "
                      "them under torch.no_grad()");
    return &t;
}
const Tensor &tensor(const char *name, PyObject *o)
{
    TORCH_CHECK_TYPE(o, name, " is None, expected a tensor");
    return *optional_tensor(name, o);
}

// ---- checks ----------------------------------------------------------------------
int element_type(const Tensor &t)
{
    switch (t.scalar_type()) {
    case at::kFloat:
        return LSTM_F32;
    case at::kBFloat16:
        return LSTM_BF16;
    case at::kHalf:
        return LSTM_F16;
    default:
        TORCH_CHECK_VALUE(false, "element type ", t.scalar_type(),
                          ", expected float32, bfloat16 or float16");
    }
}

// The matrix that gives a call its sizes.
struct Rows {
    const Tensor &t;
    int64_t rows, cols;
    at::ScalarType type;
    at::Device device;

    Rows(const char *name, const Tensor &m, int dims = 2)
        : t(m), rows(0), cols(0), type(m.scalar_type()), device(m.device())
    {
        TORCH_CHECK_VALUE(m.dim() == dims, name, " has shape ", m.sizes(), ", expected ",
                          dims == 2 ? "two" : "three", " dimensions");
        TORCH_CHECK_VALUE(device.is_cuda(), name, " is on ", device, ", expected a CUDA device");
        rows = m.size(0);
        cols = m.size(1);
    }
};

// Row stride of a matrix of the given size and type on r's device.
long long matrix(const char *name, const Tensor &m, int64_t rows, int64_t cols, at::ScalarType type,
                 const Rows &r)
{
    TORCH_CHECK_VALUE(m.dim() == 2 && m.size(0) == rows && m.size(1) == cols &&
                          m.scalar_type() == type && m.device() == r.device,
                      name, " is ", m.scalar_type(), " ", m.sizes(), " on ", m.device(),
                      ", expected ", type, " [", rows, ", ", cols, "] on ", r.device);
    TORCH_CHECK_VALUE(cols <= 1 || m.stride(1) == 1, name,
                      " needs consecutive columns, has stride ", m.stride(1), " between them");
    return m.stride(0);
}

// Address of a densely packed tensor, null for none.
void *dense(const char *name, const Tensor *m, at::IntArrayRef shape, at::ScalarType type,
            const Rows &r)
{
    if (!m)
        return nullptr;
    TORCH_CHECK_VALUE(m->sizes() == shape && m->scalar_type() == type && m->device() == r.device &&
                          m->is_contiguous(),
                      name, " is ", m->scalar_type(), " ", m->sizes(), " on ", m->device(),
                      ", expected densely packed ", type, " ", shape, " on ", r.device);
    return m->data_ptr();
}
const float *weights(const char *name, PyObject *o, at::IntArrayRef shape, const Rows &r)
{
    return static_cast<const float *>(dense(name, optional_tensor(name, o), shape, at::kFloat, r));
}
const int *indices(const char *name, PyObject *o, int64_t count, const Rows &r)
{
    return static_cast<const int *>(dense(name, optional_tensor(name, o), {count}, at::kInt, r));
}

// The last dimension of a weight, which some size of the call comes from.
int64_t last_size(const char *name, const Tensor &t)
{
    TORCH_CHECK_VALUE(t.dim() > 0, name, " has no dimensions");
    return t.size(-1);
}

// The states' arguments.
struct State {
    void *at = nullptr;
    int count = 0;
    const int *slots = nullptr;
    const int *resume = nullptr;

    State(PyObject *state, PyObject *slots_o, PyObject *resume_o, at::IntArrayRef inner,
          at::ScalarType type, int64_t sequences, const Rows &r)
    {
        const Tensor *t = optional_tensor("state", state);
        if (!t) {
            TORCH_CHECK_VALUE(!slots_o && !resume_o, "slots and resume need a state");
            return;
        }
        const int64_t n = t->dim() > 0 ? t->size(0) : 0;
        TORCH_CHECK_VALUE(slots_o || n >= sequences, sequences, " sequences without slots, a state of ",
                          n);
        int64_t shape[4] = {n};
        std::copy(inner.begin(), inner.end(), shape + 1);
        at = dense("state", t, {shape, inner.size() + 1}, type, r);
        count = as_int("state's slots", n);
        slots = indices("slots", slots_o, sequences, r);
        resume = indices("resume", resume_o, sequences, r);
    }
};

// Number of sequences and where they start.
struct Prompts {
    int64_t count;
    const int *offsets = nullptr;

    Prompts(PyObject *sequences, PyObject *offsets_o, const Rows &r) : count(number(sequences, 1))
    {
        if (!offsets_o)
            return;
        const int64_t n = tensor("offsets", offsets_o).numel() - 1;
        TORCH_CHECK_VALUE(!sequences || count == n, count, " sequences, offsets for ", n);
        count = n;
        offsets = indices("offsets", offsets_o, n + 1, r);
    }
};

// The stream that a call runs on, and outputs allocated for it.
struct Stream {
    cudaStream_t at;
    bool given;
    at::Device device;

    Stream(PyObject *o, const Rows &r) : given(o != nullptr), device(r.device)
    {
        if (!o) {
            at = c10::cuda::getCurrentCUDAStream(device.index()).stream();
            return;
        }
        PyObject *handle = PyLong_Check(o) ? Py_NewRef(o) : PyObject_GetAttrString(o, "cuda_stream");
        if (!handle)
            throw python_error();
        at = static_cast<cudaStream_t>(PyLong_AsVoidPtr(handle));
        Py_DECREF(handle);
        if (PyErr_Occurred())
            throw python_error();
    }
    Tensor empty(at::IntArrayRef shape, at::ScalarType type) const
    {
        std::optional<c10::cuda::CUDAStreamGuard> guard;
        if (given)
            guard.emplace(c10::cuda::getStreamFromExternal(at, device.index()));
        return at::empty(shape, at::TensorOptions().dtype(type).device(device));
    }
    // A given output, or a new one.
    Tensor output(const char *name, PyObject *o, at::IntArrayRef shape, at::ScalarType type) const
    {
        const Tensor *t = optional_tensor(name, o);
        return t ? *t : empty(shape, type);
    }
};

// The library's call, without the interpreter's lock (a launch waits when the
// stream's queue is full); its errors are Python's after it.
template <typename F, typename... As>
void call(F function, As... as)
{
    PyThreadState *thread = PyEval_SaveThread();
    const int status = function(as...);
    PyEval_RestoreThread(thread);
    if (status == LSTM_OK)
        return;
    PyObject *e = PyObject_CallFunction(g_error, "is", status, lstm_stack_last_error());
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw python_error();
}

// Tells autograd that the tensor of this argument, if it was given, has been
// overwritten.  (Tensors of inference mode have no count of that.)
void written(PyObject *o)
{
    if (!o)
        return;
    const Tensor &t = THPVariable_Unpack(o);
    if (!t.is_inference())
        t.unsafeGetTensorImpl()->bump_version();
}

PyObject *wrap(const Tensor &t) { return THPVariable_Wrap(t); }
PyObject *wrap(const std::optional<Tensor> &t)
{
    return t ? THPVariable_Wrap(*t) : Py_NewRef(Py_None);
}
template <typename... Ts>
PyObject *wrap_all(const Ts &...ts)
{
    PyObject *tuple = PyTuple_New(sizeof...(ts));
    if (!tuple)
        throw python_error();
    Py_ssize_t i = 0;
    (PyTuple_SET_ITEM(tuple, i++, wrap(ts)), ...);
    return tuple;
}

// ---- the functions -----------------------------------------------------------------
PyObject *causal_conv(PyObject *, PyObject *const *args, Py_ssize_t count)
{
    HANDLE_TH_ERRORS
    const Arguments<11> v(args, count);
    const Rows x("x", tensor("x", v[0]));
    const int type = element_type(x.t);
    const int64_t width = last_size("w", tensor("w", v[1]));
    const Prompts p(v[4], v[5], x);
    const State state(v[6], v[7], v[8], {width - 1, x.cols}, x.type, p.count, x);
    const long long x_stride = matrix("x", x.t, x.rows, x.cols, x.type, x);
    const float *w = weights("w", v[1], {x.cols, width}, x);
    const float *bias = weights("bias", v[2], {x.cols}, x);
    const Stream stream(v[10], x);
    const Tensor y = stream.output("y", v[9], {x.rows, x.cols}, x.type);
    call(lstm_causal_conv, x.t.data_ptr(), x_stride, type, as_int("tokens", x.rows),
                           as_int("channels", x.cols), as_int("width", width), w, bias,
                           truth(v[3], true), as_int("sequences", p.count), p.offsets, state.at,
                           state.count, state.slots, state.resume, y.data_ptr(),
                           matrix("y", y, x.rows, x.cols, x.type, x), stream.at);
    written(v[6]);
    written(v[9]);
    return wrap(y);
    END_HANDLE_TH_ERRORS
}

PyObject *causal_conv_step(PyObject *, PyObject *const *args, Py_ssize_t count)
{
    HANDLE_TH_ERRORS
    const Arguments<8> v(args, count);
    const Rows x("x", tensor("x", v[0]));
    const int type = element_type(x.t);
    const int64_t width = last_size("w", tensor("w", v[1]));
    const State state(v[3], v[5], nullptr, {width - 1, x.cols}, x.type, x.rows, x);
    const long long x_stride = matrix("x", x.t, x.rows, x.cols, x.type, x);
    const float *w = weights("w", v[1], {x.cols, width}, x);
    const float *bias = weights("bias", v[2], {x.cols}, x);
    const Stream stream(v[7], x);
    const Tensor y = stream.output("y", v[6], {x.rows, x.cols}, x.type);
    call(lstm_causal_conv_step, x.t.data_ptr(), x_stride, type, as_int("sequences", x.rows),
                                as_int("channels", x.cols), as_int("width", width), w, bias,
                                truth(v[4], true), state.at, state.count, state.slots,
                                y.data_ptr(), matrix("y", y, x.rows, x.cols, x.type, x), stream.at);
    written(v[3]);
    written(v[6]);
    return wrap(y);
    END_HANDLE_TH_ERRORS
}

// What both scan functions begin with.
struct Scan {
    const Tensor &dt, &b, &c;
    const Tensor *z;
    int64_t states, groups;
    long long u_stride, dt_stride, b_stride, c_stride, z_stride = 0;
    const float *a, *skip, *dt_bias;

    Scan(const Rows &u, PyObject *dt_o, PyObject *a_o, PyObject *b_o, PyObject *c_o, PyObject *skip_o,
         PyObject *z_o, PyObject *dt_bias_o, PyObject *groups_o)
        : dt(tensor("dt", dt_o)), b(tensor("b", b_o)), c(tensor("c", c_o)),
          z(optional_tensor("z", z_o)), states(last_size("a", tensor("a", a_o))),
          groups(number(groups_o, 1))
    {
        u_stride = matrix("u", u.t, u.rows, u.cols, u.type, u);
        dt_stride = matrix("dt", dt, u.rows, u.cols, u.type, u);
        b_stride = matrix("b", b, u.rows, groups * states, u.type, u);
        c_stride = matrix("c", c, u.rows, groups * states, u.type, u);
        if (z)
            z_stride = matrix("z", *z, u.rows, u.cols, u.type, u);
        a = weights("a", a_o, {u.cols, states}, u);
        skip = weights("skip", skip_o, {u.cols}, u);
        dt_bias = weights("dt_bias", dt_bias_o, {u.cols}, u);
    }
    const void *z_at() const { return z ? z->data_ptr() : nullptr; }
};

PyObject *selective_scan(PyObject *, PyObject *const *args, Py_ssize_t count)
{
    HANDLE_TH_ERRORS
    const Arguments<17> v(args, count);
    const Rows u("u", tensor("u", v[0]));
    const int type = element_type(u.t);
    const Scan s(u, v[1], v[2], v[3], v[4], v[5], v[6], v[7], v[9]);
    const Prompts p(v[10], v[11], u);
    const State state(v[12], v[13], v[14], {u.cols, s.states}, at::kFloat, p.count, u);
    const Stream stream(v[16], u);
    const Tensor y = stream.output("y", v[15], {u.rows, u.cols}, u.type);
    const int tokens = as_int("tokens", u.rows), channels = as_int("channels", u.cols),
              states = as_int("states", s.states), groups = as_int("groups", s.groups),
              sequences = as_int("sequences", p.count);
    const size_t bytes =
        lstm_selective_scan_workspace(tokens, channels, states, groups, sequences, !p.offsets);
    Tensor workspace;
    if (bytes)
        workspace = stream.empty({static_cast<int64_t>(bytes)}, at::kByte);
    call(lstm_selective_scan, u.t.data_ptr(), s.u_stride, s.dt.data_ptr(), s.dt_stride, s.a, s.b.data_ptr(), s.b_stride,
        s.c.data_ptr(), s.c_stride, s.skip, s.z_at(), s.z_stride, s.dt_bias, truth(v[8], true),
        type, tokens, channels, states, groups, sequences, p.offsets,
        static_cast<float *>(state.at), state.count, state.slots, state.resume, y.data_ptr(),
        matrix("y", y, u.rows, u.cols, u.type, u), bytes ? workspace.data_ptr() : nullptr, bytes,
        stream.at);
    written(v[12]);
    written(v[15]);
    return wrap(y);
    END_HANDLE_TH_ERRORS
}

PyObject *selective_scan_step(PyObject *, PyObject *const *args, Py_ssize_t count)
{
    HANDLE_TH_ERRORS
    const Arguments<14> v(args, count);
    const Rows u("u", tensor("u", v[0]));
    const int type = element_type(u.t);
    const Scan s(u, v[1], v[2], v[3], v[4], v[6], v[7], v[8], v[10]);
    const State state(v[5], v[11], nullptr, {u.cols, s.states}, at::kFloat, u.rows, u);
    const Stream stream(v[13], u);
    const Tensor y = stream.output("y", v[12], {u.rows, u.cols}, u.type);
    call(lstm_selective_scan_step, u.t.data_ptr(), s.u_stride, s.dt.data_ptr(), s.dt_stride, s.a, s.b.data_ptr(), s.b_stride,
        s.c.data_ptr(), s.c_stride, s.skip, s.z_at(), s.z_stride, s.dt_bias, truth(v[9], true),
        type, as_int("sequences", u.rows), as_int("channels", u.cols), as_int("states", s.states),
        as_int("groups", s.groups), static_cast<float *>(state.at), state.count, state.slots,
        y.data_ptr(), matrix("y", y, u.rows, u.cols, u.type, u), stream.at);
    written(v[5]);
    written(v[12]);
    return wrap(y);
    END_HANDLE_TH_ERRORS
}

PyObject *residual_rms_norm(PyObject *, PyObject *const *args, Py_ssize_t count)
{
    HANDLE_TH_ERRORS
    const Arguments<10> v(args, count);
    const Rows x("x", tensor("x", v[0]));
    const int type = element_type(x.t);
    TORCH_CHECK_TYPE(v[2], "eps is None");
    const double eps = PyFloat_AsDouble(v[2]);
    if (eps == -1.0 && PyErr_Occurred())
        throw python_error();
    const bool quantize = truth(v[5], false);
    const int group = as_int("group", number(v[6], 0));
    const Tensor *residual = optional_tensor("residual", v[3]);
    TORCH_CHECK_VALUE(residual || !v[4], "residual_out without a residual");
    const at::ScalarType y_type = quantize ? at::kFloat8_e4m3fn : x.type;
    const long long x_stride = matrix("x", x.t, x.rows, x.cols, x.type, x);
    const long long res_stride = residual ? matrix("residual", *residual, x.rows, x.cols, x.type, x) : 0;
    const float *weight = weights("weight", v[1], {x.cols}, x);
    const Stream stream(v[9], x);
    std::optional<Tensor> res_out, scales;
    long long out_stride = 0;
    if (residual) {
        res_out = stream.output("residual_out", v[4], {x.rows, x.cols}, x.type);
        out_stride = matrix("residual_out", *res_out, x.rows, x.cols, x.type, x);
    }
    const Tensor y = stream.output("y", v[7], {x.rows, x.cols}, y_type);
    float *scales_at = nullptr;
    if (quantize) {
        const int64_t shape[2] = {x.rows, group > 0 ? (x.cols + group - 1) / group : 1};
        scales = stream.output("scales", v[8], shape, at::kFloat);
        scales_at = static_cast<float *>(dense("scales", &*scales, shape, at::kFloat, x));
    }
    call(lstm_residual_rms_norm, x.t.data_ptr(), x_stride, residual ? residual->data_ptr() : nullptr, res_stride, type, weight,
        static_cast<float>(eps), as_int("rows", x.rows), as_int("columns", x.cols),
        res_out ? res_out->data_ptr() : nullptr, out_stride, y.data_ptr(),
        matrix("y", y, x.rows, x.cols, y_type, x), quantize ? static_cast<int>(LSTM_E4M3) : type,
        scales_at, group, stream.at);
    if (residual)
        written(v[4]);
    written(v[7]);
    if (quantize)
        written(v[8]);
    return wrap_all(std::optional<Tensor>(y), scales, res_out);
    END_HANDLE_TH_ERRORS
}

PyObject *token_logprobs(PyObject *, PyObject *const *args, Py_ssize_t count)
{
    HANDLE_TH_ERRORS
    const Arguments<5> v(args, count);
    const Rows x("logits", tensor("logits", v[0]));
    const int type = element_type(x.t);
    const long long stride = matrix("logits", x.t, x.rows, x.cols, x.type, x);
    const Tensor *tokens = optional_tensor("tokens", v[1]);
    const auto *tokens_at =
        static_cast<const long long *>(dense("tokens", tokens, {x.rows}, at::kLong, x));
    const int top = as_int("top", number(v[2], 0));
    const Stream stream(v[4], x);
    std::optional<Tensor> logp, entropy, top_logp, top_ids;
    if (tokens)
        logp = stream.empty({x.rows}, at::kFloat);
    if (truth(v[3], true))
        entropy = stream.empty({x.rows}, at::kFloat);
    if (top > 0 && top <= LSTM_TOP_MAX) {  // (more are refused, and may not fit)
        top_logp = stream.empty({x.rows, top}, at::kFloat);
        top_ids = stream.empty({x.rows, top}, at::kLong);
    }
    const auto floats = [](std::optional<Tensor> &t) {
        return t ? static_cast<float *>(t->data_ptr()) : nullptr;
    };
    call(lstm_token_logprobs, x.t.data_ptr(), stride, type, as_int("rows", x.rows),
                              as_int("logits of a row", x.cols), tokens_at, floats(logp),
                              floats(entropy), top, floats(top_logp),
                              top_ids ? static_cast<long long *>(top_ids->data_ptr()) : nullptr,
                              stream.at);
    return wrap_all(logp, entropy, top_logp, top_ids);
    END_HANDLE_TH_ERRORS
}

// Rows of heads [rows, heads, width]: consecutive widths, any strides between heads and rows.
struct Heads {
    const void *at;
    long long stride, head_stride;
    int count;

    Heads(const char *name, const Tensor &m, int64_t width, const Rows &r)
    {
        TORCH_CHECK_VALUE(m.dim() == 3 && m.size(0) == r.rows && m.size(2) == width &&
                              m.scalar_type() == r.type && m.device() == r.device,
                          name, " is ", m.scalar_type(), " ", m.sizes(), " on ", m.device(),
                          ", expected ", r.type, " [", r.rows, ", heads, ", width, "] on ", r.device);
        TORCH_CHECK_VALUE(width <= 1 || m.stride(2) == 1, name,
                          " needs consecutive numbers in a head, has stride ", m.stride(2),
                          " between them");
        at = m.data_ptr();
        stride = m.stride(0);
        head_stride = m.stride(1);
        count = as_int(name, m.size(1));
    }
};

// What both functions of linear attention begin with.
struct Attention {
    int64_t keys, values, heads;
    Heads q, k, v;
    const float *decay;
    long long decay_stride = 0;
    float scale;

    Attention(const Rows &r, PyObject *k_o, PyObject *v_o, PyObject *decay_o, PyObject *scale_o)
        : keys(r.t.size(2)), values(last_size("v", tensor("v", v_o))),
          heads(last_size("log_decay", tensor("log_decay", decay_o))), q("q", r.t, keys, r),
          k("k", tensor("k", k_o), keys, r), v("v", tensor("v", v_o), values, r)
    {
        const Tensor &d = tensor("log_decay", decay_o);
        if (d.dim() == 2) {
            decay_stride = matrix("log_decay", d, r.rows, heads, at::kFloat, r);
            decay = static_cast<const float *>(d.data_ptr());
        } else {
            decay = weights("log_decay", decay_o, {heads}, r);
        }
        TORCH_CHECK_TYPE(scale_o, "scale is None");
        const double s = PyFloat_AsDouble(scale_o);
        if (s == -1.0 && PyErr_Occurred())
            throw python_error();
        scale = static_cast<float>(s);
    }
    // Row stride of the outputs [rows, heads, values], a row's heads consecutive.
    long long y_stride(const Tensor &y, const Rows &r) const
    {
        const Heads h("y", y, values, r);
        TORCH_CHECK_VALUE(h.count == heads && (heads <= 1 || h.head_stride == values), "y is ",
                          y.sizes(), " with heads ", h.head_stride, " apart, expected ", heads,
                          " consecutive heads of ", values);
        return h.stride;
    }
};

PyObject *linear_attention(PyObject *, PyObject *const *args, Py_ssize_t count)
{
    HANDLE_TH_ERRORS
    const Arguments<12> v(args, count);
    const Rows q("q", tensor("q", v[0]), 3);
    const int type = element_type(q.t);
    const Attention a(q, v[1], v[2], v[3], v[4]);
    const Prompts p(v[5], v[6], q);
    const State state(v[7], v[8], v[9], {a.heads, a.keys, a.values}, at::kFloat, p.count, q);
    const Stream stream(v[11], q);
    const Tensor y = stream.output("y", v[10], {q.rows, a.heads, a.values}, q.type);
    const long long y_stride = a.y_stride(y, q);
    const int tokens = as_int("tokens", q.rows), heads = as_int("heads", a.heads),
              keys = as_int("keys", a.keys), values = as_int("values", a.values),
              sequences = as_int("sequences", p.count);
    const size_t bytes =
        lstm_linear_attention_workspace(tokens, heads, keys, values, sequences, !p.offsets);
    Tensor workspace;
    if (bytes)
        workspace = stream.empty({static_cast<int64_t>(bytes)}, at::kByte);
    call(lstm_linear_attention, a.q.at, a.q.stride, a.q.head_stride, a.q.count, a.k.at, a.k.stride,
         a.k.head_stride, a.k.count, a.v.at, a.v.stride, a.v.head_stride, a.v.count, a.decay,
         a.decay_stride, a.scale, type, tokens, heads, keys, values, sequences, p.offsets,
         static_cast<float *>(state.at), state.count, state.slots, state.resume, y.data_ptr(),
         y_stride, bytes ? workspace.data_ptr() : nullptr, bytes, stream.at);
    written(v[7]);
    written(v[10]);
    return wrap(y);
    END_HANDLE_TH_ERRORS
}

PyObject *linear_attention_step(PyObject *, PyObject *const *args, Py_ssize_t count)
{
    HANDLE_TH_ERRORS
    const Arguments<9> v(args, count);
    const Rows q("q", tensor("q", v[0]), 3);
    const int type = element_type(q.t);
    const Attention a(q, v[1], v[2], v[3], v[5]);
    const State state(v[4], v[6], nullptr, {a.heads, a.keys, a.values}, at::kFloat, q.rows, q);
    const Stream stream(v[8], q);
    const Tensor y = stream.output("y", v[7], {q.rows, a.heads, a.values}, q.type);
    const long long y_stride = a.y_stride(y, q);
    call(lstm_linear_attention_step, a.q.at, a.q.stride, a.q.head_stride, a.q.count, a.k.at,
         a.k.stride, a.k.head_stride, a.k.count, a.v.at, a.v.stride, a.v.head_stride, a.v.count,
         a.decay, a.decay_stride, a.scale, type, as_int("sequences", q.rows),
         as_int("heads", a.heads), as_int("keys", a.keys), as_int("values", a.values),
         static_cast<float *>(state.at), state.count, state.slots, y.data_ptr(), y_stride,
         stream.at);
    written(v[4]);
    written(v[7]);
    return wrap(y);
    END_HANDLE_TH_ERRORS
}

PyObject *dense_product(PyObject *, PyObject *const *args, Py_ssize_t count)
{
    HANDLE_TH_ERRORS
    const Arguments<7> v(args, count);
    const Rows x("x", tensor("x", v[0]));
    const int type = element_type(x.t);
    const long long x_stride = matrix("x", x.t, x.rows, x.cols, x.type, x);
    const Tensor &w = tensor("w", v[1]);
    const int64_t out = w.dim() > 0 ? w.size(0) : 0;
    const long long w_stride = matrix("w", w, out, x.cols, x.type, x);
    const float *bias = weights("bias", v[2], {out}, x);
    const Tensor *residual = optional_tensor("residual", v[4]);
    const long long residual_stride =
        residual ? matrix("residual", *residual, x.rows, out, x.type, x) : 0;
    const Stream stream(v[6], x);
    const Tensor y = stream.output("y", v[5], {x.rows, out}, x.type);
    const long long y_stride = matrix("y", y, x.rows, out, x.type, x);
    const int rows = as_int("rows", x.rows), in = as_int("columns of x", x.cols),
              columns = as_int("rows of w", out);
    const size_t bytes = lstm_dense_workspace(x.t.data_ptr(), x_stride, w.data_ptr(), w_stride,
                                              type, rows, in, columns);
    Tensor workspace;
    if (bytes)
        workspace = stream.empty({static_cast<int64_t>(bytes)}, at::kByte);
    call(lstm_dense, x.t.data_ptr(), x_stride, w.data_ptr(), w_stride, bias,
         as_int("activation", number(v[3], LSTM_ACT_NONE)), residual ? residual->data_ptr() : nullptr,
         residual_stride, type, rows, in, columns, y.data_ptr(), y_stride,
         bytes ? workspace.data_ptr() : nullptr, bytes, stream.at);
    written(v[5]);
    return wrap(y);
    END_HANDLE_TH_ERRORS
}

PyObject *set_error(PyObject *, PyObject *cls)
{
    Py_XSETREF(g_error, Py_NewRef(cls));
    Py_RETURN_NONE;
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)>
constexpr PyMethodDef method(const char *name)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(F)), METH_FASTCALL,
            nullptr};
}

PyMethodDef methods[] = {
    method<causal_conv>("causal_conv"),
    method<causal_conv_step>("causal_conv_step"),
    method<selective_scan>("selective_scan"),
    method<selective_scan_step>("selective_scan_step"),
    method<residual_rms_norm>("residual_rms_norm"),
    method<token_logprobs>("token_logprobs"),
    method<linear_attention>("linear_attention"),
    method<linear_attention_step>("linear_attention_step"),
    method<dense_product>("dense"),
    {"set_error", set_error, METH_O, "The class of the library's errors."},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native",
                      "The calls of binding.py's functions on torch tensors.",
                      -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__native() { return PyModule_Create(&module); }
