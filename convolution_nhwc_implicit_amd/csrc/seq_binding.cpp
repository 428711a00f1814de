// seq_binding.cpp -- the sequence operators as functions of torch tensors
// (module _sequence; sequence.py gives them their Python signatures).
//
// Checks of arguments, outputs and workspaces on the current stream, then the C
// ABI of sequence_ops.h.  A call of a few microseconds of GPU work would
// otherwise wait for its own argument handling: this takes about 4 us a call
// where ctypes and Python took 15 to 20.
//
// Types, shapes and strides are checked before the devices, so that a wrong call
// says what is wrong with it on any machine.
#include <ATen/ATen.h>
#include <ATen/core/grad_mode.h>
#include <ATen/hip/impl/HIPStreamMasqueradingAsCUDA.h>
#include <c10/core/DeviceGuard.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <string>

#include "sequence_ops.h"

namespace {

using at::Tensor;
using std::string;

[[noreturn]] void python_raise(PyObject *type, const string &m)
{
    PyErr_SetString(type, m.c_str());
    throw python_error();
}
[[noreturn]] void value_error(const string &m) { python_raise(PyExc_ValueError, m); }
[[noreturn]] void type_error(const string &m) { python_raise(PyExc_TypeError, m); }

string shape_text(at::IntArrayRef s)
{
    string r = "(";
    for (size_t i = 0; i < s.size(); ++i) r += (i ? ", " : "") + std::to_string(s[i]);
    return r + (s.size() == 1 ? ",)" : ")");
}
string type_text(at::ScalarType t)
{
    switch (t) {
        case at::kHalf: return "torch.float16";
        case at::kBFloat16: return "torch.bfloat16";
        case at::kFloat: return "torch.float32";
        case at::kInt: return "torch.int32";
        case at::kFloat8_e4m3fn: return "torch.float8_e4m3fn";
        default: return c10::toString(t);
    }
}

const Tensor *tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o)) type_error(string(name) + " must be a torch.Tensor");
    return &THPVariable_Unpack(o);
}
const Tensor *maybe(PyObject *o, const char *name) { return o == Py_None ? nullptr : tensor(o, name); }

bool truth(PyObject *o)
{
    const int r = PyObject_IsTrue(o);
    if (r < 0) throw python_error();
    return r != 0;
}

int float_code(const Tensor &t, const char *name)
{
    switch (t.scalar_type()) {
        case at::kHalf: return CONV2D_DTYPE_F16;
        case at::kBFloat16: return CONV2D_DTYPE_BF16;
        case at::kFloat: return CONV2D_DTYPE_F32;
        default: type_error(string(name) + " must be float16, bfloat16 or float32, got " + type_text(t.scalar_type()));
    }
}

// Collects what the tensors have to be; device() looks at the devices last.
struct Checks {
    const Tensor *seen[16];
    const char *names[16];
    int count = 0;

    void strided(const Tensor &t, const char *name, at::ScalarType type, at::IntArrayRef shape)
    {
        if (t.scalar_type() != type)
            type_error(string(name) + " must be " + type_text(type) + ", got " + type_text(t.scalar_type()));
        if (t.layout() != at::kStrided) type_error(string(name) + " must be a dense tensor");
        if (t.sizes() != shape)
            value_error(string(name) + " must have shape " + shape_text(shape) + ", got " + shape_text(t.sizes()));
        if (t.size(-1) > 1 && t.stride(-1) != 1) value_error(string(name) + " must have unit stride over its last axis");
        seen[count] = &t;
        names[count++] = name;
    }
    void *dense(const Tensor *t, const char *name, at::ScalarType type, at::IntArrayRef shape)
    {
        if (!t) return nullptr;
        strided(*t, name, type, shape);
        if (!t->is_contiguous()) value_error(string(name) + " must be contiguous");
        return t->data_ptr();
    }
    void device(const Tensor &first) const
    {
        for (int i = 0; i < count; ++i) {
            if (!seen[i]->is_cuda()) value_error(string(names[i]) + " must be on the GPU, got " + seen[i]->device().str());
            if (seen[i]->device() != first.device())
                value_error(string(names[i]) + " must be on " + first.device().str() + ", got " + seen[i]->device().str());
        }
    }
    // Results carry no gradient history: a warning where a caller may expect one.
    void detached(const char *where, const char *instead) const
    {
        if (!at::GradMode::is_enabled()) return;
        for (int i = 0; i < count; ++i)
            if (seen[i]->requires_grad()) {
                const string m = string(where) + ": " + names[i] + " requires a gradient, but the result carries no gradient history; " + instead;
                if (PyErr_WarnEx(PyExc_UserWarning, m.c_str(), 2) < 0) throw python_error();
                return;
            }
    }
};

const void *ptr(const Tensor *t) { return t ? t->data_ptr() : nullptr; }
void *out_ptr(const Tensor &t) { return t.defined() ? t.data_ptr() : nullptr; }

// The device's current stream.
void *stream_of(const Tensor &t)
{
    return (void *)c10::hip::getCurrentHIPStreamMasqueradingAsCUDA(t.device().index()).stream();
}

// A step has written to it: what autograd saved of it before is not its value any more.
void written(const Tensor &t)
{
    if (!t.is_inference()) t.unsafeGetTensorImpl()->bump_version();
}

Tensor new_tensor(const Tensor &like, at::IntArrayRef shape, at::ScalarType type)
{
    return at::empty(shape, like.options().dtype(type).requires_grad(false));
}
Tensor workspace(const Tensor &like, size_t bytes)
{
    return bytes ? new_tensor(like, {(int64_t)bytes}, at::kByte) : Tensor();
}

PyObject *error_class = nullptr;  // Conv2dError

void raise(int status, const char *where)
{
    if (status == CONV2D_OK) return;
    PyObject *e = PyObject_CallFunction(error_class, "is", status, where);
    if (e) {
        PyErr_SetObject(error_class, e);
        Py_DECREF(e);
    }
    throw python_error();
}

PyObject *wrap(const Tensor &t)
{
    if (!t.defined()) Py_RETURN_NONE;
    return THPVariable_Wrap(t);
}

PyObject *pair(const Tensor &a, const Tensor &b)
{
    PyObject *t = PyTuple_New(2);
    if (!t) throw python_error();
    PyTuple_SET_ITEM(t, 0, wrap(a));
    PyTuple_SET_ITEM(t, 1, wrap(b));
    return t;
}

void set_item(PyObject *d, const char *key, const Tensor &t)
{
    PyObject *v = wrap(t);
    const int r = v ? PyDict_SetItemString(d, key, v) : -1;
    Py_XDECREF(v);
    if (r < 0) {
        Py_DECREF(d);
        throw python_error();
    }
}

// The sequences of tensors whose leading axes are t's without its last `inner`.
struct Lead {
    at::IntArrayRef shape;
    seq_batch_t batch;
    int64_t seqs;
    Lead(const Tensor &t, const Tensor *start, Checks &c)
    {
        if (t.dim() < 2 || t.dim() > 3) value_error("tokens must lie along one axis, or along two as [sequences][tokens]");
        shape = t.sizes().slice(0, t.dim() - 1);
        batch = {};
        int64_t tokens;
        if (start) {
            if (shape.size() != 1) value_error("with seq_start, tokens lie along one axis");
            if (start->dim() != 1 || start->size(0) < 2)
                value_error("seq_start must be a vector with an entry for every sequence and one more");
            c.strided(*start, "seq_start", at::kInt, start->sizes());
            seqs = start->size(0) - 1;
            tokens = shape[0];
            batch.seq_start = (const int *)start->data_ptr();
        } else {
            seqs = shape.size() == 2 ? shape[0] : 1;
            if (seqs < 1) value_error("there must be at least one sequence");
            if (shape.back() > INT32_MAX) value_error("a sequence has at most 2^31 - 1 tokens");
            tokens = seqs * shape.back();
            batch.len = (int)shape.back();
        }
        if (seqs > INT32_MAX) value_error("too many sequences");
        batch.seqs = (int)seqs;
        batch.tokens = tokens;
    }
    // strides over tokens and sequences; an axis of one element has any
    seq_stride_t strides(const Tensor &t) const
    {
        const size_t n = shape.size();
        return {shape[n - 1] > 1 ? t.stride(n - 1) : 0, n == 2 && shape[0] > 1 ? t.stride(0) : 0};
    }
};

long long row_stride(const Tensor &t) { return t.size(0) > 1 ? t.stride(0) : 0; }

int int_size(int64_t v, const char *what)
{
    if (v > INT32_MAX) value_error(string(what) + " is past 2^31 - 1");
    return (int)v;
}

const int *slots_of(const Tensor *slots, int64_t rows, int64_t pool, Checks &c)
{
    if (!slots) {
        if (rows > pool) value_error("without slots, state must have a place for every row");
        return nullptr;
    }
    c.strided(*slots, "slots", at::kInt, {rows});
    return (const int *)slots->data_ptr();
}

void expect_args(Py_ssize_t have, Py_ssize_t want)
{
    if (have != want) type_error("expected " + std::to_string(want) + " arguments, got " + std::to_string(have));
}

// ------------------------------------------------------------ causal convolution
struct Conv {
    Checks c;
    const Tensor *x, *weight, *bias, *initial;
    int code;
    causal_conv_problem_t p;
    int64_t d, w, seqs;
    Conv(PyObject *const *a)
    {
        x = tensor(a[0], "x");
        weight = tensor(a[1], "weight");
        bias = maybe(a[2], "bias");
        const bool silu = truth(a[3]);
        initial = maybe(a[4], "initial_state");
        const Tensor *start = maybe(a[5], "seq_start");
        code = float_code(*x, "x");
        const at::ScalarType type = x->scalar_type();
        if (x->dim() < 2) value_error("x must be [tokens][d] or [sequences][tokens][d]");
        if (weight->dim() != 2) value_error("weight must be [d][w]");
        d = x->size(-1);
        w = weight->size(1);
        c.strided(*x, "x", type, x->sizes());
        c.dense(weight, "weight", type, {d, w});
        c.dense(bias, "bias", type, {d});
        const Lead lead(*x, start, c);
        seqs = lead.seqs;
        if (w < 1) value_error("weight must have at least one tap");
        c.dense(initial, "initial_state", type, {seqs, w - 1, d});
        p = {lead.batch, int_size(d, "d"), int_size(w, "w"), silu, lead.strides(*x), {0, 0}};
    }
};

PyObject *py_causal_conv(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    expect_args(n, 7);
    Conv v(a);
    const bool state = truth(a[6]);
    v.c.device(*v.x);
    v.c.detached("causal_conv", "causal_conv_grad computes the gradients");
    const c10::DeviceGuard guard(v.x->device());
    const Tensor y = new_tensor(*v.x, v.x->sizes(), v.x->scalar_type());
    const Tensor f = state ? new_tensor(*v.x, {v.seqs, v.w - 1, v.d}, v.x->scalar_type()) : Tensor();
    raise(causal_conv(&v.p, v.code, ptr(v.x), ptr(v.weight), ptr(v.bias), ptr(v.initial), out_ptr(y), out_ptr(f),
                      stream_of(*v.x)), "causal_conv");
    return state ? pair(y, f) : wrap(y);
    END_HANDLE_TH_ERRORS
}

PyObject *py_causal_conv_grad(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    expect_args(n, 8);
    const Tensor *dy = tensor(a[0], "dy");
    Conv v(a + 1);
    const Tensor *dfinal = maybe(a[7], "dfinal_state");
    const at::ScalarType type = v.x->scalar_type();
    v.c.strided(*dy, "dy", type, v.x->sizes());
    v.c.dense(dfinal, "dfinal_state", type, {v.seqs, v.w - 1, v.d});
    const size_t lead = v.x->dim() - 1;
    v.p.dy = {dy->size(lead - 1) > 1 ? dy->stride(lead - 1) : 0, lead == 2 && dy->size(0) > 1 ? dy->stride(0) : 0};
    v.c.device(*v.x);
    const c10::DeviceGuard guard(v.x->device());
    size_t need = 0;
    raise(causal_conv_grad_workspace_size(&v.p, v.code, &need), "causal_conv_grad_workspace_size");
    const Tensor dx = new_tensor(*v.x, v.x->sizes(), type), dw = new_tensor(*v.x, v.weight->sizes(), type);
    const Tensor db = v.bias ? new_tensor(*v.x, {v.d}, type) : Tensor();
    const Tensor di = v.initial ? new_tensor(*v.x, v.initial->sizes(), type) : Tensor();
    const Tensor ws = workspace(*v.x, need);
    raise(causal_conv_grad(&v.p, v.code, ptr(dy), ptr(v.x), ptr(v.weight), ptr(v.bias), ptr(v.initial), ptr(dfinal),
                           out_ptr(dx), out_ptr(dw), out_ptr(db), out_ptr(di), out_ptr(ws), need, stream_of(*v.x)),
          "causal_conv_grad");
    PyObject *r = PyDict_New();
    if (!r) throw python_error();
    set_item(r, "dx", dx);
    set_item(r, "dw", dw);
    set_item(r, "db", db);
    set_item(r, "dinitial_state", di);
    return r;
    END_HANDLE_TH_ERRORS
}

PyObject *py_causal_conv_step(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    expect_args(n, 6);
    const Tensor *x = tensor(a[0], "x"), *state = tensor(a[1], "state"), *weight = tensor(a[2], "weight");
    const Tensor *bias = maybe(a[3], "bias"), *slots = maybe(a[5], "slots");
    const bool silu = truth(a[4]);
    const int code = float_code(*x, "x");
    if (x->dim() != 2 || weight->dim() != 2 || state->dim() != 3)
        value_error("x must be [rows][d], weight [d][w] and state [pool][w-1][d]");
    const at::ScalarType type = x->scalar_type();
    const int64_t rows = x->size(0), d = x->size(1), w = weight->size(1), pool = state->size(0);
    if (w < 1) value_error("weight must have at least one tap");
    Checks c;
    c.strided(*x, "x", type, x->sizes());
    c.dense(weight, "weight", type, {d, w});
    c.dense(bias, "bias", type, {d});
    c.dense(state, "state", type, {pool, w - 1, d});
    const int *sp = slots_of(slots, rows, pool, c);
    const causal_conv_step_problem_t p = {int_size(rows, "rows"), int_size(pool, "pool"), int_size(d, "d"),
                                          int_size(w, "w"), silu, row_stride(*x)};
    c.device(*x);
    c.detached("causal_conv_step", "causal_conv and causal_conv_grad compute prompts and their gradients");
    const c10::DeviceGuard guard(x->device());
    const Tensor y = new_tensor(*x, {rows, d}, type);
    raise(causal_conv_step(&p, code, ptr(x), state->data_ptr(), ptr(weight), ptr(bias), sp, out_ptr(y), stream_of(*x)),
          "causal_conv_step");
    written(*state);
    return wrap(y);
    END_HANDLE_TH_ERRORS
}

// ---------------------------------------------------------------- selective scan
struct Scan {
    Checks c;
    const Tensor *x, *dt, *A, *B, *C, *D, *z, *bias;
    int code;
    int64_t d, n, groups;
    // x, dt, A, B, C, D, z, dt_bias
    Scan(PyObject *const *a)
    {
        x = tensor(a[0], "x");
        dt = tensor(a[1], "dt");
        A = tensor(a[2], "A");
        B = tensor(a[3], "B");
        C = tensor(a[4], "C");
        D = maybe(a[5], "D");
        z = maybe(a[6], "z");
        bias = maybe(a[7], "dt_bias");
        code = float_code(*x, "x");
        const at::ScalarType type = x->scalar_type();
        if (x->dim() < 2 || A->dim() != 2 || B->dim() != x->dim() + 1)
            value_error("x must be [tokens][d] or [sequences][tokens][d], A [d][n] and B [tokens][groups][n] likewise");
        d = x->size(-1);
        n = A->size(1);
        groups = B->size(-2);
        c.strided(*x, "x", type, x->sizes());
        c.strided(*dt, "dt", type, x->sizes());
        c10::SmallVector<int64_t, 4> bc(x->sizes().begin(), x->sizes().end() - 1);
        bc.push_back(groups);
        bc.push_back(n);
        c.strided(*B, "B", type, bc);
        c.strided(*C, "C", type, bc);
        if (z) c.strided(*z, "z", type, x->sizes());
        c.dense(A, "A", at::kFloat, {d, n});
        c.dense(D, "D", at::kFloat, {d});
        c.dense(bias, "dt_bias", at::kFloat, {d});
        if (groups < 1 || d % groups)
            value_error("the " + std::to_string(groups) + " groups of B must divide the " + std::to_string(d) + " channels");
    }
    long long group_stride(const Tensor &t) const { return groups > 1 ? t.stride(-2) : 0; }
};

struct ScanTokens : Scan {
    const Tensor *initial;
    selective_scan_problem_t p;
    int64_t seqs;
    // x .. dt_bias, softplus, initial_state, seq_start
    ScanTokens(PyObject *const *a) : Scan(a)
    {
        const bool soft = truth(a[8]);
        initial = maybe(a[9], "initial_state");
        const Lead lead(*x, maybe(a[10], "seq_start"), c);
        seqs = lead.seqs;
        c.dense(initial, "initial_state", at::kFloat, {seqs, d, n});
        p = {lead.batch, int_size(d, "d"), int_size(n, "n"), int_size(groups, "groups"), soft, lead.strides(*x),
             lead.strides(*dt), lead.strides(*B), lead.strides(*C), z ? lead.strides(*z) : seq_stride_t{0, 0}, {0, 0},
             group_stride(*B), group_stride(*C)};
    }
    static const float *f(const Tensor *t) { return (const float *)ptr(t); }
};

PyObject *py_selective_scan(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    expect_args(n, 12);
    ScanTokens v(a);
    const bool state = truth(a[11]);
    v.c.device(*v.x);
    v.c.detached("selective_scan", "selective_scan_grad computes the gradients");
    const c10::DeviceGuard guard(v.x->device());
    size_t need = 0;
    raise(selective_scan_workspace_size(&v.p, v.code, &need), "selective_scan_workspace_size");
    const Tensor y = new_tensor(*v.x, v.x->sizes(), v.x->scalar_type());
    const Tensor s = state ? new_tensor(*v.x, {v.seqs, v.d, v.n}, at::kFloat) : Tensor();
    const Tensor ws = workspace(*v.x, need);
    raise(selective_scan(&v.p, v.code, ptr(v.x), ptr(v.dt), v.f(v.A), ptr(v.B), ptr(v.C), v.f(v.D), ptr(v.z),
                         v.f(v.bias), v.f(v.initial), out_ptr(y), (float *)out_ptr(s), out_ptr(ws), need,
                         stream_of(*v.x)), "selective_scan");
    return state ? pair(y, s) : wrap(y);
    END_HANDLE_TH_ERRORS
}

PyObject *py_selective_scan_grad(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    expect_args(n, 13);
    const Tensor *dy = tensor(a[0], "dy");
    ScanTokens v(a + 1);
    const Tensor *dfinal = maybe(a[12], "dfinal_state");
    const at::ScalarType type = v.x->scalar_type();
    v.c.strided(*dy, "dy", type, v.x->sizes());
    v.c.dense(dfinal, "dfinal_state", at::kFloat, {v.seqs, v.d, v.n});
    const size_t lead = v.x->dim() - 1;
    v.p.dy = {dy->size(lead - 1) > 1 ? dy->stride(lead - 1) : 0, lead == 2 && dy->size(0) > 1 ? dy->stride(0) : 0};
    v.c.device(*v.x);
    const c10::DeviceGuard guard(v.x->device());
    size_t need = 0;
    raise(selective_scan_grad_workspace_size(&v.p, v.code, &need), "selective_scan_grad_workspace_size");
    auto like = [&](const Tensor *t) { return t ? new_tensor(*v.x, t->sizes(), t->scalar_type()) : Tensor(); };
    const Tensor du = like(v.x), ddt = like(v.dt), dA = like(v.A), dB = like(v.B), dC = like(v.C), dD = like(v.D);
    const Tensor dz = like(v.z), dbias = like(v.bias), di = like(v.initial);
    const Tensor ws = workspace(*v.x, need);
    const selective_scan_grads_t g = {out_ptr(du), out_ptr(ddt), (float *)out_ptr(dA), out_ptr(dB), out_ptr(dC),
                                      (float *)out_ptr(dD), out_ptr(dz), (float *)out_ptr(dbias), (float *)out_ptr(di)};
    raise(selective_scan_grad(&v.p, v.code, ptr(dy), ptr(v.x), ptr(v.dt), v.f(v.A), ptr(v.B), ptr(v.C), v.f(v.D),
                              ptr(v.z), v.f(v.bias), v.f(v.initial), v.f(dfinal), &g, out_ptr(ws), need,
                              stream_of(*v.x)), "selective_scan_grad");
    PyObject *r = PyDict_New();
    if (!r) throw python_error();
    set_item(r, "du", du);
    set_item(r, "ddt", ddt);
    set_item(r, "dA", dA);
    set_item(r, "dB", dB);
    set_item(r, "dC", dC);
    set_item(r, "dD", dD);
    set_item(r, "dz", dz);
    set_item(r, "ddt_bias", dbias);
    set_item(r, "dinitial_state", di);
    return r;
    END_HANDLE_TH_ERRORS
}

PyObject *py_selective_scan_step(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    expect_args(n, 11);
    Scan v(a);  // x, dt, A, B, C, D, z, dt_bias, then state, softplus, slots
    const Tensor *state = tensor(a[8], "state"), *slots = maybe(a[10], "slots");
    const bool soft = truth(a[9]);
    if (v.x->dim() != 2 || state->dim() != 3) value_error("x must be [rows][d] and state [pool][d][n]");
    const int64_t rows = v.x->size(0), pool = state->size(0);
    v.c.dense(state, "state", at::kFloat, {pool, v.d, v.n});
    const int *sp = slots_of(slots, rows, pool, v.c);
    const selective_scan_step_problem_t p = {
        int_size(rows, "rows"), int_size(pool, "pool"), int_size(v.d, "d"), int_size(v.n, "n"), int_size(v.groups, "groups"),
        soft, row_stride(*v.x), row_stride(*v.dt), row_stride(*v.B), row_stride(*v.C), v.z ? row_stride(*v.z) : 0,
        v.group_stride(*v.B), v.group_stride(*v.C)};
    v.c.device(*v.x);
    v.c.detached("selective_scan_step", "selective_scan and selective_scan_grad compute prompts and their gradients");
    const c10::DeviceGuard guard(v.x->device());
    const Tensor y = new_tensor(*v.x, {rows, v.d}, v.x->scalar_type());
    raise(selective_scan_step(&p, v.code, ptr(v.x), ptr(v.dt), (const float *)ptr(v.A), ptr(v.B), ptr(v.C),
                              (const float *)ptr(v.D), ptr(v.z), (const float *)ptr(v.bias), (float *)state->data_ptr(), sp,
                              out_ptr(y), stream_of(*v.x)), "selective_scan_step");
    written(*state);
    return wrap(y);
    END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------ block-scaled fp8 products
int64_t blocks_of(int64_t v) { return (v + 127) / 128; }

PyObject *py_fp8_quantize(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    expect_args(n, 3);
    const Tensor *x = tensor(a[0], "x");
    const bool transpose = truth(a[1]), blocks = truth(a[2]);
    const int code = float_code(*x, "x");
    if (x->dim() != 2) value_error("x must be [m][k]");
    if (transpose && blocks) value_error("blocks of 128 x 128 are quantised as they lie");
    Checks c;
    c.strided(*x, "x", x->scalar_type(), x->sizes());
    c.device(*x);
    c.detached("fp8_quantize", "rounding to 8 bits has none");
    const int64_t m = x->size(0), k = x->size(1), rows = transpose ? k : m, cols = transpose ? m : k;
    const int64_t pitch = (cols + 127) / 128 * 128;  // whole lines: rows that straddle them cost the products' loads
    const c10::DeviceGuard guard(x->device());
    const Tensor q = new_tensor(*x, {rows, pitch}, at::kFloat8_e4m3fn);
    const Tensor scale = new_tensor(*x, {blocks ? blocks_of(rows) : rows, blocks_of(cols)}, at::kFloat);
    raise(fp8_quantize(transpose ? FP8_TRANSPOSE : blocks ? FP8_BLOCKS : FP8_ROWS, code, int_size(m, "m"),
                       int_size(k, "k"), ptr(x), row_stride(*x), out_ptr(q), pitch, (float *)out_ptr(scale),
                       stream_of(*x)), "fp8_quantize");
    return pair(pitch == cols ? q : q.narrow(1, 0, cols), scale);
    END_HANDLE_TH_ERRORS
}

// An operand's row pitch; *blocks: whether its scales are of 128 rows together.
long long operand(const Tensor &q, const Tensor &scale, const char *name, const char *scale_name, bool *blocks, Checks &c)
{
    if (q.dim() != 2) value_error(string(name) + " must be a matrix");
    c.strided(q, name, at::kFloat8_e4m3fn, q.sizes());
    const int64_t rows = q.size(0), k = q.size(1);
    const bool by_block = blocks && scale.dim() == 2 && scale.size(0) != rows;
    c.dense(&scale, scale_name, at::kFloat, {by_block ? blocks_of(rows) : rows, blocks_of(k)});
    if (blocks) *blocks = by_block;
    const long long pitch = rows > 1 && k > 0 ? q.stride(0) : (k + 15) / 16 * 16;
    if (pitch % 16 || pitch < k)
        value_error(string(name) + "'s rows must start on 16-byte steps (fp8_quantize lays them out so)");
    return pitch;
}

PyObject *py_fp8_matmul(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    expect_args(n, 5);
    const Tensor *x = tensor(a[0], "a"), *xs = tensor(a[1], "a_scale"), *w = tensor(a[2], "b"), *ws = tensor(a[3], "b_scale");
    if (!THPDtype_Check(a[4])) type_error("out_dtype must be a torch.dtype");
    const at::ScalarType type = ((THPDtype *)a[4])->scalar_type;
    if (type != at::kHalf && type != at::kBFloat16 && type != at::kFloat)
        type_error("out_dtype must be float16, bfloat16 or float32, got " + type_text(type));
    Checks c;
    bool blocks = false;
    const long long xp = operand(*x, *xs, "a", "a_scale", nullptr, c), wp = operand(*w, *ws, "b", "b_scale", &blocks, c);
    if (w->size(1) != x->size(1))
        value_error("b must be [n][" + std::to_string(x->size(1)) + "], got " + shape_text(w->sizes()));
    c.device(*x);
    c.detached("fp8_matmul", "the gradients are products of the same kind");
    const fp8_matmul_problem_t p = {int_size(x->size(0), "m"), int_size(w->size(0), "n"), int_size(x->size(1), "k"), blocks, xp, wp};
    const int code = type == at::kHalf ? CONV2D_DTYPE_F16 : type == at::kBFloat16 ? CONV2D_DTYPE_BF16 : CONV2D_DTYPE_F32;
    const c10::DeviceGuard guard(x->device());
    size_t need = 0;
    raise(fp8_matmul_workspace_size(&p, code, &need), "fp8_matmul_workspace_size");
    const Tensor out = new_tensor(*x, {x->size(0), w->size(0)}, type), work = workspace(*x, need);
    raise(fp8_matmul(&p, code, ptr(x), (const float *)ptr(xs), ptr(w), (const float *)ptr(ws), out_ptr(out), out_ptr(work),
                     need, stream_of(*x)), "fp8_matmul");
    return wrap(out);
    END_HANDLE_TH_ERRORS
}

// ---------------------------------------------------------------- gated recurrence
struct Recur {
    Checks c;
    const Tensor *x, *r, *i, *A, *z, *r_bias, *i_bias;
    int code;
    int64_t d;
    // x, r, i, A, z, r_bias, i_bias
    Recur(PyObject *const *a)
    {
        x = tensor(a[0], "x");
        r = tensor(a[1], "r");
        i = tensor(a[2], "i");
        A = tensor(a[3], "A");
        z = maybe(a[4], "z");
        r_bias = maybe(a[5], "r_bias");
        i_bias = maybe(a[6], "i_bias");
        code = float_code(*x, "x");
        const at::ScalarType type = x->scalar_type();
        if (x->dim() < 2) value_error("x must be [tokens][d] or [sequences][tokens][d]");
        d = x->size(-1);
        c.strided(*x, "x", type, x->sizes());
        c.strided(*r, "r", type, x->sizes());
        c.strided(*i, "i", type, x->sizes());
        if (z) c.strided(*z, "z", type, x->sizes());
        c.dense(A, "A", at::kFloat, {d});
        c.dense(r_bias, "r_bias", at::kFloat, {d});
        c.dense(i_bias, "i_bias", at::kFloat, {d});
    }
    static const float *f(const Tensor *t) { return (const float *)ptr(t); }
};

struct RecurTokens : Recur {
    const Tensor *initial;
    gated_recurrence_problem_t p;
    int64_t seqs;
    // x .. i_bias, initial_state, seq_start
    RecurTokens(PyObject *const *a) : Recur(a)
    {
        initial = maybe(a[7], "initial_state");
        const Lead lead(*x, maybe(a[8], "seq_start"), c);
        seqs = lead.seqs;
        c.dense(initial, "initial_state", at::kFloat, {seqs, d});
        p = {lead.batch, int_size(d, "d"), lead.strides(*x), lead.strides(*r), lead.strides(*i),
             z ? lead.strides(*z) : seq_stride_t{0, 0}, {0, 0}};
    }
};

PyObject *py_gated_recurrence(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    expect_args(n, 10);
    RecurTokens v(a);
    const bool state = truth(a[9]);
    v.c.device(*v.x);
    v.c.detached("gated_recurrence", "gated_recurrence_grad computes the gradients");
    const c10::DeviceGuard guard(v.x->device());
    size_t need = 0;
    raise(gated_recurrence_workspace_size(&v.p, v.code, &need), "gated_recurrence_workspace_size");
    const Tensor y = new_tensor(*v.x, v.x->sizes(), v.x->scalar_type());
    const Tensor s = state ? new_tensor(*v.x, {v.seqs, v.d}, at::kFloat) : Tensor();
    const Tensor ws = workspace(*v.x, need);
    raise(gated_recurrence(&v.p, v.code, ptr(v.x), ptr(v.r), ptr(v.i), v.f(v.A), ptr(v.z), v.f(v.r_bias), v.f(v.i_bias),
                           v.f(v.initial), out_ptr(y), (float *)out_ptr(s), out_ptr(ws), need, stream_of(*v.x)),
          "gated_recurrence");
    return state ? pair(y, s) : wrap(y);
    END_HANDLE_TH_ERRORS
}

PyObject *py_gated_recurrence_grad(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    expect_args(n, 11);
    const Tensor *dy = tensor(a[0], "dy");
    RecurTokens v(a + 1);
    const Tensor *dfinal = maybe(a[10], "dfinal_state");
    v.c.strided(*dy, "dy", v.x->scalar_type(), v.x->sizes());
    v.c.dense(dfinal, "dfinal_state", at::kFloat, {v.seqs, v.d});
    const size_t lead = v.x->dim() - 1;
    v.p.dy = {dy->size(lead - 1) > 1 ? dy->stride(lead - 1) : 0, lead == 2 && dy->size(0) > 1 ? dy->stride(0) : 0};
    v.c.device(*v.x);
    const c10::DeviceGuard guard(v.x->device());
    size_t need = 0;
    raise(gated_recurrence_grad_workspace_size(&v.p, v.code, &need), "gated_recurrence_grad_workspace_size");
    auto like = [&](const Tensor *t) { return t ? new_tensor(*v.x, t->sizes(), t->scalar_type()) : Tensor(); };
    const Tensor dx = like(v.x), dr = like(v.r), di = like(v.i), dA = like(v.A), dz = like(v.z);
    const Tensor drb = like(v.r_bias), dib = like(v.i_bias), d0 = like(v.initial);
    const Tensor ws = workspace(*v.x, need);
    const gated_recurrence_grads_t g = {out_ptr(dx), out_ptr(dr), out_ptr(di), (float *)out_ptr(dA), out_ptr(dz),
                                        (float *)out_ptr(drb), (float *)out_ptr(dib), (float *)out_ptr(d0)};
    raise(gated_recurrence_grad(&v.p, v.code, ptr(dy), ptr(v.x), ptr(v.r), ptr(v.i), v.f(v.A), ptr(v.z), v.f(v.r_bias),
                                v.f(v.i_bias), v.f(v.initial), v.f(dfinal), &g, out_ptr(ws), need, stream_of(*v.x)),
          "gated_recurrence_grad");
    PyObject *r = PyDict_New();
    if (!r) throw python_error();
    set_item(r, "dx", dx);
    set_item(r, "dr", dr);
    set_item(r, "di", di);
    set_item(r, "dA", dA);
    set_item(r, "dz", dz);
    set_item(r, "dr_bias", drb);
    set_item(r, "di_bias", dib);
    set_item(r, "dinitial_state", d0);
    return r;
    END_HANDLE_TH_ERRORS
}

PyObject *py_gated_recurrence_step(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    expect_args(n, 9);
    Recur v(a);  // x, r, i, A, z, r_bias, i_bias, then state, slots
    const Tensor *state = tensor(a[7], "state"), *slots = maybe(a[8], "slots");
    if (v.x->dim() != 2 || state->dim() != 2) value_error("x must be [rows][d] and state [pool][d]");
    const int64_t rows = v.x->size(0), pool = state->size(0);
    v.c.dense(state, "state", at::kFloat, {pool, v.d});
    const int *sp = slots_of(slots, rows, pool, v.c);
    const gated_recurrence_step_problem_t p = {int_size(rows, "rows"), int_size(pool, "pool"), int_size(v.d, "d"),
                                               row_stride(*v.x), row_stride(*v.r), row_stride(*v.i), v.z ? row_stride(*v.z) : 0};
    v.c.device(*v.x);
    v.c.detached("gated_recurrence_step", "gated_recurrence and gated_recurrence_grad compute prompts and their gradients");
    const c10::DeviceGuard guard(v.x->device());
    const Tensor y = new_tensor(*v.x, {rows, v.d}, v.x->scalar_type());
    raise(gated_recurrence_step(&p, v.code, ptr(v.x), ptr(v.r), ptr(v.i), v.f(v.A), ptr(v.z), v.f(v.r_bias), v.f(v.i_bias),
                                (float *)state->data_ptr(), sp, out_ptr(y), stream_of(*v.x)), "gated_recurrence_step");
    written(*state);
    return wrap(y);
    END_HANDLE_TH_ERRORS
}

// ---------------------------------------------------------------------- layer norm
struct Norm {
    Checks c;
    const Tensor *x, *weight, *bias;
    int code, param_code;
    at::ScalarType param_type;
    int64_t d;
    layer_norm_problem_t p;
    Norm(PyObject *xo, PyObject *wo, PyObject *bo, PyObject *eps)
    {
        x = tensor(xo, "x");
        weight = maybe(wo, "weight");
        bias = maybe(bo, "bias");
        code = float_code(*x, "x");
        const double e = PyFloat_AsDouble(eps);
        if (e == -1.0 && PyErr_Occurred()) throw python_error();
        if (!(e >= 0.0) || !((float)e <= 3.402823466e38f)) value_error("eps must be finite and not negative");
        if (x->dim() < 2 || x->dim() > 3) value_error("x must be [tokens][d] or [sequences][tokens][d]");
        d = x->size(-1);
        if (d < 1) value_error("rows must have at least one element");
        c.strided(*x, "x", x->scalar_type(), x->sizes());
        const Tensor *first = weight ? weight : bias;
        param_type = first && first->scalar_type() == at::kFloat ? at::kFloat : x->scalar_type();
        param_code = param_type == at::kFloat ? CONV2D_DTYPE_F32 : code;
        c.dense(weight, "weight", param_type, {d});
        c.dense(bias, "bias", param_type, {d});
        const size_t n = x->dim();
        const int64_t seqs = n == 3 ? x->size(0) : 1, len = x->size(n - 2);
        p = {int_size(seqs, "sequences"), int_size(len, "tokens"), int_size(d, "d"), (float)e, strides(*x), {0, 0}, {0, 0}, {0, 0}};
        if (seqs * len > INT32_MAX) value_error("there are at most 2^31 - 1 rows");
    }
    seq_stride_t strides(const Tensor &t) const
    {
        const size_t n = t.dim();
        return {t.size(n - 2) > 1 ? t.stride(n - 2) : 0, n == 3 && t.size(0) > 1 ? t.stride(0) : 0};
    }
};

PyObject *py_layer_norm(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    expect_args(n, 5);
    Norm v(a[0], a[1], a[2], a[3]);
    const Tensor *residual = maybe(a[4], "residual");
    const at::ScalarType type = v.x->scalar_type();
    if (residual) {
        v.c.strided(*residual, "residual", type, v.x->sizes());
        v.p.residual = v.strides(*residual);
    }
    v.c.device(*v.x);
    v.c.detached("layer_norm", "layer_norm_grad computes the gradients");
    const c10::DeviceGuard guard(v.x->device());
    const Tensor y = new_tensor(*v.x, v.x->sizes(), type), total = residual ? new_tensor(*v.x, v.x->sizes(), type) : Tensor();
    raise(layer_norm(&v.p, v.code, v.param_code, ptr(v.x), ptr(residual), ptr(v.weight), ptr(v.bias), out_ptr(y),
                     out_ptr(total), stream_of(*v.x)), "layer_norm");
    return residual ? pair(y, total) : wrap(y);
    END_HANDLE_TH_ERRORS
}

PyObject *py_layer_norm_grad(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    expect_args(n, 6);
    const Tensor *dy = tensor(a[0], "dy");
    Norm v(a[1], a[2], a[3], a[4]);
    const Tensor *dtotal = maybe(a[5], "dtotal");
    const at::ScalarType type = v.x->scalar_type();
    v.c.strided(*dy, "dy", type, v.x->sizes());
    v.p.dy = v.strides(*dy);
    if (dtotal) {
        v.c.strided(*dtotal, "dtotal", type, v.x->sizes());
        v.p.dtotal = v.strides(*dtotal);
    }
    v.c.device(*v.x);
    const c10::DeviceGuard guard(v.x->device());
    size_t need = 0;
    raise(layer_norm_grad_workspace_size(&v.p, v.code, &need), "layer_norm_grad_workspace_size");
    const Tensor dx = new_tensor(*v.x, v.x->sizes(), type);
    const Tensor dw = v.weight ? new_tensor(*v.x, {v.d}, v.param_type) : Tensor();
    const Tensor db = v.bias ? new_tensor(*v.x, {v.d}, v.param_type) : Tensor();
    const Tensor ws = workspace(*v.x, need);
    raise(layer_norm_grad(&v.p, v.code, v.param_code, ptr(dy), ptr(v.x), ptr(v.weight), ptr(dtotal), out_ptr(dx),
                          out_ptr(dw), out_ptr(db), out_ptr(ws), need, stream_of(*v.x)), "layer_norm_grad");
    PyObject *r = PyDict_New();
    if (!r) throw python_error();
    set_item(r, "dx", dx);
    set_item(r, "dw", dw);
    set_item(r, "db", db);
    return r;
    END_HANDLE_TH_ERRORS
}

// ------------------------------------------------------------------ 4-bit products
int64_t fp4_groups(int64_t k) { return (k + 31) / 32; }

PyObject *py_fp4_quantize(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    expect_args(n, 1);
    const Tensor *x = tensor(a[0], "x");
    const int code = float_code(*x, "x");
    if (x->dim() != 2) value_error("x must be [m][k]");
    Checks c;
    c.strided(*x, "x", x->scalar_type(), x->sizes());
    c.device(*x);
    c.detached("fp4_quantize", "rounding to 4 bits has none");
    const int64_t m = x->size(0), k = x->size(1), pitch = fp4_groups(k) * 16, cols = (k + 1) / 2;
    const c10::DeviceGuard guard(x->device());
    const Tensor q = new_tensor(*x, {m, pitch}, at::kByte), scale = new_tensor(*x, {m, fp4_groups(k)}, at::kByte);
    raise(fp4_quantize(code, int_size(m, "m"), int_size(k, "k"), ptr(x), row_stride(*x), out_ptr(q), pitch, out_ptr(scale),
                       stream_of(*x)), "fp4_quantize");
    return pair(pitch == cols ? q : q.narrow(1, 0, cols), scale);
    END_HANDLE_TH_ERRORS
}

PyObject *py_fp4_matmul(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    expect_args(n, 3);
    const Tensor *x = tensor(a[0], "x"), *w = tensor(a[1], "w"), *ws = tensor(a[2], "w_scale");
    const int code = float_code(*x, "x");
    if (x->dim() != 2 || w->dim() != 2) value_error("x must be [m][k] and w [n][ceil(k/2)]");
    Checks c;
    const int64_t m = x->size(0), k = x->size(1), rows = w->size(0), groups = fp4_groups(k);
    c.strided(*x, "x", x->scalar_type(), x->sizes());
    c.strided(*w, "w", at::kByte, {rows, (k + 1) / 2});
    c.dense(ws, "w_scale", at::kByte, {rows, groups});
    const int64_t pitch = rows > 1 && k > 0 ? w->stride(0) : groups * 16;
    // whole groups are read: the last row's too has to lie in w's memory to its last group's end
    if (pitch % 16 || pitch < groups * 16 ||
        (rows > 0 && k > 0 && (w->storage_offset() + (rows - 1) * pitch + groups * 16) > (int64_t)w->storage().nbytes()))
        value_error("w's rows must start on 16-byte steps and hold whole groups of 32 values (fp4_quantize lays them out so)");
    c.device(*x);
    c.detached("fp4_matmul", "quantised weights have none");
    const fp4_matmul_problem_t p = {int_size(m, "m"), int_size(rows, "n"), int_size(k, "k"), row_stride(*x), pitch};
    const c10::DeviceGuard guard(x->device());
    size_t need = 0;
    raise(fp4_matmul_workspace_size(&p, code, &need), "fp4_matmul_workspace_size");
    const Tensor out = new_tensor(*x, {m, rows}, x->scalar_type()), work = workspace(*x, need);
    raise(fp4_matmul(&p, code, ptr(x), ptr(w), ptr(ws), out_ptr(out), out_ptr(work), need, stream_of(*x)), "fp4_matmul");
    return wrap(out);
    END_HANDLE_TH_ERRORS
}

#define FN(name) {#name, (PyCFunction)(void (*)(void))py_##name, METH_FASTCALL, nullptr}
PyMethodDef methods[] = {FN(causal_conv), FN(causal_conv_grad), FN(causal_conv_step), FN(selective_scan),
                         FN(selective_scan_grad), FN(selective_scan_step), FN(fp8_quantize), FN(fp8_matmul),
                         FN(gated_recurrence), FN(gated_recurrence_grad), FN(gated_recurrence_step), FN(layer_norm),
                         FN(layer_norm_grad), FN(fp4_quantize), FN(fp4_matmul),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_sequence", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__sequence()
{
    PyObject *binding = PyImport_ImportModule("convolution_nhwc_implicit_amd.binding");
    if (!binding) return nullptr;
    error_class = PyObject_GetAttrString(binding, "Conv2dError");
    Py_DECREF(binding);
    return error_class ? PyModule_Create(&module) : nullptr;
}
