// fp8mm_torch.cpp -- the operators of an MLP block for PyTorch tensors, as a
// CPython extension module.
//
// These calls make up to five new tensors each, and with few rows their
// kernels take 2 to 10 us, so the host's time is the call's time. Through
// ctypes, with the checks and torch.empty in Python, one token's layer norm
// with codes took 21 us a call on a Grace core, here 9.0; a product with a new
// output 14, here 3.9. The module checks arguments, makes the tensors that are
// not given, and calls the C entries, whose addresses it is handed (init); it
// runs nothing on the device itself. Errors are ValueError for arguments
// (TypeError for what is no tensor) and what `check` raises for a status.
// All tensors of a call are on one device; what is made is made there, and the
// kernels run on that device's current stream.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdarg>
#include <initializer_list>
#include <string>

#include "fp8mm.h"

namespace {

using at::ScalarType;
using at::Tensor;

struct Raised {};    // a Python exception is set

[[noreturn]] void refuse(const char *format, ...)
{
    va_list args;
    va_start(args, format);
    PyErr_FormatV(PyExc_ValueError, format, args);
    va_end(args);
    throw Raised{};
}

// ------------------------------------------------------------- C entries ---

struct {
    decltype(&fp8_scaled_mm_epilogue) mm_epilogue;
    decltype(&fp8_scaled_mm_act_grad) mm_act_grad;
    decltype(&fp8_act_grad) act_grad;
    decltype(&fp8_act_grad_workspace) act_grad_workspace;
    decltype(&fp8_layer_norm) layer_norm;
    decltype(&fp8_layer_norm_grad) layer_norm_grad;
    decltype(&fp8_layer_norm_grad_workspace) layer_norm_grad_workspace;
} api;
PyObject *check_status;      // raises for a status other than 0

void checked(int64_t rc)
{
    if (rc >= 0)
        return;
    PyObject *r = PyObject_CallFunction(check_status, "i", static_cast<int>(rc));
    if (r) {
        Py_DECREF(r);
        PyErr_Format(PyExc_RuntimeError, "status %d", static_cast<int>(rc));
    }
    throw Raised{};
}

// Other Python threads run while this one makes its tensors and launches
// (either can wait: for memory, for room in the stream's queue). Once per call:
// it costs 0.4 us.
struct Unlocked {
    PyThreadState *state = PyEval_SaveThread();
    ~Unlocked() { PyEval_RestoreThread(state); }
};

// The call's device as the current one.
struct Guard {
    c10::cuda::OptionalCUDAGuard guard;
    explicit Guard(at::Device d)
    {
        if (d.index() != c10::cuda::current_device())
            guard.set_device(d);
    }
};

void *stream() { return c10::cuda::getCurrentCUDAStream().stream(); }

// ------------------------------------------------------------- arguments ---

const Tensor *tensor(const char *name, PyObject *o, bool may_be_none = false)
{
    if (o == Py_None && may_be_none)
        return nullptr;
    if (!THPVariable_Check(o)) {
        PyErr_Format(PyExc_TypeError, "%s must be a tensor, not %s", name, Py_TYPE(o)->tp_name);
        throw Raised{};
    }
    return &THPVariable_Unpack(o);
}

int integer(PyObject *o)
{
    PyObject *i = PyNumber_Index(o);
    if (!i)
        throw Raised{};
    const long v = PyLong_AsLong(i);
    Py_DECREF(i);
    if (v == -1 && PyErr_Occurred())
        throw Raised{};
    if (v < INT32_MIN || v > INT32_MAX)
        refuse("integer argument out of range");
    return static_cast<int>(v);
}

bool truth(PyObject *o)
{
    const int t = PyObject_IsTrue(o);
    if (t < 0)
        throw Raised{};
    return t != 0;
}

ScalarType dtype(const char *name, PyObject *o)
{
    if (!THPDtype_Check(o)) {
        PyErr_Format(PyExc_TypeError, "%s must be a torch.dtype, not %s", name, Py_TYPE(o)->tp_name);
        throw Raised{};
    }
    return reinterpret_cast<THPDtype *>(o)->scalar_type;
}

// Element codes of the C entries; -1: not one of them.
int row_code(ScalarType t)
{
    return t == ScalarType::BFloat16 ? FP8MM_OUT_BF16
           : t == ScalarType::Half   ? FP8MM_OUT_F16
           : t == ScalarType::Float  ? FP8MM_OUT_F32
                                     : -1;
}
int out_code(ScalarType t) { return t == ScalarType::Float8_e4m3fn ? FP8MM_OUT_E4M3 : row_code(t); }
int fp8_code(ScalarType t)
{
    return t == ScalarType::Float8_e4m3fn ? FP8MM_TYPE_E4M3 : t == ScalarType::Float8_e5m2 ? FP8MM_TYPE_E5M2 : -1;
}
const char *row_name(ScalarType t)
{
    return t == ScalarType::BFloat16 ? "torch.bfloat16" : t == ScalarType::Half ? "torch.float16" : "torch.float32";
}

// A call's tensors are on one device: that of its first one.
void beside(const char *name, const Tensor &t, const Tensor &first)
{
    if (t.device() != first.device())
        refuse("%s is on another device than the first operand", name);
}

// Row stride of a 2-D bf16, fp16 or fp32 CUDA matrix with contiguous rows; its
// shape and type as `like`'s, where given.
int64_t rows(const char *name, const Tensor &t, const Tensor *like = nullptr, const ScalarType *type = nullptr)
{
    if (t.dim() != 2 || row_code(t.scalar_type()) < 0 || !t.is_cuda())
        refuse("%s must be a 2-D CUDA tensor of bfloat16, float16 or float32", name);
    if (like)
        beside(name, t, *like);
    const int64_t R = t.size(0), C = t.size(1);
    if (like && (R != like->size(0) || C != like->size(1)))
        refuse("%s must have shape (%lld, %lld)", name, static_cast<long long>(like->size(0)),
               static_cast<long long>(like->size(1)));
    if (type && t.scalar_type() != *type)
        refuse("%s must be %s", name, row_name(*type));
    if (t.is_contiguous())
        return C;
    if ((C > 1 && t.stride(1) != 1) || (R > 1 && t.stride(0) < C))
        refuse("%s's rows must be contiguous, their stride at least %lld", name, static_cast<long long>(C));
    return R > 1 ? t.stride(0) : C;
}

// A contiguous vector of n values, fp32 or (any) of any row type, on first's device.
void vector(const char *name, const Tensor *t, int64_t n, bool any, const Tensor &first)
{
    if (t && ((any ? row_code(t->scalar_type()) < 0 : t->scalar_type() != ScalarType::Float) || t->numel() != n ||
              !t->is_contiguous() || !t->is_cuda()))
        refuse("%s must be a contiguous CUDA tensor of %lld values of %s", name, static_cast<long long>(n),
               any ? "torch.bfloat16 or torch.float16 or torch.float32" : "torch.float32");
    if (t)
        beside(name, *t, first);
}

void *data(const Tensor *t) { return t ? t->data_ptr() : nullptr; }
float *floats(const Tensor *t) { return static_cast<float *>(data(t)); }

Tensor empty(const Tensor &like, at::IntArrayRef shape, ScalarType type)
{
    return at::empty(shape, like.options().dtype(type));
}

// A result: the tensor that was given, one to be made, or None.
struct Result {
    PyObject *given = nullptr;
    const Tensor *t = nullptr;       // given or made
    Tensor made;
    const Tensor *like = nullptr;    // to be made: of this one's device, [rows, cols] or [rows]
    int64_t rows = 0, cols = 0;
    ScalarType type = ScalarType::Float;

    void take(const char *name, PyObject *o)
    {
        t = tensor(name, o, true);
        given = t ? o : nullptr;
        if (t)
            type = t->scalar_type();
    }
    void plan(const Tensor &x, ScalarType ty, int64_t r, int64_t c = -1)
    {
        like = &x;
        type = ty;
        rows = r;
        cols = c;
    }
    bool wanted() const { return t || like; }
    // (without the interpreter's lock)
    void *make()
    {
        if (!t && like) {
            const int64_t shape[2] = {rows, cols};
            made = empty(*like, at::IntArrayRef(shape, cols < 0 ? 1 : 2), type);
            t = &made;
        }
        return t ? t->data_ptr() : nullptr;
    }
    float *make_floats() { return static_cast<float *>(make()); }
    PyObject *object()
    {
        PyObject *o = !t ? Py_None : given;
        if (!o) {
            o = THPVariable_Wrap(made);
            if (!o)
                throw Raised{};
            return o;
        }
        Py_INCREF(o);
        return o;
    }
};

PyObject *tuple(std::initializer_list<Result *> results)
{
    PyObject *all = PyTuple_New(static_cast<Py_ssize_t>(results.size()));
    if (!all)
        throw Raised{};
    Py_ssize_t i = 0;
    try {
        for (Result *r : results)
            PyTuple_SET_ITEM(all, i++, r->object());
    } catch (...) {
        Py_DECREF(all);
        throw;
    }
    return all;
}

// -------------------------------------------------------------- products ---

struct Product {
    const Tensor *A, *B, *scale_a, *scale_b;
    int mode;
    int64_t M, N, K;
    fp8mm_options options;
};

std::string shape_of(const Tensor &t)
{
    std::string s = "(";
    for (int64_t i = 0; i < t.dim(); ++i)
        s += (i ? ", " : "") + std::to_string(t.size(i));
    return s + (t.dim() == 1 ? ",)" : ")");
}

// Whether n rows (columns) of K elements lie back to back: dimension `inner` of
// t runs along K. With one of them the other stride does not matter.
bool back_to_back(const Tensor &t, int inner, int64_t n, int64_t K)
{
    return n == 0 || (t.stride(inner) == 1 && (n == 1 || t.stride(1 - inner) == K));
}

// The operands and options of a product: A, B, scale_a, scale_b, scale_mode
// from a[0], variant, tile_n, split_k from o[0].
Product product(PyObject *const *a, PyObject *const *o)
{
    Product p{};
    p.A = tensor("A", a[0]);
    p.B = tensor("B", a[1]);
    p.scale_a = tensor("scale_a", a[2]);
    p.scale_b = tensor("scale_b", a[3]);
    p.mode = integer(a[4]);
    const Tensor &A = *p.A, &B = *p.B;
    if (A.dim() != 2 || B.dim() != 2)
        refuse("A must be [M, K] and B [K, N]");
    p.M = A.size(0);
    p.K = A.size(1);
    p.N = B.size(1);
    if (B.size(0) != p.K)
        refuse("inner dimensions differ: A is %s, B is %s", shape_of(A).c_str(), shape_of(B).c_str());
    p.options.a_type = fp8_code(A.scalar_type());
    p.options.b_type = fp8_code(B.scalar_type());
    if (p.options.a_type < 0 || p.options.b_type < 0)
        refuse("A and B must be torch.float8_e4m3fn or float8_e5m2");
    if (!back_to_back(A, 1, p.M, p.K))
        refuse("A must be row-major contiguous [M, K]");
    if (!back_to_back(B, 0, p.N, p.K))
        refuse("B must be column-major [K, N] (B.t() contiguous)");
    if (p.mode != FP8MM_SCALE_TENSOR && p.mode != FP8MM_SCALE_ROWWISE)
        refuse("scale_mode must be 0 (per-tensor) or 1 (row-wise)");
    const Tensor *scales[2] = {p.scale_a, p.scale_b};
    for (int i = 0; i < 2; ++i) {
        const int64_t n = p.mode == FP8MM_SCALE_TENSOR ? 1 : i ? p.N : p.M;
        if (scales[i]->scalar_type() != ScalarType::Float || scales[i]->numel() != n || !scales[i]->is_contiguous())
            refuse("%s must be a contiguous float32 tensor of %lld values", i ? "scale_b" : "scale_a",
                   static_cast<long long>(n));
    }
    if (!A.is_cuda() || !B.is_cuda() || !p.scale_a->is_cuda() || !p.scale_b->is_cuda())
        refuse("fp8_scaled_mm takes CUDA tensors (use fp8_scaled_mm_host for host memory)");
    beside("B", B, A);
    beside("scale_a", *p.scale_a, A);
    beside("scale_b", *p.scale_b, A);
    p.options.variant = integer(o[0]);
    p.options.tile_n = integer(o[1]);
    p.options.split_k = integer(o[2]);
    return p;
}

// The product's output, given or made; its leading dimension.
void product_out(Product &p, Result &out, PyObject *given, ScalarType type)
{
    out.take("out", given);
    if (!out.t) {
        if (out_code(type) < 0)
            refuse("out must be a [M, N] tensor of bfloat16, float16, float32 or float8_e4m3fn with contiguous rows");
        out.plan(*p.A, type, p.M, p.N);
    } else {
        const Tensor &t = *out.t;
        if (out_code(t.scalar_type()) < 0 || t.dim() != 2 || t.size(0) != p.M || t.size(1) != p.N ||
            !(t.is_contiguous() || ((t.stride(1) == 1 || p.N == 1) && t.stride(0) >= p.N)))
            refuse("out must be a [M, N] tensor of bfloat16, float16, float32 or float8_e4m3fn with contiguous rows");
        if (!t.is_cuda())
            refuse("fp8_scaled_mm takes CUDA tensors (use fp8_scaled_mm_host for host memory)");
        beside("out", t, *p.A);
        p.options.ldo = t.is_contiguous() ? 0 : t.stride(0);
    }
    p.options.out_type = out_code(out.type);
}

ScalarType aux_type(const Result &out)
{
    return out.type == ScalarType::Float8_e4m3fn ? ScalarType::BFloat16 : out.type;
}

// Leading dimension of a [M, N] matrix beside out (residual, preact, z).
int64_t aux(const char *name, const Product &p, const Tensor *t, ScalarType type)
{
    if (!t)
        return 0;
    if (t->scalar_type() != type || t->dim() != 2 || t->size(0) != p.M || t->size(1) != p.N || !t->is_cuda())
        refuse("%s must be a CUDA [M, N] tensor of out's dtype (bfloat16 for a float8_e4m3fn output)", name);
    beside(name, *t, *p.A);
    if (t->is_contiguous())
        return p.N;
    if ((t->stride(1) != 1 && p.N > 1) || (t->stride(0) < p.N && p.M > 1))
        refuse("%s's rows must be contiguous, their stride at least N", name);
    return std::max(p.N, t->stride(0));
}

// A, B, scale_a, scale_b, scale_mode, bias, activation, residual, preact, out,
// out_dtype, return_preact, variant, tile_n, split_k
PyObject *mm_epilogue(PyObject *const *a)
{
    Product p = product(a, a + 12);
    const Tensor *bias = tensor("bias", a[5], true), *residual = tensor("residual", a[7], true);
    const bool return_preact = truth(a[11]);
    Result out, preact;
    product_out(p, out, a[9], dtype("out_dtype", a[10]));
    const ScalarType type = aux_type(out);
    if (bias && (bias->scalar_type() != type || bias->numel() != p.N || !bias->is_contiguous()))
        refuse("bias must be a contiguous tensor of N values of out's dtype (bfloat16 for a float8_e4m3fn output)");
    if (bias && !bias->is_cuda())
        refuse("fp8_scaled_mm takes CUDA tensors (use fp8_scaled_mm_host for host memory)");
    if (bias)
        beside("bias", *bias, *p.A);
    preact.take("preact", a[8]);
    if (return_preact && !preact.t)
        preact.plan(*p.A, type, p.M, p.N);
    fp8mm_epilogue e{};
    e.activation = integer(a[6]);
    e.residual = data(residual);
    e.ldr = aux("residual", p, residual, type);
    e.ldp = aux("preact", p, preact.t, type);
    const Guard guard(p.A->device());
    int64_t rc;
    {
        Unlocked u;
        void *to = out.make();
        e.preact = preact.make();
        rc = api.mm_epilogue(data(p.A), data(p.B), floats(p.scale_a), floats(p.scale_b), p.mode, data(bias), to, p.M, p.N,
                             p.K, stream(), &p.options, &e);
    }
    checked(rc);
    return return_preact ? tuple({&out, &preact}) : out.object();
}

// A, B, scale_a, scale_b, scale_mode, z, activation, out, out_dtype, variant,
// tile_n, split_k
PyObject *mm_act_grad(PyObject *const *a)
{
    Product p = product(a, a + 9);
    const Tensor *z = tensor("z", a[5]);
    Result out;
    product_out(p, out, a[7], a[8] == Py_None ? z->scalar_type() : dtype("out_dtype", a[8]));
    const int64_t ldz = aux("z", p, z, aux_type(out));
    const int activation = integer(a[6]);
    const Guard guard(p.A->device());
    int64_t rc;
    {
        Unlocked u;
        void *to = out.make();
        rc = api.mm_act_grad(data(p.A), data(p.B), floats(p.scale_a), floats(p.scale_b), p.mode, activation, data(z), ldz,
                             to, p.M, p.N, p.K, stream(), &p.options);
    }
    checked(rc);
    return out.object();
}

// ------------------------------------------------------------------ rows ---

// dy, z, activation, dz, dbias, return_dz, return_dbias
PyObject *act_grad(PyObject *const *a)
{
    const Tensor &dy = *tensor("dy", a[0]), *z = tensor("z", a[1], true);
    const int64_t lddy = rows("dy", dy), M = dy.size(0), N = dy.size(1);
    const ScalarType type = dy.scalar_type();
    const int64_t ldz = z ? rows("z", *z, &dy, &type) : 0;
    Result dz, dbias;
    dz.take("dz", a[3]);
    const int64_t lddz = dz.t ? rows("dz", *dz.t, &dy, &type) : 0;
    if (!dz.t && truth(a[5]))
        dz.plan(dy, type, M, N);
    dbias.take("dbias", a[4]);
    vector("dbias", dbias.t, N, false, dy);
    if (!dbias.t && truth(a[6]))
        dbias.plan(dy, ScalarType::Float, N);
    const int activation = integer(a[2]);
    const Guard guard(dy.device());
    int64_t bytes = 0, rc;
    if (dbias.wanted())
        checked(bytes = api.act_grad_workspace(M, N));
    {
        Unlocked u;
        void *to = dz.make();
        float *sums = dbias.make_floats();
        Tensor ws;
        if (bytes > 0)
            ws = empty(dy, {bytes}, ScalarType::Byte);
        rc = api.act_grad(data(&dy), lddy, data(z), ldz, row_code(type), activation, to, lddz, sums, M, N,
                          bytes > 0 ? data(&ws) : nullptr, bytes, stream());
    }
    checked(rc);
    return tuple({&dz, &dbias});
}

// x, gamma, beta, eps, y, y_dtype, q_dtype, return_y
PyObject *layer_norm(PyObject *const *a)
{
    const Tensor &x = *tensor("x", a[0]), *gamma = tensor("gamma", a[1], true), *beta = tensor("beta", a[2], true);
    const int64_t ldx = rows("x", x), R = x.size(0), C = x.size(1);
    if (R > 0 && C == 0)
        refuse("x's rows must have at least one column");
    if (gamma && beta && gamma->scalar_type() != beta->scalar_type())
        refuse("gamma and beta must have one dtype");
    vector("gamma", gamma, C, true, x);
    vector("beta", beta, C, true, x);
    const Tensor *params = gamma ? gamma : beta;
    const double eps = PyFloat_AsDouble(a[3]);
    if (eps == -1.0 && PyErr_Occurred())
        throw Raised{};
    Result y, mean, rstd, q, q_scale;
    const ScalarType y_type = a[5] == Py_None ? x.scalar_type() : dtype("y_dtype", a[5]);
    y.take("y", a[4]);
    int64_t ldy = C;
    if (y.t) {
        ldy = rows("y", *y.t, &x, a[5] == Py_None ? nullptr : &y_type);
    } else if (truth(a[7])) {
        if (row_code(y_type) < 0)
            refuse("y_dtype must be torch.bfloat16, torch.float16 or torch.float32");
        y.plan(x, y_type, R, C);
    }
    const bool codes = a[6] != Py_None;
    const ScalarType code_type = codes ? dtype("q_dtype", a[6]) : ScalarType::Float8_e4m3fn;
    if (fp8_code(code_type) < 0)
        refuse("q_dtype must be torch.float8_e4m3fn or torch.float8_e5m2");
    mean.plan(x, ScalarType::Float, R);
    rstd.plan(x, ScalarType::Float, R);
    if (codes) {
        q.plan(x, code_type, R, C);
        q_scale.plan(x, ScalarType::Float, R);
    }
    const Guard guard(x.device());
    int64_t rc;
    {
        Unlocked u;
        void *to = y.make(), *to_q = q.make();
        float *means = mean.make_floats(), *rstds = rstd.make_floats(), *scales = q_scale.make_floats();
        rc = api.layer_norm(data(&x), row_code(x.scalar_type()), ldx, data(gamma), data(beta),
                            params ? row_code(params->scalar_type()) : FP8MM_OUT_F32, static_cast<float>(eps), to,
                            y.t ? row_code(y.type) : FP8MM_OUT_F32, ldy, means, rstds, to_q, fp8_code(code_type), scales,
                            R, C, stream());
    }
    checked(rc);
    return q.t ? tuple({&y, &mean, &rstd, &q, &q_scale}) : tuple({&y, &mean, &rstd});
}

// dy, x, gamma, mean, rstd, residual_grad, dx, return_params
PyObject *layer_norm_grad(PyObject *const *a)
{
    const Tensor &dy = *tensor("dy", a[0]), &x = *tensor("x", a[1]), *gamma = tensor("gamma", a[2], true),
                 *mean = tensor("mean", a[3]), *rstd = tensor("rstd", a[4]), *res = tensor("residual_grad", a[5], true);
    const int64_t lddy = rows("dy", dy), ldx = rows("x", x, &dy), R = x.size(0), C = x.size(1);
    const ScalarType type = x.scalar_type();
    vector("gamma", gamma, C, true, dy);
    vector("mean", mean, R, false, dy);
    vector("rstd", rstd, R, false, dy);
    const int64_t lddres = res ? rows("residual_grad", *res, &x, &type) : 0;
    Result dx, dgamma, dbeta;
    dx.take("dx", a[6]);
    int64_t lddx = C;
    if (dx.t)
        lddx = rows("dx", *dx.t, &x, &type);
    else
        dx.plan(x, type, R, C);
    const Guard guard(x.device());
    int64_t bytes = 0, rc;
    if (truth(a[7])) {
        checked(bytes = api.layer_norm_grad_workspace(R, C));
        dgamma.plan(x, ScalarType::Float, C);
        dbeta.plan(x, ScalarType::Float, C);
    }
    {
        Unlocked u;
        void *to = dx.make();
        float *to_gamma = dgamma.make_floats(), *to_beta = dbeta.make_floats();
        Tensor ws;
        if (bytes > 0)
            ws = empty(x, {bytes}, ScalarType::Byte);
        rc = api.layer_norm_grad(data(&dy), row_code(dy.scalar_type()), lddy, data(&x), row_code(type), ldx, data(gamma),
                                 gamma ? row_code(gamma->scalar_type()) : FP8MM_OUT_F32, floats(mean), floats(rstd),
                                 data(res), lddres, to, lddx, to_gamma, to_beta, R, C, bytes > 0 ? data(&ws) : nullptr,
                                 bytes, stream());
    }
    checked(rc);
    return tuple({&dx, &dgamma, &dbeta});
}

// ---------------------------------------------------------------- module ---

// A function of N positional arguments.
template <PyObject *(*F)(PyObject *const *), Py_ssize_t N>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != N) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", N, n);
        return nullptr;
    }
    if (!check_status) {
        PyErr_SetString(PyExc_RuntimeError, "init() has not been called");
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Raised &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// init(check, addresses): the status check and the C entries' addresses in
// api's order.
PyObject *init(PyObject *, PyObject *args)
{
    PyObject *check;
    unsigned long long at[7];
    if (!PyArg_ParseTuple(args, "O(KKKKKKK)", &check, &at[0], &at[1], &at[2], &at[3], &at[4], &at[5], &at[6]))
        return nullptr;
    int i = 0;
    auto next = [&](auto &f) { f = reinterpret_cast<std::decay_t<decltype(f)>>(static_cast<uintptr_t>(at[i++])); };
    next(api.mm_epilogue);
    next(api.mm_act_grad);
    next(api.act_grad);
    next(api.act_grad_workspace);
    next(api.layer_norm);
    next(api.layer_norm_grad);
    next(api.layer_norm_grad_workspace);
    Py_INCREF(check);
    Py_XDECREF(check_status);
    check_status = check;
    Py_RETURN_NONE;
}

template <PyObject *(*F)(PyObject *const *), Py_ssize_t N>
PyMethodDef method(const char *name)
{
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<F, N>)), METH_FASTCALL, nullptr};
}

PyMethodDef methods[] = {
    {"init", init, METH_VARARGS, nullptr},
    method<mm_epilogue, 15>("mm_epilogue"),
    method<mm_act_grad, 12>("mm_act_grad"),
    method<act_grad, 7>("act_grad"),
    method<layer_norm, 8>("layer_norm"),
    method<layer_norm_grad, 8>("layer_norm_grad"),
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_fp8mm_torch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__fp8mm_torch() { return PyModule_Create(&module); }
