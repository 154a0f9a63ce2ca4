// bind.cpp -- the Python module _ops: argument marshalling of the operators around the expert
// layer, over the C ABI of include/cpw_moe.h.  Nothing is computed here.  Checks of shapes, types
// and devices raise ValueError / TypeError, status codes of the library raise MoeError; outputs
// and workspaces come from PyTorch's allocator on the current stream.  (These calls are a few
// microseconds of GPU work at decode sizes: marshalled in Python they took 13 to 20 us of host
// time a call.)
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/ATen.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>

#include <algorithm>
#include <climits>
#include <sstream>
#include <stdexcept>
#include <string>

#include "../../include/cpw_moe.h"

namespace {

struct ValueErr : std::runtime_error {
    using std::runtime_error::runtime_error;
};
struct TypeErr : std::runtime_error {
    using std::runtime_error::runtime_error;
};
struct MoeErr {
    int code;
    const char *what;
};
struct PyErrSet {};   // a Python error is already set

PyObject *g_moe_error = nullptr;   // native.MoeError

std::string shape_of(const at::Tensor &t)
{
    std::ostringstream s;
    s << "(";
    for (int64_t i = 0; i < t.dim(); ++i)
        s << (i ? ", " : "") << t.size(i);
    s << ")";
    return s.str();
}
std::string dtype_name(at::ScalarType t) { return c10::toString(t); }

const at::Tensor &tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o))
        throw TypeErr(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}
bool none(PyObject *o) { return o == Py_None; }

int code_of(at::ScalarType t)
{
    return t == at::kFloat ? MOE_F32 : t == at::kBFloat16 ? MOE_BF16 : t == at::kHalf ? MOE_F16 : -1;
}

int count(int64_t n, const char *name)
{
    if (n > INT_MAX || n < INT_MIN)
        throw ValueErr(std::string(name) + ": " + std::to_string(n) + " passes 31 bits");
    return static_cast<int>(n);
}

void on_device(const at::Tensor &t, const char *name, at::ScalarType dtype, int dev)
{
    if (!t.is_cuda())
        throw ValueErr(std::string(name) + " must be a CUDA tensor");
    if (t.scalar_type() != dtype)
        throw TypeErr(std::string(name) + ": dtype " + dtype_name(t.scalar_type()) + " != " + dtype_name(dtype));
    if (t.device().index() != dev)
        throw ValueErr(std::string(name) + " is not on the device of the other tensors");
}

// The matrix that the other tensors are held against: its element type and device.
struct First {
    at::ScalarType type;
    int dtype, dev;
};
First first(const at::Tensor &t, const char *name, bool half_only = false)
{
    if (half_only && t.scalar_type() != at::kBFloat16 && t.scalar_type() != at::kHalf)
        throw TypeErr(std::string(name) + ": dtype " + dtype_name(t.scalar_type()) + " is not bfloat16 or float16 (not float32)");
    if (t.dim() != 2)
        throw ValueErr(std::string(name) + ": shape " + shape_of(t) + " is not [rows, width]");
    const int dtype = code_of(t.scalar_type());
    if (dtype < 0)
        throw TypeErr(std::string(name) + ": dtype " + dtype_name(t.scalar_type()) + " is not float32, bfloat16 or float16");
    if (!t.is_cuda())
        throw ValueErr(std::string(name) + " must be a CUDA tensor");
    const int dev = t.device().index();
    if (dev != c10::cuda::current_device())
        throw ValueErr(std::string(name) + " is not on the current device");
    return {t.scalar_type(), dtype, dev};
}

// A matrix of contiguous rows that do not overlap.
struct Matrix {
    int64_t rows, width, ld;
    void *p;
};
Matrix matrix(const at::Tensor &t, const char *name, const First &f, int64_t rows = -1, int64_t width = -1)
{
    if (t.dim() != 2 || (rows >= 0 && t.size(0) != rows) || (width >= 0 && t.size(1) != width)) {
        std::ostringstream s;
        s << name << ": shape " << shape_of(t) << " is not [";
        rows >= 0 ? s << rows : s << "rows";
        s << ", ";
        width >= 0 ? s << width : s << "width";
        s << "]";
        throw ValueErr(s.str());
    }
    on_device(t, name, f.type, f.dev);
    const int64_t n = t.size(0), w = t.size(1), ld = t.stride(0), step = t.stride(1);
    if (n >= 1 && w > 1 && step != 1)
        throw ValueErr(std::string(name) + ": the elements of a row must be contiguous");
    if (n > 1 && ld < w)
        throw ValueErr(std::string(name) + ": rows must not overlap");
    // (the stride of a single row is never used and may be anything)
    return {n, w, n > 1 ? ld : std::max<int64_t>(w, 1), t.data_ptr()};
}

// An output that the caller gave has been written: what autograd saved of it is no longer there.
void written(const at::Tensor &t)
{
    if (!t.is_inference())   // (inference tensors have no version)
        t.unsafeGetTensorImpl()->bump_version();
}

// A contiguous tensor of the given shape.
void *flat(const at::Tensor &t, const char *name, at::IntArrayRef shape, at::ScalarType dtype, int dev)
{
    if (t.sizes() != shape) {
        std::ostringstream s;
        s << name << ": shape " << shape_of(t) << " != (";
        for (size_t i = 0; i < shape.size(); ++i)
            s << (i ? ", " : "") << shape[i];
        s << ")";
        throw ValueErr(s.str());
    }
    on_device(t, name, dtype, dev);
    if (!t.is_contiguous())
        throw ValueErr(std::string(name) + " must be contiguous");
    return t.data_ptr();
}
void *flat_or_null(PyObject *o, const char *name, at::IntArrayRef shape, at::ScalarType dtype, int dev)
{
    return none(o) ? nullptr : flat(tensor(o, name), name, shape, dtype, dev);
}

at::Tensor make(at::IntArrayRef shape, at::ScalarType dtype, int dev)
{
    // (at::empty without the dispatcher's 0.3 us)
    return at::detail::empty_cuda(shape, at::TensorOptions().dtype(dtype).device(at::kCUDA, static_cast<c10::DeviceIndex>(dev)));
}

// A workspace for a call: memory of the current stream, back in the allocator's hands (and so in
// that stream's order) when the call has been enqueued.
struct Workspace {
    c10::DataPtr p;
    explicit Workspace(uint64_t bytes)
    {
        if (bytes)
            p = c10::cuda::CUDACachingAllocator::get()->allocate(bytes);
    }
    void *get() const { return p.get(); }
};

void *current_stream(int dev) { return c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev)).stream(); }

void check(int rc, const char *what)
{
    if (rc != MOE_OK)
        throw MoeErr{rc, what};
}

int64_t integer(PyObject *o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred())
        throw PyErrSet{};
    return v;
}
int small(PyObject *o, const char *name) { return count(integer(o), name); }
bool truth(PyObject *o)
{
    const int v = PyObject_IsTrue(o);
    if (v < 0)
        throw PyErrSet{};
    return v != 0;
}
float real(PyObject *o)
{
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred())
        throw PyErrSet{};
    return static_cast<float>(v);
}

PyObject *tuple_of(std::initializer_list<at::Tensor> ts)
{
    PyObject *r = PyTuple_New(static_cast<Py_ssize_t>(ts.size()));
    if (!r)
        throw PyErrSet{};
    Py_ssize_t i = 0;
    for (const at::Tensor &t : ts)
        PyTuple_SET_ITEM(r, i++, THPVariable_Wrap(t));
    return r;
}

using Args = PyObject *const *;

// Runs a call of N positional arguments; C++ exceptions become Python errors.
template <Py_ssize_t N, PyObject *(*F)(Args)>
PyObject *guarded(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    try {
        if (n != N)
            throw TypeErr("wrong number of arguments");
        return F(a);
    } catch (const PyErrSet &) {
    } catch (const MoeErr &e) {
        PyObject *x = PyObject_CallFunction(g_moe_error, "is", e.code, e.what);
        if (x) {
            PyErr_SetObject(g_moe_error, x);
            Py_DECREF(x);
        }
    } catch (const ValueErr &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const TypeErr &e) {
        PyErr_SetString(PyExc_TypeError, e.what());
    } catch (const c10::Error &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    } catch (...) {
        PyErr_SetString(PyExc_RuntimeError, "unknown error");
    }
    return nullptr;
}

// ------------------------------------------------------------------ layer norm ----------
// A norm's weight and bias [H] (or None): both of x's type or both fp32.
struct Affine {
    void *weight, *bias;
    int dtype;
    at::ScalarType type;
};
Affine affine(PyObject *weight, PyObject *bias, int64_t H, const First &f)
{
    at::ScalarType type = f.type;
    if (!none(weight))
        type = tensor(weight, "weight").scalar_type();
    else if (!none(bias))
        type = tensor(bias, "bias").scalar_type();
    if (type != f.type && type != at::kFloat)
        throw TypeErr("weight and bias: dtype " + dtype_name(type) + " is neither " + dtype_name(f.type) + " nor Float");
    return {flat_or_null(weight, "weight", {H}, type, f.dev), flat_or_null(bias, "bias", {H}, type, f.dev), code_of(type), type};
}

// (x, weight, bias, eps)
PyObject *layer_norm(Args a)
{
    const at::Tensor &x = tensor(a[0], "x");
    const First f = first(x, "x");
    const Matrix m = matrix(x, "x", f);
    const Affine w = affine(a[1], a[2], m.width, f);
    at::Tensor y = make({m.rows, m.width}, f.type, f.dev), mean = make({m.rows}, at::kFloat, f.dev), rstd = make({m.rows}, at::kFloat, f.dev);
    check(moe_layer_norm(count(m.rows, "x"), count(m.width, "x"), m.p, m.ld, f.dtype, w.weight, w.bias, w.dtype, real(a[3]),
                         y.data_ptr(), mean.data_ptr<float>(), rstd.data_ptr<float>(), current_stream(f.dev)),
          "moe_layer_norm");
    return tuple_of({y, mean, rstd});
}

// (x, weight, bias, eps, pow2_scales)
PyObject *layer_norm_fp8(Args a)
{
    const at::Tensor &x = tensor(a[0], "x");
    const First f = first(x, "x");
    const Matrix m = matrix(x, "x", f);
    const Affine w = affine(a[1], a[2], m.width, f);
    at::Tensor q = make({m.rows, m.width}, at::kByte, f.dev), sf = make({m.rows, m.width / 128}, at::kFloat, f.dev);
    check(moe_layer_norm_fp8(count(m.rows, "x"), count(m.width, "x"), m.p, m.ld, f.dtype, w.weight, w.bias, w.dtype, real(a[3]),
                             truth(a[4]), q.data_ptr<uint8_t>(), sf.data_ptr<float>(), current_stream(f.dev)),
          "moe_layer_norm_fp8");
    return tuple_of({q, sf});
}

// (dy, x, weight, mean, rstd, params fp32, dweight wanted, dbias wanted)
PyObject *layer_norm_backward(Args a)
{
    const at::Tensor &x = tensor(a[1], "x");
    const First f = first(x, "x");
    const Matrix m = matrix(x, "x", f), d = matrix(tensor(a[0], "dy"), "dy", f, m.rows, m.width);
    Affine w = affine(a[2], Py_None, m.width, f);
    if (none(a[2]) && truth(a[5])) {
        w.type = at::kFloat;
        w.dtype = MOE_F32;
    }
    const void *mean = flat(tensor(a[3], "mean"), "mean", {m.rows}, at::kFloat, f.dev);
    const void *rstd = flat(tensor(a[4], "rstd"), "rstd", {m.rows}, at::kFloat, f.dev);
    const int T = count(m.rows, "x"), H = count(m.width, "x");
    const bool want_w = truth(a[6]), want_b = truth(a[7]);
    uint64_t need = 0;
    if (want_w || want_b)
        check(moe_layer_norm_backward_workspace(T, H, &need), "moe_layer_norm_backward_workspace");
    const Workspace ws(need);
    at::Tensor dx = make({m.rows, m.width}, f.type, f.dev), dweight, dbias;   // (an undefined tensor is None)
    if (want_w)
        dweight = make({m.width}, w.type, f.dev);
    if (want_b)
        dbias = make({m.width}, w.type, f.dev);
    check(moe_layer_norm_backward(T, H, d.p, d.ld, m.p, m.ld, f.dtype, w.weight, w.dtype, static_cast<const float *>(mean),
                                  static_cast<const float *>(rstd), dx.data_ptr(),
                                  want_w ? dweight.data_ptr() : nullptr, want_b ? dbias.data_ptr() : nullptr, ws.get(), need, current_stream(f.dev)),
          "moe_layer_norm_backward");
    return tuple_of({dx, dweight, dbias});
}

// ------------------------------------------------------------------ router --------------
// (logits, topk, token_mask, renormalize)
PyObject *route_topk(Args a)
{
    const at::Tensor &l = tensor(a[0], "logits");
    const First f = first(l, "logits");
    const Matrix m = matrix(l, "logits", f);
    const int k = small(a[1], "topk");
    const void *mask = flat_or_null(a[2], "token_mask", {m.rows}, at::kBool, f.dev);
    at::Tensor idx = make({m.rows, std::max(k, 0)}, at::kLong, f.dev), w = make({m.rows, std::max(k, 0)}, at::kFloat, f.dev);
    check(moe_route_topk(count(m.rows, "logits"), count(m.width, "logits"), k, m.p, m.ld, f.dtype, static_cast<const uint8_t *>(mask),
                         truth(a[3]), idx.data_ptr<int64_t>(), w.data_ptr<float>(), current_stream(f.dev)),
          "moe_route_topk");
    return tuple_of({idx, w});
}

const at::Tensor &slots(PyObject *o)
{
    const at::Tensor &idx = tensor(o, "idx");
    if (idx.dim() != 2)
        throw ValueErr("idx: shape " + shape_of(idx) + " is not [T, topk]");
    return idx;
}

// (dw, idx, w, logits, renormalize)
PyObject *route_topk_backward(Args a)
{
    const at::Tensor &l = tensor(a[3], "logits"), &idx = slots(a[1]);
    const First f = first(l, "logits");
    const Matrix m = matrix(l, "logits", f);
    const int64_t k = idx.size(1);
    const void *pi = flat(idx, "idx", {m.rows, k}, at::kLong, f.dev);
    const void *pw = flat(tensor(a[2], "w"), "w", {m.rows, k}, at::kFloat, f.dev);
    const void *pd = flat(tensor(a[0], "dw"), "dw", {m.rows, k}, at::kFloat, f.dev);
    at::Tensor d = make({m.rows, m.width}, f.type, f.dev);
    check(moe_route_topk_backward(count(m.rows, "logits"), count(m.width, "logits"), count(k, "idx"), static_cast<const float *>(pd),
                                  static_cast<const int64_t *>(pi), static_cast<const float *>(pw), m.p, m.ld, f.dtype, truth(a[4]),
                                  d.data_ptr(), current_stream(f.dev)),
          "moe_route_topk_backward");
    return THPVariable_Wrap(d);
}

// (idx, E)
PyObject *expert_order(Args a)
{
    const at::Tensor &idx = slots(a[0]);
    if (!idx.is_cuda())
        throw ValueErr("idx must be a CUDA tensor");
    const int dev = idx.device().index();
    if (dev != c10::cuda::current_device())
        throw ValueErr("idx is not on the current device");
    const int64_t T = idx.size(0), k = idx.size(1);
    const void *pi = flat(idx, "idx", {T, k}, at::kLong, dev);
    const int E = small(a[1], "E");
    uint64_t need = 0;
    check(moe_expert_order_workspace(count(T, "idx"), count(k, "idx"), E, &need), "moe_expert_order_workspace");
    const Workspace ws(need);
    at::Tensor offsets = make({E + 1}, at::kInt, dev), rows = make({T, k}, at::kInt, dev), status = make({1}, at::kInt, dev);
    check(moe_expert_order(count(T, "idx"), count(k, "idx"), E, static_cast<const int64_t *>(pi), offsets.data_ptr<int32_t>(),
                           rows.data_ptr<int32_t>(), status.data_ptr<int32_t>(), ws.get(), need,
                           current_stream(dev)),
          "moe_expert_order");
    return tuple_of({offsets, rows, status});
}

// ------------------------------------------------------------------ rows ----------------
struct Rows {
    int64_t T, k;
    const int32_t *p;
};
Rows order_rows(PyObject *o, int dev)
{
    const at::Tensor &t = tensor(o, "rows");
    if (t.dim() != 2)
        throw ValueErr("rows: shape " + shape_of(t) + " is not [T, topk]");
    return {t.size(0), t.size(1), static_cast<const int32_t *>(flat(t, "rows", {t.size(0), t.size(1)}, at::kInt, dev))};
}
struct Groups {
    int E;
    const int32_t *p;
};
Groups groups(PyObject *o, int dev, int64_t E = -1)
{
    const at::Tensor &t = tensor(o, "offsets");
    if (t.dim() != 1 || t.size(0) < 2 || (E >= 0 && t.size(0) != E + 1))
        throw ValueErr("offsets: shape " + shape_of(t) + " is not [E+1]");
    return {count(t.size(0) - 1, "offsets"), static_cast<const int32_t *>(flat(t, "offsets", {t.size(0)}, at::kInt, dev))};
}

// (x, rows, offsets)
PyObject *gather_rows(Args a)
{
    const at::Tensor &x = tensor(a[0], "x");
    const First f = first(x, "x");
    const Rows r = order_rows(a[1], f.dev);
    const Matrix m = matrix(x, "x", f, r.T);
    const Groups g = groups(a[2], f.dev);
    at::Tensor out = make({r.T * r.k, m.width}, f.type, f.dev);
    check(moe_gather_rows(count(r.T, "rows"), count(r.k, "rows"), count(m.width, "x"), g.E, r.T * r.k, m.p, m.ld, f.dtype, r.p, g.p,
                          out.data_ptr(), current_stream(f.dev)),
          "moe_gather_rows");
    return THPVariable_Wrap(out);
}

// (y, rows, w)
PyObject *combine_rows(Args a)
{
    const at::Tensor &y = tensor(a[0], "y");
    const First f = first(y, "y");
    const int64_t M = y.size(0), H = y.size(1);
    const void *py = flat(y, "y", {M, H}, f.type, f.dev);
    const Rows r = order_rows(a[1], f.dev);
    const void *pw = flat_or_null(a[2], "w", {r.T, r.k}, at::kFloat, f.dev);
    at::Tensor out = make({r.T, H}, f.type, f.dev);
    check(moe_combine_rows(count(r.T, "rows"), count(r.k, "rows"), count(H, "y"), M, py, f.dtype, r.p, static_cast<const float *>(pw),
                           out.data_ptr(), current_stream(f.dev)),
          "moe_combine_rows");
    return THPVariable_Wrap(out);
}

// (dout, y, rows, w, offsets, dw wanted)
PyObject *combine_rows_backward(Args a)
{
    const at::Tensor &y = tensor(a[1], "y");
    const First f = first(y, "y");
    const int64_t M = y.size(0), H = y.size(1);
    const void *py = flat(y, "y", {M, H}, f.type, f.dev);
    const Rows r = order_rows(a[2], f.dev);
    const Groups g = groups(a[4], f.dev);
    const Matrix d = matrix(tensor(a[0], "dout"), "dout", f, r.T, H);
    const void *pw = flat_or_null(a[3], "w", {r.T, r.k}, at::kFloat, f.dev);
    at::Tensor dy = make({M, H}, f.type, f.dev), dw;   // (an undefined tensor is None)
    if (truth(a[5]))
        dw = make({r.T, r.k}, at::kFloat, f.dev);
    check(moe_combine_rows_backward(count(r.T, "rows"), count(r.k, "rows"), count(H, "y"), g.E, M, d.p, d.ld, py, f.dtype, r.p,
                                    static_cast<const float *>(pw), g.p, dy.data_ptr(),
                                    dw.defined() ? dw.data_ptr<float>() : nullptr, current_stream(f.dev)),
          "moe_combine_rows_backward");
    return tuple_of({dy, dw});
}

// ------------------------------------------------------------------ grouped products ----
// The bytes of a tensor: rows of `width` bytes, `pitch` apart (pitch >= width).
struct Bytes {
    const char *p;
    int64_t rows, width, pitch;
};
Bytes bytes_of(const Matrix &m, size_t size)
{
    const int64_t b = static_cast<int64_t>(size);
    return {static_cast<const char *>(m.p), m.rows, m.width * b, m.ld * b};
}
Bytes bytes_of(const void *p, int64_t elements, size_t size)
{
    const int64_t n = elements * static_cast<int64_t>(size);
    return {static_cast<const char *>(p), 1, n, n};
}
bool overlap(Bytes a, Bytes b)
{
    if (a.rows == 0 || b.rows == 0 || a.width == 0 || b.width == 0)
        return false;
    if (a.p >= b.p + b.pitch * (b.rows - 1) + b.width || b.p >= a.p + a.pitch * (a.rows - 1) + a.width)
        return false;
    // the tensors lie among each other: parts of the rows of one buffer, perhaps
    if (a.rows > b.rows)
        std::swap(a, b);
    for (int64_t r = 0; r < a.rows; ++r) {
        const char *lo = a.p + r * a.pitch, *hi = lo + a.width;
        if (hi <= b.p)
            continue;
        // the last row of b that starts before this row's end is the only one of those that may pass its start
        const int64_t j = std::min((hi - 1 - b.p) / b.pitch, b.rows - 1);
        if (b.p + j * b.pitch + b.width > lo)
            return true;
    }
    return false;
}
// A product's blocks write its output while others still read the inputs.
void apart(const Bytes &out, const Bytes &in, const char *name)
{
    if (overlap(out, in))
        throw ValueErr(std::string("out overlaps ") + name);
}

struct Weights {
    int64_t E, N, K;
    const void *p;
};
Weights weights(PyObject *o, const First &f)
{
    const at::Tensor &w = tensor(o, "w");
    if (w.dim() != 3)
        throw ValueErr("w: shape " + shape_of(w) + " is not [E, N, K]");
    return {w.size(0), w.size(1), w.size(2), flat(w, "w", {w.size(0), w.size(1), w.size(2)}, f.type, f.dev)};
}

// (rows of x or dy, w, offsets, out): TO_N: out[r] = w[e] @ rows[r], else rows[r] @ w[e]
template <bool TO_N>
PyObject *grouped(Args a)
{
    const char *name = TO_N ? "x" : "dy";
    const at::Tensor &x = tensor(a[0], name);
    const First f = first(x, name, true);
    const Weights w = weights(a[1], f);
    const Matrix m = matrix(x, name, f, -1, TO_N ? w.K : w.N);
    const Groups g = groups(a[2], f.dev, w.E);
    const int64_t width = TO_N ? w.N : w.K;
    at::Tensor fresh;
    Matrix o;
    if (none(a[3])) {
        fresh = make({m.rows, width}, f.type, f.dev);
        o = {m.rows, width, std::max<int64_t>(width, 1), fresh.data_ptr()};
    } else {
        o = matrix(tensor(a[3], "out"), "out", f, m.rows, width);
        const Bytes to = bytes_of(o, 2);
        apart(to, bytes_of(m, 2), name);
        apart(to, bytes_of(w.p, w.E * w.N * w.K, 2), "w");
        apart(to, bytes_of(g.p, w.E + 1, 4), "offsets");
    }
    const auto call = TO_N ? moe_grouped_mm : moe_grouped_mm_dx;
    uint64_t need = 0;
    check(moe_grouped_mm_workspace(m.rows, count(w.E, "w"), count(w.N, "w"), count(w.K, "w"), &need), "moe_grouped_mm_workspace");
    const Workspace ws(need);
    check(call(m.rows, g.E, static_cast<int>(w.N), static_cast<int>(w.K), m.p, m.ld, w.p, g.p, o.p, o.ld, f.dtype,
               ws.get(), need, current_stream(f.dev)),
          TO_N ? "moe_grouped_mm" : "moe_grouped_mm_dx");
    if (none(a[3]))
        return THPVariable_Wrap(fresh);
    written(tensor(a[3], "out"));
    Py_INCREF(a[3]);
    return a[3];
}

// (dy, x, offsets, out, accumulate, fp32 out)
PyObject *grouped_dw(Args a)
{
    const at::Tensor &x = tensor(a[1], "x");
    const First f = first(x, "x", true);
    const Matrix m = matrix(x, "x", f), d = matrix(tensor(a[0], "dy"), "dy", f, m.rows);
    const Groups g = groups(a[2], f.dev);
    const int64_t N = d.width, K = m.width;
    const bool accumulate = truth(a[4]);
    at::Tensor fresh;
    at::ScalarType type = truth(a[5]) ? at::kFloat : f.type;
    void *po;
    if (none(a[3])) {
        if (accumulate)
            throw ValueErr("accumulate needs an out to add to");
        fresh = make({g.E, N, K}, type, f.dev);
        po = fresh.data_ptr();
    } else {
        const at::Tensor &out = tensor(a[3], "out");
        type = out.scalar_type();
        if (type != f.type && type != at::kFloat)
            throw TypeErr("out: dtype " + dtype_name(type) + " is neither " + dtype_name(f.type) + " nor Float");
        po = flat(out, "out", {g.E, N, K}, type, f.dev);
        const Bytes to = bytes_of(po, g.E * N * K, type == at::kFloat ? 4 : 2);
        apart(to, bytes_of(d, 2), "dy");
        apart(to, bytes_of(m, 2), "x");
        apart(to, bytes_of(g.p, g.E + 1, 4), "offsets");
    }
    uint64_t need = 0;
    check(moe_grouped_mm_dw_workspace(m.rows, g.E, count(N, "dy"), count(K, "x"), &need), "moe_grouped_mm_dw_workspace");
    const Workspace ws(need);
    check(moe_grouped_mm_dw(m.rows, g.E, count(N, "dy"), count(K, "x"), d.p, d.ld, m.p, m.ld, g.p, po, f.dtype, code_of(type), accumulate,
                            ws.get(), need, current_stream(f.dev)),
          "moe_grouped_mm_dw");
    if (none(a[3]))
        return THPVariable_Wrap(fresh);
    written(tensor(a[3], "out"));
    Py_INCREF(a[3]);
    return a[3];
}

// ()
PyObject *get_error(Args)
{
    int st = 0;
    void *const stream = current_stream(c10::cuda::current_device());
    int rc;
    Py_BEGIN_ALLOW_THREADS   // it waits for the stream, whose work may itself wait for a Python thread
    rc = moe_ops_get_error(&st, stream);
    Py_END_ALLOW_THREADS
    check(rc, "moe_ops_get_error");
    return PyLong_FromLong(st);
}

#define CALL(name, n, fn) {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void *>(guarded<n, fn>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {CALL("layer_norm", 4, layer_norm),
                         CALL("layer_norm_fp8", 5, layer_norm_fp8),
                         CALL("layer_norm_backward", 8, layer_norm_backward),
                         CALL("route_topk", 4, route_topk),
                         CALL("route_topk_backward", 5, route_topk_backward),
                         CALL("expert_order", 2, expert_order),
                         CALL("gather_rows", 3, gather_rows),
                         CALL("combine_rows", 3, combine_rows),
                         CALL("combine_rows_backward", 6, combine_rows_backward),
                         CALL("grouped_mm", 4, grouped<true>),
                         CALL("grouped_mm_dx", 4, grouped<false>),
                         CALL("grouped_mm_dw", 6, grouped_dw),
                         CALL("get_error", 0, get_error),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_ops", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__ops()
{
    PyObject *native = PyImport_ImportModule("combine_persistent_warp_gb300.native");
    if (!native)
        return nullptr;
    g_moe_error = PyObject_GetAttrString(native, "MoeError");
    Py_DECREF(native);
    return g_moe_error ? PyModule_Create(&module_def) : nullptr;
}
