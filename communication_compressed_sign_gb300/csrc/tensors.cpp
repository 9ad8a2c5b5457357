// tensors.cpp -- the Python module _tensors: calls of the block operators' C ABI
// (include/lioncub_block.h) from torch tensors.
//
// A small call is bound by what the host does, and a tensor's type, device, sizes
// and strides cost a Python call each: a norm of 8 rows took 7.5 us through Python
// structs, of which 1.9 are the launch.  Here they are read from the tensors
// themselves.  Nothing is allocated or copied; arguments that do not fit raise
// ValueError, and the functions return the C function's code.
#include <Python.h>

#include <ATen/core/grad_mode.h>
#include <c10/core/AutogradState.h>
#include <torch/csrc/autograd/python_variable.h>

#include <exception>
#include <sstream>
#include <string>

#include "lioncub_block.h"

namespace {

// The library's functions, by their addresses in the library that is loaded (see bind).
struct Functions {
    decltype(&lioncub_rms_norm_forward) rms_norm_forward;
    decltype(&lioncub_rms_norm_backward) rms_norm_backward;
    decltype(&lioncub_pack8) pack8;
    decltype(&lioncub_unpack8) unpack8;
    decltype(&lioncub_activation_forward) activation_forward;
    decltype(&lioncub_activation_backward) activation_backward;
    decltype(&lioncub_rotary_apply) rotary_apply;
} lib;

PyObject *n_codes, *n_scales, *n_group;  // attribute names of a Packed

// What does not fit: becomes a ValueError.
struct Refusal : std::exception {
    std::string what_;
    explicit Refusal(std::string s) : what_(std::move(s)) {}
    const char* what() const noexcept override { return what_.c_str(); }
};
struct PythonError : std::exception {};  // already set

template <typename... Parts>
[[noreturn]] void refuse(const Parts&... parts)
{
    std::ostringstream s;
    (s << ... << parts);
    throw Refusal(s.str());
}

std::string shape_of(const at::Tensor& t)
{
    std::ostringstream s;
    s << "(";
    for (int64_t i = 0; i < t.dim(); ++i)
        s << (i ? ", " : "") << t.size(i);
    s << (t.dim() == 1 ? ",)" : ")");
    return s.str();
}

const at::Tensor& tensor(PyObject* o, const char* name)
{
    if (!THPVariable_Check(o))
        refuse(name, " must be a tensor");
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.layout() != at::kStrided)
        refuse(name, " must be a dense tensor");
    if (t.is_neg())
        refuse(name, " is a negated view, whose memory holds other numbers: pass resolve_neg() of it");
    return t;
}

bool on_device(const at::Tensor& t, int64_t device) { return t.is_cuda() && t.get_device() == device; }

void check_gradient(const at::Tensor& t, const char* name)
{
    if (t.requires_grad() && at::GradMode::is_enabled())
        refuse(name, " requires a gradient, but results are not part of torch's graph: call under torch.no_grad() or pass a detached tensor");
    if (t._fw_grad(0).defined() && c10::AutogradState::get_tls_state().get_fw_grad_mode())
        refuse(name, " has a tangent (a forward-mode derivative), but results have none: pass its primal value");
}

int row_type(const at::Tensor& t, const char* name, int64_t device)
{
    const at::ScalarType type = t.scalar_type();
    if ((type != at::kBFloat16 && type != at::kFloat) || !on_device(t, device))
        refuse(name, " must be a bfloat16 or float32 tensor on cuda:", device);
    check_gradient(t, name);
    return type == at::kBFloat16 ? LIONCUB_ROWS_BF16 : LIONCUB_ROWS_F32;
}

// The distance between the rows of a tensor (..., cols) of n rows.
int64_t step_of(const at::Tensor& t, const char* name, int64_t n, int64_t cols)
{
    if (t.is_contiguous())
        return cols;
    const int64_t dims = t.dim();
    if (cols > 1 && t.stride(dims - 1) != 1)
        refuse(name, ": the columns of a row must be contiguous");
    int64_t step = cols, reach = 0;
    bool first = true;
    for (int64_t i = dims - 2; i >= 0; --i) {  // from the inner dimensions outwards
        const int64_t size = t.size(i), stride = t.stride(i);
        if (size == 1)
            continue;
        if (first)
            step = reach = stride;
        else if (stride != reach)
            refuse(name, ": its rows do not lie a fixed distance apart");
        first = false;
        reach *= size;
    }
    return n > 1 ? step : cols;
}

// What a call does with a tensor.  One that is written gets memory of its own first
// if it shares that of another until then (a lazy clone).
enum Use { kRead, kWrite };

void* address(const at::Tensor& t, Use use) { return use == kWrite ? t.mutable_data_ptr() : const_cast<void*>(t.const_data_ptr()); }

// A matrix argument; None is a null pointer.
struct Matrix {
    lioncub_rows rows;
    const lioncub_rows* p = nullptr;
    Matrix() = default;
    Matrix(PyObject* o, const char* name, int64_t n, int64_t cols, int64_t device, Use use = kRead)
    {
        if (o == Py_None)
            return;
        const at::Tensor& t = tensor(o, name);
        const int type = row_type(t, name, device);
        if (!t.dim() || t.size(-1) != cols || t.numel() != n * cols)
            refuse(name, " must have ", n, " rows of ", cols, " columns (got ", shape_of(t), ")");
        rows = {address(t, use), step_of(t, name, n, cols), type, 0};
        p = &rows;
    }
};

// A matrix in 8 bits: an object with codes, scales and group.
struct PackedMatrix {
    lioncub_packed packed;
    const lioncub_packed* p = nullptr;
    PackedMatrix() = default;
    PackedMatrix(PyObject* o, const char* name, int64_t n, int64_t cols, int64_t device, Use use = kRead)
    {
        if (o == Py_None)
            return;
        Held codes(o, n_codes), scales(o, n_scales), group(o, n_group);
        const std::string prefix(name);
        const at::Tensor& c = tensor(codes.o, (prefix + ": codes").c_str());
        const at::Tensor& s = tensor(scales.o, (prefix + ": scales").c_str());
        const long long g = PyLong_AsLongLong(group.o);
        if (g == -1 && PyErr_Occurred())
            throw PythonError();
        const at::ScalarType type = c.scalar_type();
        if ((type != at::kChar && type != at::kFloat8_e4m3fn) || !on_device(c, device))
            refuse(name, ": codes must be an int8 or float8_e4m3fn tensor on cuda:", device);
        if (s.scalar_type() != at::kFloat || !on_device(s, device))
            refuse(name, ": scales must be a float32 tensor on cuda:", device);
        check_gradient(s, name);
        const int64_t groups = g > 0 ? (cols + g - 1) / g : 1;
        if (!c.dim() || c.size(-1) != cols || c.numel() != n * cols)
            refuse(name, " must have ", n, " rows of ", cols, " columns (got ", shape_of(c), ")");
        if (!s.dim() || s.size(-1) != groups || s.numel() != n * groups)
            refuse(name, " must have ", n, " rows of ", groups, " scales (got ", shape_of(s), ")");
        packed = {address(c, use), static_cast<float*>(address(s, use)), step_of(c, name, n, cols), step_of(s, name, n, groups),
                  static_cast<int32_t>(g < -1 || g > 1 << 30 ? -1 : g), type == at::kChar ? LIONCUB_CODES_INT8 : LIONCUB_CODES_E4M3};
        p = &packed;
    }

private:
    struct Held {  // an attribute, while it is used
        PyObject* o;
        Held(PyObject* from, PyObject* name) : o(PyObject_GetAttr(from, name))
        {
            if (!o)
                throw PythonError();
        }
        ~Held() { Py_DECREF(o); }
        Held(const Held&) = delete;
        Held& operator=(const Held&) = delete;
    };
};

// An argument that is a matrix or one in 8 bits.
struct Either {
    Matrix m;
    PackedMatrix c;
    Either(PyObject* o, const char* name, int64_t n, int64_t cols, int64_t device, Use use = kRead)
    {
        if (o == Py_None)
            return;
        if (THPVariable_Check(o))
            fill(m, Matrix(o, name, n, cols, device, use));
        else
            fill(c, PackedMatrix(o, name, n, cols, device, use));
    }

private:
    static void fill(Matrix& to, const Matrix& from)
    {
        to.rows = from.rows;
        to.p = &to.rows;
    }
    static void fill(PackedMatrix& to, const PackedMatrix& from)
    {
        to.packed = from.packed;
        to.p = &to.packed;
    }
};

float* vector(PyObject* o, const char* name, int64_t n, int64_t device, Use use)
{
    if (o == Py_None)
        return nullptr;
    const at::Tensor& t = tensor(o, name);
    if (t.scalar_type() != at::kFloat || !on_device(t, device) || t.numel() != n || !t.is_contiguous())
        refuse(name, " must be a contiguous float32 tensor of ", n, " elements on cuda:", device);
    check_gradient(t, name);
    return static_cast<float*>(address(t, use));
}

int64_t integer(PyObject* o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred())
        throw PythonError();
    return v;
}

template <typename T>
T pointer(PyObject* o)
{
    void* p = PyLong_AsVoidPtr(o);
    if (!p && PyErr_Occurred())
        throw PythonError();
    return reinterpret_cast<T>(p);
}

// (rows, columns) of x, which must be on the current device
struct Size {
    int64_t n, cols;
    Size(const at::Tensor& t, const char* name, int64_t device)
    {
        if (!on_device(t, device))
            refuse(name, " must be on the current CUDA device");
        if (!t.dim())
            refuse(name, " must have at least one dimension");
        cols = t.size(-1);
        n = cols ? t.numel() / cols : 0;
    }
};

int64_t rows_of(PyObject* o, const char* name, int64_t dim)
{
    const at::Tensor& t = tensor(o, name);
    if (!t.dim() || t.size(-1) != dim)
        refuse(name, " must have rows of ", dim, " columns (got ", shape_of(t), ")");
    return t.numel() / dim;
}

template <typename Call>
PyObject* code_of(Call&& call)
{
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = call();
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

// Runs a function's body; no C++ exception leaves it.
template <typename Body>
PyObject* guarded(const char* name, Py_ssize_t got, Py_ssize_t wanted, Body&& body)
{
    if (got != wanted) {
        PyErr_Format(PyExc_TypeError, "%s takes %zd arguments (got %zd)", name, wanted, got);
        return nullptr;
    }
    try {
        return body();
    } catch (const PythonError&) {
    } catch (const Refusal& e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// (handle, dim, device, x, residual, weight, summed, saved, rstd, out, stream)
PyObject* rms_norm_forward(PyObject*, PyObject* const* a, Py_ssize_t count)
{
    return guarded("rms_norm_forward", count, 11, [&] {
        const auto h = pointer<lioncub_rms_norm_t>(a[0]);
        const int64_t D = integer(a[1]), dev = integer(a[2]), n = rows_of(a[3], "x", D);
        const Matrix x(a[3], "x", n, D, dev), residual(a[4], "residual", n, D, dev), weight(a[5], "weight", 1, D, dev),
            summed(a[6], "summed", n, D, dev, kWrite);
        const PackedMatrix saved(a[7], "saved", n, D, dev, kWrite);
        float* const rstd = vector(a[8], "rstd", n, dev, kWrite);
        const Either out(a[9], "out", n, D, dev, kWrite);
        const auto stream = pointer<lioncub_stream_t>(a[10]);
        return code_of([&] {
            return lib.rms_norm_forward(h, n, x.p, residual.p, weight.p, summed.p, saved.p, rstd, out.m.p, out.c.p, stream);
        });
    });
}

// (handle, dim, device, dout, saved, rstd, weight, residual_grad, dx, weight_base, weight_grad, again, stream)
PyObject* rms_norm_backward(PyObject*, PyObject* const* a, Py_ssize_t count)
{
    return guarded("rms_norm_backward", count, 13, [&] {
        const auto h = pointer<lioncub_rms_norm_t>(a[0]);
        const int64_t D = integer(a[1]), dev = integer(a[2]), n = rows_of(a[3], "dout", D);
        const Matrix dout(a[3], "dout", n, D, dev);
        const Either saved(a[4], "saved", n, D, dev);
        const float* const rstd = vector(a[5], "rstd", n, dev, kRead);
        const Matrix weight(a[6], "weight", 1, D, dev), residual_grad(a[7], "residual_grad", n, D, dev),
            dx(a[8], "out", n, D, dev, kWrite), base(a[9], "weight_base", 1, D, dev), grad(a[10], "weight_grad", 1, D, dev, kWrite),
            again(a[11], "again", n, D, dev, kWrite);
        const auto stream = pointer<lioncub_stream_t>(a[12]);
        return code_of([&] {
            return lib.rms_norm_backward(h, n, dout.p, saved.m.p, saved.c.p, rstd, weight.p, residual_grad.p, dx.p, base.p, grad.p, again.p,
                                         stream);
        });
    });
}

// (device, x, out, stream)
PyObject* pack8(PyObject*, PyObject* const* a, Py_ssize_t count)
{
    return guarded("pack8", count, 4, [&] {
        const int64_t dev = integer(a[0]);
        const Size size(tensor(a[1], "x"), "x", dev);
        const Matrix x(a[1], "x", size.n, size.cols, dev);
        const PackedMatrix out(a[2], "out", size.n, size.cols, dev, kWrite);
        const auto stream = pointer<lioncub_stream_t>(a[3]);
        return code_of([&] { return lib.pack8(size.n, size.cols, x.p, out.p, stream); });
    });
}

// (device, codes of x, x, out, stream)
PyObject* unpack8(PyObject*, PyObject* const* a, Py_ssize_t count)
{
    return guarded("unpack8", count, 5, [&] {
        const int64_t dev = integer(a[0]);
        const Size size(tensor(a[1], "x"), "x", dev);
        const PackedMatrix x(a[2], "x", size.n, size.cols, dev);
        const Matrix out(a[3], "out", size.n, size.cols, dev, kWrite);
        const auto stream = pointer<lioncub_stream_t>(a[4]);
        return code_of([&] { return lib.unpack8(size.n, size.cols, x.p, out.p, stream); });
    });
}

// (device, kind, x, up, out, saved, saved_up, stream)
PyObject* activation_forward(PyObject*, PyObject* const* a, Py_ssize_t count)
{
    return guarded("activation_forward", count, 8, [&] {
        const int64_t dev = integer(a[0]), kind = integer(a[1]);
        const Size size(tensor(a[2], "x"), "x", dev);
        const int64_t n = size.n, cols = size.cols;
        const Matrix x(a[2], "x", n, cols, dev), up(a[3], "up", n, cols, dev), out(a[4], "out", n, cols, dev, kWrite);
        const PackedMatrix saved(a[5], "saved", n, cols, dev, kWrite), saved_up(a[6], "saved_up", n, cols, dev, kWrite);
        const auto stream = pointer<lioncub_stream_t>(a[7]);
        return code_of([&] {
            return lib.activation_forward(n, cols, static_cast<int>(kind), x.p, up.p, out.p, saved.p, saved_up.p, stream);
        });
    });
}

// (device, kind, dout, x, up, dx, dup, again, stream)
PyObject* activation_backward(PyObject*, PyObject* const* a, Py_ssize_t count)
{
    return guarded("activation_backward", count, 9, [&] {
        const int64_t dev = integer(a[0]), kind = integer(a[1]);
        const Size size(tensor(a[2], "dout"), "dout", dev);
        const int64_t n = size.n, cols = size.cols;
        const Matrix dout(a[2], "dout", n, cols, dev);
        const Either x(a[3], "x", n, cols, dev), up(a[4], "up", n, cols, dev);
        const Matrix dx(a[5], "dx", n, cols, dev, kWrite), dup(a[6], "dup", n, cols, dev, kWrite), again(a[7], "again", n, cols, dev, kWrite);
        const auto stream = pointer<lioncub_stream_t>(a[8]);
        return code_of([&] {
            return lib.activation_backward(n, cols, static_cast<int>(kind), dout.p, x.m.p, up.m.p, x.c.p, up.c.p, dx.p, dup.p, again.p, stream);
        });
    });
}

struct HeadsArgument {
    lioncub_heads heads;
    const lioncub_heads* p = nullptr;
    HeadsArgument(PyObject* o, const char* name, int64_t batch, int64_t places, int64_t head_dim, int64_t device, Use use = kRead)
    {
        if (o == Py_None)
            return;
        const at::Tensor& t = tensor(o, name);
        const int type = row_type(t, name, device);
        const int64_t lead = t.dim() - 3;
        if ((lead != 0 && lead != 1) || (lead ? t.size(0) : 1) != batch || t.size(lead) != places || t.size(lead + 2) != head_dim)
            refuse(name, " must be (", batch, ", ", places, ", heads, ", head_dim, ") (got ", shape_of(t), ")");
        if (t.stride(lead + 2) != 1 && t.numel())
            refuse(name, ": the columns of a head must be contiguous");
        if (t.size(lead + 1) > INT32_MAX)
            refuse(name, " has too many heads");
        heads = {address(t, use), lead ? t.stride(0) : 0, t.stride(lead), t.stride(lead + 1), static_cast<int32_t>(t.size(lead + 1)), type};
        p = &heads;
    }
};

// (handle, head_dim, device, q, q_out, k, k_out, positions, first_position, inverse, stream)
PyObject* rotary_apply(PyObject*, PyObject* const* a, Py_ssize_t count)
{
    return guarded("rotary_apply", count, 11, [&] {
        const auto h = pointer<lioncub_rotary_t>(a[0]);
        const int64_t D = integer(a[1]), dev = integer(a[2]);
        const at::Tensor& first = tensor(a[3], "q");
        if (first.dim() != 3 && first.dim() != 4)
            refuse("q must be (batch, places, heads, ", D, ") (got ", shape_of(first), ")");
        const int64_t batch = first.dim() == 4 ? first.size(0) : 1, places = first.size(first.dim() - 3);
        const HeadsArgument q(a[3], "q", batch, places, D, dev), q_out(a[4], "q_out", batch, places, D, dev, kWrite),
            k(a[5], "k", batch, places, D, dev), k_out(a[6], "k_out", batch, places, D, dev, kWrite);
        lioncub_sequences s = {nullptr, batch, places, integer(a[8]), LIONCUB_INDEX_I64, 0};
        if (a[7] != Py_None) {
            const at::Tensor& t = tensor(a[7], "positions");
            const at::ScalarType type = t.scalar_type();
            if ((type != at::kLong && type != at::kInt) || !on_device(t, dev) || !t.is_contiguous() || t.numel() != batch * places)
                refuse("positions must be a contiguous int64 or int32 tensor of ", batch, " x ", places, " on cuda:", dev);
            s.positions = t.const_data_ptr();
            s.index_type = type == at::kLong ? LIONCUB_INDEX_I64 : LIONCUB_INDEX_I32;
        }
        const int64_t inverse = integer(a[9]);
        const auto stream = pointer<lioncub_stream_t>(a[10]);
        return code_of([&] { return lib.rotary_apply(h, &s, q.p, q_out.p, k.p, k_out.p, static_cast<int>(inverse), stream); });
    });
}

// (addresses of the library's functions, in the order of Functions)
PyObject* bind(PyObject*, PyObject* const* a, Py_ssize_t count)
{
    return guarded("bind", count, 7, [&]() -> PyObject* {
        Functions f;
        f.rms_norm_forward = pointer<decltype(f.rms_norm_forward)>(a[0]);
        f.rms_norm_backward = pointer<decltype(f.rms_norm_backward)>(a[1]);
        f.pack8 = pointer<decltype(f.pack8)>(a[2]);
        f.unpack8 = pointer<decltype(f.unpack8)>(a[3]);
        f.activation_forward = pointer<decltype(f.activation_forward)>(a[4]);
        f.activation_backward = pointer<decltype(f.activation_backward)>(a[5]);
        f.rotary_apply = pointer<decltype(f.rotary_apply)>(a[6]);
        lib = f;
        Py_RETURN_NONE;
    });
}

#define METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(name)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {METHOD(bind), METHOD(rms_norm_forward), METHOD(rms_norm_backward), METHOD(pack8), METHOD(unpack8),
                         METHOD(activation_forward), METHOD(activation_backward), METHOD(rotary_apply), {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensors", "The block operators' calls from torch tensors.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensors(void)
{
    n_codes = PyUnicode_InternFromString("codes");
    n_scales = PyUnicode_InternFromString("scales");
    n_group = PyUnicode_InternFromString("group");
    if (!n_codes || !n_scales || !n_group)
        return nullptr;
    return PyModule_Create(&module);
}
