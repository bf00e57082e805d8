// binding.hpp -- what the Python functions of the extension module share: their
// arguments by position or name, the checks of their tensors, and the call of
// the C entry point, or its arguments as a tuple for plan().
#pragma once

#include <Python.h>

#include <c10/hip/HIPStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>
#include <cstring>
#include <exception>
#include <string>
#include <type_traits>

#include "reduce.h"

namespace binding {

// A Python exception is set already.
struct Raised {};

[[noreturn]] inline void raise(PyObject* type, const std::string& what)
{
    PyErr_SetString(type, what.c_str());
    throw Raised();
}

// ---- arguments by position or name -------------------------------------------

struct Params {
    static constexpr int kMost = 24;
    const char* names[kMost];
    int required; // the first ones, up to here, have no default
    int count() const
    {
        int n = 0;
        while (n < kMost && names[n])
            ++n;
        return n;
    }
};

// A call's arguments in the order of its parameters; nullptr: not given.
struct Given {
    PyObject* at[Params::kMost] = {};

    Given(const char* function, const Params& p, PyObject* const* args, Py_ssize_t n,
          PyObject* names)
    {
        const int most = p.count();
        if (n > most)
            raise(PyExc_TypeError, std::string(function) + "() takes at most " +
                                       std::to_string(most) + " arguments");
        for (Py_ssize_t i = 0; i < n; ++i)
            at[i] = args[i];
        const Py_ssize_t named = names ? PyTuple_GET_SIZE(names) : 0;
        for (Py_ssize_t k = 0; k < named; ++k) {
            const char* name = PyUnicode_AsUTF8(PyTuple_GET_ITEM(names, k));
            if (!name)
                throw Raised();
            int i = 0;
            while (i < most && std::strcmp(name, p.names[i]))
                ++i;
            if (i == most)
                raise(PyExc_TypeError, std::string(function) +
                                           "() got an unexpected keyword argument '" + name + "'");
            if (at[i])
                raise(PyExc_TypeError, std::string(function) +
                                           "() got multiple values for argument '" + name + "'");
            at[i] = args[n + k];
        }
        for (int i = 0; i < p.required; ++i)
            if (!at[i])
                raise(PyExc_TypeError, std::string(function) +
                                           "() missing required argument '" + p.names[i] + "'");
    }
};

inline bool is_none(PyObject* o) { return !o || o == Py_None; }

inline float number(PyObject* o, float otherwise)
{
    if (!o)
        return otherwise;
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred())
        throw Raised();
    return (float)v;
}

inline int truth(PyObject* o)
{
    if (!o)
        return 0;
    const int v = PyObject_IsTrue(o);
    if (v < 0)
        throw Raised();
    return v;
}

// None: the current stream; a torch stream; or a handle.
inline red_stream_t stream_of(PyObject* o)
{
    if (is_none(o))
        return c10::hip::getCurrentHIPStream().stream();
    PyObject* handle = PyObject_GetAttrString(o, "cuda_stream");
    if (!handle) {
        PyErr_Clear();
        handle = PyNumber_Long(o);
    }
    if (!handle)
        throw Raised();
    void* p = PyLong_AsVoidPtr(handle);
    Py_DECREF(handle);
    if (!p && PyErr_Occurred())
        throw Raised();
    return p;
}

// ---- tensors -----------------------------------------------------------------

inline const char* type_name(at::ScalarType t)
{
    switch (t) {
    case at::kFloat: return "torch.float32";
    case at::kHalf: return "torch.float16";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kLong: return "torch.int64";
    default: return c10::toString(t);
    }
}

inline const at::Tensor& tensor(PyObject* o, at::ScalarType type, const char* what)
{
    if (!THPVariable_Check(o))
        raise(PyExc_TypeError, std::string(what) + " must be a torch.Tensor");
    const at::Tensor& t = THPVariable_Unpack(o);
    if (t.scalar_type() != type)
        raise(PyExc_TypeError, std::string(what) + " must be " + type_name(type) + ", got " +
                                   type_name(t.scalar_type()));
    if (!t.is_cuda())
        raise(PyExc_ValueError, std::string(what) + " must be a device (cuda/HIP) tensor");
    return t;
}

// A 2-D tensor whose rows are contiguous; the row stride may exceed the
// columns.
struct Matrix {
    void* p = nullptr;
    size_t rows = 0, cols = 0, ld = 0;
    int device = 0;
};

inline Matrix matrix(PyObject* o, at::ScalarType type, const char* what)
{
    const at::Tensor& t = tensor(o, type, what);
    if (t.dim() != 2)
        raise(PyExc_ValueError, std::string(what) + " must be 2-D");
    const int64_t rows = t.size(0), cols = t.size(1);
    int64_t ld = t.stride(0);
    if (t.stride(1) != 1 && cols > 1)
        raise(PyExc_ValueError, std::string("the rows of ") + what + " must be contiguous");
    if (rows <= 1)
        ld = cols;
    else if (ld < cols)
        raise(PyExc_ValueError, std::string("the rows of ") + what + " must not overlap");
    return {t.data_ptr(), (size_t)rows, (size_t)cols, (size_t)ld, t.get_device()};
}

// The checks of one call's tensors, which lie on the logits' device.
struct Tensors {
    Matrix z;
    at::ScalarType type;

    Tensors() = default;
    Tensors(PyObject* logits, at::ScalarType t) : z(matrix(logits, t, "logits")), type(t) {}

    void same_device(const at::Tensor& t) const
    {
        if (t.get_device() != z.device)
            raise(PyExc_ValueError, "all tensors must be on the device of logits");
    }
    // A contiguous tensor of n elements.
    template <class E>
    E* values(PyObject* o, at::ScalarType t, size_t n, const char* what) const
    {
        const at::Tensor& v = tensor(o, t, what);
        if (!v.is_contiguous())
            raise(PyExc_ValueError, std::string(what) + " must be contiguous");
        if ((size_t)v.numel() != n)
            raise(PyExc_ValueError, std::string(what) + " must have " + std::to_string(n) +
                                        " element(s), has " + std::to_string(v.numel()));
        same_device(v);
        return static_cast<E*>(v.data_ptr());
    }
    float* floats(PyObject* o, size_t n, const char* what) const
    {
        return values<float>(o, at::kFloat, n, what);
    }
    float* maybe_floats(PyObject* o, size_t n, const char* what) const
    {
        return is_none(o) ? nullptr : floats(o, n, what);
    }
    int64_t* targets(PyObject* o) const
    {
        return values<int64_t>(o, at::kLong, z.rows, "targets");
    }
    // The gradient's pointer and row stride.
    Matrix gradient(PyObject* o, bool optional) const
    {
        if (optional && is_none(o))
            return {};
        const Matrix d = matrix(o, type, "dlogits");
        if (d.rows != z.rows || d.cols != z.cols)
            raise(PyExc_ValueError, "dlogits must have the shape of logits");
        if (d.device != z.device)
            raise(PyExc_ValueError, "all tensors must be on the device of logits");
        return d;
    }
};

// ---- the call ----------------------------------------------------------------

enum class Mode { Call, Marshal };

inline PyObject* boxed(const void* p) { return p ? PyLong_FromVoidPtr(const_cast<void*>(p)) : Py_NewRef(Py_None); }
inline PyObject* boxed(size_t v) { return PyLong_FromSize_t(v); }
inline PyObject* boxed(int v) { return PyLong_FromLong(v); }
inline PyObject* boxed(float v) { return PyFloat_FromDouble(v); }

[[noreturn]] inline void raise_status(int status, const char* function)
{
    PyObject* m = PyImport_ImportModule("fp32_reductions_amd");
    PyObject* type = m ? PyObject_GetAttrString(m, "ReduceError") : nullptr;
    PyObject* e =
        type ? PyObject_CallFunction(type, "is", status, (std::string("red_") + function).c_str())
             : nullptr;
    if (e)
        PyErr_SetObject(type, e);
    Py_XDECREF(e);
    Py_XDECREF(type);
    Py_XDECREF(m);
    throw Raised();
}

template <class... P, class... A>
PyObject* enter(Mode mode, const char* function, int (*fn)(P...), A... a)
{
    static_assert(sizeof...(P) == sizeof...(A), "an argument for each parameter");
    if (mode == Mode::Marshal) {
        PyObject* t = PyTuple_New(sizeof...(P));
        if (!t)
            throw Raised();
        Py_ssize_t i = 0;
        bool ok = true;
        auto put = [&](PyObject* o) {
            ok = ok && o;
            PyTuple_SET_ITEM(t, i++, o);
        };
        (put(boxed((P)a)), ...);
        if (!ok) {
            Py_DECREF(t);
            throw Raised();
        }
        return t;
    }
    int status;
    Py_BEGIN_ALLOW_THREADS
    status = fn((P)a...);
    Py_END_ALLOW_THREADS
    if (status != RED_OK)
        raise_status(status, function);
    Py_RETURN_NONE;
}

// One Python function: an operator on an element type.
template <class Op, class T, Mode mode>
PyObject* function(PyObject* name, PyObject* const* args, Py_ssize_t n, PyObject* names)
{
    try {
        const char* called = PyUnicode_AsUTF8(name);
        if (!called)
            return nullptr;
        const Given g(called, Op::params, args, n, names);
        return Op::template run<T>(mode, called, g.at);
    } catch (const Raised&) {
    } catch (const std::exception& e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

// The functions, calling and marshalling, with their names and documentation.
struct Function {
    PyMethodDef call, marshal;
    std::string name, doc;
};

template <class Op, class T>
Function make(const char* op, const char* type, const char* doc)
{
    Function f;
    f.name = std::string(op) + "_" + type;
    f.doc = f.name + doc;
    f.call = {nullptr, (PyCFunction)(void*)function<Op, T, Mode::Call>,
              METH_FASTCALL | METH_KEYWORDS, nullptr};
    f.marshal = {nullptr, (PyCFunction)(void*)function<Op, T, Mode::Marshal>,
                 METH_FASTCALL | METH_KEYWORDS, nullptr};
    return f;
}

// An operator's functions on the element types T..., each of which names itself.
template <class Op, class... T>
void add(PyObject* calls, PyObject* marshals, const char* op, const char* doc)
{
    static Function of[] = {make<Op, T>(op, T::name, doc)...};
    for (Function& f : of) {
        f.call.ml_name = f.marshal.ml_name = f.name.c_str();
        f.call.ml_doc = f.marshal.ml_doc = f.doc.c_str();
        PyObject* name = PyUnicode_FromString(f.name.c_str());
        PyObject* module = PyUnicode_FromString("fp32_reductions_amd");
        PyObject* call = name && module ? PyCFunction_NewEx(&f.call, name, module) : nullptr;
        PyObject* marshal = call ? PyCFunction_NewEx(&f.marshal, name, module) : nullptr;
        if (!marshal || PyDict_SetItem(calls, name, call) || PyDict_SetItem(marshals, name, marshal))
            throw Raised();
        Py_DECREF(call);
        Py_DECREF(marshal);
        Py_DECREF(module);
        Py_DECREF(name);
    }
}

// The operators around the output layer (layer_binding.cpp), added to the module.
void add_layer_functions(PyObject* calls, PyObject* marshals);

} // namespace binding
