// rowloss_binding.cpp -- the Python functions of the losses over rows of
// logits: each checks its tensors, takes their pointers, sizes and strides,
// and calls the C entry point of include/reduce.h of the same name.
//
// Such a call has up to twenty arguments, and where the logits are small its
// checks take longer than its kernel: a policy loss took 10.5 us of host time
// a call with them in Python and ctypes, and takes 3.9 us here, of which the
// launch is 3.  With `Mode::Marshal` the same checks give the entry point's
// arguments as a tuple, for plan().
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

namespace {

// A Python exception is set already.
struct Raised {};

[[noreturn]] void raise(PyObject* type, const std::string& what)
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

bool is_none(PyObject* o) { return !o || o == Py_None; }

float number(PyObject* o, float otherwise)
{
    if (!o)
        return otherwise;
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred())
        throw Raised();
    return (float)v;
}

int truth(PyObject* o)
{
    if (!o)
        return 0;
    const int v = PyObject_IsTrue(o);
    if (v < 0)
        throw Raised();
    return v;
}

// None: the current stream; a torch stream; or a handle.
red_stream_t stream_of(PyObject* o)
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

const char* type_name(at::ScalarType t)
{
    switch (t) {
    case at::kFloat: return "torch.float32";
    case at::kHalf: return "torch.float16";
    case at::kBFloat16: return "torch.bfloat16";
    case at::kLong: return "torch.int64";
    default: return c10::toString(t);
    }
}

const at::Tensor& tensor(PyObject* o, at::ScalarType type, const char* what)
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

Matrix matrix(PyObject* o, at::ScalarType type, const char* what)
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

PyObject* boxed(const void* p) { return p ? PyLong_FromVoidPtr(const_cast<void*>(p)) : Py_NewRef(Py_None); }
PyObject* boxed(size_t v) { return PyLong_FromSize_t(v); }
PyObject* boxed(int v) { return PyLong_FromLong(v); }
PyObject* boxed(float v) { return PyFloat_FromDouble(v); }

[[noreturn]] void raise_status(int status, const char* function)
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

// The entry points of one element type.
struct F32 {
    static constexpr at::ScalarType type = at::kFloat;
    static constexpr auto logprob = red_token_logprob_f32;
    static constexpr auto logprob_grad = red_token_logprob_grad_f32;
    static constexpr auto distill = red_distill_topk_f32;
    static constexpr auto policy = red_policy_loss_f32;
    static constexpr auto preference = red_preference_loss_f32;
    typedef float S;
};
struct F16 {
    static constexpr at::ScalarType type = at::kHalf;
    static constexpr auto logprob = red_token_logprob_f16;
    static constexpr auto logprob_grad = red_token_logprob_grad_f16;
    static constexpr auto distill = red_distill_topk_f16;
    static constexpr auto policy = red_policy_loss_f16;
    static constexpr auto preference = red_preference_loss_f16;
    typedef uint16_t S;
};
struct BF16 {
    static constexpr at::ScalarType type = at::kBFloat16;
    static constexpr auto logprob = red_token_logprob_bf16;
    static constexpr auto logprob_grad = red_token_logprob_grad_bf16;
    static constexpr auto distill = red_distill_topk_bf16;
    static constexpr auto policy = red_policy_loss_bf16;
    static constexpr auto preference = red_preference_loss_bf16;
    typedef uint16_t S;
};

struct Logprob {
    static constexpr Params params = {
        {"logits", "targets", "logp", "lse", "entropy", "scale", "stream"}, 4};
    template <class T>
    static PyObject* run(Mode mode, const char* name, PyObject* const* a)
    {
        const Tensors t(a[0], T::type);
        const size_t n = t.z.rows;
        return enter(mode, name, T::logprob, (const typename T::S*)t.z.p, n, t.z.cols, t.z.ld,
                     t.targets(a[1]), number(a[5], 1.0f), t.floats(a[2], n, "logp"),
                     t.floats(a[3], n, "lse"), t.maybe_floats(a[4], n, "entropy"),
                     stream_of(a[6]));
    }
};

struct LogprobGrad {
    static constexpr Params params = {{"logits", "targets", "lse", "glogp", "dlogits", "entropy",
                                       "gentropy", "scale", "stream"},
                                      5};
    template <class T>
    static PyObject* run(Mode mode, const char* name, PyObject* const* a)
    {
        const Tensors t(a[0], T::type);
        const size_t n = t.z.rows;
        const Matrix d = t.gradient(a[4], false);
        if (!is_none(a[6]) && is_none(a[5]))
            raise(PyExc_ValueError, "gentropy needs entropy");
        return enter(mode, name, T::logprob_grad, (const typename T::S*)t.z.p, n, t.z.cols,
                     t.z.ld, t.targets(a[1]), number(a[7], 1.0f), t.floats(a[2], n, "lse"),
                     t.maybe_floats(a[5], n, "entropy"), t.floats(a[3], n, "glogp"),
                     t.maybe_floats(a[6], n, "gentropy"), (typename T::S*)d.p, d.ld,
                     stream_of(a[8]));
    }
};

struct Distill {
    static constexpr Params params = {{"logits", "idx", "val", "loss", "dlogits", "teacher_lse",
                                       "weight", "row_loss", "scale", "accum", "stream"},
                                      4};
    template <class T>
    static PyObject* run(Mode mode, const char* name, PyObject* const* a)
    {
        const Tensors t(a[0], T::type);
        const size_t n = t.z.rows;
        const Matrix i = matrix(a[1], at::kLong, "idx"), v = matrix(a[2], at::kFloat, "val");
        if (i.rows != n || v.rows != n || v.cols != i.cols)
            raise(PyExc_ValueError, "idx and val must both be (rows, K)");
        if (i.ld != v.ld)
            raise(PyExc_ValueError, "idx and val must have the same row stride");
        if (i.device != t.z.device || v.device != t.z.device)
            raise(PyExc_ValueError, "all tensors must be on the device of logits");
        const Matrix d = t.gradient(a[4], true);
        return enter(mode, name, T::distill, (const typename T::S*)t.z.p, n, t.z.cols, t.z.ld,
                     (const int64_t*)i.p, (const float*)v.p, i.cols, i.ld,
                     t.maybe_floats(a[5], n, "teacher_lse"), t.maybe_floats(a[6], n, "weight"),
                     number(a[8], 1.0f), t.floats(a[3], 1, "loss"), truth(a[9]),
                     t.maybe_floats(a[7], n, "row_loss"), (typename T::S*)d.p, d.ld,
                     stream_of(a[10]));
    }
};

struct Policy {
    static constexpr Params params = {
        {"logits", "targets", "old_logp", "advantage", "loss", "logp", "dlogits", "ref_logp",
         "weight", "entropy", "scale", "clip_low", "clip_high", "kl_coef", "entropy_coef", "accum",
         "stream"},
        6};
    template <class T>
    static PyObject* run(Mode mode, const char* name, PyObject* const* a)
    {
        const Tensors t(a[0], T::type);
        const size_t n = t.z.rows;
        const Matrix d = t.gradient(a[6], true);
        const float kl = number(a[13], 0.0f);
        if (kl != 0.0f && is_none(a[7]))
            raise(PyExc_ValueError, "kl_coef needs ref_logp");
        return enter(mode, name, T::policy, (const typename T::S*)t.z.p, n, t.z.cols, t.z.ld,
                     t.targets(a[1]), t.floats(a[2], n, "old_logp"),
                     t.maybe_floats(a[7], n, "ref_logp"), t.floats(a[3], n, "advantage"),
                     t.maybe_floats(a[8], n, "weight"), number(a[10], 1.0f), number(a[11], 0.2f),
                     number(a[12], 0.2f), kl, number(a[14], 0.0f), t.floats(a[4], 1, "loss"),
                     truth(a[15]), t.floats(a[5], n, "logp"), t.maybe_floats(a[9], n, "entropy"),
                     (typename T::S*)d.p, d.ld, stream_of(a[16]));
    }
};

struct Preference {
    static constexpr Params params = {
        {"logits", "targets", "starts", "loss", "seq_logp", "dlogits", "ref_logp", "weight",
         "kind", "beta", "margin", "smoothing", "average", "accum", "stream"},
        5};
    static int kind_of(PyObject* o)
    {
        if (!o)
            return RED_PREF_SIGMOID;
        const char* k = PyUnicode_Check(o) ? PyUnicode_AsUTF8(o) : nullptr;
        if (k && !std::strcmp(k, "sigmoid"))
            return RED_PREF_SIGMOID;
        if (k && !std::strcmp(k, "hinge"))
            return RED_PREF_HINGE;
        if (k && !std::strcmp(k, "squared"))
            return RED_PREF_SQUARED;
        raise(PyExc_ValueError, "kind must be one of hinge, sigmoid, squared");
    }
    template <class T>
    static PyObject* run(Mode mode, const char* name, PyObject* const* a)
    {
        const Tensors t(a[0], T::type);
        const at::Tensor& s = tensor(a[2], at::kLong, "starts");
        if (!s.is_contiguous())
            raise(PyExc_ValueError, "starts must be contiguous");
        if (s.numel() % 2 == 0)
            raise(PyExc_ValueError, "starts must have 2 * pairs + 1 elements");
        t.same_device(s);
        const size_t pairs = (size_t)s.numel() / 2;
        const int kind = kind_of(a[8]);
        const Matrix d = t.gradient(a[5], true);
        return enter(mode, name, T::preference, (const typename T::S*)t.z.p, t.z.rows, t.z.cols,
                     t.z.ld, t.targets(a[1]), (const int64_t*)s.data_ptr(), pairs,
                     t.maybe_floats(a[6], 2 * pairs, "ref_logp"),
                     t.maybe_floats(a[7], pairs, "weight"), kind, number(a[9], 0.1f),
                     number(a[10], 0.0f), number(a[11], 0.0f), truth(a[12]),
                     t.floats(a[3], 1, "loss"), truth(a[13]),
                     t.floats(a[4], 2 * pairs, "seq_logp"), (typename T::S*)d.p, d.ld,
                     stream_of(a[14]));
    }
};

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

const char kLogprobDoc[] =
    "($self, logits, targets, logp, lse, entropy=None, scale=1.0, stream=None)\n--\n\n"
    "logp[r] = ln p_target, lse[r] = ln sum exp(scale * logits[r]) and, where\n"
    "given, entropy[r] of each row's softmax p at inverse temperature `scale`.\n\n"
    "logits (rows, V) with contiguous rows of any stride; targets int64 (a\n"
    "target outside [0, V) gives logp 0); logp, lse, entropy fp32.";
const char kLogprobGradDoc[] =
    "($self, logits, targets, lse, glogp, dlogits, entropy=None, gentropy=None, scale=1.0, "
    "stream=None)\n--\n\n"
    "dlogits from the gradients glogp (of logp) and gentropy (of entropy) of\n"
    "token_logprob, whose lse and entropy the caller kept.  dlogits may be\n"
    "logits itself.";
const char kDistillDoc[] =
    "($self, logits, idx, val, loss, dlogits=None, teacher_lse=None, weight=None, "
    "row_loss=None, scale=1.0, accum=False, stream=None)\n--\n\n"
    "loss[0] = [loss[0] +] sum_r weight[r] KL(teacher || softmax(scale *\n"
    "logits[r])) for a teacher given by K columns idx (rows, K) int64 and\n"
    "their logits val (rows, K) fp32; columns outside [0, V) are padding.\n"
    "Without teacher_lse the teacher is the softmax of its entries; with the\n"
    "log-sum-exp of its whole scaled row, the columns not listed count as one\n"
    "more.  weight: 1 / rows each when None; 0 leaves a row out.  dlogits\n"
    "takes the gradient (it may be logits itself), row_loss the rows' losses.";
const char kPolicyDoc[] =
    "($self, logits, targets, old_logp, advantage, loss, logp, dlogits=None, ref_logp=None, "
    "weight=None, entropy=None, scale=1.0, clip_low=0.2, clip_high=0.2, kl_coef=0.0, "
    "entropy_coef=0.0, accum=False, stream=None)\n--\n\n"
    "loss[0] = [loss[0] +] sum_r weight[r] (-min(ratio A, clip(ratio) A) +\n"
    "kl_coef (exp(d) - d - 1) - entropy_coef H) with ratio = exp(logp[r] -\n"
    "old_logp[r]) clipped to [1 - clip_low, 1 + clip_high], A = advantage[r],\n"
    "d = ref_logp[r] - logp[r] and H the entropy of softmax(scale *\n"
    "logits[r]).  logp and entropy take the rows' values, dlogits the gradient\n"
    "(it may be logits itself).  weight: 1 / rows each when None; rows of\n"
    "weight 0, or without a target in [0, V), do not count.";
const char kPreferenceDoc[] =
    "($self, logits, targets, starts, loss, seq_logp, dlogits=None, ref_logp=None, weight=None, "
    "kind=\"sigmoid\", beta=0.1, margin=0.0, smoothing=0.0, average=False, accum=False, "
    "stream=None)\n--\n\n"
    "loss[0] = [loss[0] +] sum_p weight[p] l(beta D_p - margin), D_p the\n"
    "log-ratio of pair p's chosen sequence (number p) over its rejected one\n"
    "(number pairs + p), each against ref_logp; l is \"sigmoid\" (with label\n"
    "smoothing), \"hinge\" or \"squared\".  Sequence i has the rows starts[i] to\n"
    "starts[i + 1] (int64, 2 * pairs + 1 of them); seq_logp (2 * pairs) takes\n"
    "the sums (average: means) of their targets' log-probabilities, dlogits the\n"
    "gradient (it may be logits itself).  weight: 1 / pairs each when None.";

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

template <class Op>
void add(PyObject* calls, PyObject* marshals, const char* op, const char* doc)
{
    static Function of[3] = {make<Op, F32>(op, "f32", doc), make<Op, F16>(op, "f16", doc),
                             make<Op, BF16>(op, "bf16", doc)};
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

PyModuleDef definition = {PyModuleDef_HEAD_INIT, "_rowloss",
                          "The losses over rows of logits: calls and marshalling by name.", -1,
                          nullptr};

} // namespace

PyMODINIT_FUNC PyInit__rowloss()
{
    PyObject* m = PyModule_Create(&definition);
    PyObject* calls = PyDict_New();
    PyObject* marshals = PyDict_New();
    if (!m || !calls || !marshals)
        return nullptr;
    try {
        add<Logprob>(calls, marshals, "token_logprob", kLogprobDoc);
        add<LogprobGrad>(calls, marshals, "token_logprob_grad", kLogprobGradDoc);
        add<Distill>(calls, marshals, "distill_topk", kDistillDoc);
        add<Policy>(calls, marshals, "policy_loss", kPolicyDoc);
        add<Preference>(calls, marshals, "preference_loss", kPreferenceDoc);
    } catch (const Raised&) {
        return nullptr;
    }
    if (PyModule_AddObject(m, "CALLS", calls) || PyModule_AddObject(m, "MARSHALS", marshals))
        return nullptr;
    return m;
}
