// rowloss_binding.cpp -- the Python functions of the losses over rows of
// logits: each checks its tensors, takes their pointers, sizes and strides,
// and calls the C entry point of include/reduce.h of the same name.
//
// Such a call has up to twenty arguments, and where the logits are small its
// checks take longer than its kernel: a policy loss took 10.5 us of host time
// a call with them in Python and ctypes, and takes 3.9 us here, of which the
// launch is 3.  With `Mode::Marshal` the same checks give the entry point's
// arguments as a tuple, for plan().
#include "binding.hpp"

namespace {

using namespace binding;

// The entry points of one element type.
struct F32 {
    static constexpr const char* name = "f32";
    static constexpr at::ScalarType type = at::kFloat;
    static constexpr auto logprob = red_token_logprob_f32;
    static constexpr auto logprob_grad = red_token_logprob_grad_f32;
    static constexpr auto distill = red_distill_topk_f32;
    static constexpr auto policy = red_policy_loss_f32;
    static constexpr auto preference = red_preference_loss_f32;
    typedef float S;
};
struct F16 {
    static constexpr const char* name = "f16";
    static constexpr at::ScalarType type = at::kHalf;
    static constexpr auto logprob = red_token_logprob_f16;
    static constexpr auto logprob_grad = red_token_logprob_grad_f16;
    static constexpr auto distill = red_distill_topk_f16;
    static constexpr auto policy = red_policy_loss_f16;
    static constexpr auto preference = red_preference_loss_f16;
    typedef uint16_t S;
};
struct BF16 {
    static constexpr const char* name = "bf16";
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

PyModuleDef definition = {PyModuleDef_HEAD_INIT, "_rowloss",
                          "The losses over rows of logits and the operators around the output layer:\n"
                          "calls and marshalling by name.", -1,
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
        add<Logprob, F32, F16, BF16>(calls, marshals, "token_logprob", kLogprobDoc);
        add<LogprobGrad, F32, F16, BF16>(calls, marshals, "token_logprob_grad", kLogprobGradDoc);
        add<Distill, F32, F16, BF16>(calls, marshals, "distill_topk", kDistillDoc);
        add<Policy, F32, F16, BF16>(calls, marshals, "policy_loss", kPolicyDoc);
        add<Preference, F32, F16, BF16>(calls, marshals, "preference_loss", kPreferenceDoc);
        add_layer_functions(calls, marshals);
    } catch (const Raised&) {
        return nullptr;
    }
    if (PyModule_AddObject(m, "CALLS", calls) || PyModule_AddObject(m, "MARSHALS", marshals))
        return nullptr;
    return m;
}
