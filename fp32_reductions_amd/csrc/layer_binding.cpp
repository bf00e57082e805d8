// layer_binding.cpp -- the Python functions of the operators around the output
// layer: the norm, the router's balance loss, the layer's cross entropy.  Part
// of the extension module of rowloss_binding.cpp.
#include "binding.hpp"

#include <ATen/ATen.h>
#include <c10/hip/HIPFunctions.h>

namespace binding {
namespace {

struct F32 {
    static constexpr const char* name = "f32";
    static constexpr at::ScalarType type = at::kFloat;
    static constexpr auto norm = red_add_rmsnorm_f32;
    static constexpr auto norm_grad = red_rmsnorm_grad_f32;
    static constexpr auto router = red_router_balance_f32;
    typedef float S;
};
struct F16 {
    static constexpr const char* name = "f16";
    static constexpr at::ScalarType type = at::kHalf;
    static constexpr auto norm = red_add_rmsnorm_f16;
    static constexpr auto norm_grad = red_rmsnorm_grad_f16;
    static constexpr auto router = red_router_balance_f16;
    static constexpr auto linear = red_linear_ce_f16;
    static constexpr auto linear_bytes = red_linear_ce_workspace_f16;
    typedef uint16_t S;
};
struct BF16 {
    static constexpr const char* name = "bf16";
    static constexpr at::ScalarType type = at::kBFloat16;
    static constexpr auto norm = red_add_rmsnorm_bf16;
    static constexpr auto norm_grad = red_rmsnorm_grad_bf16;
    static constexpr auto router = red_router_balance_bf16;
    static constexpr auto linear = red_linear_ce_bf16;
    static constexpr auto linear_bytes = red_linear_ce_workspace_bf16;
    typedef uint16_t S;
};

// Tensors of a call, all on the current device: its first matrix is `z`.
struct Call : Tensors {
    const char* first;
    Call(PyObject* matrix, at::ScalarType t, const char* what) : Tensors(matrix_of(matrix, t, what)), first(what)
    {
        if (z.device != c10::hip::current_device())
            raise(PyExc_ValueError, std::string(what) + " must be on the current device");
    }
    // Another matrix of the same shape; null where it is optional and not given.
    Matrix like(PyObject* o, at::ScalarType t, bool optional, const char* what) const
    {
        if (optional && is_none(o))
            return {};
        const Matrix m = matrix(o, t, what);
        if (m.rows != z.rows || m.cols != z.cols)
            raise(PyExc_ValueError, std::string(what) + " must have the shape of " + first);
        here(m.device);
        return m;
    }
    Matrix like(PyObject* o, bool optional, const char* what) const { return like(o, type, optional, what); }
    template <class E>
    E* vector(PyObject* o, at::ScalarType t, size_t n, const char* what) const
    {
        const at::Tensor& v = tensor(o, t, what);
        if (!v.is_contiguous())
            raise(PyExc_ValueError, std::string(what) + " must be contiguous");
        if ((size_t)v.numel() != n)
            raise(PyExc_ValueError, std::string(what) + " must have " + std::to_string(n) +
                                        " element(s), has " + std::to_string(v.numel()));
        here(v.get_device());
        return static_cast<E*>(v.data_ptr());
    }
    float* numbers(PyObject* o, size_t n, const char* what) const
    {
        return vector<float>(o, at::kFloat, n, what);
    }
    float* maybe_numbers(PyObject* o, size_t n, const char* what) const
    {
        return is_none(o) ? nullptr : numbers(o, n, what);
    }
    void here(int device) const
    {
        if (device != z.device)
            raise(PyExc_ValueError, std::string("all tensors must be on the device of ") + first);
    }

  private:
    static Tensors matrix_of(PyObject* o, at::ScalarType t, const char* what)
    {
        Tensors v;
        v.z = matrix(o, t, what);
        v.type = t;
        return v;
    }
};

struct AddRmsnorm {
    static constexpr Params params = {
        {"x", "weight", "y", "residual", "sum", "y8", "yscale", "rstd", "eps", "stream"}, 3};
    template <class T>
    static PyObject* run(Mode mode, const char* name, PyObject* const* a)
    {
        typedef typename T::S S;
        const Call t(a[0], T::type, "x");
        const size_t n = t.z.rows;
        // y of the rows' type or of 8 bits, or both: y and y8.
        PyObject *y = a[2], *y8 = a[5];
        if (!is_none(y) && THPVariable_Check(y) &&
            THPVariable_Unpack(y).scalar_type() == at::kFloat8_e4m3fn) {
            if (!is_none(y8))
                raise(PyExc_ValueError, "y and y8 are both of 8 bits");
            y8 = y;
            y = Py_None;
        }
        const Matrix my = t.like(y, true, "y"), m8 = t.like(y8, at::kFloat8_e4m3fn, true, "y8"),
                     r = t.like(a[3], true, "residual"), s = t.like(a[4], true, "sum");
        if (is_none(y) && is_none(y8))
            raise(PyExc_ValueError, "y or y8 must be given");
        if (is_none(y8) != is_none(a[6]))
            raise(PyExc_ValueError, "an output of 8 bits needs yscale, and yscale one");
        return enter(mode, name, T::norm, (const S*)t.z.p, n, t.z.cols, t.z.ld, (const S*)r.p, r.ld,
                     t.template vector<const S>(a[1], T::type, t.z.cols, "weight"),
                     number(a[8], 1e-6f), (S*)s.p, s.ld, (S*)my.p, my.ld, (uint8_t*)m8.p, m8.ld,
                     t.maybe_numbers(a[6], n, "yscale"), t.maybe_numbers(a[7], n, "rstd"),
                     stream_of(a[9]));
    }
};

struct RmsnormGrad {
    static constexpr Params params = {
        {"h", "weight", "rstd", "dy", "dx", "dsum", "dweight", "accum", "stream"}, 5};
    template <class T>
    static PyObject* run(Mode mode, const char* name, PyObject* const* a)
    {
        typedef typename T::S S;
        const Call t(a[0], T::type, "h");
        const Matrix dy = t.like(a[3], false, "dy"), dx = t.like(a[4], false, "dx"),
                     ds = t.like(a[5], true, "dsum");
        return enter(mode, name, T::norm_grad, (const S*)t.z.p, t.z.rows, t.z.cols, t.z.ld,
                     t.template vector<const S>(a[1], T::type, t.z.cols, "weight"),
                     t.numbers(a[2], t.z.rows, "rstd"), (const S*)dy.p, dy.ld, (const S*)ds.p, ds.ld,
                     (S*)dx.p, dx.ld, t.maybe_numbers(a[6], t.z.cols, "dweight"), truth(a[7]),
                     stream_of(a[8]));
    }
};

struct RouterBalance {
    static constexpr Params params = {{"logits", "experts", "loss", "counts", "dlogits", "weight",
                                       "prob", "balance_coef", "z_coef", "accum", "stream"},
                                      4};
    template <class T>
    static PyObject* run(Mode mode, const char* name, PyObject* const* a)
    {
        typedef typename T::S S;
        const Call t(a[0], T::type, "logits");
        const size_t n = t.z.rows, E = t.z.cols;
        const Matrix k = matrix(a[1], at::kLong, "experts");
        if (k.rows != n)
            raise(PyExc_ValueError, "experts must be (rows, K)");
        t.here(k.device);
        const Matrix d = t.like(a[4], true, "dlogits");
        return enter(mode, name, T::router, (const S*)t.z.p, n, E, t.z.ld, (const int64_t*)k.p,
                     k.cols, k.ld, t.maybe_numbers(a[5], n, "weight"), number(a[7], 0.01f),
                     number(a[8], 0.0f), t.numbers(a[2], 1, "loss"), truth(a[9]),
                     t.template vector<int64_t>(a[3], at::kLong, E, "counts"),
                     t.maybe_numbers(a[6], E, "prob"), (S*)d.p, d.ld, stream_of(a[10]));
    }
};

struct LinearCe {
    static constexpr Params params = {{"hidden", "weight", "targets", "loss", "logp", "lse",
                                       "dhidden", "dweight", "row_weight", "scale", "z_coef",
                                       "accum", "workspace", "stream"},
                                      4};
    template <class T>
    static PyObject* run(Mode mode, const char* name, PyObject* const* a)
    {
        const Call t(a[0], T::type, "hidden");
        const size_t n = t.z.rows, D = t.z.cols;
        const Matrix w = matrix(a[1], T::type, "weight");
        if (w.cols != D)
            raise(PyExc_ValueError, "weight must be (V, D) for hidden rows of D");
        t.here(w.device);
        const Matrix dh = t.like(a[6], true, "dhidden");
        Matrix dw;
        if (!is_none(a[7])) {
            dw = matrix(a[7], T::type, "dweight");
            if (dw.rows != w.rows || dw.cols != D)
                raise(PyExc_ValueError, "dweight must have the shape of weight");
            t.here(dw.device);
        }
        const int64_t* y = t.template vector<const int64_t>(a[2], at::kLong, n, "targets");
        float* loss = t.numbers(a[3], 1, "loss");
        const red_stream_t stream = stream_of(a[13]);
        // Given, or of torch's allocator for this call.
        at::Tensor own;
        void* p = nullptr;
        size_t bytes = 0;
        if (!is_none(a[12])) {
            const at::Tensor& s = tensor(a[12], at::kByte, "workspace");
            if (!s.is_contiguous())
                raise(PyExc_ValueError, "workspace must be contiguous");
            t.here(s.get_device());
            p = s.data_ptr();
            bytes = (size_t)s.numel();
        } else if (mode == Mode::Marshal) {
            raise(PyExc_ValueError, "a plan needs a workspace of its own");
        } else if (n && D && w.rows) {
            const int status = T::linear_bytes(n, D, w.rows, dh.p != nullptr, dw.p != nullptr, &bytes);
            if (status != RED_OK)
                raise_status(status, name);
            own = at::empty({(int64_t)bytes}, THPVariable_Unpack(a[0]).options().dtype(at::kByte));
            const auto current = c10::hip::getCurrentHIPStream();
            if (stream != (red_stream_t)current.stream())
                raise(PyExc_ValueError,
                      "on another stream than the current one the call needs a workspace");
            p = own.data_ptr();
        }
        return enter(mode, name, T::linear, (const uint16_t*)t.z.p, n, D, t.z.ld,
                     (const uint16_t*)w.p, w.rows, w.ld, y, t.maybe_numbers(a[8], n, "row_weight"),
                     number(a[9], 1.0f), number(a[10], 0.0f), loss, truth(a[11]),
                     t.maybe_numbers(a[4], n, "logp"), t.maybe_numbers(a[5], n, "lse"),
                     (uint16_t*)dh.p, dh.ld, (uint16_t*)dw.p, dw.ld, p, bytes, stream);
    }
};

const char kNormDoc[] =
    "($self, x, weight, y, residual=None, sum=None, y8=None, yscale=None, rstd=None, eps=1e-6, "
    "stream=None)\n--\n\n"
    "Root-mean-square norm of rows: h = x + residual, rstd = (mean h^2 +\n"
    "eps)^-1/2, y = h * rstd * weight; sum takes h, rstd (rows, fp32) what\n"
    "rmsnorm_grad needs.  y is of x's type, or torch.float8_e4m3fn with\n"
    "yscale (rows, fp32): y * yscale is the row.  y8 is the 8-bit output\n"
    "beside a y of x's type (y may be None then).  sum and y may each be x or\n"
    "residual themselves.  A row with an infinity has rstd 0, NaN there and zeros\n"
    "elsewhere.";
const char kNormGradDoc[] =
    "($self, h, weight, rstd, dy, dx, dsum=None, dweight=None, accum=False, stream=None)\n--\n\n"
    "The gradient of add_rmsnorm from its h (sum) and rstd: dx of x and of the\n"
    "residual, with dsum, the gradient of sum, added; dweight (fp32) [+]= the\n"
    "weight's.  dx may be h, dy or dsum itself.";
const char kRouterDoc[] =
    "($self, logits, experts, loss, counts, dlogits=None, weight=None, prob=None, "
    "balance_coef=0.01, z_coef=0.0, accum=False, stream=None)\n--\n\n"
    "loss[0] = [loss[0] +] balance_coef * E * sum_e f_e P_e + z_coef * sum_r\n"
    "weight[r] lse_r^2 of a router's logits (rows, E): counts (E, int64) takes\n"
    "how often the rows that count chose each expert in experts (rows, K)\n"
    "int64, f its share, prob (E, fp32) P = sum_r weight[r] softmax(logits[r]).\n"
    "dlogits takes the gradient, for which counts is constant (it may be logits\n"
    "itself).  weight: 1 / rows each when None; 0 leaves a row out.";
const char kLinearDoc[] =
    "($self, hidden, weight, targets, loss, logp=None, lse=None, dhidden=None, dweight=None, "
    "row_weight=None, scale=1.0, z_coef=0.0, accum=False, workspace=None, stream=None)\n--\n\n"
    "loss[0] = [loss[0] +] sum_r row_weight[r] (-logp[r] + z_coef lse[r]^2),\n"
    "the cross entropy of softmax(scale * hidden @ weight.T) without a matrix\n"
    "of logits: hidden (rows, D), weight (V, D), targets (rows) int64.  logp and\n"
    "lse (fp32) take the rows' values, dhidden and dweight the gradients.\n"
    "row_weight: 1 / rows each when None; rows of weight 0, or without a target\n"
    "in [0, V), do not count.  D a multiple of 8, weight's rows 16-byte aligned.\n"
    "workspace: a uint8 tensor of linear_ce_workspace() bytes; torch allocates\n"
    "one for the call when None.";

} // namespace

void add_layer_functions(PyObject* calls, PyObject* marshals)
{
    add<AddRmsnorm, F32, F16, BF16>(calls, marshals, "add_rmsnorm", kNormDoc);
    add<RmsnormGrad, F32, F16, BF16>(calls, marshals, "rmsnorm_grad", kNormGradDoc);
    add<RouterBalance, F32, F16, BF16>(calls, marshals, "router_balance", kRouterDoc);
    add<LinearCe, F16, BF16>(calls, marshals, "linear_ce", kLinearDoc);
}

} // namespace binding
