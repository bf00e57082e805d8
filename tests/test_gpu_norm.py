"""The root-mean-square norm and its gradient on the GPU against the fp64
reference (layer_reference.py), whose bounds follow from the formats.

Widths sit on both sides of every boundary of the kernels: shorter than a
vector, around each number of threads and vectors a row is given, for few rows
and for many; bases aligned to their element only; padded strides; everything
around a row holds NaN or a mark."""
import math

import pytest

import layer_reference as ref
from gpu_helpers import say
from test_gpu_rowloss import DTYPES, place, untouched

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

WIDTHS = [1, 3, 4, 7, 8, 9, 31, 33, 63, 64, 65, 127, 128, 129, 256, 257, 511, 513, 1000, 1024,
          1025, 2047, 2049, 4096, 4099, 8192, 8200, 16384]
CASES = [(rows, D, t) for D in WIDTHS for rows in (1, 5) for t in DTYPES]
# more rows than compute units: other shapes, and several rows a workgroup
CASES += [(rows, D, t) for D, rows in [(9, 4099), (65, 1201), (128, 3000), (260, 2100),
                                       (600, 700), (1025, 777), (2048, 520), (4100, 300),
                                       (8192, 513), (9000, 300), (16384, 260)] for t in DTYPES]


@pytest.fixture(scope="module")
def red():
    import fp32_reductions_amd
    return fp32_reductions_amd


def matrix(g, rows, D, t, std=2.0):
    return (torch.randn(rows, D, generator=g) * std).to(DTYPES[t])


def mark(x, shift, pad):
    return place(torch.full_like(x, 7.0), shift, pad, 5.0)


@pytest.mark.parametrize("rows,D,t", CASES)
def test_norm(red, rows, D, t):
    say("norm %d x %d %s" % (rows, D, t))
    g = torch.Generator().manual_seed(rows * 31 + D)
    x, r, w = matrix(g, rows, D, t), matrix(g, rows, D, t), matrix(g, 1, D, t, 1.0)[0]
    shift, pad = (1, 3) if D % 2 else (0, 8)
    for residual in (None, r):
        want = ref.add_rmsnorm(x, residual, w, 1e-5)
        xd, _ = place(x, shift, pad)
        rd = None if residual is None else place(r, 2 * shift, pad + 1)[0]
        s, sflat = mark(x, shift, pad)
        y, yflat = mark(x, 0, pad)
        rstd = torch.empty(rows, device="cuda")
        y8 = torch.empty(rows, D + pad, dtype=ref.E4M3, device="cuda")
        y8.view(torch.uint8).fill_(0x55)
        scale = torch.empty(rows, device="cuda")
        getattr(red, "add_rmsnorm_" + t)(xd, w.cuda(), y, residual=rd, sum=s, y8=y8[:, :D],
                                         yscale=scale, rstd=rstd, eps=1e-5)
        for k, v in (("sum", s), ("rstd", rstd), ("y", y)):
            ref.same(k, v, *want[k])
        ref.check_8bit(y8[:, :D], scale, want["exact"])
        assert untouched(sflat, shift, rows, D, pad, 5.0) and untouched(yflat, 0, rows, D, pad, 5.0)
        assert (y8[:, D:].contiguous().view(torch.uint8) == 0x55).all()
        # each output alone is the same, bit for bit
        y2, only8 = torch.empty(rows, D, dtype=x.dtype, device="cuda"), torch.empty_like(y8)
        getattr(red, "add_rmsnorm_" + t)(xd, w.cuda(), y2, residual=rd, eps=1e-5)
        assert torch.equal(y2, y)
        getattr(red, "add_rmsnorm_" + t)(xd, w.cuda(), only8[:, :D], residual=rd, yscale=scale,
                                         eps=1e-5)
        assert torch.equal(only8[:, :D].contiguous().view(torch.uint8),
                           y8[:, :D].contiguous().view(torch.uint8))


@pytest.mark.parametrize("rows,D,t", CASES)
def test_gradient(red, rows, D, t):
    say("norm gradient %d x %d %s" % (rows, D, t))
    g = torch.Generator().manual_seed(rows * 37 + D)
    h, dy, ds = matrix(g, rows, D, t), matrix(g, rows, D, t, 0.1), matrix(g, rows, D, t, 0.1)
    w = matrix(g, 1, D, t, 1.0)[0]
    rstd = (h.double().square().mean(1) + 1e-5).rsqrt().float()
    old = torch.randn(D, generator=g)
    shift, pad = (1, 3) if D % 2 else (0, 8)
    hd, dyd, dsd = (place(v, i * shift, pad + i)[0] for i, v in enumerate((h, dy, ds)))
    for dsum, weight, accum in ((None, False, False), (ds, True, False), (ds, True, True)):
        want = ref.rmsnorm_grad(h, w, rstd, dy, dsum)
        dx, flat = mark(h, shift, pad)
        dw = old.cuda() if weight else None
        getattr(red, "rmsnorm_grad_" + t)(hd, w.cuda(), rstd.cuda(), dyd, dx,
                                          dsum=None if dsum is None else dsd, dweight=dw,
                                          accum=accum)
        ref.same("dx", dx, *want["dx"])
        assert untouched(flat, shift, rows, D, pad, 5.0)
        if weight:
            v, b = want["dweight"]
            if accum:
                v = v + old.double()
                b = b + v.abs() * 2 ** -23 + old.abs() * 2 ** -23
            ref.same("dweight", dw, v, b)


@pytest.mark.parametrize("t", DTYPES)
def test_outputs_over_inputs(red, t):
    g = torch.Generator().manual_seed(5)
    f, fg = getattr(red, "add_rmsnorm_" + t), getattr(red, "rmsnorm_grad_" + t)
    for rows, D in ((3, 1000), (700, 264)):
        say("in place %d x %d %s" % (rows, D, t))
        x, r, w = (v.cuda() for v in (matrix(g, rows, D, t), matrix(g, rows, D, t),
                                      matrix(g, 1, D, t)[0]))
        s, y, rstd = torch.empty_like(x), torch.empty_like(x), torch.empty(rows, device="cuda")
        f(x, w, y, residual=r, sum=s, rstd=rstd)
        a, b = x.clone(), r.clone()
        f(a, w, a, residual=b, sum=b)
        assert torch.equal(a, y) and torch.equal(b, s)
        a, b = x.clone(), r.clone()
        f(a, w, b, residual=b, sum=a)
        assert torch.equal(b, y) and torch.equal(a, s)
        dx = torch.empty_like(x)
        fg(s, w, rstd, x, dx, dsum=r)
        for i in range(3):
            args = [s.clone(), x.clone(), r.clone()]
            fg(args[0], w, rstd, args[1], args[i], dsum=args[2])
            assert torch.equal(args[i], dx)


@pytest.mark.parametrize("t", DTYPES)
def test_special_rows(red, t):
    """Zeros, infinities and NaN, the largest and smallest values: each row for
    itself."""
    info = torch.finfo(DTYPES[t])
    D = 1000
    g = torch.Generator().manual_seed(6)
    x = matrix(g, 8, D, t)
    x[1] = 0.0
    x[2, 7] = math.inf
    x[3, 999] = math.nan
    x[4] = info.max
    x[5] = info.tiny
    x[6, 1:] = 0.0
    w = matrix(g, 1, D, t, 1.0)[0]
    for eps in (1e-6, 0.0):
        say("special rows %s eps %g" % (t, eps))
        want = ref.add_rmsnorm(x, None, w, eps)
        y, y8 = torch.empty_like(x, device="cuda"), torch.empty(8, D, dtype=ref.E4M3, device="cuda")
        scale, rstd = torch.empty(8, device="cuda"), torch.empty(8, device="cuda")
        getattr(red, "add_rmsnorm_" + t)(x.cuda(), w.cuda(), y, y8=y8, yscale=scale, rstd=rstd,
                                         eps=eps)
        fine = [0, 4, 6, 7] + ([1, 5] if eps else [])
        for k, v in (("y", y), ("rstd", rstd)):
            val, b = want[k]
            ref.same(k, v.cpu()[fine], val[fine], b[fine])
        assert y[3].isnan().all() and rstd[3].isnan()
        assert y[2, 7].isnan() and (y[2, :7] == 0).all() and rstd[2] == 0
        q = y8.cpu().float()
        assert q[3].isnan().all() and q[2, 7].isnan() and (q[2, :7] == 0).all()
        assert scale[2] == 0 and scale[3] == 0
        if eps:
            assert (y[1] == 0).all() and (q[1] == 0).all() and scale[1] == 0
            ref.check_8bit(y8[[0, 4, 6, 7]], scale[[0, 4, 6, 7]].cpu(),
                           want["exact"][[0, 4, 6, 7]])
        else:
            assert y[1].isnan().all()


def test_wide_range_of_f32(red):
    """Squares past fp32's range in both directions."""
    g = torch.Generator().manual_seed(7)
    x = torch.randn(4, 777, generator=g) * torch.tensor([[1e30], [1e-30], [1e37], [1e-37]])
    w = torch.randn(777, generator=g)
    want = ref.add_rmsnorm(x, None, w, 0.0)
    y, rstd = torch.empty(4, 777, device="cuda"), torch.empty(4, device="cuda")
    red.add_rmsnorm_f32(x.cuda(), w.cuda(), y, rstd=rstd, eps=0.0)
    ref.same("rstd", rstd, *want["rstd"])
    ref.same("y", y, *want["y"])


@pytest.mark.parametrize("t", DTYPES)
def test_nan_stays_in_its_row(red, t):
    g = torch.Generator().manual_seed(8)
    h, dy, w = matrix(g, 300, 520, t), matrix(g, 300, 520, t), matrix(g, 1, 520, t)[0]
    rstd = (h.double().square().mean(1) + 1e-5).rsqrt().float()
    want, _ = ref.rmsnorm_grad(h, w, rstd, dy, None)["dx"]
    h[17, 3] = math.nan
    dx, dw = torch.empty_like(h, device="cuda"), torch.empty(520, device="cuda")
    getattr(red, "rmsnorm_grad_" + t)(h.cuda(), w.cuda(), rstd.cuda(), dy.cuda(), dx, dweight=dw)
    keep = torch.arange(300) != 17
    assert dx[17].isnan().all()
    _, b = ref.rmsnorm_grad(h[keep], w, rstd[keep], dy[keep], None)["dx"]
    ref.same("dx", dx.cpu()[keep], want[keep], b)
    assert dw[3].isnan() and dw.isnan().sum() == 1


def test_refusals(red):
    x = torch.zeros(4, 16, device="cuda")
    w, y, s = torch.zeros(16, device="cuda"), torch.zeros_like(x), torch.zeros(4, device="cuda")
    y8 = torch.zeros(4, 16, dtype=ref.E4M3, device="cuda")
    f = red.add_rmsnorm_f32
    for bad in (dict(y=None), dict(y=y8), dict(y8=y8), dict(yscale=s), dict(residual=x[:3]),
                dict(sum=x[:, :8]), dict(rstd=s[:3]), dict(y=y.t()), dict(weight=w[:8]),
                dict(weight=torch.zeros(32, device="cuda")[::2])):
        args = dict(x=x, weight=w, y=y)
        args.update(bad)
        with pytest.raises(ValueError):
            f(**args)
    for bad in (dict(y=y.half()), dict(residual=x.bfloat16()), dict(y8=y, yscale=s)):
        args = dict(x=x, weight=w, y=y)
        args.update(bad)
        with pytest.raises(TypeError):
            f(**args)
    with pytest.raises(red.ReduceError):
        f(x, w, x, sum=x)
    with pytest.raises(red.ReduceError):
        f(x, w, y, eps=-1.0)
    wide = torch.zeros(2, 16385, device="cuda")
    with pytest.raises(red.ReduceError):
        f(wide, wide[0], torch.empty_like(wide))
