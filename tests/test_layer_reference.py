"""The fp64 references of the operators around the output layer: their
gradients against automatic differentiation and against differences of the
definitions, written here a second time."""
import math

import pytest

torch = pytest.importorskip("torch")

import layer_reference as ref  # noqa: E402

G = torch.Generator().manual_seed(11)


def normal(*shape):
    return torch.randn(*shape, generator=G, dtype=torch.float64)


def differences(f, x, n=12, step=1e-5):
    """(indices, central differences of the scalar f there)."""
    flat = x.reshape(-1)
    at = torch.randperm(flat.numel(), generator=G)[:n]
    out = []
    for i in at.tolist():
        d = torch.zeros_like(flat)
        d[i] = step
        out.append((f(x + d.view_as(x)) - f(x - d.view_as(x))) / (2 * step))
    return at, torch.stack(out)


def close(a, b, tol):
    assert ((a - b).abs() <= tol * (1e-3 + b.abs().max())).all(), (a - b).abs().max()


def test_norm():
    h, w, dy, ds = normal(5, 9), normal(9), normal(5, 9), normal(5, 9)
    eps = 0.01

    def f(h, w=w):
        return (dy * h * w / (h.square().mean(1, keepdim=True) + eps).sqrt()).sum() + (ds * h).sum()

    r = (h.square().mean(1) + eps).rsqrt()
    got = ref.rmsnorm_grad(h, w, r, dy, ds)
    hg, wg = h.clone().requires_grad_(), w.clone().requires_grad_()
    dh, dw = torch.autograd.grad(f(hg, wg), [hg, wg])
    close(got["dx"][0], dh, 1e-12)
    close(got["dweight"][0], dw, 1e-12)
    at, d = differences(f, h)
    close(got["dx"][0].reshape(-1)[at], d, 1e-8)


@pytest.mark.parametrize("weighted", [False, True])
def test_router(weighted):
    z = normal(7, 5)
    experts = torch.tensor([[0, 1], [1, 2], [4, -1], [0, 5], [3, 3], [1, 0], [2, 4]])
    w = torch.tensor([0.5, 0.0, 1.0, 2.0, 0.25, 0.0, 1.0]) if weighted else None
    n = torch.tensor([2, 1, 1, 2, 2]) if weighted else torch.tensor([3, 3, 2, 2, 2])
    got = ref.router_balance(z, experts, w, 0.25, 0.125)
    assert torch.equal(got["counts"][0], n.double())
    ww = torch.full((7,), 1 / 7.0) if w is None else w

    def f(z):
        total = 0.0
        for r in range(7):
            p = torch.softmax(z[r], 0)
            total = total + ww[r].double() * (0.25 * 5 * (n.double() / n.sum() * p).sum()
                                              + 0.125 * torch.logsumexp(z[r], 0) ** 2)
        return total

    close(got["loss"][0], f(z), 1e-7)
    zg = z.clone().requires_grad_()
    close(got["dlogits"][0], torch.autograd.grad(f(zg), zg)[0], 1e-7)
    at, d = differences(f, z)
    close(got["dlogits"][0].reshape(-1)[at], d, 1e-6)


@pytest.mark.parametrize("scale,zc", [(1.0, 0.0), (0.5, 0.25)])
def test_linear(scale, zc):
    h, W = normal(6, 8).bfloat16(), normal(11, 8).bfloat16()
    y = torch.tensor([0, 10, -100, 3, 11, 5])
    w = torch.tensor([1.0, 0.5, 1.0, 0.0, 2.0, 0.25])
    got = ref.linear_ce(h, W, y, w, scale, zc)

    def f(h, W=W.double()):
        total = 0.0
        for r in (0, 1, 5):
            z = scale * (W @ h[r])
            lse = torch.logsumexp(z, 0)
            total = total + w[r].double() * (lse - z[y[r]] + zc * lse ** 2)
        return total

    hg, wg = h.double().requires_grad_(), W.double().requires_grad_()
    dh, dw = torch.autograd.grad(f(hg, wg), [hg, wg])
    close(got["loss"][0], f(h.double()), 1e-12)
    close(got["dhidden"][0], dh, 1e-12)
    close(got["dweight"][0], dw, 1e-12)
    at, d = differences(f, h.double())
    close(got["dhidden"][0].reshape(-1)[at], d, 1e-7)
    at, d = differences(lambda v: f(h.double(), v), W.double())
    close(got["dweight"][0].reshape(-1)[at], d, 1e-7)


def test_bounds_are_tight_enough():
    """A bound is of the order of the type's rounding, not larger than the
    result: a wrong formula cannot hide in it."""
    h, W = normal(20, 64).bfloat16(), (normal(300, 64) / 4).bfloat16()
    y = torch.randint(300, (20,), generator=G)
    got = ref.linear_ce(h, W, y, None, 1.0, 0.0)
    for k in ("dhidden", "dweight"):
        v, b = got[k]
        assert b.norm() <= 0.05 * v.norm(), k
    for k in ("loss", "logp", "lse"):
        v, b = got[k]
        assert (b <= 1e-4 * v.abs()).all(), k
    z = normal(50, 16)
    got = ref.router_balance(z.float(), torch.randint(16, (50, 2), generator=G), None, 0.01, 0.001)
    assert (got["dlogits"][1] <= 1e-3 * got["dlogits"][0].abs().max()).all()
    x = normal(4, 100).float()
    got = ref.add_rmsnorm(x, None, x[0], 1e-6)
    assert (got["y"][1] <= 1e-6 * (1e-6 + got["y"][0].abs())).all()
    assert math.isfinite(got["rstd"][1].sum())
