"""The norm, the router's loss and the output layer's cross entropy together, as the
example's training step calls them: every gradient against the formulas in fp64 and
against differences of the whole loss, and the step captured into a graph."""
import importlib.util
import os

import pytest

import layer_reference as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location(
        "train_step", os.path.join(ROOT, "examples", "train_step.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_the_example_runs(example):
    losses = example.main(steps=3)
    assert len(losses) == 3 and all(v == v and abs(v) < 1e6 for v in losses)


def whole_loss(example, x, residual, norm, layer, router, targets, weight, experts):
    """The step's loss in fp64, without a rounding on the way."""
    h = x + residual
    y = h * (h.square().mean(1, keepdim=True) + 1e-6).rsqrt() * norm
    z = y @ layer.t()
    lse = z.logsumexp(1)
    w = weight.double()
    at = z.gather(1, targets.unsqueeze(1)).squeeze(1)
    loss = (w * (lse - at + example.Z_HEAD * lse ** 2)).sum()
    r = y @ router.t()
    counts = torch.bincount(experts[weight != 0].reshape(-1), minlength=example.EXPERTS).double()
    P = (torch.softmax(r, 1) * w.unsqueeze(1)).sum(0)
    loss = loss + example.BALANCE * example.EXPERTS * (counts / counts.sum() * P).sum()
    return loss + example.Z_ROUTER * (w * r.logsumexp(1) ** 2).sum()


def test_gradients_of_the_step(example):
    g = torch.Generator(device="cuda").manual_seed(3)
    step = example.Step(g)
    x, residual, targets, weight = example.batch(g)
    dx, dnorm, dlayer, drouter = step.losses(x, residual, targets, weight)

    h = (x.double() + residual.double()).bfloat16()
    y = torch.empty_like(x)
    import fp32_reductions_amd as red
    red.add_rmsnorm_bf16(x, step.norm, y, residual=residual)
    experts = (y @ step.router.t()).topk(example.CHOSEN, dim=1).indices
    leaves = [v.double().requires_grad_() for v in (x, residual, step.norm, step.layer, step.router)]
    loss = whole_loss(example, *leaves, targets, weight, experts)
    want = torch.autograd.grad(loss, leaves)

    # Every value on the way is rounded to bf16 (half a step, 2^-8 of itself at most):
    # the sum and the norm's output, the gradient of each logit, the two parts of dy and
    # their sum, the layers' and the results.  So each gradient is off by at most eight
    # such steps of the terms that make it, and those of random signs by far less: 8 x
    # 2^-8 of the whole gradient's norm.
    assert abs(step.loss.item() - loss.item()) <= 2 ** -8 * abs(loss.item())
    for name, got, value in (("x", dx, want[0]), ("norm", dnorm, want[2]),
                             ("layer", dlayer, want[3]), ("router", drouter, want[4])):
        off = (got.double() - value).norm() / value.norm()
        assert off <= 8 * 2 ** -8, (name, off.item())
    assert torch.equal(want[0], want[1])
    assert (dx[weight == 0] == 0).all()

    # The definition's own differences along the gradient found: the loss moves by its norm.
    direction = dx.double() / dx.double().norm()
    moved = [whole_loss(example, leaves[0].detach() + s * direction, *(v.detach() for v in leaves[1:]),
                        targets, weight, experts) for s in (1e-3, -1e-3)]
    slope = (moved[0] - moved[1]) / 2e-3
    assert abs(slope - want[0].norm()) <= 8 * 2 ** -8 * want[0].norm()
    assert h.shape == x.shape


def test_the_norm_alone_is_exact(example):
    """The same step's norm and gradient to the reference's bounds."""
    g = torch.Generator(device="cuda").manual_seed(4)
    step = example.Step(g)
    x, residual, _, _ = example.batch(g)
    import fp32_reductions_amd as red
    h, y, dx = (torch.empty_like(x) for _ in range(3))
    red.add_rmsnorm_bf16(x, step.norm, y, residual=residual, sum=h, rstd=step.rstd)
    want = ref.add_rmsnorm(x, residual, step.norm, 1e-6)
    for k, v in (("sum", h), ("y", y), ("rstd", step.rstd)):
        ref.same(k, v, *want[k])
    dnorm = torch.empty(example.WIDTH, device="cuda")
    red.rmsnorm_grad_bf16(h, step.norm, step.rstd, residual, dx, dweight=dnorm)
    want = ref.rmsnorm_grad(h, step.norm, step.rstd, residual, None)
    ref.same("dx", dx, *want["dx"])
    ref.same("dnorm", dnorm, *want["dweight"])


def test_captured_and_replayed(example):
    """The library's part of the step in a graph, replayed with new rows between eager
    work: every replay equals the eager call."""
    import fp32_reductions_amd as red

    g = torch.Generator(device="cuda").manual_seed(5)
    step = example.Step(g)
    x, residual, targets, weight = example.batch(g)
    logits = torch.randn(example.TOKENS, example.EXPERTS, device="cuda", generator=g).bfloat16()
    experts = logits.topk(example.CHOSEN, dim=1).indices
    bufs = {k: torch.empty_like(x) for k in ("h", "y", "dy", "dx")}
    bufs.update(dlayer=torch.empty_like(step.layer), dlogits=torch.empty_like(logits),
                dnorm=torch.empty(example.WIDTH, device="cuda"))
    room = torch.empty(red.linear_ce_workspace(x, step.layer), dtype=torch.uint8, device="cuda")

    def run():
        red.add_rmsnorm_bf16(x, step.norm, bufs["y"], residual=residual, sum=bufs["h"],
                             rstd=step.rstd)
        red.linear_ce_bf16(bufs["y"], step.layer, targets, step.loss, logp=step.logp,
                           dhidden=bufs["dy"], dweight=bufs["dlayer"], row_weight=weight,
                           workspace=room)
        red.router_balance_bf16(logits, experts, step.loss, step.counts, dlogits=bufs["dlogits"],
                                weight=weight, z_coef=0.001, accum=True)
        red.rmsnorm_grad_bf16(bufs["h"], step.norm, step.rstd, bufs["dy"], bufs["dx"],
                              dweight=bufs["dnorm"])

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        run()  # makes the stream's workspace
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            run()
    torch.cuda.synchronize()
    for seed in range(4):
        g.manual_seed(100 + seed)
        for old, new in zip((x, residual, targets, weight), example.batch(g)):
            old.copy_(new)
        with torch.cuda.stream(s):
            graph.replay()
        s.synchronize()
        got = {k: v.clone() for k, v in bufs.items()}
        got.update(loss=step.loss.clone(), counts=step.counts.clone())
        for v in bufs.values():
            v.fill_(7.0)
        run()
        torch.cuda.synchronize()
        for k, v in bufs.items():
            assert torch.equal(got[k], v), (seed, k)
        assert torch.equal(got["loss"], step.loss) and torch.equal(got["counts"], step.counts)


def test_two_streams_at_once():
    """Calls on two streams, each with workspaces of its own, at the same time."""
    import fp32_reductions_amd as red

    g = torch.Generator(device="cuda").manual_seed(6)
    z = torch.randn(20000, 64, device="cuda", generator=g)
    e = z.topk(4, dim=1).indices
    h = torch.randn(3000, 520, device="cuda", generator=g).bfloat16()
    W = torch.randn(5000, 520, device="cuda", generator=g).bfloat16() * 0.05
    y = torch.randint(5000, (3000,), device="cuda", generator=g)
    w = torch.ones(520, device="cuda").bfloat16()
    rstd = torch.ones(3000, device="cuda")

    def work(room):
        out = [torch.empty(1, device="cuda"), torch.empty(64, dtype=torch.int64, device="cuda"),
               torch.empty_like(z), torch.empty(1, device="cuda"), torch.empty_like(h),
               torch.empty_like(W), torch.empty_like(h), torch.empty(520, device="cuda")]
        red.router_balance_f32(z, e, out[0], out[1], dlogits=out[2])
        red.linear_ce_bf16(h, W, y, out[3], dhidden=out[4], dweight=out[5], workspace=room)
        red.rmsnorm_grad_bf16(h, w, rstd, h, out[6], dweight=out[7])
        return out

    size = red.linear_ce_workspace(h, W)
    rooms = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(2)]
    want = work(rooms[0])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(3):
        for s, room in zip(streams, rooms):
            with torch.cuda.stream(s):
                got.append(work(room))
    torch.cuda.synchronize()
    for out in got:
        assert all(torch.equal(a, b) for a, b in zip(out, want))
