"""The norm, linear layers and gated blocks as torch functions (layers.py): values and
gradients against autograd in 64 bits at what is kept, refusals, streams, graphs, and
a block of them together."""
import gc
import threading

import pytest
import torch

import tests.ff_ref as F
import zero_sharded_optimizer_step_gb300 as z

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF = torch.bfloat16
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def randn(g, *shape, dtype=BF, sigma=1.0, grad=False):
    t = (torch.randn(*shape, generator=g, device=DEV) * sigma).to(dtype)
    return t.requires_grad_() if grad else t


def near(got, want, halves):
    """Relative to the whole: `halves` roundings of the type, each at most half a step."""
    u = torch.finfo(got.dtype).eps / 2
    off = (got.double() - want).norm()
    assert float(off) <= halves * u * float(want.norm()) + 1e-30, float(off / want.norm() / u)


def kept(v, keep8, dtype):
    """What the backward pass sees of v."""
    if keep8:
        return F.rounded(F.pack(v)[0], dtype).double()
    return v.to(dtype).double()


@pytest.mark.parametrize("keep8", [False, True])
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n,k", [(6, 40, 72), (300, 513, 136)])
def test_linear(act, m, n, k, keep8):
    """The output is rounded once (one half step, and what fp32 sums lose); a gradient
    is a product with dz rounded to the type, and rounded itself: two half steps
    at the most, as norms, and a quarter more for what is kept next to a border."""
    g = gen(m)
    x, w = randn(g, 2, m // 2, k, grad=True), randn(g, n, k, sigma=k ** -0.5, grad=True)
    b, r = randn(g, n, grad=True), randn(g, 2, m // 2, n, grad=True)
    y = z.linear(x, w, b, act, r, keep8)
    dy = randn(g, 2, m // 2, n)
    y.backward(dy)
    x64, w64, d64 = x.detach().double().view(m, k), w.detach().double(), dy.double().view(m, n)
    v = x64 @ w64.t() + b.detach().double()
    kind = ACTS.index(act)
    near(y.detach().view(m, n), F.activation(v, kind)[0] + r.detach().double().view(m, n), 1.1)
    dz = d64 * (F.activation(kept(v, keep8, BF), kind)[1] if act != "none" else 1.0)
    if keep8:
        x64 = F.rounded(F.pack(x64)[0], BF).double()
    near(x.grad.view(m, k), dz @ w64, 2.25)
    near(w.grad, dz.t() @ x64, 2.25)
    near(b.grad, dz.sum(0), 1.25)
    assert torch.equal(r.grad, dy)


@pytest.mark.parametrize("keep8", [False, True])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh", "none"])
@pytest.mark.parametrize("m,n,k", [(6, 40, 72), (300, 513, 136)])
def test_gated(act, m, n, k, keep8):
    g = gen(m + 1)
    x = randn(g, 3, m // 3, k, grad=True)
    wg, wu = (randn(g, n, k, sigma=k ** -0.5, grad=True) for _ in range(2))
    h = z.gated(x, wg, wu, act, keep8)
    dh = randn(g, 3, m // 3, n)
    h.backward(dh)
    x64, d64 = x.detach().double().view(m, k), dh.double().view(m, n)
    wg64, wu64 = wg.detach().double(), wu.detach().double()
    gate, up, kind = x64 @ wg64.t(), x64 @ wu64.t(), ACTS.index(act)
    near(h.detach().view(m, n), F.activation(gate, kind)[0] * up, 1.1)
    gate, up = kept(gate, keep8, BF), kept(up, keep8, BF)
    f, slope = F.activation(gate, kind)
    dg, du = d64 * up * slope, d64 * f
    if keep8:
        x64 = F.rounded(F.pack(x64)[0], BF).double()
    near(x.grad.view(m, k), dg @ wg64 + du @ wu64, 2.25)
    near(wg.grad, dg.t() @ x64, 2.25)
    near(wu.grad, du.t() @ x64, 2.25)


@pytest.mark.parametrize("dtype", [torch.float32, BF, torch.float16])
@pytest.mark.parametrize("with_residual", [False, True])
def test_rms_norm(dtype, with_residual):
    g = gen(3)
    x = randn(g, 4, 30, 200, dtype=dtype, grad=True)
    r = randn(g, 4, 30, 200, dtype=dtype, grad=True) if with_residual else None
    w = randn(g, 200, dtype=dtype, grad=True)
    out = z.rms_norm(x, w, r, eps=1e-4)
    y, total = out if with_residual else (out, None)
    dy, dt = randn(g, 4, 30, 200, dtype=dtype), randn(g, 4, 30, 200, dtype=dtype)
    s64 = x.detach().double()
    if with_residual:
        s64 = (s64 + r.detach().double()).to(dtype).double()
        assert torch.equal(total.detach().double(), s64)
        torch.autograd.backward([y, total], [dy, dt])
    else:
        y.backward(dy)
    s64 = s64.requires_grad_()
    w64 = w.detach().double().requires_grad_()
    y64 = s64 * ((s64 * s64).mean(-1, keepdim=True) + 1e-4) ** -0.5 * w64
    loss = (y64 * dy.double()).sum() + ((s64 * dt.double()).sum() if with_residual else 0.0)
    loss.backward()
    # one rounding; in fp32 the sums' own errors, 200 (120 rows: 120) terms and a few roundings
    halves = 64 if dtype == torch.float32 else 1.25
    near(y.detach(), y64.detach(), halves)
    near(x.grad, s64.grad, halves)
    near(w.grad, w64.grad, halves)
    if with_residual:
        assert torch.equal(r.grad, x.grad)


def test_rms_norm_only_through_its_sum_or_its_norm():
    g = gen(4)
    for which in (0, 1):
        x, r, w = randn(g, 5, 64, grad=True), randn(g, 5, 64), randn(g, 64, grad=True)
        out = z.rms_norm(x, w, r)[which]
        d = randn(g, 5, 64)
        out.backward(d)
        if which:
            assert torch.equal(x.grad, d) and (w.grad is None or not w.grad.any())
        else:
            assert bool(x.grad.any()) and bool(w.grad.any())


def test_packed_norm_feeds_a_layer():
    """The norm's 8-bit output as what the layer keeps of its input."""
    g = gen(5)
    x, w = randn(g, 40, 96), randn(g, 96)
    weight = randn(g, 64, 96, sigma=0.1, grad=True)
    y, q = z.rms_norm(x, w, packed=True)
    dy = randn(g, 40, 64)
    z.linear(y, weight, keep8=q).backward(dy)
    near(weight.grad, dy.double().t() @ q.values(BF).double(), 1.25)
    first, weight.grad = weight.grad, None
    z.linear(y, weight, keep8=True).backward(dy)          # packed from the rounded norm
    assert float((weight.grad.double() - first.double()).norm()) < 0.05 * float(first.double().norm())


def test_pack8_round_trip():
    x = randn(gen(6), 30, 100, dtype=torch.float32)
    p = z.pack8(x)
    assert torch.equal(p.values(), F.rounded(F.pack(x.double())[0], torch.float32))
    assert torch.equal(z.pack8(x.t().contiguous().t()[:, :40].contiguous()).values(),
                       F.rounded(F.pack(x[:, :40].double())[0], torch.float32))


def test_matmul_writes_and_adds_where_a_rank_keeps_its_gradients():
    g = gen(7)
    x, dy = randn(g, 50, 72), randn(g, 50, 40)
    want, err = F.product(dy.double().t(), x.double().t())
    for dtype in (torch.float32, BF):
        buf = torch.full((40 * 72 + 6,), 3.0, dtype=dtype, device=DEV)
        grad = buf[3:-3].view(40, 72)
        z.matmul(dy, x, True, True, out=grad, accumulate=True)
        F.within(grad, want + 3.0, err + 2.0 ** -24 * (want.abs() + 3.0))
        z.matmul(dy, x, True, True, out=grad)
        F.within(grad, want, err)
        assert buf[:3].tolist() == [3.0] * 3 and buf[-3:].tolist() == [3.0] * 3


def test_nothing_is_kept_where_no_backward_pass_can_follow():
    g = gen(8)
    x, w = randn(g, 512, 256), randn(g, 512, 256, grad=True)
    for call in (lambda: z.linear(x, w, activation="gelu"), lambda: z.gated(x, w, w)):
        with torch.no_grad():
            call()
            torch.cuda.synchronize()
            torch.cuda.reset_peak_memory_stats()
            before = torch.cuda.memory_allocated()
            y = call()
            assert torch.cuda.max_memory_allocated() - before == 512 * 512 * 2
        assert not y.requires_grad


def test_gradients_of_awkward_shapes():
    """Expanded, transposed and empty ones."""
    g = gen(9)
    x, w = randn(g, 6, 72, grad=True), randn(g, 40, 72, grad=True)
    z.linear(x, w, activation="silu").sum().backward()          # an expanded gradient
    first = x.grad.clone(), w.grad.clone()
    x.grad = w.grad = None
    z.linear(x, w, activation="silu").backward(torch.ones(40, 6, dtype=BF, device=DEV).t())
    assert torch.equal(x.grad, first[0]) and torch.equal(w.grad, first[1])
    e = torch.empty(0, 72, dtype=BF, device=DEV, requires_grad=True)
    b = randn(g, 40, grad=True)
    w.grad = None
    y = z.linear(e, w, b, "gelu")
    assert y.shape == (0, 40)
    y.sum().backward()
    assert e.grad.shape == (0, 72) and not w.grad.any() and not b.grad.any()
    w.grad = None
    h = z.gated(e, w, w.detach())
    h.sum().backward()
    assert not w.grad.any()
    nw = randn(g, 72, grad=True)
    z.rms_norm(e, nw).sum().backward()
    assert not nw.grad.any()
    xt = randn(g, 72, 6).t()                                      # rows that are not runs
    assert torch.equal(z.linear(xt, w.detach()), z.linear(xt.contiguous(), w.detach()))


def test_rows_of_nothing():
    """No columns to go through: a product is its bias, a norm has no elements."""
    g = gen(17)
    x = torch.empty(2, 3, 0, dtype=BF, device=DEV, requires_grad=True)
    w = torch.empty(40, 0, dtype=BF, device=DEV, requires_grad=True)
    b = randn(g, 40, grad=True)
    y = z.linear(x, w, b, "relu")
    assert torch.equal(y, b.detach().relu().expand(2, 3, 40))
    y.sum().backward()
    assert x.grad.shape == x.shape and w.grad.shape == w.shape
    assert torch.equal(b.grad, 6 * (b.detach() > 0).to(BF))
    assert not z.gated(x, w, w).any()
    nw = torch.empty(0, dtype=BF, device=DEV, requires_grad=True)
    y, total, q = z.rms_norm(x, nw, residual=x, packed=True)
    assert y.shape == total.shape == x.shape and (q.rows, q.cols) == (6, 0)
    (y.sum() + total.sum()).backward()
    assert nw.grad.shape == (0,)
    assert z.linear(randn(g, 5, 64), torch.empty(0, 64, dtype=BF, device=DEV)).shape == (5, 0)


@pytest.mark.parametrize("keep8", [False, True])
def test_what_is_kept_is_freed_with_the_output(keep8):
    """At once, without the collector: no reference goes round in a circle."""
    p = params(gen(18))
    h = randn(gen(19), 70, 64)
    block(p, h, keep8)                           # what the first calls make is there
    gc.collect()
    gc.disable()
    try:
        before = torch.cuda.memory_allocated()
        y = block(p, h, keep8)
        assert torch.cuda.memory_allocated() > before
        del y
        assert torch.cuda.memory_allocated() == before
    finally:
        gc.enable()


def test_second_derivatives_are_refused():
    g = gen(10)
    x, w = randn(g, 4, 64, grad=True), randn(g, 64, 64, grad=True)
    nw = randn(g, 64, grad=True)
    for out, leaves in ((z.linear(x, w, activation="gelu"), (x, w)), (z.gated(x, w, w), (x, w)),
                        (z.rms_norm(x, nw), (x, nw))):
        grads = torch.autograd.grad(out.float().square().sum(), leaves, create_graph=True)
        for gr in grads:
            with pytest.raises(RuntimeError, match="once"):
                torch.autograd.grad(gr.float().sum(), leaves, allow_unused=True,
                                    retain_graph=True)


def test_refusals():
    g = gen(11)
    x, w, b = randn(g, 4, 64), randn(g, 40, 64), randn(g, 40)
    f = x.float()
    for bad in (lambda: z.linear(x, w[:, :60]), lambda: z.linear(f, w.float()),
                lambda: z.linear(x, w.half()), lambda: z.linear(x, w, b[:3]),
                lambda: z.linear(x, w, b.float()), lambda: z.linear(x, w, activation="tanh"),
                lambda: z.linear(x, w, residual=x), lambda: z.linear(x, w.cpu()),
                lambda: z.linear(x, w, keep8=z.pack8(w)), lambda: z.gated(x, w, w[:30]),
                lambda: z.gated(x, w, w.half()), lambda: z.gated(f, w, w),
                lambda: z.rms_norm(x, b), lambda: z.rms_norm(x, w[0].float()),
                lambda: z.rms_norm(x, w[0], residual=w), lambda: z.rms_norm(x.long(), w[0]),
                lambda: z.matmul(x, w, accumulate=True), lambda: z.matmul(x, w, a2=x),
                lambda: z.matmul(x, w, out=x), lambda: z.matmul(x, w, a_cols=True),
                lambda: z.matmul(x, w, kept=torch.empty(4, 40, device=DEV)),
                lambda: z.matmul(x, w, packed=z.pack8(x)), lambda: z.pack8(x.view(2, 2, 64)),
                lambda: z.matmul(x, w, residual=torch.empty(4, 40, device=DEV))):
        with pytest.raises(ValueError):
            bad()


def block(p, h, keep8):
    """A pre-norm feed-forward block on the residual stream h, twice: gated and
    with a bias and GELU."""
    y, h = z.rms_norm(p["x"], p["n1"], residual=h)
    y = z.gated(y, p["wg"], p["wu"], keep8=keep8)
    h = z.linear(y, p["wd"], residual=h, keep8=keep8)
    y, total = z.rms_norm(z.linear(h, p["w1"], p["b1"], "gelu_tanh", keep8=keep8), p["n2"],
                          residual=torch.zeros(h.shape[0], p["n2"].numel(), dtype=h.dtype,
                                               device=h.device))
    return z.linear(y, p["w2"], p["b2"], residual=h, keep8=keep8) + 0.0 * total.sum()


def plain_block(p, h):
    def norm(v, w):
        return v * ((v * v).mean(-1, keepdim=True) + 1e-5) ** -0.5 * w

    s = p["x"] + h
    y = norm(s, p["n1"])
    h = (torch.nn.functional.silu(y @ p["wg"].t()) * (y @ p["wu"].t())) @ p["wd"].t() + s
    y = norm(torch.nn.functional.gelu(h @ p["w1"].t() + p["b1"], approximate="tanh"), p["n2"])
    return y @ p["w2"].t() + p["b2"] + h


def params(g, m=70, d=64, hidden=136, dtype=BF):
    def r(*s, sigma):
        return (torch.randn(*s, generator=g, device=DEV) * sigma).to(dtype).requires_grad_()

    return dict(x=r(m, d, sigma=1), n1=r(d, sigma=1), wg=r(hidden, d, sigma=d ** -0.5),
                wu=r(hidden, d, sigma=d ** -0.5), wd=r(d, hidden, sigma=hidden ** -0.5),
                w1=r(hidden, d, sigma=d ** -0.5), b1=r(hidden, sigma=0.1), n2=r(hidden, sigma=1),
                w2=r(d, hidden, sigma=hidden ** -0.5), b2=r(d, sigma=0.1))


@pytest.mark.parametrize("keep8", [False, True])
def test_a_block_of_them_together(keep8):
    """Values and gradients of the whole against autograd in 64 bits.  A dozen roundings
    to bf16 lie between a leaf and its gradient, each of half a step at most and
    carried on by factors of about one: 16 of them, as norms; 8-bit kept values are
    off by up to 2^-4, a third of that as a norm (uniform over a step that is between
    2^-4 and 2^-3 of the value), in each of the activations that a gradient goes through."""
    g = gen(12)
    p = params(g)
    h = randn(g, 70, 64)
    out = block(p, h, keep8)
    dy = randn(g, 70, 64)
    out.backward(dy)
    p64 = {k: v.detach().double().requires_grad_() for k, v in p.items()}
    want = plain_block(p64, h.double())
    want.backward(dy.double())
    near(out.detach(), want.detach(), 16)
    for name in p:
        allowed = 16 if not keep8 else 16 + 3 * 2.0 ** -4 / 2.0 ** -8 / 3
        near(p[name].grad, p64[name].grad, allowed)
    assert z.zero_matmul_timeouts() == 0


@pytest.mark.parametrize("keep8", [False, True])
def test_forward_and_backward_in_a_captured_graph(keep8):
    g = gen(13)
    p = params(g)
    leaves = list(p.values())
    h, dy = randn(g, 70, 64), randn(g, 70, 64)

    def step():
        return torch.autograd.grad(block(p, h, keep8), leaves, dy)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = [t.clone() for t in step()]
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = step()
    torch.cuda.current_stream().wait_stream(side)
    with torch.no_grad():
        for _ in range(2):
            for t in got:
                t.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        # new inputs in the same places
        h.copy_(randn(g, 70, 64))
        graph.replay()
        torch.cuda.synchronize()
        first = [t.clone() for t in got]
    assert all(torch.equal(a, b) for a, b in zip(step(), first))


def test_two_streams_and_two_threads_at_once():
    """Each call's workspaces are its own."""
    g = gen(14)
    sets = [params(gen(20 + k), m=201, d=65, hidden=133) for k in range(2)]
    h = randn(g, 201, 65)
    dy = randn(g, 201, 65)
    want = [[t.clone() for t in torch.autograd.grad(block(p, h, True), list(p.values()), dy)]
            for p in sets]
    torch.cuda.synchronize()
    wrong = []

    def work(k):
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(10):
                got = torch.autograd.grad(block(sets[k], h, True), list(sets[k].values()), dy)
                torch.cuda.current_stream().synchronize()
                if not all(torch.equal(a, b) for a, b in zip(got, want[k])):
                    wrong.append(k)

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong


def test_a_block_trains_under_the_optimizer():
    """Gradients of the block into the ranks' buffers, a step, and the weights move."""
    g = gen(15)
    p = params(g)
    leaves = [p[k] for k in p if k != "x"]
    opt = z.ZeroAdam(leaves, world=2, lr=1e-2)
    before = [t.detach().clone() for t in leaves]
    for k in range(2):
        h, dy = randn(g, 70, 64), randn(g, 70, 64)
        for buf, grad in zip(opt.rank_grads(k), torch.autograd.grad(block(p, h, True), leaves, dy)):
            buf.copy_(grad)
    opt.step()
    assert all(torch.isfinite(t).all() and not torch.equal(t, b) for t, b in zip(leaves, before))
