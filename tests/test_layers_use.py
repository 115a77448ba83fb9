"""The layer operators as a program uses them: a whole model's gradients, the
example, gradients against differences, graphs, streams, in-place calls, long
buffers and the binding's refusals on device tensors."""
import math
import os
import sys

import numpy as np
import pytest

import software_pipelined_tiled_pgemm_amd as pg

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import ffn_lm
    finally:
        sys.path.pop(0)
    return ffn_lm


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_example_trains_and_generates(dtype):
    ex = example()
    model, losses, permutation = ex.train(steps=150, tokens=4096, vocab=500, dtype=dtype)
    assert losses[0] > 0.8 * math.log(500)
    assert losses[-1] < 0.35 * losses[0]
    text = model.generate(7, 10)
    assert sum(int(permutation[a]) == b for a, b in zip(text, text[1:])) >= 9


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_example_gradients(dtype):
    """The model's gradients against torch's in binary64 on the same 16-bit
    weights.  Each activation and gradient between operators is rounded to the
    type once per operator (4 forward, 4 backward, h and d inside): the norms
    of the errors add to less than 12 roundings of half a unit each."""
    ex = example()
    model = ex.Model(vocab=333, width=72, hidden=136, layers=2, dtype=dtype)
    g = torch.Generator(device="cuda").manual_seed(5)
    t = torch.randint(0, 333, (300,), generator=g, device="cuda")
    target = torch.randint(0, 333, (300,), generator=g, device="cuda")
    target[::7] = -100
    loss, grads = model.loss_and_grads(t, target)
    p = {k: v.double().requires_grad_() for k, v in model.weights.items()}
    x = p["embed"][t]
    for i in range(2):
        w, b, w_in, w_out = (p[n + str(i)] for n in ex.NAMES)
        y = torch.nn.functional.gelu(x @ w + b) + x
        gate, up = (y @ w_in).chunk(2, dim=1)
        x = (torch.nn.functional.silu(gate) * up) @ w_out + y
    exact = torch.nn.functional.cross_entropy(x * model.scale @ p["embed"].t(), target)
    exact.backward()
    u = 2.0 ** -11 if dtype is torch.float16 else 2.0 ** -8
    assert abs(float(loss) - float(exact)) <= 12 * u * float(exact)
    for k, v in grads.items():
        err = (v.double() - p[k].grad).norm() / p[k].grad.norm()
        assert float(err) <= 12 * u, (k, float(err))


def test_gradients_against_differences():
    """sum(y * c) of the block and of the linear layer, and the loss, moved
    along random directions: central differences of the binary64 formulas at
    the 16-bit inputs against the operators' gradients.  The gradients' entries
    carry at most 3 roundings of 2^-8 with random signs; along a direction of
    thousands of entries 2 % of |gradient| |direction| / sqrt(entries) times 4
    covers them."""
    torch.manual_seed(3)
    dt = torch.bfloat16
    M, D, F, V = 96, 72, 104, 301
    x = torch.randn(M, D, device="cuda").to(dt)
    wi = (torch.randn(D, 2 * F, device="cuda") * D ** -0.5).to(dt)
    wo = (torch.randn(F, D, device="cuda") * F ** -0.5).to(dt)
    wv = (torch.randn(V, D, device="cuda") * D ** -0.5).to(dt)
    c = torch.randn(M, D, device="cuda").to(dt)
    t = torch.randint(0, V, (M,), device="cuda")

    def ffn(x, wi, wo):
        g, u = (x @ wi).chunk(2, dim=1)
        return ((torch.sigmoid(g) * g * u) @ wo * c.double()).sum()

    def xent(x, wv):
        return torch.nn.functional.cross_entropy(x @ wv.t(), t)

    gu = torch.empty(M, 2 * F, dtype=dt, device="cuda")
    pg.pffn(x, wi, wo, gate_up=gu)
    _, lse = pg.pxent(x, wv, t)
    cases = [(ffn, (x, wi, wo), pg.pffn_bwd(c, x, wi, wo, gu)),
             (xent, (x, wv), pg.pxent_bwd(x, wv, t, lse))]
    for f, args, grads in cases:
        for i, grad in enumerate(grads):
            for seed in range(3):
                d = torch.randn(args[i].shape, device="cuda", dtype=torch.float64,
                                generator=torch.Generator(device="cuda").manual_seed(seed))
                h = 1e-5
                a = [v.double() for v in args]
                a[i] = a[i] + h * d
                up = f(*a)
                a[i] = a[i] - 2 * h * d
                slope = float((up - f(*a)) / (2 * h))
                got = float((grad.double() * d).sum())
                scale = float(grad.double().norm() * d.norm()) / math.sqrt(d.numel())
                assert abs(got - slope) <= 0.08 * scale + 1e-6, (f.__name__, i, got, slope)


def test_same_bits_call_after_call():
    torch.manual_seed(1)
    M, D, F, V = 300, 264, 520, 1003
    for dt in (torch.float16, torch.bfloat16):
        x = torch.randn(M, D, device="cuda").to(dt)
        wi = torch.randn(D, 2 * F, device="cuda").mul(0.06).to(dt)
        wo = torch.randn(F, D, device="cuda").mul(0.04).to(dt)
        wv = torch.randn(V, D, device="cuda").mul(0.06).to(dt)
        t = torch.randint(0, V, (M,), device="cuda")

        def everything():
            gu = torch.empty(M, 2 * F, dtype=dt, device="cuda")
            y = pg.pffn(x, wi, wo, residual=x, gate_up=gu)
            loss, lse = pg.pxent(y, wv, t)
            dy, dw = pg.pxent_bwd(y, wv, t, lse)
            rest = pg.pffn_bwd(dy, x, wi, wo, gu)
            z = torch.empty(M, D, dtype=dt, device="cuda")
            u = pg.plinear(x, wo[:D], act="gelu", preact=z)
            grads = [dw, *rest, *pg.plinear_bwd(u, x, wo[:D], preact=z, act="gelu")]
            norm = pg.pclip_grad_norm(grads, 0.5)
            return [y, loss, lse, dy, u, norm] + grads
        first = everything()
        for _ in range(3):
            for a, b in zip(first, everything()):
                assert torch.equal(a, b)


def test_graph_replay():
    """A captured step replayed several times, with eager work in between,
    gives the eager results."""
    torch.manual_seed(2)
    dt = torch.bfloat16
    M, D, F, V = 130, 128, 200, 517
    x = torch.randn(M, D, device="cuda").to(dt)
    wi = torch.randn(D, 2 * F, device="cuda").mul(0.09).to(dt)
    wo = torch.randn(F, D, device="cuda").mul(0.07).to(dt)
    wv = torch.randn(V, D, device="cuda").mul(0.09).to(dt)
    t = torch.randint(0, V, (M,), device="cuda")
    gu = torch.empty(M, 2 * F, dtype=dt, device="cuda")

    def step():
        y = pg.pffn(x, wi, wo, residual=x, gate_up=gu)
        loss, lse = pg.pxent(y, wv, t)
        dy, dw = pg.pxent_bwd(y, wv, t, lse)
        grads = [dw, *pg.pffn_bwd(dy, x, wi, wo, gu, dx_residual=dy)]
        norm = pg.pclip_grad_norm(grads, 0.1)
        return [y, loss, norm] + grads
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for i in range(4):
        x.copy_(torch.randn(M, D, device="cuda").to(dt))
        t.copy_(torch.randint(0, V, (M,), device="cuda"))
        g.replay()
        torch.cuda.synchronize()
        replayed = [o.clone() for o in out]
        for a, b in zip(replayed, step()):
            assert torch.equal(a, b)
        torch.cuda.synchronize()


def test_other_stream():
    """Calls on a stream of their own, outputs and workspaces from its pool,
    while the current stream is busy."""
    torch.manual_seed(4)
    x = torch.randn(200, 1000, device="cuda").half()
    w = torch.randn(1000, 700, device="cuda").mul(0.03).half()
    ref = pg.plinear(x, w, act="silu")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(20):
        big = torch.randn(4096, 4096, device="cuda") @ torch.randn(4096, 4096, device="cuda")
        outs.append(pg.plinear(x, w, act="silu", stream=s))
        del big
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)


def test_in_place():
    torch.manual_seed(6)
    x = torch.randn(70, 64, device="cuda").bfloat16()
    w = torch.randn(64, 64, device="cuda").mul(0.1).bfloat16()
    r = torch.randn(70, 64, device="cuda").bfloat16()
    ref = pg.plinear(x, w, residual=r)
    buf = r.clone()
    assert pg.plinear(x, w, residual=buf, out=buf) is buf and torch.equal(buf, ref)
    wi = torch.randn(64, 96, device="cuda").mul(0.1).bfloat16()
    wo = torch.randn(48, 64, device="cuda").mul(0.1).bfloat16()
    ref = pg.pffn(x, wi, wo, residual=x)
    buf = x.clone()
    assert torch.equal(pg.pffn(buf, wi, wo, residual=buf, out=buf), ref)
    ref = pg.plinear_bwd(r, x, w, dx_residual=r)[0]
    acc = r.clone()
    got = pg.plinear_bwd(r, x, w, dx_residual=acc, dx=acc, needs=(True, False, False))
    assert torch.equal(got[0], ref) and got[1] is None and got[2] is None


def test_offsets_past_32_bits():
    """A row pitch and row count whose products pass 2^32 bytes, on each side
    of a product; only the ends are compared (they sit in the last rows)."""
    M, K, N, pitch = 2100, 64, 72, (1 << 20) + 8
    buf = torch.zeros(M * pitch, dtype=torch.float16, device="cuda")
    x = buf.view(M, pitch)[:, :K]
    y = buf.view(M, pitch)[:, 512:512 + N]
    torch.manual_seed(8)
    x.copy_(torch.randn(M, K, device="cuda"))
    w = torch.randn(K, N, device="cuda").mul(0.1).half()
    pg.plinear(x, w, act="relu", out=y)
    assert torch.equal(y, pg.plinear(x.contiguous(), w, act="relu"))
    dw = pg.plinear_bwd(y, x, w, needs=(False, True, False))[1]
    assert torch.equal(dw, pg.plinear_bwd(y.contiguous(), x.contiguous(), w,
                                          needs=(False, True, False))[1])
    # a vocabulary of strided rows past 2^32 bytes
    V, t = 2100, torch.arange(9, device="cuda") * 200
    wv = buf.view(M, pitch)[:, :K]
    loss, lse = pg.pxent(x[:9].contiguous(), wv, t)
    loss2, lse2 = pg.pxent(x[:9].contiguous(), wv.contiguous(), t)
    assert torch.equal(loss, loss2) and torch.equal(lse, lse2)
    dx, dwv = pg.pxent_bwd(x[:9].contiguous(), wv, t, lse)
    dx2, dwv2 = pg.pxent_bwd(x[:9].contiguous(), wv.contiguous(), t, lse)
    assert torch.equal(dx, dx2) and torch.equal(dwv, dwv2) and dwv.shape == (V, K)


def test_masked_rows_reach_no_gradient():
    x = torch.randn(90, 40, device="cuda").half()
    w = torch.randn(77, 40, device="cuda").mul(0.2).half()
    t = torch.randint(0, 77, (90,), device="cuda")
    t[10:40] = -100
    _, lse = pg.pxent(x, w, t)
    ref = pg.pxent_bwd(x, w, t, lse)
    y = x.clone()
    y[10:20], y[20:30], y[30:40] = float("nan"), float("inf"), 65504.0
    _, lse = pg.pxent(y, w, t)
    got = pg.pxent_bwd(y, w, t, lse)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    assert not bool(got[0][10:40].any())


def test_empty_sizes():
    f = lambda *s: torch.randn(*s, device="cuda").half()  # noqa: E731
    assert pg.plinear(f(0, 8), f(8, 16)).shape == (0, 16)
    assert pg.plinear(f(5, 8), f(8, 0)).shape == (5, 0)
    r = f(5, 16)
    assert torch.equal(pg.plinear(f(5, 0), f(0, 16), residual=r), r)
    dx, dw, db = pg.plinear_bwd(f(0, 16), f(0, 8), f(8, 16))
    assert dx.shape == (0, 8) and not bool(dw.any()) and not bool(db.any())
    dx, dw, db = pg.plinear_bwd(f(5, 0), f(5, 8), f(8, 0))
    assert not bool(dx.any()) and dw.shape == (8, 0) and db.shape == (0,)
    gu = f(0, 12)
    assert pg.pffn(f(0, 8), f(8, 12), f(6, 4), gate_up=gu).shape == (0, 4)
    dx, dwi, dwo = pg.pffn_bwd(f(0, 4), f(0, 8), f(8, 12), f(6, 4), gu)
    assert not bool(dwi.any()) and not bool(dwo.any())
    t = torch.zeros(0, dtype=torch.int64, device="cuda")
    loss, lse = pg.pxent(f(0, 8), f(9, 8), t)
    assert float(loss) == 0.0 and lse.shape == (0,)
    dx, dw = pg.pxent_bwd(f(0, 8), f(9, 8), t, lse)
    assert dx.shape == (0, 8) and not bool(dw.any())


def test_refusals_on_device_tensors():
    x = torch.zeros(4, 8, device="cuda").half()
    w = torch.zeros(8, 6, device="cuda").half()
    for bad in (lambda: pg.plinear(x, w.t()), lambda: pg.plinear(x, w.float()),
                lambda: pg.plinear(x, torch.zeros(9, 6, device="cuda").half()),
                lambda: pg.plinear(x, torch.zeros(6, 8, device="cuda").half().t()),
                lambda: pg.plinear(x, w, bias=torch.zeros(7, device="cuda").half()),
                lambda: pg.plinear(x, w, residual=torch.zeros(4, 7, device="cuda").half()),
                lambda: pg.plinear(x[:1].expand(4, 8), w),
                lambda: pg.plinear(x.view(4, 2, 4), w),
                lambda: pg.plinear_bwd(x, x, torch.zeros(8, 8, device="cuda").half(), act="silu"),
                lambda: pg.pffn(x, torch.zeros(8, 5, device="cuda").half(), w),
                lambda: pg.pxent(x, torch.zeros(9, 8, device="cuda").half(),
                                 torch.zeros(4, device="cuda", dtype=torch.int32)),
                lambda: pg.pxent(x, torch.zeros(9, 8, device="cuda").half(),
                                 torch.zeros(4, device="cuda", dtype=torch.int64),
                                 reduction="median"),
                lambda: pg.pclip_grad_norm([x.t()], 1.0),
                lambda: pg.pclip_grad_norm([x], 1.0, out=[x[:2].contiguous()]),
                lambda: pg.pclip_grad_norm([x.double()], 1.0)):
        with pytest.raises((TypeError, ValueError)):
            bad()
    with pytest.raises(pg.PgemmError):
        pg.plinear(x, torch.zeros(8, 8, device="cuda").half(), out=x)   # out is x
    with pytest.raises(pg.PgemmError):
        pg.pclip_grad_norm([x, x], 1.0)                                  # one tensor twice
    with pytest.raises(pg.PgemmError):
        pg.plinear(x[:, 1:], torch.zeros(7, 6, device="cuda").half(),
                   workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    assert np.isfinite(float(pg.pclip_grad_norm([x.clone()], 1.0)))
