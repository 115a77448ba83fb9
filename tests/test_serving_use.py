"""The norm, the microscaled product and sampling as a program uses them:
together, a whole model's gradients, graphs, streams, long buffers and the
binding's refusals on device tensors."""
import os
import sys

import numpy as np
import pytest

import software_pipelined_tiled_pgemm_amd as pg

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
UNIT = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


def example():
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import served_lm
    finally:
        sys.path.pop(0)
    return served_lm


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
def test_example_runs(dtype):
    ex = example()
    model, losses, _ = ex.train(steps=3, tokens=512, vocab=300, dtype=dtype)
    assert np.isfinite(losses).all()
    served = ex.Served(model)
    text = served.generate(7, 5, temperature=0.8, top_k=20, top_p=0.9, min_p=0.01)
    assert len(text) == 6 and all(0 <= t < 300 for t in text)
    assert text == served.generate(7, 5, temperature=0.8, top_k=20, top_p=0.9, min_p=0.01)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_example_gradients(dtype):
    """The model's gradients against torch's in binary64 on the same 16-bit
    weights.  What is rounded to the type on the way: the stream, n and the
    block's output once a layer, h and [dg | du] inside the block, dn and dh once a
    layer, and the gradient itself: with two layers less than 14 roundings of
    half a unit each."""
    ex = example()
    model = ex.Model(vocab=333, width=72, hidden=136, layers=2, dtype=dtype)
    for i in range(3):  # norms of their own
        model.master["norm%d" % i].add_(torch.linspace(-0.3, 0.3, 72, device="cuda"))
    model.refresh()
    g = torch.Generator(device="cuda").manual_seed(5)
    t = torch.randint(0, 333, (300,), generator=g, device="cuda")
    target = torch.randint(0, 333, (300,), generator=g, device="cuda")
    target[::7] = -100
    loss, grads = model.loss_and_grads(t, target)
    p = {k: v.double().requires_grad_() for k, v in model.weights.items()}

    def norm(h, w):
        return h / torch.sqrt((h * h).mean(dim=1, keepdim=True) + ex.EPS) * w
    h = p["embed"][t]
    for i in range(2):
        gate, up = (norm(h, p["norm%d" % i]) @ p["w_in%d" % i]).chunk(2, dim=1)
        h = h + (torch.nn.functional.silu(gate) * up) @ p["w_out%d" % i]
    exact = torch.nn.functional.cross_entropy(norm(h, p["norm2"]) @ p["embed"].t(), target)
    exact.backward()
    u = UNIT[dtype]
    assert abs(float(loss) - float(exact.detach())) <= 14 * u * float(exact.detach())
    assert sorted(grads) == sorted(p)
    for k, v in grads.items():
        err = (v.double() - p[k].grad).norm() / p[k].grad.norm()
        assert float(err) <= 14 * u, (k, float(err))


def decode_parts(dtype, M=3, D=320, F=448, V=5003):
    g = torch.Generator(device="cuda").manual_seed(1)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)
    return {"x": normal(M, D), "r": normal(M, D), "n1": 1 + 0.2 * normal(D), "n2": 1 + 0.2 * normal(D),
            "w": pg.pmx_quantize(normal(F, D, std=D ** -0.5), "e2m1"),
            "v": pg.pmx_quantize(normal(D, F, std=F ** -0.5), "e2m1"),
            "b": normal(F, std=0.1),
            "head": pg.pmx_quantize(normal(V, D, std=3.0 * D ** -0.5), "e2m1"),
            "u": torch.rand(M, generator=g, device="cuda")}


def decode(p):
    """A decoding step: norm, two projections, norm, logits, tokens."""
    h = torch.empty_like(p["x"])
    n = pg.prmsnorm(p["x"], p["n1"], residual=p["r"], h=h, format="e4m3")
    z = pg.pmx_linear(n, p["w"], bias=p["b"], act="silu", dtype=h.dtype)
    y = pg.pmx_linear(z, p["v"], residual=h)
    n = pg.prmsnorm(y, p["n2"], format="e4m3")
    logits = pg.pmx_linear(n, p["head"], dtype=h.dtype)
    return [logits, *pg.psample(logits, p["u"], temperature=0.8, top_k=30, top_p=0.9)]


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("M", [1, 3, 40, 200])
def test_decoding_step(M, dtype):
    """The step against the formulas in binary64, each operator on what the one
    before gave: an 8-bit operand differs from the exact one only where a value
    lies next to a rounding border, so the logits are compared from the operands
    that the kernels made, and these from their inputs by half a step."""
    p = decode_parts(dtype, M)
    u = UNIT[dtype]
    h = torch.empty_like(p["x"])
    n = pg.prmsnorm(p["x"], p["n1"], residual=p["r"], h=h, format="e4m3")
    s = p["x"].double() + p["r"].double()
    want = s / torch.sqrt((s * s).mean(dim=1, keepdim=True) + 1e-6) * p["n1"].double()
    nv = pg.pmx_dequantize(n, dtype=torch.bfloat16).double()  # exact: 4 significant bits
    assert ((nv - want).abs() <= (2.0 ** -4 + 2.0 ** -14) * want.abs() + 2.0 ** -10 * 2.0 ** 2).all()
    assert float((nv - want).norm() / want.norm()) <= 2.0 ** -4
    wv = {k: pg.pmx_dequantize(p[k], dtype=torch.bfloat16).double() for k in ("w", "v", "head")}
    z = pg.pmx_linear(n, p["w"], bias=p["b"], act="silu", dtype=dtype)
    want = torch.nn.functional.silu(nv @ wv["w"].t() + p["b"].double())
    # norm of the error: one rounding, and 2^-14 for the sums and the activation
    assert float((z.double() - want).norm() / want.norm()) <= u + 2.0 ** -14
    y = pg.pmx_linear(z, p["v"], residual=h)
    zv = pg.pmx_dequantize(pg.pmx_quantize(z, "e4m3"), dtype=torch.bfloat16).double()
    want = zv @ wv["v"].t() + h.double()
    assert float((y.double() - want).norm() / want.norm()) <= u + 2.0 ** -14
    n = pg.prmsnorm(y, p["n2"], format="e4m3")
    logits = pg.pmx_linear(n, p["head"], dtype=dtype)
    want = pg.pmx_dequantize(n, dtype=torch.bfloat16).double() @ wv["head"].t()
    assert float((logits.double() - want).norm() / want.norm()) <= u + 2.0 ** -14
    tokens, logprobs = pg.psample(logits, p["u"], temperature=0.8, top_k=30, top_p=0.9)
    got = decode(p)
    assert torch.equal(got[0], logits) and torch.equal(got[1], tokens) and torch.equal(got[2], logprobs)
    top = torch.topk(logits.double(), 31, dim=1).values
    chosen = logits.double().gather(1, tokens[:, None])[:, 0]
    assert (chosen >= top[:, 29]).all() and (logprobs <= 0).all()


@pytest.mark.parametrize("M", [1, 40, 200])
def test_graph_replay(M):
    """A captured decoding step and a captured norm step, replayed several times
    with eager work in between, give the eager results."""
    p = decode_parts(torch.bfloat16, M)
    dy, dh = torch.randn_like(p["x"]), torch.randn_like(p["x"])

    def step():
        h = torch.empty_like(p["x"])
        y = pg.prmsnorm(p["x"], p["n1"], residual=p["r"], h=h)
        back = pg.prmsnorm_bwd(dy, h, p["n1"], dh=dh)
        flat = pg.psample(p["x"], p["u"], top_p=0.9, min_p=0.01)  # without top-k
        return decode(p) + [y, h, *back, *flat]
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for i in range(4):
        p["x"].copy_(torch.randn_like(p["x"]))
        dy.copy_(torch.randn_like(dy))
        p["u"].copy_(torch.rand(M, device="cuda"))
        g.replay()
        torch.cuda.synchronize()
        replayed = [o.clone() for o in out]
        for a, b in zip(replayed, step()):
            assert torch.equal(a, b)
        torch.cuda.synchronize()


def test_two_graphs_share_workspaces():
    """Two captured graphs that were given the same workspaces, replayed in turn."""
    V = 70000
    l = torch.randn(2, V, device="cuda") * 3
    u = torch.rand(2, device="cuda")
    x = torch.randn(100, 600, device="cuda").half()
    w = pg.pmx_quantize(torch.randn(300, 600, device="cuda").half(), "e2m1")
    h, dy = torch.randn(500, 600, device="cuda").half(), torch.randn(500, 600, device="cuda").half()
    n = torch.ones(600, device="cuda").half()
    ws = torch.full((1 << 23,), 0xFF, dtype=torch.uint8, device="cuda")

    def step(k):
        return [*pg.psample(l * (k + 1), u, top_p=0.9, workspace=ws),
                pg.pmx_linear(x, w, format=("e2m1", "e4m3")[k], workspace=ws),
                *pg.prmsnorm_bwd(dy, h, n, eps=0.1 * k, workspace=ws)]
    eager = [step(0), step(1)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for k in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step(k))
        graphs.append(g)
    for _ in range(3):
        for k in (0, 1, 1, 0):
            graphs[k].replay()
            torch.cuda.synchronize()
            for a, b in zip(outs[k], eager[k]):
                assert torch.equal(a, b)


def test_other_stream():
    """Calls on a stream of their own, outputs and workspaces from its pool,
    while the current stream is busy; and two streams at once."""
    p = decode_parts(torch.bfloat16, 70)
    l = torch.randn(5, 60000, device="cuda") * 4
    u = torch.rand(5, device="cuda")
    h, dy = torch.randn(900, 700, device="cuda").half(), torch.randn(900, 700, device="cuda").half()
    n = torch.ones(700, device="cuda").half()

    def calls(s):
        m = pg.prmsnorm(p["x"], p["n1"], format="e2m1", stream=s)
        return [pg.pmx_linear(m, p["w"], bias=p["b"], dtype=torch.bfloat16, stream=s),
                pg.pmx_linear(p["x"], p["w"], stream=s), pg.pmx_dequantize(m, stream=s),
                *pg.psample(l, u, top_k=9, stream=s), *pg.psample(l, u, top_p=0.8, stream=s),
                *pg.prmsnorm_bwd(dy, h, n, stream=s)]
    ref = calls(None)
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    outs = []
    for _ in range(10):
        big = torch.randn(4096, 4096, device="cuda") @ torch.randn(4096, 4096, device="cuda")
        outs += [calls(a), calls(b)]
        del big
    torch.cuda.synchronize()
    for out in outs:
        assert all(torch.equal(x, y) for x, y in zip(out, ref))


def test_same_bits_call_after_call():
    p = decode_parts(torch.float16, 130)
    l = (torch.randn(200, 9000, device="cuda") * 2).half()
    u = torch.rand(200, device="cuda")

    def everything():
        return decode(p) + [*pg.psample(l, u, top_p=0.95), *pg.psample(l[:9], u[:9], top_k=700),
                            *pg.prmsnorm_bwd(l, l, l[0])]
    first = everything()
    for _ in range(3):
        for a, b in zip(first, everything()):
            assert torch.equal(a, b)


def test_rows_stay():
    """Rows and columns behind the outputs, and outputs that another call made, are
    left as they were."""
    x = torch.randn(5, 300, device="cuda").bfloat16()
    w = pg.pmx_quantize(torch.randn(70, 300, device="cuda").bfloat16(), "e2m1")
    for rows in (5, 90, 300):
        big = torch.full((rows + 3, 90), 7.0, dtype=torch.bfloat16, device="cuda")
        xs = x[:1].expand(rows, 300).contiguous()
        pg.pmx_linear(xs, w, out=big[:rows, 8:78])
        assert (big[rows:] == 7).all() and (big[:, :8] == 7).all() and (big[:, 78:] == 7).all()
    y = torch.full((9, 310), 7.0, dtype=torch.bfloat16, device="cuda")
    h = y.clone()
    pg.prmsnorm(x, residual=x, h=h[:5, 3:303], out=y[:5, 3:303])
    dx = y.clone()
    pg.prmsnorm_bwd(x, x, dx=dx[:5, 3:303])
    for t in (y, h, dx):
        assert (t[5:] == 7).all() and (t[:, :3] == 7).all() and (t[:, 303:] == 7).all()


@pytest.mark.parametrize("M,D", [((1 << 22) + 37, 8), ((1 << 20) + 3, 2056), ((1 << 22) + 70000, 128),
                                 ((1 << 18) + 5, 1001)])
def test_more_rows_than_workgroups(M, D):
    """Launches whose workgroups walk the rows: the ends' rows are what they are by
    themselves."""
    print(M, D, flush=True)
    x = torch.randn(M, D, device="cuda", dtype=torch.bfloat16)
    w = torch.randn(D, device="cuda").bfloat16()
    ends = [slice(0, 40), slice(M - 40, M)]
    y = pg.prmsnorm(x, w)
    for e in ends:
        assert torch.equal(y[e], pg.prmsnorm(x[e], w))
    y = pg.pmx_dequantize(pg.prmsnorm(x, w, format="e2m1"))
    for e in ends:
        assert torch.equal(y[e], pg.pmx_dequantize(pg.prmsnorm(x[e], w, format="e2m1")))
    m = pg.pmx_quantize(x, "e4m3")
    y = pg.pmx_dequantize(m)
    for e in ends:
        q = pg.pmx_quantize(x[e], "e4m3")
        assert torch.equal(m.codes[e], q.codes)
        assert torch.equal(y[e], pg.pmx_dequantize(q))
    y, dw = pg.prmsnorm_bwd(x, x, w)
    for e in ends:
        assert torch.equal(y[e], pg.prmsnorm_bwd(x[e], x[e], w, needs=(True, False))[0])
    # dw: n 2^-17 off; up to M / 512 + 512 additions; its rounding
    exact, size = torch.zeros(D, device="cuda").double(), torch.zeros(D, device="cuda").double()
    for r in range(0, M, 1 << 18):
        c = x[r:r + (1 << 18)].double()
        c = c * c / (c.square().mean(dim=1, keepdim=True) + 1e-6).sqrt()
        exact += c.sum(dim=0)
        size += c.abs().sum(dim=0)
    bound = 2.0 ** -8 * exact.abs() + ((M / 512 + 512) * 2.0 ** -24 + 2.0 ** -17) * size
    assert ((dw.double() - exact).abs() <= bound).all()


@pytest.mark.parametrize("V,dtype,k", [(16, torch.float32, 0), (70, torch.float16, 5),
                                       (8192, torch.bfloat16, 600)])
def test_more_sampled_rows_than_workgroups(V, dtype, k):
    M = (1 << 20) + 90
    print(M, V, flush=True)
    l = torch.randn(M, V, device="cuda", dtype=dtype) * 3
    u = torch.rand(M, device="cuda")
    tokens, logprobs = pg.psample(l, u, top_k=k, top_p=0.9)
    for e in (slice(0, 80), slice(M - 80, M)):
        t, p = pg.psample(l[e], u[e], top_k=k, top_p=0.9)
        assert torch.equal(tokens[e], t) and torch.equal(logprobs[e], p)


@pytest.mark.parametrize("by_row", [False, True])
def test_long_rows_of_16_bits_in_a_graph(by_row):
    """Many long rows: replays with other logits in the same places, and another call
    on a second stream meanwhile."""
    M, V = 90, 50000
    l, u = torch.empty(M, V, dtype=torch.bfloat16, device="cuda"), torch.rand(M, device="cuda")
    k = torch.arange(M, dtype=torch.int32, device="cuda") * 9 if by_row else 0
    ls = [(torch.randn(M, V, device="cuda") * s).bfloat16() for s in (3, 0.1, 40)]
    ref = [pg.psample(x, u, top_k=k, top_p=0.9) for x in ls]
    l.copy_(ls[0])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = pg.psample(l, u, top_k=k, top_p=0.9)
    for _ in range(2):
        for x, r in zip(ls, ref):
            l.copy_(x)
            other = pg.psample(ls[1], u, top_k=k, top_p=0.9, stream=s)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out[0], r[0]) and torch.equal(out[1], r[1])
            assert torch.equal(other[0], ref[1][0])


def test_offsets_past_32_bits():
    """Row pitches and row counts whose products pass 2^32 bytes."""
    M, K, pitch = 2100, 200, (1 << 20) + 8
    buf = torch.zeros(M * pitch, dtype=torch.float16, device="cuda")
    x = buf.view(M, pitch)[:, :K]
    y = buf.view(M, pitch)[:, 512:512 + K]
    torch.manual_seed(8)
    x.copy_(torch.randn(M, K, device="cuda"))
    n = torch.randn(K, device="cuda").half()
    ref = pg.prmsnorm(x.contiguous(), n)
    pg.prmsnorm(x, n, out=y)
    assert torch.equal(y, ref)
    got, want = pg.prmsnorm_bwd(y, x, n), pg.prmsnorm_bwd(ref, x.contiguous(), n)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    m, q = pg.pmx_quantize(x, "e4m3"), pg.pmx_quantize(x.contiguous(), "e4m3")
    assert torch.equal(m.codes, q.codes) and torch.equal(m.scales[:, :8], q.scales[:, :8])
    u = torch.rand(M, device="cuda")
    a, b = pg.psample(x, u, top_k=9), pg.psample(x.contiguous(), u, top_k=9)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    a, b = pg.psample(x[-9:], u[-9:], top_p=0.9), pg.psample(x[-9:].contiguous(), u[-9:], top_p=0.9)
    assert torch.equal(a[0], b[0])
    del buf, x, y
    # codes and scales of 2^32 bytes and more
    codes = torch.zeros(2100, 1 << 21, dtype=torch.uint8, device="cuda")
    w = pg.MxMatrix(codes[:, 64:320], q.scales, K, "e4m3")
    w.codes.copy_(q.codes)
    for rows in (3, 100, 2100):
        xs = pg.MxMatrix(q.codes[:rows], q.scales[:rows], K, "e4m3")
        assert torch.equal(pg.pmx_linear(xs, w), pg.pmx_linear(xs, q))
        wide = pg.MxMatrix(w.codes[-rows:], q.scales[-rows:], K, "e4m3")
        near = pg.MxMatrix(q.codes[-rows:], q.scales[-rows:], K, "e4m3")
        assert torch.equal(pg.pmx_linear(wide, q), pg.pmx_linear(near, q))
    assert torch.equal(pg.pmx_dequantize(w), pg.pmx_dequantize(q))


def test_refusals_on_device_tensors():
    x = torch.zeros(4, 64, device="cuda").half()
    w = pg.pmx_quantize(torch.zeros(6, 64, device="cuda").half(), "e2m1")
    m = pg.pmx_quantize(x, "e4m3")
    v = torch.zeros(64, device="cuda").half()
    l, u = torch.zeros(3, 9, device="cuda"), torch.zeros(3, device="cuda")
    for bad in (lambda: pg.prmsnorm(x, v[:63]), lambda: pg.prmsnorm(x, v.float()),
                lambda: pg.prmsnorm(x, residual=x[:3]), lambda: pg.prmsnorm(x, residual=x.bfloat16()),
                lambda: pg.prmsnorm(x.t()), lambda: pg.prmsnorm(x, eps=-1.0),
                lambda: pg.prmsnorm(x, eps=float("nan")), lambda: pg.prmsnorm(x, format="fp4"),
                lambda: pg.prmsnorm(x, format="e2m1", out=m), lambda: pg.prmsnorm(x, out=m),
                lambda: pg.prmsnorm(x, h=x[:, :8]), lambda: pg.prmsnorm(x[:1].expand(4, 64)),
                lambda: pg.prmsnorm_bwd(x, x[:3]), lambda: pg.prmsnorm_bwd(x, x, v, dh=v),
                lambda: pg.prmsnorm_bwd(x, x, v, dweight=v[:3]),
                lambda: pg.pmx_quantize(x, "e4m3", out=w), lambda: pg.pmx_quantize(x.float()),
                lambda: pg.pmx_dequantize(x), lambda: pg.pmx_dequantize(m, dtype=torch.float32),
                lambda: pg.pmx_dequantize(m, out=x[:3]),
                lambda: pg.pmx_linear(x, x), lambda: pg.pmx_linear(x[:, :63], w),
                lambda: pg.pmx_linear(m, w, act="tanh"), lambda: pg.pmx_linear(x, w, format="f8"),
                lambda: pg.pmx_linear(m, w, bias=v), lambda: pg.pmx_linear(m, w, dtype=torch.float32),
                lambda: pg.pmx_linear(x, w, dtype=torch.bfloat16),
                lambda: pg.pmx_linear(m, w, out=x), lambda: pg.pmx_linear(x.float(), w),
                lambda: pg.psample(l, u[:2]), lambda: pg.psample(l, u.half()),
                lambda: pg.psample(l[0], u), lambda: pg.psample(l, u, temperature=-0.5),
                lambda: pg.psample(l, u, temperature=u.double()), lambda: pg.psample(l, u, top_k=-1),
                lambda: pg.psample(l, u, top_k=u), lambda: pg.psample(l, u, top_p=float("nan")),
                lambda: pg.psample(l, u, min_p=1.5), lambda: pg.psample(l[:, :0], u),
                lambda: pg.psample(l, u, tokens=u), lambda: pg.psample(l.long(), u)):
        with pytest.raises((TypeError, ValueError)):
            bad()
    big = torch.randn(30, 3000, device="cuda").half()
    wide = pg.pmx_quantize(torch.zeros(6, 3000, device="cuda").half(), "e2m1")
    for bad in (lambda: pg.prmsnorm(x, v, h=x, out=x),                    # y is h
                lambda: pg.prmsnorm_bwd(x, x, v, dx=x),                   # dx is dy
                lambda: pg.pmx_linear(big, wide, workspace=torch.empty(8, dtype=torch.uint8,
                                                                       device="cuda")),
                lambda: pg.psample(l, u, logprobs=u)):                    # logprobs are u
        with pytest.raises(pg.PgemmError):
            bad()
    # formats of other types that hold bytes
    q = pg.MxMatrix(m.codes.view(torch.float8_e4m3fn), m.scales.view(torch.float8_e8m0fnu), 64, "e4m3")
    assert torch.equal(pg.pmx_dequantize(q), pg.pmx_dequantize(m))
