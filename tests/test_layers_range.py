"""The layer operators at the ends of their types' ranges: pre-activations that
overflow, infinities, NaN and tails, against the formulas in binary64.

Tolerances, derived before the first run: u is the output type's rounding
(2^-11 for float16, 2^-8 for bfloat16); a value that passes through one 16-bit
intermediate carries 2 u; the activations' few fp32 roundings and their
exponential and reciprocal (1 ulp each) are below 2^-19 of the value where its
argument is of ordinary size."""
import numpy as np
import pytest

import software_pipelined_tiled_pgemm_amd as pg

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

UNIT = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -126}
DTYPES = [torch.float16, torch.bfloat16]
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
E32 = 2.0 ** -23
inf, nan = float("inf"), float("nan")


def value(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return torch.where(z == -inf, 0.0, z * torch.special.ndtr(z))
    if act == "gelu_tanh":
        return torch.where(z < -1e3, 0.0, z * torch.sigmoid(2 * (2 / np.pi) ** 0.5 * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return torch.where(z == -inf, 0.0, z * torch.sigmoid(z))
    return z


def slope(z, act):
    far = z.clamp(-1e3, 1e3)
    if act == "relu":
        return (z > 0).double()
    if act == "gelu":
        return torch.special.ndtr(z) + far * torch.exp(-far * far / 2) / (2 * np.pi) ** 0.5
    if act == "gelu_tanh":
        c = (2 / np.pi) ** 0.5
        s = torch.sigmoid(2 * c * (far + 0.044715 * far ** 3))
        return s + far * s * (1 - s) * 2 * c * (1 + 3 * 0.044715 * far * far)
    if act == "silu":
        s = torch.sigmoid(far)
        return s * (1 + far * (1 - s))
    return torch.ones_like(z)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ACTS)
def test_linear_gradient_at_the_ends(act, dtype):
    top = float(torch.finfo(dtype).max)
    z = torch.tensor([[-inf, -top, -1e4, -100.0, -30.0, -12.0, -0.0, 0.0, 12.0, 30.0, 100.0, 1e4, top, inf]],
                     dtype=torch.float64).to(dtype).cuda()
    n = z.shape[1]
    x, w = torch.ones((1, 1), dtype=dtype, device="cuda"), torch.ones((1, n), dtype=dtype, device="cuda")
    dy = torch.full((1, n), 3.0, dtype=dtype, device="cuda")
    dx, dw, db = pg.plinear_bwd(dy, x, w, preact=z, act=act)
    exact = 3.0 * slope(z.double(), act)[0]
    tol = UNIT[dtype] * exact.abs() + 2.0 ** -19 * exact.abs() + 1e-6
    assert bool(((db.double() - exact).abs() <= tol).all()), (db, exact)
    assert bool(((dw[0].double() - exact).abs() <= 2 * tol).all())
    assert bool(torch.isfinite(dx).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_linear_gradient_of_nan(act, dtype):
    z = torch.tensor([[1.0, nan, -2.0]], dtype=dtype, device="cuda")
    one = torch.ones((1, 1), dtype=dtype, device="cuda")
    db = pg.plinear_bwd(torch.ones_like(z), one, torch.ones_like(z), preact=z, act=act)[2]
    assert torch.isnan(db).tolist() == [False, True, False]


@pytest.mark.parametrize("act", ACTS)
def test_linear_step_that_overflows_its_preact(act):
    x = torch.tensor([[300.0, 1.0], [1.0, 1.0]], device="cuda").half()
    w = torch.tensor([[300.0, -300.0, 1.0], [0.5, 0.25, -1.0]], device="cuda").half()
    z = torch.empty((2, 3), dtype=torch.float16, device="cuda")
    pg.plinear(x, w, act=act, preact=z)
    assert torch.isinf(z[0, :2]).all()
    dy = torch.tensor([[0.5, 0.25, 1.0], [1.0, 2.0, 0.5]], device="cuda").half()
    got = pg.plinear_bwd(dy, x, w, preact=z, act=act)
    X, W, DY = x.double(), w.double(), dy.double()
    DZ = DY * slope(X @ W, act)
    for g, e, s in zip(got, (DZ @ W.t(), X.t() @ DZ, DZ.sum(0)),
                       (DZ.abs() @ W.abs().t(), X.t() @ DZ.abs(), DZ.abs().sum(0))):
        assert bool(((g.double() - e).abs() <= 2.0 ** -10 * s + 1e-6).all()), (g, e)


@pytest.mark.parametrize("act", ["relu", "gelu", "gelu_tanh", "silu"])
def test_ffn_gate_below_the_range(act):
    """A gate of -90000, which float16 keeps as -inf: the forward pass's h is 0
    there, and so are the gradients of that row."""
    x = torch.tensor([[300.0], [1.0]], device="cuda").half()
    wi = torch.tensor([[-300.0, 0.01]], device="cuda").half()
    wo = torch.tensor([[0.5]], device="cuda").half()
    gu = torch.empty((2, 2), dtype=torch.float16, device="cuda")
    y = pg.pffn(x, wi, wo, act=act, gate_up=gu)
    assert bool(torch.isfinite(y).all()) and float(gu[0, 0]) == -inf
    dy = torch.tensor([[2.0], [0.0]], device="cuda").half()
    for grad in pg.pffn_bwd(dy, x, wi, wo, gu, act=act):
        assert not bool(grad.any()) and bool(torch.isfinite(grad).all())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("F", [1, 8])
def test_ffn_infinite_rows(F, dtype):
    """An infinite row of x or dy gives the formula's infinities, also where F
    is padded to whole 16-byte pieces."""
    x = torch.tensor([[inf], [1.0]], dtype=dtype, device="cuda")
    wi = torch.ones((1, 2 * F), dtype=dtype, device="cuda")
    wo = torch.full((F, 1), 2.0, dtype=dtype, device="cuda")
    assert pg.pffn(x, wi, wo, act="relu").tolist() == [[inf], [2.0 * F]]
    one = torch.ones((2, 1), dtype=dtype, device="cuda")
    gu = torch.empty((2, 2 * F), dtype=dtype, device="cuda")
    pg.pffn(one, wi, wo, act="relu", gate_up=gu)
    dx, dwi, dwo = pg.pffn_bwd(x, one, wi, wo, gu, act="relu")
    assert dx.tolist() == [[inf], [4.0 * F]]
    assert dwi.tolist() == [[inf] * (2 * F)] and dwo.tolist() == [[inf]] * F


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("F", [0, 6, 24])
def test_ffn_without_outputs(F, dtype):
    """N = 0: gate_up is written all the same, and the gradients are 0."""
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn(5, 8, generator=g, device="cuda").to(dtype)
    wi = torch.randn(8, 2 * F, generator=g, device="cuda").to(dtype)
    wo = torch.empty((F, 0), dtype=dtype, device="cuda")
    gu = torch.full((5, 2 * F), nan, dtype=dtype, device="cuda")
    y = pg.pffn(x, wi, wo, gate_up=gu)
    assert y.shape == (5, 0)
    full = torch.full((5, 2 * F), nan, dtype=dtype, device="cuda")
    pg.pffn(x, wi, torch.ones((F, 3), dtype=dtype, device="cuda"), gate_up=full)
    assert torch.equal(gu.view(torch.int16), full.view(torch.int16))
    assert not bool(torch.isnan(gu).any())
    dx, dwi, dwo = pg.pffn_bwd(torch.empty((5, 0), dtype=dtype, device="cuda"), x, wi, wo, gu)
    assert not bool(dx.any()) and not bool(dwi.any()) and dwo.shape == (F, 0)


@pytest.mark.parametrize("dtype", DTYPES)
def test_gelu_tail(dtype):
    """z Phi(z) and its derivative to one rounding of the type down the tail: the
    fp32 evaluation adds 2^-19 and, by the rounded argument of exp(-z^2 / 2), z^2
    2^-22 of the value (of each term of the derivative)."""
    z = torch.linspace(-13.0, 6.0, 3001, dtype=torch.float64).to(dtype).cuda()[None]
    n = z.shape[1]
    one = torch.ones((1, 1), dtype=dtype, device="cuda")
    y = pg.plinear(one, z, act="gelu")
    Z = z.double()
    rel = UNIT[dtype] + 2.0 ** -19 + Z * Z * 2.0 ** -22
    cdf = torch.special.erfc(-Z.cpu() * 0.5 ** 0.5).cuda() / 2   # (ndtr cancels in the tail)
    E = Z * cdf
    ratio = ((y.double() - E).abs() - TINY[dtype]) / (rel * E.abs() + 1e-300)
    assert float(ratio.max()) <= 1, (float(ratio.max()), float(Z[0, int(ratio.argmax())]))
    db = pg.plinear_bwd(torch.ones_like(z), one, torch.ones_like(z), preact=z, act="gelu")[2]
    a, b = cdf, Z * torch.exp(-Z * Z / 2) / (2 * np.pi) ** 0.5
    tol = UNIT[dtype] * (a + b).abs() + (rel - UNIT[dtype]) * (a + b.abs()) + TINY[dtype]
    assert bool(((db.double() - (a + b)[0]).abs() <= tol[0]).all())


# (M, D, F, N): an edge, whole and broken 16-byte rows, a split contraction
# (dh through the finish kernel), whole 128x128 and 256x256 tiles
BEYOND = [(3, 16, 5, 4), (70, 40, 136, 72), (130, 72, 129, 600), (256, 64, 256, 64),
          (4096, 64, 4096, 128)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("shape", BEYOND)
def test_ffn_gradients_beyond_the_kept_range(shape, act, dtype):
    """Columns of g and u whose values the 16 bits that they are kept in do not
    hold (fp16: beyond 65504; bf16: beyond 2^33 and below 2^-30), in a block
    whose activations and gradients are of ordinary size: gate column c is scaled by
    a, up column c by b and row c of W_out by 1 / (a b).

    Bound: a kept value carries its rounding (2^-11, for bf16 2^-10, fp16
    subnormals 2^-25) and the fp32 sum's error, a value computed again the
    latter; |act'| and |act''| are at most 1.13; relu' may differ where |g| is
    below its error.  Entries of [dg | du] and h are rounded once (u, subnormals
    TINY)."""
    M, D, F, N = shape
    print("beyond", shape, act, dtype, flush=True)
    g = torch.Generator(device="cuda").manual_seed(7)

    def rnd(*s):
        return torch.randn(*s, generator=g, device="cuda", dtype=torch.float64)
    x = rnd(M, D).to(dtype)
    x[M // 2] = 0.0  # g and u of exactly 0
    a, b = (torch.ones(F, dtype=torch.float64, device="cuda") for _ in range(2))
    if dtype is torch.float16:
        a[1::5], b[1::5], a[3::5], b[3::5] = 5e4, 1e-2, 1e-2, 5e4
    else:
        a[1::5], b[1::5], a[3::5], b[3::5], a[4::5] = 1e14, 1e-13, 1e-20, 1e16, 1e-12
    wi = (rnd(D, 2 * F) * D ** -0.5 * torch.cat([a, b])).to(dtype)
    wo = (rnd(F, N) * F ** -0.5 / (a * b)[:, None]).to(dtype)
    dy = rnd(M, N).to(dtype)
    gu = torch.empty((M, 2 * F), dtype=dtype, device="cuda")
    y = pg.pffn(x, wi, wo, act=act, gate_up=gu)
    assert bool(torch.isfinite(y).all())
    dx, dwi, dwo = pg.pffn_bwd(dy, x, wi, wo, gu, act=act)

    X, WI, WO, DY = x.double(), wi.double(), wo.double(), dy.double()
    Z, S = X @ WI, X.abs() @ WI.abs()
    u, tiny = UNIT[dtype], TINY[dtype]
    KU = u if dtype is torch.float16 else u / 4
    E = KU * Z.abs() + (D + 16) * E32 * S + (2.0 ** -25 if dtype is torch.float16 else 0.0)
    if dtype is torch.float16:
        assert int((Z.abs() > 65520).sum()) > 0
    else:
        assert int((Z.abs() > 2.0 ** 34).sum()) > 0 and int((Z.abs() < 2.0 ** -31).sum()) > F
    G, U, EG, EU = Z[:, :F], Z[:, F:], E[:, :F], E[:, F:]
    DH = DY @ WO.t()
    EDH = (N + 17) * E32 * (DY.abs() @ WO.abs().t())
    A, P = value(G, act), slope(G, act)
    DIN = torch.cat([DH * U * P, DH * A], 1)
    H = A * U
    unsure = (G.abs() <= EG) * (DH * U).abs() if act == "relu" else 0.0
    # the activations' own fp32 evaluation: 1e-6 of their argument
    EDIN = torch.cat([1.13 * (EDH * U.abs() + DH.abs() * (EU + U.abs() * EG)) + unsure + 1e-6 * (DH * U).abs(),
                      EDH * A.abs() + DH.abs() * (1.13 * EG + 1e-6 * G.abs())], 1)
    EH = A.abs() * EU + U.abs() * (1.13 * EG + 1e-6 * G.abs())
    EDIN = 1.01 * EDIN + u * DIN.abs() + tiny
    EH = 1.01 * EH + u * H.abs() + tiny
    for name, got, exact, err, scale, n in (
            ("dx", dx, DIN @ WI.t(), EDIN @ WI.abs().t(), DIN.abs() @ WI.abs().t(), 2 * F),
            ("dw_in", dwi, X.t() @ DIN, X.abs().t() @ EDIN, X.abs().t() @ DIN.abs(), M),
            ("dw_out", dwo, H.t() @ DY, EH.t() @ DY.abs(), H.abs().t() @ DY.abs(), M)):
        bound = u * exact.abs() + 1.01 * err + (n + 16) * E32 * scale + tiny
        bad = ~((got.double() - exact).abs() <= bound)
        # sums beyond the output type's own range are its infinity
        bad &= ~((exact.abs() + bound > torch.finfo(dtype).max) & (got == exact.sign() * inf))
        assert not bool(bad.any()), (name, int(bad.sum()), got[bad][:4], exact[bad][:4], bound[bad][:4])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("M,F", [(70, 51), (256, 256)])
def test_ffn_gradients_keep_nan(M, F, dtype):
    """A NaN row of x: its own row of dx is NaN, the others keep their bits."""
    g = torch.Generator(device="cuda").manual_seed(8)
    x = torch.randn(M, 40, generator=g, device="cuda").to(dtype)
    wi = torch.randn(40, 2 * F, generator=g, device="cuda").mul(0.16).to(dtype)
    wo = torch.randn(F, 24, generator=g, device="cuda").mul(0.1).to(dtype)
    dy = torch.randn(M, 24, generator=g, device="cuda").to(dtype)
    gu = torch.empty((M, 2 * F), dtype=dtype, device="cuda")
    pg.pffn(x, wi, wo, gate_up=gu)
    ref = pg.pffn_bwd(dy, x, wi, wo, gu)[0]
    x[5] = nan
    pg.pffn(x, wi, wo, gate_up=gu)
    dx, dwi, dwo = pg.pffn_bwd(dy, x, wi, wo, gu)
    assert bool(torch.isnan(dx[5]).all()) and bool(torch.isnan(dwi).all()) and bool(torch.isnan(dwo).all())
    dx[5] = ref[5]
    assert torch.equal(dx, ref)


def test_ffn_kept_codes():
    """bf16's kept form: gradual underflow below 2^-30, nothing but 0 becomes 0,
    and without x the topmost code stands for NaN."""
    v = [0.0, 2.0 ** -30, 2.0 ** -31, -(2.0 ** -33), 2.0 ** -39, 1e-30, -1e-37, 2.0 ** 34, -1e38, inf, nan, 1.0]
    w = torch.tensor([v + v], dtype=torch.float64).to(torch.bfloat16).cuda()
    one = torch.ones((1, 1), dtype=torch.bfloat16, device="cuda")
    wo = torch.ones((12, 1), dtype=torch.bfloat16, device="cuda")
    gu = torch.empty((1, 24), dtype=torch.bfloat16, device="cuda")
    pg.pffn(one, w, wo, gate_up=gu)
    codes = [c & 0xFFFF for c in gu.view(torch.int16)[0, :12].tolist()]
    assert codes[:7] == [0, 1 << 9, 1 << 8, 0x8000 | 1 << 6, 1, 1, 0x8001]
    assert all(c & 0x7FFF == 0x7FFF for c in codes[7:11]) and codes[11] == 31 << 9

    # dW_out = h^T dy alone, without x: act "none", h = g u
    L = pg.lib()
    dwo = torch.empty((12, 1), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    for x in (None, one.data_ptr()):
        rc = L.pffn_bwd(1, one.data_ptr(), 1, x, 1, w.data_ptr(), 24, wo.data_ptr(), 1, gu.data_ptr(), 24,
                        None, 0, None, 0, None, 0, dwo.data_ptr(), 1, 1, 1, 12, 1, 0, ws.data_ptr(),
                        ws.numel(), torch.cuda.current_stream().cuda_stream)
        assert rc == pg.PGEMM_OK
        got = dwo.double().cpu()[:, 0]
        exact = w[0, :12].double().cpu() ** 2
        if x is None:
            assert torch.isnan(got[7:11]).all()
            assert bool(((got - exact)[:7].abs() <= 2.0 ** -8 * exact[:7] + 2.0 ** -78).all())
        else:
            assert float(got[7]) == 2.0 ** 68 and got[8] == inf and got[9] == inf and torch.isnan(got[10])
            fits = exact > 2.0 ** -126   # (-1e-37 squared is below the type's range)
            fits[7:] = False
            assert bool(((got - exact).abs() <= 2.0 ** -8 * exact)[fits].all())


def test_gate_up_as_int16():
    """bfloat16's kept form in an int16 tensor: the same bits and gradients;
    float16 keeps its values in float16 alone."""
    g = torch.Generator(device="cuda").manual_seed(10)
    x, wi, wo = (torch.randn(*s, generator=g, device="cuda").bfloat16() for s in ((9, 8), (8, 12), (6, 4)))
    kept = [torch.empty((9, 12), dtype=t, device="cuda") for t in (torch.bfloat16, torch.int16)]
    for gu in kept:
        pg.pffn(x, wi, wo, gate_up=gu)
    assert torch.equal(kept[0].view(torch.int16), kept[1])
    dy = torch.randn(9, 4, generator=g, device="cuda").bfloat16()
    for a, b in zip(*(pg.pffn_bwd(dy, x, wi, wo, gu) for gu in kept)):
        assert torch.equal(a, b)
    for bad in (torch.float16, torch.float32, torch.int32):
        with pytest.raises(TypeError):
            pg.pffn(x, wi, wo, gate_up=torch.empty((9, 12), dtype=bad, device="cuda"))
        with pytest.raises(TypeError):
            pg.pffn_bwd(dy, x, wi, wo, torch.empty((9, 12), dtype=bad, device="cuda"))
    with pytest.raises(TypeError):
        pg.pffn(x.half(), wi.half(), wo.half(), gate_up=kept[1])


@pytest.mark.parametrize("V", [3, 300])
def test_xent_at_the_ends_of_fp32(V):
    """Logits of bfloat16's lowest and largest values: a row of nothing but the
    lowest, one with a single ordinary entry, one with the largest; lse to fp32's
    rounding (log V is far below it at 3e38)."""
    top = float(torch.finfo(torch.bfloat16).max)
    w = torch.ones((V, 3), dtype=torch.float64)
    w[1, 1], w[2, 2] = 0.0, 0.5
    w = w.to(torch.bfloat16).cuda()
    x = torch.tensor([[-top, 0, 0], [0, -top, 0], [0, 0, top]], dtype=torch.float64).to(torch.bfloat16).cuda()
    t = torch.tensor([0, 1, 2], device="cuda")
    loss, lse = pg.pxent(x, w, t, reduction="none")
    logits = x.double() @ w.double().t()
    exact = torch.logsumexp(logits, 1)
    assert bool(((lse.double() - exact).abs() <= 2.0 ** -22 * exact.abs()).all()), (lse, exact)
    each = exact - logits[torch.arange(3), t.cpu()]
    assert bool(((loss.double() - each).abs() <= 2.0 ** -22 * (exact.abs() + each.abs())).all())
