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
