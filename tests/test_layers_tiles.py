"""The layer operators at sizes whose products take 256x256 tiles: contractions
of several passes of the 5-step ring (704 = 22 steps of 32 and more), in the
three operand layouts, whole tiles and edges, with and without a K split, and
the statistics of the cross entropy with workgroups that walk several tiles.
Each test first asserts, with the library's own rule, that its products take
the tiles that it is about.

The reference is binary64 on the device.  Tolerances, derived before the first
run: u is the output type's rounding (2^-11 for float16, 2^-8 for bfloat16);
an output that is a sum of terms t_i with at most c stored 16-bit roundings in
each satisfies |got - exact| <= u |exact| + c u sum|t_i| + (n + 16) 2^-23 sum|t_i| +
tiny, n being the length of the sum, the third part fp32 accumulation in any
order with the activations' fp32 roundings."""
import ctypes

import pytest

import software_pipelined_tiled_pgemm_amd as pg

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

UNIT = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -126}
DTYPES = [torch.float16, torch.bfloat16]
E32 = 2.0 ** -23


class Cut(ctypes.Structure):
    _fields_ = [("big", ctypes.c_bool), ("splits", ctypes.c_int), ("chunk", ctypes.c_int64)]


def cut(M, N, K, most=16):
    """(256x256 tiles, K splits) of a product, by the library's rule."""
    f = pg.lib()._ZN5pgemm5layer10choose_cutElllii
    f.restype, f.argtypes = Cut, [ctypes.c_int64] * 3 + [ctypes.c_int] * 2
    c = f(M, N, K, torch.cuda.get_device_properties(0).multi_processor_count, most)
    return c.big, c.splits


def rand(shape, dtype, seed, std=1.0, pad=0):
    """Normal values; with `pad`, rows that lie pad elements apart, NaN between."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    v = (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)
    if not pad:
        return v
    view = gaps(shape, dtype, pad)
    view.copy_(v)
    return view


def gaps(shape, dtype, pad):
    """An uninitialised (NaN) matrix of rows pad elements apart."""
    r, c = shape
    return torch.full((r, c + pad), float("nan"), dtype=dtype, device="cuda")[:, :c]


def gaps_kept(t):
    r, c = t.shape
    ld = t.stride(0)
    whole = torch.as_strided(t, (r, ld), (ld, 1), t.storage_offset())
    return bool(torch.isnan(whole[:, c:]).all())


def near(got, exact, scale, n, c, what):
    u = UNIT[got.dtype]
    g = got.double()
    bound = u * exact.abs() + (c * u + (n + 16) * E32) * scale + TINY[got.dtype]
    bad = ~((g - exact).abs() <= bound)
    if bool(bad.any()):
        i = tuple(int(v) for v in bad.nonzero()[0])
        pytest.fail("%s: %d of %d outside; first %s: got %r, exact %r, bound %r" % (
            what, int(bad.sum()), bad.numel(), i, float(g[i]), float(exact[i]), float(bound[i])))


def silu(z):
    return z * torch.sigmoid(z)


def silu_grad(z):
    p = torch.sigmoid(z)
    return p * (1 + z * (1 - p))


def say(*a):
    print(*a, flush=True)


# (M, N, K), elements between rows: whole tiles, edges with odd rows, a split contraction
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape,splits,pad", [
    ((4096, 4096, 704), 1, 0), ((4096, 4096, 704), 1, 8), ((4093, 4100, 701), 1, 0),
    ((4093, 4096, 712), 1, 3), ((2304, 2304, 4096), 3, 0), ((2300, 2310, 4100), 2, 5)])
def test_linear_forward(shape, splits, pad, dtype):
    M, N, K = shape
    assert cut(M, N, K) == (True, splits)
    say("linear", shape, splits, pad, dtype)
    x, w = rand((M, K), dtype, 1, pad=pad), rand((K, N), dtype, 2, std=K ** -0.5, pad=pad)
    b, r = rand((N,), dtype, 3, std=0.3), rand((M, N), dtype, 4, pad=pad)
    z, y = gaps((M, N), dtype, pad), gaps((M, N), dtype, pad)
    pg.plinear(x, w, bias=b, residual=r, act="silu", preact=z, out=y)
    X, W, B, R = x.double(), w.double(), b.double(), r.double()
    Z = X @ W + B
    S = X.abs() @ W.abs() + B.abs()
    near(z, Z, S, K, 0, "preact")
    near(y, silu(Z) + R, 1.2 * S + R.abs(), K, 0, "y")  # |silu'| < 1.1
    assert gaps_kept(z) and gaps_kept(y)
    again = pg.plinear(x, w, bias=b, residual=r, act="silu")
    assert torch.equal(again, y)


# (M, N, K), splits of dx (NT) and dw (TN)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape,splits,pad", [
    ((4096, 3840, 2304), (1, 1), 0), ((4096, 3840, 2304), (1, 1), 8),
    ((2300, 4100, 2310), (2, 1), 0), ((2300, 4100, 2310), (2, 1), 3),
    ((2304, 4096, 2304), (3, 1), 0)])
def test_linear_backward(shape, splits, pad, dtype):
    M, N, K = shape
    assert cut(M, K, N) == (True, splits[0]) and cut(K, N, M) == (True, splits[1])
    say("linear backward", shape, splits, pad, dtype)
    x, w = rand((M, K), dtype, 11, pad=pad), rand((K, N), dtype, 12, std=K ** -0.5, pad=pad)
    z, dy = rand((M, N), dtype, 13, pad=pad), rand((M, N), dtype, 14, pad=pad)
    a = rand((M, K), dtype, 15, pad=pad)
    dx, dw = gaps((M, K), dtype, pad), gaps((K, N), dtype, pad)
    db = pg.plinear_bwd(dy, x, w, preact=z, act="silu", dx_residual=a, dx=dx, dw=dw)[2]
    X, W, A, DY = x.double(), w.double(), a.double(), dy.double()
    DZ, mag = DY * silu_grad(z.double()), DY.abs() * 1.1
    near(dx, DZ @ W.t() + A, mag @ W.abs().t() + A.abs(), N, 1, "dx")
    near(dw, X.t() @ DZ, X.abs().t() @ mag, M, 1, "dw")
    near(db, DZ.sum(0), mag.sum(0), M, 0, "dbias")
    assert gaps_kept(dx) and gaps_kept(dw)
    again = pg.plinear_bwd(dy, x, w, preact=z, act="silu", dx_residual=a)
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw) and torch.equal(again[2], db)


def kept(t):
    """The values that pffn kept in gate_up: float16 as they are, for bfloat16
    1 sign, 6 exponent (bias 31) and 9 fraction bits."""
    if t.dtype is torch.float16:
        return t.double()
    c = t.contiguous().view(torch.int16).long() & 0xFFFF
    v = torch.ldexp(1.0 + (c & 511).double() / 512.0, ((c >> 9) & 63) - 31)
    v = torch.where((c >> 9) & 63 > 0, v, torch.zeros_like(v))
    return torch.where(c >> 15 != 0, -v, v)


# (M, D, F, N), cuts of the projections, dh, dx and dw_in (None: not the test's concern)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape,splits,pad", [
    ((4096, 704, 4096, 704), (1, 1, 4, 2), 0), ((4096, 704, 4096, 704), (1, 1, 4, 2), 8),
    ((4093, 701, 4100, 700), (1, 1, 4, 2), 0), ((4093, 704, 4097, 704), (1, 1, 4, 2), 3),
    ((2304, 4096, 1152, 704), (3, None, None, 1), 0), ((2304, 704, 2304, 4096), (None, 3, None, None), 0)])
def test_ffn(shape, splits, pad, dtype):
    M, D, F, N = shape
    f8 = (F + 7) // 8 * 8
    for s, c in zip(splits, ((M, 2 * f8, D), (M, F, N), (M, D, 2 * f8), (D, 2 * f8, M))):
        assert s is None or cut(*c) == (True, s)
    say("ffn", shape, splits, pad, dtype)
    x = rand((M, D), dtype, 31, pad=pad)
    wi = rand((D, 2 * F), dtype, 32, std=D ** -0.5, pad=pad)
    wo = rand((F, N), dtype, 33, std=F ** -0.5, pad=pad)
    r, gu, y = rand((M, N), dtype, 34, pad=pad), gaps((M, 2 * F), dtype, pad), gaps((M, N), dtype, pad)
    pg.pffn(x, wi, wo, residual=r, act="silu", gate_up=gu, out=y)
    X, WI, WO, R = x.double(), wi.double(), wo.double(), r.double()
    Z, S = X @ WI, X.abs() @ WI.abs()
    u = UNIT[dtype]
    KU = u / (1 if dtype is torch.float16 else 4)  # the kept form's rounding
    GU = kept(gu)
    tol = KU * Z.abs() + (D + 16) * E32 * S + 2.0 ** -24
    assert bool(((GU - Z).abs() <= tol).all())
    A, H = silu(Z[:, :F]), silu(Z[:, :F]) * Z[:, F:]
    HE = (D + 16) * E32 * 1.2 * (S[:, :F] * Z[:, F:].abs() + A.abs() * S[:, F:])
    Y = H @ WO + R
    tol = (u * Y.abs() + (u + (F + 16) * E32) * (H.abs() @ WO.abs() + R.abs())
           + 1.01 * (HE @ WO.abs()) + TINY[dtype] * (1 + WO.abs().sum(0)))
    assert bool(((y.double() - Y).abs() <= tol).all())
    assert gaps_kept(y)

    dy, a = rand((M, N), dtype, 35, pad=pad), rand((M, D), dtype, 36, pad=pad)
    dx, dwi, dwo = gaps((M, D), dtype, pad), gaps((D, 2 * F), dtype, pad), gaps((F, N), dtype, pad)
    pg.pffn_bwd(dy, x, wi, wo, gu, act="silu", dx_residual=a, dx=dx, dw_in=dwi, dw_out=dwo)
    DY, G, U = dy.double(), GU[:, :F], GU[:, F:]
    DH, DHS = DY @ WO.t(), DY.abs() @ WO.abs().t()
    AG, DG = silu(G), silu_grad(G)
    DIN = torch.cat([DH * U * DG, DH * AG], dim=1)
    # the rounding of an entry, and dh's fp32 accumulation where it cancels
    mag = DIN.abs() + 2 * (N + 17) * E32 / u * torch.cat(
        [DHS * U.abs() * 1.2, DHS * (AG.abs() + 1e-6 * G.abs())], dim=1)
    A = a.double()
    near(dx, DIN @ WI.t() + A, mag @ WI.abs().t() + A.abs(), 2 * F, 1, "dx")
    near(dwi, X.t() @ DIN, X.abs().t() @ mag, M, 1, "dw_in")
    near(dwo, (AG * U).t() @ DY, (AG.abs() * U.abs() * 1.0001 + 1e-6 * (G * U).abs()).t() @ DY.abs(),
         M, 1, "dw_out")
    assert gaps_kept(dx) and gaps_kept(dwi) and gaps_kept(dwo)
    again = pg.pffn_bwd(dy, x, wi, wo, gu, act="silu", dx_residual=a)
    assert all(torch.equal(p, q) for p, q in zip(again, (dx, dwi, dwo)))
    assert torch.equal(pg.pffn(x, wi, wo, residual=r, act="silu"), y)


# (M, D, V), pieces of the backward pass, whether its dx and dw take 256x256 tiles
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape,pieces,grads,pad", [
    ((4093, 168, 5003), 1, False, 0),   # 320 tiles: workgroups walk
    ((4096, 704, 4864), 1, False, 0),   # 304 whole tiles
    ((4001, 2300, 4099), 1, True, 0), ((4096, 2304, 4352), 1, True, 8),
    ((33000, 520, 9000), 2, True, 0)])
def test_xent(shape, pieces, grads, pad, dtype):
    M, D, V = shape
    step = V if pieces == 1 else -(-V // pieces // 256) * 256
    assert cut(M, V, D, 1)[0] and cut(M, step, D)[0] and -(-V // step) == pieces
    assert not grads or (cut(M, D, step)[0] and cut(step, D, M)[0])
    say("xent", shape, pieces, pad, dtype)
    x, w = rand((M, D), dtype, 51, pad=pad), rand((V, D), dtype, 52, std=2 * D ** -0.5, pad=pad)
    g = torch.Generator(device="cuda").manual_seed(53)
    t = torch.randint(0, V, (M,), generator=g, device="cuda")
    t[torch.rand(M, generator=g, device="cuda") < 0.2] = -100
    loss, lse = pg.pxent(x, w, t, reduction="none")
    X, W = x.double(), w.double()
    L = X @ W.t()
    LSE = torch.logsumexp(L, 1)
    S = (X.abs() @ W.abs().t()).amax(1)
    # a logit's fp32 accumulation, exp and log of fp32 values near |lse|
    e = (D + 8) * E32 * S + 16 * E32 * (LSE.abs() + 1)
    assert bool(((lse.double() - LSE).abs() <= e).all())
    valid = t >= 0
    at = t.clamp(min=0)
    rows = torch.arange(M, device="cuda")
    EACH = torch.where(valid, LSE - L[rows, at], torch.zeros_like(LSE))
    assert bool(((loss.double() - EACH).abs() <= 2 * e * valid + E32 * EACH.abs()).all())
    mean = pg.pxent(x, w, t)[0]
    n = int(valid.sum())
    assert abs(float(mean) - float(EACH.sum()) / n) <= float((2 * e * valid).sum() + 2 * E32 * EACH.sum()) / n
    again = pg.pxent(x, w, t, reduction="none")
    assert torch.equal(again[0], loss) and torch.equal(again[1], lse)

    dx, dw = gaps((M, D), dtype, pad), gaps((V, D), dtype, pad)
    pg.pxent_bwd(x, w, t, lse, reduction="sum", dx=dx, dw=dw)
    u = UNIT[dtype]
    P = torch.exp(L - LSE[:, None]) * valid[:, None]
    # dl: one rounding; the error of the logit and of lse in the exponent; in
    # float16 the subnormals of dl scaled by 2^15
    mag = P * (2 * e[:, None] + 8 * E32 * (1 + (L - LSE[:, None]).abs())) / u
    del L
    P[rows, at] -= valid.double()
    mag += P.abs()
    if dtype is torch.float16:
        mag += valid[:, None] * 2.0 ** -39 / u
    near(dx, P @ W, mag @ W.abs(), V, 1, "dx")
    near(dw, P.t() @ X, mag.t() @ X.abs(), M, 1, "dw")
    assert gaps_kept(dx) and gaps_kept(dw) and not bool(dx[~valid].any())
    again = pg.pxent_bwd(x, w, t, lse, reduction="sum")
    assert torch.equal(again[0], dx) and torch.equal(again[1], dw)
