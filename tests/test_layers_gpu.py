"""The layer operators on the GPU against plain formulas in binary64 on the
CPU (numpy), written apart from the kernels.

Tolerances, derived before the first run.  u is the output type's rounding
(2^-11 for float16, 2^-8 for bfloat16: half an ulp relative to the value), and
a stored intermediate adds another rounding of the same relative size to each
term that it enters.  For an output that is a sum of terms t_i, each carrying
relative errors of at most c roundings, |got - exact| <= u |exact| + c u sum|t_i|
+ (n + 16) 2^-23 sum|t_i| + tiny, where the third part is fp32 accumulation
over n terms in any order with the activations' few fp32 roundings, and tiny
covers the type's subnormals.  Each test states its c (0 where no intermediate
is rounded)."""
import sys

import numpy as np
import pytest

import software_pipelined_tiled_pgemm_amd as pg

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

UNIT = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -126}
DTYPES = [torch.float16, torch.bfloat16]
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def rand(shape, dtype, seed, std=1.0, pitch=None, offset=0):
    """Normal values of the type on the device, rows `pitch` apart (default:
    dense), the first one `offset` elements into its buffer; the gaps hold
    NaN."""
    rng = np.random.default_rng(seed)
    v = torch.from_numpy(rng.normal(0.0, std, size=shape)).to(dtype)
    if pitch is None and offset == 0:
        return v.cuda()
    r, c = shape
    pitch = pitch or c
    buf = torch.full((offset + r * pitch + 16,), float("nan"), dtype=dtype)
    view = buf.cuda()[offset:offset + r * pitch].view(r, pitch)[:, :c]
    view.copy_(v)
    return view


def f64(t):
    torch.cuda.synchronize()
    return t.detach().cpu().double().numpy()


def erf(x):
    return torch.special.erf(torch.from_numpy(np.ascontiguousarray(x))).numpy()


def act_exact(z, act):
    if act == "relu":
        return np.maximum(z, 0.0)
    if act == "gelu":
        return z * 0.5 * (1 + erf(z / np.sqrt(2)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + np.tanh(np.sqrt(2 / np.pi) * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z / (1 + np.exp(-z))
    return z


def grad_exact(z, act):
    if act == "relu":
        return (z > 0).astype(np.float64)
    if act == "gelu":
        return 0.5 * (1 + erf(z / np.sqrt(2))) + z * np.exp(-z * z / 2) / np.sqrt(2 * np.pi)
    if act == "gelu_tanh":
        t = np.tanh(np.sqrt(2 / np.pi) * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * np.sqrt(2 / np.pi) * (1 + 3 * 0.044715 * z * z)
    if act == "silu":
        p = 1 / (1 + np.exp(-z))
        return p * (1 + z * (1 - p))
    return np.ones_like(z)


def assert_near(got, exact, scale, dtype, n, c, what):
    """scale: sum of the terms' magnitudes."""
    g = f64(got)
    u = UNIT[dtype]
    bound = u * np.abs(exact) + (c * u + (n + 16) * 2.0 ** -23) * scale + TINY[dtype]
    err = np.abs(g - exact)
    bad = ~(err <= bound)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        pytest.fail("%s: %d of %d outside; first %s: got %r, exact %r, bound %r"
                    % (what, bad.sum(), bad.size, i, g[i], exact[i], bound[i]))


# M, N, K: one row and column, tile corners, whole 16-byte rows and not, an
# empty sum, K around the ring's 5 steps of 32, a split K, large
SHAPES = [(1, 1, 1), (1, 8, 8), (3, 5, 7), (17, 24, 40), (64, 256, 512), (127, 129, 131),
          (128, 128, 160), (256, 256, 288), (257, 264, 320), (130, 72, 0), (300, 520, 999),
          (16, 4096, 1024), (5, 1000, 2056), (511, 768, 1024), (33, 40, 8192), (1100, 1032, 96)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_linear_forward(shape, dtype):
    M, N, K = shape
    act = ACTS[(M + N + K) % len(ACTS)]
    say("linear", shape, dtype, act)
    x = rand((M, K), dtype, 1)
    w = rand((K, N), dtype, 2, std=max(K, 1) ** -0.5)
    b = rand((N,), dtype, 3, std=0.3)
    r = rand((M, N), dtype, 4)
    z = torch.full((M, N), float("nan"), dtype=dtype, device="cuda")
    y = pg.plinear(x, w, bias=b, residual=r, act=act, preact=z)
    X, W, B, R = f64(x), f64(w), f64(b), f64(r)
    Z = X @ W + B
    S = np.abs(X) @ np.abs(W) + np.abs(B)
    assert_near(z, Z, S, dtype, K, 0, "preact")
    # an activation moves by at most 1.2 of its argument's error
    assert_near(y, act_exact(Z, act) + R, 1.2 * S + np.abs(R), dtype, K, 0, "y")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_linear_backward(shape, dtype):
    M, N, K = shape
    act = ACTS[(M + N + K + 1) % len(ACTS)]
    say("linear backward", shape, dtype, act)
    x = rand((M, K), dtype, 11)
    w = rand((K, N), dtype, 12, std=max(K, 1) ** -0.5)
    z = rand((M, N), dtype, 13)
    dy = rand((M, N), dtype, 14)
    a = rand((M, K), dtype, 15)
    dx, dw, db = pg.plinear_bwd(dy, x, w, preact=z, act=act, dx_residual=a)
    X, W, Z, DY, A = f64(x), f64(w), f64(z), f64(dy), f64(a)
    DZ = DY * grad_exact(Z, act)
    mag = np.abs(DY) * 1.2  # |act'| is below 1.13 everywhere
    c = 1 if act != "none" else 0  # dz is rounded once
    assert_near(dx, DZ @ W.T + A, mag @ np.abs(W).T + np.abs(A), dtype, N, c, "dx")
    assert_near(dw, X.T @ DZ, np.abs(X).T @ mag, dtype, M, c, "dw")
    assert_near(db, DZ.sum(0), mag.sum(0), dtype, M, 0, "dbias")


# (pitch beyond the row, offset of the first element): whole 16-byte rows,
# rows off by some elements, an address off by one element
STRIDES = [(8, 0), (64, 8), (3, 0), (0, 1), (5, 3), (16, 4)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pad,offset", STRIDES)
@pytest.mark.parametrize("shape", [(130, 136, 72), (4, 264, 520), (37, 51, 43)])
def test_linear_strides(shape, pad, offset, dtype):
    M, N, K = shape
    say("linear strides", shape, pad, offset, dtype)
    x = rand((M, K), dtype, 21, pitch=K + pad, offset=offset)
    w = rand((K, N), dtype, 22, std=K ** -0.5, pitch=N + pad, offset=offset)
    r = rand((M, N), dtype, 23, pitch=N + pad, offset=offset)
    out = rand((M, N), dtype, 24, pitch=N + pad, offset=offset)
    z = rand((M, N), dtype, 25, pitch=N + pad, offset=offset)
    got = pg.plinear(x, w, residual=r, act="silu", preact=z, out=out)
    assert got is out
    dense = pg.plinear(x.contiguous(), w.contiguous(), residual=r.contiguous(), act="silu")
    assert torch.equal(out, dense)
    # the gaps between rows keep their NaN
    if pad:
        whole = torch.as_strided(out, (M, N + pad), (N + pad, 1), out.storage_offset())
        assert bool(torch.isnan(whole[:, N:]).all())
    dy = rand((M, N), dtype, 26, pitch=N + pad, offset=offset)
    g = pg.plinear_bwd(dy, x, w, preact=z, act="silu")
    h = pg.plinear_bwd(dy.contiguous(), x.contiguous(), w.contiguous(), preact=z.contiguous(),
                       act="silu")
    for u, v in zip(g, h):
        assert torch.equal(u, v)


# (M, D, F, N): single values, whole and broken 16-byte rows, tile edges, a
# split contraction, more outputs than inputs, an empty block
FFN = [(1, 1, 1, 1), (1, 64, 96, 64), (5, 37, 51, 29), (130, 72, 129, 72), (64, 512, 256, 512),
       (257, 264, 520, 136), (3, 1024, 2048, 1024), (300, 100, 36, 260), (40, 8, 0, 16),
       (129, 4096, 136, 24)]


def kept(t):
    """The values that pffn kept in gate_up: float16 as they are, for bfloat16
    1 sign, 6 exponent (bias 31) and 9 fraction bits."""
    if t.dtype is torch.float16:
        return f64(t)
    torch.cuda.synchronize()
    c = t.contiguous().view(torch.int16).cpu().numpy().astype(np.int64) & 0xFFFF
    exponent, fraction = (c >> 9) & 63, c & 511
    v = np.where(exponent > 0, np.ldexp(1.0 + fraction / 512.0, exponent - 31), 0.0)
    v = np.where((c & 0x7FFF) == 0x7FFF, np.nan, v)
    return np.where(c >> 15, -v, v)


def test_ffn_kept_range():
    """Kept values of every size: g = x * w_in with one input and x = 1."""
    v = np.array([0.0, 1.0, -1.5, 2.0 ** -30, 2.0 ** -31, -(2.0 ** 32), 2.0 ** 34, 1e38, np.inf,
                  np.nan, 255.0, -(2.0 ** -29)])
    w = torch.from_numpy(np.concatenate([v, v])[None]).to(torch.bfloat16).cuda()
    gu = torch.empty((1, 24), dtype=torch.bfloat16, device="cuda")
    pg.pffn(torch.ones((1, 1), dtype=torch.bfloat16, device="cuda"), w,
            torch.zeros((12, 1), dtype=torch.bfloat16, device="cuda"), gate_up=gu)
    exact = f64(w)[0]
    a = np.abs(exact)
    exact = np.where(a < 2.0 ** -30, 0.0, np.where(a < 2.0 ** 33, exact, np.nan))
    assert np.array_equal(kept(gu)[0], exact, equal_nan=True)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", FFN)
def test_ffn(shape, dtype):
    M, D, F, N = shape
    act = ACTS[(M + D + F) % len(ACTS)]
    say("ffn", shape, dtype, act)
    x = rand((M, D), dtype, 31)
    wi = rand((D, 2 * F), dtype, 32, std=D ** -0.5)
    wo = rand((F, N), dtype, 33, std=max(F, 1) ** -0.5)
    r = rand((M, N), dtype, 34)
    gu = torch.full((M, 2 * F), float("nan"), dtype=dtype, device="cuda")
    y = pg.pffn(x, wi, wo, residual=r, act=act, gate_up=gu)
    X, WI, WO, R = f64(x), f64(wi), f64(wo), f64(r)
    G, U = (X @ WI)[:, :F], (X @ WI)[:, F:]
    S = np.abs(X) @ np.abs(WI)
    KU = UNIT[dtype] / (1 if dtype is torch.float16 else 4)  # the kept form's rounding
    GU = kept(gu)
    assert (np.abs(GU - X @ WI) <= KU * np.abs(X @ WI) + (D + 16) * 2.0 ** -23 * S + 2.0 ** -30).all()
    H = act_exact(G, act) * U
    # an error of g or u (fp32 accumulation) reaches h through the product
    e32 = (D + 16) * 2.0 ** -23
    HE = e32 * 1.2 * (S[:, :F] * np.abs(U) + np.abs(act_exact(G, act)) * S[:, F:])
    Y = H @ WO + R
    bound = HE @ np.abs(WO)
    exact_scale = np.abs(H) @ np.abs(WO) + np.abs(R)
    u = UNIT[dtype]
    tol = (u * np.abs(Y) + (u + (F + 16) * 2.0 ** -23) * exact_scale + bound * 1.01 + TINY[dtype]
           + TINY[dtype] * np.abs(WO).sum(0))
    assert (np.abs(f64(y) - Y) <= tol).all()

    # the backward pass takes gate_up as kept
    dy = rand((M, N), dtype, 35)
    a = rand((M, D), dtype, 36)
    dx, dwi, dwo = pg.pffn_bwd(dy, x, wi, wo, gu, act=act, dx_residual=a)
    DY, A = f64(dy), f64(a)
    G, U = GU[:, :F], GU[:, F:]
    DH = DY @ WO.T
    DHS = np.abs(DY) @ np.abs(WO).T
    AG, DG = act_exact(G, act), grad_exact(G, act)
    DIN = np.concatenate([DH * U * DG, DH * AG], axis=1)
    # magnitudes: the rounding of an entry, and fp32 accumulation over N in dh
    # (17 + N of 2^-23 of DHS) is far below half a rounding of it only where dh does
    # not cancel, so it is added
    mag = np.abs(DIN) + 2 * (N + 17) * 2.0 ** -23 / u * np.concatenate(
        [DHS * np.abs(U) * 1.2, DHS * (np.abs(AG) + 1e-6 * np.abs(G))], axis=1)
    assert_near(dx, DIN @ WI.T + A, mag @ np.abs(WI).T + np.abs(A), dtype, 2 * F, 1, "dx")
    assert_near(dwi, X.T @ DIN, np.abs(X).T @ mag, dtype, M, 1, "dw_in")
    assert_near(dwo, (AG * U).T @ DY, (np.abs(AG) * np.abs(U) * 1.0001 + 1e-6 * np.abs(G * U)).T
                @ np.abs(DY), dtype, M, 1, "dw_out")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("pad,offset", STRIDES)
@pytest.mark.parametrize("shape", [(130, 72, 136, 40), (4, 264, 520, 264), (37, 51, 43, 27)])
def test_ffn_strides(shape, pad, offset, dtype):
    M, D, F, N = shape
    say("ffn strides", shape, pad, offset, dtype)
    x = rand((M, D), dtype, 41, pitch=D + pad, offset=offset)
    wi = rand((D, 2 * F), dtype, 42, std=D ** -0.5, pitch=2 * F + pad, offset=offset)
    wo = rand((F, N), dtype, 43, std=F ** -0.5, pitch=N + pad, offset=offset)
    gu = rand((M, 2 * F), dtype, 44, pitch=2 * F + pad, offset=offset)
    gu2 = torch.empty((M, 2 * F), dtype=dtype, device="cuda")
    y = pg.pffn(x, wi, wo, gate_up=gu)
    z = pg.pffn(x.contiguous(), wi.contiguous(), wo.contiguous(), gate_up=gu2)
    assert torch.equal(y, z) and torch.equal(gu, gu2)
    dy = rand((M, N), dtype, 45, pitch=N + pad, offset=offset)
    g = pg.pffn_bwd(dy, x, wi, wo, gu)
    h = pg.pffn_bwd(dy.contiguous(), x.contiguous(), wi.contiguous(), wo.contiguous(), gu2)
    for u, v in zip(g, h):
        assert torch.equal(u, v)


def xent_exact(X, W, t, V, ignore=-100):
    L = X @ W.T
    top = L.max(1, keepdims=True)
    lse = top[:, 0] + np.log(np.exp(L - top).sum(1))
    valid = t != ignore
    at = np.where(valid, t, 0)
    loss = np.where(valid, lse - L[np.arange(len(t)), at], 0.0)
    p = np.exp(L - lse[:, None])
    p[np.arange(len(t)), at] -= 1.0
    return L, lse, loss, p * valid[:, None], valid


# (M, D, V): single values, odd vocabularies, tile edges, several pieces of the
# backward pass (V > 1024 only with many rows: see below), a long row
XENT = [(1, 1, 1), (1, 64, 1000), (7, 40, 257), (130, 72, 511), (33, 100, 1025), (300, 264, 640),
        (5, 1024, 5003), (257, 37, 300)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
@pytest.mark.parametrize("shape", XENT)
def test_xent(shape, reduction, dtype):
    M, D, V = shape
    say("xent", shape, reduction, dtype)
    x = rand((M, D), dtype, 51)
    w = rand((V, D), dtype, 52, std=2 * D ** -0.5)
    rng = np.random.default_rng(53)
    t = rng.integers(0, V, size=M)
    t[rng.random(M) < 0.3] = -100
    target = torch.from_numpy(t).cuda()
    loss, lse = pg.pxent(x, w, target, reduction=reduction)
    X, W = f64(x), f64(w)
    L, LSE, EACH, P, valid = xent_exact(X, W, t, V)
    S = np.abs(X) @ np.abs(W).T
    # a logit's fp32 accumulation, exp and log of fp32 values near |lse|
    e = (D + 8) * 2.0 ** -23 * S.max(1) + 16 * 2.0 ** -23 * (np.abs(LSE) + 1)
    assert (np.abs(f64(lse) - LSE) <= e).all()
    n = max(1, int(valid.sum()))
    e2 = 2 * e * valid
    if reduction == "none":
        assert (np.abs(f64(loss) - EACH) <= e2 + 2.0 ** -23 * np.abs(EACH)).all()
    else:
        k = n if reduction == "mean" else 1
        assert abs(f64(loss) - EACH.sum() / k) <= (e2.sum() + 2.0 ** -22 * np.abs(EACH).sum()) / k

    if reduction == "none":
        g = rng.normal(0, 1, size=M).astype(np.float32)
        g[::3] *= 1e-3
        dloss = torch.from_numpy(g).cuda()
        G = g.astype(np.float64)
    else:
        dloss = torch.tensor(0.37, device="cuda")
        G = np.full(M, float(np.float32(0.37)) / (n if reduction == "mean" else 1))
    dx, dw = pg.pxent_bwd(x, w, target, lse, dloss=dloss, reduction=reduction)
    DL = P * G[:, None]
    # dl: one rounding, and the absolute error of the logit and lse in the exponent
    q = np.exp(L - LSE[:, None]) * valid[:, None] * np.abs(G)[:, None]
    u = UNIT[dtype]
    top = np.abs(G).max()
    mag = np.abs(DL) + q * (2 * e[:, None] + 8 * 2.0 ** -23 * (1 + np.abs(L - LSE[:, None]))) / u
    if dtype is torch.float16:  # subnormals of the scaled dl
        mag = mag + valid[:, None] * top * 2.0 ** -15 * 2.0 ** -24 / u
    assert_near(dx, DL @ W, mag @ np.abs(W), dtype, V, 1, "dx")
    assert_near(dw, DL.T @ X, mag.T @ np.abs(X), dtype, M, 1, "dw")


@pytest.mark.parametrize("dtype", DTYPES)
def test_xent_pieces_and_strides(dtype):
    """Rows enough that the backward pass takes the vocabulary in pieces, the
    last one shorter; strided and misaligned operands give the same bits."""
    M, D, V = 140000, 24, 4500
    say("xent pieces", M, D, V, dtype)
    x = rand((M, D), dtype, 61)
    w = rand((V, D), dtype, 62, std=2 * D ** -0.5)
    target = torch.from_numpy(np.random.default_rng(63).integers(0, V, size=M)).cuda()
    loss, lse = pg.pxent(x, w, target)
    dx, dw = pg.pxent_bwd(x, w, target, lse, reduction="sum")
    X, W, T = x.double(), w.double(), target
    L = X @ W.t()
    LSE = torch.logsumexp(L, 1)
    each = LSE - L[torch.arange(M, device="cuda"), T]
    assert abs(float(loss) - float(each.mean())) <= 1e-5
    P = torch.exp(L - LSE[:, None])
    P[torch.arange(M, device="cuda"), T] -= 1.0
    u = UNIT[dtype]
    A = P.abs() + 2.0 ** -30
    DX, DW = P @ W, P.t() @ X
    ex = 1.5 * u * DX.abs() + (1.5 * u + (V + 64) * 2.0 ** -23) * (A @ W.abs()) + 1e-6
    ew = 1.5 * u * DW.abs() + (1.5 * u + (M + 64) * 2.0 ** -23) * (A.t() @ X.abs()) + 1e-6
    assert bool(((dx.double() - DX).abs() <= ex).all())
    assert bool(((dw.double() - DW).abs() <= ew).all())

    xs = rand((M, D), dtype, 61, pitch=D + 3, offset=1)
    ws = rand((V, D), dtype, 62, std=2 * D ** -0.5, pitch=D + 5, offset=3)
    loss2, lse2 = pg.pxent(xs, ws, target)
    assert torch.equal(loss, loss2) and torch.equal(lse, lse2)
    dx2, dw2 = pg.pxent_bwd(xs, ws, target, lse, reduction="sum")
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2)


def test_xent_masks():
    """All rows ignored; targets outside the vocabulary; ignored rows with
    infinite and NaN values in x."""
    M, D, V = 70, 64, 300
    x = rand((M, D), torch.bfloat16, 71)
    w = rand((V, D), torch.bfloat16, 72, std=0.2)
    t = torch.full((M,), -100, device="cuda")
    loss, lse = pg.pxent(x, w, t)
    dx, dw = pg.pxent_bwd(x, w, t, lse)
    assert float(loss) == 0.0 and not bool(dx.any()) and not bool(dw.any())
    assert not bool(pg.pxent(x, w, t, reduction="none")[0].any())

    t = torch.arange(M, device="cuda")
    t[5], t[9] = V, -1
    loss, lse = pg.pxent(x, w, t, reduction="none")
    bad = torch.isnan(loss)
    assert bad[5] and bad[9] and int(bad.sum()) == 2
    dx, dw = pg.pxent_bwd(x, w, t, lse, reduction="none")
    rows = torch.isnan(dx).all(1)
    assert rows[5] and rows[9] and int(torch.isnan(dx).any(1).sum()) == 2
    assert int(pg.pxent(x, w, t, ignore_index=V, reduction="none")[0].isnan().sum()) == 1

    clean = torch.arange(M, device="cuda")
    clean[[3, 40]] = -100
    y = x.clone()
    y[3], y[40] = float("inf"), float("nan")
    loss, lse = pg.pxent(y, w, clean)
    ref, _ = pg.pxent(x, w, clean)
    assert torch.equal(loss, ref)
    dx, _ = pg.pxent_bwd(y, w, clean, lse, needs=(True, False))
    ref, _ = pg.pxent_bwd(x, w, clean, pg.pxent(x, w, clean)[1], needs=(True, False))
    assert torch.equal(dx, ref) and not bool(dx[3].any()) and not bool(dx[40].any())


CLIP_KINDS = [[torch.float32], [torch.float16], [torch.bfloat16],
              [torch.float32, torch.float16, torch.bfloat16]]


@pytest.mark.parametrize("inplace", [False, True])
@pytest.mark.parametrize("kinds", CLIP_KINDS)
@pytest.mark.parametrize("sizes", [[1], [7, 0, 4096, 33], [5] * 300, [40000, 1 << 20, 3],
                                   [17000001, 32768, 32769, 9]])
def test_clip(sizes, kinds, inplace):
    say("clip", len(sizes), sum(sizes), kinds, inplace)
    rng = np.random.default_rng(81)
    grads = []
    for i, n in enumerate(sizes):
        k = kinds[i % len(kinds)]
        v = torch.from_numpy(rng.normal(0, 1, size=n).astype(np.float32)).to(k)
        off = i % 5  # elements off a 16-byte boundary
        buf = torch.empty(n + 8, dtype=k, device="cuda")
        t = buf[off:off + n]
        t.copy_(v)
        grads.append(t)
    exact = [f64(t) for t in grads]
    norm = np.sqrt(sum((e * e).sum() for e in exact))
    for factor in (0.3, 2.0):
        out = None if inplace else [torch.full_like(t, float("nan")) for t in grads]
        src = [t.clone() for t in grads] if inplace else grads
        got = pg.pclip_grad_norm(src, factor * norm, out=out)
        # fp64 sums (8 fp16 squares in fp32 first), one rounding to fp32
        assert abs(f64(got) - norm) <= 2.0 ** -22 * norm
        c = min(1.0, float(np.float32(factor * norm)) / (norm + 1e-6))
        for e, o in zip(exact, src if inplace else out):
            u = UNIT.get(o.dtype, 2.0 ** -24)
            tiny = TINY.get(o.dtype, 2.0 ** -126)
            # the factor's and the product's fp32 roundings, and the type's
            assert (np.abs(f64(o) - e * c) <= (u + 2.0 ** -22) * np.abs(e * c) + tiny).all()
            if factor > 1:
                assert np.array_equal(f64(o), e)


def test_clip_extremes():
    """Squares beyond fp32's range; NaN and infinite gradients."""
    big = torch.full((1000,), 1e30, dtype=torch.bfloat16, device="cuda")
    small = torch.full((1000,), 1e-30, device="cuda")
    e = f64(big)
    n = pg.pclip_grad_norm([big.clone()], float("inf"))
    assert abs(f64(n) - np.sqrt((e * e).sum())) <= 1e-6 * f64(n)
    n = pg.pclip_grad_norm([small.clone()], 1.0)
    assert abs(f64(n) - f64(small)[0] * np.sqrt(1000)) <= 1e-6 * f64(n)
    x = [torch.ones(100, device="cuda"), torch.ones(50, dtype=torch.float16, device="cuda")]
    x[1][7] = float("nan")
    n = pg.pclip_grad_norm(x, 1.0)
    assert bool(torch.isnan(n)) and all(bool(torch.isnan(t).all()) for t in x)
    y = [torch.ones(100, device="cuda")]
    y[0][3] = float("inf")
    n = pg.pclip_grad_norm(y, 1.0)
    assert bool(torch.isinf(n)) and int((y[0] == 0).sum()) == 99
