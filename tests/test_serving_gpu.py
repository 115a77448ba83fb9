"""The norm, the microscaled matrices and sampling on the GPU against plain
formulas in binary64 on the CPU (numpy), written apart from the kernels.

Tolerances, derived before the first run.  u is the output type's rounding
(2^-11 for float16, 2^-8 for bfloat16: half a step relative to the value).
 - The norm: s = x + r in fp32 is off by 2^-24 of s; a sum of up to 100 squares one
   after the other and a tree of 16 additions by at most 120 2^-24 of it, half of
   that in the root; the reciprocal root, the mean's and the three other products
   by 2^-23 each: 2^-17 of y in all, beside its own rounding u.
 - Its gradient: terms (g - n mean(g n)) / rms, each with a few such errors, and
   mean(g n) 2^-17 of mean|g n|; h is the stored one in the reference too.
 - Quantisation and back: no tolerance.
 - The product: exact operands; fp32 sums of K products in any order, (K + 16)
   2^-23 of the sum of magnitudes; with 8-bit elements on either side the matrix
   instruction may drop what lies below 2^-11 of the largest of 128 products: the
   bound per instruction is 2^-10 of its largest product (128 such losses of one
   sign would be more, and do not occur together).  The epilogue
   adds a few fp32 roundings, the activation's of up to 2^-19 relative.
 - Sampling: tokens are equal; logprobs within 2^-22 (1 + |logprob|)."""
import sys

import numpy as np
import pytest

import software_pipelined_tiled_pgemm_amd as pg

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

UNIT = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float16: 2.0 ** -24, torch.bfloat16: 2.0 ** -126}
DTYPES = [torch.float16, torch.bfloat16]
FORMATS = ["e2m1", "e4m3"]


def say(*a):
    print(*a, flush=True)
    sys.stdout.flush()


def rand(shape, dtype, seed, std=1.0, pitch=None, offset=0):
    """Normal values on the device, rows `pitch` apart, the first one `offset`
    elements into its buffer; the gaps hold NaN."""
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


def near(got, exact, bound, what):
    g = f64(got)
    err = np.abs(g - exact)
    bad = ~(err <= bound)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        pytest.fail("%s: %d of %d outside; first %s: got %r, exact %r, bound %r"
                    % (what, bad.sum(), bad.size, i, g[i], exact[i], np.broadcast_to(bound, err.shape)[i]))


# ---- microscaled numbers -------------------------------------------------------

GRID = {"e2m1": np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6]),
        "e4m3": np.array([i * 2.0 ** -9 for i in range(8)] +
                         [(8 + i) * 2.0 ** (e - 10) for e in range(1, 16) for i in range(8)][:-1])}


def mx_reference(v, to):
    """(codes by element, scale codes) of v [rows, cols] in binary64, columns
    padded to a multiple of 128."""
    rows, cols = v.shape
    pad = -cols % 128
    v = np.concatenate([v, np.zeros((rows, pad))], axis=1).reshape(rows, -1, 32)
    grid = GRID[to]
    most = np.abs(v).max(axis=2)
    fine = np.isfinite(v).all(axis=2)
    m, e = np.frexp(np.where(fine, most, 0.0))
    # most = m 2^e; the smallest s with most <= grid[-1] 2^s
    s = np.ceil(np.log2(np.maximum(m, 0.5) / grid[-1])).astype(int) + e
    s += most > grid[-1] * np.exp2(s.astype(float))
    s -= (most <= grid[-1] * np.exp2(s - 1.0))
    s = np.where(most > 0, np.maximum(s, -127), -127)
    a = np.where(fine[:, :, None], np.abs(v), 0.0) / np.exp2(s.astype(float))[:, :, None]
    hi = np.minimum(np.searchsorted(grid, a), len(grid) - 1)
    lo = np.maximum(hi - 1, 0)
    up, down = grid[hi] - a, a - grid[lo]
    code = np.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    sign = (np.signbit(v) & fine[:, :, None]) * (8 if to == "e2m1" else 128)
    return (code + sign).reshape(rows, -1), np.where(fine, s + 127, 255)


def codes_of(m):
    """Elements one by one, and the scales of the blocks."""
    torch.cuda.synchronize()
    groups = (m.cols + 127) // 128
    c = m.codes.cpu().numpy().astype(int)
    if m.format == "e2m1":
        c = c[:, :64 * groups]
        c = np.stack([c & 15, c >> 4], axis=2).reshape(len(c), -1)
    return c[:, :128 * groups], m.scales.cpu().numpy()[:, :4 * groups].astype(int)


def values_of(m):
    c, s = codes_of(m)
    grid = np.concatenate([GRID[m.format], [np.nan] if m.format == "e4m3" else []])
    half = len(grid)
    v = grid[c % half] * np.where(c >= half, -1.0, 1.0)
    scale = np.where(s == 255, np.nan, np.exp2(s - 127.0))
    return (v * scale.repeat(32, axis=1))[:, :m.cols]


@pytest.mark.parametrize("to", FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_quantize_every_value(dtype, to):
    """Every 16-bit pattern, in blocks of neighbours and in shuffled blocks."""
    bits = np.arange(65536).astype(np.uint16)
    shuffled = np.random.default_rng(1).permutation(bits)
    mild = bits[np.abs(torch.from_numpy(bits.view(np.int16)).view(dtype).float().numpy()) < 100]
    mild = np.random.default_rng(2).permutation(np.resize(mild, 65536))
    x = np.stack([bits, shuffled, mild]).reshape(3 * 64, 1024)
    t = torch.from_numpy(x.view(np.int16)).view(dtype)
    say("quantize every value", dtype, to)
    m = pg.pmx_quantize(t.cuda(), to)
    got_c, got_s = codes_of(m)
    want_c, want_s = mx_reference(t.double().numpy(), to)
    assert np.array_equal(got_s, want_s)
    assert np.array_equal(got_c, want_c)


@pytest.mark.parametrize("to", FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape,pitch,offset", [((1, 1), None, 0), ((3, 31), None, 0), ((2, 32), 40, 8),
                                                ((5, 33), 35, 1), ((4, 127), None, 0),
                                                ((7, 128), 129, 3), ((33, 513), 600, 0),
                                                ((300, 2050), None, 0), ((2, 9000), None, 0)])
def test_quantize_shapes(shape, pitch, offset, dtype, to):
    x = rand(shape, dtype, 5, pitch=pitch, offset=offset)
    say("quantize", shape, pitch, offset, dtype, to)
    m = pg.pmx_quantize(x, to)
    c, s = codes_of(m)
    want_c, want_s = mx_reference(f64(x), to)
    assert np.array_equal(s, want_s) and np.array_equal(c, want_c)
    # back: rounded once
    for out in DTYPES:
        y = torch.full(shape, float("nan"), dtype=out, device="cuda")
        assert pg.pmx_dequantize(m, out=y) is y
        want = torch.from_numpy(values_of(m)).to(out)
        torch.cuda.synchronize()
        assert torch.equal(y.cpu(), want)


@pytest.mark.parametrize("to", FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
def test_dequantize_every_code(dtype, to):
    """Every element under every scale, subnormals, overflow and NaN included."""
    n = 16 if to == "e2m1" else 256
    c = np.tile(np.arange(n), (256, 1))
    codes = (c[:, 0::2] | (c[:, 1::2] << 4)) if to == "e2m1" else c
    pad = 128 if to == "e4m3" else 64
    codes = np.pad(codes, ((0, 0), (0, -codes.shape[1] % pad))).astype(np.uint8)
    scales = np.repeat(np.arange(256)[:, None], 16, axis=1).astype(np.uint8)
    m = pg.MxMatrix(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), n, to)
    say("dequantize every code", dtype, to)
    y = pg.pmx_dequantize(m, dtype=dtype).cpu()
    want = torch.from_numpy(values_of(m)).to(dtype)
    assert torch.equal(y.isnan(), want.isnan())
    assert torch.equal(y.nan_to_num(0.0), want.nan_to_num(0.0))


def test_quantize_strided_matrix():
    """Codes and scales as parts of wider buffers, whose other bytes stay."""
    x = rand((9, 200), torch.bfloat16, 3)
    codes = torch.full((9, 512), 0xAA, dtype=torch.uint8, device="cuda")
    scales = torch.full((9, 64), 0xAA, dtype=torch.uint8, device="cuda")
    m = pg.MxMatrix(codes[:, 128:384], scales[:, 16:32], 200, "e4m3")
    assert pg.pmx_quantize(x, "e4m3", out=m) is m
    plain = pg.pmx_quantize(x, "e4m3")
    torch.cuda.synchronize()
    assert torch.equal(m.codes, plain.codes) and torch.equal(m.scales[:, :8], plain.scales[:, :8])
    assert (codes[:, :128] == 0xAA).all() and (codes[:, 384:] == 0xAA).all()
    assert (scales[:, :16] == 0xAA).all() and (scales[:, 32:] == 0xAA).all()


# ---- the norm --------------------------------------------------------------------

NORM_SHAPES = [(1, 1), (3, 7), (5, 64), (17, 129), (64, 512), (33, 1000), (9, 1025), (9, 2048),
               (7, 2056), (5, 4096), (3, 4104), (3, 8192), (2, 16384), (3, 20001), (2, 32768), (2, 32776),
               (3, 70001), (1000, 72)]


def norm_exact(x, r, w, eps):
    s = x if r is None else x + r
    n = s / np.sqrt((s * s).mean(axis=1, keepdims=True) + eps)
    return s, n if w is None else n * w


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", NORM_SHAPES)
def test_norm_forward(shape, dtype):
    M, D = shape
    odd = (M + D) % 2
    say("norm", shape, dtype)
    x = rand(shape, dtype, 1, pitch=D + 5 if odd else None, offset=odd)
    r = rand(shape, dtype, 2, std=2.0, pitch=None if odd else D + 8)
    w = rand((D,), dtype, 3)
    h = torch.full(shape, float("nan"), dtype=dtype, device="cuda")
    y = pg.prmsnorm(x, w, residual=r, eps=1e-5, h=h)
    S, Y = norm_exact(f64(x), f64(r), f64(w), 1e-5)
    u = UNIT[dtype]
    near(h, S, (u + 2.0 ** -23) * np.abs(S) + TINY[dtype], "h")
    near(y, Y, (u + 2.0 ** -17) * np.abs(Y) + TINY[dtype], "y")
    # without residual and weight; in place
    _, Y = norm_exact(f64(x), None, None, 1e-5)
    near(pg.prmsnorm(x, eps=1e-5), Y, (u + 2.0 ** -17) * np.abs(Y) + TINY[dtype], "plain y")
    a, b = x.clone(), r.contiguous()
    assert pg.prmsnorm(a, w, residual=b, eps=1e-5, h=b, out=a) is a
    torch.cuda.synchronize()
    assert torch.equal(a, y) and torch.equal(b, h)


@pytest.mark.parametrize("to", FORMATS)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", NORM_SHAPES)
def test_norm_quantized(shape, dtype, to):
    M, D = shape
    say("norm", shape, dtype, to)
    x, r, w = rand(shape, dtype, 4, pitch=D + 3), rand(shape, dtype, 5), rand((D,), dtype, 6)
    h = torch.empty(shape, dtype=dtype, device="cuda")
    m = pg.prmsnorm(x, w, residual=r, h=h, format=to)
    assert m.shape == shape and m.format == to
    S, Y = norm_exact(f64(x), f64(r), f64(w), 1e-6)
    near(h, S, (UNIT[dtype] + 2.0 ** -23) * np.abs(S) + TINY[dtype], "h")
    c, s = codes_of(m)
    scale = np.exp2(s - 127.0)
    padded = np.pad(np.abs(Y), ((0, 0), (0, -D % 128)))
    most = padded.reshape(M, -1, 32).max(axis=2)
    top = GRID[to][-1]
    slack = 1 + 2.0 ** -16
    assert (most <= top * scale * slack).all() and ((most * slack > top * scale / 2) | (s == 0)).all()
    # half a step: 2^-4 of the value (e4m3), 2^-2 (e2m1), or half the smallest element
    rel, least = (2.0 ** -2, 0.25) if to == "e2m1" else (2.0 ** -4, 2.0 ** -10)
    bound = (rel + 2.0 ** -14) * np.abs(Y) + least * scale.repeat(32, axis=1)[:, :D]
    near(torch.from_numpy(values_of(m)), Y, bound, "values")
    assert (c[:, D:] == 0).all()


@pytest.mark.parametrize("D", [40, 4096, 33000])
def test_norm_extremes(D):
    """Squares outside fp32's range, empty rows, infinities and NaN, each row
    apart from the others."""
    bf = torch.bfloat16
    base = rand((8, D), bf, 7).float().cpu()
    rows = torch.stack([base[0] * 1e30, base[1] * 3e37, base[2] * 1e-30, base[3] * 1e-38, base[4] * 0,
                        base[5], base[6], base[7]]).to(bf)
    rows[5, D // 2] = float("inf")
    rows[6, 0] = float("nan")
    x = rows.cuda()
    u = 2.0 ** -8
    for eps in (0.0, 1e-30, 1e-5):
        say("norm extremes", D, eps)
        y = f64(pg.prmsnorm(x, eps=eps))
        X = rows.double().numpy()
        with np.errstate(all="ignore"):
            Y = X / np.sqrt((X * X).mean(axis=1, keepdims=True) + float(np.float32(eps)))
        for i in (0, 1, 2, 3, 7):
            err = np.abs(y[i] - Y[i])
            assert (err <= (u + 2.0 ** -16) * np.abs(Y[i]) + 2.0 ** -133).all(), (i, eps, err.max())
        assert np.isnan(y[4]).all() if eps == 0 else (y[4] == 0).all()
        assert np.isnan(y[5, D // 2]) and (np.delete(y[5], D // 2) == 0).all()
        assert np.isnan(y[6]).all()
        m = pg.prmsnorm(x, eps=eps, format="e4m3")
        s = codes_of(m)[1]
        assert (s[7] < 255).all() and (s[0] < 255).all()
        assert (s[6, :(D + 31) // 32] == 255).all() and s[5, D // 64] == 255
    big = torch.full((2, D), 65504.0, dtype=torch.float16, device="cuda")
    h = torch.empty_like(big)
    y = pg.prmsnorm(big, residual=big, h=h)
    assert (f64(y) == 1.0).all() and np.isinf(f64(h)).all()


def norm_grad_exact(dy, h, w, dh, eps):
    inv = 1.0 / np.sqrt((h * h).mean(axis=1, keepdims=True) + eps)
    n = h * inv
    g = dy if w is None else dy * w
    mean = (g * n).mean(axis=1, keepdims=True)
    dx = inv * (g - n * mean)
    size = inv * (np.abs(g) + np.abs(n) * np.abs(g * n).mean(axis=1, keepdims=True))
    if dh is not None:
        dx, size = dx + dh, size + np.abs(dh)
    return dx, size, (dy * n).sum(axis=0), np.abs(dy * n).sum(axis=0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", NORM_SHAPES + [(5000, 64), (2100, 520), (700, 4100), (130, 33000)])
def test_norm_backward(shape, dtype):
    M, D = shape
    odd = (M + D) % 2
    say("norm backward", shape, dtype)
    dy = rand(shape, dtype, 11, pitch=D + 3 if odd else None)
    h = rand(shape, dtype, 12, std=3.0, pitch=None if odd else D + 8)
    w, dh = rand((D,), dtype, 13), rand(shape, dtype, 14, pitch=D + 1)
    dx, dw = pg.prmsnorm_bwd(dy, h, w, eps=1e-5, dh=dh)
    DX, size, DW, wsize = norm_grad_exact(f64(dy), f64(h), f64(w), f64(dh), 1e-5)
    u = UNIT[dtype]
    near(dx, DX, u * np.abs(DX) + 2.0 ** -16 * size + TINY[dtype], "dx")
    # a column's sum: its products 2^-17 off, M of them added in any order
    near(dw, DW, u * np.abs(DW) + (2.0 ** -17 + M * 2.0 ** -24) * wsize + TINY[dtype], "dw")
    # each alone, without weight, in place of dh
    only, none = pg.prmsnorm_bwd(dy, h, w, eps=1e-5, dh=dh, needs=(True, False), dx=dh)
    assert none is None and only is dh
    none, only = pg.prmsnorm_bwd(dy, h, w, eps=1e-5, needs=(False, True))
    torch.cuda.synchronize()
    assert none is None and torch.equal(only, dw) and torch.equal(dh, dx)
    plain, none = pg.prmsnorm_bwd(dy, h, eps=1e-5)
    DX, size, _, _ = norm_grad_exact(f64(dy), f64(h), None, None, 1e-5)
    assert none is None
    near(plain, DX, u * np.abs(DX) + 2.0 ** -16 * size + TINY[dtype], "plain dx")


def test_norm_backward_extremes():
    bf = torch.bfloat16
    D = 300
    scale = torch.tensor([1e30, 3e37, 1e-30, 1.0])[:, None]
    h = (rand((4, D), bf, 21).float().cpu() * scale).to(bf)
    dy = rand((4, D), bf, 22)
    dx, dw = pg.prmsnorm_bwd(dy, h.cuda(), torch.ones(D, dtype=bf, device="cuda"), eps=1e-38)
    H = h.double().numpy()
    DX, size, DW, wsize = norm_grad_exact(f64(dy), H, None, None, 1e-38)
    near(dx, DX, 2.0 ** -8 * np.abs(DX) + 2.0 ** -15 * size + 2.0 ** -133, "dx")
    near(dw, DW, 2.0 ** -8 * np.abs(DW) + 2.0 ** -16 * wsize, "dw")


def test_norm_empty():
    w = torch.ones(8, dtype=torch.float16, device="cuda")
    x = torch.empty(0, 8, dtype=torch.float16, device="cuda")
    assert pg.prmsnorm(x, w).shape == (0, 8)
    assert pg.prmsnorm(x, w, format="e2m1").shape == (0, 8)
    dx, dw = pg.prmsnorm_bwd(x, x, w)
    assert dx.shape == (0, 8) and (f64(dw) == 0).all()
    e = torch.empty(3, 0, dtype=torch.float16, device="cuda")
    assert pg.prmsnorm(e).shape == (3, 0) and pg.pmx_quantize(e).shape == (3, 0)


def test_norm_gradient_against_differences():
    """The backward pass against central differences of the forward pass in
    binary64, and of the kernel's own loss along a direction."""
    M, D, eps = 3, 50, 1e-3
    rng = np.random.default_rng(31)
    H, W, DY = rng.normal(size=(M, D)), rng.normal(size=D), rng.normal(size=(M, D))
    t = [torch.from_numpy(v).half() for v in (H, W, DY)]
    H, W, DY = (v.double().numpy() for v in t)
    dx, dw = pg.prmsnorm_bwd(t[2].cuda(), t[0].cuda(), t[1].cuda(), eps=eps)
    dx, dw = f64(dx), f64(dw)

    def loss(h, w):
        return (norm_exact(h, None, w, eps)[1] * DY).sum()
    d = 1e-5
    for m, k in [(0, 0), (1, 17), (2, 49)]:
        e = np.zeros_like(H)
        e[m, k] = d
        slope = (loss(H + e, W) - loss(H - e, W)) / (2 * d)
        assert abs(dx[m, k] - slope) <= 2.0 ** -11 * abs(slope) + 2.0 ** -13 * np.abs(DY[m] * W).max()
        e = np.zeros_like(W)
        e[k] = d
        slope = (loss(H, W + e) - loss(H, W - e)) / (2 * d)
        assert abs(dw[k] - slope) <= 2.0 ** -11 * abs(slope) + 2.0 ** -16 * np.abs(DY[:, k]).sum()


# ---- the product -------------------------------------------------------------------

def act_exact(z, act):
    if act == "relu":
        return np.maximum(z, 0.0)
    if act == "gelu":
        e = torch.special.erf(torch.from_numpy(np.ascontiguousarray(z / np.sqrt(2)))).numpy()
        return z * 0.5 * (1 + e)
    if act == "gelu_tanh":
        return 0.5 * z * (1 + np.tanh(np.sqrt(2 / np.pi) * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z / (1 + np.exp(-z))
    return z


ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def check_mx(y, x, w, bias, residual, act, dtype, what):
    """y against the values of the MxMatrices x and w."""
    X, W = values_of(x), values_of(w)
    K = X.shape[1]
    Z = X @ W.T
    size = np.abs(X) @ np.abs(W).T
    drop = np.zeros_like(Z)
    if "e4m3" in (x.format, w.format):
        for k in range(0, K, 128):
            a, b = np.abs(X[:, k:k + 128]), np.abs(W[:, k:k + 128])
            # at most the product of the largest of each, row by row
            drop += 2.0 ** -10 * np.minimum((a @ b.T), a.max(axis=1)[:, None] * b.max(axis=1)[None, :])
    if bias is not None:
        Z, size = Z + f64(bias), size + np.abs(f64(bias))
    Y = act_exact(Z, act)
    # the activations' slopes stay below 1.13
    off = 1.13 * ((K + 16) * 2.0 ** -23 * size + drop) + 2.0 ** -18 * np.abs(Y)
    if act in ("gelu", "gelu_tanh", "silu"):
        off = off + 2.0 ** -18 * np.abs(Z)
    if residual is not None:
        Y = Y + f64(residual)
        off = off + 2.0 ** -23 * np.abs(Y)
    near(y, Y, UNIT[dtype] * np.abs(Y) + off * 1.01 + TINY[dtype], what)


# M, N, K: single ones, groups of 128 and 512 columns not filled, blocks of rows not
# filled, few rows and many, an empty sum
MX_SHAPES = [(1, 1, 1), (1, 16, 128), (2, 17, 129), (5, 100, 200), (16, 64, 512), (17, 33, 640), (33, 50, 2050),
             (64, 256, 1024), (65, 255, 96), (130, 130, 1153), (128, 256, 4096), (257, 384, 768),
             (300, 520, 999), (512, 512, 2560), (3, 40, 0), (1, 1000, 8192), (31, 4100, 300),
             (700, 72, 5000), (1100, 1032, 384), (4, 200, 4096), (3, 70, 5000), (4, 30, 4097),
             (20, 300, 5000), (50, 40, 9000), (64, 24, 6000), (90, 500, 16384)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("xf,wf", [("e2m1", "e2m1"), ("e4m3", "e2m1"), ("e4m3", "e4m3"), ("e2m1", "e4m3")])
@pytest.mark.parametrize("shape", MX_SHAPES)
def test_mx_linear(shape, xf, wf, dtype):
    M, N, K = shape
    act = ACTS[(M + N + K) % len(ACTS)]
    say("mx linear", shape, xf, wf, dtype, act)
    x = rand((M, K), dtype, 1)
    w = pg.pmx_quantize(rand((N, K), dtype, 2, std=max(K, 1) ** -0.5), wf)
    b, r = rand((N,), dtype, 3, std=0.3), rand((M, N), dtype, 4, pitch=N + 3)
    q = pg.pmx_quantize(x, xf)
    y = pg.pmx_linear(q, w, bias=b, residual=r, act=act)
    assert y.dtype is dtype
    check_mx(y, q, w, b, r, act, dtype, "y")
    # quantised within the call: the same bits; again: the same bits
    out = torch.full((M, N + 1), float("nan"), dtype=dtype, device="cuda")
    same = pg.pmx_linear(x, w, bias=b, residual=r, act=act, format=xf, out=out[:, :N])
    again = pg.pmx_linear(q, w, bias=b, residual=r, act=act)
    torch.cuda.synchronize()
    assert torch.equal(same, y) and torch.equal(again, y)
    assert out[:, N].isnan().all()
    plain = pg.pmx_linear(q, w, dtype=dtype)
    check_mx(plain, q, w, None, None, "none", dtype, "plain")
    assert pg.pmx_linear(q, w, bias=b, residual=r, act=act, out=r) is r
    torch.cuda.synchronize()
    assert torch.equal(r, y)


@pytest.mark.parametrize("xf,wf", [("e2m1", "e2m1"), ("e4m3", "e2m1"), ("e4m3", "e4m3"), ("e2m1", "e4m3")])
@pytest.mark.parametrize("shape", [(4100, 4110, 1200), (8200, 2040, 130), (300, 20000, 4224)])
def test_mx_linear_many_tiles(shape, xf, wf):
    """More 256-row tiles than compute units, edges and steps that fill nothing:
    every output against the product of the same values in fp32, some rows
    against binary64."""
    M, N, K = shape
    dtype = torch.bfloat16 if M > 5000 else torch.float16
    say("mx linear, many tiles", shape, xf, wf)
    x, w = rand((M, K), dtype, 1), rand((N, K), dtype, 2, std=K ** -0.5)
    q, w = pg.pmx_quantize(x, xf), pg.pmx_quantize(w, wf)
    b, r = rand((N,), dtype, 3, std=0.3), rand((M, N), dtype, 4)
    y = pg.pmx_linear(q, w, bias=b, residual=r, act="gelu")
    rows = np.unique(np.concatenate([[0, 15, 16, 127, 128, 255, 256, M - 1, M - 2],
                                     np.random.default_rng(1).integers(0, M, 20)]))
    some = pg.MxMatrix(q.codes[rows].contiguous(), q.scales[rows].contiguous(), K, xf)
    check_mx(y[rows], some, w, b, r[rows], "gelu", dtype, "rows")
    X = torch.from_numpy(values_of(q)).float().cuda()
    W = torch.from_numpy(values_of(w)).float().cuda()
    Z = X @ W.t() + b.float()
    ref = torch.nn.functional.gelu(Z) + r.float()
    # as in check_mx, the reference's own fp32 sum added; |products| by their norms
    size = X.norm(dim=1)[:, None] * W.norm(dim=1)[None, :]
    drop = 0.0
    if "e4m3" in (xf, wf):
        drop = -(-K // 128) * 2.0 ** -10 * X.abs().amax(dim=1)[:, None] * W.abs().amax(dim=1)[None, :]
    bound = UNIT[dtype] * ref.abs() + 1.13 * (2 * (K + 16) * 2.0 ** -23 * size + drop) \
        + 2.0 ** -17 * (Z.abs() + r.float().abs() + ref.abs()) + TINY[dtype]
    bad = ~((y.float() - ref).abs() <= bound)
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[0].tolist())


def test_mx_linear_wide_scales():
    """Scales over their whole range in one product: the ends of fp32 and NaN."""
    K, N = 256, 40
    rng = np.random.default_rng(5)
    codes = torch.from_numpy(rng.integers(0, 256, (N, 128)).astype(np.uint8)).cuda()
    scales = np.full((N, 16), 127, np.uint8)
    scales[:, :8] = rng.integers(100, 150, (N, 8))
    scales[3, 2] = 255
    scales[4, :8] = 0
    w = pg.MxMatrix(codes, torch.from_numpy(scales).cuda(), K, "e2m1")
    x = pg.pmx_quantize(rand((20, K), torch.bfloat16, 6), "e2m1")
    y = pg.pmx_linear(x, w)
    assert f64(y[:, 3]).shape == (20,) and np.isnan(f64(y[:, 3])).all()
    keep = [n for n in range(N) if n != 3]
    X, W = values_of(x), values_of(w)[keep]
    bound = 2.0 ** -8 * np.abs(X @ W.T) + 300 * 2.0 ** -23 * (np.abs(X) @ np.abs(W).T) + 2.0 ** -126
    near(y[:, keep], X @ W.T, bound, "wide scales")


def test_mx_linear_nan_rows():
    """A row of x with an infinity gives NaN in its own row alone."""
    x = rand((70, 300), torch.float16, 8)
    x[5, 7] = float("inf")
    w = pg.pmx_quantize(rand((90, 300), torch.float16, 9), "e2m1")
    for f in FORMATS:
        y = f64(pg.pmx_linear(x, w, format=f))
        assert np.isnan(y[5]).all() and np.isfinite(np.delete(y, 5, axis=0)).all()


# ---- sampling ----------------------------------------------------------------------

def sample_exact(l, u, t=1.0, k=0, p=1.0, m=0.0):
    """(token, logprob) of one row in binary64."""
    if np.isnan(l).any() or (l == -np.inf).all():
        return -1, np.nan
    order = np.argsort(-l, kind="stable")
    if not t > 0:
        return order[0], 0.0
    v = l[order]
    with np.errstate(all="ignore"):
        w = np.where(v == v[0], 1.0, np.exp((v - v[0]) / t))
    w = np.where(np.isfinite(v) | (v == v[0]), w, 0.0)
    n = np.count_nonzero(w >= 2.0 ** -41)
    if k > 0:
        n = min(n, k)
    c = np.cumsum(w)
    if p < 1:
        n = min(n, 1 + int(np.searchsorted(c[:n], p * c[n - 1], side="left")))
    n = max(1, min(n, int(np.count_nonzero(w >= min(m, 1.0)))))
    at = min(int(np.searchsorted(c[:n], u * c[n - 1], side="right")), n - 1)
    return order[at], np.log(w[at] / c[n - 1])


def check_sample(l, u, got, what, t=1.0, k=0, p=1.0, m=0.0):
    tokens, logprobs = (f64(g) for g in got)
    L, U = f64(l), f64(u)
    M = L.shape[0]

    def each(v):
        return f64(v) if isinstance(v, torch.Tensor) else np.full(M, np.float32(v), np.float64)
    T, K, P, Q = each(t), each(k).astype(int), each(p), each(m)
    for i in range(M):
        tok, lp = sample_exact(L[i], U[i], T[i], K[i], P[i], Q[i])
        assert tokens[i] == tok, (what, i, tokens[i], tok, U[i])
        if np.isnan(lp):
            assert np.isnan(logprobs[i])
        else:
            assert abs(logprobs[i] - lp) <= 2.0 ** -22 * (1 + abs(lp)), (what, i, logprobs[i], lp)


def uniform(M, seed):
    u = np.random.default_rng(seed).random(M).astype(np.float32)
    u[0] = 0.0
    if M > 1:
        u[1] = 1 - 2.0 ** -24
    return torch.from_numpy(u).cuda()


SETTINGS = [dict(), dict(t=0.7, k=1), dict(t=0.0), dict(k=40), dict(p=0.9), dict(m=0.05),
            dict(t=1.3, k=200, p=0.8, m=0.01), dict(t=0.05, p=0.5), dict(t=50.0, k=3000, p=0.99),
            dict(p=0.0), dict(m=1.0), dict(k=10 ** 6), dict(k=512), dict(k=513, p=0.95),
            dict(t=0.02, k=30), dict(t=20.0, p=0.999), dict(p=0.97, m=0.3), dict(t=3.0, k=7, m=0.2)]


@pytest.mark.parametrize("dtype", DTYPES + [torch.float32])
@pytest.mark.parametrize("V", [1, 2, 7, 1000, 4097, 32001, 131072])
def test_sample(V, dtype):
    M = 6
    l = rand((M, V), dtype, V, std=3.0, pitch=V + (V % 3), offset=V % 2)
    u = uniform(M, V)
    for s in SETTINGS:
        say("sample", V, dtype, s)
        got = pg.psample(l, u, temperature=s.get("t", 1.0), top_k=s.get("k", 0), top_p=s.get("p", 1.0),
                         min_p=s.get("m", 0.0))
        check_sample(l, u, got, (V, dtype, s), **s)


@pytest.mark.parametrize("M,V,dtype", [(66, 40000, torch.float32), (65, 33001, torch.float16),
                                       (65, 70003, torch.bfloat16), (65, 16385, torch.bfloat16)])
def test_sample_many_rows(M, V, dtype):
    """Long rows of a workgroup each: kept in LDS and read again."""
    l = rand((M, V), dtype, V, std=3.0, pitch=V + 1)
    u = uniform(M, V)
    for s in (dict(), dict(k=50, p=0.9), dict(p=0.8, m=0.02), dict(k=2000), dict(t=0.0)):
        say("sample, many rows", M, V, dtype, s)
        got = pg.psample(l, u, temperature=s.get("t", 1.0), top_k=s.get("k", 0), top_p=s.get("p", 1.0),
                         min_p=s.get("m", 0.0))
        check_sample(l, u, got, s, **s)
    # ties and crowds
    l[:, ::3] = 2.0
    for s in (dict(), dict(k=V // 2, p=0.9), dict(k=100)):
        got = pg.psample(l, u, top_k=s.get("k", 0), top_p=s.get("p", 1.0))
        check_sample(l, u, got, s, **s)


@pytest.mark.parametrize("M,V", [(300, 1000), (70, 20000), (513, 130)])
def test_sample_settings_by_row(M, V):
    rng = np.random.default_rng(M)
    l = rand((M, V), torch.bfloat16, 17, std=2.5)
    l[:, ::5] = float("-inf")
    t = torch.from_numpy(rng.uniform(0.3, 1.5, M).astype(np.float32))
    t[::7] = 0.0
    k = torch.from_numpy(rng.integers(-1, 60, M).astype(np.int32)).cuda()
    p = torch.from_numpy(rng.uniform(0.5, 1.1, M).astype(np.float32)).cuda()
    m = torch.from_numpy(rng.uniform(-0.05, 0.1, M).astype(np.float32)).cuda()
    t, u = t.cuda(), uniform(M, 3)
    say("sample by row", M, V)
    got = pg.psample(l, u, temperature=t, top_k=k, top_p=p, min_p=m)
    check_sample(l, u, got, "by row", t=t, k=k, p=p, m=m)


@pytest.mark.parametrize("V", [1024, 3000, 100000])
def test_sample_ties(V):
    """Equal logits by index: more of them than are ranked at once, and by
    halves."""
    u = torch.tensor([0.0, 0.25, 0.5, 0.75, 1 - 2.0 ** -24], device="cuda")
    l = torch.zeros(5, V, dtype=torch.float32, device="cuda")
    say("ties", V)
    got = pg.psample(l, u)
    check_sample(l, u, got, "equal")
    for k in (1, 5, V // 2 + 1):
        check_sample(l, u, pg.psample(l, u, top_k=k), "equal, k", k=k)
    check_sample(l, u, pg.psample(l, u, top_p=0.5), "equal, p", p=0.5)
    l[:, ::2] = -1.0
    l[:, 5] = -0.0
    check_sample(l, u, pg.psample(l, u, top_k=V // 2 + 7), "two values", k=V // 2 + 7)


@pytest.mark.parametrize("V", [8200, 32768, 65537, 100001])
@pytest.mark.parametrize("dtype", DTYPES)
def test_sample_long_rows_of_16_bits(V, dtype):
    """Rows that share few values: both zeros, masked logits, infinities, more equal
    ones than 16 bits count, one alone among them; top-k of many and by row."""
    M, rng = 66, np.random.default_rng(V)
    l = torch.from_numpy((rng.integers(-40, 41, (M, V)) / 8.0).astype(np.float32))
    l[0] = 0.0
    l[1] = 0.0
    l[1, ::2] = -0.0
    l[2] = -3.0
    l[2, V - 1] = -2.5
    l[3] = float("-inf")
    l[3, [5, V - 2]] = -60000.0
    l[4, : V - 3] = float("-inf")
    l[5, 7] = float("inf")
    l[6, V // 2] = float("nan")
    l[7] = float("-inf")
    l[8] = -1.0
    l[8, 1000:1003] = 20.0
    l[9, :] = torch.from_numpy(rng.standard_normal(V).astype(np.float32)) * 1e-7
    l[10, 70:] = 1.0
    l[10, :70] = 1.5
    l[11:40] = torch.from_numpy(rng.standard_normal((29, V)).astype(np.float32)) * 4
    l[20:60, ::7] = float("-inf")
    l = l.to(dtype).cuda()
    u = uniform(M, V)
    u[2:11] = 0.7
    for s in (dict(), dict(k=600), dict(k=V // 2, p=0.9), dict(t=8.0, p=0.7, m=0.3), dict(t=0.0),
              dict(k=V - 1, m=0.02), dict(t=1e-3, k=5000)):
        say("long rows", V, dtype, s)
        got = pg.psample(l, u, temperature=s.get("t", 1.0), top_k=s.get("k", 0), top_p=s.get("p", 1.0),
                         min_p=s.get("m", 0.0))
        check_sample(l, u, got, s, **s)
    k = torch.from_numpy(rng.integers(-1, V, M).astype(np.int32)).cuda()
    k[::3] = torch.from_numpy(rng.integers(1, 90, 22).astype(np.int32)).cuda()
    p = torch.from_numpy(rng.uniform(0.2, 1.1, M).astype(np.float32)).cuda()
    check_sample(l, u, pg.psample(l, u, top_k=k, top_p=p), "by row", k=k, p=p)


def test_sample_crowded():
    """Far more logits next to each other than are ranked at once, all distinct
    or nearly so, at the top and behind a peak."""
    rng = np.random.default_rng(9)
    V = 60000
    rows = [rng.permutation(V) * 2.0 ** -24 + 1.0, rng.integers(0, 5000, V) * 2.0 ** -20 + 4.0,
            rng.random(V) * 1e-3, np.where(np.arange(V) == 777, 3.0, rng.random(V) * 1e-4),
            rng.random(V) * 1e-38, np.where(rng.random(V) < 0.5, 1e30, 1e30 * (1 - 2.0 ** -23))]
    l = torch.from_numpy(np.stack(rows).astype(np.float32)).cuda()
    u = uniform(len(rows), 10)
    for s in (dict(), dict(k=12345), dict(p=0.7), dict(k=50000, p=0.3, m=0.5), dict(t=1e-3, p=0.9)):
        say("crowded", s)
        got = pg.psample(l, u, temperature=s.get("t", 1.0), top_k=s.get("k", 0), top_p=s.get("p", 1.0),
                         min_p=s.get("m", 0.0))
        check_sample(l, u, got, s, **s)


def test_sample_special_rows():
    inf, nan = float("inf"), float("nan")
    l = torch.zeros(9, 500)
    l[0] = -inf
    l[1, 3] = nan
    l[2, [7, 9]] = inf
    l[3] = -inf
    l[3, 499] = -5.0
    l[4] = torch.linspace(-3e38, 3e38, 500)
    l[5, 100:] = -inf
    l[6] = torch.linspace(0, 1e-40, 500)
    l[7, 250] = 88.0
    l = l.cuda()
    u = torch.tensor([0.5, 0.5, 0.6, 0.9, 0.3, 0.999, 0.4, 0.7, 0.2], device="cuda")
    for t in (1.0, 0.0, 1e-30, 1e30, inf):
        say("special rows", t)
        check_sample(l, u, pg.psample(l, u, temperature=t), t, t=t)
        check_sample(l, u, pg.psample(l, u, temperature=t, top_p=0.5), t, t=t, p=0.5)
    tokens, logprobs = pg.psample(l.half(), u)
    assert int(tokens[0]) == -1 and int(tokens[1]) == -1 and bool(logprobs[0].isnan())
    assert int(tokens[3]) == 499 and int(tokens[5]) < 100
    # random numbers outside [0, 1)
    bad = torch.tensor([nan, -1.0, 1.0, 2.0, inf], device="cuda")
    x = torch.arange(5.0, device="cuda").repeat(5, 1)
    assert pg.psample(x, bad)[0].tolist() == [4, 4, 0, 0, 0]


def test_sample_frequencies():
    """Evenly spread random numbers draw each token as often as it is probable:
    to within one of n p, since the tokens' stretches of [0, 1) do not
    overlap."""
    n = 4096
    l = torch.tensor([0.1, 2.0, -1.0, 0.7, 0.7, -3.0], device="cuda").repeat(n, 1)
    u = ((torch.arange(n, dtype=torch.float64) + 0.5) / n).float().cuda()
    tokens = pg.psample(l, u)[0].cpu()
    p = torch.softmax(l[0].double().cpu(), 0)
    counts = torch.bincount(tokens, minlength=6).double()
    assert ((counts - n * p).abs() <= 1.0).all()
