"""Calls of the norm, the microscaled operators and sampling that their other GPU
tests do not make, against plain formulas in binary64 on the CPU.  Tolerances as
derived in test_serving_gpu.py."""
import numpy as np
import pytest

import software_pipelined_tiled_pgemm_amd as pg
from .test_serving_gpu import (DTYPES, NORM_SHAPES, TINY, UNIT, check_mx, check_sample, f64, near,
                              norm_grad_exact, rand, say, uniform)

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", NORM_SHAPES + [(5000, 64), (2100, 520), (700, 4100), (300, 17000),
                                                 (130, 33000)])
def test_norm_backward_at_the_sum(shape, dtype):
    """The gradient at x + residual as the forward pass normed it, in fp32: no rounding
    but the results' own."""
    M, D = shape
    odd = (M + D) % 2
    say("norm backward at the sum", shape, dtype)
    dy = rand(shape, dtype, 11, pitch=D + 3 if odd else None)
    x = rand(shape, dtype, 12, std=3.0, pitch=None if odd else D + 8)
    r = rand(shape, dtype, 15, std=2.0, pitch=D + 5 if odd else None, offset=odd)
    w, dh = rand((D,), dtype, 13), rand(shape, dtype, 14, pitch=D + 1)
    kept = r.clone()
    dx, dw = pg.prmsnorm_bwd(dy, x, w, eps=1e-5, dh=dh, residual=r)
    DX, size, DW, wsize = norm_grad_exact(f64(dy), f64(x) + f64(r), f64(w), f64(dh), 1e-5)
    u = UNIT[dtype]
    near(dx, DX, u * np.abs(DX) + 2.0 ** -16 * size + TINY[dtype], "dx")
    near(dw, DW, u * np.abs(DW) + (2.0 ** -17 + M * 2.0 ** -24) * wsize + TINY[dtype], "dw")
    # each alone, in place of dh; without weight
    only, none = pg.prmsnorm_bwd(dy, x, w, eps=1e-5, dh=dh, needs=(True, False), dx=dh, residual=r)
    assert none is None and only is dh
    none, only = pg.prmsnorm_bwd(dy, x, w, eps=1e-5, needs=(False, True), residual=r)
    torch.cuda.synchronize()
    assert none is None and torch.equal(only, dw) and torch.equal(dh, dx) and torch.equal(kept, r)
    plain, none = pg.prmsnorm_bwd(dy, x, eps=1e-5, residual=r)
    DX, size, _, _ = norm_grad_exact(f64(dy), f64(x) + f64(r), None, None, 1e-5)
    assert none is None
    near(plain, DX, u * np.abs(DX) + 2.0 ** -16 * size + TINY[dtype], "plain dx")
    # a zero residual: the other form's bits
    a = pg.prmsnorm_bwd(dy, x, w, eps=1e-5, residual=torch.zeros_like(r))
    for p, q in zip(a, pg.prmsnorm_bwd(dy, x, w, eps=1e-5)):
        assert torch.equal(p, q)


def test_norm_backward_at_a_sum_beyond_the_type():
    """x + residual past float16's largest, and squares outside fp32's range."""
    D = 300
    x, r = rand((3, D), torch.float16, 1).cpu(), rand((3, D), torch.float16, 2).cpu()
    x[1], r[1] = 60000.0, x[1].sign() * 50000.0
    r[2] = -x[2]
    dy = rand((3, D), torch.float16, 3)
    dx, dw = pg.prmsnorm_bwd(dy, x.cuda(), torch.ones(D, device="cuda").half(), eps=1e-5,
                             residual=r.cuda())
    S = x.double().numpy() + r.double().numpy()
    DX, size, DW, wsize = norm_grad_exact(f64(dy), S, None, None, 1e-5)
    near(dx, DX, 2.0 ** -11 * np.abs(DX) + 2.0 ** -16 * size + TINY[torch.float16], "dx")
    near(dw, DW, 2.0 ** -11 * np.abs(DW) + 2.0 ** -16 * wsize + TINY[torch.float16], "dw")
    bf = torch.bfloat16
    scale = torch.tensor([1e30, 1e37, 1e-30, 1.0])[:, None]
    x, r = ((rand((4, D), bf, s).float().cpu() * scale).to(bf) for s in (4, 5))
    dy = rand((4, D), bf, 6)
    dx, dw = pg.prmsnorm_bwd(dy, x.cuda(), torch.ones(D, device="cuda").to(bf), eps=1e-38,
                             residual=r.cuda())
    S = x.double().numpy() + r.double().numpy()
    DX, size, DW, wsize = norm_grad_exact(f64(dy), S, None, None, 1e-38)
    near(dx, DX, 2.0 ** -8 * np.abs(DX) + 2.0 ** -15 * size + 2.0 ** -133, "dx")
    near(dw, DW, 2.0 ** -8 * np.abs(DW) + 2.0 ** -16 * wsize, "dw")


def test_norm_backward_at_the_sum_refusals_and_graph():
    x = torch.randn(9, 64, device="cuda").half()
    w = torch.ones(64, device="cuda").half()
    for bad in (x[:3], x.bfloat16(), x.cpu(), x.t()):
        with pytest.raises((TypeError, ValueError)):
            pg.prmsnorm_bwd(x, x, w, residual=bad)
    with pytest.raises(pg.PgemmError):
        pg.prmsnorm_bwd(x, x, w, residual=x.clone(), dx=x)
    r, dy = torch.randn_like(x), torch.randn_like(x)
    with pytest.raises(pg.PgemmError):
        pg.prmsnorm_bwd(dy, x, w, residual=r, dx=r)
    pg.prmsnorm_bwd(dy, x, w, residual=r)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = pg.prmsnorm_bwd(dy, x, w, residual=r)
    for _ in range(3):
        r.copy_(torch.randn_like(r))
        g.replay()
        torch.cuda.synchronize()
        for a, b in zip(out, pg.prmsnorm_bwd(dy, x, w, residual=r)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("M,V,dtype", [(3, 500, torch.float32), (3, 40000, torch.float32),
                                       (66, 500, torch.bfloat16), (66, 40000, torch.bfloat16),
                                       (70, 40000, torch.float32), (2, 40000, torch.bfloat16)])
def test_sample_differences_beyond_fp32(M, V, dtype):
    """Finite logits further apart than fp32's largest, at temperatures that leave them
    weight: for each way that rows go."""
    l = torch.empty(M, V)
    l[0] = torch.linspace(-3e38, 3e38, V)
    l[1:] = torch.from_numpy(np.random.default_rng(V).uniform(-3.3e38, 3.3e38, (M - 1, V))).float()
    l[1, ::2] = -3e38
    l[1, 1::2] = 3e38
    l = l.to(dtype).cuda()
    u = uniform(M, V + 1)
    u[:M] = torch.tensor(([0.9, 0.999, 1 - 2.0 ** -24] + u[3:].tolist())[:M])
    for s in (dict(t=1e36), dict(t=1e37), dict(t=1.3e37), dict(t=1e38), dict(t=3e38, k=V // 2 + 3),
              dict(t=1e38, k=100), dict(t=2e38, p=0.9), dict(t=1e38, p=0.999, m=0.01)):
        say("differences beyond fp32", M, V, dtype, s)
        got = pg.psample(l, u, temperature=s["t"], top_k=s.get("k", 0), top_p=s.get("p", 1.0),
                         min_p=s.get("m", 0.0))
        check_sample(l, u, got, s, **s)


@pytest.mark.parametrize("M,V,dtype", [(6, 2, torch.float32), (6, 300, torch.float16),
                                       (6, 40000, torch.float32), (66, 40000, torch.bfloat16)])
def test_sample_numbers_outside_the_interval(M, V, dtype):
    """A random number of 1 and more draws as the largest float32 below 1 does, not
    the least likely token; one below 0, and NaN, as 0 does."""
    l = torch.full((M, V), -25.0, dtype=dtype)  # 1.4e-11 of the largest each
    l[:, V // 2] = 0.0
    l = l.cuda()
    below = 1 - 2.0 ** -24
    u = torch.tensor([1.0, 2.0, float("inf"), -1.0, float("nan"), float("-inf")] * (M // 6), device="cuda")
    near_u = torch.tensor([below, below, below, 0.0, 0.0, 0.0] * (M // 6), device="cuda")
    for s in (dict(), dict(top_k=V), dict(top_k=min(V, 40)), dict(top_p=0.9999999)):
        say("numbers outside", M, V, dtype, s)
        got, want = pg.psample(l, u, **s), pg.psample(l, near_u, **s)
        if V <= 300:  # all of the others together are less than 2^-24 of the row
            assert (want[0] == V // 2).all()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), s


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(1, 16384), (5, 16385), (130, 16392), (70, 20481), (65, 24576),
                                   (64, 32768), (3, 32775)])
def test_norm_backward_wide(shape, dtype):
    """Rows on both sides of what the backward pass holds in registers."""
    M, D = shape
    say("norm backward, wide", shape, dtype)
    dy, h = rand(shape, dtype, 1, pitch=D + D % 2), rand(shape, dtype, 2, std=3.0, pitch=D + 3)
    w, dh = rand((D,), dtype, 3), rand(shape, dtype, 4)
    dx, dw = pg.prmsnorm_bwd(dy, h, w, eps=1e-5, dh=dh)
    DX, size, DW, wsize = norm_grad_exact(f64(dy), f64(h), f64(w), f64(dh), 1e-5)
    u = UNIT[dtype]
    near(dx, DX, u * np.abs(DX) + 2.0 ** -16 * size + TINY[dtype], "dx")
    near(dw, DW, u * np.abs(DW) + (2.0 ** -17 + M * 2.0 ** -24) * wsize + TINY[dtype], "dw")
    assert pg.prmsnorm_bwd(dy, h, w, eps=1e-5, dh=dh, needs=(True, False), dx=dh)[0] is dh
    torch.cuda.synchronize()
    assert torch.equal(dh, dx)


@pytest.mark.parametrize("D", [2056, 2051])
def test_norm_past_the_caches(D):
    """Calls larger than the memory-side cache, which store and read past it, give the
    bits of calls on parts of their rows."""
    M, dtype = 33000, torch.float16
    say("norm past the caches", M, D)
    x, r, dy, dh = (torch.randn(M, D, device="cuda", dtype=dtype) for _ in range(4))
    w = torch.randn(D, device="cuda").to(dtype)
    parts = [slice(a, a + 5000) for a in range(0, M, 5000)]
    h = torch.empty_like(x)
    y = pg.prmsnorm(x, w, residual=r, h=h)
    h8 = torch.empty_like(x)
    m = pg.prmsnorm(x, w, residual=r, h=h8, format="e4m3")
    v = pg.pmx_dequantize(m, dtype=dtype)
    dx, dw = pg.prmsnorm_bwd(dy, h, w, dh=dh)
    sx, sw = pg.prmsnorm_bwd(dy, x, w, dh=dh, residual=r)
    for p in parts:
        hp = torch.empty_like(x[p])
        assert torch.equal(y[p], pg.prmsnorm(x[p], w, residual=r[p], h=hp)) and torch.equal(h[p], hp)
        q = pg.prmsnorm(x[p], w, residual=r[p], format="e4m3")
        assert torch.equal(m.codes[p], q.codes) and torch.equal(h8[p], hp)
        assert torch.equal(v[p], pg.pmx_dequantize(q, dtype=dtype))
        assert torch.equal(dx[p], pg.prmsnorm_bwd(dy[p], h[p], w, dh=dh[p])[0])
        assert torch.equal(sx[p], pg.prmsnorm_bwd(dy[p], x[p], w, dh=dh[p], residual=r[p])[0])


@pytest.mark.parametrize("xf,wf", [("e2m1", "e2m1"), ("e4m3", "e2m1"), ("e4m3", "e4m3"), ("e2m1", "e4m3")])
@pytest.mark.parametrize("shape", [(1, 65500, 1100), (3, 32700, 2050), (16, 32700, 1153), (17, 16400, 4096),
                                   (33, 9001, 8192), (64, 16300, 640), (64, 20000, 0), (2, 131000, 129)])
def test_mx_linear_few_rows_of_many_columns(shape, xf, wf):
    """Fewer rows than a tile has, by so many columns that they go by tiles."""
    M, N, K = shape
    dtype = torch.bfloat16 if M % 2 else torch.float16
    say("mx linear, few rows of many columns", shape, xf, wf)
    x = rand((M, K), dtype, 1)
    w = pg.pmx_quantize(rand((N, K), dtype, 2, std=max(K, 1) ** -0.5), wf)
    b, r = rand((N,), dtype, 3, std=0.3), rand((M, N), dtype, 4, pitch=N + 3)
    q = pg.pmx_quantize(x, xf)
    out = torch.full((M + 2, N + 1), 7.0, dtype=dtype, device="cuda")
    y = pg.pmx_linear(q, w, bias=b, residual=r, act="silu", out=out[:M, :N])
    check_mx(y, q, w, b, r, "silu", dtype, "y")
    assert (out[M:] == 7).all() and (out[:, N] == 7).all()
    # quantised within the call; in place of the residual
    assert torch.equal(pg.pmx_linear(x, w, bias=b, residual=r, act="silu", format=xf), y)
    assert pg.pmx_linear(q, w, bias=b, residual=r, act="silu", out=r) is r
    torch.cuda.synchronize()
    assert torch.equal(r, y)


@pytest.mark.parametrize("M", [15, 16, 17, 40])
@pytest.mark.parametrize("V,dtype", [(9001, torch.float32), (50000, torch.float32), (40001, torch.bfloat16),
                                     (33000, torch.float16)])
def test_sample_on_both_sides_of_pieces(M, V, dtype):
    """As many long rows as are cut into pieces, and more."""
    l = rand((M, V), dtype, V, std=3.0, pitch=V + 1)
    l[M - 1, ::2] = 3.0
    l[M - 2] = float("-inf")
    u = uniform(M, M)
    for s in (dict(), dict(k=50, p=0.95), dict(p=0.9, m=0.01), dict(k=1000), dict(t=8.0, p=0.9),
              dict(t=0.0)):
        say("both sides of pieces", M, V, dtype, s)
        got = pg.psample(l, u, temperature=s.get("t", 1.0), top_k=s.get("k", 0), top_p=s.get("p", 1.0),
                         min_p=s.get("m", 0.0))
        check_sample(l, u, got, s, **s)
