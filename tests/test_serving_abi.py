"""Argument checks of the norm, the microscaled matrices and sampling that need
no GPU: every refusal is decided on the host before any HIP call."""
import os

import pytest

import software_pipelined_tiled_pgemm_amd as pg
from software_pipelined_tiled_pgemm_amd import _lib

EINVAL, EUNSUP, OK = pg.PGEMM_EINVAL, pg.PGEMM_EUNSUPPORTED, pg.PGEMM_OK
F16, BF16, F32 = 0, 1, 2
NONE, E2M1, E4M3 = -1, 0, 1
NAN, INF = float("nan"), float("inf")
# Fake, never dereferenced addresses, 256 MiB apart.
X, R, W, H, Y, S, WS, Z = (0x10000000 * (i + 1) for i in range(8))


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(_lib.LIB_PATH):
        from software_pipelined_tiled_pgemm_amd import build
        build.build()
    return pg.lib()


def test_pitches(L):
    assert [L.pmx_codes_pitch(E2M1, n) for n in (0, 1, 128, 129, 4096)] == [0, 64, 64, 128, 2048]
    assert [L.pmx_codes_pitch(E4M3, n) for n in (0, 1, 128, 129, 4096)] == [0, 128, 128, 256, 4096]
    assert [L.pmx_scales_pitch(n) for n in (0, 1, 512, 513, 4096)] == [0, 16, 16, 32, 128]
    assert L.pmx_codes_pitch(E2M1, -1) == EINVAL and L.pmx_scales_pitch(-1) == EINVAL
    assert L.pmx_codes_pitch(2, 8) == EUNSUP and L.pmx_codes_pitch(NONE, 8) == EUNSUP
    assert L.pmx_codes_pitch(E4M3, 1 << 22) == EUNSUP and L.pmx_scales_pitch(1 << 22) == EUNSUP


def norm(L, dtype=F16, x=X, ldx=64, r=R, ldr=64, w=W, h=H, ldh=64, fmt=NONE, y=Y, ldy=64, s=None,
         lds=0, M=4, D=64, eps=1e-6):
    return L.prmsnorm(dtype, x, ldx, r, ldr, w, h, ldh, fmt, y, ldy, s, lds, M, D, eps, None)


@pytest.mark.parametrize("change,expected", [
    (dict(M=-1), EINVAL), (dict(D=-1), EINVAL), (dict(x=None), EINVAL), (dict(y=None), EINVAL),
    (dict(ldx=63), EINVAL), (dict(ldr=63), EINVAL), (dict(ldh=63), EINVAL), (dict(ldy=63), EINVAL),
    (dict(eps=-1e-6), EINVAL), (dict(eps=NAN), EINVAL), (dict(eps=INF), EINVAL),
    (dict(dtype=F32), EUNSUP), (dict(dtype=-1), EUNSUP), (dict(fmt=2), EUNSUP),
    (dict(fmt=-2), EUNSUP), (dict(x=X + 1), EUNSUP), (dict(w=W + 1), EUNSUP),
    (dict(D=1 << 22, ldx=1 << 22), EUNSUP), (dict(M=1 << 31), EUNSUP),
    (dict(y=W), EINVAL), (dict(h=W), EINVAL), (dict(y=H), EINVAL), (dict(y=H + 2), EINVAL),
    (dict(y=X + 2), EINVAL), (dict(y=X, ldy=80), EINVAL), (dict(h=R + 4), EINVAL),
    (dict(y=X, h=X), EINVAL),
    (dict(fmt=E4M3, ldy=128, s=None), EINVAL), (dict(fmt=E4M3, ldy=64, s=S, lds=16), EINVAL),
    (dict(fmt=E4M3, ldy=128, s=S, lds=8), EINVAL), (dict(fmt=E4M3, ldy=136, s=S, lds=16), EUNSUP),
    (dict(fmt=E4M3, ldy=128, s=S, lds=20), EUNSUP), (dict(fmt=E4M3, ldy=128, s=S + 4, lds=16), EUNSUP),
    (dict(fmt=E4M3, y=Y + 8, ldy=128, s=S, lds=16), EUNSUP),
    (dict(fmt=E4M3, ldy=128, s=Y + 16, lds=16), EINVAL), (dict(fmt=E4M3, ldy=128, s=X, lds=16), EINVAL),
    (dict(fmt=E2M1, y=X, ldy=64, s=S, lds=16), EINVAL), (dict(fmt=E2M1, y=H, s=S, lds=16), EINVAL),
    (dict(M=0), OK), (dict(D=0), OK), (dict(M=0, x=None, y=None), OK),
])
def test_norm_checks(L, change, expected):
    assert norm(L, **change) == expected


def norm_bwd(L, dtype=F16, dy=X, lddy=64, h=H, ldh=64, w=W, dh=R, lddh=64, dx=Y, lddx=64, dw=Z, M=4,
             D=64, eps=1e-6, ws=WS, nws=1 << 20):
    return L.prmsnorm_bwd(dtype, dy, lddy, h, ldh, w, dh, lddh, dx, lddx, dw, M, D, eps, ws, nws, None)


@pytest.mark.parametrize("change,expected", [
    (dict(M=-1), EINVAL), (dict(D=-1), EINVAL), (dict(dy=None), EINVAL), (dict(h=None), EINVAL),
    (dict(lddy=63), EINVAL), (dict(ldh=63), EINVAL), (dict(lddh=63), EINVAL), (dict(lddx=63), EINVAL),
    (dict(eps=NAN), EINVAL), (dict(dtype=F32), EUNSUP), (dict(dy=X + 1), EUNSUP),
    (dict(dx=X), EINVAL), (dict(dx=H), EINVAL), (dict(dx=W), EINVAL), (dict(dx=R + 2), EINVAL),
    (dict(dw=X + 64), EINVAL), (dict(dw=R), EINVAL), (dict(dw=W), EINVAL), (dict(dx=Z), EINVAL),
    (dict(ws=None, nws=0), EINVAL), (dict(nws=16), EINVAL), (dict(ws=WS + 8), EUNSUP),
    (dict(ws=X), EINVAL), (dict(ws=Z), EINVAL),
    (dict(D=0), OK), (dict(dx=None, dw=None, dy=None), OK),
])
def test_norm_bwd_checks(L, change, expected):
    assert norm_bwd(L, **change) == expected


def test_norm_bwd_workspace(L):
    need = L.prmsnorm_bwd_workspace_bytes(F16, 4, 64, 1, 1)
    assert 0 < need <= 1 << 20
    assert L.prmsnorm_bwd_workspace_bytes(F16, 4, 64, 1, 0) == 0
    assert L.prmsnorm_bwd_workspace_bytes(F16, 4, 0, 1, 1) == 0
    assert L.prmsnorm_bwd_workspace_bytes(F16, -1, 64, 1, 1) == EINVAL
    assert L.prmsnorm_bwd_workspace_bytes(7, 4, 64, 1, 1) == EUNSUP
    assert norm_bwd(L, nws=need - 1) == EINVAL


def quantize(L, dtype=BF16, x=X, ldx=200, fmt=E2M1, c=Y, ldc=128, s=S, lds=16, M=4, K=200):
    return L.pmx_quantize(dtype, x, ldx, fmt, c, ldc, s, lds, M, K, None)


def dequantize(L, dtype=BF16, x=X, ldx=200, fmt=E2M1, c=Y, ldc=128, s=S, lds=16, M=4, K=200):
    return L.pmx_dequantize(fmt, c, ldc, s, lds, dtype, x, ldx, M, K, None)


@pytest.mark.parametrize("call", [quantize, dequantize])
@pytest.mark.parametrize("change,expected", [
    (dict(M=-1), EINVAL), (dict(K=-1), EINVAL), (dict(x=None), EINVAL), (dict(c=None), EINVAL),
    (dict(s=None), EINVAL), (dict(ldx=199), EINVAL), (dict(ldc=112), EINVAL), (dict(lds=0), EINVAL),
    (dict(fmt=NONE), EUNSUP), (dict(fmt=3), EUNSUP), (dict(dtype=F32), EUNSUP),
    (dict(fmt=E4M3), EINVAL), (dict(ldc=136), EUNSUP), (dict(lds=24), EUNSUP), (dict(c=Y + 8), EUNSUP),
    (dict(s=S + 8), EUNSUP), (dict(x=X + 1), EUNSUP), (dict(c=X), EINVAL), (dict(s=X + 16), EINVAL),
    (dict(K=(1 << 22) - 64, ldx=(1 << 22) - 64, ldc=1 << 21, lds=1 << 17), EUNSUP),
    (dict(M=0), OK), (dict(K=0), OK),
])
def test_quantize_checks(L, call, change, expected):
    assert call(L, **change) == expected


def test_quantize_outputs_apart(L):
    assert quantize(L, s=Y + 128) == EINVAL


def linear(L, dtype=F16, xf=E4M3, x=X, ldx=128, xs=S, ldxs=16, wf=E2M1, w=W, ldw=64, ws_=Z, ldws=16,
           b=None, r=None, ldr=0, y=Y, ldy=32, M=16, N=32, K=128, act=0, ws=WS, nws=1 << 20):
    return L.pmx_linear(dtype, xf, x, ldx, xs, ldxs, wf, w, ldw, ws_, ldws, b, r, ldr, y, ldy, M, N, K,
                        act, ws, nws, None)


@pytest.mark.parametrize("change,expected", [
    (dict(M=-1), EINVAL), (dict(N=-1), EINVAL), (dict(K=-1), EINVAL),
    (dict(x=None), EINVAL), (dict(w=None), EINVAL), (dict(y=None), EINVAL), (dict(ws_=None), EINVAL),
    (dict(ldx=112), EINVAL), (dict(ldw=48), EINVAL), (dict(ldy=31), EINVAL), (dict(ldws=0), EINVAL),
    (dict(dtype=F32), EUNSUP), (dict(act=5), EUNSUP), (dict(xf=NONE), EUNSUP), (dict(wf=2), EUNSUP),
    (dict(ldw=72), EUNSUP), (dict(ldx=136), EUNSUP), (dict(w=W + 8), EUNSUP), (dict(ws_=Z + 4), EUNSUP),
    (dict(xs=S + 4), EUNSUP), (dict(b=H + 1), EUNSUP), (dict(y=Y + 1), EUNSUP),
    (dict(N=1 << 22, ldy=1 << 22), EUNSUP), (dict(M=1 << 31), EUNSUP), (dict(K=1 << 22), EUNSUP),
    (dict(M=1 << 30), EUNSUP),                        # too many tiles for a launch
    (dict(y=X), EINVAL), (dict(y=S), EINVAL), (dict(y=W), EINVAL), (dict(y=Z), EINVAL),
    (dict(b=Y), EINVAL), (dict(r=Y + 2, ldr=32), EINVAL), (dict(r=R, ldr=31), EINVAL),
    # x in 16 bits, which is quantised into the workspace
    (dict(xs=None, ws=None, nws=0), EINVAL), (dict(xs=None, nws=16), EINVAL),
    (dict(xs=None, ldx=127), EINVAL), (dict(xs=None, x=X + 1), EUNSUP),
    (dict(xs=None, ws=WS + 8), EUNSUP), (dict(xs=None, ws=Y), EINVAL), (dict(xs=None, ws=X), EINVAL),
    (dict(M=0), OK), (dict(N=0), OK),
])
def test_mx_linear_checks(L, change, expected):
    assert linear(L, **change) == expected


def test_mx_linear_workspace(L):
    need = L.pmx_linear_workspace_bytes(F16, E4M3, 1, E2M1, 16, 32, 128)
    assert need > 0 and linear(L, xs=None, nws=need - 1) == EINVAL
    # a token's few values are quantised by the kernel itself
    assert L.pmx_linear_workspace_bytes(F16, E4M3, 1, E2M1, 1, 32, 128) == 0
    assert L.pmx_linear_workspace_bytes(F16, E4M3, 0, E2M1, -4, 32, 128) == EINVAL
    assert L.pmx_linear_workspace_bytes(F16, 5, 0, E2M1, 4, 32, 128) == EUNSUP


def sample(L, dtype=F32, l=X, ld=100, u=R, t=1.0, ts=None, k=0, ks=None, p=1.0, ps=None, m=0.0, ms=None,
           tok=Y, lp=Z, M=4, V=100, ws=WS, nws=1 << 24):
    return L.psample(dtype, l, ld, u, t, ts, k, ks, p, ps, m, ms, tok, lp, M, V, ws, nws, None)


@pytest.mark.parametrize("change,expected", [
    (dict(M=-1), EINVAL), (dict(V=0), EINVAL), (dict(l=None), EINVAL), (dict(u=None), EINVAL),
    (dict(tok=None), EINVAL), (dict(ld=99), EINVAL), (dict(t=-1.0), EINVAL), (dict(t=NAN), EINVAL),
    (dict(p=-0.5), EINVAL), (dict(p=NAN), EINVAL), (dict(m=-0.5), EINVAL), (dict(m=1.5), EINVAL),
    (dict(m=NAN), EINVAL), (dict(dtype=3), EUNSUP), (dict(dtype=-1), EUNSUP),
    (dict(l=X + 2), EUNSUP), (dict(u=R + 2), EUNSUP), (dict(tok=Y + 4), EUNSUP), (dict(ts=H + 1), EUNSUP),
    (dict(V=1 << 22, ld=1 << 22), EUNSUP), (dict(ld=1 << 22), EUNSUP), (dict(M=1 << 31), EUNSUP),
    (dict(tok=X), EINVAL), (dict(lp=R), EINVAL), (dict(tok=H, ks=H), EINVAL), (dict(lp=Y + 8), EINVAL),
    (dict(M=0), OK),
])
def test_sample_checks(L, change, expected):
    assert sample(L, **change) == expected


def test_python_refusals():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        pg.prmsnorm(x)  # not on a device
    with pytest.raises(TypeError):
        pg.prmsnorm(x.float())
    with pytest.raises(ValueError):
        pg.pmx_quantize(x, "e5m2")
    codes, scales = torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(4, 16, dtype=torch.uint8)
    m = pg.MxMatrix(codes, scales, 100, "e2m1")
    assert m.shape == (4, 100) and "e2m1" in repr(m)
    for bad in [(codes, scales, 129, "e2m1"), (codes, scales, 100, "e4m3"),
                (codes, scales[:3], 100, "e2m1"), (codes, scales[:, :4], 100, "e2m1"),
                (codes, scales, -1, "e2m1"), (codes[0], scales, 100, "e2m1")]:
        with pytest.raises(ValueError):
            pg.MxMatrix(*bad)
    with pytest.raises(TypeError):
        pg.MxMatrix(x, scales, 64, "e2m1")
    with pytest.raises(ValueError):
        pg.pmx_dequantize(m)  # not on a device
    with pytest.raises(TypeError):
        pg.pmx_linear(x, codes)
    with pytest.raises(TypeError):
        pg.psample(torch.zeros(2, 5, dtype=torch.int32), torch.zeros(2))
