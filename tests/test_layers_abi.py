"""Argument checks of the layer operators that need no GPU: every refusal is
decided on the host before any HIP call."""
import array
import os

import pytest

import software_pipelined_tiled_pgemm_amd as pg
from software_pipelined_tiled_pgemm_amd import _lib

EINVAL, EUNSUP, OK = pg.PGEMM_EINVAL, pg.PGEMM_EUNSUPPORTED, pg.PGEMM_OK
F16, BF16, F32 = 0, 1, 2
# Fake, never dereferenced addresses, 256 MiB apart.
X, W, B, R, Y, P, WS, Z = (0x10000000 * (i + 1) for i in range(8))


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(_lib.LIB_PATH):
        from software_pipelined_tiled_pgemm_amd import build
        build.build()
    return pg.lib()


def linear(L, dtype=F16, x=X, ldx=64, w=W, ldw=32, bias=None, res=None, ldr=0, y=Y, ldy=32, pre=None,
           ldp=0, M=16, N=32, K=64, act=0, ws=WS, nws=1 << 20):
    return L.plinear(dtype, x, ldx, w, ldw, bias, res, ldr, y, ldy, pre, ldp, M, N, K, act, ws, nws,
                     None)


@pytest.mark.parametrize("change,expected", [
    (dict(M=-1), EINVAL), (dict(N=-1), EINVAL), (dict(K=-1), EINVAL),
    (dict(x=None), EINVAL), (dict(w=None), EINVAL), (dict(y=None), EINVAL),
    (dict(ldx=63), EINVAL), (dict(ldw=31), EINVAL), (dict(ldy=31), EINVAL),
    (dict(res=R, ldr=31), EINVAL), (dict(pre=P, ldp=31), EINVAL),
    (dict(dtype=F32), EUNSUP), (dict(dtype=-1), EUNSUP), (dict(dtype=7), EUNSUP),
    (dict(act=-1), EUNSUP), (dict(act=5), EUNSUP),
    (dict(x=X + 1), EUNSUP), (dict(y=Y + 1), EUNSUP), (dict(bias=B + 1), EUNSUP),
    (dict(ldx=1 << 22), EUNSUP), (dict(K=1 << 22, ldx=1 << 22), EUNSUP),
    (dict(M=1 << 31), EUNSUP), (dict(N=1 << 22, ldw=1 << 22, ldy=1 << 22), EUNSUP),
    (dict(y=X), EINVAL), (dict(y=W + 8), EINVAL), (dict(bias=Y + 4), EINVAL),
    (dict(pre=Y, ldp=32), EINVAL), (dict(pre=X + 64, ldp=32), EINVAL),
    (dict(res=Y + 2, ldr=32), EINVAL), (dict(res=Y, ldr=40), EINVAL),
    (dict(pre=R, ldp=32, res=R, ldr=32), EINVAL),
    (dict(x=X + 2, ws=None, nws=0), EINVAL),          # x has to be padded: a workspace
    (dict(x=X + 2, nws=16), EINVAL),
    (dict(x=X + 2, ws=WS + 8), EUNSUP),
    (dict(x=X + 2, ws=Y), EINVAL),                    # the workspace is y
    (dict(M=0), OK), (dict(N=0), OK), (dict(M=0, x=None, w=None, y=None, ws=None, nws=0), OK),
])
def test_linear_checks(L, change, expected):
    assert linear(L, **change) == expected


def test_linear_bwd_checks(L):
    def call(dtype=F16, dy=X, lddy=32, x=W, ldx=64, w=B, ldw=32, pre=None, ldp=0, add=None, lda=0,
             dx=R, lddx=64, dw=Y, lddw=32, db=P, M=16, N=32, K=64, act=0, ws=WS, nws=1 << 22):
        return L.plinear_bwd(dtype, dy, lddy, x, ldx, w, ldw, pre, ldp, add, lda, dx, lddx, dw, lddw,
                             db, M, N, K, act, ws, nws, None)
    assert call(dy=None) == EINVAL
    assert call(x=None) == EINVAL and call(w=None) == EINVAL
    assert call(act=4) == EINVAL                       # no preact
    assert call(act=9) == EUNSUP
    assert call(dx=X) == EINVAL and call(dw=W) == EINVAL and call(db=B) == EINVAL
    assert call(dx=Y) == EINVAL                        # dx and dw are one
    assert call(add=R + 2, lda=64) == EINVAL           # dx may be add, not meet it
    assert call(add=Y, lda=64) == EINVAL
    assert call(lddx=63) == EINVAL
    assert call(ws=None, nws=0) == EINVAL              # the bias gradient's partial sums
    need = L.plinear_bwd_workspace_bytes(F16, 16, 32, 16, 64, 16, 32, 16, 32, 64, 0, 1, 1, 1)
    assert 0 < need < 1 << 22
    assert call(nws=need - 1) == EINVAL
    assert L.plinear_bwd_workspace_bytes(F16, 16, 32, 16, 64, 16, 32, -1, 32, 64, 0, 1, 1, 1) == EINVAL
    assert L.plinear_bwd_workspace_bytes(F16, 16, 32, 16, 64, 16, 32, 16, 32, 64, 0, 0, 0, 0) == 0


def test_columns_of_one_buffer_do_not_overlap(L):
    """x and y as column ranges of one buffer of pitch 128 are accepted up to
    the next check, overlapping ranges are not."""
    assert linear(L, x=X, ldx=128, y=X + 2 * 64, ldy=128, w=W + 1) == EUNSUP  # reaches w's check
    assert linear(L, x=X, ldx=128, y=X + 2 * 48, ldy=128) == EINVAL
    assert linear(L, x=X, ldx=128, y=X + 2 * 112, ldy=128) == EINVAL          # wraps into the next row


def test_ffn_checks(L):
    def call(dtype=BF16, x=X, ldx=64, wi=W, ldwi=96, wo=B, ldwo=64, res=None, ldr=0, y=Y, ldy=64,
             gu=None, ldgu=0, M=16, D=64, F=48, N=64, act=4, ws=WS, nws=1 << 22):
        return L.pffn(dtype, x, ldx, wi, ldwi, wo, ldwo, res, ldr, y, ldy, gu, ldgu, M, D, F, N, act,
                      ws, nws, None)
    for k in ("M", "D", "F", "N"):
        assert call(**{k: -1}) == EINVAL
    assert call(x=None) == EINVAL and call(wi=None) == EINVAL and call(wo=None) == EINVAL
    assert call(y=None) == EINVAL
    assert call(ldwi=95) == EINVAL and call(gu=P, ldgu=95) == EINVAL
    assert call(F=1 << 21, ldwi=(1 << 22) - 8) == EUNSUP
    assert call(M=1 << 28, F=1 << 10, ldwi=1 << 11) == EUNSUP   # M 2F above 2^37
    assert call(dtype=F32) == EUNSUP and call(act=17) == EUNSUP
    assert call(gu=Y, ldgu=96) == EINVAL and call(gu=X, ldgu=96) == EINVAL
    assert call(y=W) == EINVAL
    assert call(ws=None, nws=0) == EINVAL              # h
    assert call(ws=X) == EINVAL
    assert call(M=0) == OK
    need = L.pffn_workspace_bytes(BF16, 16, 64, 16, 96, 16, 64, 16, 64, 48, 64)
    assert need >= 16 * 48 * 2 and call(nws=need - 1) == EINVAL

    def bwd(dy=X, x=W, wi=B, wo=R, gu=P, dx=Y, dwi=Z, dwo=Z + (1 << 24), add=None, lda=0, nws=1 << 22):
        return L.pffn_bwd(BF16, dy, 64, x, 64, wi, 96, wo, 64, gu, 96, add, lda, dx, 64, dwi, 96,
                          dwo, 64, 16, 64, 48, 64, 4, WS, nws, None)
    for k in ("dy", "x", "wi", "wo", "gu"):
        assert bwd(**{k: None}) == EINVAL
    assert bwd(dx=X) == EINVAL and bwd(dwi=B) == EINVAL and bwd(dwo=R) == EINVAL
    assert bwd(dwo=Z) == EINVAL and bwd(dx=P) == EINVAL
    assert bwd(add=Y + 2, lda=64) == EINVAL
    assert bwd(nws=64) == EINVAL
    assert bwd(dx=None, dwi=None, dwo=None) == OK


def test_xent_checks(L):
    def call(dtype=F16, x=X, ldx=64, w=W, ldw=64, t=B, red=1, loss=R, lse=Y, M=16, V=100, D=64, ws=WS,
             nws=1 << 22):
        return L.pxent(dtype, x, ldx, w, ldw, t, -100, red, loss, lse, M, V, D, ws, nws, None)
    assert call(M=-1) == EINVAL and call(D=-1) == EINVAL
    assert call(V=0) == EINVAL
    assert call(red=3) == EUNSUP and call(red=-1) == EUNSUP and call(dtype=F32) == EUNSUP
    for k in ("x", "w", "t", "loss", "lse"):
        assert call(**{k: None}) == EINVAL
    assert call(t=B + 4) == EUNSUP and call(lse=Y + 2) == EUNSUP
    assert call(loss=Y) == EINVAL and call(lse=X) == EINVAL and call(loss=W) == EINVAL
    assert call(M=1 << 20, V=1 << 20, ldx=64) == EUNSUP     # M V above 2^37
    assert call(ws=None, nws=0) == EINVAL and call(ws=Y) == EINVAL
    assert call(M=0, red=0) == OK

    def bwd(x=X, w=W, t=B, lse=R, g=None, dx=Y, dw=P, ws=WS, nws=1 << 24):
        return L.pxent_bwd(F16, x, 64, w, 64, t, -100, 1, lse, g, dx, 64, dw, 64, 16, 100, 64, ws,
                           nws, None)
    for k in ("x", "w", "t", "lse"):
        assert bwd(**{k: None}) == EINVAL
    assert bwd(dx=X) == EINVAL and bwd(dw=W) == EINVAL and bwd(dw=Y) == EINVAL
    assert bwd(g=Y) == EINVAL and bwd(nws=100) == EINVAL
    assert bwd(dx=None, dw=None) == OK


def test_clip_checks(L):
    def call(ptrs=(X, W), outs=None, sizes=(100, 50), dtypes=(F16, F32), norm=B, max_norm=1.0, ws=WS,
             nws=1 << 20, count=None):
        n = len(ptrs)
        a, s, d = array.array("Q", ptrs), array.array("q", sizes), array.array("i", dtypes)
        o = array.array("Q", outs) if outs else None
        return L.pclip_grad_norm(a.buffer_info()[0], o.buffer_info()[0] if o else None,
                                 s.buffer_info()[0], d.buffer_info()[0], n if count is None else count,
                                 max_norm, norm, ws, nws, None)
    assert call(count=-1) == EINVAL
    assert call(norm=None) == EINVAL and call(norm=B + 2) == EUNSUP
    assert call(max_norm=-1.0) == EINVAL and call(max_norm=float("nan")) == EINVAL
    assert call(sizes=(100, -1)) == EINVAL
    assert call(dtypes=(F16, 3)) == EUNSUP
    assert call(ptrs=(X, 0)) == EINVAL and call(outs=(Y, 0)) == EINVAL
    assert call(ptrs=(X + 1, W)) == EUNSUP and call(ptrs=(X, W + 2)) == EUNSUP
    assert call(ptrs=(X, X)) == EINVAL                     # one tensor twice
    assert call(ptrs=(X, X + 196)) == EINVAL               # they meet
    assert call(outs=(W, Y)) == EINVAL                     # an output is another gradient
    assert call(outs=(X + 4, Y)) == EINVAL
    assert call(norm=X + 8) == EINVAL and call(ws=X) == EINVAL
    assert call(ws=None) == EINVAL and call(ws=WS + 4) == EUNSUP
    assert call(nws=L.pclip_grad_norm_workspace_bytes(2) - 1) == EINVAL
    assert call(sizes=(1 << 41, 50)) == EUNSUP
    assert L.pclip_grad_norm_workspace_bytes(-1) == EINVAL


def test_python_refusals():
    torch = pytest.importorskip("torch")
    x = torch.zeros((4, 8), dtype=torch.float16)
    w = torch.zeros((8, 4), dtype=torch.float16)
    with pytest.raises(ValueError):
        pg.plinear(x, w)                       # no device tensor
    with pytest.raises(ValueError):
        pg.plinear(x, w, act="tanh")
    with pytest.raises(TypeError):
        pg.plinear(x.float(), w)
    with pytest.raises(TypeError):
        pg.plinear([1.0], w)
    with pytest.raises(ValueError):
        pg.pffn(x, w, w)
    with pytest.raises(ValueError):
        pg.pxent(x, x, torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError):
        pg.pclip_grad_norm([], 1.0)
    with pytest.raises(ValueError):
        pg.pclip_grad_norm([torch.zeros(3)], 1.0)
    with pytest.raises(TypeError):
        pg.pclip_grad_norm([1.0], 1.0)
