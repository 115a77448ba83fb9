"""Argument checks of the norm's backward pass at x + residual, without a GPU:
every refusal is decided on the host before any HIP call."""
import pytest

import software_pipelined_tiled_pgemm_amd as pg
from .test_serving_abi import BF16, F16, F32, H, L, NAN, R, W, WS, X, Y, Z  # noqa: F401

EINVAL, EUNSUP, OK = pg.PGEMM_EINVAL, pg.PGEMM_EUNSUPPORTED, pg.PGEMM_OK
DH = 0x90000000  # one more address that is never dereferenced


def bwd(L, dtype=F16, dy=X, lddy=64, x=H, ldx=64, r=R, ldr=64, w=W, dh=DH, lddh=64, dx=Y, lddx=64,
        dw=Z, M=4, D=64, eps=1e-6, ws=WS, nws=1 << 20):
    return L.prmsnorm_bwd_sum(dtype, dy, lddy, x, ldx, r, ldr, w, dh, lddh, dx, lddx, dw, M, D, eps, ws,
                              nws, None)


@pytest.mark.parametrize("change,expected", [
    (dict(M=-1), EINVAL), (dict(D=-1), EINVAL), (dict(dy=None), EINVAL), (dict(x=None), EINVAL),
    (dict(r=None), EINVAL), (dict(lddy=63), EINVAL), (dict(ldx=63), EINVAL), (dict(ldr=63), EINVAL),
    (dict(lddh=63), EINVAL), (dict(lddx=63), EINVAL), (dict(eps=NAN), EINVAL), (dict(eps=-1.0), EINVAL),
    (dict(dtype=F32), EUNSUP), (dict(r=R + 1), EUNSUP), (dict(ldr=1 << 22), EUNSUP),
    (dict(dx=X), EINVAL), (dict(dx=H), EINVAL), (dict(dx=R), EINVAL), (dict(dx=W), EINVAL),
    (dict(dx=DH + 2), EINVAL), (dict(dw=R + 64), EINVAL), (dict(dw=W), EINVAL), (dict(dx=Z), EINVAL),
    (dict(ws=None, nws=0), EINVAL), (dict(nws=16), EINVAL), (dict(ws=WS + 8), EUNSUP),
    (dict(ws=R), EINVAL), (dict(ws=H), EINVAL),
    (dict(D=0), OK), (dict(dx=None, dw=None, dy=None), OK),
])
def test_norm_bwd_sum_checks(L, change, expected):  # noqa: F811
    assert bwd(L, **change) == expected


def test_mx_linear_few_rows_of_many_columns(L):  # noqa: F811
    """A few rows by a vocabulary's columns go by tiles, whose operand is quantised in the
    workspace; by few columns they are quantised by the kernel itself."""
    need = L.pmx_linear_workspace_bytes
    for M in (1, 4):
        assert need(F16, 1, 1, 0, M, 131072, 4096) > 0
        assert need(F16, 1, 1, 0, M, 4096, 4096) == 0


def test_sample_workspace(L):  # noqa: F811
    """Up to 16 long rows are cut into pieces, which meet in the workspace."""
    need = L.psample_workspace_bytes
    for dtype, V in ((F16, 20000), (BF16, 131072), (F32, 9000)):
        assert need(dtype, 1, V) > 0 and need(dtype, 16, V) > 0 and need(dtype, 17, V) == 0
    assert need(F32, 1, 8192) == 0 and need(BF16, 1, 16384) == 0
