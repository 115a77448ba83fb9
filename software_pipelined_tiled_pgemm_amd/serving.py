"""The operators around a model's low-precision projections (include/pgemm.h,
third part) on torch tensors: the root-mean-square norm with the residual's
addition and its backward pass, microscaled matrices and their product, and the
sampling of tokens from logits.

They check, allocate and run like the layer operators (layers.py): matrices are
2-D tensors whose last dimension is contiguous, results carry no graph, and
with stream=None a call runs on the current stream.
"""
from __future__ import annotations

from . import layers as _l
from ._lib import lib
from .layers import (_act, _at, _call, _dtype, _flat, _invoke, _mat, _need, _new, _out, _ptr, _vec,
                     _workspace)

FORMATS = {"e2m1": 0, "e4m3": 1}


def _torch():
    return _l._torch or _l._base()


def _rows(t, name, like, M, D):
    """_mat for a matrix like the call's first one, which most are: contiguous, of
    its type, shape and device."""
    if (isinstance(t, _l._TENSOR) and t.dtype is like.dtype and t.shape == like.shape
            and t.is_contiguous() and t.get_device() == like.get_device()):
        return D or 1
    return _mat(t, name, like, M, D)


def _empty_like(x, M, D, stream):
    """A new matrix of x's type and shape."""
    if stream is None and x.is_contiguous():
        return _l._torch.empty_like(x)
    return _new((M, D), x.dtype, x.device, stream)


def _format(f):
    c = FORMATS.get(f) if isinstance(f, str) else None
    if c is None:
        raise ValueError("format must be one of %s, got %r" % (", ".join(FORMATS), f))
    return c


class MxMatrix:
    """A microscaled matrix: `codes` [rows, pitch] and `scales` [rows, pitch],
    uint8 tensors laid out as include/pgemm.h says (codes of "e4m3" may be a
    float8_e4m3fn tensor, scales a float8_e8m0fnu one), for `cols` columns in the
    format "e2m1" or "e4m3".  shape is (rows, cols)."""
    __slots__ = ("cols", "format", "_code", "_codes", "_scales", "_rows", "_pitch", "_whole")

    def __init__(self, codes, scales, cols, format):
        self._code = _format(format)
        self.cols, self.format = int(cols), format
        for t, name in ((codes, "codes"), (scales, "scales")):
            if not isinstance(t, _torch().Tensor):
                raise TypeError("%s must be a torch.Tensor" % name)
            if t.element_size() != 1:
                raise TypeError("%s must hold bytes, got %s" % (name, t.dtype))
            if t.dim() != 2:
                raise ValueError("%s must have 2 dimensions" % name)
        if self.cols < 0 or scales.shape[0] != codes.shape[0]:
            raise ValueError("codes and scales must have as many rows as each other")
        groups = (self.cols + 127) // 128
        if codes.shape[1] < groups * (128 if self._code else 64) or \
                scales.shape[1] < (groups + 3) // 4 * 16:
            raise ValueError("codes %s and scales %s are too short for %d columns"
                             % (tuple(codes.shape), tuple(scales.shape), self.cols))
        self._codes, self._scales, self._rows, self._whole = codes, scales, codes.shape[0], None

    @classmethod
    def _new(cls, rows, cols, code, like, stream):
        """Codes and scales in one allocation (a small matrix's costs more than its
        kernel); the tensors are made when they are asked for."""
        pitch = _pitches.get((code, cols))
        if pitch is None:
            L = lib()
            pitch = (L.pmx_codes_pitch(code, cols), L.pmx_scales_pitch(cols))
            if min(pitch) < 0:
                raise ValueError("%d columns are too many for a microscaled matrix" % cols)
            if len(_pitches) >= 4096:
                _pitches.clear()
            _pitches[code, cols] = pitch
        m = cls.__new__(cls)
        m.cols, m.format, m._code, m._rows, m._pitch = cols, _NAMES[code], code, rows, pitch
        # (codes' rows are multiples of 64 bytes: the scales are aligned too)
        m._whole = _new(rows * (pitch[0] + pitch[1]), _torch().uint8, like.device, stream)
        m._codes = m._scales = None
        return m

    def _split(self):
        n, (pc, ps) = self._rows, self._pitch
        self._codes = self._whole[:n * pc].view(n, pc)
        self._scales = self._whole[n * pc:].view(n, ps)

    @property
    def codes(self):
        if self._codes is None:
            self._split()
        return self._codes

    @property
    def scales(self):
        if self._scales is None:
            self._split()
        return self._scales

    @property
    def _any(self):
        """A tensor of the matrix's, for its device."""
        return self._codes if self._whole is None else self._whole

    @property
    def shape(self):
        return (self._rows, self.cols)

    @property
    def device(self):
        return self._any.device

    def __repr__(self):
        return "MxMatrix(%s, %s, %s)" % (self.shape, self.format, self.device)


_NAMES = ("e2m1", "e4m3")
_pitches = {}


def _pitched(t, name, like):
    if not t.is_cuda or t.get_device() != like.get_device():
        raise ValueError("%s must be on the other tensors' device" % name)
    r, c = t.shape
    if r == 0 or c == 0:
        return 0
    s0, s1 = t.stride()
    if c > 1 and s1 != 1:
        raise ValueError("%s must be contiguous along its rows" % name)
    if r > 1 and s0 < c:
        raise ValueError("%s must not have overlapping rows" % name)
    return s0 if r > 1 else c


def _mx(m, name, like, rows=None, cols=None, format=None):
    """(address and pitch of the codes, and of the scales) of a microscaled
    argument."""
    if not isinstance(m, MxMatrix):
        raise TypeError("%s must be an MxMatrix" % name)
    if (rows is not None and m._rows != rows) or (cols is not None and m.cols != cols):
        raise ValueError("%s must have shape (%s, %s), got %s"
                         % (name, "any" if rows is None else rows, "any" if cols is None else cols,
                            m.shape))
    if format is not None and m._code != format:
        raise ValueError("%s is %s" % (name, m.format))
    whole = m._whole
    if whole is not None:
        if whole.get_device() != like.get_device():
            raise ValueError("%s must be on the other tensors' device" % name)
        p, (pc, ps) = whole.data_ptr(), m._pitch
        return p, pc, p + m._rows * pc, ps
    c, s = m._codes, m._scales
    return (c.data_ptr(), _pitched(c, name + ".codes", like), s.data_ptr(),
            _pitched(s, name + ".scales", like))


def prmsnorm(x, weight=None, residual=None, eps=1e-6, h=None, format=None, out=None, stream=None):
    """s / sqrt(mean(s^2) + eps) * weight along the rows of s = x + residual, for x
    and residual [M,D], weight [D] (float16 or bfloat16).

    h: an [M,D] tensor that receives s (the residual stream, and what prmsnorm_bwd
    takes); it may be x or residual.  format: None for a result of x's type, which
    out may hold (x or residual, too), or "e2m1" or "e4m3" for an MxMatrix, the
    operand of pmx_linear."""
    dt = _dtype(x, "x")
    ldx = _mat(x, "x", x)
    M, D = x.shape
    ldr = _rows(residual, "residual", x, M, D) if residual is not None else 0
    if weight is not None:
        _vec(weight, "weight", x, D)
    ldh = _rows(h, "h", x, M, D) if h is not None else 0
    eps = float(eps)
    if not 0.0 <= eps < float("inf"):
        raise ValueError("eps must be finite and at least 0, got %r" % eps)
    if format is None:
        code, scales, lds = -1, None, 0
        if out is None:
            out, ldy = _empty_like(x, M, D, stream), D or 1
        else:
            ldy = _rows(out, "out", x, M, D)
        y = out.data_ptr()
    else:
        code = _format(format)
        if out is None:
            out = MxMatrix._new(M, D, code, x, stream)
        y, ldy, scales, lds = _mx(out, "out", x, M, D, code)
    L = lib()

    def run(s):
        return L.prmsnorm(dt, x.data_ptr(), ldx, _ptr(residual), ldr, _ptr(weight), _ptr(h), ldh, code,
                          y, ldy, scales, lds, M, D, eps, s)
    _call(_invoke(x, stream, run), "prmsnorm")
    return out


def prmsnorm_bwd(dy, h, weight=None, eps=1e-6, dh=None, needs=(True, True), dx=None, dweight=None,
                 workspace=None, stream=None, residual=None):
    """(dx, dweight) of prmsnorm for the gradient dy [M,D] of its result.  h: as
    prmsnorm wrote it (x, where there was no residual), rounded to its type; or, with
    prmsnorm's residual given, its x: the sum is taken in fp32 then, as prmsnorm normed
    it, and dweight has one rounding less, for one matrix more to read.  dx is the
    gradient of x and of residual; dh [M,D], the gradient that reaches h by other
    ways, is added to it.  `needs` says which are computed (without a weight dweight is
    not)."""
    dt = _dtype(dy, "dy")
    lddy = _mat(dy, "dy", dy)
    M, D = dy.shape
    ldh = _rows(h, "h", dy, M, D)
    ldr = _rows(residual, "residual", dy, M, D) if residual is not None else 0
    if weight is not None:
        _vec(weight, "weight", dy, D)
    lddh = _rows(dh, "dh", dy, M, D) if dh is not None else 0
    eps = float(eps)
    if not 0.0 <= eps < float("inf"):
        raise ValueError("eps must be finite and at least 0, got %r" % eps)
    needs = (bool(needs[0]), bool(needs[1]) and weight is not None)
    lddx = 0
    if needs[0]:
        if dx is None:
            dx, lddx = _empty_like(dy, M, D, stream), D or 1
        else:
            lddx = _rows(dx, "dx", dy, M, D)
    if needs[1]:
        if dweight is None:
            dweight = _new((D,), dy.dtype, dy.device, stream)
        _vec(dweight, "dweight", dy, D)
    dx, dweight = (t if n else None for t, n in zip((dx, dweight), needs))
    L = lib()
    need = _need(L.prmsnorm_bwd_workspace_bytes, dy, dt, M, D, *map(int, needs))
    ws, nws, keep = _workspace(need, workspace, dy, stream)

    def run(s):
        if residual is not None:
            return L.prmsnorm_bwd_sum(dt, dy.data_ptr(), lddy, h.data_ptr(), ldh, residual.data_ptr(),
                                      ldr, _ptr(weight), _ptr(dh), lddh, _ptr(dx), lddx,
                                      _ptr(dweight), M, D, eps, ws, nws, s)
        return L.prmsnorm_bwd(dt, dy.data_ptr(), lddy, h.data_ptr(), ldh, _ptr(weight), _ptr(dh), lddh,
                              _ptr(dx), lddx, _ptr(dweight), M, D, eps, ws, nws, s)
    _call(_invoke(dy, stream, run), "prmsnorm_bwd")
    return dx, dweight


def pmx_quantize(x, format="e2m1", out=None, stream=None):
    """x [M,K] (float16 or bfloat16) as an MxMatrix of the format "e2m1" or
    "e4m3"."""
    dt = _dtype(x, "x")
    code = _format(format)
    ldx = _mat(x, "x", x)
    M, K = x.shape
    if out is None:
        out = MxMatrix._new(M, K, code, x, stream)
    codes, ldc, scales, lds = _mx(out, "out", x, M, K, code)
    L = lib()

    def run(s):
        return L.pmx_quantize(dt, x.data_ptr(), ldx, code, codes, ldc, scales, lds, M, K, s)
    _call(_invoke(x, stream, run), "pmx_quantize")
    return out


def pmx_dequantize(m, dtype=None, out=None, stream=None):
    """The values of an MxMatrix as a tensor of `dtype` (float16 or bfloat16, the
    default)."""
    torch = _torch()
    if not isinstance(m, MxMatrix):
        raise TypeError("m must be an MxMatrix")
    like = m._any
    if not like.is_cuda:
        raise ValueError("m must be on a device (HIP), got %s" % like.device)
    codes, ldc, scales, lds = _mx(m, "m", like)
    M, K = m.shape
    if out is None:
        if dtype is None:
            dtype = torch.bfloat16
        if dtype not in (torch.float16, torch.bfloat16):
            raise TypeError("dtype must be float16 or bfloat16, got %s" % dtype)
        out = _new((M, K), dtype, like.device, stream)
    elif dtype is not None and out.dtype is not dtype:
        raise TypeError("out must be %s, got %s" % (dtype, out.dtype))
    dt = _dtype(out, "out")
    if out.get_device() != like.get_device():
        raise ValueError("out is on another device than m")
    ldy = _mat(out, "out", out, M, K)
    L = lib()

    def run(s):
        return L.pmx_dequantize(m._code, codes, ldc, scales, lds, dt, out.data_ptr(), ldy, M, K, s)
    _call(_invoke(like, stream, run), "pmx_dequantize")
    return out


def pmx_linear(x, w, bias=None, residual=None, act="none", format="e4m3", dtype=None, out=None,
               workspace=None, stream=None):
    """act(x @ w.T + bias) + residual for microscaled w [N,K] and x [M,K]: an
    MxMatrix, or a float16 or bfloat16 matrix, which is quantised to `format`
    first.

    act: as plinear's.  bias, residual and the result are of x's type where it has
    one, else of `dtype` (the type of out, residual or bias, where one is given,
    or bfloat16).  out may be residual."""
    torch = _torch()
    a = _act(act)
    if not isinstance(w, MxMatrix):
        raise TypeError("w must be an MxMatrix")
    if isinstance(x, MxMatrix):
        like, xcode, quantizes = x._any, x._code, 0
        if not like.is_cuda:
            raise ValueError("x must be on a device (HIP), got %s" % like.device)
        px, ldx, pxs, ldxs = _mx(x, "x", like)
        if dtype is None:
            dtype = next((t.dtype for t in (out, residual, bias) if t is not None), torch.bfloat16)
    else:
        _dtype(x, "x")
        like, xcode, quantizes = x, _format(format), 1
        ldx, ldxs = _mat(x, "x", x), 0
        if dtype is not None and dtype is not x.dtype:
            raise TypeError("dtype must be x's, %s, got %s" % (x.dtype, dtype))
        dtype = x.dtype
        px, pxs = x.data_ptr(), None
    if dtype not in (torch.float16, torch.bfloat16):
        raise TypeError("dtype must be float16 or bfloat16, got %s" % dtype)
    M, K = x.shape
    pw, ldw, pws, ldws = _mx(w, "w", like, cols=K)
    N = w._rows
    if out is None:
        out, ldy = _new((M, N), dtype, like.device, stream), N or 1
    else:
        if _dtype(out, "out") != (0 if dtype is torch.float16 else 1):
            raise TypeError("out must be %s, got %s" % (dtype, out.dtype))
        if out.get_device() != like.get_device():
            raise ValueError("out is on another device than the other tensors")
        ldy = _mat(out, "out", out, M, N)
    if bias is not None:
        _vec(bias, "bias", out, N)
    ldr = _rows(residual, "residual", out, M, N) if residual is not None else 0
    dt = 0 if dtype is torch.float16 else 1
    L = lib()
    need = _need(L.pmx_linear_workspace_bytes, like, dt, xcode, quantizes, w._code, M, N, K)
    ws, nws, keep = _workspace(need, workspace, like, stream)

    def run(s):
        return L.pmx_linear(dt, xcode, px, ldx, pxs, ldxs, w._code, pw, ldw, pws, ldws, _ptr(bias),
                            _ptr(residual), ldr, out.data_ptr(), ldy, M, N, K, a, ws, nws, s)
    _call(_invoke(like, stream, run), "pmx_linear")
    return out


def _setting(v, name, like, M, dtype, number, least, most):
    """(number, tensor or None) of a setting."""
    if isinstance(v, _torch().Tensor):
        _flat(v, name, like, dtype, (M,))
        return number(0), v
    n = number(v)
    if not least <= n <= most:
        raise ValueError("%s must lie between %s and %s, got %r" % (name, least, most, v))
    return n, None


def psample(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, tokens=None, logprobs=None,
            workspace=None, stream=None):
    """(tokens, logprobs): a token drawn from each row of logits [M,V] (float16,
    bfloat16 or float32) with the random numbers u [M] (float32 in [0, 1)), and
    the logarithm of its probability among the tokens kept.

    Each setting is a number, or a tensor [M] (float32; top_k int32) with one for
    each row.  temperature 0: the first of the largest logits.  top_k: so many
    tokens are kept, 0 for all.  top_p: of those the fewest that hold this part of
    their probability.  min_p: of those the ones with at least this part of the
    largest probability.  include/pgemm.h has the definition."""
    torch = _torch()
    if not isinstance(logits, torch.Tensor):
        raise TypeError("logits must be a torch.Tensor")
    if logits.dtype is torch.float32:
        dt = 2
    else:
        try:
            dt = _dtype(logits, "logits")
        except TypeError:
            raise TypeError("logits must be float16, bfloat16 or float32, got %s"
                            % logits.dtype) from None
    ld = _mat(logits, "logits", logits)
    M, V = logits.shape
    if V < 1:
        raise ValueError("logits must have at least one column")
    _flat(u, "u", logits, torch.float32, (M,))
    inf, f32 = float("inf"), torch.float32
    t, ts = _setting(temperature, "temperature", logits, M, f32, float, 0.0, inf)
    k, ks = _setting(top_k, "top_k", logits, M, torch.int32, int, 0, 2 ** 31 - 1)
    p, ps = _setting(top_p, "top_p", logits, M, f32, float, 0.0, inf)
    m, ms = _setting(min_p, "min_p", logits, M, f32, float, 0.0, 1.0)
    if tokens is None:
        tokens = _new((M,), torch.int64, logits.device, stream)
    _flat(tokens, "tokens", logits, torch.int64, (M,))
    if logprobs is None:
        logprobs = _new((M,), f32, logits.device, stream)
    _flat(logprobs, "logprobs", logits, f32, (M,))
    L = lib()
    ws, nws, keep = _workspace(_need(L.psample_workspace_bytes, logits, dt, M, V), workspace, logits,
                               stream)

    def run(s):
        return L.psample(dt, logits.data_ptr(), ld, u.data_ptr(), t, _ptr(ts), k, _ptr(ks), p,
                         _ptr(ps), m, _ptr(ms), tokens.data_ptr(), logprobs.data_ptr(), M, V, ws,
                         nws, s)
    _call(_invoke(logits, stream, run), "psample")
    return tokens, logprobs
