"""The layer operators of libpgemm (include/pgemm.h, second part) on torch
tensors: the linear layer, the gated feed-forward block, the softmax cross
entropy over a vocabulary and gradient clipping, each with its backward pass.

As in the rest of the package the functions check arguments, allocate the
outputs and workspaces that were not given (from the pool of the stream the
call runs on) and pass pointers.  Matrices are 2-D tensors whose last
dimension is contiguous; their rows may be strided.  They know nothing of
torch's autograd: a result carries no graph, also where an input requires
grad, and gradients are what the _bwd functions return.  With stream=None a call
runs on the current stream; on another one the caller orders it after the
work that produces its inputs and keeps them alive, as for any torch tensor
used on a stream that is not its own.
"""
from __future__ import annotations

import array
import sys

from . import _lib
from ._lib import PgemmError, lib

_pkg = sys.modules[__package__]  # its helpers, defined before this module is imported
_new, _invoke = _pkg._new, _pkg._invoke

ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
REDUCTIONS = {"none": 0, "mean": 1, "sum": 2}


# torch, looked up at the first call (importing the package does not import
# torch).  A token's kernels take a few microseconds, so what a call does here
# is kept short: the checks are single expressions in the common case, and
# the sizes of workspaces are remembered by what they depend on.
_torch = None
_TENSOR = None
_F16 = _BF16 = _F32 = None


def _base():
    global _torch, _TENSOR, _F16, _BF16, _F32
    if _torch is None:
        t = _pkg._torch()
        _TENSOR, _F16, _BF16, _F32 = t.Tensor, t.float16, t.bfloat16, t.float32
        _torch = t
    return _torch


def _act(act):
    a = ACTIVATIONS.get(act) if isinstance(act, str) else None
    if a is None:
        raise ValueError("act must be one of %s, got %r" % (", ".join(ACTIVATIONS), act))
    return a


def _dtype(t, name):
    torch = _torch or _base()
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    dt = t.dtype
    if dt is _F16:
        return 0
    if dt is _BF16:
        return 1
    raise TypeError("%s must be float16 or bfloat16, got %s" % (name, dt))


def _mat(t, name, like, rows=None, cols=None, also=None):
    """Checks a matrix against the call's first tensor `like` (type, device)
    and a shape; returns its row pitch in elements.  `also`: another type that
    it may have."""
    if not isinstance(t, _TENSOR):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a device (HIP) tensor, got %s" % (name, t.device))
    if t is not like:
        if t.dtype is not like.dtype and (also is None or t.dtype is not also):
            raise TypeError("%s must be %s, got %s" % (name, like.dtype, t.dtype))
        if t.get_device() != like.get_device():
            raise ValueError("%s is on another device than the other tensors" % name)
    if t.dim() != 2:
        raise ValueError("%s must have 2 dimensions" % name)
    r, c = t.shape
    if (rows is not None and r != rows) or (cols is not None and c != cols):
        raise ValueError("%s must have shape (%s, %s), got %s"
                         % (name, "any" if rows is None else rows, "any" if cols is None else cols,
                            tuple(t.shape)))
    if r == 0 or c == 0:  # no element: torch's strides mean nothing
        return max(c, 1)
    s0, s1 = t.stride()
    if c > 1 and s1 != 1:
        raise ValueError("%s must be contiguous along its rows" % name)
    if r > 1 and s0 < c:
        raise ValueError("%s must not have overlapping rows" % name)
    return s0 if r > 1 else c


def _vec(t, name, like, n):
    if not isinstance(t, _TENSOR):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda or t.get_device() != like.get_device():
        raise ValueError("%s must be on the other tensors' device" % name)
    if t.dtype is not like.dtype:
        raise TypeError("%s must be %s, got %s" % (name, like.dtype, t.dtype))
    if t.dim() != 1 or t.shape[0] != n or not t.is_contiguous():
        raise ValueError("%s must be a contiguous vector of %d elements" % (name, n))


def _ptr(t):
    return None if t is None else t.data_ptr()


def _out(t, name, like, shape, stream):
    if t is None:
        return _new(shape, like.dtype, like.device, stream), max(shape[1], 1)
    return t, _mat(t, name, like, *shape)


_needs = {}


def _need(fn, like, *args):
    """fn(*args), a workspace size, remembered: it depends on the arguments
    (pointers: on their alignment alone, which is what is passed) and on the
    device."""
    key = (fn.__name__, like.get_device()) + args
    need = _needs.get(key)
    if need is None:
        with _base().cuda.device(key[1]):
            need = fn(*args)
        if need < 0:
            raise PgemmError(int(need), fn.__name__)
        if len(_needs) >= 4096:
            _needs.clear()
        _needs[key] = need
    return need


def _at(t):
    """An address of t's alignment."""
    return 16 + (t.data_ptr() & 15)


def _workspace(need, given, like, stream):
    """(pointer, bytes, tensor to keep alive) of a call's workspace."""
    if given is not None:
        if given.device != like.device or not given.is_contiguous():
            raise ValueError("workspace must be a contiguous tensor on %s" % like.device)
        return given.data_ptr(), given.numel() * given.element_size(), given
    if need == 0:
        return None, 0, None
    w = _new(need, _torch.uint8, like.device, stream)
    return w.data_ptr(), need, w


def _call(rc, what):
    if rc != _lib.PGEMM_OK:
        raise PgemmError(rc, what)


def plinear(x, w, bias=None, residual=None, act="none", preact=None, out=None, workspace=None,
            stream=None):
    """act(x @ w + bias) + residual for x [M,K], w [K,N] (float16 or bfloat16).

    act: "none", "relu", "gelu", "gelu_tanh" or "silu".  preact: an [M,N] tensor
    that receives x @ w + bias, which plinear_bwd needs unless act is "none".
    out may be residual."""
    dt = _dtype(x, "x")
    a = _act(act)
    ldx = _mat(x, "x", x)
    M, K = x.shape
    ldw = _mat(w, "w", x, rows=K)
    N = w.shape[1]
    if bias is not None:
        _vec(bias, "bias", x, N)
    ldr = _mat(residual, "residual", x, M, N) if residual is not None else 0
    ldp = _mat(preact, "preact", x, M, N) if preact is not None else 0
    out, ldy = _out(out, "out", x, (M, N), stream)
    L = lib()

    need = _need(L.plinear_workspace_bytes, x, dt, _at(x), ldx, _at(w), ldw, M, N, K)
    ws, nws, keep = _workspace(need, workspace, x, stream)

    def run(h):
        return L.plinear(dt, x.data_ptr(), ldx, w.data_ptr(), ldw, _ptr(bias), _ptr(residual), ldr,
                         out.data_ptr(), ldy, _ptr(preact), ldp, M, N, K, a, ws, nws, h)
    _call(_invoke(x, stream, run), "plinear")
    return out


def plinear_bwd(dy, x, w, preact=None, act="none", dx_residual=None, needs=(True, True, True),
                dx=None, dw=None, dbias=None, workspace=None, stream=None):
    """(dx, dw, dbias) of plinear for the gradient dy [M,N] of its output
    (which is also the gradient of its residual).  `needs` says which are
    computed; the others are None.  dx_residual [M,K] is added to dx (dy, where
    x was also the residual)."""
    dt = _dtype(dy, "dy")
    a = _act(act)
    lddy = _mat(dy, "dy", dy)
    M, N = dy.shape
    ldx = _mat(x, "x", dy, rows=M)
    K = x.shape[1]
    ldw = _mat(w, "w", dy, K, N)
    if a and preact is None and any(needs):
        raise ValueError("preact is needed for act=%r" % act)
    ldp = _mat(preact, "preact", dy, M, N) if preact is not None else 0
    lda = _mat(dx_residual, "dx_residual", dy, M, K) if dx_residual is not None else 0
    lddx = lddw = 0
    if needs[0]:
        dx, lddx = _out(dx, "dx", dy, (M, K), stream)
    if needs[1]:
        dw, lddw = _out(dw, "dw", dy, (K, N), stream)
    if needs[2]:
        if dbias is None:
            dbias = _new((N,), dy.dtype, dy.device, stream)
        _vec(dbias, "dbias", dy, N)
    dx, dw, dbias = (t if n else None for t, n in zip((dx, dw, dbias), needs))
    L = lib()

    need = _need(L.plinear_bwd_workspace_bytes, dy, dt, _at(dy), lddy, _at(x), ldx, _at(w), ldw, M,
                 N, K, a, *map(int, map(bool, needs)))
    ws, nws, keep = _workspace(need, workspace, dy, stream)

    def run(h):
        return L.plinear_bwd(dt, dy.data_ptr(), lddy, x.data_ptr(), ldx, w.data_ptr(), ldw,
                             _ptr(preact), ldp, _ptr(dx_residual), lda, _ptr(dx), lddx, _ptr(dw),
                             lddw, _ptr(dbias), M, N, K, a, ws, nws, h)
    _call(_invoke(dy, stream, run), "plinear_bwd")
    return dx, dw, dbias


def _gate_up(t, like, rows, cols):
    """gate_up's row pitch.  bfloat16's kept form is not bfloat16, so it may be
    held as what it is to everyone but pffn_bwd: 16 bits."""
    return _mat(t, "gate_up", like, rows, cols,
                _torch.int16 if like.dtype is _BF16 else None)


def pffn(x, w_in, w_out, residual=None, act="silu", gate_up=None, out=None, workspace=None,
         stream=None):
    """(act(g) * u) @ w_out + residual with [g | u] = x @ w_in: the gated
    feed-forward block for x [M,D], w_in [D,2F], w_out [F,N].

    gate_up: an [M,2F] tensor that receives [g | u] for pffn_bwd, of x's type; for
    bfloat16 in a 16-bit form of its own (include/pgemm.h), whose numbers mean
    nothing as bfloat16, so an int16 tensor is taken too, and is the better
    choice: it cannot be read, or passed on, as activations by mistake.
    out may be residual or x."""
    dt = _dtype(x, "x")
    a = _act(act)
    ldx = _mat(x, "x", x)
    M, D = x.shape
    ldwi = _mat(w_in, "w_in", x, rows=D)
    if w_in.shape[1] % 2:
        raise ValueError("w_in must have an even number of columns (gate, then up)")
    F = w_in.shape[1] // 2
    ldwo = _mat(w_out, "w_out", x, rows=F)
    N = w_out.shape[1]
    ldr = _mat(residual, "residual", x, M, N) if residual is not None else 0
    ldgu = _gate_up(gate_up, x, M, 2 * F) if gate_up is not None else 0
    out, ldy = _out(out, "out", x, (M, N), stream)
    L = lib()

    need = _need(L.pffn_workspace_bytes, x, dt, _at(x), ldx, _at(w_in), ldwi, _at(w_out), ldwo, M,
                 D, F, N)
    ws, nws, keep = _workspace(need, workspace, x, stream)

    def run(h):
        return L.pffn(dt, x.data_ptr(), ldx, w_in.data_ptr(), ldwi, w_out.data_ptr(), ldwo,
                      _ptr(residual), ldr, out.data_ptr(), ldy, _ptr(gate_up), ldgu, M, D, F, N, a,
                      ws, nws, h)
    _call(_invoke(x, stream, run), "pffn")
    return out


def pffn_bwd(dy, x, w_in, w_out, gate_up, act="silu", dx_residual=None, needs=(True, True, True),
             dx=None, dw_in=None, dw_out=None, workspace=None, stream=None):
    """(dx, dw_in, dw_out) of pffn for the gradient dy [M,N] of its output
    (which is also the gradient of its residual).  gate_up: as pffn wrote it, with
    the same x and w_in (not a product of the caller's own).  `needs` says which are
    computed; the others are None.  dx_residual [M,D] is added to dx (dy, where
    x was also the residual)."""
    dt = _dtype(dy, "dy")
    a = _act(act)
    lddy = _mat(dy, "dy", dy)
    M, N = dy.shape
    ldx = _mat(x, "x", dy, rows=M)
    D = x.shape[1]
    ldwi = _mat(w_in, "w_in", dy, rows=D)
    if w_in.shape[1] % 2:
        raise ValueError("w_in must have an even number of columns (gate, then up)")
    F = w_in.shape[1] // 2
    ldwo = _mat(w_out, "w_out", dy, F, N)
    ldgu = _gate_up(gate_up, dy, M, 2 * F)
    lda = _mat(dx_residual, "dx_residual", dy, M, D) if dx_residual is not None else 0
    lddx = lddwi = lddwo = 0
    if needs[0]:
        dx, lddx = _out(dx, "dx", dy, (M, D), stream)
    if needs[1]:
        dw_in, lddwi = _out(dw_in, "dw_in", dy, (D, 2 * F), stream)
    if needs[2]:
        dw_out, lddwo = _out(dw_out, "dw_out", dy, (F, N), stream)
    dx, dw_in, dw_out = (t if n else None for t, n in zip((dx, dw_in, dw_out), needs))
    L = lib()

    need = _need(L.pffn_bwd_workspace_bytes, dy, dt, _at(dy), lddy, _at(x), ldx, _at(w_in), ldwi,
                 _at(w_out), ldwo, M, D, F, N, *map(int, map(bool, needs)))
    ws, nws, keep = _workspace(need, workspace, dy, stream)

    def run(h):
        return L.pffn_bwd(dt, dy.data_ptr(), lddy, x.data_ptr(), ldx, w_in.data_ptr(), ldwi,
                          w_out.data_ptr(), ldwo, gate_up.data_ptr(), ldgu, _ptr(dx_residual), lda,
                          _ptr(dx), lddx, _ptr(dw_in), lddwi, _ptr(dw_out), lddwo, M, D, F, N, a,
                          ws, nws, h)
    _call(_invoke(dy, stream, run), "pffn_bwd")
    return dx, dw_in, dw_out


def _reduction(reduction):
    try:
        return REDUCTIONS[reduction]
    except (KeyError, TypeError):
        raise ValueError("reduction must be one of %s, got %r"
                         % (", ".join(REDUCTIONS), reduction)) from None


def _flat(t, name, like, dtype, shape):
    torch = _base()
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda or t.get_device() != like.get_device():
        raise ValueError("%s must be on the other tensors' device" % name)
    if t.dtype is not dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError("%s must be a contiguous tensor of shape %s" % (name, shape))


def _xent_operands(x, w, target):
    torch = _base()
    dt = _dtype(x, "x")
    ldx = _mat(x, "x", x)
    ldw = _mat(w, "w", x, cols=x.shape[1])
    _flat(target, "target", x, torch.int64, (x.shape[0],))
    return dt, ldx, ldw


def pxent(x, w, target, ignore_index=-100, reduction="mean", loss=None, lse=None, workspace=None,
          stream=None):
    """(loss, lse) of the softmax cross entropy of x [M,D] against the rows of
    w [V,D] at target [M] (int64): loss is a float32 scalar tensor ("mean" over
    the rows that are not ignored, "sum") or [M] ("none"), lse [M] the rows'
    log-sum-exp, which pxent_bwd needs.  The logits are not kept."""
    torch = _base()
    dt, ldx, ldw = _xent_operands(x, w, target)
    red = _reduction(reduction)
    (M, D), V = x.shape, w.shape[0]
    shape = (M,) if red == 0 else ()
    if loss is None:
        loss = _new(shape, torch.float32, x.device, stream)
    _flat(loss, "loss", x, torch.float32, shape)
    if lse is None:
        lse = _new((M,), torch.float32, x.device, stream)
    _flat(lse, "lse", x, torch.float32, (M,))
    L = lib()

    need = _need(L.pxent_workspace_bytes, x, dt, _at(x), ldx, _at(w), ldw, red, M, V, D)
    ws, nws, keep = _workspace(need, workspace, x, stream)

    def run(h):
        return L.pxent(dt, x.data_ptr(), ldx, w.data_ptr(), ldw, target.data_ptr(),
                       int(ignore_index), red, loss.data_ptr(), lse.data_ptr(), M, V, D, ws, nws, h)
    _call(_invoke(x, stream, run), "pxent")
    return loss, lse


def pxent_bwd(x, w, target, lse, dloss=None, ignore_index=-100, reduction="mean",
              needs=(True, True), dx=None, dw=None, workspace=None, stream=None):
    """(dx, dw) of pxent, called with the same x, w, target, ignore_index and
    reduction, for the gradient dloss of its loss (a float32 tensor of the
    loss's shape; None: 1).  `needs` says which are computed."""
    torch = _base()
    dt, ldx, ldw = _xent_operands(x, w, target)
    red = _reduction(reduction)
    (M, D), V = x.shape, w.shape[0]
    _flat(lse, "lse", x, torch.float32, (M,))
    if dloss is not None:
        _flat(dloss, "dloss", x, torch.float32, (M,) if red == 0 else ())
    lddx = lddw = 0
    if needs[0]:
        dx, lddx = _out(dx, "dx", x, (M, D), stream)
    if needs[1]:
        dw, lddw = _out(dw, "dw", x, (V, D), stream)
    dx, dw = (t if n else None for t, n in zip((dx, dw), needs))
    L = lib()

    need = _need(L.pxent_bwd_workspace_bytes, x, dt, _at(x), ldx, _at(w), ldw, M, V, D,
                 *map(int, map(bool, needs)))
    ws, nws, keep = _workspace(need, workspace, x, stream)

    def run(h):
        return L.pxent_bwd(dt, x.data_ptr(), ldx, w.data_ptr(), ldw, target.data_ptr(),
                           int(ignore_index), red, lse.data_ptr(), _ptr(dloss), _ptr(dx), lddx,
                           _ptr(dw), lddw, M, V, D, ws, nws, h)
    _call(_invoke(x, stream, run), "pxent_bwd")
    return dx, dw


def pclip_grad_norm(tensors, max_norm, out=None, norm=None, workspace=None, stream=None):
    """Scales the tensors (contiguous; float16, bfloat16 or float32, mixed as
    they come) by min(1, max_norm / (norm + 1e-6)), norm being that of all
    their elements together: in place, or into the list `out`.  Returns the
    norm before clipping as a float32 scalar tensor on the device."""
    torch = _torch or _base()
    tensors = list(tensors)
    n = len(tensors)
    if not n:
        raise ValueError("tensors must not be empty")
    every = tensors if out is None else tensors + list(out)
    if out is not None and len(every) != 2 * n:
        raise ValueError("out must have %d tensors" % n)
    # Unbound methods over the whole list: a model has hundreds of gradients,
    # and the calls' own time is most of the host's.
    T = _TENSOR
    devices = set(map(T.get_device, every))  # (TypeError if one is no tensor)
    first = tensors[0]
    if len(devices) != 1 or not first.is_cuda:
        raise ValueError("tensors and out must be on one HIP device")
    if not all(map(T.is_contiguous, every)):
        raise ValueError("tensors and out must be contiguous")
    kinds = list(map({torch.float16: 0, torch.bfloat16: 1, torch.float32: 2}.get,
                     [t.dtype for t in every]))
    if None in kinds:
        raise TypeError("tensors must be float16, bfloat16 or float32")
    counts = list(map(T.numel, every))
    if out is not None and (kinds[:n] != kinds[n:] or counts[:n] != counts[n:]):
        raise ValueError("out must have the tensors' types and sizes")
    pointers = array.array("Q", map(T.data_ptr, every))
    sizes, dtypes = array.array("q", counts), array.array("i", kinds)
    grads = pointers.buffer_info()[0]
    outs = None if out is None else grads + n * pointers.itemsize
    if norm is None:
        norm = _new((), torch.float32, first.device, stream)
    else:
        _flat(norm, "norm", first, torch.float32, ())
    L = lib()
    ws, nws, keep = _workspace(_need(L.pclip_grad_norm_workspace_bytes, first, n), workspace, first,
                               stream)

    def run(h):
        return L.pclip_grad_norm(grads, outs, sizes.buffer_info()[0], dtypes.buffer_info()[0], n,
                                 float(max_norm), norm.data_ptr(), ws, nws, h)
    _call(_invoke(first, stream, run), "pclip_grad_norm")
    return norm
