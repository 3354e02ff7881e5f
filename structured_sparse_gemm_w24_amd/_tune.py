"""Binding of the calls that tune and serve pruned layers: layer norm, low-rank
adapters, the cross entropy of a linear head.

Same manner as ``_lib``: torch device tensors in and out, one library call on
torch's current stream, ``SsgError`` on a nonzero status, no fallback.  Rows may
be strided (a 2-D tensor whose last axis is contiguous); workspaces come from
torch's caching allocator, whose reuse is ordered by the stream.  The gradients
are calls of their own and no autograd functions: results carry no history, also
where an input requires a gradient.
"""

from __future__ import annotations

import contextlib
import ctypes as ct
import functools

from . import _lib
from ._lib import SSG_OK, SsgError

SSG_DT_F16, SSG_DT_BF16, SSG_DT_F32 = 0, 1, 2
_SAME = contextlib.nullcontext()


@functools.lru_cache(maxsize=None)
def _torch():
    import torch
    return torch


def load():
    return _lib._LIB or _lib.load()


def _check(rc):
    if rc != SSG_OK:
        raise SsgError(rc, load().ssg_last_error().decode())


@functools.lru_cache(maxsize=None)
def _codes():
    torch = _torch()
    return {torch.float16: SSG_DT_F16, torch.bfloat16: SSG_DT_BF16, torch.float32: SSG_DT_F32}


@functools.lru_cache(maxsize=None)
def _raw_stream():
    """device index -> its current stream's handle (torch's own lookup where it has one: it
    builds no Stream object, 0.1 instead of 1.8 us a call)."""
    torch = _torch()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw or (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _stream(t):
    return _raw_stream()(t.get_device())


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _on(t):
    """Makes the tensors' device current for the launch."""
    torch = _torch()
    index = t.get_device()
    return _SAME if index == torch.cuda.current_device() else torch.cuda.device(index)


def _code(t, name, allowed=(SSG_DT_F16, SSG_DT_BF16, SSG_DT_F32)):
    if not isinstance(t, _torch().Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a torch tensor on a HIP device")
    code = _codes().get(t.dtype)
    if code is None or code not in allowed:
        raise TypeError(f"{name} has type {t.dtype}, which this call does not take")
    return code


def _refuse(t, dtype, shape, like, name):
    """Says what is wrong with a tensor that failed the checks of its caller."""
    if not isinstance(t, _torch().Tensor) or t.device != like.device:
        raise TypeError(f"{name} must be a torch tensor on {like.device}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


# (the checks below are one expression each: they run eight times in a call of
# 12 us, most of whose time is the host's)
def _rows(t, like, shape, name):
    """A [M, N] matrix of like's type and device with contiguous rows; returns its row stride."""
    dtype = like.dtype
    if not (isinstance(t, _torch().Tensor) and t.dtype is dtype and t.shape == shape
            and t.get_device() == like.get_device()):
        _refuse(t, dtype, shape, like, name)
    if t.is_contiguous():
        return shape[1] or 1
    ld, last = t.stride()
    if last != 1 and shape[1] > 1:
        raise ValueError(f"{name} must have contiguous rows")
    if shape[0] <= 1:
        return shape[1] or 1
    if ld < shape[1]:
        raise ValueError(f"{name} has overlapping rows")
    return ld


def _flat(t, dtype, shape, like, name):
    """A contiguous tensor of the given type and shape on like's device."""
    if not (isinstance(t, _torch().Tensor) and t.dtype is dtype and t.shape == shape
            and t.get_device() == like.get_device() and t.is_contiguous()):
        _refuse(t, dtype, shape, like, name)
    return t


def _matrix(t, name):
    if t.dim() != 2:
        raise ValueError(f"{name} must be a matrix, got shape {tuple(t.shape)}")
    return t.shape


def _out(out, like, shape, name="out"):
    """The caller's output (rows may be strided) or a new one; returns it and its row stride."""
    if out is None:
        if like.shape == shape and like.is_contiguous():
            return _torch().empty_like(like), shape[1] or 1
        return like.new_empty(shape), shape[1] or 1
    return out, _rows(out, like, shape, name)


def _workspace(n, like, ws=None):
    torch = _torch()
    if ws is not None:
        return _flat(ws, torch.uint8, ws.shape, like, "workspace")
    return like.new_empty(n if n > 16 else 16, dtype=torch.uint8)


# ------------------------------------------------------------------ layer norm
def _norm_params(x, n, weight, bias):
    torch = _torch()
    wt = None
    for p, name in ((weight, "weight"), (bias, "bias")):
        if p is None:
            continue
        if wt is None:
            wt = p.dtype
            if wt not in (x.dtype, torch.float32):
                raise TypeError(f"{name} must be {x.dtype} or torch.float32, got {wt}")
        _flat(p, wt, (n,), x, name)
    return _codes()[wt if wt is not None else x.dtype]


def layer_norm(x, weight=None, bias=None, eps=1e-5, residual=None, out=None, sum_out=None):
    """y = (s - mean) * rstd * weight + bias over the last axis of x [M, N], where s = x, or
    x + residual rounded to x's type.  Returns (y, mean, rstd), with a residual
    (y, mean, rstd, s); mean and rstd are fp32 [M].  x: float16, bfloat16 or float32;
    weight and bias [N]: both of x's type or both float32."""
    torch = _torch()
    dt = _code(x, "x")
    shape = _matrix(x, "x")
    m, n = shape
    ldx = _rows(x, x, shape, "x")
    wt = _norm_params(x, n, weight, bias)
    y, ldy = _out(out, x, shape)
    ldr = lds = n
    s = None
    if residual is not None:
        ldr = _rows(residual, x, shape, "residual")
        s, lds = _out(sum_out, x, shape, "sum_out")
    elif sum_out is not None:
        raise ValueError("sum_out needs a residual")
    mean = x.new_empty(m, dtype=torch.float32)
    rstd = torch.empty_like(mean)
    with _on(x):
        _check(load().layer_norm_forward(dt, _ptr(x), ldx, _ptr(residual), ldr, _ptr(weight), _ptr(bias), wt, eps,
                                         _ptr(y), ldy, _ptr(s), lds, _ptr(mean), _ptr(rstd), m, n, _stream(x)))
    return (y, mean, rstd) if residual is None else (y, mean, rstd, s)


def layer_norm_backward(dy, x, mean, rstd, weight=None, dres=None, out=None, param_grads=True, workspace=None):
    """Gradients of layer_norm: x is its normalised input (the sum s, if there was a residual),
    mean and rstd what it returned.  Returns (dx, dweight, dbias); dx has dres added when that is
    given, dweight and dbias are fp32 [N] (None with param_grads=False: frozen norms)."""
    torch = _torch()
    dt = _code(x, "x")
    shape = _matrix(x, "x")
    m, n = shape
    ldx = _rows(x, x, shape, "x")
    lddy = _rows(dy, x, shape, "dy")
    _flat(mean, torch.float32, (m,), x, "mean")
    _flat(rstd, torch.float32, (m,), x, "rstd")
    wt = _norm_params(x, n, weight, None)
    ldres = _rows(dres, x, shape, "dres") if dres is not None else n
    dx, lddx = _out(out, x, shape)
    dw = db = ws = None
    lib = load()
    if param_grads:
        dw = x.new_empty(n, dtype=torch.float32)
        db = torch.empty_like(dw)
        ws = _workspace(lib.layer_norm_workspace_bytes(dt, m, n), x, workspace)
    with _on(x):
        _check(lib.layer_norm_backward(dt, _ptr(dy), lddy, _ptr(x), ldx, _ptr(mean), _ptr(rstd), _ptr(weight), wt,
                                       _ptr(dres), ldres, _ptr(dx), lddx, _ptr(dw), _ptr(db), m, n, _ptr(ws),
                                       ws.numel() if ws is not None else 0, _stream(x)))
    return dx, dw, db


# -------------------------------------------------------------------- adapters
class _LowRank(ct.Structure):
    _fields_ = [("down", ct.c_void_p), ("up", ct.c_void_p), ("scale", ct.c_void_p), ("ranks", ct.c_void_p),
                ("index", ct.c_void_p), ("dtype", ct.c_int32), ("adapters", ct.c_int32), ("R", ct.c_int32)]


def _pool(x, n, down, up, index, scale, ranks):
    """The C description of an adapter pool for rows x [M, K] and N = n output channels."""
    torch = _torch()
    dt = _code(x, "x", (SSG_DT_F16, SSG_DT_BF16))
    m, k = _matrix(x, "x")
    if not isinstance(down, torch.Tensor) or down.dim() != 3:
        raise ValueError("down must be a tensor of shape [adapters, R, K]")
    a, r, _ = down.shape
    _flat(down, x.dtype, (a, r, k), x, "down")
    _flat(up, x.dtype, (a, n, r), x, "up")
    _flat(index, torch.int32, (m,), x, "index")
    if scale is not None:
        _flat(scale, torch.float32, (a,), x, "scale")
    if ranks is not None:
        _flat(ranks, torch.int32, (a,), x, "ranks")
    return _LowRank(down.data_ptr(), up.data_ptr(), scale.data_ptr() if scale is not None else None,
                    ranks.data_ptr() if ranks is not None else None, index.data_ptr(), dt, a, r)


def _channels(up):
    if not isinstance(up, _torch().Tensor) or up.dim() != 3:
        raise ValueError("up must be a tensor of shape [adapters, N, R]")
    return up.shape[1]


def low_rank_add(base, x, down, up, index, scale=None, ranks=None, out=None, workspace=None):
    """out[m] = base[m] + scale[a] * up[a] . (down[a] . x[m]) with a = index[m] (-1: base alone).

    x [M, K], base [M, N] (None: zeros) and out (may be base): float16 or bfloat16, row strides in
    multiples of 8.  down [adapters, R, K] and up [adapters, N, R] hold the pool, R a multiple of 8
    up to 128; ranks int32 [adapters] are the slots in use (None: all R), scale float32 [adapters].
    index int32 [M], any order; a token with another index outside the pool gets NaN."""
    n = _channels(up)
    lr = _pool(x, n, down, up, index, scale, ranks)
    m, k = x.shape
    ldx = _rows(x, x, x.shape, "x")
    ldb = _rows(base, x, (m, n), "base") if base is not None else n
    out, ldo = _out(out, x, (m, n))
    lib = load()
    need = lib.low_rank_workspace_bytes(m, lr.R)
    ws = _workspace(need, x, workspace) if need > 0 else None
    with _on(x):
        _check(lib.low_rank_add(ct.byref(lr), _ptr(x), ldx, _ptr(base), ldb, _ptr(out), ldo, m, n, k, _ptr(ws),
                                ws.numel() if ws is not None else 0, _stream(x)))
    return out


def w24_low_rank_gemm_f16(A, vals, meta, down, up, index, scale=None, ranks=None, out=None, workspace=None):
    """C = A . W + the adapters' part in one pass: w24_gemm_f16 with a pool of adapters beside its 2:4
    weight (arguments as there and as in low_rank_add; everything float16, A contiguous)."""
    torch = _torch()
    _code(A, "A", (SSG_DT_F16,))
    m, k = _matrix(A, "A")
    _flat(A, torch.float16, A.shape, A, "A")
    n = vals.shape[0]
    _flat(vals, torch.float16, (n, k // 2), A, "vals")
    _flat(meta, torch.int32, (n, -(-k // 32)), A, "meta")
    lr = _pool(A, n, down, up, index, scale, ranks)
    if out is None:
        out = A.new_empty((m, n))
    else:
        _flat(out, torch.float16, (m, n), A, "out")
    lib = load()
    ws = _workspace(lib.w24_low_rank_workspace_bytes(m, n, k, lr.R), A, workspace)
    with _on(A):
        _check(lib.w24_low_rank_gemm_f16(_ptr(A), _ptr(vals), _ptr(meta), ct.byref(lr), _ptr(out), m, n, k, _ptr(ws),
                                         ws.numel(), _stream(A)))
    return out


def low_rank_backward(dy, x, down, up, index, scale=None, ranks=None, base=None, out=None, workspace=None):
    """Gradients of the adapters' part for dy [M, N] and the forward pass's x [M, K]: returns
    (dx, ddown, dup).  dx [M, K] has base (the shared projection's input gradient) added when that is
    given; ddown and dup are shaped and typed as the pool, zero where a slot or an adapter has no use."""
    torch = _torch()
    n = _channels(up)
    lr = _pool(x, n, down, up, index, scale, ranks)
    m, k = x.shape
    ldx = _rows(x, x, x.shape, "x")
    lddy = _rows(dy, x, (m, n), "dy")
    ldb = _rows(base, x, x.shape, "base") if base is not None else k
    dx, lddx = _out(out, x, x.shape)
    ddown, dup = torch.empty_like(down), torch.empty_like(up)
    lib = load()
    ws = _workspace(lib.low_rank_backward_workspace_bytes(lr.adapters, lr.R, m, n, k), x, workspace)
    with _on(x):
        _check(lib.low_rank_backward(ct.byref(lr), _ptr(dy), lddy, _ptr(x), ldx, _ptr(base), ldb, _ptr(dx), lddx,
                                     _ptr(ddown), _ptr(dup), m, n, k, _ptr(ws), ws.numel(), _stream(x)))
    return dx, ddown, dup


# ------------------------------------------------------------------------ loss
def _head(x, w, target):
    torch = _torch()
    dt = _code(x, "x", (SSG_DT_F16, SSG_DT_BF16))
    m, d = _matrix(x, "x")
    if not isinstance(w, torch.Tensor) or w.dim() != 2:
        raise ValueError("w must be a matrix [V, D]")
    v = w.shape[0]
    ldx = _rows(x, x, x.shape, "x")
    ldw = _rows(w, x, (v, d), "w")
    _flat(target, torch.int64, (m,), x, "target")
    return dt, m, v, d, ldx, ldw


def linear_cross_entropy(x, w, target, ignore_index=-100, workspace=None):
    """Softmax cross entropy of the logits x . w^T, which are never stored: x [M, D] and w [V, D] float16
    or bfloat16 (rows may be strided), target int64 [M].  Returns (loss, lse), float32 [M]: a row's loss (0
    where its target is ignore_index, NaN for a target outside the vocabulary) and its log-sum-exp, which
    the backward pass takes."""
    torch = _torch()
    dt, m, v, d, ldx, ldw = _head(x, w, target)
    loss = x.new_empty(m, dtype=torch.float32)
    lse = torch.empty_like(loss)
    lib = load()
    ws = _workspace(lib.linear_cross_entropy_workspace_bytes(dt, m, v, d, ldx, ldw, 0), x, workspace)
    with _on(x):
        _check(lib.linear_cross_entropy_forward(dt, _ptr(x), ldx, _ptr(w), ldw, _ptr(target), ignore_index, _ptr(loss),
                                                _ptr(lse), m, v, d, _ptr(ws), ws.numel(), _stream(x)))
    return loss, lse


def linear_cross_entropy_backward(dloss, x, w, target, lse, ignore_index=-100, out=None, dw_out=None, workspace=None):
    """Gradient of linear_cross_entropy for dloss float32 [M] (the derivative by each row's loss: 1 / rows for
    their mean) and its lse.  Returns (dx, dw) in x's type; the logits are computed again in pieces of the
    vocabulary.  In float16 a row whose |dloss| is below about 2^-18 of the largest loses digits of its dx."""
    torch = _torch()
    dt, m, v, d, ldx, ldw = _head(x, w, target)
    _flat(dloss, torch.float32, (m,), x, "dloss")
    _flat(lse, torch.float32, (m,), x, "lse")
    dx, lddx = _out(out, x, x.shape)
    dw, lddw = _out(dw_out, w, w.shape, "dw_out")
    lib = load()
    ws = _workspace(lib.linear_cross_entropy_workspace_bytes(dt, m, v, d, ldx, ldw, 1), x, workspace)
    with _on(x):
        _check(lib.linear_cross_entropy_backward(dt, _ptr(dloss), _ptr(x), ldx, _ptr(w), ldw, _ptr(target),
                                                 ignore_index, _ptr(lse), _ptr(dx), lddx, _ptr(dw), lddw, m, v, d,
                                                 _ptr(ws), ws.numel(), _stream(x)))
    return dx, dw
