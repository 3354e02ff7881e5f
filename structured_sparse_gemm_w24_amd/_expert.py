"""Binding of the calls for layers of experts: products grouped by expert with their
gradients, microscaled 4-bit (MXFP4) operands, the global gradient norm and clipping.

Same manner as ``_tune``: torch device tensors in and out, one library call on torch's
current stream, ``SsgError`` on a nonzero status, no fallback; rows may be strided, the
gradients are calls of their own and results carry no history.  An output or a workspace
that overlaps an input is refused.
"""

from __future__ import annotations

from array import array

from ._tune import (SSG_DT_BF16, SSG_DT_F16, _check, _code, _codes, _flat, _matrix, _on, _out, _ptr, _rows, _stream,
                    _torch, _workspace, load)

BLOCK, PAD = 32, 128  # values that share a scale; packed rows hold a multiple of this many
_HALF = (SSG_DT_F16, SSG_DT_BF16)


def _experts(w, name="w"):
    if not isinstance(w, _torch().Tensor) or w.dim() != 3:
        raise ValueError(f"{name} must be a tensor with an expert, a row and a column axis")
    return w.shape


def _offsets(offsets, e, like):
    _flat(offsets, _torch().int32, (e + 1,), like, "offsets")


# ------------------------------------------------------------ grouped products
def grouped_gemm(x, w, offsets, out=None):
    """out[m] = w[e] . x[m] for every row m of expert e: x [M, K], w [E, N, K], both float16 or bfloat16;
    offsets int32 [E + 1] on the device, expert e's rows are offsets[e] .. offsets[e + 1] (it may have none).
    Rows of no expert are left as they are in out, and undefined without one.  N and K multiples of 8;
    rows of x and out may be strided, in multiples of 8."""
    dt = _code(x, "x", _HALF)
    m, k = _matrix(x, "x")
    e, n, _ = _experts(w)
    ldx = _rows(x, x, x.shape, "x")
    _flat(w, x.dtype, (e, n, k), x, "w")
    _offsets(offsets, e, x)
    out, ldo = _out(out, x, (m, n))
    with _on(x):
        _check(load().grouped_gemm(dt, _ptr(x), ldx, _ptr(w), _ptr(offsets), e, _ptr(out), ldo, m, n, k, _stream(x)))
    return out


def grouped_gemm_backward(dy, x, w, offsets, out=None, dw_out=None, x_grad=True, w_grad=True, workspace=None):
    """Gradients of grouped_gemm for dy [M, N]: returns (dx, dw), dx [M, K] (rows of no expert as in
    grouped_gemm) and dw [E, N, K] (zeros for an expert without rows), in x's type; None for one that is
    not asked for."""
    dt = _code(x, "x", _HALF)
    m, k = _matrix(x, "x")
    e, n, _ = _experts(w)
    ldx = _rows(x, x, x.shape, "x")
    lddy = _rows(dy, x, (m, n), "dy")
    _flat(w, x.dtype, (e, n, k), x, "w")
    _offsets(offsets, e, x)
    dx = dw = None
    lddx = k
    if x_grad:
        dx, lddx = _out(out, x, (m, k))
    lib, ws = load(), None
    if w_grad:
        dw = _torch().empty_like(w) if dw_out is None else _flat(dw_out, x.dtype, (e, n, k), x, "dw_out")
        need = lib.grouped_gemm_backward_workspace_bytes(e, m, n, k)
        if need > 0:
            ws = _workspace(need, x, workspace)
    with _on(x):
        _check(lib.grouped_gemm_backward(dt, _ptr(dy), lddy, _ptr(x), ldx, _ptr(w), _ptr(offsets), e, _ptr(dx), lddx,
                                         _ptr(dw), m, n, k, _ptr(ws), ws.numel() if ws is not None else 0, _stream(x)))
    return dx, dw


def expert_tile(product, experts, m, n, k):
    """The entry of the library's table of tiles that a product of expert layers runs on (ssg_expert_tile in
    ssg.h: 0 grouped_gemm, 1 dx, 2 dw, 3 dx and dw in one launch, 4 the 4-bit products)."""
    return int(load().ssg_expert_tile(product, experts, m, n, k))


# ------------------------------------------------------------ microscaled 4 bit
def _padded(k):
    return -(-k // PAD) * PAD


def _packed(codes, scales, shape, k, like, name):
    """Codes [..., kp / 2] and scales [..., kp / 32] of rows of k values."""
    torch, kp = _torch(), _padded(k)
    _flat(codes, torch.uint8, (*shape, kp // 2), like, name)
    _flat(scales, torch.uint8, (*shape, kp // BLOCK), like, name + "'s scales")


def mxfp4_quantize(x, codes_out=None, scales_out=None):
    """x [M, K] (float16, bfloat16 or float32) as microscaled 4-bit rows: (codes, scales), uint8 of
    kp / 2 and kp / 32 columns with kp = K rounded up to 128.  Every 32 values along K share the scale
    2^(byte - 127), byte - 127 = floor(log2 of the largest) - 2; value 2i is in the low half of byte i."""
    torch = _torch()
    dt = _code(x, "x")
    m, k = _matrix(x, "x")
    ldx = _rows(x, x, x.shape, "x")
    kp = _padded(k)
    if codes_out is None:
        codes_out = x.new_empty((m, kp // 2), dtype=torch.uint8)
    else:
        _flat(codes_out, torch.uint8, (m, kp // 2), x, "codes_out")
    if scales_out is None:
        scales_out = x.new_empty((m, kp // BLOCK), dtype=torch.uint8)
    else:
        _flat(scales_out, torch.uint8, (m, kp // BLOCK), x, "scales_out")
    with _on(x):
        _check(load().mxfp4_quantize(dt, _ptr(x), ldx, _ptr(codes_out), _ptr(scales_out), m, k, _stream(x)))
    return codes_out, scales_out


def mxfp4_dequantize(codes, scales, k, dtype=None, out=None):
    """The values [M, k] that mxfp4_quantize's codes and scales stand for, as dtype (float32)."""
    torch = _torch()
    dtype = dtype or (out.dtype if out is not None else torch.float32)
    if dtype not in _codes():
        raise TypeError(f"dtype {dtype}, which this call does not write")
    if not isinstance(codes, torch.Tensor) or not codes.is_cuda or codes.dim() != 2:
        raise TypeError("codes must be a matrix on a HIP device")
    m = codes.shape[0]
    _packed(codes, scales, (m,), k, codes, "codes")
    if out is None:
        out, ldo = codes.new_empty((m, k), dtype=dtype), k
    else:
        if out.dtype is not dtype:
            raise TypeError(f"out must be {dtype}, got {out.dtype}")
        if out.device != codes.device:
            raise TypeError(f"out must be a torch tensor on {codes.device}")
        ldo = _rows(out, out, (m, k), "out")
    with _on(codes):
        _check(load().mxfp4_dequantize(_ptr(codes), _ptr(scales), _codes()[dtype], _ptr(out), ldo, m, k,
                                       _stream(codes)))
    return out


def mxfp4_gemm(a, a_scales, w, w_scales, k, dtype=None, offsets=None, out=None):
    """out[m, n] = sum over k of a[m] w[n], both packed by mxfp4_quantize from rows of k values; fp32 sums,
    one rounding to dtype (float16; bfloat16 or float32).  With offsets (as in grouped_gemm) w is
    [E, N, kp / 2] and row m meets its expert's matrix."""
    torch = _torch()
    dtype = dtype or (out.dtype if out is not None else torch.float16)
    if dtype not in _codes():
        raise TypeError(f"dtype {dtype}, which this call does not write")
    if not isinstance(a, torch.Tensor) or not a.is_cuda or a.dim() != 2:
        raise TypeError("a must be a matrix on a HIP device")
    m = a.shape[0]
    _packed(a, a_scales, (m,), k, a, "a")
    e, n = _mx_weight(w, w_scales, offsets, k, a)
    if out is None:
        out, ldo = a.new_empty((m, n), dtype=dtype), n
    else:
        if out.dtype is not dtype:
            raise TypeError(f"out must be {dtype}, got {out.dtype}")
        if out.device != a.device:
            raise TypeError(f"out must be a torch tensor on {a.device}")
        ldo = _rows(out, out, (m, n), "out")
    with _on(a):
        _check(load().mxfp4_gemm(_ptr(a), _ptr(a_scales), _ptr(w), _ptr(w_scales), _ptr(offsets), e, _codes()[dtype],
                                 _ptr(out), ldo, m, n, k, _stream(a)))
    return out


def _mx_weight(w, w_scales, offsets, k, like):
    if offsets is None:
        if not isinstance(w, _torch().Tensor) or w.dim() != 2:
            raise ValueError("w must be a matrix of packed rows")
        e, n = 1, w.shape[0]
        _packed(w, w_scales, (n,), k, like, "w")
    else:
        e, n, _ = _experts(w)
        _packed(w, w_scales, (e, n), k, like, "w")
        _offsets(offsets, e, like)
    return e, n


def _mx_linear(x, w, w_scales, offsets, out, workspace):
    dt = _code(x, "x", _HALF)
    m, k = _matrix(x, "x")
    ldx = _rows(x, x, x.shape, "x")
    e, n = _mx_weight(w, w_scales, offsets, k, x)
    out, ldo = _out(out, x, (m, n))
    lib = load()
    ws = _workspace(lib.mxfp4_linear_workspace_bytes(m, k), x, workspace)
    with _on(x):
        _check(lib.mxfp4_linear(dt, _ptr(x), ldx, _ptr(w), _ptr(w_scales), _ptr(offsets), e, _ptr(out), ldo, m, n, k,
                                _ptr(ws), ws.numel(), _stream(x)))
    return out


def mxfp4_linear(x, w, w_scales, out=None, workspace=None):
    """x . w^T of x [M, K] (float16 or bfloat16, quantised in the call as mxfp4_quantize does) and a weight
    of N packed rows, in x's type."""
    return _mx_linear(x, w, w_scales, None, out, workspace)


def mxfp4_grouped_linear(x, w, w_scales, offsets, out=None, workspace=None):
    """mxfp4_linear with an expert's weight for every row: w [E, N, kp / 2], offsets and the rows of no
    expert as in grouped_gemm."""
    if offsets is None:
        raise TypeError("offsets must be an int32 tensor")
    return _mx_linear(x, w, w_scales, offsets, out, workspace)


# ---------------------------------------------------------------- gradient norm
def _dense(t):
    """Whether t's elements fill one run of memory, in whatever order of its axes."""
    if t.is_contiguous():
        return True
    step = 1
    for stride, size in sorted(zip(t.stride(), t.shape)):
        if size != 1:
            if stride != step:
                return False
            step *= size
    return True


# (a model has hundreds of tensors, and each look at one from Python is 50 to 100 ns: what the checks
# of a good list need is asked for once, in comprehensions, and a bad one is looked at again)
def _list(grads, name):
    """Checks a list of tensors on one device; returns it, whether all are contiguous, its device, sizes and
    types, and the C arrays of addresses, sizes and types."""
    codes = _codes()
    grads = list(grads)
    if not grads:
        raise ValueError(f"{name} is empty")
    try:
        devices = {t.get_device() for t in grads}
        types = [codes.get(t.dtype, -1) for t in grads]
        plain = all([t.is_contiguous() for t in grads])
        sizes = [t.numel() for t in grads]
        ptrs = array("Q", [t.data_ptr() for t in grads])
    except AttributeError:  # not all are tensors
        _refuse_list(grads, name)
        raise
    if len(devices) != 1 or -1 in devices or -1 in types or not (plain or all([_dense(t) for t in grads])):
        _refuse_list(grads, name)
    return grads, plain, devices, sizes, types, ptrs, array("q", sizes), array("i", types)


def _refuse_list(grads, name):
    torch, codes = _torch(), _codes()
    for t in grads:
        if not isinstance(t, torch.Tensor) or not t.is_cuda:
            raise TypeError(f"{name} must be torch tensors on a HIP device")
        if t.device != grads[0].device:
            raise TypeError(f"{name} must be on one device, got {grads[0].device} and {t.device}")
        if t.dtype not in codes:
            raise TypeError(f"{name} of type {t.dtype}, which this call does not take")
        if not _dense(t):
            raise ValueError(f"{name} must each fill one run of memory, got strides {t.stride()} of {tuple(t.shape)}")


def _at(a):
    """Address of an array's items."""
    return a.buffer_info()[0]


def grad_norm(grads, workspace=None):
    """The 2-norm of all elements of the tensors (float16, bfloat16, float32, mixed) as a float32 scalar
    tensor; squares are summed in 64 bits, in a fixed order."""
    torch = _torch()
    grads, _, _, _, _, ptrs, sizes, types = _list(grads, "grads")
    like = grads[0]
    norm = like.new_empty((), dtype=torch.float32)
    lib = load()
    ws = _norm_workspace(lib, len(grads), like, workspace)
    with _on(like):
        _check(lib.grad_norm(len(grads), _at(ptrs), _at(sizes), _at(types), _ptr(norm), _ptr(ws), ws.numel(), _stream(like)))
    return norm


def clip_grad_norm(grads, max_norm, norm=None, out=None, workspace=None):
    """Every gradient times min(1, max_norm / (norm + 1e-6)): returns (norm, clipped).  norm: grad_norm of
    the list, or a float32 scalar tensor to clip by instead (one that was reduced over ranks); an infinite one
    makes the factor 0.  (The list's own norm clips in 64 bits, also where float32 holds it as infinite.)  out: the
    tensors to write, grads themselves for clipping in place (left untouched where nothing is clipped);
    None makes new ones.  Tensors that share elements with one that is written are refused."""
    torch = _torch()
    given_grads = grads
    grads, plain, devices, numels, codes, ptrs, sizes, types = _list(grads, "grads")
    like = grads[0]
    n = len(grads)
    if out is None:
        out = [torch.empty_like(t) for t in grads]
        outs = array("Q", [t.data_ptr() for t in out])
    elif out is given_grads:
        out, outs = grads, ptrs
    else:
        out = list(out)
        if len(out) != n:
            raise ValueError(f"{len(out)} outputs for {n} gradients")
        out, oplain, odevices, onumels, ocodes, outs, _, _ = _list(out, "out")
        if ocodes != codes or odevices != devices:
            raise TypeError("out must have the types of grads, on their device")
        if onumels != numels or not (plain and oplain or all([
                (o.is_contiguous() and t.is_contiguous()) or (o.shape == t.shape and o.stride() == t.stride())
                for o, t in zip(out, grads)])):
            raise ValueError("out must be contiguous with grads' sizes, or have the shapes and strides of grads")
    lib = load()
    ws, given = None, norm
    if given is None:
        norm = like.new_empty((), dtype=torch.float32)
        ws = _norm_workspace(lib, n, like, workspace)
    elif not isinstance(given, torch.Tensor) or given.numel() != 1:
        raise ValueError("norm must be a tensor of one element")
    else:
        _flat(given, torch.float32, given.shape, like, "norm")
    with _on(like):
        _check(lib.clip_grad_norm(n, _at(ptrs), _at(outs), _at(sizes), _at(types), float(max_norm), _ptr(given),
                                  _ptr(norm) if given is None else None, _ptr(ws), ws.numel() if ws is not None else 0,
                                  _stream(like)))
    return norm, out


def _norm_workspace(lib, n, like, workspace):
    torch = _torch()
    if workspace is not None:
        return _flat(workspace, torch.uint8, workspace.shape, like, "workspace")
    return like.new_empty(lib.grad_norm_workspace_bytes(n), dtype=torch.uint8)
