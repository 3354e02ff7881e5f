"""Outputs that overlap inputs are refused on the host; rows of one buffer beside each other are not (no GPU:
a call that passes these checks fails for want of a device, or would only ask for one)."""

import ctypes as ct

import pytest

F16, F32 = 0, 2
E, M, N, K = 2, 40, 64, 64
FAR = 1 << 30


def _p(v):
    return ct.c_void_p(v)


def _fwd(r, x=1 << 20, ldx=K, w=2 << 20, offsets=3 << 20, out=4 << 20, ldo=N):
    return r.grouped_gemm(F16, _p(x), ldx, _p(w), _p(offsets), E, _p(out), ldo, M, N, K, None)


def _bwd(r, dy=1 << 20, lddy=N, x=2 << 20, w=3 << 20, offsets=4 << 20, dx=5 << 20, lddx=K, dw=6 << 20, m=M, e=E,
         ws=FAR):
    return r.grouped_gemm_backward(F16, _p(dy), lddy, _p(x), K, _p(w), _p(offsets), e, _p(dx), lddx, _p(dw), m, N, K,
                                   _p(ws), 1 << 29, None)


def _quant(r, x=1 << 20, ldx=100, codes=2 << 20, scales=3 << 20, dtype=F16, m=M):
    return r.mxfp4_quantize(dtype, _p(x), ldx, _p(codes), _p(scales), m, 100, None)


def _dequant(r, codes=1 << 20, scales=2 << 20, out=3 << 20, ldo=100):
    return r.mxfp4_dequantize(_p(codes), _p(scales), F32, _p(out), ldo, M, 100, None)


def _gemm(r, a=1 << 20, sa=2 << 20, w=3 << 20, sw=4 << 20, offsets=5 << 20, out=6 << 20, ldo=N):
    return r.mxfp4_gemm(_p(a), _p(sa), _p(w), _p(sw), _p(offsets), E, F16, _p(out), ldo, M, N, 100, None)


def _linear(r, x=1 << 20, ldx=100, w=2 << 20, sw=3 << 20, offsets=4 << 20, out=5 << 20, ldo=N, ws=6 << 20):
    return r.mxfp4_linear(F16, _p(x), ldx, _p(w), _p(sw), _p(offsets), E, _p(out), ldo, M, N, 100, _p(ws), 1 << 20,
                          None)


def _norm(r, grads=(1 << 20,), norm=2 << 20, ws=3 << 20):
    n = len(grads)
    return r.grad_norm(n, (ct.c_void_p * n)(*grads), (ct.c_int64 * n)(*[8] * n), (ct.c_int32 * n)(*[F32] * n),
                       _p(norm), _p(ws), 1 << 20, None)


def _clip(r, grads=(1 << 20,), outs=(4 << 20,), norm=2 << 20, ws=3 << 20, norm_in=None):
    n = len(grads)
    return r.clip_grad_norm(n, (ct.c_void_p * n)(*grads), (ct.c_void_p * n)(*outs), (ct.c_int64 * n)(*[8] * n),
                            (ct.c_int32 * n)(*[F32] * n), 1.0, _p(norm_in), _p(norm), _p(ws), 1 << 20, None)


MB = 1 << 20
ROW = 2 * N
REFUSED = [
    (lambda r: _fwd(r, out=MB), "out overlaps x"),
    (lambda r: _fwd(r, out=MB + (M - 1) * ROW), "out overlaps x"),
    (lambda r: _fwd(r, out=MB - (M - 1) * ROW - 16), "out overlaps x"),
    (lambda r: _fwd(r, out=2 * MB + E * N * K * 2 - 16), "out overlaps w"),
    (lambda r: _fwd(r, out=3 * MB - M * ROW + 16), "out overlaps offsets"),
    # columns 0..63 and 56..119 of rows of 128; rows 0, 2, 4 .. and 3, 6, 9 ..
    (lambda r: _fwd(r, ldx=128, ldo=128, out=MB + 112), "out overlaps x"),
    (lambda r: _fwd(r, ldx=2 * N, ldo=3 * N, out=MB + 3 * ROW), "out overlaps x"),
    (lambda r: _bwd(r, dx=MB), "dx overlaps dy"),
    (lambda r: _bwd(r, dx=2 * MB), "dx overlaps x"),
    (lambda r: _bwd(r, dx=3 * MB), "dx overlaps w"),
    (lambda r: _bwd(r, dw=3 * MB), "dw overlaps w"),
    (lambda r: _bwd(r, dw=5 * MB), "dx overlaps dw"),
    (lambda r: _bwd(r, dw=4 * MB), "dw overlaps offsets"),
    (lambda r: _bwd(r, e=1, m=9000, dy=16 * MB, dx=None, dw=8 * MB, ws=2 * MB), "workspace overlaps x"),
    (lambda r: _quant(r, codes=MB), "codes overlaps x"),
    (lambda r: _quant(r, scales=2 * MB + 64), "codes overlaps scales"),
    (lambda r: _dequant(r, out=MB), "out overlaps codes"),
    (lambda r: _dequant(r, out=2 * MB + 4), "out overlaps scales"),
    (lambda r: _gemm(r, out=MB), "out overlaps a"),
    (lambda r: _gemm(r, out=2 * MB), "out overlaps a's scales"),
    (lambda r: _gemm(r, out=3 * MB + N * 64), "out overlaps w"),
    (lambda r: _gemm(r, out=4 * MB + N * 4), "out overlaps w's scales"),
    (lambda r: _linear(r, out=MB + 2), "out overlaps x"),
    (lambda r: _linear(r, ws=MB), "workspace overlaps x"),
    (lambda r: _linear(r, ws=5 * MB), "out overlaps the workspace"),
    (lambda r: _norm(r, norm=MB + 28), "norm overlaps a tensor (entry 0)"),
    (lambda r: _norm(r, grads=(MB, 3 * MB + 64)), "workspace overlaps a tensor (entry 1)"),
    (lambda r: _norm(r, norm=3 * MB + 8), "norm overlaps the workspace"),
    (lambda r: _clip(r, norm=4 * MB), "norm overlaps an output"),
    (lambda r: _clip(r, norm=MB + 4), "norm overlaps a tensor"),
    (lambda r: _clip(r, ws=4 * MB - 32), "workspace overlaps an output"),
]


@pytest.mark.parametrize("call,msg", REFUSED)
def test_refused(lib, call, msg):
    raw = lib.load()
    assert call(raw) == 1, raw.ssg_last_error().decode()  # SSG_EINVAL
    assert msg in raw.ssg_last_error().decode(), raw.ssg_last_error().decode()


APART = [
    lambda r: _fwd(r),
    lambda r: _fwd(r, out=MB + M * ROW),
    lambda r: _fwd(r, out=MB - M * ROW),
    lambda r: _fwd(r, ldx=128, ldo=128, out=MB + 128),             # columns 0..63 and 64..127
    lambda r: _fwd(r, ldx=128, ldo=128, x=MB + 128, out=MB),
    lambda r: _fwd(r, ldx=128, ldo=128, out=MB + 128 + 256 * 7),   # rows further down
    lambda r: _fwd(r, ldx=2 * N, ldo=2 * N, out=MB + ROW),         # even rows and odd ones
    lambda r: _fwd(r, ldx=4 * N, ldo=2 * N, out=MB + ROW),
    lambda r: _fwd(r, ldo=128, offsets=4 * MB + 128),              # behind a row, before the next
    lambda r: _bwd(r, dw=None, x=5 * MB),                          # (x is not read)
    lambda r: _bwd(r, dx=None, w=6 * MB),                          # (nor w)
    lambda r: _quant(r, dtype=F32, m=1, ldx=1 << 61),              # one row, of any stride
    lambda r: _norm(r, norm=MB + 32),
    lambda r: _clip(r, norm=MB + 32),
    lambda r: _clip(r, norm=4 * MB, ws=MB, norm_in=5 * MB),        # (neither is used)
]


@pytest.mark.parametrize("call", APART)
def test_not_refused(lib, call):
    """The checks pass: what is left is to find a device (there is none here, or the process sees none)."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("would launch on made-up addresses")
    raw = lib.load()
    assert call(raw) > 1, raw.ssg_last_error().decode()  # SSG_ENODEV


@pytest.mark.gpu
def test_columns_of_one_buffer(lib, gpu):
    import torch
    g = torch.Generator().manual_seed(2)
    both = torch.randn(M, 160, generator=g).half().cuda()
    w = torch.randn(E, N, K, generator=g).half().cuda() / 8
    offsets = torch.tensor([0, 11, M], dtype=torch.int32, device="cuda")
    x = both[:, 8:72].contiguous()
    want = lib.grouped_gemm(x, w, offsets)
    lib.grouped_gemm(both[:, 8:72], w, offsets, out=both[:, 72:136])
    assert torch.equal(both[:, 72:136], want) and torch.equal(both[:, 8:72], x)
    for out in (both[:, 8:72], both[:, 64:128]):
        with pytest.raises(lib.SsgError, match="out overlaps x"):
            lib.grouped_gemm(both[:, 8:72], w, offsets, out=out)
    codes, scales = lib.mxfp4_quantize(w[0])
    with pytest.raises(lib.SsgError, match="out overlaps x"):
        lib.mxfp4_linear(x, codes, scales, out=x)
    with pytest.raises(lib.SsgError, match="dx overlaps dy"):
        lib.grouped_gemm_backward(x, x.clone(), w, offsets, out=x)
