"""The calls for layers of experts: refusals on the host, workspace sizes, and the
register, LDS and scratch budget of their kernels (no GPU)."""

import ctypes as ct
import os
import re
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
KDIR = os.path.join(ROOT, "structured_sparse_gemm_w24_amd", "csrc", "kernels")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
F16, BF16, F32 = 0, 1, 2


def _p(v):
    return ct.c_void_p(v)


def _fwd(r, dtype=F16, x=16, ldx=64, w=16, offsets=16, experts=2, out=16, ldo=64, m=4, n=64, k=64):
    return r.grouped_gemm(dtype, _p(x), ldx, _p(w), _p(offsets), experts, _p(out), ldo, m, n, k, None)


def _bwd(r, dtype=F16, dy=16, lddy=64, x=16, ldx=64, w=16, offsets=16, experts=2, dx=16, lddx=64, dw=16, m=4, n=64,
         k=64, ws=16, size=1 << 30):
    return r.grouped_gemm_backward(dtype, _p(dy), lddy, _p(x), ldx, _p(w), _p(offsets), experts, _p(dx), lddx, _p(dw),
                                   m, n, k, _p(ws), size, None)


def _quant(r, dtype=F16, x=16, ldx=100, codes=16, scales=16, m=4, k=100):
    return r.mxfp4_quantize(dtype, _p(x), ldx, _p(codes), _p(scales), m, k, None)


def _dequant(r, dtype=F16, codes=16, scales=16, out=16, ldo=100, m=4, k=100):
    return r.mxfp4_dequantize(_p(codes), _p(scales), dtype, _p(out), ldo, m, k, None)


def _gemm(r, a=16, sa=16, w=16, sw=16, offsets=None, experts=1, dtype=F16, out=16, ldo=70, m=4, n=70, k=100):
    return r.mxfp4_gemm(_p(a), _p(sa), _p(w), _p(sw), _p(offsets), experts, dtype, _p(out), ldo, m, n, k, None)


def _linear(r, dtype=F16, x=16, ldx=100, w=16, sw=16, offsets=None, experts=1, out=16, ldo=70, m=4, n=70, k=100, ws=16,
            size=1 << 20):
    return r.mxfp4_linear(dtype, _p(x), ldx, _p(w), _p(sw), _p(offsets), experts, _p(out), ldo, m, n, k, _p(ws), size,
                          None)


def _lists(grads, sizes, types, outs=None):
    n = len(grads)
    arr = lambda t, v: (t * max(n, 1))(*v)
    return (n, arr(ct.c_void_p, grads), arr(ct.c_void_p, outs if outs is not None else grads), arr(ct.c_int64, sizes),
            arr(ct.c_int32, types))


def _norm(r, grads=(4096,), sizes=(8,), types=(F16,), norm=16, ws=16, size=1 << 20):
    n, g, _, s, t = _lists(grads, sizes, types)
    return r.grad_norm(n, g, s, t, _p(norm), _p(ws), size, None)


def _clip(r, grads=(4096,), sizes=(8,), types=(F16,), outs=None, most=1.0, norm_in=None, norm=16, ws=16, size=1 << 20):
    n, g, o, s, t = _lists(grads, sizes, types, outs)
    return r.clip_grad_norm(n, g, o, s, t, most, _p(norm_in), _p(norm), _p(ws), size, None)


@pytest.mark.parametrize("call,msg", [
    (lambda r: _fwd(r, dtype=F32), "must be fp16 or bf16"),
    (lambda r: _fwd(r, m=-1), "M=-1"),
    (lambda r: _fwd(r, n=60), "multiples of 8"),
    (lambda r: _fwd(r, k=4), "multiples of 8"),
    (lambda r: _fwd(r, n=1 << 22), "2^22"),
    (lambda r: _fwd(r, n=1 << 16, k=1 << 15, ldx=1 << 15, ldo=1 << 16), "2 GiB"),
    (lambda r: _fwd(r, m=1 << 29), "2^29"),
    (lambda r: _fwd(r, experts=0), "experts=0"),
    (lambda r: _fwd(r, experts=65536), "experts=65536"),
    (lambda r: _fwd(r, offsets=None), "offsets"),
    (lambda r: _fwd(r, offsets=18), "offsets"),
    (lambda r: _fwd(r, ldx=56), "row stride"),
    (lambda r: _fwd(r, ldo=68), "row stride"),
    (lambda r: _fwd(r, ldx=1 << 22), "row stride"),
    (lambda r: _fwd(r, x=None), "x null"),
    (lambda r: _fwd(r, x=24), "16-byte aligned"),
    (lambda r: _fwd(r, w=None), "w null"),
    (lambda r: _fwd(r, out=None), "out null"),
    (lambda r: _fwd(r, m=(1 << 29) - 1, n=1 << 20, ldo=1 << 20), "too large"),
    (lambda r: _bwd(r, dy=None), "dy null"),
    (lambda r: _bwd(r, lddy=60), "row stride"),
    (lambda r: _bwd(r, w=None), "w null"),
    (lambda r: _bwd(r, x=None), "x null"),
    (lambda r: _bwd(r, lddx=60), "row stride"),
    (lambda r: _bwd(r, dw=24), "16-byte aligned"),
    (lambda r: _bwd(r, m=9000, experts=1, ws=None), "workspace null"),
    (lambda r: _bwd(r, m=9000, experts=1, size=64), "needed"),
    (lambda r: _quant(r, dtype=3), "unknown dtype"),
    (lambda r: _quant(r, k=0), "K=0"),
    (lambda r: _quant(r, k=1 << 22), "2^22"),
    (lambda r: _quant(r, ldx=99), "row stride"),
    (lambda r: _quant(r, x=17), "aligned to its elements"),
    (lambda r: _quant(r, codes=8), "16-byte aligned"),
    (lambda r: _quant(r, scales=18), "4-byte aligned"),
    (lambda r: _quant(r, scales=None), "null"),
    (lambda r: _dequant(r, dtype=-1), "unknown dtype"),
    (lambda r: _dequant(r, out=None), "out null"),
    (lambda r: _dequant(r, ldo=64), "row stride"),
    (lambda r: _gemm(r, dtype=5), "unknown dtype"),
    (lambda r: _gemm(r, n=0), "N=0"),
    (lambda r: _gemm(r, m=1 << 29), "2^29"),
    (lambda r: _gemm(r, m=(1 << 29) - 64, n=1 << 21, k=128, ldo=1 << 21), "too large"),
    (lambda r: _quant(r, m=(1 << 31) - 1, k=1000, ldx=1000), "2^36"),
    (lambda r: _gemm(r, experts=2), "without offsets"),
    (lambda r: _gemm(r, offsets=16, experts=0), "experts=0"),
    (lambda r: _gemm(r, a=None), "codes of a"),
    (lambda r: _gemm(r, sw=None), "codes of w"),
    (lambda r: _gemm(r, ldo=69), "row stride"),
    (lambda r: _gemm(r, n=1 << 21, k=1 << 13, ldo=1 << 21), "2 GiB"),
    (lambda r: _linear(r, dtype=F32), "must be fp16 or bf16"),
    (lambda r: _linear(r, x=None), "x null"),
    (lambda r: _linear(r, ws=None), "workspace null"),
    (lambda r: _linear(r, size=4 * 64 + 4 * 4 - 1), "needed"),
    (lambda r: _norm(r, types=(7,)), "unknown dtype"),
    (lambda r: _norm(r, sizes=(-1,)), "elements"),
    (lambda r: _norm(r, grads=(None,)), "tensor 0 null"),
    (lambda r: _norm(r, grads=(4097,)), "aligned to its elements"),
    (lambda r: _norm(r, norm=None), "norm null"),
    (lambda r: _norm(r, ws=None), "workspace null"),
    (lambda r: _norm(r, size=8), "needed"),
    (lambda r: r.grad_norm(-1, None, None, None, _p(16), _p(16), 0, None), "n=-1"),
    (lambda r: r.grad_norm(1, None, None, None, _p(16), _p(16), 1 << 20, None), "null list"),
    (lambda r: _clip(r, most=-0.5), "max_norm"),
    (lambda r: _clip(r, most=float("nan")), "max_norm"),
    (lambda r: _clip(r, outs=(None,)), "output 0 null"),
    (lambda r: _clip(r, outs=(4098,)), "overlaps"),
    (lambda r: _clip(r, grads=(4096, 4096), sizes=(8, 8), types=(F16, F16)), "overlaps"),
    (lambda r: _clip(r, grads=(4096, 4100), sizes=(8, 8), types=(F16, F32)), "overlaps"),
    (lambda r: _clip(r, grads=(4096, 8192), outs=(8192, 12288), sizes=(8, 8), types=(F16, F16)), "overlaps"),
    (lambda r: _clip(r, grads=(4096, 8192), outs=(12288, 12296), sizes=(8, 8), types=(F16, F16)), "overlaps"),
    (lambda r: _clip(r, norm=None), "norm null"),
    (lambda r: _clip(r, norm_in=18), "norm_in"),
    (lambda r: _clip(r, norm_in=4108), "norm_in overlaps"),
    (lambda r: _norm(r, grads=(4096,) * 5, sizes=((1 << 40) - 1,) * 5, types=(F32,) * 5), "16 TiB"),
    (lambda r: r.grad_norm((1 << 20) + 1, _p(16), _p(16), _p(16), _p(16), _p(16), 1 << 30, None), "2^20"),
])
def test_refused_on_host(lib, call, msg):
    raw = lib.load()
    assert call(raw) == 1, raw.ssg_last_error().decode()  # SSG_EINVAL
    assert msg in raw.ssg_last_error().decode(), raw.ssg_last_error().decode()


def test_no_rows_is_ok_without_touching_the_device(lib):
    raw = lib.load()
    assert _fwd(raw, m=0, x=None, w=None, out=None) == 0
    assert _bwd(raw, m=0, dy=None, x=None, w=None, dw=None, ws=None, size=0) == 0
    assert _bwd(raw, dx=None, dw=None, w=None, x=None, ws=None, size=0) == 0
    assert _quant(raw, m=0, x=None, codes=None, scales=None) == 0
    assert _dequant(raw, m=0, codes=None, scales=None, out=None) == 0
    assert _gemm(raw, m=0, a=None, sa=None, w=None, sw=None, out=None) == 0
    assert _linear(raw, m=0, x=None, w=None, sw=None, out=None, ws=None, size=0) == 0


def test_workspace_sizes(lib):
    raw = lib.load()
    assert raw.mxfp4_linear_workspace_bytes(3, 100) == 3 * (64 + 4)
    assert raw.mxfp4_linear_workspace_bytes(0, 100) == 0
    assert raw.mxfp4_linear_workspace_bytes(-1, 100) == 0
    assert raw.grad_norm_workspace_bytes(0) == 0 and raw.grad_norm_workspace_bytes(-3) == 0
    assert 0 < raw.grad_norm_workspace_bytes(1) <= raw.grad_norm_workspace_bytes(1000) <= 1 << 17
    # the weight gradient: nothing where its tiles fill the device; slices within 256 MiB else
    assert raw.grouped_gemm_backward_workspace_bytes(16, 16384, 4096, 1024) == 0
    assert raw.grouped_gemm_backward_workspace_bytes(0, 16384, 4096, 1024) == 0
    assert raw.grouped_gemm_backward_workspace_bytes(2, 100, 60, 64) == 0
    for e in (1, 2, 7, 64):
        for m in (0, 1, 100, 5000, 100000, (1 << 29) - 1):
            for n, k in ((8, 8), (64, 720), (1024, 1024), (8192, 4096)):
                w = raw.grouped_gemm_backward_workspace_bytes(e, m, n, k)
                assert w % (e * n * k * 4) == 0 and w <= 256 << 20


def _kernels(asm):
    out = {}
    for m in re.finditer(r"^\s*\.amdhsa_kernel (\S+)\n(.*?)\.end_amdhsa_kernel", asm, re.M | re.S):
        val = lambda k: int(re.search(r"\.amdhsa_" + k + r"\s+(\d+)", m.group(2)).group(1))
        out[m.group(1)] = dict(lds=val("group_segment_fixed_size"), vgpr=val("next_free_vgpr"),
                               scratch=val("private_segment_fixed_size"))
    return out


@pytest.mark.parametrize("source,least", [("grouped.hip", 40), ("mxfp4.hip", 40), ("grad_norm.hip", 3)])
def test_no_spills_and_lds_fits(source, least, tmp_path):
    if shutil.which(HIPCC) is None and not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    from structured_sparse_gemm_w24_amd.build import HIP_FLAGS
    flags = [f for f in HIP_FLAGS if f not in ("-fPIC", "-fvisibility=hidden")]
    out = tmp_path / "k.s"
    p = subprocess.run([HIPCC, *flags, "--cuda-device-only", "-S", os.path.join(KDIR, source), "-o", str(out)],
                       capture_output=True, text=True)
    assert p.returncode == 0, p.stderr
    asm = out.read_text()
    found = _kernels(asm)
    assert len(found) >= least, len(found)
    assert {k: v["scratch"] for k, v in found.items() if v["scratch"]} == {}
    assert {k: v["lds"] for k, v in found.items() if v["lds"] > 160 * 1024} == {}
    assert not re.search(r"^\s*v_pk_(fma|mul|add)_f32", asm, re.M)
