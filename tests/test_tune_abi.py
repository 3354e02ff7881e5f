"""The calls that tune and serve pruned layers: refusals on the host, workspace
sizes, and the register, LDS and scratch budget of their kernels (no GPU)."""

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


def _lr(dtype=F16, adapters=2, R=16, down=16, up=16, scale=16, ranks=16, index=16):
    from structured_sparse_gemm_w24_amd._tune import _LowRank
    return ct.byref(_LowRank(down, up, scale, ranks, index, dtype, adapters, R))


def _norm(r, dtype=F16, x=16, ldx=32, res=None, w=16, b=16, wt=F16, eps=1e-5, y=16, ldy=32, s=None, mean=16, rstd=16,
          m=4, n=32):
    return r.layer_norm_forward(dtype, _p(x), ldx, _p(res), 32, _p(w), _p(b), wt, eps, _p(y), ldy, _p(s), 32, _p(mean),
                                _p(rstd), m, n, None)


def _norm_bwd(r, dtype=F16, w=16, wt=F16, dw=16, db=16, m=4, n=32, ws=16, size=1 << 20, lddx=32, mean=16):
    return r.layer_norm_backward(dtype, _p(16), 32, _p(16), 32, _p(mean), _p(16), _p(w), wt, None, 32, _p(16), lddx,
                                 _p(dw), _p(db), m, n, _p(ws), size, None)


def _add(r, lr=None, x=16, ldx=64, ldo=64, out=16, m=200, n=64, k=64, ws=16, size=1 << 20):
    return r.low_rank_add(lr if lr is not None else _lr(), _p(x), ldx, _p(16), 64, _p(out), ldo, m, n, k, _p(ws), size,
                          None)


def _w24(r, lr=None, m=200, n=64, k=64, meta=16, ws=16, size=1 << 20):
    return r.w24_low_rank_gemm_f16(_p(16), _p(16), _p(meta), lr if lr is not None else _lr(), _p(16), m, n, k, _p(ws),
                                   size, None)


def _lr_bwd(r, lr=None, ddown=16, m=200, n=64, k=64, lddy=64, size=1 << 24):
    return r.low_rank_backward(lr if lr is not None else _lr(), _p(16), lddy, _p(16), 64, None, 0, _p(16), 64,
                               _p(ddown), _p(16), m, n, k, _p(16), size, None)


def _loss(r, dtype=F16, x=16, ldx=64, ldw=64, target=16, loss=16, m=4, v=100, d=64, size=1 << 24):
    return r.linear_cross_entropy_forward(dtype, _p(x), ldx, _p(16), ldw, _p(target), -100, _p(loss), _p(16), m, v, d,
                                          _p(16), size, None)


def _loss_bwd(r, dw=16, dloss=16, lddx=64, m=4, v=100, d=64, size=1 << 24):
    return r.linear_cross_entropy_backward(F16, _p(dloss), _p(16), 64, _p(16), 64, _p(16), -100, _p(16), _p(16), lddx,
                                           _p(dw), 64, m, v, d, _p(16), size, None)


@pytest.mark.parametrize("call,msg", [
    (lambda r: _norm(r, dtype=3), "unknown dtype"),
    (lambda r: _norm(r, wt=BF16), "weight type"),
    (lambda r: _norm(r, n=0), "N=0"),
    (lambda r: _norm(r, m=-1), "M=-1"),
    (lambda r: _norm(r, eps=-1e-5), "eps"),
    (lambda r: _norm(r, ldx=31), "row stride"),
    (lambda r: _norm(r, ldy=0), "row stride"),
    (lambda r: _norm(r, x=None), "null"),
    (lambda r: _norm(r, x=17), "aligned"),
    (lambda r: _norm(r, res=16), "go together"),
    (lambda r: _norm(r, mean=None), "go together"),
    (lambda r: _norm_bwd(r, dw=None), "go together"),
    (lambda r: _norm_bwd(r, lddx=8), "row stride"),
    (lambda r: _norm_bwd(r, mean=None), "null"),
    (lambda r: _norm_bwd(r, ws=None), "workspace null"),
    (lambda r: _norm_bwd(r, size=255), "needed"),
    (lambda r: _add(r, lr=_lr(dtype=F32)), "must be fp16 or bf16"),
    (lambda r: _add(r, lr=_lr(R=12)), "multiple of 8"),
    (lambda r: _add(r, lr=_lr(R=136)), "at most 128"),
    (lambda r: _add(r, lr=_lr(adapters=0)), "adapters=0"),
    (lambda r: _add(r, lr=_lr(down=None)), "null"),
    (lambda r: _add(r, lr=_lr(up=24)), "16-byte aligned"),
    (lambda r: _add(r, lr=_lr(index=18)), "misaligned"),
    (lambda r: _add(r, k=60), "multiples of 8"),
    (lambda r: _add(r, ldx=68), "row stride"),
    (lambda r: _add(r, ldo=56), "row stride"),
    (lambda r: _add(r, out=None), "out is null"),
    (lambda r: _add(r, ws=None), "workspace null"),
    (lambda r: _add(r, size=64), "needed"),
    (lambda r: _w24(r, lr=_lr(dtype=BF16)), "must be fp16"),
    (lambda r: _w24(r, n=96), "multiple of 64"),
    (lambda r: _w24(r, meta=None), "meta"),
    (lambda r: _w24(r, size=64), "needed"),
    (lambda r: _w24(r, m=8, size=8 * 64 * 4 - 1), "needed"),
    (lambda r: _lr_bwd(r, ddown=None), "ddown"),
    (lambda r: _lr_bwd(r, lddy=72 + 4), "row stride"),
    (lambda r: _lr_bwd(r, size=64), "needed"),
    (lambda r: _loss(r, dtype=F32), "must be fp16 or bf16"),
    (lambda r: _loss(r, v=0), "V=0"),
    (lambda r: _loss(r, ldw=63), "row stride"),
    (lambda r: _loss(r, x=24), "aligned"),
    (lambda r: _loss(r, target=None), "null"),
    (lambda r: _loss(r, loss=None), "loss"),
    (lambda r: _loss(r, size=16), "needed"),
    (lambda r: _loss(r, m=1 << 25, ldx=64), "x below 4 GiB"),
    (lambda r: _loss_bwd(r, dw=None), "dw"),
    (lambda r: _loss_bwd(r, dloss=None), "dloss"),
    (lambda r: _loss_bwd(r, lddx=60), "row stride"),
    (lambda r: _loss_bwd(r, size=16), "needed"),
])
def test_refused_on_host(lib, call, msg):
    raw = lib.load()
    assert call(raw) == 1  # SSG_EINVAL
    assert msg in raw.ssg_last_error().decode(), raw.ssg_last_error().decode()


def test_no_rows_is_ok_without_touching_the_device(lib):
    raw = lib.load()
    assert _norm(raw, m=0, x=None, y=None) == 0
    assert _norm_bwd(raw, m=0, dw=None, db=None, ws=None, size=0) == 0
    assert _add(raw, m=0, lr=_lr(down=None, up=None, index=None), x=None, out=None, ws=None, size=0) == 0
    assert _w24(raw, m=0, meta=None, ws=None, size=0) == 0
    assert _loss(raw, m=0, x=None, target=None, loss=None, size=0) == 0


def test_workspace_sizes(lib):
    raw = lib.load()
    # layer norm: one slice of two fp32 rows a persistent workgroup, at most one a CU
    assert raw.layer_norm_workspace_bytes(F16, 1, 768) == 2 * 768 * 4
    assert 0 < raw.layer_norm_workspace_bytes(F16, 12608, 768) <= 256 * 2 * 768 * 4
    assert raw.layer_norm_workspace_bytes(F16, 0, 768) == 0
    # adapters: two planes of 16-bit values in blocks of 32 tokens x 16 slots; none for few tokens
    assert raw.low_rank_workspace_bytes(129, 8) == 160 * 16 * 4
    assert raw.low_rank_workspace_bytes(16, 8) == 0
    # few tokens beside a 2:4 product: its fp32 sums
    assert raw.w24_low_rank_workspace_bytes(16, 1024, 1024, 8) == 16 * 1024 * 4
    assert raw.w24_low_rank_workspace_bytes(4096, 1024, 1024, 64) == 4096 * 64 * 4
    # the gradients' slices stay within 256 MiB beside the values themselves, for large pools too
    for a, r in ((1, 8), (64, 64), (1000, 128)):
        w = raw.low_rank_backward_workspace_bytes(a, r, 8192, 4096, 1024)
        assert 0 < w <= (256 << 20) + 4 * 8192 * 128 * 4 + 64 * a * 4 + 4096, (a, r, w)
    # cross entropy: nothing near the logits' size (forward), one piece of 256 MiB (backward)
    assert raw.linear_cross_entropy_workspace_bytes(F16, 8192, 128000, 1024, 1024, 1024, 0) < 8192 * 128000 * 2 // 50
    assert raw.linear_cross_entropy_workspace_bytes(F16, 8192, 128000, 1024, 1024, 1024, 1) <= (300 << 20)
    # a very tall batch keeps a piece's G inside the products' 4 GiB
    assert raw.linear_cross_entropy_workspace_bytes(F16, 4_000_000, 5000, 64, 64, 64, 1) < \
        (4 << 30) + 4_000_000 * 64 * 4 + 4096
    for m in (0, 1, 63, 64, 1000, 1 << 20):
        for v in (1, 7, 255, 50257):
            for d in (1, 100, 2048):
                for back in (0, 1):
                    assert raw.linear_cross_entropy_workspace_bytes(BF16, m, v, d, d, d, back) >= 0


def _kernels(asm):
    out = {}
    for m in re.finditer(r"^\s*\.amdhsa_kernel (\S+)\n(.*?)\.end_amdhsa_kernel", asm, re.M | re.S):
        val = lambda k: int(re.search(r"\.amdhsa_" + k + r"\s+(\d+)", m.group(2)).group(1))
        out[m.group(1)] = dict(lds=val("group_segment_fixed_size"), vgpr=val("next_free_vgpr"),
                               scratch=val("private_segment_fixed_size"))
    return out


@pytest.mark.parametrize("source,least", [("layer_norm.hip", 60), ("low_rank.hip", 20), ("low_rank_gemm.hip", 5),
                                          ("loss.hip", 25)])
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
