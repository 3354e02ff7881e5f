"""Every tile that the experts' products may run on: ragged groups (an empty one, one of a single row) with rows
of no expert before and behind them, widths that end inside a tile, sums that end inside a stage of 64 values
(4 bits: of 256, and inside a block of scales).

16-bit values are -1, 0 and 1, 4-bit ones have scales of 1/2 to 2: every sum is a whole number (4 bits: of
1/16) below 2^24 and exact in fp32 in any order, so results equal the 64-bit ones but for the output's one rounding."""

import random

import numpy as np
import pytest

FORWARD, DX, DW, JOINT, MX = range(5)  # the products of expert_tile
# (tile, experts, M, N, K)
FORWARDS = [(0, 3, 42, 72, 424), (1, 22, 6214, 72, 400), (2, 36, 137, 1360, 400), (3, 39, 10040, 136, 400),
            (4, 17, 18775, 136, 400), (5, 36, 2741, 1592, 408), (6, 33, 21420, 272, 408)]
# N ends inside a stage, then with one (and K inside a tile, so that loads reach past a weight's last row)
DXS = [(0, 4, 45, 408, 72), (1, 13, 6694, 592, 72), (2, 30, 94, 400, 848), (3, 34, 7862, 400, 136),
       (4, 20, 636, 432, 1616), (5, 40, 14388, 400, 136), (6, 33, 19780, 400, 264),
       (0, 3, 41, 384, 80), (1, 33, 6435, 640, 72), (2, 37, 148, 384, 592), (3, 38, 7269, 384, 136),
       (4, 29, 941, 448, 1136), (5, 39, 14975, 384, 136), (6, 19, 1668, 384, 3080)]
# (tile, whether the rows are split, ...)
DWS = [(0, False, 3, 941, 72, 80), (0, True, 3, 5127, 72, 80), (1, False, 39, 11828, 272, 72),
       (1, True, 10, 28233, 136, 72), (2, False, 35, 11139, 136, 392), (2, True, 3, 18122, 712, 72),
       (3, False, 39, 12013, 200, 136), (3, True, 3, 12037, 776, 72), (4, False, 36, 10925, 656, 136),
       (4, True, 3, 28953, 824, 136), (5, False, 15, 4561, 2256, 136)]
JOINTS = [(-1, 40, 125, 592, 424), (0, 4, 45, 408, 72), (1, 36, 130, 432, 136), (2, 33, 6156, 456, 144)]
# 16 and up: the kernels of few rows; experts 0: one weight
MXS = [(0, 0, 531, 101, 1583), (0, 24, 208, 101, 2122), (1, 0, 527, 101, 1041), (1, 6, 541, 101, 1079),
       (2, 0, 6670, 202, 1045), (2, 31, 99, 969, 1030), (3, 0, 10120, 269, 1061), (3, 12, 10006, 274, 1050),
       (4, 0, 13729, 522, 1033), (4, 38, 3108, 1439, 1036), (5, 0, 12302, 780, 1082), (5, 34, 3994, 1667, 1034),
       (16, 0, 9, 102, 261), (16, 3, 25, 118, 267), (17, 0, 3, 101, 1037), (17, 3, 4, 107, 1036),
       (18, 0, 97, 2224, 264), (18, 30, 242, 303, 262)]


def test_shapes_run_on_their_tiles_and_reach_all(lib):
    for product, shapes in ((FORWARD, FORWARDS), (DX, DXS), (JOINT, JOINTS), (MX, MXS)):
        for tile, *shape in shapes:
            assert lib.expert_tile(product, *shape) == tile, (product, tile, shape)
    for tile, split, *shape in DWS:
        got = lib.expert_tile(DW, *shape)
        assert (got % 256, got // 256 > 1) == (tile, split), (tile, split, shape)
    have = {FORWARD: {s[0] for s in FORWARDS}, DX: {s[0] for s in DXS}, JOINT: {s[0] for s in JOINTS},
            MX: {(s[0], s[1] > 0) for s in MXS}, DW: {s[:2] for s in DWS}}
    rng = random.Random(0)
    size = lambda lo, hi: int(round(lo * (hi / lo) ** rng.random()))
    for _ in range(60000):
        e, m, n, k = size(1, 200), size(1, 40000), 8 * size(1, 1000), 8 * size(1, 1000)
        for product in (FORWARD, DX, JOINT):
            assert lib.expert_tile(product, e, m, n, k) in have[product], (product, e, m, n, k)
        dw = lib.expert_tile(DW, e, m, n, k)
        assert (dw % 256, dw // 256 > 1) in have[DW], (e, m, n, k)
        n, k = size(1, 8000), size(1, 8000)
        for experts in (0, e):
            assert (lib.expert_tile(MX, experts, m, n, k), experts > 0) in have[MX], (experts, m, n, k)
    for bad in ((-1, 1, 1, 8, 8), (5, 1, 1, 8, 8), (0, 0, 1, 8, 8), (0, 1, 0, 8, 8), (2, 1, 1, 12, 8), (4, 0, 1, 0, 8)):
        assert lib.expert_tile(*bad) == -2


@pytest.mark.parametrize("m,n,k", [(157, 288, 6100), (193, 120, 5304), (12, 352, 7724)])
def test_long_sums_are_not_taken_by_the_few_rows_kernels_for_the_host_s_sake(lib, m, n, k):
    """One launch takes up to twice the time of two on the device there (27.3 us and 13.3 for the first)."""
    assert 0 <= lib.expert_tile(MX, 0, m, n, k) < 16


def _dt(name):
    import torch
    return {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}[name]


def _cuts(m, e, seed):
    """Offsets of ragged groups in m rows: 2 before, 3 behind (few rows: fewer), the second empty, the third of one row."""
    rng = np.random.default_rng(seed)
    before, behind = (2, 3) if m >= 12 else (0, 1)
    share = np.exp(rng.normal(size=e))
    share[1] = share[2] = 0
    counts = rng.multinomial(m - before - behind - 1, share / share.sum())
    counts[2] = 1
    return (before + np.concatenate([[0], np.cumsum(counts)])).tolist()


def _trits(g, *shape, dt):
    import torch
    return torch.randint(-1, 2, shape, generator=g, device="cuda", dtype=torch.int8).to(dt)


def _operands(m, n, k, e, dt):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(m + n + k)
    o = _cuts(m, e, m + n + k)
    x, dy, w = _trits(g, m, k, dt=_dt(dt)), _trits(g, m, n, dt=_dt(dt)), _trits(g, e, n, k, dt=_dt(dt))
    for t in (x, dy):  # what lies in rows of no expert must reach nothing
        t[:o[0]], t[o[-1]:] = float("nan"), float("inf")
    return x, dy, w, o, torch.tensor(o, dtype=torch.int32, device="cuda")


def _same(got, want, dt):
    import torch
    want = want.to(_dt(dt))
    assert torch.equal(got, want), (got != want).nonzero()[:4].tolist()


def _groups(got, o, product, dt):
    """got: rows filled with 7 before the call; product(e, rows): the 64-bit result of an expert's rows."""
    for e, (a, b) in enumerate(zip(o, o[1:])):
        if b > a:
            _same(got[a:b], product(e, slice(a, b)), dt)
    assert bool((got[:o[0]] == 7).all()) and bool((got[o[-1]:] == 7).all())


def _sevens(m, n, dt):
    import torch
    return torch.full((m, n), 7.0, dtype=_dt(dt), device="cuda")


def _check_dw(dw, x, dy, o, dt):
    for e, (a, b) in enumerate(zip(o, o[1:])):
        _same(dw[e], dy[a:b].double().t().contiguous() @ x[a:b].double(), dt)


def _check_dx(dx, dy, w, o, dt):
    _groups(dx, o, lambda e, rows: dy[rows].double() @ w[e].double(), dt)


HALF = pytest.mark.parametrize("dt", ["f16", "bf16"])


@pytest.mark.gpu
@pytest.mark.parametrize("tile,e,m,n,k", FORWARDS)
@HALF
def test_forward(lib, gpu, tile, e, m, n, k, dt):
    x, _, w, o, offsets = _operands(m, n, k, e, dt)
    got = lib.grouped_gemm(x, w, offsets, out=_sevens(m, n, dt))
    _groups(got, o, lambda i, rows: x[rows].double() @ w[i].double().t().contiguous(), dt)


@pytest.mark.gpu
@pytest.mark.parametrize("tile,e,m,n,k", DXS)
@HALF
def test_dx(lib, gpu, tile, e, m, n, k, dt):
    x, dy, w, o, offsets = _operands(m, n, k, e, dt)
    dx, _ = lib.grouped_gemm_backward(dy, x, w, offsets, out=_sevens(m, k, dt), w_grad=False)
    _check_dx(dx, dy, w, o, dt)


@pytest.mark.gpu
@pytest.mark.parametrize("tile,split,e,m,n,k", DWS)
@HALF
def test_dw(lib, gpu, tile, split, e, m, n, k, dt):
    x, dy, w, o, offsets = _operands(m, n, k, e, dt)
    _, dw = lib.grouped_gemm_backward(dy, x, w, offsets, x_grad=False)
    _check_dw(dw, x, dy, o, dt)


@pytest.mark.gpu
@pytest.mark.parametrize("tile,e,m,n,k", JOINTS)
@HALF
def test_dx_and_dw(lib, gpu, tile, e, m, n, k, dt):
    x, dy, w, o, offsets = _operands(m, n, k, e, dt)
    dx, dw = lib.grouped_gemm_backward(dy, x, w, offsets, out=_sevens(m, k, dt))
    _check_dx(dx, dy, w, o, dt)
    _check_dw(dw, x, dy, o, dt)


def _values(codes, scales, k):
    """float64 values of packed rows."""
    import torch
    c = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=codes.device)
    v = torch.where(c >= 8, -1.0, 1.0) * table[c & 7]
    return (v * torch.exp2(scales.double() - 127).repeat_interleave(32, -1))[..., :k].contiguous()


def _packed(g, rows, k):
    import torch
    kp = -(-k // 128) * 128
    codes = torch.randint(0, 256, (rows, kp // 2), generator=g, device="cuda", dtype=torch.uint8)
    codes[:, (k + 1) // 2:] = 0
    if k % 2:
        codes[:, k // 2] &= 15
    return codes, torch.randint(126, 129, (rows, kp // 32), generator=g, device="cuda", dtype=torch.uint8)


@pytest.mark.gpu
@pytest.mark.parametrize("tile,e,m,n,k", MXS)
@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
def test_4_bits(lib, gpu, tile, e, m, n, k, dt):
    import torch
    g = torch.Generator(device="cuda")
    g.manual_seed(m + n + k)
    a, sa = _packed(g, m, k)
    w, sw = _packed(g, max(e, 1) * n, k)
    va, vw = _values(a, sa, k), _values(w, sw, k)
    out = torch.full((m, n + 3), 7.0, dtype=_dt(dt), device="cuda")  # (rows at odd strides)
    if not e:
        lib.mxfp4_gemm(a, sa, w, sw, k, out=out[:, 1:n + 1])
        _same(out[:, 1:n + 1], va @ vw.t().contiguous(), dt)
    else:
        o = _cuts(m, e, m)
        offsets = torch.tensor(o, dtype=torch.int32, device="cuda")
        sa[:o[0]], sa[o[-1]:] = 255, 255  # (NaN in rows of no expert)
        lib.mxfp4_gemm(a, sa, w.view(e, n, -1), sw.view(e, n, -1), k, offsets=offsets, out=out[:, 1:n + 1])
        _groups(out[:, 1:n + 1], o, lambda i, rows: va[rows] @ vw[i * n:(i + 1) * n].t().contiguous(), dt)
    assert bool((out[:, 0] == 7).all()) and bool((out[:, n + 1:] == 7).all())
    if dt == "f32":
        return
    # the same from 16-bit rows, quantised in the call
    x = torch.randn(m, k, generator=g, device="cuda").to(_dt(dt))
    if not e:
        got, want = lib.mxfp4_linear(x, w, sw), lib.mxfp4_gemm(*lib.mxfp4_quantize(x), w, sw, k, _dt(dt))
    else:
        x[:o[0]], x[o[-1]:] = float("nan"), float("inf")
        w, sw = w.view(e, n, -1), sw.view(e, n, -1)
        got = lib.mxfp4_grouped_linear(x, w, sw, offsets, out=_sevens(m, n, dt))
        want = lib.mxfp4_gemm(*lib.mxfp4_quantize(x), w, sw, k, offsets=offsets, out=_sevens(m, n, dt))
    assert torch.equal(got, want)
