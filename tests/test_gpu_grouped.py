"""Products grouped by expert and their gradients against 64-bit sums.

Bound of an error: products of 16-bit values are exact in fp32 (bf16; fp16's too, 22
bits), n additions in any order are off by at most n 2^-24 sum|a||b| to first order
(twice that is allowed), the output's rounding by half a step."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def _dt(name):
    import torch
    return {"f16": torch.float16, "bf16": torch.bfloat16}[name]


def _close(got, a, b, dt):
    """got = a . b of float64 CPU matrices."""
    import torch
    want, size = a @ b, a.abs() @ b.abs()
    half, eps = torch.finfo(_dt(dt)).eps / 2, torch.finfo(_dt(dt)).eps
    bound = half * want.abs() + (1 + half) * 2 * max(a.shape[1], 1) * 2.0 ** -24 * size
    bound = bound + torch.finfo(_dt(dt)).smallest_normal * eps
    miss = (got.double().cpu() - want).abs()
    assert bool((miss <= bound).all()), float((miss - bound).max())


def _offsets(lengths, first=0):
    import torch
    return torch.tensor([first] + (first + np.cumsum(lengths)).tolist(), dtype=torch.int32)


# lengths of the experts' rows, rows before the first and behind the last, N, K
CASES = [
    ([1], 0, 0, 8, 8), ([3, 0, 1], 0, 0, 64, 64), ([0, 0], 0, 3, 16, 24), ([5, 0, 0, 27], 2, 3, 136, 72),
    ([33, 31, 1, 64, 65], 0, 0, 128, 128), ([64, 2, 200], 1, 9, 200, 264), ([127, 128, 129, 0], 0, 5, 256, 192),
    ([300, 3, 257], 0, 0, 264, 520), ([1000, 700], 4, 4, 520, 136), ([2] * 70 + [0] * 5 + [3] * 60, 0, 1, 72, 200),
    ([513, 900, 1100], 0, 0, 1032, 776), ([0, 4097], 0, 0, 256, 256),
]


def _case(lengths, before, behind, n, k, dt, seed=0):
    import torch
    g = torch.Generator().manual_seed(seed + n + k)
    m, e = before + sum(lengths) + behind, len(lengths)
    x = torch.randn(m, k, generator=g).to(_dt(dt))
    dy = torch.randn(m, n, generator=g).to(_dt(dt))
    w = (torch.randn(e, n, k, generator=g) / k ** 0.5).to(_dt(dt))
    return x, dy, w, _offsets(lengths, before)


@pytest.mark.parametrize("lengths,before,behind,n,k", CASES)
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_forward(lib, gpu, lengths, before, behind, n, k, dt):
    import torch
    x, _, w, offsets = _case(lengths, before, behind, n, k, dt)
    out = torch.full((x.shape[0], n), 7.0, dtype=_dt(dt), device="cuda")
    got = lib.grouped_gemm(x.cuda(), w.cuda(), offsets.cuda(), out=out)
    o = offsets.tolist()
    for e in range(len(lengths)):
        if lengths[e]:
            _close(got[o[e]:o[e + 1]], x[o[e]:o[e + 1]].double(), w[e].double().t(), dt)
    assert bool((got[:before] == 7).all()) and bool((got[o[-1]:] == 7).all())
    if before == behind == 0:
        assert torch.equal(lib.grouped_gemm(x.cuda(), w.cuda(), offsets.cuda()), got)


@pytest.mark.parametrize("lengths,before,behind,n,k", CASES)
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_backward(lib, gpu, lengths, before, behind, n, k, dt):
    import torch
    x, dy, w, offsets = _case(lengths, before, behind, n, k, dt, 1)
    # what lies in rows of no expert must reach nothing
    for t in (x, dy):
        t[:before] = float("nan")
        t[t.shape[0] - behind:] = float("inf") if behind else 0
    out = torch.full((x.shape[0], k), 7.0, dtype=_dt(dt), device="cuda")
    dx, dw = lib.grouped_gemm_backward(dy.cuda(), x.cuda(), w.cuda(), offsets.cuda(), out=out)
    o = offsets.tolist()
    for e in range(len(lengths)):
        rows = slice(o[e], o[e + 1])
        if lengths[e]:
            _close(dx[rows], dy[rows].double(), w[e].double(), dt)
            _close(dw[e], dy[rows].double().t(), x[rows].double(), dt)
        else:
            assert not bool(dw[e].any())
    assert bool((dx[:before] == 7).all()) and bool((dx[o[-1]:] == 7).all())
    a, b = lib.grouped_gemm_backward(dy.cuda(), x.cuda(), w.cuda(), offsets.cuda(), out=out, w_grad=False)
    assert b is None and torch.equal(a, dx)
    a, b = lib.grouped_gemm_backward(dy.cuda(), x.cuda(), w.cuda(), offsets.cuda(), x_grad=False)
    assert a is None and torch.equal(b, dw)


def test_gradients_against_differences(lib, gpu):
    """<grad, direction> against (f(+h) - f(-h)) / 2h of f = <dy, forward>, linear in either argument, so
    exact up to roundings: the forward's (half a step of every output, and the sums') and the gradients'."""
    import torch
    x, dy, w, offsets = _case([40, 0, 75, 9], 0, 0, 96, 160, "f16", 2)
    dx, dw = lib.grouped_gemm_backward(dy.cuda(), x.cuda(), w.cuda(), offsets.cuda())
    g = torch.Generator().manual_seed(5)
    f = lambda x, w: (dy.double() * lib.grouped_gemm(x.cuda(), w.cuda(), offsets.cuda()).double().cpu()).sum()
    for grad, at in ((dx, "x"), (dw, "w")):
        base = x if at == "x" else w
        # steps that 16 bits hold: both points are rounded first, their true distance is used
        d = torch.randn(base.shape, generator=g) * base.float().abs().mean()
        up, down = (base.float() + d).half(), (base.float() - d).half()
        diff = f(up, w) - f(down, w) if at == "x" else f(x, up) - f(x, down)
        step = up.double() - down.double()
        want = (grad.double().cpu() * step).sum()
        size = (grad.double().cpu().abs() * step.abs()).sum()
        outs = sum(lib.grouped_gemm(*((p.cuda(), w.cuda()) if at == "x" else (x.cuda(), p.cuda())),
                                    offsets.cuda()).double().cpu().abs() for p in (up, down))
        bound = 2.0 ** -11 * (size + (dy.double().abs() * outs).sum()) * 1.01
        assert abs(diff - want) <= bound, (at, float(diff - want), float(bound))


def test_strided_rows(lib, gpu):
    import torch
    x, dy, w, offsets = _case([40, 100, 0, 7], 0, 2, 96, 72, "bf16", 3)
    m = x.shape[0]
    wx, wy = torch.randn(m, 120).bfloat16().cuda(), torch.randn(m, 200).bfloat16().cuda()
    wx[:, 16:88], wy[:, 24:120] = x.cuda(), dy.cuda()
    sx, sy = wx[:, 16:88], wy[:, 24:120]
    w, offsets = w.cuda(), offsets.cuda()
    out = torch.full((m, 136), 4.0, dtype=torch.bfloat16, device="cuda")
    lib.grouped_gemm(sx, w, offsets, out=out[:, 8:104])
    live = slice(0, m - 2)
    assert torch.equal(out[live, 8:104], lib.grouped_gemm(x.cuda(), w, offsets)[live])
    assert bool((out[:, :8] == 4).all()) and bool((out[:, 104:] == 4).all()) and bool((out[m - 2:] == 4).all())
    a, b = lib.grouped_gemm_backward(sy, sx, w, offsets), lib.grouped_gemm_backward(dy.cuda(), x.cuda(), w, offsets)
    assert torch.equal(a[0][live], b[0][live]) and torch.equal(a[1], b[1])


def test_what_is_not_finite_stays_with_its_row_or_expert(lib, gpu):
    import torch
    for k in (64, 72):  # (72: K ends inside a stage)
        x, dy, w, offsets = _case([30, 50, 20], 0, 0, 88, k, "f16", 4)
        clean = lib.grouped_gemm(x.cuda(), w.cuda(), offsets.cuda())
        dclean = lib.grouped_gemm_backward(dy.cuda(), x.cuda(), w.cuda(), offsets.cuda())
        x[35, 3], w[2, 5, 1], dy[36, 0] = float("nan"), float("inf"), float("inf")
        got = lib.grouped_gemm(x.cuda(), w.cuda(), offsets.cuda())
        keep = torch.ones(100, 88, dtype=torch.bool)
        keep[35], keep[80:, 5] = False, False
        assert torch.equal(got.cpu()[keep], clean.cpu()[keep]) and not bool(torch.isfinite(got.cpu()[~keep]).any())
        dx, dw = lib.grouped_gemm_backward(dy.cuda(), x.cuda(), w.cuda(), offsets.cuda())
        rows = torch.ones(100, k, dtype=torch.bool)
        rows[36], rows[80:, 1] = False, False
        assert torch.equal(dx.cpu()[rows], dclean[0].cpu()[rows])
        assert torch.equal(dw[[0, 2]], dclean[1][[0, 2]])
        keep = torch.ones(88, k, dtype=torch.bool)
        keep[0], keep[:, 3] = False, False
        assert torch.equal(dw[1].cpu()[keep], dclean[1][1].cpu()[keep])


@pytest.mark.parametrize("bad,same", [([0, 50, 20, 90], [0, 50, 50, 90]), ([-5, 10, 300, 200], [0, 10, 100, 100]),
                                      ([70, 30, 100, 100], [70, 70, 100, 100]), ([0, 0, 0, 2 ** 31 - 1], [0, 0, 0, 100])])
def test_offsets_that_are_not_in_order(lib, gpu, bad, same):
    import torch
    x, dy, w, _ = _case([100, 0, 0], 0, 0, 64, 64, "f16", 5)
    run = lambda o: (lib.grouped_gemm(x.cuda(), w.cuda(), torch.tensor(o, dtype=torch.int32).cuda(),
                                      out=torch.zeros(100, 64, dtype=torch.float16, device="cuda")),
                     *lib.grouped_gemm_backward(dy.cuda(), x.cuda(), w.cuda(), torch.tensor(o, dtype=torch.int32).cuda(),
                                                out=torch.zeros(100, 64, dtype=torch.float16, device="cuda")))
    for a, b in zip(run(bad), run(same)):
        assert torch.equal(a, b)


def test_no_rows(lib, gpu):
    import torch
    x, dy, w, _ = _case([1, 0], 0, 0, 64, 72, "f16")
    offsets = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert lib.grouped_gemm(x[:0].cuda(), w.cuda(), offsets).shape == (0, 64)
    dx, dw = lib.grouped_gemm_backward(dy[:0].cuda(), x[:0].cuda(), w.cuda(), offsets,
                                       dw_out=torch.ones(2, 64, 72, dtype=torch.float16, device="cuda"))
    assert dx.shape == (0, 72) and not bool(dw.any())


@pytest.mark.parametrize("lengths,n,k", [([9000], 64, 136), ([0, 3000, 1, 5000], 72, 80), ([20000, 300], 128, 256)])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_weight_gradient_of_many_rows(lib, gpu, lengths, n, k, dt):
    """Few tiles, long sums: the rows are split and the slices added."""
    import torch
    m, e = sum(lengths), len(lengths)
    need = lib.load().grouped_gemm_backward_workspace_bytes(e, m, n, k)
    assert need > 0 and need % (e * n * k * 4) == 0
    x, dy, w, offsets = _case(lengths, 0, 0, n, k, dt, 7)
    args = [t.cuda() for t in (dy, x, w, offsets)]
    _, dw = lib.grouped_gemm_backward(*args, x_grad=False)
    o = offsets.tolist()
    for i in range(e):
        _close(dw[i], dy[o[i]:o[i + 1]].double().t(), x[o[i]:o[i + 1]].double(), dt)
    again = lib.grouped_gemm_backward(*args, x_grad=False, workspace=torch.full((need,), 255, dtype=torch.uint8,
                                                                               device="cuda"))[1]
    assert torch.equal(dw, again)
    with pytest.raises(lib.SsgError, match="needed"):
        lib.grouped_gemm_backward(*args, workspace=torch.empty(need - 16, dtype=torch.uint8, device="cuda"))
