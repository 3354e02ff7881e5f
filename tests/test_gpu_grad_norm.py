"""The gradient norm and clipping against 64-bit sums.

The norm's square is summed in fp64 from exact squares: after the square root and the
rounding to fp32 it is within 2^-24 (half a step) and 1e-12 of the norm.  The factor is rounded to
fp32 once more (2^-24), then the product to the tensor's type (half a step)."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu


def _dt(name):
    import torch
    return {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}[name]


def _tensors(sizes, kinds, seed=0, std=1.0):
    import torch
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * std).to(_dt(kinds[i % len(kinds)])) for i, n in enumerate(sizes)]


def _norm(ts):
    return float(np.sqrt(sum(float((t.double() ** 2).sum()) for t in ts)))


def _check(ts, norm, outs, max_norm):
    import torch
    want = _norm(ts)
    assert abs(float(norm) - want) <= 2.0 ** -24 * want + 1e-12 * want
    by = min(1.0, max_norm / (want + 1e-6))
    for t, o in zip(ts, outs):
        assert o.dtype == t.dtype and o.shape == t.shape
        exact = t.double() * by
        half, tiny = torch.finfo(t.dtype).eps / 2, torch.finfo(t.dtype).smallest_normal * torch.finfo(t.dtype).eps
        bound = exact.abs() * (half + 2.0 ** -24 * (1 + half) + 1e-11) + tiny
        assert bool(((o.double().cpu() - exact).abs() <= bound).all())


SIZES = [[1], [0, 5, 0], [7, 8192, 8193, 1, 16385, 100000], [3] * 500, [4096, 0, 4097, 12288, 12289],
         [1000003], [50000] * 137 + [11]]


@pytest.mark.parametrize("sizes", SIZES)
@pytest.mark.parametrize("kinds", [["f16"], ["bf16"], ["f32"], ["f16", "f32", "bf16"]])
def test_norm_and_clip(lib, gpu, sizes, kinds):
    import torch
    ts = _tensors(sizes, kinds, len(sizes))
    dev = [t.cuda() for t in ts]
    norm = lib.grad_norm(dev)
    assert norm.shape == () and norm.dtype == torch.float32
    for most in (0.5, 1e9):
        got, outs = lib.clip_grad_norm(dev, most)
        assert torch.equal(got, norm) and all(torch.equal(a.cpu(), b) for a, b in zip(dev, ts))
        _check(ts, got, outs, most)
        again = [t.clone() for t in dev]
        got, same = lib.clip_grad_norm(again, most, out=again)
        assert torch.equal(got, norm) and all(a is b for a, b in zip(same, again))
        assert all(torch.equal(a, b) for a, b in zip(same, outs))
        got, by_norm = lib.clip_grad_norm(dev, most, norm=norm)
        _check(ts, got, by_norm, most)


def test_views_at_any_element(lib, gpu):
    import torch
    flat = torch.randn(100000, generator=torch.Generator().manual_seed(1)).half()
    cuts = [1, 2, 5, 4000, 4001, 30003, 99999]
    views = lambda f: [f[a:b] for a, b in zip(cuts, cuts[1:])]
    dev, out = flat.cuda(), torch.full((100000,), 3.0, dtype=torch.float16, device="cuda")
    norm, outs = lib.clip_grad_norm(views(dev), 1.0, out=views(out))
    _check(views(flat), norm, [o.cpu() for o in outs], 1.0)
    assert float(out[0]) == 3.0 and float(out[-1]) == 3.0
    norm2, _ = lib.clip_grad_norm(views(dev), 1.0, out=views(dev))
    assert torch.equal(dev[1:99999], out[1:99999]) and torch.equal(norm, norm2)


def test_shapes_and_axis_orders(lib, gpu):
    import torch
    a = torch.randn(30, 40).cuda().t()
    b = torch.randn(4, 5, 6).cuda().permute(2, 0, 1).bfloat16()
    assert not a.is_contiguous()
    norm, (ca, cb) = lib.clip_grad_norm([a, b], 0.1)
    _check([a.cpu(), b.cpu()], norm, [ca, cb], 0.1)
    with pytest.raises(ValueError, match="run of memory"):
        lib.grad_norm([torch.randn(8, 8, device="cuda")[:, :3]])
    with pytest.raises(ValueError, match="strides"):
        lib.clip_grad_norm([a], 1.0, out=[torch.empty(40, 30, device="cuda")])


def test_large_and_small_values(lib, gpu):
    import torch
    for value, dt in ((3e38, torch.float32), (1e-40, torch.float32), (6e4, torch.float16), (6e-8, torch.float16),
                      (3e38, torch.bfloat16)):
        t = torch.full((5000,), value).to(dt)
        norm, out = lib.clip_grad_norm([t.cuda()], 1.0)
        want = float(t[0].double()) * 5000 ** 0.5
        if want < 3.4e38:
            # (a subnormal norm has steps of 2^-149)
            assert abs(float(norm) - want) <= 2.0 ** -24 * want + 2.0 ** -150
        else:
            assert float(norm) == float("inf")
        by = min(1.0, 1.0 / (want + 1e-6))  # (from the 64-bit norm, also where fp32 has none)
        exact = t.double() * by
        fi = torch.finfo(dt)
        assert bool(((out[0].double().cpu() - exact).abs() <=
                     exact.abs() * (fi.eps + 2.0 ** -22) + fi.smallest_normal * fi.eps + by * 0).all()) or by < 1e-37


def test_not_finite(lib, gpu):
    import torch
    nan, inf = float("nan"), float("inf")
    t = torch.ones(100)
    t[3] = inf
    norm, (o, p) = lib.clip_grad_norm([t.cuda(), torch.ones(5).cuda()], 1.0)
    assert float(norm) == inf and bool(torch.isnan(o[3])) and float(o[4]) == 0 and not bool(p.any())
    t[3] = nan
    norm, (o,) = lib.clip_grad_norm([t.cuda()], 1.0)
    assert bool(torch.isnan(norm)) and bool(torch.isnan(o).all())
    norm, (o,) = lib.clip_grad_norm([torch.ones(7).cuda()], 1.0, norm=torch.tensor(nan).cuda())
    assert bool(torch.isnan(o).all())


def test_repeats_bit_for_bit(lib, gpu):
    import torch
    dev = [t.cuda() for t in _tensors([300000, 17, 5000, 70001], ["bf16", "f32"], 3)]
    first = lib.grad_norm(dev)
    for _ in range(5):
        assert torch.equal(lib.grad_norm(dev), first)


def test_refusals(lib, gpu):
    import torch
    t = torch.randn(64).cuda()
    for bad, why in (([t, t], "overlaps"), ([t[:40], t[30:]], "overlaps")):
        with pytest.raises(lib.SsgError, match=why):
            lib.clip_grad_norm(bad, 1.0, out=bad)
        assert float(lib.grad_norm(bad)) > 0  # (the norm alone writes nothing)
    with pytest.raises(lib.SsgError, match="overlaps"):
        lib.clip_grad_norm([t[:32]], 1.0, out=[t[16:48]])
    with pytest.raises(lib.SsgError, match="max_norm"):
        lib.clip_grad_norm([t], -1.0)
    with pytest.raises(lib.SsgError, match="max_norm"):
        lib.clip_grad_norm([t], float("nan"))
    with pytest.raises(ValueError, match="outputs for"):
        lib.clip_grad_norm([t], 1.0, out=[])
    with pytest.raises(ValueError, match="empty"):
        lib.grad_norm([])
    with pytest.raises(TypeError, match="torch tensors"):
        lib.grad_norm([torch.ones(3)])
    with pytest.raises(TypeError, match="does not take"):
        lib.grad_norm([torch.ones(3, device="cuda", dtype=torch.float64)])
    with pytest.raises(ValueError, match="one element"):
        lib.clip_grad_norm([t], 1.0, norm=torch.ones(2).cuda())
    with pytest.raises(lib.SsgError, match="workspace"):
        lib.grad_norm([t], workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
