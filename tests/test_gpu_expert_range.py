"""The experts' calls at the ends of their ranges: operands past 4 GiB, thousands of experts, no rows.

Values are -1, 0 and 1, so every sum below 2^24 is exact in fp32 whatever its order, the 4-bit form
holds each value exactly (a block's scale is 1/4 or, of zeros alone, the smallest), and what is left is
the output's one rounding: results are compared for equality."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

ROWS, WIDE = 2_200_003, 1024  # 16-bit rows of 4.2 GiB


def _trits(shape, dt):
    import torch
    return torch.randint(-1, 2, shape, device="cuda", dtype=torch.int8).to(dt)


@pytest.fixture(scope="module")
def large(lib, gpu):
    import torch
    torch.manual_seed(5)
    x = _trits((ROWS, WIDE), torch.bfloat16)
    offsets = [1, 700_001, 700_001, ROWS - 2]
    yield x, offsets, torch.tensor(offsets, dtype=torch.int32, device="cuda")
    del x
    torch.cuda.empty_cache()


def _around(offsets):
    """Rows at both ends, at the experts' ends and on both sides of 2 and 4 GiB."""
    at = [0, ROWS - 1, (1 << 30) // WIDE, (1 << 31) // WIDE] + offsets
    return sorted({r for a in at for r in range(a - 2, a + 3) if 0 <= r < ROWS})


def _expert_of(row, offsets):
    return next((e for e in range(len(offsets) - 1) if offsets[e] <= row < offsets[e + 1]), None)


def test_forward_past_4_gib(lib, large):
    import torch
    x, offsets, dev = large
    w = _trits((3, 64, WIDE), torch.bfloat16)
    out = torch.full((ROWS, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    lib.grouped_gemm(x, w, dev, out=out)
    for r in _around(offsets):
        e = _expert_of(r, offsets)
        want = torch.full((64,), 7.0) if e is None else (w[e].double().cpu() @ x[r].double().cpu())
        assert torch.equal(out[r].cpu(), want.to(torch.bfloat16)), r


def test_backward_past_4_gib(lib, large):
    import torch
    x, offsets, dev = large
    w, dy = _trits((3, 64, WIDE), torch.bfloat16), _trits((ROWS, 64), torch.bfloat16)
    out = torch.full_like(x, 7.0)
    _, dw = lib.grouped_gemm_backward(dy, x, w, dev, out=out)
    for r in _around(offsets):
        e = _expert_of(r, offsets)
        want = torch.full((WIDE,), 7.0) if e is None else (w[e].double().cpu().t() @ dy[r].double().cpu())
        assert torch.equal(out[r].cpu(), want.to(torch.bfloat16)), r
    for e in range(3):
        want = torch.zeros(64, WIDE, dtype=torch.float64, device="cuda")
        for at in range(offsets[e], offsets[e + 1], 100_000):
            to = min(at + 100_000, offsets[e + 1])
            want += dy[at:to].double().t().contiguous() @ x[at:to].double()
        assert torch.equal(dw[e], want.to(torch.bfloat16)), e


def test_4_bit_past_4_gib(lib, large):
    import torch
    x, offsets, dev = large
    codes, scales = lib.mxfp4_quantize(x)
    back = torch.empty_like(x)
    lib.mxfp4_dequantize(codes, scales, WIDE, out=back)
    assert torch.equal(back, x)
    del back
    w = _trits((3, 512, WIDE), torch.bfloat16)
    wc, ws = lib.mxfp4_quantize(w.reshape(-1, WIDE))
    wc, ws = wc.reshape(3, 512, -1), ws.reshape(3, 512, -1)
    for grouped in (False, True):
        out = torch.full((ROWS, 512), 7.0, device="cuda")
        if grouped:
            lib.mxfp4_gemm(codes, scales, wc, ws, WIDE, offsets=dev, out=out)
        else:
            lib.mxfp4_gemm(codes, scales, wc[1].contiguous(), ws[1].contiguous(), WIDE, out=out)
        for r in _around(offsets):
            e = _expert_of(r, offsets) if grouped else 1
            want = torch.full((512,), 7.0) if e is None else (w[e].double().cpu() @ x[r].double().cpu()).float()
            assert torch.equal(out[r].cpu(), want), (grouped, r)


def test_clip_past_4_gib(lib, large):
    import torch
    n = ROWS * WIDE + 3
    g, small = torch.ones(n, dtype=torch.bfloat16, device="cuda"), torch.ones(5, device="cuda")
    total = float(np.sqrt(np.float64(n + 5)))
    norm, (a, b) = lib.clip_grad_norm([g, small], 3.0)
    assert norm.item() == np.float32(total)
    by = torch.tensor(3.0 / (total + 1e-6), dtype=torch.float32, device="cuda")
    assert bool((a == by.to(torch.bfloat16)).all()) and bool((b == by).all())


@pytest.mark.parametrize("experts,rows", [(4999, 7003), (65535, 300)])
def test_thousands_of_experts(lib, gpu, experts, rows):
    import torch
    g = np.random.default_rng(3)
    ends = np.sort(g.integers(0, rows + 1, experts))
    ends[-1] = rows
    lengths = np.diff(np.concatenate([[0], ends]))
    offsets = torch.tensor(np.concatenate([[0], ends]), dtype=torch.int32, device="cuda")
    of = torch.tensor(np.repeat(np.arange(experts), lengths), device="cuda")
    x, dy = _trits((rows, 40), torch.float16), _trits((rows, 24), torch.float16)
    w = _trits((experts, 24, 40), torch.float16)
    out = lib.grouped_gemm(x, w, offsets)
    mine = w[of].float()
    assert torch.equal(out.float(), (mine * x.float()[:, None, :]).sum(2))
    dx, dw = lib.grouped_gemm_backward(dy, x, w, offsets)
    assert torch.equal(dx.float(), (mine * dy.float()[:, :, None]).sum(1))
    want = torch.zeros(experts, 24, 40, device="cuda")
    want.index_add_(0, of, dy.float()[:, :, None] * x.float()[:, None, :])  # (integers: in any order)
    assert torch.equal(dw.float(), want)
    wc, ws = lib.mxfp4_quantize(w.reshape(-1, 40))
    out = lib.mxfp4_grouped_linear(x, wc.reshape(experts, 24, -1), ws.reshape(experts, 24, -1), offsets)
    assert torch.equal(out.float(), (mine * x.float()[:, None, :]).sum(2))


def test_no_rows(lib, gpu):
    import torch
    x = torch.empty(0, 72, dtype=torch.bfloat16, device="cuda")
    w = _trits((2, 40, 72), torch.bfloat16)
    offsets = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert lib.grouped_gemm(x, w, offsets).shape == (0, 40)
    dx, dw = lib.grouped_gemm_backward(x.new_empty(0, 40), x, w, offsets, dw_out=torch.full_like(w, 7.0))
    assert dx.shape == (0, 72) and not bool(dw.any())
    codes, scales = lib.mxfp4_quantize(x)
    assert codes.shape == (0, 64) and scales.shape == (0, 4)
    assert lib.mxfp4_dequantize(codes, scales, 72).shape == (0, 72)
    wc, ws = lib.mxfp4_quantize(w.reshape(-1, 72))
    wc, ws = wc.reshape(2, 40, -1), ws.reshape(2, 40, -1)
    assert lib.mxfp4_gemm(codes, scales, wc[0], ws[0], 72).shape == (0, 40)
    assert lib.mxfp4_gemm(codes, scales, wc, ws, 72, offsets=offsets).shape == (0, 40)
    assert lib.mxfp4_linear(x, wc[0], ws[0]).shape == (0, 40)
    assert lib.mxfp4_grouped_linear(x, wc, ws, offsets).shape == (0, 40)


def test_clip_by_infinite_and_no_norms(lib, gpu):
    import torch
    g = [torch.tensor([1.0, -2.0, 2.0], device="cuda")]
    for most, norm, want in ((float("inf"), None, [1, -2, 2]), (0.0, None, [0, 0, 0]), (6.0, None, [1, -2, 2]),
                             (1.0, float("inf"), [0, 0, 0]), (0.5, 0.0, [1, -2, 2])):
        given = None if norm is None else torch.tensor(norm, device="cuda")
        told, (out,) = lib.clip_grad_norm(g, most, norm=given)
        assert out.tolist() == want, (most, norm)
        assert told.item() == (3.0 if norm is None else norm)
    _, (out,) = lib.clip_grad_norm(g, 1.0, norm=torch.tensor(float("nan"), device="cuda"))
    assert bool(out.isnan().all())
    flat = torch.ones(9, device="cuda")
    with pytest.raises(lib.SsgError, match="norm_in overlaps"):
        lib.clip_grad_norm([flat], 1.0, norm=flat[2], out=[flat])
