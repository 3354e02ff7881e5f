"""The experts' calls on pools of weights past 4 GiB and on the longest rows.  Values are -1, 0 and 1: every sum
below 2^24 is exact in fp32, and results equal the 64-bit ones but for the output's one rounding."""

import pytest

pytestmark = pytest.mark.gpu


def _trits(*shape):
    import torch
    return torch.randint(-1, 2, shape, device="cuda", dtype=torch.int8).bfloat16()


def _offsets(*ends):
    import torch
    return torch.tensor(ends, dtype=torch.int32, device="cuda")


@pytest.fixture(scope="module")
def pool(gpu):
    """20 experts of 256 MiB: 5 GiB."""
    import torch
    torch.manual_seed(3)
    w = _trits(20, 8192, 16384)
    yield w
    del w
    torch.cuda.empty_cache()


def test_pools_past_4_gib(lib, pool):
    import torch
    experts, n, k = pool.shape
    ends = [0] * 7 + [3] + [3] * 8 + [40] * 4 + [77]  # expert 6: 3 rows, 15: 37, 19: 37
    offsets = _offsets(*ends)
    x, dy = _trits(77, k), _trits(77, n)
    out = lib.grouped_gemm(x, pool, offsets)
    for e in (6, 15, 19):
        rows = slice(ends[e], ends[e + 1])
        assert torch.equal(out[rows], (x[rows].double() @ pool[e].double().t().contiguous()).bfloat16()), e
    dx, dw = lib.grouped_gemm_backward(dy, x, pool, offsets)
    for e in range(experts):
        rows = slice(ends[e], ends[e + 1])
        if ends[e] == ends[e + 1]:
            assert not bool(dw[e].any()), e
            continue
        assert torch.equal(dx[rows], (dy[rows].double() @ pool[e].double()).bfloat16()), e
        assert torch.equal(dw[e], (dy[rows].double().t().contiguous() @ x[rows].double()).bfloat16()), e


def test_4_bit_pools_past_4_gib(lib, gpu):
    import torch
    experts, n, k = 72, 8192, 16384  # 64 MiB of codes each, 4.5 GiB
    some = _trits(3, n, k)
    codes = torch.zeros(experts, n, k // 2, dtype=torch.uint8, device="cuda")
    scales = torch.full((experts, n, k // 32), 255, dtype=torch.uint8, device="cuda")  # (NaN where no row may look)
    for i, e in enumerate((1, 40, 71)):
        c, s = lib.mxfp4_quantize(some[i])
        codes[e], scales[e] = c, s
    for lengths in ((2, 3, 4), (300, 40, 513)):  # few rows, and the tiles
        ends, at = [0], 0
        for e in range(experts):
            at += lengths[(1, 40, 71).index(e)] if e in (1, 40, 71) else 0
            ends.append(at)
        x = _trits(at, k)
        out = lib.mxfp4_grouped_linear(x, codes, scales, _offsets(*ends))
        for i, e in enumerate((1, 40, 71)):
            rows = slice(ends[e], ends[e + 1])
            want = x[rows].double() @ some[i].double().t().contiguous()
            assert torch.equal(out[rows], want.bfloat16()), (lengths, e)


@pytest.mark.parametrize("m", [3, 300])
def test_longest_rows_of_16_bits(lib, gpu, m):
    """K just below 2^22, N = 8, and the other way round."""
    import torch
    torch.manual_seed(m)
    wide, narrow = (1 << 22) - 8, 8
    offsets = _offsets(0, m // 2, m)
    x, w, dy = _trits(m, wide), _trits(2, narrow, wide), _trits(m, narrow)
    halves = ((0, slice(0, m // 2)), (1, slice(m // 2, m)))
    out = lib.grouped_gemm(x, w, offsets)
    dx, dw = lib.grouped_gemm_backward(dy, x, w, offsets)
    for e, rows in halves:
        assert torch.equal(out[rows], (x[rows].double() @ w[e].double().t().contiguous()).bfloat16())
        assert torch.equal(dx[rows], (dy[rows].double() @ w[e].double()).bfloat16())
        assert torch.equal(dw[e], (dy[rows].double().t().contiguous() @ x[rows].double()).bfloat16())
    w, x, dy = w.view(2, wide, narrow), dy, x
    out = lib.grouped_gemm(x, w, offsets)
    dx, dw = lib.grouped_gemm_backward(dy, x, w, offsets)
    for e, rows in halves:
        assert torch.equal(out[rows], (x[rows].double() @ w[e].double().t().contiguous()).bfloat16())
        assert torch.equal(dx[rows], (dy[rows].double() @ w[e].double()).bfloat16())
        assert torch.equal(dw[e], (dy[rows].double().t().contiguous() @ x[rows].double()).bfloat16())


@pytest.mark.parametrize("m,n", [(2, 3), (300, 40), (600, 5)])
def test_longest_rows_of_4_bits(lib, gpu, m, n):
    import torch
    torch.manual_seed(m)
    k = (1 << 22) - 1
    x, w = _trits(m, k), _trits(n, k)
    codes, scales = lib.mxfp4_quantize(w)
    assert torch.equal(lib.mxfp4_dequantize(codes, scales, k, torch.bfloat16), w)
    out = lib.mxfp4_linear(x, codes, scales)
    want = x.double() @ w.double().t().contiguous()
    assert torch.equal(out, want.bfloat16())
