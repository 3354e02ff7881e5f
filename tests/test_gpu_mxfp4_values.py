"""4-bit quantisation of every 16-bit value below a larger one, and products at the ends of the scales' range."""

import numpy as np
import pytest
from test_gpu_mxfp4 import _cpu, _dt, ref_quantize, ref_values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("top", [1.0, 1.75, 1.9921875])
def test_quantize_every_16_bit_value_below_a_larger_one(lib, gpu, dt, top):
    """Every bit pattern, as the second value of a block whose first one, `top` times a power of two, sets the
    scale 2^0 .. 2^4 above it."""
    import torch
    v = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(_dt(dt))
    f = v.double().abs()
    lead = torch.where(torch.isfinite(f) & (f > 0), torch.exp2(torch.floor(torch.log2(f.clamp_min(1e-45)))), 1.0)
    x = torch.zeros(65536, 32, dtype=_dt(dt))
    x[:, 0] = (lead * top * torch.exp2((torch.arange(65536) % 5).double())).to(_dt(dt))
    x[:, 1] = v
    codes, scales = lib.mxfp4_quantize(x.cuda())
    want = ref_quantize(x.double().numpy())
    assert np.array_equal(_cpu(scales), want[1])
    assert np.array_equal(_cpu(codes), want[0])


def _operands(m, n, k, first, g):
    """Random codes; the scales of block b of a and w are 2^(first[b] - 127) and 2^(127 - first[b]), times 1 to 4."""
    import torch
    codes = lambda rows: torch.randint(0, 256, (rows, k // 2), generator=g, dtype=torch.uint8)
    near = lambda rows: torch.randint(0, 3, (rows, k // 32), generator=g)
    a, w = codes(m), codes(n)
    return a, (first + near(m)).to(torch.uint8), w, (254 - first - near(n)).clamp_min(0).to(torch.uint8)


@pytest.mark.parametrize("m,n,k", [(5, 40, 256), (20, 70, 512), (70, 128, 384), (400, 300, 640), (2100, 300, 256)])
def test_products_at_every_scale(lib, gpu, m, n, k):
    """One operand's scales from 2^-127 to 2^126 where the other's undo them: every sum is a whole number of
    quarters below 2^20 and exact."""
    import torch
    g = torch.Generator().manual_seed(m + k)
    blocks = k // 32
    for low in (0, 1, 2, 60, 128, 200, 244):
        first = low + torch.arange(blocks) % 8
        a, sa, w, sw = _operands(m, n, k, first, g)
        got = lib.mxfp4_gemm(a.cuda(), sa.cuda(), w.cuda(), sw.cuda(), k, torch.float32)
        want = ref_values(a.numpy(), sa.numpy(), k) @ ref_values(w.numpy(), sw.numpy(), k).T
        assert np.array_equal(_cpu(got.double()), want), low


@pytest.mark.parametrize("m", [5, 70, 700])
def test_products_below_the_normal_values(lib, gpu, m):
    """Scales whose product is 2^-140 and 2^-254: whole numbers of 2^-142, which fp32 holds, and nothing that it does."""
    import torch
    g = torch.Generator().manual_seed(m)
    n, k = 72, 256
    a, w = (torch.randint(0, 256, (rows, k // 2), generator=g, dtype=torch.uint8) for rows in (m, n))
    for sa, sw in ((100, 14), (14, 100), (0, 0)):
        fa, fw = (torch.full((rows, k // 32), s, dtype=torch.uint8) for rows, s in ((m, sa), (n, sw)))
        got = lib.mxfp4_gemm(a.cuda(), fa.cuda(), w.cuda(), fw.cuda(), k, torch.float32)
        want = ref_values(a.numpy(), fa.numpy(), k) @ ref_values(w.numpy(), fw.numpy(), k).T
        assert np.array_equal(_cpu(got.double()), want.astype(np.float32).astype(np.float64)), (sa, sw)
