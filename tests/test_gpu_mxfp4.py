"""Microscaled 4-bit rows: quantisation and its inverse bit for bit against the
format's definition, products against 64-bit sums.

Bound of a product's error: the products of two 4-bit values and their power-of-two
scales are exact, so only sums and the last rounding count; n fp32 additions in any
order are off by at most n 2^-24 sum|a||w| (to first order; twice that is allowed), and
the rounding to the output by half a step, eps / 2 of the value."""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

MAGS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def padded(k):
    return -(-k // 128) * 128


def ref_quantize(x):
    """x float64 [M, K] -> (codes [M, kp/2], scales [M, kp/32]) uint8."""
    m, k = x.shape
    kp = padded(k)
    v = np.zeros((m, kp))
    v[:, :k] = x
    v = v.reshape(m, kp // 32, 32)
    fine = np.isfinite(v).all(2)
    top = np.where(fine, np.abs(np.where(np.isfinite(v), v, 0)).max(2), 0)
    e = np.frexp(np.where(top > 0, top, 1.0))[1] - 1  # floor(log2)
    byte = np.where(top > 0, np.clip(e - 2 + 127, 0, 254), 0)
    a = np.abs(np.where(fine[..., None], v, 0)) * np.exp2(127.0 - byte)[..., None]
    away = np.abs(a[..., None] - MAGS)
    near = away.min(-1, keepdims=True)
    code = np.zeros(a.shape, int)
    for i in (1, 3, 5, 7, 0, 2, 4, 6):  # (the even code last: it wins a tie)
        code = np.where(away[..., i] == near[..., 0], i, code)
    code = np.where(a >= 6, 7, code) | np.where(np.signbit(v), 8, 0)
    code = np.where(fine[..., None], code, 0).reshape(m, kp).astype(np.uint8)
    return code[:, ::2] | code[:, 1::2] << 4, np.where(fine, byte, 255).astype(np.uint8)


def ref_values(codes, scales, k):
    c = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1)
    v = MAGS[c & 7] * np.where(c >= 8, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, np.exp2(scales.astype(np.float64) - 127))
    return (v * np.repeat(s, 32, 1))[:, :k]


def _dt(name):
    import torch
    return {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}[name]


def _cpu(t):
    return t.cpu().numpy()


def _random(m, k, dt, seed):
    import torch
    g = torch.Generator().manual_seed(seed)
    spread = torch.exp2(torch.randint(-14, 12, (m, 1), generator=g).float())
    return (torch.randn(m, k, generator=g) * spread).to(_dt(dt))


@pytest.mark.parametrize("dt", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("m,k", [(1, 1), (1, 31), (3, 32), (2, 33), (5, 127), (7, 128), (4, 130), (1, 1000), (33, 2049),
                                 (300, 264), (1000, 1024)])
def test_quantize(lib, gpu, m, k, dt):
    x = _random(m, k, dt, m + k)
    codes, scales = lib.mxfp4_quantize(x.cuda())
    want = ref_quantize(x.double().numpy())
    assert np.array_equal(_cpu(scales), want[1])
    assert np.array_equal(_cpu(codes), want[0])
    for out in ("f16", "bf16", "f32"):
        back = _cpu(lib.mxfp4_dequantize(codes, scales, k, _dt(out)).double())
        import torch
        assert np.array_equal(back, torch.from_numpy(ref_values(*want, k)).to(_dt(out)).double().numpy())


@pytest.mark.parametrize("dt", ["f16", "bf16"])
@pytest.mark.parametrize("top", [1.0, 1.75, 1.9921875])
def test_quantize_every_16_bit_value(lib, gpu, dt, top):
    """Every bit pattern, as the second value of a block whose first one sets the scale 2^0 .. 2^4 above it."""
    import torch
    v = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(_dt(dt))
    x = torch.zeros(65536, 32, dtype=_dt(dt))
    x[:, 1] = v
    f = v.double().abs()
    lead = torch.where(torch.isfinite(f) & (f > 0), torch.exp2(torch.floor(torch.log2(f.clamp_min(1e-45)))), 1.0)
    x[:, 0] = (lead * top * torch.exp2((torch.arange(65536) % 5).double())).to(_dt(dt))
    codes, scales = lib.mxfp4_quantize(x.cuda())
    want = ref_quantize(x.double().numpy())
    assert np.array_equal(_cpu(scales), want[1])
    assert np.array_equal(_cpu(codes), want[0])


def test_quantize_extremes(lib, gpu):
    import torch
    inf, nan = float("inf"), float("nan")
    rows = [[0.0] * 32, [-0.0] * 32, [1e-45] + [0.0] * 31, [2.0 ** -126] * 32, [2.0 ** -125, 2.0 ** -127] + [2.0 ** -129] * 30,
            [3.4e38, -3.4e38] + [1e38] * 30, [inf] + [1.0] * 31, [1.0] * 31 + [nan], [-inf, nan] + [0.0] * 30,
            [5.0, 2.5, 3.5, 0.25, 0.75, 1.25, 1.75, -5.0, 7.0, 6.5] + [0.0] * 22]
    x = torch.tensor(rows)
    codes, scales = lib.mxfp4_quantize(x.cuda())
    want = ref_quantize(x.double().numpy())
    assert np.array_equal(_cpu(scales), want[1]) and np.array_equal(_cpu(codes), want[0])
    back = _cpu(lib.mxfp4_dequantize(codes, scales, 32).double())
    assert np.isnan(back[6:9]).all() and np.array_equal(back, ref_values(*want, 32), equal_nan=True)


@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_quantize_every_16_bit_value(lib, gpu, dt):
    """Each bit pattern, in blocks of its neighbours, of values up to 2^5 times as large and beside its
    ties: quantised in a call of its own and inside a product of few rows and of many."""
    import torch
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    near = bits.view(_dt(dt)).view(2048, 32)
    g = torch.Generator().manual_seed(7)
    finite = near.flatten()[torch.isfinite(near.flatten())]
    spread = finite[torch.randint(0, len(finite), (4096, 32), generator=g)].double()
    top = spread[:, :1].abs()
    spread = (top * 2.0 ** torch.randint(-5, 1, (4096, 32), generator=g) * (1 + torch.rand(4096, 32, generator=g) / 2))
    ties = top * torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 4.0] * 4) / 4
    x = torch.cat([near, spread.to(_dt(dt)), ties.to(_dt(dt))])
    codes, scales = lib.mxfp4_quantize(x.cuda())
    want = ref_quantize(x.double().numpy())
    assert np.array_equal(_cpu(scales), want[1]) and np.array_equal(_cpu(codes), want[0])
    # a product with 1 at one place of each block gives that value back
    eye = torch.zeros(32, 32)
    eye.fill_diagonal_(1.0)
    w = lib.mxfp4_quantize(eye.cuda())
    values = torch.from_numpy(ref_values(*want, 32)).to(_dt(dt))
    values[values.isnan().any(1)] = float("nan")
    for at in list(range(0, len(x), 512)) + [None]:
        part = x if at is None else x[at:at + 31]
        got = lib.mxfp4_linear(part.cuda(), *w).cpu()
        assert torch.equal(got.isnan(), values[at:at + 31].isnan() if at is not None else values.isnan())
        assert torch.equal(got.nan_to_num(), (values if at is None else values[at:at + 31]).nan_to_num())


def test_dequantize_every_code_and_scale(lib, gpu):
    import torch
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(1, 256).repeat(256, 1)
    scales = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(256, 1).repeat(1, 16)
    want = ref_values(codes.numpy(), scales.numpy(), 512)
    for dt in ("f16", "bf16", "f32"):
        got = lib.mxfp4_dequantize(codes.cuda(), scales.cuda(), 512, _dt(dt))
        assert np.array_equal(_cpu(got.double()), torch.from_numpy(want).to(_dt(dt)).double().numpy(), equal_nan=True)


@pytest.mark.parametrize("dt", ["f16", "f32"])
def test_strided_rows(lib, gpu, dt):
    import torch
    wide = _random(9, 300, dt, 3).cuda()
    x = wide[:, 7:207]
    codes, scales = lib.mxfp4_quantize(x)
    same = lib.mxfp4_quantize(x.contiguous())
    assert torch.equal(codes, same[0]) and torch.equal(scales, same[1])
    out = torch.full_like(wide, 9.0)
    lib.mxfp4_dequantize(codes, scales, 200, out=out[:, 7:207])
    assert torch.equal(out[:, 7:207], lib.mxfp4_dequantize(codes, scales, 200, _dt(dt)))
    assert bool((out[:, :7] == 9).all()) and bool((out[:, 207:] == 9).all())


def _weight(n, k, seed, lo=117, hi=123):
    import torch
    g = torch.Generator().manual_seed(seed)
    codes = torch.randint(0, 256, (n, padded(k) // 2), generator=g, dtype=torch.uint8)
    codes[:, (k + 1) // 2:] = 0
    if k % 2:
        codes[:, k // 2] &= 15
    return codes, torch.randint(lo, hi, (n, padded(k) // 32), generator=g, dtype=torch.uint8)


def _close(got, a, w, dt):
    """The bound of the module's docstring."""
    import torch
    want, size = a @ w.T, np.abs(a) @ np.abs(w).T
    half = torch.finfo(_dt(dt)).eps / 2
    tiny = torch.finfo(_dt(dt)).smallest_normal * torch.finfo(_dt(dt)).eps
    bound = half * np.abs(want) + (1 + half) * 2 * a.shape[1] * 2.0 ** -24 * size + tiny
    miss = np.abs(_cpu(got.double()) - want)
    assert (miss <= bound).all(), float((miss - bound).max())


SIZES = [(1, 1, 1), (1, 64, 64), (2, 100, 128), (4, 4096, 1024), (17, 129, 257), (31, 96, 4000), (33, 128, 640),
         (64, 200, 1000), (65, 130, 384), (128, 512, 512), (257, 259, 1100), (300, 1024, 2048), (700, 513, 768),
         (1031, 264, 130), (2100, 2111, 300)]


@pytest.mark.parametrize("m,n,k", SIZES)
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_linear(lib, gpu, m, n, k, dt):
    x = _random(m, k, dt, m)
    codes, scales = _weight(n, k, n)
    got = lib.mxfp4_linear(x.cuda(), codes.cuda(), scales.cuda())
    assert got.dtype == _dt(dt) and got.shape == (m, n)
    a = ref_values(*ref_quantize(x.double().numpy()), k)
    w = ref_values(codes.numpy(), scales.numpy(), k)
    if dt == "f16":  # (values beyond its range are another test's)
        keep = (np.abs(a) @ np.abs(w).T).max(1) < 6e4
        assert keep.any()
        got, a = got[:, :].cpu()[np.flatnonzero(keep)], a[keep]
    _close(got, a, w, dt)


# rows that share a tile of 32 in every way that it takes them, K of one and of many units of 256 values,
# whole, half and odd
@pytest.mark.parametrize("m", [1, 2, 3, 8, 9, 32, 33, 70])
@pytest.mark.parametrize("n,k", [(1, 3), (33, 128), (70, 385), (40, 1030), (96, 2500), (130, 5001), (31, 8320)])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_few_rows(lib, gpu, m, n, k, dt):
    import torch
    wide = _random(m, k + 5, "f32", m + n).clamp(-8, 8).to(_dt(dt)).cuda()
    x = wide[:, 3:3 + k]  # (rows at any element)
    codes, scales = _weight(n, k, n + m)
    out = torch.full((m, n + 3), 5.0, dtype=_dt(dt), device="cuda")
    lib.mxfp4_linear(x, codes.cuda(), scales.cuda(), out=out[:, 1:1 + n])
    packed = lib.mxfp4_quantize(x)
    assert torch.equal(out[:, 1:1 + n], lib.mxfp4_gemm(*packed, codes.cuda(), scales.cuda(), k, _dt(dt)))
    assert bool((out[:, 0] == 5).all()) and bool((out[:, 1 + n:] == 5).all())
    a = ref_values(*ref_quantize(_cpu(x.double())), k)
    _close(out[:, 1:1 + n], a, ref_values(codes.numpy(), scales.numpy(), k), dt)


@pytest.mark.parametrize("m,n,k", [(3, 70, 200), (40, 65, 513), (200, 131, 129), (600, 300, 256)])
def test_gemm_fp32_is_linear_before_its_rounding(lib, gpu, m, n, k):
    import torch
    x = _random(m, k, "bf16", 5).cuda()
    codes, scales = (t.cuda() for t in _weight(n, k, 6))
    full = lib.mxfp4_gemm(*lib.mxfp4_quantize(x), codes, scales, k, torch.float32)
    assert torch.equal(full.bfloat16(), lib.mxfp4_linear(x, codes, scales))
    _close(full, ref_values(*ref_quantize(_cpu(x.double())), k), ref_values(_cpu(codes), _cpu(scales), k), "f32")


def test_codes_are_exact_in_the_matrix_instruction(lib, gpu):
    """Whole numbers small enough that every sum is exact: the product is, bit for bit, at every scale."""
    import torch
    g = torch.Generator().manual_seed(1)
    for m, n, k in ((5, 40, 256), (70, 128, 384), (400, 300, 640)):
        a = torch.randint(0, 256, (m, k // 2), generator=g, dtype=torch.uint8)
        w = torch.randint(0, 256, (n, k // 2), generator=g, dtype=torch.uint8)
        sa = torch.randint(125, 129, (m, k // 32), generator=g, dtype=torch.uint8)
        sw = torch.randint(125, 129, (n, k // 32), generator=g, dtype=torch.uint8)
        got = lib.mxfp4_gemm(a.cuda(), sa.cuda(), w.cuda(), sw.cuda(), k, torch.float32)
        want = ref_values(a.numpy(), sa.numpy(), k) @ ref_values(w.numpy(), sw.numpy(), k).T
        assert np.array_equal(_cpu(got.double()), want)


@pytest.mark.parametrize("m", [4, 50, 300])
def test_nan_blocks_stay_in_their_row_and_column(lib, gpu, m):
    import torch
    k, n = 500, 90
    x = _random(m, k, "bf16", 2)
    clean = x.clone()
    x[1, 40], x[2, 499] = float("nan"), float("inf")
    codes, scales = _weight(n, k, 3)
    broken = scales.clone()
    broken[7, 3] = 255
    got = lib.mxfp4_linear(x.cuda(), codes.cuda(), broken.cuda()).cpu()
    want = lib.mxfp4_linear(clean.cuda(), codes.cuda(), scales.cuda()).cpu()
    bad = torch.zeros(m, n, dtype=torch.bool)
    bad[1:3], bad[:, 7] = True, True
    assert bool(torch.isnan(got[bad]).all()) and torch.equal(got[~bad], want[~bad])


def test_out_strided_and_kept(lib, gpu):
    import torch
    x = _random(70, 300, "f16", 4).cuda() / 64
    codes, scales = (t.cuda() for t in _weight(77, 300, 5))
    wide = torch.full((72, 101), 3.0, dtype=torch.float16, device="cuda")
    out = lib.mxfp4_linear(x, codes, scales, out=wide[1:71, 5:82])
    assert out.data_ptr() == wide[1:71, 5:82].data_ptr()
    assert torch.equal(out, lib.mxfp4_linear(x, codes, scales))
    wide[1:71, 5:82] = 3
    assert bool((wide == 3).all())


def _groups(m, e, seed, used=1.0):
    import torch
    g = torch.Generator().manual_seed(seed)
    pick = torch.randint(0, e, (int(m * used),), generator=g) ** 2 // max(e, 1)
    return torch.cat([torch.zeros(1), torch.cumsum(torch.bincount(pick, minlength=e)[:e], 0)]).to(torch.int32)


@pytest.mark.parametrize("m,n,k,e,used", [(1, 64, 128, 1, 1.0), (5, 70, 100, 8, 1.0), (40, 256, 512, 3, 1.0),
                                          (130, 96, 640, 70, 1.0), (200, 131, 257, 2, 0.9), (900, 300, 384, 5, 0.8),
                                          (3000, 260, 256, 4, 0.95), (64, 40, 64, 200, 1.0)])
@pytest.mark.parametrize("dt", ["f16", "bf16"])
def test_grouped_linear(lib, gpu, m, n, k, e, used, dt):
    import torch
    x = (torch.randn(m, k, generator=torch.Generator().manual_seed(m))).to(_dt(dt))
    codes, scales = _weight(e * n, k, e)
    offsets = _groups(m, e, m + e, used)
    out = torch.full((m, n), 5.0, dtype=_dt(dt), device="cuda")
    got = lib.mxfp4_grouped_linear(x.cuda(), codes.view(e, n, -1).cuda(), scales.view(e, n, -1).cuda(), offsets.cuda(),
                                   out=out)
    a, w = ref_values(*ref_quantize(x.double().numpy()), k), ref_values(codes.numpy(), scales.numpy(), k)
    o = offsets.tolist()
    for i in range(e):
        if o[i + 1] > o[i]:
            _close(got[o[i]:o[i + 1]], a[o[i]:o[i + 1]], w[i * n:(i + 1) * n], dt)
    assert bool((got[o[-1]:] == 5).all())
