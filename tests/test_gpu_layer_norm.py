"""Layer norm forward and backward against a plain 64-bit implementation.

Tolerances (set before the first run).  Let u be the unit roundoff of the output
type (2^-11 fp16, 2^-8 bf16, 2^-24 fp32) and e = 2^-24.
  y      one final rounding u|y|; before it the fp32 chain: (s - mean) carries
         e|s|-sized errors of the mean (a tree sum of N terms, log2(N) + few
         roundings of sums of |s|), amplified by rstd |w|.  Allowed:
         u |y| + 64 e (rstd |w| (|s| + mean|s|) + |xh w| + |b|) + the type's
         smallest step.
  mean   32 e mean|s|;  rstd 64 e rstd (1 + rstd^2 mean(s^2) ...) -- with the
         two-sweep variance the relative error of rstd is a few e plus the
         error of the mean squared, so 64 e rstd.
  dx     u |dx| + 256 e rstd (|g| + mean|g| + |xh| mean|g xh|) + 4 e |dres| (added in
         fp32, before the one rounding) + smallest step.
  dw, db sums of M terms in fp32, a chain of at most ceil(M / slices) + 64
         additions: e (chain + 8) sum |term|, taken with chain <= M.
"""

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

E = 2.0 ** -24


def _types():
    import torch
    return {"f16": (torch.float16, 2.0 ** -11, 2.0 ** -24), "bf16": (torch.bfloat16, 2.0 ** -8, 1e-38),
            "f32": (torch.float32, 2.0 ** -24, 1e-38)}


def _case(seed, dtype, m, n, wdtype=None, offset=0.3):
    import torch
    dt = _types()[dtype][0]
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")
    wt = torch.float32 if wdtype == "f32" else dt
    return dict(x=(r(m, n) + offset).to(dt), res=r(m, n).to(dt), w=(1 + 0.3 * r(n)).to(wt), b=(0.2 * r(n)).to(wt),
                dy=r(m, n).to(dt), dres=r(m, n).to(dt))


def _check_forward(out, s, w, b, dtype, eps=1e-5):
    import torch
    _, u, tiny = _types()[dtype]
    y, mean, rstd = (t.double() for t in out[:3])
    s, n = s.double(), s.shape[1]
    w = torch.ones(n, device="cuda").double() if w is None else w.double()
    b = torch.zeros(n, device="cuda").double() if b is None else b.double()
    mu = s.sum(1) / n
    off = s - mu[:, None]
    rs = 1 / torch.sqrt((off * off).sum(1) / n + eps)
    ref = off * rs[:, None] * w + b
    size = s.abs().mean(1)
    assert ((mean - mu).abs() <= 32 * E * size + 1e-38).all()
    assert ((rstd - rs).abs() <= 64 * E * rs).all()
    xh = off * rs[:, None]
    bound = u * ref.abs() + 64 * E * (rs[:, None] * w.abs() * (s.abs() + size[:, None]) + (xh * w).abs() + b.abs()) + tiny
    bad = (y - ref).abs() > bound
    assert not bad.any(), (bad.sum().item(), ((y - ref).abs() / bound).max().item())


def _check_backward(got, dy, x, mean, rstd, w, dres, dtype):
    import torch
    _, u, tiny = _types()[dtype]
    m, n = x.shape
    dx, dw, db = got
    dy, x = dy.double(), x.double()
    wd = torch.ones(n, device="cuda").double() if w is None else w.double()
    rs = rstd.double()[:, None]
    xh = (x - mean.double()[:, None]) * rs
    g = dy * wd
    c1, c2 = g.sum(1, keepdim=True) / n, (g * xh).sum(1, keepdim=True) / n
    ref = rs * (g - c1 - xh * c2)
    size = rs * (g.abs() + g.abs().mean(1, keepdim=True) + xh.abs() * (g * xh).abs().mean(1, keepdim=True))
    if dres is not None:
        ref = ref + dres.double()
        size = size + dres.double().abs()
    bound = u * ref.abs() + 256 * E * size + tiny
    bad = (dx.double() - ref).abs() > bound
    assert not bad.any(), (bad.sum().item(), ((dx.double() - ref).abs() / bound).max().item())
    for have, term in ((dw, dy * xh), (db, dy)):
        if have is not None:
            off = (have.double() - term.sum(0)).abs()
            assert (off <= E * (m + 72) * term.abs().sum(0) + 1e-38).all()


# widths around every boundary of the register forms, odd ones, and past them all
SHAPES = [(1, 1), (1, 1024), (3, 7), (5, 64), (17, 511), (33, 512), (34, 513), (64, 768), (129, 1023), (130, 1025),
          (9, 2047), (9, 2049), (6, 4096), (6, 4097), (5, 8192), (5, 8193), (3, 16384), (3, 16385), (2, 40001)]


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("m,n", SHAPES)
def test_forward_and_backward(lib, gpu, dtype, m, n):
    c = _case(m * 100003 + n, dtype, m, n)
    out = lib.layer_norm(c["x"], c["w"], c["b"])
    _check_forward(out, c["x"], c["w"], c["b"], dtype)
    got = lib.layer_norm_backward(c["dy"], c["x"], out[1], out[2], c["w"])
    _check_backward(got, c["dy"], c["x"], out[1], out[2], c["w"], None, dtype)


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("m,n", [(37, 768), (5, 1537), (3, 4100), (2, 20000), (2500, 130)])
def test_residual_and_float_params(lib, gpu, dtype, m, n):
    import torch
    c = _case(n, dtype, m, n, wdtype="f32")
    y, mean, rstd, s = lib.layer_norm(c["x"], c["w"], c["b"], residual=c["res"])
    assert torch.equal(s, (c["x"].float() + c["res"].float()).to(c["x"].dtype))
    _check_forward((y, mean, rstd), s, c["w"], c["b"], dtype)
    got = lib.layer_norm_backward(c["dy"], s, mean, rstd, c["w"], dres=c["dres"])
    _check_backward(got, c["dy"], s, mean, rstd, c["w"], c["dres"], dtype)


@pytest.mark.parametrize("m,n", [(21, 384), (4, 3001), (2, 33000)])
def test_without_affine_and_frozen(lib, gpu, m, n):
    import torch
    c = _case(7, "f16", m, n)
    out = lib.layer_norm(c["x"])
    _check_forward(out, c["x"], None, None, "f16")
    only_b = lib.layer_norm(c["x"], None, c["b"])
    _check_forward(only_b, c["x"], None, c["b"], "f16")
    dx, dw, db = lib.layer_norm_backward(c["dy"], c["x"], out[1], out[2], param_grads=False)
    assert dw is None and db is None
    _check_backward((dx, None, None), c["dy"], c["x"], out[1], out[2], None, None, "f16")
    full = lib.layer_norm_backward(c["dy"], c["x"], out[1], out[2])
    assert torch.equal(full[0], dx)


@pytest.mark.parametrize("dtype", ["f16", "f32"])
@pytest.mark.parametrize("n", [96, 1001])
def test_strides_and_in_place(lib, gpu, dtype, n):
    import torch
    m = 19
    wide = _case(3, dtype, m, 3 * n + 5)
    x, res, dy = (wide[k][:, n + 1:2 * n + 1] for k in ("x", "res", "dy"))
    w, b = wide["w"][:n].contiguous(), wide["b"][1:n + 1]
    y, mean, rstd, s = lib.layer_norm(x, w, b, residual=res)
    y2, mean2, rstd2, s2 = lib.layer_norm(x.contiguous(), w, b.contiguous(), residual=res.contiguous())
    assert torch.equal(y, y2) and torch.equal(s, s2) and torch.equal(mean, mean2) and torch.equal(rstd, rstd2)
    dx, dw, db = lib.layer_norm_backward(dy, s, mean, rstd, w, dres=res)
    dx2, dw2, db2 = lib.layer_norm_backward(dy.contiguous(), s2, mean2, rstd2, w, dres=res.contiguous())
    assert torch.equal(dx, dx2) and torch.equal(dw, dw2) and torch.equal(db, db2)
    # outputs over their inputs
    keep = res.clone()
    before = wide["x"].clone()
    lib.layer_norm(x, w, b, residual=res, out=x, sum_out=res)
    assert torch.equal(x, y) and torch.equal(res, s)
    assert torch.equal(wide["x"][:, :n + 1], before[:, :n + 1]) and torch.equal(wide["x"][:, 2 * n + 1:],
                                                                               before[:, 2 * n + 1:])
    lib.layer_norm_backward(dy, s, mean, rstd, w, dres=keep, out=keep)
    assert torch.equal(keep, dx)


def test_large_offset_keeps_its_digits(lib, gpu):
    """A mean a thousand times the spread: the two-sweep variance loses nothing."""
    c = _case(11, "f32", 6, 1000, offset=1000.0)
    _check_forward(lib.layer_norm(c["x"], c["w"], c["b"]), c["x"], c["w"], c["b"], "f32")


def test_constant_rows_and_non_finite_values(lib, gpu):
    import torch
    x = torch.randn(6, 777, device="cuda").half()
    x[1] = 3.0  # no spread: rstd = 1 / sqrt(eps)
    x[2, 5] = float("inf")
    x[3, 700] = float("nan")
    w = torch.ones(777, device="cuda").half()
    b = torch.full((777,), 0.5, device="cuda").half()
    y, mean, rstd = lib.layer_norm(x, w, b)
    ref = torch.nn.functional.layer_norm(x.float().cpu(), (777,), w.float().cpu(), b.float().cpu())
    fine = [0, 1, 4, 5]
    assert (y[fine].float().cpu() - ref[fine]).abs().max() < 4e-3
    assert (y[1] == 0.5).all() and abs(rstd[1].item() - 1e-5 ** -0.5) < 1e-3
    assert not torch.isfinite(y[2].float()).any() and torch.isnan(y[3]).all()
    assert torch.isfinite(y[fine].float()).all()


def test_empty_and_single(lib, gpu):
    import torch
    x = torch.empty((0, 640), device="cuda").half()
    y, mean, rstd = lib.layer_norm(x)
    assert y.shape == (0, 640) and mean.shape == (0,)
    dx, dw, db = lib.layer_norm_backward(x, x, mean, rstd)
    assert dx.shape == (0, 640) and (dw == 0).all() and (db == 0).all()
    one = torch.full((4, 1), 2.0, device="cuda")
    y, mean, rstd = lib.layer_norm(one)
    assert (y == 0).all() and (mean == 2).all()


def test_gradient_against_differences(lib, gpu):
    """dx against central differences of the fp32 forward pass through a fixed linear functional."""
    import torch
    c = _case(5, "f32", 4, 37)
    x, w, b, dy = c["x"], c["w"], c["b"], c["dy"]
    out = lib.layer_norm(x, w, b)
    dx, dw, db = lib.layer_norm_backward(dy, x, out[1], out[2], w)

    def f(x, w, b):
        return (lib.layer_norm(x, w, b)[0].double() * dy.double()).sum().item()
    h = 2.0 ** -7
    # central differences: h^2 / 6 times a third derivative of order |dy| |w| N^0 plus rounding 2^-20 / h
    for i, j in ((0, 0), (1, 17), (3, 36)):
        step = torch.zeros_like(x)
        step[i, j] = h
        d = (f(x + step, w, b) - f(x - step, w, b)) / (2 * h)
        assert abs(d - dx[i, j].item()) < 2e-3, (d, dx[i, j].item())
    for j in (0, 20):
        step = torch.zeros_like(w)
        step[j] = h
        assert abs((f(x, w + step, b) - f(x, w - step, b)) / (2 * h) - dw[j].item()) < 2e-3
        assert abs((f(x, w, b + step) - f(x, w, b - step)) / (2 * h) - db[j].item()) < 2e-3


def test_repeatable_and_on_another_stream(lib, gpu):
    import torch
    c = _case(8, "bf16", 3001, 768)
    out = lib.layer_norm(c["x"], c["w"], c["b"])
    first = lib.layer_norm_backward(c["dy"], c["x"], out[1], out[2], c["w"])
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        out2 = lib.layer_norm(c["x"], c["w"], c["b"])
        again = lib.layer_norm_backward(c["dy"], c["x"], out2[1], out2[2], c["w"])
    torch.cuda.current_stream().wait_stream(st)
    for p, q in zip(first + out, again + out2):
        assert torch.equal(p, q)


def test_refusals(lib, gpu):
    import torch
    x = torch.zeros((4, 32), device="cuda", dtype=torch.float16)
    s = torch.zeros(4, device="cuda")
    with pytest.raises(TypeError):
        lib.layer_norm(x.cpu())
    with pytest.raises(TypeError):
        lib.layer_norm(x.double())
    with pytest.raises(ValueError):
        lib.layer_norm(x.t())
    with pytest.raises(ValueError):
        lib.layer_norm(x, torch.ones(31, device="cuda").half())
    with pytest.raises(TypeError):
        lib.layer_norm(x, torch.ones(32, device="cuda").bfloat16())
    with pytest.raises(lib.SsgError, match="eps"):
        lib.layer_norm(x, eps=-1.0)
    with pytest.raises(lib.SsgError, match="eps"):
        lib.layer_norm(x, eps=float("nan"))
    with pytest.raises(ValueError):
        lib.layer_norm_backward(x, x, s[:3], s)
    with pytest.raises(lib.SsgError, match="workspace"):
        lib.layer_norm_backward(x, x, s, s, workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))


@pytest.mark.parametrize("dtype", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("n", list(range(1, 18)) + [505, 1023, 2051, 4093, 8190, 16383])
def test_every_tail_of_a_row(lib, gpu, dtype, n):
    """Rows that end in part of a 16-byte piece: the values, nothing written beside them, and the same
    bits for a row wherever in the batch it lies."""
    import torch
    m = 9
    c = _case(n, dtype, m, n)
    dt = c["x"].dtype
    wide = [torch.full((m, n + 3), 7.0, dtype=dt, device="cuda") for _ in range(3)]
    y, s, dx = (t[:, 1:n + 1] for t in wide)
    out = lib.layer_norm(c["x"], c["w"], c["b"], residual=c["res"], out=y, sum_out=s)
    assert torch.equal(s, (c["x"].float() + c["res"].float()).to(dt))
    _check_forward(out, s, c["w"], c["b"], dtype)
    mean, rstd = out[1:3]
    got = lib.layer_norm_backward(c["dy"], s, mean, rstd, c["w"], dres=c["dres"], out=dx)
    _check_backward(got, c["dy"], s, mean, rstd, c["w"], c["dres"], dtype)
    for t in wide:
        assert (t[:, 0] == 7).all() and (t[:, n + 1:] == 7).all()
    for i in (0, 5):
        one = lib.layer_norm(c["x"][i:i + 1], c["w"], c["b"], residual=c["res"][i:i + 1])
        assert torch.equal(one[0], y[i:i + 1]) and torch.equal(one[2], rstd[i:i + 1])


def test_parameter_gradients_of_a_very_long_row(lib, gpu):
    """A row past 2^26 elements: the column sums' launch stays below 2^32 threads."""
    import torch
    m, n = 2, (1 << 26) + 5
    g = torch.Generator(device="cuda").manual_seed(1)
    x, dy = (torch.randn(m, n, generator=g, device="cuda", dtype=torch.float16) for _ in range(2))
    mean = torch.tensor([0.1, -0.2], device="cuda")
    rstd = torch.tensor([0.9, 1.3], device="cuda")
    dx, dw, db = lib.layer_norm_backward(dy, x, mean, rstd)
    at = torch.cat([torch.arange(0, n, 9973, device="cuda"), torch.arange(n - 70, n, device="cuda")])
    d = dy[:, at].double()
    xh = (x[:, at].double() - mean.double()[:, None]) * rstd.double()[:, None]
    # (the difference, the product and m sums in fp32: 2^-24 each)
    assert ((dw[at].double() - (d * xh).sum(0)).abs() <= E * (m + 8) * (d.abs() * (xh.abs() + 1)).sum(0)).all()
    assert ((db[at].double() - d.sum(0)).abs() <= E * (m + 8) * d.abs().sum(0)).all()
    assert torch.isfinite(dx[:, at]).all()
