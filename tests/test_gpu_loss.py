"""Linear cross entropy (forward and backward) against a plain 64-bit implementation.

Tolerances, set before the first run; e = 2^-24, u the unit roundoff of the type.
  lse, loss  a logit carries e (D + 64) |x| . |w| (an fp32 chain over D exact
             products); lse adds its own logarithm and sums, 64 e (1 + |lse|).
  G          p carries the logit's and lse's error, its exponential (64 e of the
             exponent's size), and one rounding u of |G|; fp16 cannot go below
             2^-24 of a scaled value, 2^-36 of the largest |dloss|.
  dx, dw     u |ref| + sum over |G error| |w| (or |x|) + e (chain + 64) sum |G| |w|
             + the type's smallest step."""

import pytest

pytestmark = pytest.mark.gpu
E = 2.0 ** -24


def _kind(dtype):
    import torch
    return {"f16": (torch.float16, 2.0 ** -11, 2.0 ** -24), "bf16": (torch.bfloat16, 2.0 ** -8, 1e-37)}[dtype]


def make(seed, dtype, m, v, d, spread=1.5, ignore=0.1):
    import torch
    dt = _kind(dtype)[0]
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = (torch.randn(v, d, generator=g, device="cuda") * spread / d ** 0.5).to(dt)
    t = torch.randint(0, v, (m,), generator=g, device="cuda")
    x = (torch.randn(m, d, generator=g, device="cuda") + 3 * torch.rand(m, 1, generator=g, device="cuda") *
         w[t].float()).to(dt)
    t[torch.rand(m, generator=g, device="cuda") < ignore] = -100
    return x, w, t, torch.randn(m, generator=g, device="cuda")


def check_forward(got, x, w, t):
    import torch
    loss, lse = got
    z = x.double() @ w.double().t()
    size = (x.double().abs() @ w.double().abs().t()).amax(1)
    ref = torch.logsumexp(z, 1)
    keep = t != -100
    ref_loss = torch.where(keep, ref - z.gather(1, t.clamp(min=0)[:, None])[:, 0], 0.0)
    bound = E * (x.shape[1] + 64) * size + 64 * E * (1 + ref.abs())
    assert ((lse.double() - ref).abs() <= bound).all(), ((lse.double() - ref).abs() / bound).max().item()
    assert ((loss.double() - ref_loss).abs() <= 2 * bound).all()
    assert (loss[~keep] == 0).all()


def gradient(x, w, t, dloss, lse):
    import torch
    z = x.double() @ w.double().t()
    p = torch.exp(z - lse.double()[:, None])
    keep = t != -100
    g = p.clone()
    g[torch.arange(len(t), device="cuda"), t.clamp(min=0)] -= 1
    c = torch.where(keep, dloss.double(), 0.0)[:, None]
    return z, p, g * c, c


def check_backward(got, x, w, t, dloss, lse, dtype):
    import torch
    _, u, tiny = _kind(dtype)
    dx, dw = got
    z, p, g, c = gradient(x, w, t, dloss, lse)
    xa, wa = x.double().abs(), w.double().abs()
    size = xa @ wa.t()
    dz = E * (x.shape[1] + 64) * size + 64 * E * (1 + (z - lse.double()[:, None]).abs())
    low = 2.0 ** -36 * c.abs().max() * (dtype == "f16")
    dg = u * g.abs() + c.abs() * p * dz * 2 + 4 * E * g.abs() + low
    for have, ref, err, chain in ((dx, g @ w.double(), dg @ wa + E * (len(w) + 64) * (g.abs() @ wa), 0),
                                  (dw, g.t() @ x.double(), dg.t() @ xa + E * (len(x) + 64) * (g.abs().t() @ xa), 0)):
        off, bound = (have.double() - ref).abs(), u * ref.abs() + err + tiny
        assert (off <= bound).all(), (off / bound).max().item()


SHAPES = [(1, 1, 1), (1, 100, 64), (3, 7, 5), (64, 1000, 768), (65, 64, 64), (130, 257, 100), (200, 4097, 72),
          (257, 999, 520), (2050, 515, 128), (1000, 8200, 192), (300, 30001, 64), (7000, 2500, 64)]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,v,d", SHAPES)
def test_forward_and_backward(lib, gpu, dtype, m, v, d):
    x, w, t, dloss = make(m + v + d, dtype, m, v, d)
    got = lib.linear_cross_entropy(x, w, t)
    check_forward(got, x, w, t)
    check_backward(lib.linear_cross_entropy_backward(dloss, x, w, t, got[1]), x, w, t, dloss, got[1], dtype)


@pytest.mark.parametrize("m,v,d", [(4100, 9001, 64), (16500, 4500, 64)])
def test_several_pieces_of_the_vocabulary(lib, gpu, m, v, d):
    """Enough rows that the gradient works through the vocabulary in more than one piece."""
    x, w, t, dloss = make(m, "f16", m, v, d)
    got = lib.linear_cross_entropy(x, w, t)
    check_backward(lib.linear_cross_entropy_backward(dloss, x, w, t, got[1]), x, w, t, dloss, got[1], "f16")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,v,d", [(1, 2049, 64), (38, 4306, 1210), (187, 5382, 264), (9000, 20001, 64)])
def test_split_sum_over_the_vocabulary(lib, gpu, dtype, m, v, d):
    """Few tiles of dx against a long vocabulary (the last with two pieces): its sum is split, the
    same way in every call, and a row without weight holds zeros whatever its input is."""
    x, w, t, dloss = make(m + v, dtype, m, v, d, ignore=0.0)
    _, lse = lib.linear_cross_entropy(x, w, t)
    got = lib.linear_cross_entropy_backward(dloss, x, w, t, lse)
    check_backward(got, x, w, t, dloss, lse, dtype)
    again = lib.linear_cross_entropy_backward(dloss, x, w, t, lse)
    assert got[0].equal(again[0]) and got[1].equal(again[1])
    t[m // 2] = -100
    dx, _ = lib.linear_cross_entropy_backward(dloss, x, w, t, lse)
    assert (dx[m // 2] == 0).all()


def test_more_tiles_than_one_launch_takes(lib, gpu):
    """Rows times entries past the 2^32 threads of one launch: the statistics come from two."""
    import torch
    m, v, d = 7_990_001, 69_000, 64
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randn(m, d, generator=g, device="cuda", dtype=torch.float16)
    w = (torch.randn(v, d, generator=g, device="cuda") * 0.2).half()
    t = torch.randint(0, v, (m,), generator=g, device="cuda")
    loss, lse = lib.linear_cross_entropy(x, w, t)
    at = torch.cat([torch.arange(0, m, 79_861, device="cuda"), torch.arange(m - 40, m, device="cuda")])
    check_forward((loss[at], lse[at]), x[at], w, t[at])
    assert torch.isfinite(loss).all() and torch.isfinite(lse).all()


def test_strides(lib, gpu):
    import torch
    x, w, t, dloss = make(1, "f16", 77, 300, 3 * 128)
    xs, ws = x[:, 65:65 + 128], w[:, 129:129 + 128]
    a = lib.linear_cross_entropy(xs, ws, t)
    b = lib.linear_cross_entropy(xs.contiguous(), ws.contiguous(), t)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    ga = torch.zeros_like(x), torch.zeros_like(w)
    lib.linear_cross_entropy_backward(dloss, xs, ws, t, a[1], out=ga[0][:, 3:131], dw_out=ga[1][:, 8:136])
    gb = lib.linear_cross_entropy_backward(dloss, xs.contiguous(), ws.contiguous(), t, a[1])
    for p, q, c in ((ga[0], gb[0], 3), (ga[1], gb[1], 8)):
        assert torch.equal(p[:, c:c + 128], q) and (p[:, :c] == 0).all() and (p[:, c + 128:] == 0).all()


def test_confident_and_extreme_rows(lib, gpu):
    """Logits of several hundred: no overflow, losses from 0 to over 20, gradients to match."""
    import torch
    x, w, t, dloss = make(2, "f16", 96, 640, 64, spread=40.0)
    got = lib.linear_cross_entropy(x, w, t)
    check_forward(got, x, w, t)
    assert got[1].max() > 300 and got[0].max() > 20 and got[0][t != -100].min() < 1e-3  # (what the inputs are for)
    check_backward(lib.linear_cross_entropy_backward(dloss, x, w, t, got[1]), x, w, t, dloss, got[1], "f16")


def test_gradient_scale_spans_its_rows(lib, gpu):
    """Row weights from 1 to 1e-4, and a common factor far below fp16's range: the rows keep their digits."""
    import torch
    x, w, t, _ = make(3, "bf16", 128, 500, 64, ignore=0.0)
    lse = lib.linear_cross_entropy(x, w, t)[1]
    dloss = torch.logspace(0, -4, 128, device="cuda") * 1e-9
    check_backward(lib.linear_cross_entropy_backward(dloss, x, w, t, lse), x, w, t, dloss, lse, "bf16")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("value", [float("inf"), float("-inf"), float("nan")])
@pytest.mark.parametrize("m,v,d", [(1, 50, 64), (90, 300, 64), (70, 4306, 72), (4100, 9001, 64)])
def test_a_weight_that_is_not_finite_stays_with_its_row(lib, gpu, dtype, value, m, v, d):
    """dloss[m] infinite or NaN: dx of that row and dw are not finite, the other rows of dx are what
    they are beside a zero there (the same bits: the rows' common factor is the largest finite one)."""
    import torch
    x, w, t, dloss = make(m + v, dtype, m, v, d)
    bad = m // 2
    t[bad] = v // 3
    lse = lib.linear_cross_entropy(x, w, t)[1]
    plain, broken = dloss.clone(), dloss.clone()
    plain[bad], broken[bad] = 0.0, value
    others = torch.arange(m, device="cuda") != bad
    ref = lib.linear_cross_entropy_backward(plain, x, w, t, lse)
    dx, dw = lib.linear_cross_entropy_backward(broken, x, w, t, lse)
    assert torch.equal(dx[others], ref[0][others])
    assert not torch.isfinite(dx[bad]).any() and not torch.isfinite(dw).any()
    # every finite weight zero
    zero = torch.zeros_like(dloss)
    zero[bad] = value
    dx, _ = lib.linear_cross_entropy_backward(zero, x, w, t, lse)
    assert (dx[others] == 0).all() and not torch.isfinite(dx[bad]).any()
    # in an ignored row it is not looked at
    t[bad] = -100
    for p, q in zip(lib.linear_cross_entropy_backward(broken, x, w, t, lse),
                    lib.linear_cross_entropy_backward(plain, x, w, t, lse)):
        assert torch.equal(p, q)


def test_row_weights_of_a_wide_range_in_fp16(lib, gpu):
    """Weights from 1 to 2^-30 in fp16: G's step of 2^-36 of the largest bounds every row, and the rows
    down to 2^-18 of it keep their digits.  For those: G's rounding and dx's (2^-11 each), and over a row
    of 500 entries of size 1.5 / 8 steps of at most 2^-37 each, beside a gradient of about 2^-18 times that
    size: 2^-9 of the row's norm in all."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(11)
    w = (torch.randn(500, 64, generator=g, device="cuda") * 1.5 / 8).half()
    x = torch.randn(124, 64, generator=g, device="cuda").half()
    t = torch.randint(0, 500, (124,), generator=g, device="cuda")
    dloss = torch.exp2(-0.25 * torch.arange(124, device="cuda").float())
    lse = lib.linear_cross_entropy(x, w, t)[1]
    # (a common factor that keeps the lightest rows above fp16's smallest step)
    dloss *= 1024.0
    got = lib.linear_cross_entropy_backward(dloss, x, w, t, lse)
    check_backward(got, x, w, t, dloss, lse, "f16")
    _, _, grad, _ = gradient(x, w, t, dloss, lse)
    ref, heavy = grad @ w.double(), dloss >= 1024.0 * 2.0 ** -18
    off = (got[0].double() - ref).norm(dim=1)
    assert heavy.sum() == 73 and (off[heavy] <= 2.0 ** -9 * ref.norm(dim=1)[heavy]).all()


def test_ignored_rows_and_zero_weights(lib, gpu):
    import torch
    x, w, t, dloss = make(4, "f16", 70, 200, 64)
    x[5] = float("nan")
    x[9] = float("inf")
    t[5] = t[9] = -100
    loss, lse = lib.linear_cross_entropy(x, w, t)
    assert loss[5] == 0 and loss[9] == 0
    dx, dw = lib.linear_cross_entropy_backward(dloss, x, w, t, lse)
    assert (dx[t == -100] == 0).all()
    everything = torch.full_like(t, -100)
    y = torch.nan_to_num(x, 0, 0, 0)
    loss, lse = lib.linear_cross_entropy(y, w, everything)
    assert (loss == 0).all() and torch.isfinite(lse).all()
    for g in lib.linear_cross_entropy_backward(dloss, y, w, everything, lse):
        assert (g == 0).all()
    for g in lib.linear_cross_entropy_backward(torch.zeros_like(dloss), y, w, t, lse):
        assert (g == 0).all()
    other = lib.linear_cross_entropy(y, w, torch.where(t == -100, 7, t), ignore_index=7)
    assert (other[0][t == -100] == 0).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,v,d", [(1, 30, 64), (70, 200, 64), (70, 200, 72), (300, 9001, 8), (2050, 515, 128),
                                   (4100, 9001, 64)])
def test_ignored_rows_leave_no_trace_in_the_gradients(lib, gpu, dtype, m, v, d):
    """Whatever an ignored row's input holds, dx of all rows and dw are what they are with zeros there."""
    import torch
    x, w, t, dloss = make(m + v + d, dtype, m, v, d, ignore=0.2)
    t[m // 2] = -100
    rows = (t == -100).nonzero()[:, 0]
    clean = x.clone()
    clean[rows] = 0
    lse = lib.linear_cross_entropy(clean, w, t)[1]
    ref = lib.linear_cross_entropy_backward(dloss, clean, w, t, lse)
    for i, value in enumerate((float("nan"), float("inf"), float("-inf"))):
        x[rows[i::3], i % d] = value
    x[rows[0]] = float("nan")
    loss, lse = lib.linear_cross_entropy(x, w, t)
    assert (loss[rows] == 0).all()
    got = lib.linear_cross_entropy_backward(dloss, x, w, t, lse)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    wide = torch.full((m, d + 24), float("nan"), device="cuda", dtype=x.dtype)
    wide[:, 8:d + 8] = x
    got = lib.linear_cross_entropy_backward(dloss, wide[:, 8:d + 8], w, t, lse)
    assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])


def test_targets_outside_the_vocabulary_and_non_finite_rows(lib, gpu):
    import torch
    x, w, t, dloss = make(5, "f16", 130, 300, 64, ignore=0.0)
    bad = torch.zeros(130, dtype=torch.bool, device="cuda")
    for i, v in ((0, 300), (64, -1), (129, 2 ** 40)):
        t[i] = v
        bad[i] = True
    x[7, 3] = float("inf")
    bad[7] = True
    loss, lse = lib.linear_cross_entropy(x, w, t)
    assert torch.isnan(loss[bad]).all() and torch.isfinite(loss[~bad]).all()
    dx, dw = lib.linear_cross_entropy_backward(dloss, x, w, t, lse)
    assert torch.isnan(dx[bad]).any(1).all() and torch.isfinite(dx[~bad]).all()


def test_no_rows(lib, gpu):
    import torch
    x, w, t, dloss = make(6, "f16", 0, 50, 24)
    loss, lse = lib.linear_cross_entropy(x, w, t)
    assert loss.shape == (0,)
    dx, dw = lib.linear_cross_entropy_backward(dloss, x, w, t, lse)
    assert dx.shape == (0, 24) and (dw == 0).all()


def test_gradient_against_differences(lib, gpu):
    """Central differences of the 64-bit loss along random directions."""
    import torch
    x, w, t, dloss = make(7, "f16", 40, 90, 64)
    lse = lib.linear_cross_entropy(x, w, t)[1]
    grads = lib.linear_cross_entropy_backward(dloss, x, w, t, lse)

    def f(x, w):
        z = x @ w.t()
        keep = t != -100
        loss = torch.logsumexp(z, 1) - z.gather(1, t.clamp(min=0)[:, None])[:, 0]
        return (torch.where(keep, loss, 0.0) * dloss.double()).sum()
    g = torch.Generator(device="cuda").manual_seed(2)
    xd, wd = x.double(), w.double()
    h = 2.0 ** -12
    for k, grad in enumerate(grads):
        way = torch.randn(grad.shape, generator=g, device="cuda").double()
        args = [[xd, wd], [xd, wd]]
        args[0][k], args[1][k] = args[0][k] + h * way, args[1][k] - h * way
        diff = (f(*args[0]) - f(*args[1])) / (2 * h)
        # fp16 rounding of G and of the result (2 x 2^-11) of every entry, and the difference's h^2 term
        bound = 2.0 ** -9 * (grad.double() * way).abs().sum() + 1e-4
        assert (diff - (grad.double() * way).sum()).abs() <= bound


def test_repeatable_and_on_another_stream(lib, gpu):
    import torch
    x, w, t, dloss = make(8, "bf16", 700, 5000, 128)

    def call():
        loss, lse = lib.linear_cross_entropy(x, w, t)
        return (loss, lse, *lib.linear_cross_entropy_backward(dloss, x, w, t, lse))
    first = call()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        again = call()
    torch.cuda.current_stream().wait_stream(st)
    for p, q in zip(first, again):
        assert torch.equal(p, q)


def test_refusals(lib, gpu):
    import torch
    x, w, t, dloss = make(9, "f16", 10, 20, 64)
    with pytest.raises(TypeError):
        lib.linear_cross_entropy(x.float(), w.float(), t)
    with pytest.raises(TypeError):
        lib.linear_cross_entropy(x, w.bfloat16(), t)
    with pytest.raises(TypeError):
        lib.linear_cross_entropy(x, w, t.int())
    with pytest.raises(ValueError):
        lib.linear_cross_entropy(x, w[:, :32], t)
    with pytest.raises(ValueError):
        lib.linear_cross_entropy_backward(dloss[:9], x, w, t, dloss)
    with pytest.raises(lib.SsgError, match="workspace"):
        lib.linear_cross_entropy(x, w, t, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(lib.SsgError, match="aligned"):
        flat = torch.zeros(10 * 64 + 4, device="cuda").half()
        lib.linear_cross_entropy(flat[4:].view(10, 64), w, t)
