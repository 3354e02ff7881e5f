"""What the gradient norm and clipping promise beyond ordinary values: a norm past fp32, one norm from
both calls, long lists."""

import pytest

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.mark.parametrize("dt", ["float32", "bfloat16"])
@pytest.mark.parametrize("most", [1.0, 1e-6, 1e30, INF])
def test_a_norm_past_fp32(lib, gpu, dt, most):
    """The call that sums the squares clips by its 64-bit norm, also where norm[0] is infinite; an infinite
    norm that is given makes the factor 0.  Roundings: the product to fp32, then to the type."""
    import torch
    t = torch.full((5000,), 3e38).to(getattr(torch, dt))
    small = torch.tensor([1.0, -2.0]).to(t.dtype)
    want = float(t[0].double()) * 5000 ** 0.5
    by = min(1.0, most / (want + 1e-6))
    g = [t.cuda(), small.cuda()]
    norm, outs = lib.clip_grad_norm(g, most)
    told = lib.grad_norm(g)
    assert norm.item() == INF and told.item() == INF
    fi = torch.finfo(t.dtype)
    for a, have in zip((t, small), outs):
        exact = a.double() * by
        bound = exact.abs() * ((fi.eps / 2 if dt == "bfloat16" else 0) + 2.0 ** -23 + 1e-11)
        bound = bound + fi.smallest_normal * fi.eps
        assert bool(((have.cpu().double() - exact).abs() <= bound).all())
    for have in lib.clip_grad_norm(g, most, norm=told)[1]:
        assert not bool(have.any()) and not bool(have.isnan().any())
    g[0][17] = INF  # (infinite times zero)
    norm, (a, b) = lib.clip_grad_norm(g, most)
    assert norm.item() == INF and a.isnan().nonzero().flatten().tolist() == [17]
    assert not bool(a.nan_to_num().any()) and not bool(b.any())


@pytest.mark.parametrize("top,most", [(3e38, 1.0), (3e38, 1e-3), (1e38, 1e-6), (1e30, 1e-12)])
def test_factors_below_the_normal_fp32_values(lib, gpu, top, most):
    """The factor keeps its digits below 2^-126: roundings of the factor (2^-24 where fp32 holds it) and of the
    product (2^-24, or half of the smallest value)."""
    import torch
    t = torch.tensor([top, -top / 4, 1.0])
    want = float(t.double().norm())
    assert want < 3.4e38
    norm, (out,) = lib.clip_grad_norm([t.cuda()], most)
    by = most / (want + 1e-6)
    bound = t.double().abs() * by * (2.0 ** -23 + 1e-11) + 2.0 ** -150
    assert abs(norm.item() - want) <= 2.0 ** -24 * want * (1 + 1e-9)
    assert bool(((out.cpu().double() - t.double() * by).abs() <= bound).all())


def test_both_calls_add_in_one_order(lib, gpu):
    """Squares whose sum lies half way between two norms, and a few that are lost or not, as the order has it."""
    import torch
    g = torch.zeros(1024, 4096, device="cuda")  # a piece a row, a partial sum each
    g[0, :4] = torch.tensor([2.0 ** 24, 4096.0, 4096.0, 1.0])  # (2^24 + 1)^2
    for row in (256, 512, 768):
        g[row, 0] = g[row + 32, 0] = 0.1677  # (its square: 0.45 of the sum's last place)
    norm = lib.grad_norm([g])
    told, _ = lib.clip_grad_norm([g], 1.0)
    assert torch.equal(norm, told), (norm.item(), told.item())


def _replayed_us(f):
    """Least time of a captured call (without the host's part)."""
    import torch
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        f()
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        f()
    best = INF
    for _ in range(5):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        graph.replay()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b) * 1e3)
    return best


def test_long_lists_take_no_longer_than_their_norm_and_their_scaling(lib, gpu):
    """Experts kept as separate matrices: 12000 tensors of 100 KB, 64512 partial sums."""
    import torch
    flat = torch.randn(12000, 51200, device="cuda", dtype=torch.bfloat16)
    g, out = list(flat), list(torch.empty_like(flat))
    norm = lib.grad_norm(g)
    want = sum(part.double().square().sum().item() for part in flat.split(1000)) ** 0.5
    assert abs(norm.item() - want) <= 2.0 ** -24 * want * (1 + 1e-9)
    told, _ = lib.clip_grad_norm(g, 1.0, out=out)
    assert torch.equal(told, norm)
    by = 1.0 / (want + 1e-6)
    for i in (0, 189, 190, 5999, 11999):  # (half a step of the product's rounding to 16 bits, and fp32's two)
        exact = flat[i].double() * by
        assert bool(((out[i].double() - exact).abs() <= exact.abs() * (2.0 ** -8 + 2.0 ** -22)).all())
    apart = _replayed_us(lambda: lib.grad_norm(g)) + _replayed_us(lambda: lib.clip_grad_norm(g, 1.0, norm=norm, out=out))
    both = _replayed_us(lambda: lib.clip_grad_norm(g, 1.0, out=out))
    assert both <= 1.5 * apart, (both, apart)
