"""What the gradient norm and clipping promise beyond ordinary values: one norm from both calls, long lists."""

import pytest

pytestmark = pytest.mark.gpu

INF = float("inf")


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
