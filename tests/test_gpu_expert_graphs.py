"""Capture and replay of the expert calls: a captured step, replayed on new inputs and
new group boundaries with the eager step and synchronisations between the replays, gives
the eager results bit for bit; two graphs and two streams at once do not disturb each other."""

import pytest

pytestmark = pytest.mark.gpu


def _offsets(m, e, seed):
    import torch
    g = torch.Generator().manual_seed(seed)
    cuts = torch.randint(0, m + 1, (e - 1,), generator=g).sort().values
    return torch.cat([torch.zeros(1, dtype=torch.int64), cuts, torch.tensor([m])]).to(torch.int32)


def _step(lib, seed, m=500, n=160, k=264, e=5):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    s = dict(x=rnd(m, k).half(), dy=rnd(m, n).half(), w=rnd(e, n, k).half() / 16, offsets=_offsets(m, e, seed).cuda(),
             out=torch.zeros(m, n, device="cuda", dtype=torch.float16),
             dx=torch.zeros(m, k, device="cuda", dtype=torch.float16),
             yq=torch.zeros(m, n, device="cuda", dtype=torch.float16), long=rnd(6000, 64).half(),
             one=torch.tensor([0, 6000], dtype=torch.int32).cuda())
    codes, scales = lib.mxfp4_quantize(s["w"].view(e * n, k))
    codes, scales = codes.view(e, n, -1), scales.view(e, n, -1)

    def step():
        y = lib.grouped_gemm(s["x"], s["w"], s["offsets"], out=s["out"])
        dx, dw = lib.grouped_gemm_backward(s["dy"], s["x"], s["w"], s["offsets"], out=s["dx"])
        _, dw1 = lib.grouped_gemm_backward(s["long"], s["long"], s["w"][:1, :64, :64].contiguous(), s["one"],
                                           x_grad=False)  # (split sums)
        norm, clipped = lib.clip_grad_norm([dw, dw1], 1.0)
        q, qs = lib.mxfp4_quantize(s["x"])
        back = lib.mxfp4_dequantize(q, qs, k)
        yq = lib.mxfp4_grouped_linear(s["x"], codes, scales, s["offsets"], out=s["yq"])
        y1 = lib.mxfp4_linear(s["x"][:7], codes[0], scales[0])
        return [y, dx, dw, dw1, norm, *clipped, q, qs, back, yq, y1]
    return s, step


def _capture(step):
    import torch
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step()
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        outs = step()
    return graph, outs


def test_captured_step_replays(lib, gpu):
    import torch
    s, step = _step(lib, 0)
    graph, outs = _capture(step)
    for turn in range(4):
        for key in ("x", "dy", "long"):
            s[key].copy_(torch.randn_like(s[key]))
        s["offsets"].copy_(_offsets(500, 5, 10 + turn))
        want = [t.clone() for t in step()]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i, (p, q) in enumerate(zip(outs, want)):
            assert torch.equal(p, q), (turn, i)


def test_two_graphs_and_two_streams(lib, gpu):
    import torch
    sides = [_step(lib, seed, m=m, n=n) for seed, m, n in ((1, 700, 136), (2, 300, 264))]
    want = [[t.clone() for t in step()] for _, step in sides]
    graphs = [_capture(step) for _, step in sides]
    streams = [torch.cuda.Stream() for _ in sides]
    torch.cuda.synchronize()
    for turn in range(3):
        for (graph, _), st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
        torch.cuda.synchronize()
        for (_, outs), w in zip(graphs, want):
            assert all(torch.equal(a, b) for a, b in zip(outs, w)), turn
        eager = []
        for (_, step), st in zip(sides, streams):
            with torch.cuda.stream(st):
                eager.append([t.clone() for t in step()])
        torch.cuda.synchronize()
        for e, w in zip(eager, want):
            assert all(torch.equal(a, b) for a, b in zip(e, w)), turn
