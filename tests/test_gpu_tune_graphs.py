"""Capture and replay of the calls that tune and serve pruned layers: a captured
step, replayed three times on new inputs with the eager step and a
synchronisation between the replays, gives the eager results bit for bit."""

import pytest

pytestmark = pytest.mark.gpu


def _steps(lib):
    import torch
    g = torch.Generator(device="cuda").manual_seed(0)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    m, k, n, r, a, v = 300, 256, 320, 16, 3, 700
    s = dict(x=rnd(m, k).half(), res=rnd(m, k).half(), w=rnd(k).half(), b=rnd(k).half(), dy=rnd(m, n).half(),
             base=rnd(m, n).half(), down=rnd(a, r, k).half() / 16, up=rnd(a, n, r).half() / 4,
             index=torch.randint(-1, a, (m,), generator=g, device="cuda").to(torch.int32),
             head=rnd(v, k).half() / 8, target=torch.randint(0, v, (m,), generator=g, device="cuda"), dloss=rnd(m))

    def step():
        y, mean, rstd, t = lib.layer_norm(s["x"], s["w"], s["b"], residual=s["res"])
        o = lib.low_rank_add(s["base"], y, s["down"], s["up"], s["index"])
        few = lib.low_rank_add(s["base"][:5], y[:5], s["down"], s["up"], s["index"][:5])
        dx, ddown, dup = lib.low_rank_backward(s["dy"], y, s["down"], s["up"], s["index"], base=s["res"])
        loss, lse = lib.linear_cross_entropy(y, s["head"], s["target"])
        dh, dw = lib.linear_cross_entropy_backward(s["dloss"], y, s["head"], s["target"], lse)
        dn = lib.layer_norm_backward(dh, t, mean, rstd, s["w"], dres=dx)
        return [y, t, o, few, dx, ddown, dup, loss, lse, dh, dw, *dn]
    return s, step


def test_captured_step_replays(lib, gpu):
    import torch
    s, step = _steps(lib)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        step()
    st.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        outs = step()
    for turn in range(3):
        for key in ("x", "dy", "dloss"):
            s[key].copy_(torch.randn_like(s[key]))
        want = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i, (p, q) in enumerate(zip(outs, want)):
            assert torch.equal(p, q), (turn, i)


def test_captured_adapters_beside_the_sparse_product(lib, gpu):
    import numpy as np
    import torch

    import workloads as wl
    w = wl.random_24_f16(np.random.default_rng(0), 1, 256, 320)["Wp"]
    vals, meta = lib.w24_pack_f16(w)
    vals, meta = torch.from_numpy(vals).cuda(), torch.from_numpy(meta.view(np.int32)).cuda()
    s, _ = _steps(lib)
    for m in (20, 300):
        x, index = s["x"][:m].contiguous(), s["index"][:m].contiguous()
        call = lambda: lib.w24_low_rank_gemm_f16(x, vals, meta, s["down"], s["up"], index)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            call()
        st.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            out = call()
        for _ in range(3):
            x.copy_(torch.randn_like(x))
            want = call()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, want)
