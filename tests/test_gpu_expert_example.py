"""The expert-layer example end to end: it trains, its gradients match torch's own on
the same layer in fp32, and its 4-bit answers are the dequantised layer's."""

import importlib.util
import math
import os

import pytest

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "expert_layer.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("expert_layer", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_it_trains(gpu, example):
    losses, norms, _, _ = example.train(steps=5, tokens=300, verbose=False)
    assert all(math.isfinite(v) for v in losses + norms) and all(v > 0 for v in norms)


def test_gradients_match_autograd(gpu, example):
    """Relative to each gradient's norm: fp16 activations, weights and gradients on the way (half a
    step, 2^-11, each, fewer than a dozen of them) against fp32 throughout."""
    import torch
    g = torch.Generator().manual_seed(3)
    layer = example.Layer(g)
    t = torch.randn(333, example.D, generator=g).half().cuda()
    router = torch.randn(example.D, example.EXPERTS, generator=g).cuda()
    dout = torch.randn(333, example.D, generator=g).half().cuda()
    routes = example.route(t, router)
    out, saved = layer.forward(t, routes)
    grads = layer.backward(dout, saved, routes)
    w1, w2 = (p.half().float().requires_grad_() for p in layer.parameters())
    token, gate, offsets = routes
    o = offsets.tolist()
    rows = []
    for e in range(example.EXPERTS):
        x = t[token[o[e]:o[e + 1]]].float()
        rows.append(torch.nn.functional.gelu(x @ w1[e].t()) @ w2[e].t())
    want = example.combine(torch.cat(rows), token, gate, len(t))
    assert (out - want).norm() <= 12 * 2.0 ** -11 * want.norm()
    want.backward(dout.float())
    for have, w in zip(grads, (w1, w2)):
        assert (have.float() - w.grad).norm() <= 12 * 2.0 ** -11 * w.grad.norm()


def test_served_tokens(gpu, lib, example):
    import torch
    _, _, layer, router = example.train(steps=2, tokens=300, verbose=False)
    packed = layer.packed()
    t = torch.randn(40, example.D, generator=torch.Generator().manual_seed(1)).half().cuda()
    served = example.serve(packed, t, router)
    for i in (0, 17, 39):  # no token depends on the others
        assert torch.equal(example.serve(packed, t[i:i + 1].contiguous(), router)[0], served[i])
    # the same layer from dequantised operands, in fp32
    e = example.EXPERTS
    w1 = lib.mxfp4_dequantize(packed[0][0].flatten(0, 1), packed[0][1].flatten(0, 1), example.D).view(e, example.F, -1)
    w2 = lib.mxfp4_dequantize(packed[1][0].flatten(0, 1), packed[1][1].flatten(0, 1), example.F).view(e, example.D, -1)
    values = lambda x: lib.mxfp4_dequantize(*lib.mxfp4_quantize(x), x.shape[1])
    token, gate, offsets = example.route(t, router)
    x, o = values(t[token]), offsets.tolist()
    h = torch.cat([x[o[i]:o[i + 1]] @ w1[i].t() for i in range(e)]).half()
    a = values(torch.nn.functional.gelu(h))
    y = torch.cat([a[o[i]:o[i + 1]] @ w2[i].t() for i in range(e)]).half()
    want = example.combine(y, token, gate, len(t))
    # a value of h that rounds to the other 16-bit neighbour may move its 4-bit code by a step: half
    # a step in 2^-11 of the values, and no more than a quarter of the value each
    assert (served - want).norm() <= 0.01 * want.norm()
