"""The adapter-tuning example end to end: the loss falls, a step's gradients match
torch's own on the same block in fp32, and a served token does not depend on the
requests beside it."""

import importlib.util
import math
import os

import pytest

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "tune_adapters.py")


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("tune_adapters", PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_the_loss_falls(gpu, example):
    losses, _ = example.tune(steps=40, verbose=False)
    assert all(math.isfinite(v) for v in losses)
    assert losses[-1] < 0.7 * losses[0], (losses[0], losses[-1])


def test_served_tokens_do_not_depend_on_their_neighbours(gpu, example):
    import torch
    _, block = example.tune(steps=2, verbose=False)
    z, t, index = example.serve(block, requests=32)
    for i in (0, 7, 31):
        alone = block.forward(t[i:i + 1].contiguous(), index[i:i + 1].contiguous())[0]
        assert torch.equal(alone[0], z[i])


def test_gradients_match_autograd(gpu, example):
    """Relative to each gradient's norm: fp16 activations and gradients on the way (2^-11 each, a
    dozen of them) against fp32 throughout."""
    import torch
    g = torch.Generator().manual_seed(3)
    weights = example.sparse_weight(g, example.D, example.F), example.sparse_weight(g, example.F, example.D)
    block = example.Block(g, weights, 0.5)
    t = torch.randn(200, example.D, generator=g).half().cuda()
    index = torch.randint(-1, example.ADAPTERS, (200,), generator=g).to(torch.int32).cuda()
    dz = torch.randn(200, example.D, generator=g).half().cuda()
    z, saved = block.forward(t, index)
    grads = block.backward(dz, saved, index)

    p = [q.detach().clone().half().float().requires_grad_() if i < 4 else q.detach().clone().requires_grad_()
         for i, q in enumerate(block.parameters())]
    one = (index[:, None] == torch.arange(example.ADAPTERS, device="cuda")).float() * 2.0

    def project(x, w, down, up):
        low = torch.matmul(x, down.reshape(-1, x.shape[1]).t()).view(len(x), example.ADAPTERS, -1) * one[:, :, None]
        return x @ w.float() + torch.matmul(low.flatten(1), up.transpose(1, 2).reshape(-1, up.shape[1]))
    x = t.float()
    y = torch.nn.functional.layer_norm(x, (example.D,), p[4], p[5])
    o = project(torch.nn.functional.gelu(project(y, weights[0][2], p[0], p[1])), weights[1][2], p[2], p[3])
    out = torch.nn.functional.layer_norm(x + o, (example.D,), p[6], p[7])
    assert (z.float() - out).norm() <= 12 * 2.0 ** -11 * out.norm()
    out.backward(dz.float())
    for have, want in zip(grads, p):
        assert (have.float() - want.grad).norm() <= 12 * 2.0 ** -11 * want.grad.norm()
