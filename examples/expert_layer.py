"""Train a layer of experts in 16 bits, then serve it with 4-bit weights.

Every token goes to the two experts that a fixed router likes best.  The chosen
(token, expert) pairs are sorted by expert, which makes one ragged batch of rows:

    x = t[row's token] -> grouped_gemm w1 -> gelu -> grouped_gemm w2 -> sum over a token's rows, gated

and back, with the gradients of both products, clipped together.  The targets come
from a teacher layer with other experts.  Afterwards both weights are packed to
microscaled 4-bit rows once and the layer answers single tokens.

    python examples/expert_layer.py [--steps 40]
"""

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import structured_sparse_gemm_w24_amd as ssg  # noqa: E402

D, F, EXPERTS, CHOICES = 256, 512, 8, 2


def route(t, router):
    """Rows sorted by expert: (token of every row, its gate, offsets int32 [EXPERTS + 1])."""
    score, expert = (t.float() @ router).topk(CHOICES, dim=1)
    gate = score.softmax(1).flatten()
    by_expert = expert.flatten().argsort(stable=True)
    counts = (expert.flatten()[:, None] == torch.arange(EXPERTS, device=t.device)).sum(0)
    offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    return by_expert // CHOICES, gate[by_expert], offsets


def combine(rows, token, gate, n):
    """out[token of row] += gate * row, fp32; a token's rows are added in a fixed order."""
    order = token.argsort(stable=True)
    return (rows.float() * gate[:, None])[order].view(n, CHOICES, -1).sum(1)


class Layer:
    """fp32 parameters, fp16 copies for the kernels."""

    def __init__(self, g):
        self.w1 = (torch.randn(EXPERTS, F, D, generator=g) / math.sqrt(D)).cuda()
        self.w2 = (torch.randn(EXPERTS, D, F, generator=g) / math.sqrt(F)).cuda()

    def parameters(self):
        return [self.w1, self.w2]

    def forward(self, t, routes):
        token, gate, offsets = routes
        x = t[token]
        h = ssg.grouped_gemm(x, self.w1.half(), offsets)
        a = torch.nn.functional.gelu(h)
        y = ssg.grouped_gemm(a, self.w2.half(), offsets)
        return combine(y, token, gate, len(t)), (x, h, a)

    def backward(self, dout, saved, routes):
        """Gradients of w1 and w2 (the router is fixed)."""
        token, gate, offsets = routes
        x, h, a = saved
        dy = (dout[token].float() * gate[:, None]).half()
        da, dw2 = ssg.grouped_gemm_backward(dy, a, self.w2.half(), offsets)
        hf = h.float()
        cdf = 0.5 * (1 + torch.erf(hf / math.sqrt(2)))
        dh = (da.float() * (cdf + hf * torch.exp(-0.5 * hf * hf) / math.sqrt(2 * math.pi))).half()
        _, dw1 = ssg.grouped_gemm_backward(dh, x, self.w1.half(), offsets, x_grad=False)
        return [dw1, dw2]

    def packed(self):
        """Both weights as microscaled 4-bit rows."""
        out = []
        for w in self.parameters():
            e, n, k = w.shape
            codes, scales = ssg.mxfp4_quantize(w.view(e * n, k))
            out.append((codes.view(e, n, -1), scales.view(e, n, -1)))
        return out


def serve(packed, t, router):
    """The layer's answer with 4-bit weights."""
    token, gate, offsets = route(t, router)
    h = ssg.mxfp4_grouped_linear(t[token], *packed[0], offsets)
    y = ssg.mxfp4_grouped_linear(torch.nn.functional.gelu(h), *packed[1], offsets)
    return combine(y, token, gate, len(t))


def train(steps=40, tokens=1024, seed=0, lr=2e-3, scale=1024.0, verbose=True):
    """Returns the mean squared error of every step, the gradient norms, the layer and its router."""
    g = torch.Generator().manual_seed(seed)
    teacher, layer = Layer(g), Layer(g)
    router = torch.randn(D, EXPERTS, generator=g).cuda()
    t = torch.randn(tokens, D, generator=g).half().cuda()
    routes = route(t, router)
    target = teacher.forward(t, routes)[0]
    moments = [(torch.zeros_like(p), torch.zeros_like(p)) for p in layer.parameters()]
    losses, norms = [], []
    for step in range(1, steps + 1):
        out, saved = layer.forward(t, routes)
        miss = out - target
        dout = (miss * (2.0 * scale / miss.numel())).half()
        grads = layer.backward(dout, saved, routes)
        norm, grads = ssg.clip_grad_norm(grads, 0.05 * scale, out=grads)
        for p, grad, (m1, m2) in zip(layer.parameters(), grads, moments):
            grad = grad.float() / scale
            m1.mul_(0.9).add_(grad, alpha=0.1)
            m2.mul_(0.99).addcmul_(grad, grad, value=0.01)
            p.sub_(lr * (m1 / (1 - 0.9 ** step)) / ((m2 / (1 - 0.99 ** step)).sqrt() + 1e-8))
        losses.append(float((miss * miss).mean()))
        norms.append(float(norm) / scale)
        if verbose and (step == 1 or step % 10 == 0):
            print(f"step {step:4d}  loss {losses[-1]:.4f}  gradient norm {norms[-1]:.4f}", flush=True)
    return losses, norms, layer, router


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=40)
    ap.add_argument("--tokens", type=int, default=1024)
    a = ap.parse_args()
    losses, _, layer, router = train(a.steps, a.tokens)
    t = torch.randn(16, D, generator=torch.Generator().manual_seed(1)).half().cuda()
    full = layer.forward(t, route(t, router))[0]
    served = serve(layer.packed(), t, router)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f}; 4-bit answers to {len(t)} tokens differ from the 16-bit ones by "
          f"{float((served - full).norm() / full.norm()):.3f} of their norm")


if __name__ == "__main__":
    main()
