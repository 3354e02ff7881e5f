"""Tune low-rank adapters and norms of a pruned feed-forward block, then serve them.

A 2:4 weight is packed once and stays as it is.  What is tuned sits beside it:
two requests' (or tasks') adapters next to both projections, and the norms.  One
training step, all on the library's kernels except the elementwise activation
and the update:

    t  -> layer_norm -> y -> fc1 (2:4 + adapters) -> gelu -> fc2 (2:4 + adapters) -> o
    s = t + o -> layer_norm -> z -> cross entropy against the vocabulary `head`

and back.  The targets come from a teacher whose adapters differ, so the loss has
somewhere to go.  Afterwards every adapter serves single tokens of many requests.

    python examples/tune_adapters.py [--steps 60]
"""

import argparse
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import structured_sparse_gemm_w24_amd as ssg  # noqa: E402
import workloads as wl  # noqa: E402

D, F, V, RANK, ADAPTERS = 256, 1024, 2000, 16, 2


def sparse_weight(g, k, n):
    """A 2:4 weight: packed for the forward product, and dense [k, n] for the input gradient."""
    w = torch.randn(k, n, generator=g) / math.sqrt(k / 2)
    w = w.half().numpy()
    w = wl.prune24_magnitude(w)
    vals, meta = ssg.w24_pack_f16(w)
    return torch.from_numpy(vals).cuda(), torch.from_numpy(meta.view("int32")).cuda(), torch.from_numpy(w).cuda()


class Adapters:
    """A pool of adapters next to a k x n projection: fp32 parameters, fp16 copies for the kernels."""

    def __init__(self, g, k, n, spread):
        self.scale = torch.full((ADAPTERS,), 2.0, device="cuda")
        self.down = (torch.randn(ADAPTERS, RANK, k, generator=g) / math.sqrt(k)).cuda()
        self.up = (torch.randn(ADAPTERS, n, RANK, generator=g) * spread / math.sqrt(RANK)).cuda()

    def half(self):
        return self.down.half(), self.up.half()


class Block:
    def __init__(self, g, weights, spread):
        self.w1, self.w2 = weights
        self.a1, self.a2 = Adapters(g, D, F, spread), Adapters(g, F, D, spread)
        self.norms = [torch.ones(D, device="cuda"), torch.zeros(D, device="cuda"),
                      torch.ones(D, device="cuda"), torch.zeros(D, device="cuda")]

    def forward(self, t, index):
        n1w, n1b, n2w, n2b = self.norms
        y, mean1, rstd1 = ssg.layer_norm(t, n1w, n1b)
        h = ssg.w24_low_rank_gemm_f16(y, *self.w1[:2], *self.a1.half(), index, self.a1.scale)
        a = torch.nn.functional.gelu(h)
        o = ssg.w24_low_rank_gemm_f16(a, *self.w2[:2], *self.a2.half(), index, self.a2.scale)
        z, mean2, rstd2, s = ssg.layer_norm(o, n2w, n2b, residual=t)
        return z, (t, y, mean1, rstd1, h, a, s, mean2, rstd2)

    def backward(self, dz, saved, index):
        """Gradients of the parameters, in the order of parameters()."""
        t, y, mean1, rstd1, h, a, s, mean2, rstd2 = saved
        n1w, _, n2w, _ = self.norms
        ds, dn2w, dn2b = ssg.layer_norm_backward(dz, s, mean2, rstd2, n2w)
        da = ssg.dense_gemm_f16(ds, self.w2[2])  # the shared weight's part: ds . W2^T
        da, ddown2, dup2 = ssg.low_rank_backward(ds, a, *self.a2.half(), index, self.a2.scale, base=da)
        hf = h.float()
        cdf = 0.5 * (1 + torch.erf(hf / math.sqrt(2)))
        dh = (da.float() * (cdf + hf * torch.exp(-0.5 * hf * hf) / math.sqrt(2 * math.pi))).half()
        dy = ssg.dense_gemm_f16(dh, self.w1[2])
        dy, ddown1, dup1 = ssg.low_rank_backward(dh, y, *self.a1.half(), index, self.a1.scale, base=dy)
        _, dn1w, dn1b = ssg.layer_norm_backward(dy, t, mean1, rstd1, n1w, dres=ds)
        return [ddown1, dup1, ddown2, dup2, dn1w, dn1b, dn2w, dn2b]

    def parameters(self):
        return [self.a1.down, self.a1.up, self.a2.down, self.a2.up, *self.norms]


def tune(steps=60, tokens=512, seed=0, lr=3e-3, loss_scale=1024.0, verbose=True):
    """Returns the mean loss of every step, and the tuned block."""
    g = torch.Generator().manual_seed(seed)
    weights = sparse_weight(g, D, F), sparse_weight(g, F, D)
    teacher, block = Block(g, weights, 1.5), Block(g, weights, 0.1)
    head = (torch.randn(V, D, generator=g) * 4 / math.sqrt(D)).half().cuda()
    t = torch.randn(tokens, D, generator=g).half().cuda()
    # ragged requests: a first task, tokens without an adapter, a second task
    index = torch.zeros(tokens, dtype=torch.int32)
    index[tokens // 2:] = 1
    index[tokens // 2 - 20:tokens // 2 + 17] = -1
    index = index.cuda()
    target = (teacher.forward(t, index)[0].float() @ head.float().t()).argmax(1)
    target[::11] = -100  # not every token counts
    rows = int((target != -100).sum())
    dloss = torch.full((tokens,), loss_scale / rows, device="cuda")
    moments = [(torch.zeros_like(p), torch.zeros_like(p)) for p in block.parameters()]
    losses = []
    for step in range(1, steps + 1):
        z, saved = block.forward(t, index)
        loss, lse = ssg.linear_cross_entropy(z, head, target)
        dz, _ = ssg.linear_cross_entropy_backward(dloss, z, head, target, lse)
        for p, grad, (m1, m2) in zip(block.parameters(), block.backward(dz, saved, index), moments):
            grad = grad.float() / loss_scale
            m1.mul_(0.9).add_(grad, alpha=0.1)
            m2.mul_(0.99).addcmul_(grad, grad, value=0.01)
            p.sub_(lr * (m1 / (1 - 0.9 ** step)) / ((m2 / (1 - 0.99 ** step)).sqrt() + 1e-8))
        losses.append(loss.sum().item() / rows)
        if verbose and (step == 1 or step % 10 == 0):
            print(f"step {step:4d}  loss {losses[-1]:.4f}", flush=True)
    return losses, block


def serve(block, requests=32, seed=1):
    """One decode step: a single token each of many requests, mixed adapters."""
    g = torch.Generator().manual_seed(seed)
    t = torch.randn(requests, D, generator=g).half().cuda()
    index = torch.randint(-1, ADAPTERS, (requests,), generator=g).to(torch.int32).cuda()
    return block.forward(t, index)[0], t, index


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--tokens", type=int, default=512)
    a = ap.parse_args()
    losses, block = tune(a.steps, a.tokens)
    z, t, index = serve(block)
    print(f"loss {losses[0]:.4f} -> {losses[-1]:.4f}; served {len(index)} tokens, "
          f"{int((index >= 0).sum())} with an adapter, finite: {bool(torch.isfinite(z).all())}")


if __name__ == "__main__":
    main()
