"""Measured cases of the adapter-tuning operators: layer norm, low-rank adapters
beside a shared projection, and the cross entropy of a linear head.

Every case is one call a user makes while serving or tuning low-rank adapters on
a pruned transformer: the norm in front of a projection (forward, and backward
with the weight's gradient), the 2:4 projection with the adapters of many
requests beside it (single tokens, long ragged batches, and the gradients), and
the loss over the vocabulary with its gradient.

``run`` computes the plain form (elementary torch operations in 32 bits) unless
``own`` is true; then it calls the library.
"""

import math

import torch

own = False

EPS = 1e-5
IGNORE = -100
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one token of a decode step: the norm after the residual sum
        dict(name="norm_fwd_token", op="norm_fwd", dtype="f16", m=1, n=1024, res=True),
        # a ViT-Base batch (64 images of 197 tokens): residual sum and norm
        dict(name="norm_fwd_batch", op="norm_fwd", dtype="f16", m=12608, n=768, res=True),
        # the same norm's backward pass, with the residual branch's gradient
        dict(name="norm_bwd_batch", op="norm_bwd", dtype="f16", m=12608, n=768, res=True),
        # an odd width and row count in bf16, no residual branch
        dict(name="norm_bwd_odd", op="norm_bwd", dtype="bf16", m=4099, n=1537, res=False),
        # a decode step: 32 requests of one token, 24 adapters of up to rank 16
        dict(name="adapter_decode", op="adapter_w24", dtype="f16", m=32, k=1024, n=4096, rank=16, adapters=24,
             requests=32, ranks=True),
        # one 2:4 fc1 layer over ragged prompts of many requests, ranks up to 64
        dict(name="adapter_prefill", op="adapter_w24", dtype="f16", m=4096, k=1024, n=4096, rank=64, adapters=12,
             requests=17, ranks=True),
        # adapters added to another projection's output (bf16, an odd token count and width)
        dict(name="adapter_add_ragged", op="adapter_add", dtype="bf16", m=1531, k=768, n=2312, rank=32, adapters=8,
             requests=9, ranks=False),
        # tuning: gradients of four adapters of a projection, ViT-Large's fc1 width
        dict(name="adapter_bwd_batch", op="adapter_bwd", dtype="f16", m=6144, k=1024, n=4096, rank=16, adapters=4,
             requests=8, ranks=False),
        # tuning one bf16 adapter on a short, odd batch
        dict(name="adapter_bwd_small", op="adapter_bwd", dtype="bf16", m=333, k=768, n=768, rank=8, adapters=1,
             requests=1, ranks=False),
        # a classification head: one batch of images against 1000 classes
        dict(name="loss_fwd_classes", op="loss_fwd", dtype="f16", m=64, d=768, v=1000),
        # a language model's loss over a large vocabulary
        dict(name="loss_fwd_vocab", op="loss_fwd", dtype="f16", m=8192, d=1024, v=32000),
        # its gradient to the hidden states and the head's weight; an odd vocabulary
        dict(name="loss_bwd_vocab", op="loss_bwd", dtype="bf16", m=6144, d=1024, v=30001),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["norm_fwd", "norm_bwd", "adapter_w24", "adapter_add", "adapter_bwd", "loss_fwd", "loss_bwd"])
        if op.startswith("norm"):
            c = dict(op=op, dtype=rng.choice(["f16", "bf16", "f32"]), m=_log_int(rng, 1, 16000),
                     n=_log_int(rng, 64, 8192), res=rng.random() < 0.5)
        elif op.startswith("adapter"):
            n_req = _log_int(rng, 1, 64)
            c = dict(op=op, dtype=rng.choice(["f16", "bf16"]), m=_log_int(rng, n_req, 8192),
                     k=8 * _log_int(rng, 16, 512), n=8 * _log_int(rng, 16, 512), rank=8 * _log_int(rng, 1, 8),
                     adapters=_log_int(rng, 1, 32), requests=n_req, ranks=rng.random() < 0.5)
            if op == "adapter_w24":  # what the 2:4 product takes
                c.update(dtype="f16", k=64 * _log_int(rng, 4, 64), n=64 * _log_int(rng, 4, 64))
        else:
            c = dict(op=op, dtype=rng.choice(["f16", "bf16"]), m=_log_int(rng, 1, 8192), d=_log_int(rng, 64, 2048),
                     v=_log_int(rng, 100, 60000))
        if _cost(c) <= most:
            return c


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / 50)


def work(case):
    """Bytes with every input read and every output written once, and the multiply-adds of the products."""
    e = 4 if case.get("dtype") == "f32" else 2
    op, m = case["op"], case["m"]
    if op == "norm_fwd":
        n = case["n"]
        return {"bytes": m * n * e * (4 if case["res"] else 2) + 8 * m + 8 * n, "flops": 8 * m * n}
    if op == "norm_bwd":
        n = case["n"]
        return {"bytes": m * n * e * (4 if case["res"] else 3) + 8 * m + 12 * n, "flops": 12 * m * n}
    if op.startswith("adapter"):
        k, n, r = case["k"], case["n"], case["rank"]
        used = min(case["adapters"], case["requests"])  # adapters that a batch can touch
        pool = used * r * (k + n) * 2
        low = 2 * m * r * (k + n)
        if op == "adapter_w24":  # kept values, 2-bit positions, and the half of the products that is kept
            return {"bytes": 2 * m * (k + n) + n * k + n * k // 8 + pool + 4 * m, "flops": m * k * n + low}
        if op == "adapter_add":
            return {"bytes": 2 * m * (k + 2 * n) + pool + 4 * m, "flops": low}
        return {"bytes": 2 * m * (3 * k + n) + 2 * pool + 4 * m, "flops": 3 * low - 2 * m * r * n}
    d, v = case["d"], case["v"]
    if op == "loss_fwd":
        return {"bytes": 2 * (m * d + v * d) + 16 * m, "flops": 2 * m * v * d}
    return {"bytes": 4 * (m * d + v * d) + 20 * m, "flops": 6 * m * v * d}


# ----------------------------------------------------------------- the inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, std=1.0, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda").mul_(std).to(dtype)


def _pack24(g, k, n):
    """A random 2:4 weight in the library's compressed layout: kept values [n, k/2] and the
    2-bit positions of the kept values, 16 to a word [n, k/32]."""
    first = torch.randint(0, 3, (n, k // 4), generator=g, device="cuda")
    more = (torch.rand(n, k // 4, generator=g, device="cuda") * (3 - first)).long()
    second = torch.clamp(first + 1 + more, max=3)
    pos = torch.stack([first, second], -1).reshape(n, k // 32, 16)
    word = (pos << (2 * torch.arange(16, device="cuda"))).sum(-1)
    meta = torch.where(word >= 2 ** 31, word - 2 ** 32, word).to(torch.int32)
    return _randn(g, n, k // 2, std=1 / math.sqrt(k / 2), dtype=torch.float16), meta


def _requests(g, m, requests, adapters):
    """Adapter of every token: `requests` runs of ragged length, one in eight without an adapter."""
    cuts = torch.randperm(max(m - 1, 1), generator=g, device="cuda")[: max(requests - 1, 0)].sort().values + 1
    run_of = torch.bucketize(torch.arange(m, device="cuda"), cuts, right=True)
    one = torch.randint(0, adapters, (requests + 1,), generator=g, device="cuda")
    if requests > 1:
        one = torch.where(torch.rand(requests + 1, generator=g, device="cuda") < 0.125, torch.full_like(one, -1), one)
    return one[run_of].to(torch.int32)


def prepare(case, seed):
    g, op, m = _gen(seed), case["op"], case["m"]
    dt = DTYPES[case["dtype"]]
    s = {"case": dict(case)}
    if op.startswith("norm"):
        n = case["n"]
        # hidden states with an offset and a few large features, as residual streams have
        wide = 1 + 10 * (torch.rand(n, generator=g, device="cuda") < 0.01)
        s["x"] = (_randn(g, m, n) * wide + 0.2).to(dt)
        s["w"] = (1 + 0.2 * _randn(g, n)).to(dt)
        s["b"] = _randn(g, n, std=0.1, dtype=dt)
        if op == "norm_fwd":
            s["res"] = _randn(g, m, n, dtype=dt) if case["res"] else None
            return s
        xf = s["x"].float()
        s["mean"] = xf.mean(1)
        s["rstd"] = torch.rsqrt((xf - s["mean"][:, None]).square().mean(1) + EPS)
        s["dy"] = _randn(g, m, n, std=0.05, dtype=dt)
        s["dres"] = _randn(g, m, n, std=0.05, dtype=dt) if case["res"] else None
        return s
    if op.startswith("adapter"):
        k, n, r, a = case["k"], case["n"], case["rank"], case["adapters"]
        s["x"] = _randn(g, m, k, dtype=dt)
        s["down"] = _randn(g, a, r, k, std=1 / math.sqrt(k), dtype=dt)
        s["up"] = _randn(g, a, n, r, std=0.3 / math.sqrt(r), dtype=dt)
        s["scale"] = torch.rand(a, generator=g, device="cuda") + 0.5
        s["ranks"] = torch.randint(max(1, r // 4), r + 1, (a,), generator=g, device="cuda").to(torch.int32) \
            if case["ranks"] else None
        s["index"] = _requests(g, m, case["requests"], a)
        if op == "adapter_w24":
            s["vals"], s["meta"] = _pack24(g, k, n)
        elif op == "adapter_add":
            s["base"] = _randn(g, m, n, dtype=dt)
        else:
            s["dy"] = _randn(g, m, n, std=0.05, dtype=dt)
            s["base"] = _randn(g, m, k, std=0.05, dtype=dt)  # the shared projection's part of the input gradient
        return s
    d, v = case["d"], case["v"]
    s["w"] = _randn(g, v, d, std=1.5 / math.sqrt(d), dtype=dt)
    t = torch.randint(0, v, (m,), generator=g, device="cuda")
    # some rows lean towards their target, so that the losses run from near 0 to several times log(v)
    lean = 6 * torch.rand(m, 1, generator=g, device="cuda").square()
    s["x"] = (_randn(g, m, d) + lean * s["w"][t].float()).to(dt)
    s["target"] = torch.where(torch.rand(m, generator=g, device="cuda") < 0.1, torch.full_like(t, IGNORE), t)
    if op == "loss_bwd":
        z = s["x"].float() @ s["w"].float().t()
        s["lse"] = torch.logsumexp(z, 1)
        s["dloss"] = torch.full((m,), 1.0 / max(1, m), device="cuda") * 1024.0  # mean over the rows, loss scale 1024
    return s


def _lib():
    import structured_sparse_gemm_w24_amd as ssg
    return ssg


# ------------------------------------------------------------------- one pass
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    ssg, op = _lib(), s["case"]["op"]
    if op == "norm_fwd":
        return ssg.layer_norm(s["x"], s["w"], s["b"], EPS, residual=s["res"])
    if op == "norm_bwd":
        return ssg.layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["w"], dres=s["dres"])
    if op == "adapter_w24":
        return ssg.w24_low_rank_gemm_f16(s["x"], s["vals"], s["meta"], s["down"], s["up"], s["index"],
                                         s["scale"], s["ranks"])
    if op == "adapter_add":
        return ssg.low_rank_add(s["base"], s["x"], s["down"], s["up"], s["index"], s["scale"], s["ranks"])
    if op == "adapter_bwd":
        return ssg.low_rank_backward(s["dy"], s["x"], s["down"], s["up"], s["index"], s["scale"], s["ranks"],
                                     base=s["base"])
    if op == "loss_fwd":
        return ssg.linear_cross_entropy(s["x"], s["w"], s["target"], IGNORE)
    return ssg.linear_cross_entropy_backward(s["dloss"], s["x"], s["w"], s["target"], s["lse"], IGNORE)


def _dense24(vals, meta):
    """Dense [n, k] fp32 weight of the compressed one."""
    n, half = vals.shape
    pos = (meta.long()[:, :, None] >> (2 * torch.arange(16, device=vals.device))) & 3
    at = pos.reshape(n, half) + 4 * (torch.arange(half, device=vals.device) // 2)
    return torch.zeros(n, 2 * half, device=vals.device).scatter_(1, at, vals.float())


def _live(s):
    """1 where a token's adapter and a rank within it meet, [m, adapters, rank]."""
    a, r = s["down"].shape[:2]
    mine = s["index"][:, None] == torch.arange(a, device=s["index"].device)
    if s["ranks"] is None:
        return mine[:, :, None].expand(-1, a, r)
    return mine[:, :, None] & (torch.arange(r, device=mine.device) < s["ranks"][:, None])


def _run_plain(s):
    op = s["case"]["op"]
    dt = DTYPES[s["case"]["dtype"]]
    if op == "norm_fwd":
        x = s["x"] if s["res"] is None else (s["x"].float() + s["res"].float()).to(dt)
        xf = x.float()
        mean = xf.mean(1)
        rstd = torch.rsqrt((xf - mean[:, None]).square().mean(1) + EPS)
        y = ((xf - mean[:, None]) * rstd[:, None] * s["w"].float() + s["b"].float()).to(dt)
        return (y, mean, rstd) if s["res"] is None else (y, mean, rstd, x)
    if op == "norm_bwd":
        dy = s["dy"].float()
        xh = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
        gy = dy * s["w"].float()
        dx = (gy - gy.mean(1, keepdim=True) - xh * (gy * xh).mean(1, keepdim=True)) * s["rstd"][:, None]
        if s["dres"] is not None:
            dx = dx + s["dres"].float()
        return dx.to(dt), (dy * xh).sum(0), dy.sum(0)
    if op.startswith("adapter"):
        a, r, k = s["down"].shape
        x = s["x"].float()
        m = x.shape[0]
        down = s["down"].float().reshape(a * r, k)
        up = s["up"].float().transpose(1, 2).reshape(a * r, -1)
        live = _live(s)
        # every token against every adapter, what is not its own taken out; a pool's unused rows are left out too
        low = torch.where(live, (x @ down.t()).reshape(m, a, r) * s["scale"][:, None], 0.0).reshape(m, a * r)
        if op == "adapter_w24":
            return (x @ _dense24(s["vals"], s["meta"]).t() + low @ up).to(dt)
        if op == "adapter_add":
            return (s["base"].float() + low @ up).to(dt)
        dy = s["dy"].float()
        dlow = torch.where(live, (dy @ up.t()).reshape(m, a, r) * s["scale"][:, None], 0.0).reshape(m, a * r)
        dx = s["base"].float() + dlow @ down
        ddown = (dlow.t() @ x).reshape(a, r, k)
        dup = (low.t() @ dy).reshape(a, r, -1).transpose(1, 2).contiguous()
        return dx.to(dt), ddown.to(dt), dup.to(dt)
    x, w, t = s["x"].float(), s["w"].float(), s["target"]
    keep = t != IGNORE
    at = torch.where(keep, t, 0)
    z = x @ w.t()
    if op == "loss_fwd":
        top = z.max(1).values
        lse = top + (z - top[:, None]).exp().sum(1).log()
        return torch.where(keep, lse - z.gather(1, at[:, None])[:, 0], 0.0), lse
    p = (z - s["lse"][:, None]).exp()
    p.scatter_add_(1, at[:, None], torch.full_like(p[:, :1], -1.0))
    p = p * torch.where(keep, s["dloss"], 0.0)[:, None]
    return (p @ w).to(dt), (p.t() @ x).to(dt)


# ------------------------------------------------------ the definition, 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    f = {q: v.double() for q, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    op, m = case["op"], case["m"]
    if op.startswith("norm"):
        n = case["n"]
        if op == "norm_fwd":
            total = f["x"] if s["res"] is None else (f["x"] + f["res"]).to(s["x"].dtype).double()
            mean = total.sum(1) / n
            off = total - mean.unsqueeze(1)
            rstd = 1 / torch.sqrt((off * off).sum(1) / n + EPS)
            y = off * rstd.unsqueeze(1) * f["w"] + f["b"]
            return (y, mean, rstd) if s["res"] is None else (y, mean, rstd, total)
        xh = (f["x"] - f["mean"].unsqueeze(1)) * f["rstd"].unsqueeze(1)
        gy = f["dy"] * f["w"]
        c1, c2 = gy.sum(1) / n, (gy * xh).sum(1) / n
        dx = f["rstd"].unsqueeze(1) * (gy - c1.unsqueeze(1) - xh * c2.unsqueeze(1))
        return dx + (f["dres"] if s["dres"] is not None else 0), (f["dy"] * xh).sum(0), f["dy"].sum(0)
    if op.startswith("adapter"):
        # adapter by adapter, on the tokens that carry it
        n, r = case["n"], case["rank"]
        if op == "adapter_w24":
            k = case["k"]
            slots = torch.arange(k // 2, device="cuda")
            pos = (s["meta"][:, slots // 16].long() >> (slots % 16 * 2)) % 4
            kept = f["vals"].unsqueeze(2) * (pos.unsqueeze(2) == torch.arange(4, device="cuda"))
            out = f["x"] @ kept.view(n, k // 4, 2, 4).sum(2).view(n, k).t()
        else:
            out = f["base"].clone()
        ddown, dup = torch.zeros_like(f["down"]), torch.zeros_like(f["up"])
        for a in range(case["adapters"]):
            rows = (s["index"] == a).nonzero()[:, 0]
            q = int(s["ranks"][a]) if s["ranks"] is not None else r
            low, up, c = f["down"][a, :q], f["up"][a, :, :q], f["scale"][a]
            x = f["x"][rows]
            if op == "adapter_bwd":
                dy = f["dy"][rows]
                out[rows] += c * (dy @ up) @ low
                ddown[a, :q] = c * (dy @ up).t() @ x
                dup[a, :, :q] = c * dy.t() @ (x @ low.t())
            else:
                out[rows] += c * (x @ low.t()) @ up.t()
        return (out, ddown, dup) if op == "adapter_bwd" else out
    z = f["x"] @ f["w"].t()
    keep = s["target"] != IGNORE
    at = torch.where(keep, s["target"], torch.zeros_like(s["target"]))
    if op == "loss_fwd":
        lse = torch.logsumexp(z, 1)
        return (lse - z[torch.arange(m, device="cuda"), at]) * keep, lse
    gz = torch.exp(z - f["lse"].unsqueeze(1))
    gz[torch.arange(m, device="cuda"), at] -= 1
    gz *= (f["dloss"] * keep).unsqueeze(1)
    return gz @ f["w"], gz.t() @ f["x"]
