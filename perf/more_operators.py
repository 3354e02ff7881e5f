"""Measured cases of the expert-layer operators: microscaled 4-bit floating point
(quantisation and products), products grouped by expert with their gradients, and
the global gradient norm with clipping.

Every case is one call, or one pair of calls, that a user makes while training a
layer of experts in 16 bits and serving it, or any projection, with 4-bit weights.

``run`` computes the plain form (elementary torch operations, products in 32 bits)
unless ``own`` is true; then it calls the library.
"""

import math

import torch

own = False

BLOCK = 32    # values that share a scale
PAD = 128     # packed rows hold a multiple of this many values
CLIP_EPS = 1e-6
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
# magnitudes of the 4-bit codes 0..7; code 8 + c is minus code c
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # one token's activations on their way into a 4-bit product
        dict(name="quant_token", op="quant", dtype="bf16", m=1, k=1024),
        # the activations of a long prompt batch, or a weight being converted
        dict(name="quant_batch", op="quant", dtype="f16", m=8192, k=4096),
        # a decode step of four requests through a 4-bit projection
        dict(name="linear_token", op="linear", dtype="f16", m=4, n=4096, k=1024),
        # a prompt batch through a square 4-bit projection
        dict(name="linear_batch", op="linear", dtype="bf16", m=8192, n=4096, k=4096),
        # a decode step through 4-bit experts: 16 tokens of two experts each, 32 experts
        dict(name="experts_decode", op="experts", dtype="bf16", m=32, n=2048, k=1024, e=32, used=1.0),
        # prompts through 4-bit experts: ragged groups, odd widths, rows behind the last group
        dict(name="experts_prefill", op="experts", dtype="f16", m=7001, n=4100, k=2000, e=12, used=0.95),
        # a decode step through 16-bit experts
        dict(name="group_fwd_decode", op="group_fwd", dtype="bf16", m=64, n=1024, k=2048, e=32, used=1.0),
        # a training batch through 16-bit experts
        dict(name="group_fwd_batch", op="group_fwd", dtype="f16", m=16384, n=4096, k=1024, e=16, used=1.0),
        # that batch's gradients, to the tokens and to the experts
        dict(name="group_bwd_batch", op="group_bwd", dtype="bf16", m=16384, n=4096, k=1024, e=16, used=1.0),
        # gradients of a short batch of odd widths, rows behind the last group
        dict(name="group_bwd_odd", op="group_bwd", dtype="f16", m=1531, n=776, k=1000, e=6, used=0.9),
        # clipping the gradients of a few adapters and norms
        dict(name="clip_adapters", op="clip", dtype="f16", tensors=24, total=400000, max_norm=1.0, align=64),
        # clipping the gradients of a whole model, matrices and vectors of both types
        dict(name="clip_model", op="clip", dtype="mixed", tensors=290, total=120000000, max_norm=1.0, align=64),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["quant", "linear", "experts", "group_fwd", "group_bwd", "clip"])
        if op == "quant":
            c = dict(op=op, dtype=rng.choice(["f16", "bf16", "f32"]), m=_log_int(rng, 1, 16000),
                     k=_log_int(rng, 32, 16384))
        elif op == "linear":
            c = dict(op=op, dtype=rng.choice(["f16", "bf16"]), m=_log_int(rng, 1, 16384), n=_log_int(rng, 64, 16384),
                     k=_log_int(rng, 64, 8192))
        elif op == "clip":
            tensors = _log_int(rng, 1, 400)
            c = dict(op=op, dtype=rng.choice(["f16", "bf16", "f32", "mixed"]), tensors=tensors,
                     total=_log_int(rng, max(1000, 20 * tensors), 150000000), max_norm=rng.choice([0.1, 1.0, 1e6]),
                     align=rng.choice([1, 64]))
        else:
            c = dict(op=op, dtype=rng.choice(["f16", "bf16"]), m=_log_int(rng, 1, 16384), n=8 * _log_int(rng, 8, 512),
                     k=8 * _log_int(rng, 8, 512), e=_log_int(rng, 1, 64), used=rng.choice([1.0, 0.9]))
            if op == "experts":  # any width
                c.update(n=_log_int(rng, 64, 4096), k=_log_int(rng, 64, 4096))
        if _cost(c) <= most:
            return c


def _cost(c):
    w = work(c)
    return max(w["bytes"], w["flops"] / (600 if c["op"] in ("linear", "experts") else 150))


def work(case):
    """Bytes with every input read and every output written once, and the multiply-adds of the products."""
    op = case["op"]
    if op == "clip":
        e = {"f32": 4, "mixed": 3}.get(case["dtype"], 2)
        return {"bytes": 2 * e * case["total"] + 4, "flops": 3 * case["total"]}
    e = 4 if case["dtype"] == "f32" else 2
    m, k = case["m"], case["k"]
    if op == "quant":  # in, codes and scales, and the values they stand for
        return {"bytes": 2 * m * k * e + m * k * 17 // 32, "flops": 2 * m * k}
    n = case["n"]
    if op == "linear":
        return {"bytes": 2 * m * (k + n) + n * k * 17 // 32, "flops": 2 * m * n * k}
    rows = _used(case)
    live = min(case["e"], rows)  # experts that the rows can reach
    if op == "experts":
        return {"bytes": 2 * rows * (k + n) + live * n * k * 17 // 32, "flops": 2 * rows * n * k}
    if op == "group_fwd":
        return {"bytes": 2 * rows * (k + n) + 2 * live * n * k, "flops": 2 * rows * n * k}
    # dy, x and the weights read, dx and dw written
    return {"bytes": 2 * rows * (2 * k + n) + 2 * live * n * k + 2 * case["e"] * n * k, "flops": 4 * rows * n * k}


# ----------------------------------------------------------------- the inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _randn(g, *shape, std=1.0, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda").mul_(std).to(dtype)


def _used(case):
    return max(1, int(case["m"] * case["used"]))


def _cuts(case, seed):
    """Group boundaries of a router's ragged choice: some experts popular, some without a row."""
    g = torch.Generator().manual_seed(int(seed) + 7)
    e, rows = case["e"], _used(case)
    share = torch.exp(0.7 * torch.randn(e, generator=g))
    if e > 2:
        share[torch.randint(0, e, (max(1, e // 8),), generator=g)] = 0.0
    if float(share.sum()) == 0.0:
        share[0] = 1.0
    pick = torch.multinomial(share, rows, replacement=True, generator=g)
    return [0] + torch.cumsum(torch.bincount(pick, minlength=e), 0).tolist()


def _padded(k):
    return -(-k // PAD) * PAD


def _packed_weight(g, rows, k):
    """A random 4-bit weight in the library's layout: codes [rows, kp / 2], value 2i in the low half of
    byte i, and scales [rows, kp / 32], 2 to the power byte - 127; zeros past k."""
    kp = _padded(k)
    codes = torch.randint(0, 256, (rows, kp // 2), generator=g, device="cuda", dtype=torch.uint8)
    codes[:, (k + 1) // 2:] = 0
    if k % 2:
        codes[:, k // 2] &= 15
    near = 127 - int(round(math.log2(3 * math.sqrt(k))))
    scales = torch.randint(near - 1, near + 2, (rows, kp // BLOCK), generator=g, device="cuda", dtype=torch.uint8)
    return codes, scales


def _sizes(case):
    """Sizes of a model's tensors: matrices that hold most of it, and many short vectors."""
    n, total = case["tensors"], case["total"]
    g = torch.Generator().manual_seed(n + total)
    share = torch.exp(2.0 * torch.randn(n, generator=g, dtype=torch.float64))
    size = (share / share.sum() * (total - n)).long() + 1
    size[0] += total - int(size.sum())
    return size.tolist()


def _buckets(case, sizes):
    """Zeroed flat buffers, one a type, and a view for every tensor: how a trainer keeps its gradients."""
    kinds = ["f16", "f32"] if case["dtype"] == "mixed" else [case["dtype"]]
    a, ends, spans = case["align"], dict.fromkeys(kinds, 0), []
    for i, n in enumerate(sizes):
        kind = kinds[i % len(kinds)]
        spans.append((kind, ends[kind], n))
        ends[kind] += -(-n // a) * a
    flat = {q: torch.zeros(n, dtype=DTYPES[q], device="cuda") for q, n in ends.items()}
    return [flat[q] for q in kinds], [flat[q][at:at + n] for q, at, n in spans]


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = {"case": dict(case)}
    if op == "clip":
        sizes = _sizes(case)
        _, s["grads"] = _buckets(case, sizes)
        for t in s["grads"]:
            t.copy_(_randn(g, t.numel(), std=0.01))
        s["flat"], s["out"] = _buckets(case, sizes)
        return s
    dt, m, k = DTYPES[case["dtype"]], case["m"], case["k"]
    # hidden states with a few large features, as residual streams have
    wide = 1 + 10 * (torch.rand(k, generator=g, device="cuda") < 0.01)
    s["x"] = (_randn(g, m, k) * wide).to(dt)
    if op == "quant":
        return s
    n = case["n"]
    if op == "linear":
        s["w"], s["ws"] = _packed_weight(g, n, k)
        return s
    e = case["e"]
    s["cuts"] = _cuts(case, seed)
    s["offsets"] = torch.tensor(s["cuts"], dtype=torch.int32, device="cuda")
    if op == "experts":
        w, ws = _packed_weight(g, e * n, k)
        s["w"], s["ws"] = w.view(e, n, -1), ws.view(e, n, -1)
    else:
        s["w"] = _randn(g, e, n, k, std=1 / math.sqrt(k), dtype=dt)
    if op == "group_bwd":
        s["x"] = _randn(g, m, k, dtype=dt)
        s["dy"] = _randn(g, m, n, std=0.05, dtype=dt)
        s["out"] = torch.zeros(m, k, dtype=dt, device="cuda")
    else:
        s["out"] = torch.zeros(m, n, dtype=dt, device="cuda")
    return s


def _lib():
    import structured_sparse_gemm_w24_amd as ssg
    return ssg


# ------------------------------------------------------------------- one pass
def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    ssg, op = _lib(), s["case"]["op"]
    if op == "quant":
        codes, scales = ssg.mxfp4_quantize(s["x"])
        return ssg.mxfp4_dequantize(codes, scales, s["x"].shape[1], s["x"].dtype)
    if op == "linear":
        return ssg.mxfp4_linear(s["x"], s["w"], s["ws"])
    if op == "experts":
        return ssg.mxfp4_grouped_linear(s["x"], s["w"], s["ws"], s["offsets"], out=s["out"])
    if op == "group_fwd":
        return ssg.grouped_gemm(s["x"], s["w"], s["offsets"], out=s["out"])
    if op == "group_bwd":
        return ssg.grouped_gemm_backward(s["dy"], s["x"], s["w"], s["offsets"], out=s["out"])
    norm, _ = ssg.clip_grad_norm(s["grads"], s["case"]["max_norm"], out=s["out"])
    return [norm, *s["flat"]]


def _quantised(x):
    """The values that x's 4-bit codes and scales stand for, fp32 [m, k]: blocks of 32 share the scale
    2^(floor(log2 max) - 2), values round to the nearest of the eight magnitudes (ties to the even code)."""
    m, k = x.shape
    f = torch.nn.functional.pad(x.float(), (0, _padded(k) - k)).view(m, -1, BLOCK)
    top = f.abs().amax(2, keepdim=True)
    e = torch.where(top > 0, torch.frexp(top).exponent - 3, -127).clamp(-127, 127)
    q = torch.ldexp(f.double(), -e).abs()  # (64 bits: 2^127 times the largest value)
    step = torch.where(q < 2, 0.5, torch.where(q < 4, 1.0, 2.0))
    q = torch.clamp(torch.round(q / step) * step, max=6.0)
    v = torch.copysign(torch.ldexp(q, e), f.double()).float()
    return v.view(m, -1)[:, :k]


def _values(codes, scales, k):
    """fp32 values of packed rows."""
    table = torch.tensor(MAGNITUDES + tuple(-v for v in MAGNITUDES), device=codes.device)
    v = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
    v = table[v.int()].unflatten(-1, (-1, BLOCK)) * torch.exp2(scales.float() - 127).unsqueeze(-1)
    return v.flatten(-2)[..., :k]


def _run_plain(s):
    case = s["case"]
    op = case["op"]
    if op == "clip":
        total = sum(t.float().square().sum().double() for t in s["grads"])
        norm = total.sqrt()
        by = torch.clamp(case["max_norm"] / (norm + CLIP_EPS), max=1.0).float()
        for o, t in zip(s["out"], s["grads"]):
            o.copy_(t.float() * by)
        return [norm.float(), *s["flat"]]
    dt = DTYPES[case["dtype"]]
    if op == "quant":
        return _quantised(s["x"]).to(dt)
    if op == "linear":
        return (_quantised(s["x"]) @ _values(s["w"], s["ws"], case["k"]).t()).to(dt)
    out = s["out"]
    spans = [(e, a, b) for e, (a, b) in enumerate(zip(s["cuts"], s["cuts"][1:])) if b > a]
    if op == "experts":
        x = _quantised(s["x"])
        for e, a, b in spans:
            out[a:b] = (x[a:b] @ _values(s["w"][e], s["ws"][e], case["k"]).t()).to(dt)
        return out
    if op == "group_fwd":
        for e, a, b in spans:
            out[a:b] = (s["x"][a:b].float() @ s["w"][e].float().t()).to(dt)
        return out
    dw = torch.zeros_like(s["w"])
    for e, a, b in spans:
        dy = s["dy"][a:b].float()
        out[a:b] = (dy @ s["w"][e].float()).to(dt)
        dw[e] = (dy.t() @ s["x"][a:b].float()).to(dt)
    return out, dw


# ------------------------------------------------------ the definition, 64 bits
def _exact_quant(x):
    """Nearest magnitude by looking at all eight distances; a tie goes to the even code."""
    m, k = x.shape
    out = torch.empty(m, k, dtype=torch.float64, device=x.device)
    mags = torch.tensor(MAGNITUDES, dtype=torch.float64, device=x.device)
    for c in range(0, k, BLOCK):
        v = x[:, c:c + BLOCK].double()
        top = v.abs().max(1, keepdim=True).values
        # floor(log2) by comparison with the powers themselves: a rounded logarithm may pass an integer
        p = torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top))))
        p = torch.where(torch.exp2(p) > top, p - 1, p)
        p = torch.where(torch.exp2(p + 1) <= top, p + 1, p)
        scale = torch.exp2(torch.where(top > 0, torch.clamp(p - 2, -127, 127), torch.full_like(p, -127)))
        best = mags[0].expand_as(v).clone()
        miss = (v.abs() / scale - best).abs()
        for i in range(1, 8):
            off = (v.abs() / scale - mags[i]).abs()
            take = (off < miss) | ((off == miss) & (i % 2 == 0))
            best, miss = torch.where(take, mags[i], best), torch.where(take, off, miss)
        out[:, c:c + BLOCK] = torch.sign(v) * best * scale
    return out


def _exact_weight(codes, scales, k):
    n = codes.shape[0]
    out = torch.empty(n, 2 * codes.shape[1], dtype=torch.float64, device=codes.device)
    for half in (0, 1):
        c = (codes.long() >> (4 * half)) % 16
        expo, frac = (c % 8) // 2, (c % 2).double()
        mag = torch.where(expo == 0, frac * 0.5, (1 + frac / 2) * torch.exp2((expo - 1).double()))
        out[:, half::2] = torch.where(c >= 8, -mag, mag)
    return (out * torch.exp2(scales.double() - 127).repeat_interleave(BLOCK, 1))[:, :k]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "clip":
        squares = torch.stack([(t.double() ** 2).sum() for t in s["grads"]])
        norm = torch.sqrt(squares.sum())
        by = torch.minimum(case["max_norm"] / (norm + CLIP_EPS), torch.ones_like(norm))
        flat, views = _buckets(case, _sizes(case))
        wide = [torch.zeros(b.shape, dtype=torch.float64, device="cuda") for b in flat]
        for v, t in zip(views, s["grads"]):
            i = [b.dtype for b in flat].index(v.dtype)
            wide[i][v.storage_offset():v.storage_offset() + t.numel()] = t.double() * by
        return [norm, *wide]
    if op == "quant":
        return _exact_quant(s["x"])
    if op == "linear":
        return _exact_quant(s["x"]) @ _exact_weight(s["w"], s["ws"], case["k"]).t()
    cuts, f64 = s["cuts"], torch.float64
    out = torch.zeros(s["out"].shape, dtype=f64, device="cuda")
    dw = torch.zeros(s["w"].shape, dtype=f64, device="cuda") if op == "group_bwd" else None
    for e in range(case["e"]):
        rows = torch.arange(cuts[e], cuts[e + 1], device="cuda")
        if rows.numel() == 0:
            continue
        if op == "group_bwd":
            dy = s["dy"][rows].to(f64)
            out[rows] = dy @ s["w"][e].to(f64)
            dw[e] = dy.t() @ s["x"][rows].to(f64)
        elif op == "group_fwd":
            out[rows] = s["x"][rows].to(f64) @ s["w"][e].to(f64).t()
        else:
            out[rows] = _exact_quant(s["x"][rows]) @ _exact_weight(s["w"][e], s["ws"][e], case["k"]).t()
    return (out, dw) if op == "group_bwd" else out
