"""Low-rank adapters (added to a base, beside the 2:4 product, and their
gradients) against a plain 64-bit implementation.

Tolerance of every output, set before the first run: one rounding to the output
type, u |ref|, plus (split + 2^-24 L) S, where S is the same sum taken over
absolute values, L the length of the longest fp32 chain (K, N or the tokens)
plus 64, and split what the pair of 16-bit values that carries the low-rank
values can lose: twice 2^-21 for fp16 (11 + 11 bits), twice 2^-16 for bf16; plus
the type's smallest step (and for fp16 the low-rank values' own, 2^-24, times
the pool's size)."""

import numpy as np
import pytest

import workloads as wl

pytestmark = pytest.mark.gpu


def _kind(dtype):
    import torch
    return {"f16": (torch.float16, 2.0 ** -11, 2.0 ** -20, 2.0 ** -24),
            "bf16": (torch.bfloat16, 2.0 ** -8, 2.0 ** -15, 1e-37)}[dtype]


def make(seed, dtype, m, n, k, r, adapters, index="runs", ranks=True, scale=True, strided=False):
    import torch
    dt = _kind(dtype)[0]
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")
    ints = lambda lo, hi, s: torch.randint(lo, hi, s, generator=g, device="cuda").to(torch.int32)

    def rows(c):
        if strided:
            return rnd(m, c + 24).to(dt)[:, 8:8 + c]
        return rnd(m, c).to(dt)
    c = dict(x=rows(k), base=rows(n), dy=rows(n), xbase=rows(k),
             down=(rnd(adapters, r, k) / k ** 0.5).to(dt), up=(rnd(adapters, n, r) / r ** 0.5).to(dt),
             scale=(rnd(adapters).abs() + 0.25) if scale else None,
             ranks=ints(0, r + 1, (adapters,)) if ranks else None)
    if index == "runs":
        i = torch.arange(m, device="cuda") * 5 // max(m, 1)
        c["index"] = (ints(-1, adapters, (8,))[i.long()]).to(torch.int32)
    elif index == "mixed":
        c["index"] = ints(-1, adapters, (m,))
    else:
        c["index"] = torch.full((m,), index, dtype=torch.int32, device="cuda")
    return c


def reference(c, backward=False):
    """(value, sum of absolute values) of delta, or of dx, ddown and dup without the base."""
    import torch
    x, dy, down, up = (c[q].double() for q in ("x", "dy", "down", "up"))
    a, r, k = down.shape
    n, m = up.shape[1], x.shape[0]
    z = lambda *s: torch.zeros(*s, dtype=torch.float64, device="cuda")
    delta, dx, ddown, dup = (z(m, n), z(m, n)), (z(m, k), z(m, k)), (z(a, r, k), z(a, r, k)), (z(a, n, r), z(a, n, r))
    for i in range(a):
        t = (c["index"] == i).nonzero()[:, 0]
        q = r if c["ranks"] is None else int(c["ranks"][i])
        s = 1.0 if c["scale"] is None else c["scale"][i].double()
        d, u = down[i, :q], up[i, :, :q]
        for v, f in ((0, lambda w: w), (1, torch.abs)):
            low, dlow = s * f(x[t]) @ f(d).t(), s * f(dy[t]) @ f(u)
            delta[v][t] = low @ f(u).t()
            if backward:
                dx[v][t] = dlow @ f(d)
                ddown[v][i, :q] = dlow.t() @ f(x[t])
                dup[v][i, :, :q] = f(dy[t]).t() @ low
    return (dx, ddown, dup) if backward else delta


def close(got, ref, size, dtype, chain, pool=1.0):
    _, u, split, tiny = _kind(dtype)
    bound = u * ref.abs() + (split + 2.0 ** -24 * (chain + 64)) * size + tiny * (1 + pool)
    off = (got.double() - ref).abs()
    assert (off <= bound).all(), ((off / bound).max().item(), (off > bound).sum().item())


SHAPES = [
    # m, n, k, R, adapters, index
    (1, 8, 8, 8, 1, 0), (1, 1024, 768, 16, 4, "mixed"), (7, 264, 72, 8, 3, "mixed"), (32, 4096, 1024, 16, 24, "mixed"),
    (128, 520, 200, 128, 5, "mixed"), (129, 520, 200, 128, 5, "runs"), (130, 256, 64, 24, 9, "mixed"),
    (257, 776, 392, 40, 300, "mixed"), (640, 1024, 1000, 64, 6, "runs"), (1531, 2312, 768, 32, 8, "runs"),
    (2500, 136, 2056, 16, 2, "runs"), (300, 768, 768, 8, 1, 0), (200, 128, 128, 16, 3, -1),
]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,n,k,r,a,index", SHAPES)
def test_add(lib, gpu, dtype, m, n, k, r, a, index):
    c = make(m + n + k, dtype, m, n, k, r, a, index)
    out = lib.low_rank_add(c["base"], c["x"], c["down"], c["up"], c["index"], c["scale"], c["ranks"])
    delta, size = reference(c)
    base = c["base"].double()
    close(out, base + delta, base.abs() + size, dtype, k + r, r)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,n,k,r,a,index", SHAPES + [
    (6200, 256, 136, 16, 2, "runs"), (4100, 64, 64, 8, 1, 0), (5000, 1024, 512, 128, 400, "runs"),
    (4500, 2048, 1024, 64, 500, "mixed")])
def test_backward(lib, gpu, dtype, m, n, k, r, a, index):
    c = make(m * 3 + n + k, dtype, m, n, k, r, a, index)
    got = lib.low_rank_backward(c["dy"], c["x"], c["down"], c["up"], c["index"], c["scale"], c["ranks"],
                                base=c["xbase"])
    dx, ddown, dup = reference(c, backward=True)
    base = c["xbase"].double()
    close(got[0], base + dx[0], base.abs() + dx[1], dtype, n + r, r)
    # (the low values' own smallest step, fp16: 2^-24 of a value that is then multiplied by up to M tokens)
    close(got[1], ddown[0], ddown[1], dtype, n + m, m ** 0.5)
    close(got[2], dup[0], dup[1], dtype, k + m, m ** 0.5)


@pytest.mark.parametrize("m,n,k,r,a,index", [
    (1, 64, 64, 8, 1, 0), (3, 192, 128, 16, 2, "mixed"), (32, 4096, 1024, 16, 24, "mixed"), (64, 1024, 4096, 8, 70, "mixed"),
    (128, 256, 512, 32, 3, "runs"), (129, 256, 512, 32, 3, "mixed"), (200, 512, 256, 64, 2, "runs"),
    (520, 1024, 1024, 16, 4, "runs"), (512, 4096, 1024, 24, 4, "runs"), (1024, 1024, 4096, 128, 3, "runs"),
    (4096, 3072, 768, 40, 7, "runs"), (700, 320, 320, 16, 90, "mixed")])
def test_beside_the_sparse_product(lib, gpu, m, n, k, r, a, index):
    import torch
    c = make(m * 7 + n, "f16", m, n, k, r, a, index)
    w = wl.random_24_f16(np.random.default_rng(m + n), 1, k, n)["Wp"]
    vals, meta = lib.w24_pack_f16(w)
    vals, meta = torch.from_numpy(vals).cuda(), torch.from_numpy(meta.view(np.int32)).cuda()
    x = c["x"]
    out = lib.w24_low_rank_gemm_f16(x, vals, meta, c["down"], c["up"], c["index"], c["scale"], c["ranks"])
    wd = torch.from_numpy(w).cuda().double()
    delta, size = reference(c)
    close(out, x.double() @ wd + delta, x.double().abs() @ wd.abs() + size, "f16", k + r, r)
    if index == -1 or m == 520:  # without adapters: the plain product, bit for bit
        none = torch.full_like(c["index"], -1)
        plain = lib.w24_gemm_f16(x, vals, meta, splits=1)
        assert torch.equal(lib.w24_low_rank_gemm_f16(x, vals, meta, c["down"], c["up"], none), plain)


@pytest.mark.parametrize("m", [20, 300])
def test_pool_slots_past_the_rank_are_not_used(lib, gpu, m):
    """NaN in every unused slot of the pool, and in every adapter nobody has, changes nothing."""
    import torch
    c = make(5, "f16", m, 256, 128, 24, 6, "mixed")
    c["index"][c["index"] == 4] = -1
    args = lambda d, u: (c["base"], c["x"], d, u, c["index"], c["scale"], c["ranks"])
    down, up = c["down"].clone(), c["up"].clone()
    for i in range(6):
        q = 0 if i == 4 else int(c["ranks"][i])
        down[i, q:], up[i, :, q:] = float("nan"), float("nan")
    assert torch.equal(lib.low_rank_add(*args(down, up)), lib.low_rank_add(*args(c["down"], c["up"])))
    bwd = lambda d, u: lib.low_rank_backward(c["dy"], c["x"], d, u, c["index"], c["scale"], c["ranks"], c["xbase"])
    for p, q in zip(bwd(down, up), bwd(c["down"], c["up"])):
        assert torch.equal(p, q) and torch.isfinite(p).all()


@pytest.mark.parametrize("m", [30, 150, 700])
def test_a_broken_adapter_stays_with_its_tokens(lib, gpu, m):
    """One request's adapter holds NaN and infinities: no other token changes, in any form."""
    import torch
    c = make(15, "f16", m, 256, 128, 16, 5, "mixed")
    w = wl.random_24_f16(np.random.default_rng(3), 1, 128, 256)["Wp"]
    vals, meta = lib.w24_pack_f16(w)
    vals, meta = torch.from_numpy(vals).cuda(), torch.from_numpy(meta.view(np.int32)).cuda()
    c["ranks"][2] = 16
    others = c["index"] != 2
    x = c["x"].clone()
    x[~others, 7] = float("inf")  # and inputs of its own that are not finite
    down, up = c["down"].clone(), c["up"].clone()
    down[2, 3] = float("nan")
    up[2, 5:9] = float("inf")
    rest = (c["index"], c["scale"], c["ranks"])

    def outputs(x, down, up):
        return (lib.low_rank_add(c["base"], x, down, up, *rest), lib.w24_low_rank_gemm_f16(x, vals, meta, down, up, *rest),
                *lib.low_rank_backward(c["dy"], x, down, up, *rest, base=c["xbase"]))
    good, bad = outputs(c["x"], c["down"], c["up"]), outputs(x, down, up)
    for p, q in zip(good[:3], bad[:3]):
        assert torch.equal(p[others], q[others])
        assert not torch.isfinite(q[~others].float()).all()
    for p, q in zip(good[3:], bad[3:]):
        keep = [0, 1, 3, 4]
        assert torch.equal(p[keep], q[keep])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,n,k,r,a", [(30, 64, 72, 24, 5), (300, 128, 64, 40, 5), (1500, 1024, 128, 8, 3),
                                       (5000, 256, 512, 128, 5)])
def test_slots_past_the_rank_get_zeros_beside_inputs_that_are_not_finite(lib, gpu, dtype, m, n, k, r, a):
    """Infinities and NaN in x and in dy of one adapter's tokens: its gradients' slots past its rank
    are zeros all the same, and the other adapters and tokens keep their values."""
    import torch
    c = make(m + n, dtype, m, n, k, r, a, "mixed")
    c["ranks"][1] = r - 3
    pool = (c["down"], c["up"], c["index"], c["scale"], c["ranks"])
    ref = lib.low_rank_backward(c["dy"], c["x"], *pool, base=c["xbase"])
    mine = (c["index"] == 1).nonzero()[:, 0]
    others = c["index"] != 1
    keep = [i for i in range(a) if i != 1]
    for key, value in (("x", float("inf")), ("x", float("nan")), ("dy", float("inf")), ("dy", float("nan"))):
        d = {q: c[q].clone() for q in ("x", "dy")}
        d[key][mine[0], 5] = value
        d[key][mine[-1]] = value
        dx, ddown, dup = lib.low_rank_backward(d["dy"], d["x"], *pool, base=c["xbase"])
        assert (ddown[1, r - 3:] == 0).all() and (dup[1, :, r - 3:] == 0).all()
        assert not torch.isfinite(ddown[1, :r - 3]).all() and not torch.isfinite(dup[1, :, :r - 3]).all()
        assert torch.equal(dx[others], ref[0][others])
        assert torch.equal(ddown[keep], ref[1][keep]) and torch.equal(dup[keep], ref[2][keep])


TILES = [  # tokens, channels, the tile that the product takes there
    (150, 256, (32, 32)), (512, 2048, (64, 64)), (1024, 2048, (64, 128)), (1100, 2048, (128, 128)),
    (4500, 2816, (256, 256))]


def _fused(lib, m, n, k, r, a, seed):
    """A call of the fused product with every tile's tokens mixed over the adapters, and its pieces."""
    import torch
    c = make(seed, "f16", m, n, k, r, a, "mixed")
    w = wl.random_24_f16(np.random.default_rng(seed), 1, k, n)["Wp"]
    vals, meta = lib.w24_pack_f16(w)
    vals, meta = torch.from_numpy(vals).cuda(), torch.from_numpy(meta.view(np.int32)).cuda()

    def call(down=None, up=None, index=None, x=None):
        return lib.w24_low_rank_gemm_f16(c["x"] if x is None else x, vals, meta, c["down"] if down is None else down,
                                         c["up"] if up is None else up, c["index"] if index is None else index,
                                         c["scale"], c["ranks"])
    return c, torch.from_numpy(w).cuda().double(), call


@pytest.mark.parametrize("r,a", [(24, 5), (128, 5), (128, 2)])
@pytest.mark.parametrize("m,n,tile", TILES)
def test_every_tile_of_the_fused_product(lib, gpu, m, n, tile, r, a):
    """Each tile of the fused product (with and without loader waves, one and more waves, one and two
    rounds of 64 slots): its values, and what NaN past the ranks, a broken adapter and
    an index outside the pool do."""
    import torch
    assert lib.tile_choice(1, m, n, 128) == tile
    c, w, call = _fused(lib, m, n, 128, r, a, m + r)
    c["ranks"][1] = r
    out = call()
    delta, size = reference(c)
    x = c["x"].double()
    close(out, x @ w + delta, x.abs() @ w.abs() + size, "f16", 128 + r, r)

    # slots past the ranks
    down, up = c["down"].clone(), c["up"].clone()
    for i in range(a):
        q = int(c["ranks"][i])
        down[i, q:], up[i, :, q:] = float("nan"), float("inf")
    assert torch.equal(call(down, up), out)

    # a broken adapter: its own tokens, in the broken channels
    mine = c["index"] == 1
    slots = [0, r // 2, r - 1]
    channels = torch.tensor([0, 7, 31, 32, n // 2 + 5, n - 1], device="cuda")
    up = c["up"].clone()
    for i, ch in enumerate(channels.tolist()):
        up[1, ch, slots[i % 3]] = (float("nan"), float("inf"), float("-inf"))[i % 3]
    got = call(up=up)
    expect = torch.zeros(m, n, dtype=torch.bool, device="cuda")
    expect[:, channels] = mine[:, None].expand(-1, len(channels))
    assert torch.equal(torch.isfinite(got), ~expect)
    assert torch.equal(got[~expect], out[~expect])
    down = c["down"].clone()
    down[1, r - 1, 3] = float("nan")
    got = call(down=down)
    assert torch.isnan(got[mine]).all() and torch.equal(got[~mine], out[~mine])

    # a token whose input is not finite
    x = c["x"].clone()
    x[m // 2] = float("nan")
    got = call(x=x)
    others = torch.arange(m, device="cuda") != m // 2
    assert torch.isnan(got[m // 2]).all() and torch.equal(got[others], out[others])

    # indices outside the pool
    index, none = c["index"].clone(), c["index"].clone()
    bad = torch.zeros(m, dtype=torch.bool, device="cuda")
    for i, v in ((0, a), (33, -2), (64, 2 ** 31 - 1), (m - 1, -2 ** 31), (m // 2, 65535)):
        index[i], none[i], bad[i] = v, -1, True
    got, ref = call(index=index), call(index=none)
    assert torch.isnan(got[bad]).all() and torch.equal(got[~bad], ref[~bad])


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m", [60, 300])
@pytest.mark.parametrize("r", [24, 128])
def test_broken_weights_mark_their_channels(lib, gpu, dtype, m, r):
    """Values of `up` that are not finite, in any slot in use: beside a base, exactly their adapter's tokens
    in exactly their channels are not finite, and nothing else changes; the same of `down` in dx."""
    import torch
    n, k, a = 200, 136, 5
    c = make(m + r, dtype, m, n, k, r, a, "mixed")
    c["ranks"][1] = r
    rest = (c["index"], c["scale"], c["ranks"])
    mine = c["index"] == 1
    for key, width, call in (
            ("up", n, lambda p: lib.low_rank_add(c["base"], c["x"], c["down"], p, *rest)),
            ("down", k, lambda p: lib.low_rank_backward(c["dy"], c["x"], p, c["up"], *rest, base=c["xbase"])[0])):
        out = call(c[key])
        pool = c[key].clone()
        channels = torch.tensor([0, 7, 31, 64, width - 1], device="cuda")
        for i, ch in enumerate(channels.tolist()):
            slot = (0, r // 2, r - 1)[i % 3]
            at = (1, ch, slot) if key == "up" else (1, slot, ch)
            pool[at] = (float("nan"), float("inf"), float("-inf"))[i % 3]
        got = call(pool)
        expect = torch.zeros(m, width, dtype=torch.bool, device="cuda")
        expect[:, channels] = mine[:, None].expand(-1, len(channels))
        assert torch.equal(torch.isfinite(got), ~expect)
        assert torch.equal(got[~expect], out[~expect])


@pytest.mark.parametrize("m", [40, 260])
def test_index_outside_the_pool_gives_nan_rows(lib, gpu, m):
    import torch
    c = make(6, "f16", m, 192, 64, 8, 3, "mixed")
    bad = torch.zeros(m, dtype=torch.bool, device="cuda")
    good = c["index"].clone()
    for i, v in ((0, 3), (17, -2), (m - 1, 2 ** 31 - 1), (33, -2 ** 31)):
        c["index"][i] = v
        bad[i] = True
        good[i] = -1
    out = lib.low_rank_add(c["base"], c["x"], c["down"], c["up"], c["index"], c["scale"], c["ranks"])
    ref = lib.low_rank_add(c["base"], c["x"], c["down"], c["up"], good, c["scale"], c["ranks"])
    assert torch.isnan(out[bad]).all() and torch.equal(out[~bad], ref[~bad])
    got = lib.low_rank_backward(c["dy"], c["x"], c["down"], c["up"], c["index"], c["scale"], c["ranks"], c["xbase"])
    ref = lib.low_rank_backward(c["dy"], c["x"], c["down"], c["up"], good, c["scale"], c["ranks"], c["xbase"])
    assert torch.isnan(got[0][bad]).all() and torch.equal(got[0][~bad], ref[0][~bad])
    assert torch.equal(got[1], ref[1]) and torch.equal(got[2], ref[2])


@pytest.mark.parametrize("m", [128, 129, 700])
@pytest.mark.parametrize("size", [18, 5, -9, -13, -20])
@pytest.mark.parametrize("forward", [True, False])
def test_low_rank_values_of_any_size(lib, gpu, m, size, forward):
    """Low-rank values far above fp16's largest number and far below its steps (about 2^size, times 2^-6
    to 2^6 by token), in pools whose other side brings the result back into range: the tolerance of every
    other case, in every call, and the same on both sides of the few tokens' form."""
    import torch
    n, k, r, a = 320, 192, 24, 4
    c = make(m + size, "f16", m, n, k, r, a, "mixed", ranks=False)
    g = torch.Generator(device="cuda").manual_seed(3)
    by_token = torch.exp2(torch.randint(-6, 7, (m, 1), generator=g, device="cuda").double())
    # (first . input) is the low-rank value: forward down . x, in the gradient up^T . dy
    first, second, key, other = ("down", "up", "x", "dy") if forward else ("up", "down", "dy", "x")
    pool, back = 2.0 ** min(max(size / 2, -10), 11), 2.0 ** min(max(-size, -12), 14)
    for q, f in ((first, pool), (second, back), (key, by_token * 2.0 ** min(size - np.log2(pool), 7)),
                 (other, 2.0 ** (max(-size, -12) - 3 if size > 0 else -size // 2 - 8))):
        c[q] = (c[q].double() * f).half()
        assert torch.isfinite(c[q]).all()
    args = (c["down"], c["up"], c["index"], c["scale"])

    def check(have, ref, total, chain):
        inside = ref.abs() < 65000  # (a result past fp16's largest number is infinite)
        assert inside.double().mean() > 0.5
        close(have[inside], ref[inside], total[inside], "f16", chain)
    if forward:
        w = wl.random_24_f16(np.random.default_rng(m), 1, k, n)["Wp"]
        vals, meta = lib.w24_pack_f16(w)
        vals, meta = torch.from_numpy(vals).cuda(), torch.from_numpy(meta.view(np.int32)).cuda()
        delta, total = reference(c)
        base, x, w = c["base"].double(), c["x"].double(), torch.from_numpy(w).cuda().double()
        check(lib.low_rank_add(c["base"], c["x"], *args), base + delta, base.abs() + total, k + r)
        check(lib.w24_low_rank_gemm_f16(c["x"], vals, meta, *args), x @ w + delta, x.abs() @ w.abs() + total, k + r)
    dx, ddown, dup = lib.low_rank_backward(c["dy"], c["x"], *args, base=c["xbase"])
    ref = reference(c, backward=True)
    base = c["xbase"].double()
    check(dx, base + ref[0][0], base.abs() + ref[0][1], n + r)
    check(ddown, *ref[1], n + m)
    check(dup, *ref[2], k + m)


@pytest.mark.parametrize("m", [40, 200])
@pytest.mark.parametrize("r", [8, 24])
def test_opposite_low_rank_values_cancel_exactly(lib, gpu, m, r):
    """Two tokens whose low-rank values are 2^15 and -2^15, just past fp16's own range, with the same other
    side: powers of two throughout, so their gradients' sums are zero to the last bit."""
    import torch
    n = k = 64
    zeros = lambda *s: torch.zeros(*s, dtype=torch.float16, device="cuda")
    x, dy, down, up = zeros(m, k), zeros(m, n), zeros(1, r, k), zeros(1, n, r)
    index = torch.full((m,), -1, dtype=torch.int32, device="cuda")
    index[3] = index[m - 2] = 0
    down[0, :, 0] = up[0, 0, :] = 2.0 ** 7
    for value, same, first, second in (("x", "dy", x, dy), ("dy", "x", dy, x)):
        first[3], first[m - 2], second[3], second[m - 2] = 2.0 ** 8, -2.0 ** 8, 1.0, 1.0
        _, ddown, dup = lib.low_rank_backward(dy, x, down, up, index)
        grad = dup if value == "x" else ddown  # sums low . dy, or dlow . x, over both tokens
        assert (grad == 0).all()
    out = lib.low_rank_add(None, x, down, up, index)  # (x is 1 here: 2^7 . 2^7 . r of every slot)
    assert (out[3, 0] == 2.0 ** 14 * r if 2.0 ** 14 * r < 65504 else torch.isinf(out[3, 0])) and (out[3, 1:] == 0).all()


@pytest.mark.parametrize("m,n,k,r,a,index", [
    (100, 136, 512, 24, 26, "mixed"), (600, 128, 128, 16, 60, "mixed"), (3000, 64, 64, 8, 40, "runs"),
    (6200, 256, 136, 16, 2, "runs"), (5000, 1024, 512, 128, 400, "mixed")])
def test_gradients_of_tokens_of_mixed_sizes(lib, gpu, m, n, k, r, a, index):
    """Low-rank values from 2^-25 to 2^19 within an adapter's tokens: one and several ranges, adapters dealt
    over workgroups, and a large pool's one long range; every call twice the same."""
    import torch
    c = make(m + a, "f16", m, n, k, r, a, index)
    g = torch.Generator(device="cuda").manual_seed(4)
    for key in ("x", "dy"):
        size = torch.exp2(torch.randint(-18, 12, (m, 1), generator=g, device="cuda").double())
        c[key] = (c[key].double() * size).half()
    for key in ("down", "up"):
        size = torch.exp2(torch.randint(-7, 7, (a, 1, 1), generator=g, device="cuda").double())
        c[key] = (c[key].double() * size).half()
    assert all(torch.isfinite(c[q]).all() for q in ("x", "dy", "down", "up"))
    args = (c["dy"], c["x"], c["down"], c["up"], c["index"], c["scale"], c["ranks"], c["xbase"])
    got = lib.low_rank_backward(*args)
    dx, ddown, dup = reference(c, backward=True)
    base = c["xbase"].double()
    for have, ref, total, chain in ((got[0], base + dx[0], base.abs() + dx[1], n + r), (got[1], *ddown, n + m),
                                    (got[2], *dup, k + m)):
        inside = ref.abs() < 65000
        assert inside.double().mean() > 0.5
        close(have[inside], ref[inside], total[inside], "f16", chain)
    for p, q in zip(got, lib.low_rank_backward(*args)):
        assert torch.equal(p, q)
    out = lib.low_rank_add(c["base"], c["x"], *args[2:7])
    delta, total = reference(c)
    ref = c["base"].double() + delta
    inside = ref.abs() < 65000
    close(out[inside], ref[inside], (c["base"].double().abs() + total)[inside], "f16", k + r)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,r,rank", [(60, 8, 8), (60, 24, 13), (200, 8, 8), (200, 24, 13), (200, 128, 100)])
def test_infinite_low_rank_values_follow_the_formula(lib, gpu, dtype, m, r, rank):
    """A token whose input makes its low-rank values infinite gets the formula's infinities of either sign
    (no NaN from a difference of infinities, or from the slots that are not used), in both forms."""
    import torch
    c = make(2, dtype, m, 64, 64, r, 1, 0)
    c["ranks"][0] = rank
    sign = torch.sign(c["up"][0, :, :1])
    c["down"] = c["down"].abs() + 0.5
    c["up"][0] = (c["up"][0].abs() + 0.5) * sign
    c["x"][5] = 1.0
    c["x"][5, 7] = float("inf")
    others = torch.arange(m, device="cuda") != 5
    out = lib.low_rank_add(c["base"], c["x"], c["down"], c["up"], c["index"], c["scale"], c["ranks"])
    assert torch.isfinite(out[others]).all()
    assert torch.equal(out[5].double(), sign[:, 0].double() * float("inf"))


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m", [9, 211])
def test_strides_in_place_and_without_base(lib, gpu, dtype, m):
    import torch
    c = make(8, dtype, m, 328, 136, 16, 3, "mixed", strided=True)
    pool = (c["down"], c["up"], c["index"], c["scale"], c["ranks"])
    flat = {q: c[q].contiguous() for q in ("x", "base", "dy", "xbase")}
    out = lib.low_rank_add(c["base"], c["x"], *pool)
    assert torch.equal(out, lib.low_rank_add(flat["base"], flat["x"], *pool))
    for p, q in zip(lib.low_rank_backward(c["dy"], c["x"], *pool, base=c["xbase"]),
                    lib.low_rank_backward(flat["dy"], flat["x"], *pool, base=flat["xbase"])):
        assert torch.equal(p, q)
    alone = lib.low_rank_add(None, c["x"], *pool)
    assert torch.equal(alone, lib.low_rank_add(torch.zeros_like(flat["base"]), c["x"], *pool))
    lib.low_rank_add(c["base"], c["x"], *pool, out=c["base"])
    assert torch.equal(c["base"], out)
    dx = lib.low_rank_backward(c["dy"], c["x"], *pool, base=c["xbase"])[0]
    lib.low_rank_backward(c["dy"], c["x"], *pool, base=c["xbase"], out=c["xbase"])
    assert torch.equal(c["xbase"], dx)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("m,n,k,r,a,index", [
    (1, 64, 64, 8, 1, 0), (32, 136, 512, 24, 26, "mixed"), (7, 64, 64, 8, 900, "mixed"), (600, 128, 128, 16, 60, "mixed"),
    (5000, 64, 64, 8, 40, "runs")])
def test_backward_with_adapters_dealt_over_workgroups(lib, gpu, dtype, m, n, k, r, a, index):
    """Narrow matrices, where one range of tokens is worked through by several workgroups: every
    adapter's gradient is written once, zeros for those without a token."""
    c = make(m * 5 + a, dtype, m, n, k, r, a, index)
    got = lib.low_rank_backward(c["dy"], c["x"], c["down"], c["up"], c["index"], c["scale"], c["ranks"],
                                base=c["xbase"])
    _, ddown, dup = reference(c, backward=True)
    close(got[1], ddown[0], ddown[1], dtype, n + m, m ** 0.5)
    close(got[2], dup[0], dup[1], dtype, k + m, m ** 0.5)
    unused = [i for i in range(a) if not (c["index"] == i).any()]
    assert (got[1][unused] == 0).all() and (got[2][unused] == 0).all()


def test_no_tokens(lib, gpu):
    import torch
    c = make(9, "bf16", 0, 64, 64, 8, 2, -1)
    assert lib.low_rank_add(c["base"], c["x"], c["down"], c["up"], c["index"]).shape == (0, 64)
    dx, ddown, dup = lib.low_rank_backward(c["dy"], c["x"], c["down"], c["up"], c["index"])
    assert dx.shape == (0, 64) and (ddown == 0).all() and (dup == 0).all()


def test_gradients_against_differences(lib, gpu):
    """Central differences of the 64-bit forward formula through the returned gradients: the loss
    sum(dy * delta) is linear in x, in down and in up, so a difference along one of them is exact."""
    import torch
    c = make(10, "f16", 150, 64, 48, 8, 2, "mixed", ranks=False)
    got = lib.low_rank_backward(c["dy"], c["x"], c["down"], c["up"], c["index"], c["scale"], None)
    g = torch.Generator(device="cuda").manual_seed(1)
    for key, grad in (("x", got[0]), ("down", got[1]), ("up", got[2])):
        way = torch.randn(c[key].shape, generator=g, device="cuda").double()
        loss = []
        for sign in (1, -1):
            d = dict(c, **{key: c[key].double() + sign * way})
            loss.append((d["dy"].double() * reference(d)[0]).sum())
        diff = (loss[0] - loss[1]) / 2
        # every entry of the gradient was rounded once to fp16 (2^-11) from sums good to 2^-19
        bound = (2.0 ** -11 + 2.0 ** -19) * (grad.double() * way).abs().sum() + 1e-6
        assert (diff - (grad.double() * way).sum()).abs() <= bound


def test_repeatable_and_on_another_stream(lib, gpu):
    import torch
    c = make(11, "f16", 3000, 512, 256, 16, 5, "runs")
    call = lambda: (lib.low_rank_add(c["base"], c["x"], c["down"], c["up"], c["index"], c["scale"]),
                    *lib.low_rank_backward(c["dy"], c["x"], c["down"], c["up"], c["index"], c["scale"], None, c["xbase"]))
    first = call()
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        again = call()
    torch.cuda.current_stream().wait_stream(st)
    for p, q in zip(first, again):
        assert torch.equal(p, q)


def test_refusals(lib, gpu):
    import torch
    c = make(12, "f16", 200, 64, 64, 16, 2, "mixed")
    pool = (c["down"], c["up"], c["index"])
    with pytest.raises(TypeError):
        lib.low_rank_add(c["base"], c["x"].float(), *pool)
    with pytest.raises(TypeError):
        lib.low_rank_add(c["base"], c["x"], c["down"], c["up"], c["index"].long())
    with pytest.raises(ValueError):
        lib.low_rank_add(c["base"], c["x"], c["down"], c["up"], c["index"][:-1].contiguous())
    with pytest.raises(TypeError):
        lib.low_rank_add(c["base"], c["x"], c["down"].bfloat16(), c["up"], c["index"])
    with pytest.raises(lib.SsgError, match="multiple of 8"):
        lib.low_rank_add(c["base"], c["x"], c["down"][:, :12].contiguous(), c["up"][:, :, :12].contiguous(), c["index"])
    with pytest.raises(lib.SsgError, match="row stride"):
        wide = torch.zeros((200, 68), device="cuda").half()
        lib.low_rank_add(c["base"], wide[:, :64], *pool)
    with pytest.raises(lib.SsgError, match="aligned"):
        wide = torch.zeros((200, 72), device="cuda").half()
        lib.low_rank_add(c["base"], wide[:, 4:68], *pool)
    with pytest.raises(lib.SsgError, match="workspace"):
        lib.low_rank_add(c["base"], c["x"], *pool, workspace=torch.empty(32, dtype=torch.uint8, device="cuda"))
    with pytest.raises(lib.SsgError, match="multiples of 8"):
        lib.low_rank_add(c["base"][:, :60], c["x"], c["down"], c["up"][:, :60].contiguous(), c["index"])
    with pytest.raises(lib.SsgError, match="multiple of 64"):
        y = torch.zeros((96, 32), device="cuda").half()
        lib.w24_low_rank_gemm_f16(c["x"], y, torch.zeros((96, 2), dtype=torch.int32, device="cuda"), c["down"],
                                  torch.zeros((2, 96, 16), device="cuda").half(), c["index"])
