"""Ends of the routing and of the adapters: where memory ends, whose bits depend on what,
and bits that the small pieces of sums hold.  Oracle and tolerances as in
tests/test_gpu_route.py and tests/test_gpu_lora.py, or derived at the test."""
import numpy as np
import pytest

from oracle import serve_oracle as S
from tests import _gpu as G
from tests import test_gpu_lora as L
from tests import test_gpu_route as R

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# routing
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("t,experts,topk,groups,topk_groups", [(1 << 21, 2, 2, 1, 1), (2048, 2, 2, 1, 1),
                                                               (1 << 20, 4, 1, 4, 2), (1 << 19, 8, 3, 2, 1),
                                                               (1 << 18, 16, 5, 8, 3)])
def test_route_logits_that_end_with_their_memory(t, experts, topk, groups, topk_groups, scoring):
    """Balanced scores of fewer allowed experts than the lists of choices hold: the lanes
    past the choices hold no expert, and read no logit of one.  16 MB (16 KB in one case)
    of logits, behind which their memory ends."""
    import torch
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(experts)
    rule = R.rule_of(experts, topk, rng.standard_normal(experts) * 0.1, scoring=scoring, groups=groups,
                     topk_groups=topk_groups)
    l = (rng.standard_normal((400, experts)) * 1.5).astype(np.float32)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    buf = torch.zeros((t, experts), device=G.dev())
    buf[-400:] = G.to_dev(l)
    ids, w = X.exl3_route_topk(buf, rule)
    R.check(ids[-400:], w[-400:], l, rule)


@pytest.mark.parametrize("t", [5, 2100])
@pytest.mark.parametrize("balanced", [False, True])
@pytest.mark.parametrize("experts,topk,groups,topk_groups", [(576, 16, 64, 5), (64, 8, 64, 9), (128, 4, 64, 3),
                                                             (66, 5, 33, 4), (576, 8, 64, 63), (192, 8, 64, 7)])
def test_route_many_small_groups(experts, topk, groups, topk_groups, balanced, t):
    """Places past the experts, up to the next size that lanes hold, are of no group: their
    number may be past 64."""
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(experts + t)
    l = (rng.standard_normal((t, experts)) * 1.5).astype(np.float32)
    rule = R.rule_of(experts, topk, rng.standard_normal(experts) * 0.1 if balanced else None, scoring="sigmoid",
                     groups=groups, topk_groups=topk_groups)
    ids, w = X.exl3_route_topk(G.to_dev(l), rule)
    R.check(ids, w, l, rule)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("scoring,balanced,group_score", [("softmax", False, "max"), ("softmax", True, "max"),
                                                          ("softmax", True, "top2"), ("softmax", False, "top2"),
                                                          ("sigmoid", True, "top2"), ("sigmoid", False, "max")])
@pytest.mark.parametrize("experts,topk,groups,topk_groups", [(256, 8, 8, 4), (256, 16, 1, 1), (250, 3, 1, 1),
                                                             (160, 6, 8, 3), (128, 8, 4, 2), (96, 4, 2, 1),
                                                             (65, 8, 1, 1), (64, 6, 1, 1), (60, 4, 4, 2), (33, 2, 1, 1),
                                                             (8, 8, 1, 1), (5, 1, 1, 1), (300, 5, 1, 1)])
def test_a_tokens_route_does_not_depend_on_the_others(experts, topk, groups, topk_groups, scoring, balanced,
                                                      group_score, f32):
    """The same bits among thousands of tokens, among a few and alone."""
    import torch
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(experts + topk)
    b = rng.standard_normal(experts) * (0.1 if scoring == "sigmoid" else 0.5 / experts) if balanced else None
    rule = R.rule_of(experts, topk, b, scoring=scoring, groups=groups, topk_groups=topk_groups,
                     group_score=group_score, renormalize=topk % 2 == 0)
    l = G.to_dev((rng.standard_normal((4500, experts)) * 1.5).astype(np.float32 if f32 else np.float16))
    ids, w = X.exl3_route_topk(l, rule)
    for rows in (slice(0, 2049), slice(0, 2048), slice(2048, 4096), slice(4096, 4500), slice(7, 8), slice(4499, 4500)):
        i, v = X.exl3_route_topk(l[rows], rule)
        assert torch.equal(i, ids[rows]), rows
        assert torch.equal(v, w[rows]), rows


def test_a_tokens_route_beside_bad_tokens():
    """Tokens of the same wave with NaN and infinite logits leave a token's bits alone."""
    import torch
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(2)
    for experts in (60, 256):
        for scoring in ("softmax", "sigmoid"):
            rule = R.rule_of(experts, 6, rng.standard_normal(experts) * 0.1, scoring=scoring, groups=4, topk_groups=2,
                             group_score="top2")
            l = (rng.standard_normal((4096, experts)) * 1.5).astype(np.float32)
            want = X.exl3_route_topk(G.to_dev(l), rule)
            bad = l.copy()
            bad[1::4, 3], bad[2::4, ::5], bad[3::8, 7] = np.nan, -np.inf, np.inf
            for t in (4096, 2000):
                got = X.exl3_route_topk(G.to_dev(bad[:t]), rule)
                for a, b in zip(got, want):
                    assert torch.equal(a[::4], b[:t:4])


def near_bound(w, l, scoring):
    """As tests/test_gpu_route.py's, with the span of one token's logits that can have a
    say: a softmax's terms 110 below its largest are below 2^-158, and a sigmoid, which
    takes no difference of logits, has none."""
    finite = l[np.isfinite(l)]
    span = 0.0
    if scoring == "softmax" and finite.size:
        span = float(finite.max() - finite[finite >= finite.max() - 110].min())
    return (2 * span + 44) * 2.0 ** -24 * np.abs(w) + 2.0 ** -120


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("experts", [8, 60, 256, 1024])
def test_route_weights_beside_masks_of_the_lowest_value(experts, renormalize, scoring):
    """Weights of tokens with masked, far and infinite logits, each within the bound of its
    own token, and masks of the type's lowest value give the bits of infinite ones."""
    import torch
    import gemm_exl3_linear_amd as X
    for f32 in (True, False):
        l = R.special_logits(experts)
        l = np.delete(l, [7, 15] if renormalize else [], axis=0)  # weights divided by a sum of subnormals, or of 0
        if not f32:
            l = np.clip(l, np.finfo(np.float16).min, np.finfo(np.float16).max,
                        where=np.isfinite(l), out=l.copy()).astype(np.float16)
        rule = R.rule_of(experts, 4, None, scoring=scoring, renormalize=renormalize, scale=2.5)
        ids, w = X.exl3_route_topk(G.to_dev(l), rule)
        ref_ids, ref = S.route(l, 4, scoring, renormalize=renormalize, scale=2.5)
        np.testing.assert_array_equal(ids.cpu().numpy(), ref_ids)
        got = w.cpu().numpy().astype(np.float64)
        for i, row in enumerate(l.astype(np.float64)):
            np.testing.assert_array_equal(np.isnan(got[i]), np.isnan(ref[i]))
            ok = ~np.isnan(ref[i])
            assert (np.abs(got[i] - ref[i])[ok] <= near_bound(ref[i], row, scoring)[ok]).all(), (i, got[i], ref[i])
        # masks
        rng = np.random.default_rng(experts)
        dt = np.float32 if f32 else np.float16
        l = (rng.standard_normal((40, experts)) * 1.5).astype(dt)
        masked = rng.random(l.shape) < 0.5
        masked[::5] = True
        masked[::5, experts // 2] = False
        b = rng.standard_normal(experts) * 0.1
        for balance in (None, b):
            rule = R.rule_of(experts, 4, balance, scoring=scoring, renormalize=renormalize)
            low = X.exl3_route_topk(G.to_dev(np.where(masked, np.finfo(dt).min, l)), rule)
            inf = X.exl3_route_topk(G.to_dev(np.where(masked, dt(-np.inf), l)), rule)
            assert torch.equal(low[0], inf[0])  # 0 / 0 is NaN on either side
            assert torch.equal(low[1].view(torch.int32), inf[1].view(torch.int32))


# both in a call: tokens in one launch, in rows, in tiles, in shares of either, past 2048
@pytest.mark.parametrize("scoring,balanced,group_score", [("softmax", False, "max"), ("softmax", True, "top2"),
                                                          ("sigmoid", True, "max")])
@pytest.mark.parametrize("t,hidden,experts", [(1, 2048, 256), (4, 2048, 256), (3, 520, 40), (16, 5120, 256),
                                              (16, 1024, 60), (9, 4096, 1000), (33, 2048, 256), (64, 5120, 256),
                                              (333, 1440, 60), (700, 4104, 130), (2049, 5120, 60), (4000, 5120, 60),
                                              (2500, 264, 256)])
def test_router_routes_its_own_logits(t, hidden, experts, scoring, balanced, group_score):
    """The choices and weights of exl3_router are the bits of exl3_route_topk of its
    logits, the same without memory for them, and the logits exl3_router_linear's to
    rounding: the bound of either, twice."""
    import torch
    import gemm_exl3_linear_amd as X
    x, w, c = R.router_case(t, hidden, experts, True, seed=21)
    rng = np.random.default_rng(t)
    b = rng.standard_normal(experts) * (0.1 if scoring == "sigmoid" else 0.5 / experts) if balanced else None
    groups = 4 if experts % 4 == 0 else 1
    rule = R.rule_of(experts, 5, b, scoring=scoring, groups=groups, topk_groups=max(1, groups // 2),
                     group_score=group_score, scale=2.5)
    r, xd = R.handle(w, c), G.to_dev(x)
    logits = torch.full((t, experts + 3), 7.0, device=G.dev())
    ids, wt = X.exl3_router(xd, r, rule, logits=logits[:, :experts])
    for got in (X.exl3_route_topk(logits[:, :experts], rule), X.exl3_route_topk(logits[:, :experts].contiguous(), rule),
                X.exl3_router(xd, r, rule)):
        assert torch.equal(ids, got[0]) and torch.equal(wt, got[1])
    apart = X.exl3_router_linear(xd, r)
    _, mag = S.logits(x, w, c)
    assert (np.abs((apart.double() - logits[:, :experts].double()).cpu().numpy()) <= 2 * R.logit_bound(mag, hidden)).all()


# ---------------------------------------------------------------------------
# adapters: what is kept of A x between the two products
# ---------------------------------------------------------------------------
# rows and adapters by the kernels they take: segments of 16 found by ballots, by search
# and by the plan, of 64 by search and by the plan
SEGMENTS = [(20, 3), (333, 40), (1100, 300), (600, 3), (2100, 2)]


@pytest.mark.parametrize("m,adapters", SEGMENTS)
@pytest.mark.parametrize("rank", [8, 16, 24, 32, 40, 64, 104, 128, 256])
def test_lora_keeps_the_low_bits_of_the_inner_sums(rank, m, adapters):
    """Whole numbers again, with inner sums that need more than the 11 bits of one fp16:
    sums below 2^24 are exact in two pieces, and in fp32 in any order.  One piece would
    give other sums (checked here)."""
    import torch
    import gemm_exl3_linear_amd as X
    g = torch.Generator(device=G.dev()).manual_seed(rank * 7 + m)
    whole = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device=G.dev())
    k = 104
    for n in (8, 70, 521):
        x, a = whole(-40, 41, m, k).half(), whole(-40, 41, adapters, rank, k).half()
        b, rows = whole(-1, 2, adapters, n, rank).half(), whole(-1, adapters, m).int()
        base = whole(-99, 100, m, n).float()
        ref, one = base.double(), base.double()
        most = 0.0
        for i in range(adapters):
            mine = rows == i
            h = x[mine].double() @ a[i].double().T
            most = max(most, float(h.abs().sum(-1).max()) if h.numel() else 0.0)
            ref[mine] += h @ b[i].double().T
            step = torch.exp2(torch.floor(torch.log2(h.abs().clamp(min=1))) - 10)
            one[mine] += (torch.round(h / step) * step) @ b[i].double().T
        assert most + 99 < 2 ** 24 and not torch.equal(one, ref)
        y = X.exl3_lora(x, X.Exl3Lora(a, b), rows, base)
        assert torch.equal(y.double(), ref), n


@pytest.mark.parametrize("m,adapters", SEGMENTS)
@pytest.mark.parametrize("rank", [8, 16, 24, 32, 64, 128, 256])
def test_lora_keeps_small_inner_sums_beside_large_ones(rank, m, adapters):
    """B is the unit matrix, so that y_c is the kept value of (A x)_c, whose sums of two
    products are exact in fp32.  Kept: each within 2^-23 of itself down to 2^-29 of the
    row's largest, below that within 2^-51 of the largest; and a rounding of the sum of
    the pieces, 2^-24."""
    import torch
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(rank + m)
    k, n = 72, rank
    x = np.zeros((m, k))
    x[:, 3], x[:, 70] = 1.0, 2.0 ** -12
    a = np.zeros((adapters, rank, k))
    size = np.exp2(rng.integers(-22, 5, (adapters, rank)))  # the least fp16 that holds 11 bits: 2^-24 * 1024
    size[:, rng.integers(rank)] = 2.0 ** 5
    sign = rng.choice([-1.0, 1.0], (adapters, rank))
    a[:, :, 3] = sign * rng.integers(1024, 2048, (adapters, rank)) * size
    a[:, :, 70] = rng.integers(-2047, 2048, (adapters, rank)) * size
    b = np.broadcast_to(np.eye(rank), (adapters, n, rank))
    a16, x16 = a.astype(np.float16), x.astype(np.float16)
    assert (a16 == a).all() and (x16 == x).all()
    rows = rng.integers(0, adapters, m).astype(np.int32)
    h = np.einsum("mk,mrk->mr", x[:, [3, 70]], a[rows][:, :, [3, 70]])
    assert (h == h.astype(np.float32)).all()
    lora = X.Exl3Lora(G.to_dev(a16), G.to_dev(b.astype(np.float16).copy()))
    y = X.exl3_lora(G.to_dev(x16), lora, G.to_dev(rows), out_dtype=torch.float32).cpu().numpy().astype(np.float64)
    top = np.abs(h).max(-1, keepdims=True)
    assert (np.abs(h) < top * 2.0 ** -22).any() and (np.abs(h) > 0).all()
    limit = np.where(np.abs(h) >= top * 2.0 ** -29, 2.0 ** -23 * np.abs(h), 2.0 ** -51 * top) + 2.0 ** -24 * np.abs(h)
    bad = np.abs(y - h) > limit
    assert not bad.any(), (f"{bad.sum()} of {bad.size}: {y[bad][0]!r} for {h[bad][0]!r}, "
                           f"row's largest {np.broadcast_to(top, h.shape)[bad][0]!r}")


@pytest.mark.parametrize("m,adapters", SEGMENTS)
@pytest.mark.parametrize("rank", [8, 16, 32, 40, 128, 256])
@pytest.mark.parametrize("weight", [2.0 ** -24, 2.0 ** -22, 2.0 ** -16, 1.0])
def test_lora_inner_sums_times_subnormal_weights(weight, rank, m, adapters):
    """y_c is one inner sum of 22 bits times one weight, a power of two: the inner sum
    kept to 2^-23, and the sum of its pieces' products.  Those are exact for the high
    piece (its last place times the weight's is at least 2^-21, and a matrix instruction
    cuts about 2^-24 of an fp16 of exponent 14 times a subnormal); the low piece's are cut
    there too, which its factor makes 2^-36 beside a result of 2^-11 at least.  One
    rounding, 2^-24."""
    import torch
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(rank + m)
    k, n = 72, rank + 3
    x, a = np.zeros((m, k)), np.zeros((adapters, rank, k))
    x[:, 5], a[:, :, 5] = rng.integers(1024, 2048, m), rng.integers(1024, 2048, (adapters, rank))
    b = np.zeros((adapters, n, rank))
    b[:, :rank] = np.eye(rank) * weight
    rows = (np.arange(m) % adapters).astype(np.int32)
    want = np.zeros((m, n))
    want[:, :rank] = x[:, 5:6] * a[rows][:, :, 5] * weight
    lora = X.Exl3Lora(*(G.to_dev(v.astype(np.float16)) for v in (a, b)))
    y = X.exl3_lora(G.to_dev(x.astype(np.float16)), lora, G.to_dev(rows), out_dtype=torch.float32).cpu().numpy()
    bad = np.abs(y - want) > 4 * 2.0 ** -24 * want
    assert not bad.any(), f"{bad.sum()} of {bad.size}: {y[bad][0]!r} for {want[bad][0]!r}"


@pytest.mark.parametrize("m,adapters", [(1, 4)] + SEGMENTS)
@pytest.mark.parametrize("rank", [8, 40, 256])
def test_lora_scales_at_the_ends_of_fp32(rank, m, adapters):
    """Adapter i has a large scale and small weights, or a small one and large weights,
    or columns of B that are 0 beside inner sums and a scale of any size: results inside
    fp32 are right, and 0 stays 0.  y_c is one inner sum, kept to 2^-23 of itself, times
    one weight, one scale: three roundings of 2^-24 more."""
    import torch
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(rank + m)
    k, n = 72, rank + 3
    x, a = np.zeros((m, k)), np.zeros((adapters, rank, k))
    b, scales = np.zeros((adapters, n, rank)), np.zeros(adapters, dtype=np.float32)
    x[:, 5] = rng.integers(1024, 2048, m)                        # [2^10, 2^11)
    kinds = np.arange(adapters) % 4
    a[:, :, 5] = rng.integers(1024, 2048, (adapters, rank))
    for i, kind in enumerate(kinds):
        h = (2.0 ** 4, 2.0 ** -22, 2.0 ** 4, 2.0 ** -20)[kind]   # inner sums about 2^25, 2^-1, 2^25, 2
        a[i] *= h
        w = (2.0 ** -22, 2.0 ** 15, 0.0, 2.0 ** 14)[kind]
        b[i, :rank] = np.eye(rank) * w
        scales[i] = np.float32((1.1 * 2.0 ** 120, 1.1 * 2.0 ** -125, 3e38, 1.1 * 2.0 ** 110)[kind])
    a16, b16, x16 = a.astype(np.float16), b.astype(np.float16), x.astype(np.float16)
    assert (a16 == a).all() and (b16 == b).all() and (x16 == x).all()
    rows = (np.arange(m) % adapters).astype(np.int32)
    want = np.zeros((m, n))
    want[:, :rank] = (x[:, 5:6] * a[rows][:, :, 5]) * b[rows][:, np.arange(rank), np.arange(rank)]
    want *= scales[rows].astype(np.float64)[:, None]
    assert (np.abs(want[want != 0]) < 2.0 ** 127).all() and (np.abs(want[want != 0]) > 2.0 ** -126).all()
    lora = X.Exl3Lora(G.to_dev(a16), G.to_dev(b16), scales=G.to_dev(scales))
    y = X.exl3_lora(G.to_dev(x16), lora, G.to_dev(rows), out_dtype=torch.float32).cpu().numpy().astype(np.float64)
    assert (y[want == 0] == 0).all()
    bad = ~(np.abs(y - want) <= 5 * 2.0 ** -24 * np.abs(want))
    assert not bad.any(), f"{bad.sum()} of {bad.size}: {y[bad][0]!r} for {want[bad][0]!r}"


# ---------------------------------------------------------------------------
# the largest sizes
# ---------------------------------------------------------------------------
def test_route_of_the_most_tokens():
    """2^24 tokens: the bits of a sixteenth at a time, and the oracle at the last."""
    import torch
    import gemm_exl3_linear_amd as X
    t, experts = 1 << 24, 5
    g = torch.Generator(device=G.dev()).manual_seed(3)
    l = torch.randn(t, experts, generator=g, device=G.dev()).half()
    rule = R.rule_of(experts, 2, np.random.default_rng(3).standard_normal(experts) * 0.1, scoring="softmax")
    ids, w = X.exl3_route_topk(l, rule)
    for i in range(0, t, t // 16):
        part = X.exl3_route_topk(l[i:i + t // 16], rule)
        assert torch.equal(part[0], ids[i:i + t // 16]) and torch.equal(part[1], w[i:i + t // 16])
    # fp16 logits that are equal give s + b of two experts that may be, to rounding: none here
    R.check(ids[-500:], w[-500:], l[-500:].cpu().numpy().astype(np.float64), rule)


@pytest.mark.parametrize("t,hidden,experts", [(1 << 24, 8, 3), ((1 << 20) + 5, 64, 70), (3, 65536, 1024),
                                              (40, 65536, 1024)])
def test_router_of_the_largest_sizes(t, hidden, experts):
    """Whole numbers, whose sums are exact; choices by the logits' order."""
    import torch
    import gemm_exl3_linear_amd as X
    g = torch.Generator(device=G.dev()).manual_seed(experts)
    x = torch.randint(-2, 3, (t, hidden), generator=g, device=G.dev(), dtype=torch.int8).half()
    w = torch.randint(-2, 3, (experts, hidden), generator=g, device=G.dev(), dtype=torch.int8).half()
    r, rule = X.Exl3Router(w), X.Exl3RouteRule(experts, min(2, experts))
    logits = torch.empty((t, experts), device=G.dev())
    ids, wt = X.exl3_router(x, r, rule, logits=logits)
    apart = X.exl3_router_linear(x, r)
    step = min(t, 1 << 20)
    for i in range(0, t, step):
        ref = x[i:i + step].double() @ w.double().t()
        assert torch.equal(logits[i:i + step].double(), ref) and torch.equal(apart[i:i + step].double(), ref)
        order = torch.sort(ref, dim=-1, descending=True, stable=True).indices[:, :rule.topk]
        assert torch.equal(ids[i:i + step].long(), order)
    again = X.exl3_route_topk(logits, rule)
    assert torch.equal(again[0], ids) and torch.equal(again[1], wt)


@pytest.mark.parametrize("m,k,n,rank,adapters", [(1 << 24, 8, 9, 8, 3), (1 << 24, 8, 1, 8, 2), (1 << 21, 8, 5, 8, 4096),
                                                 (5, 1 << 20, 64, 8, 2), (70, 64, 1 << 20, 16, 2),
                                                 (600, 64, 1 << 20, 256, 1)])
def test_lora_of_the_largest_sizes(m, k, n, rank, adapters):
    """Whole numbers below 2^24 at every step (k 4 times rank at most), in place."""
    import torch
    import gemm_exl3_linear_amd as X
    g = torch.Generator(device=G.dev()).manual_seed(adapters)
    whole = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device=G.dev(), dtype=torch.int8)
    x, a, b = whole(-1, 2, m, k).half(), whole(-1, 2, adapters, rank, k).half(), whole(-1, 2, adapters, n, rank).half()
    rows = torch.randint(-1, adapters, (m,), generator=g, device=G.dev()).int()
    base = whole(-9, 10, m, n)
    y = base.float()
    X.exl3_lora(x, X.Exl3Lora(a, b), rows, y, out=y)
    step = max(1, min(m, (1 << 24) // max(n, k)))
    if adapters > 100:  # one product a row
        ref = lambda i, r: torch.bmm(b[r].float(), torch.bmm(a[r].float(), x[i].float().unsqueeze(-1))).squeeze(-1)
    for i0 in range(0, m, step):
        want = base[i0:i0 + step].double()
        if adapters > 100:
            for j in range(i0, min(m, i0 + step), 1 << 16):
                i = torch.arange(j, min(m, i0 + step, j + (1 << 16)), device=G.dev())
                i = i[rows[i] >= 0]
                want[i - i0] += ref(i, rows[i].long()).double()
        else:
            for e in range(adapters):
                mine = rows[i0:i0 + step] == e
                want[mine] += ((x[i0:i0 + step][mine].float() @ a[e].float().t()).double() @ b[e].double().t())
        assert torch.equal(y[i0:i0 + step].double(), want), i0
