"""Routing to experts on the GPU against the float64 oracle.

Tolerances.  Logits: products are exact in fp32 (22 significand bits); a sum over h
goes through the matrix cores in blocks of at least 32 and then through fp32 additions,
so, as for the other fp16 products of this library, |l - l64| <= 2 (h/32 + 104) 2^-24
sum |x||w|.  Choices are exact: whole numbers, equal to the oracle's, which compares in
64 bits (two random values closer than the library's 2^-42 do not occur in these inputs:
a few million pairs).  Weights, relative: the exponent l - max is rounded once, which is
worth R 2^-24 for a range R of the logits, in the numerator and in the sum; each
exponential is off by up to 2^-22 (two ulps); a sum of up to 1024 positive terms in a
tree and in runs of 16 takes at most 24 roundings, the sum of the chosen 6; divisions and
the factor three times two roundings: (2 R + 2 * 4 + 24 + 6 + 6) 2^-24 <= (2 R + 44)
2^-24.  Below the normals 2^-126 of any exponential may be lost, 2^-120 of a weight."""
import numpy as np
import pytest

from oracle import serve_oracle as S
from tests import _gpu as G

pytestmark = pytest.mark.gpu


def logit_bound(mag, hidden):
    return 2 * (hidden / 32 + 104) * 2.0 ** -24 * mag + 2.0 ** -149


def weight_bound(w, logits):
    finite = logits[np.isfinite(logits)]
    span = float(finite.max() - finite.min()) if finite.size else 0.0
    return (2 * span + 44) * 2.0 ** -24 * np.abs(w) + 2.0 ** -120


def oracle(logits, rule):
    b = None if rule.balance is None else rule.balance.cpu().numpy()
    return S.route(logits, rule.topk, rule.scoring, b, rule.groups, rule.topk_groups, rule.group_score,
                   rule.renormalize, rule.scale)


def check(ids, weights, logits, rule, what=""):
    """logits: what the library routed, as numpy."""
    ref_ids, ref_w = oracle(logits, rule)
    np.testing.assert_array_equal(ids.cpu().numpy(), ref_ids, err_msg=f"{what} ids")
    got = weights.cpu().numpy().astype(np.float64)
    np.testing.assert_array_equal(np.isnan(got), np.isnan(ref_w), err_msg=f"{what} NaN weights")
    ok = ~np.isnan(ref_w)
    bad = ok & ~(np.abs(got - np.where(ok, ref_w, 0)) <= weight_bound(np.where(ok, ref_w, 0), logits))
    assert not bad.any(), f"{what} {bad.sum()} weights, first {got[bad][0]!r} for {ref_w[bad][0]!r}"


def rule_of(experts, topk, balance=None, **kw):
    import gemm_exl3_linear_amd as X
    return X.Exl3RouteRule(experts, topk, balance=None if balance is None else G.to_dev(balance.astype(np.float32)),
                           **kw)


RULES = [  # t, experts, topk, groups, topk_groups, group_score
    (1, 1, 1, 1, 1, "max"), (3, 4, 4, 1, 1, "max"), (5, 7, 3, 1, 1, "max"), (64, 60, 4, 1, 1, "max"),
    (9, 64, 6, 1, 1, "max"), (33, 65, 8, 1, 1, "max"), (17, 128, 16, 1, 1, "max"), (100, 256, 8, 1, 1, "max"),
    (7, 257, 9, 1, 1, "max"), (13, 500, 2, 1, 1, "max"), (6, 1000, 16, 1, 1, "max"), (21, 1024, 8, 1, 1, "max"),
    (40, 256, 8, 8, 4, "top2"), (40, 256, 8, 8, 3, "max"), (11, 160, 6, 8, 3, "max"), (19, 60, 4, 15, 4, "top2"),
    (23, 60, 9, 4, 1, "top2"), (8, 64, 16, 32, 9, "max"), (8, 64, 3, 64, 3, "max"), (15, 128, 16, 64, 8, "top2"),
    (10, 1024, 8, 64, 5, "top2"), (12, 1020, 16, 17, 2, "top2"), (31, 16, 2, 8, 1, "top2"), (14, 48, 5, 16, 16, "max"),
    (4099, 256, 8, 1, 1, "max"), (1025, 256, 8, 8, 4, "top2"), (2051, 60, 4, 1, 1, "max"), (777, 512, 8, 1, 1, "max"),
]


@pytest.mark.parametrize("balanced", [False, True])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("t,experts,topk,groups,topk_groups,group_score", RULES)
def test_route(t, experts, topk, groups, topk_groups, group_score, scoring, balanced):
    import torch
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(t * 7 + experts * 3 + topk)
    l = (rng.standard_normal((t, experts)) * 1.5).astype(np.float32)
    b = rng.standard_normal(experts) * (0.1 if scoring == "sigmoid" else 0.5 / experts) if balanced else None
    rule = rule_of(experts, topk, b, scoring=scoring, groups=groups, topk_groups=topk_groups, group_score=group_score,
                   renormalize=bool(t % 2), scale=1.0 if t % 3 else 2.5)
    ids, w = X.exl3_route_topk(G.to_dev(l), rule)
    assert ids.dtype == torch.int32 and w.dtype == torch.float32
    check(ids, w, l, rule)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("pad,offset", [(0, 0), (1, 0), (3, 1), (8, 0), (64, 5)])
def test_route_strided_logits(f32, pad, offset):
    import torch
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(pad + offset)
    for t, experts in ((1, 256), (5, 60), (70, 256), (33, 1024)):
        dt = np.float32 if f32 else np.float16
        buf = (rng.standard_normal((t, experts + pad + offset)) * 2).astype(dt)
        rule = rule_of(experts, min(8, experts))
        ids, w = X.exl3_route_topk(G.to_dev(buf)[:, offset:offset + experts], rule)
        check(ids, w, buf[:, offset:offset + experts].astype(np.float64), rule, f"{t} {experts}")


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,topk_groups,group_score", [(1, 1, "max"), (4, 2, "max"), (4, 2, "top2")])
def test_route_equal_values_go_to_the_lower(scoring, groups, topk_groups, group_score):
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(3)
    for experts in (16, 64, 256, 1024):
        l = rng.integers(-2, 3, (50, experts)).astype(np.float32)
        l[:3] = np.array([[0.0], [-0.0], [5.0]])
        l[3] = np.where(np.arange(experts) % 2, 0.0, -0.0)
        l[4] = -7.5
        for b in (None, np.zeros(experts), rng.integers(-1, 2, experts)):
            if b is not None and scoring == "softmax" and b.any():
                continue  # s + 1 and s + 1 of other rows: equal or not by a rounding of the softmax
            rule = rule_of(experts, 8, b, scoring=scoring, groups=groups, topk_groups=topk_groups,
                           group_score=group_score)
            ids, w = X.exl3_route_topk(G.to_dev(l), rule)
            check(ids, w, l, rule, f"{experts}")


def test_route_values_that_32_bits_cannot_tell_apart():
    """sigmoid(l) + b for b of 1: scores of 1.5e-8, the next best about 2^-36 below, which
    fp32 rounds to the same value.  The values are compared to 42 significant bits: each
    is cut by less than 2^-42 of itself, so two that lie more than 2^-42 |v| apart, with
    2^-50 |v| for the 64-bit arithmetic of either side, are told apart, and a sum of two
    cut ones is off by less than 2^-42 of itself and cut once more.  Rows in which a
    neighbouring pair among the best lies closer than 2^-41 |v|, or the grades about the
    last kept group closer than 2^-40 |grade|, are open, and left out (about 5 in 100)."""
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(5)
    for experts in (60, 256, 1024):
        l = (-18.0 + rng.standard_normal((64, experts)) * 1e-2).astype(np.float32)
        b = np.ones(experts, dtype=np.float32)
        for groups, tg, score in ((1, 1, "max"), (4, 2, "top2")):
            rule = rule_of(experts, 8, b, scoring="sigmoid", groups=groups, topk_groups=tg, group_score=score)
            ids, w = X.exl3_route_topk(G.to_dev(l), rule)
            v = 1.0 / (1.0 + np.exp(-l.astype(np.float64))) + 1.0
            clear = np.ones(64, dtype=bool)
            if groups > 1:
                parts = v.reshape(64, groups, -1)
                grade = np.sort(np.sort(parts, -1)[..., -2:].sum(-1), -1)[:, ::-1]
                clear &= grade[:, tg - 1] - grade[:, tg] > 2.0 ** -40 * grade[:, tg]
                kept = np.zeros((64, groups), dtype=bool)
                order = np.argsort(-np.sort(parts, -1)[..., -2:].sum(-1), axis=-1, kind="stable")[:, :tg]
                np.put_along_axis(kept, order, True, axis=1)
                v = np.where(np.repeat(kept, experts // groups, axis=1), v, 0.0)
            best = np.sort(v, -1)[:, ::-1][:, :9]
            clear &= (best[:, :-1] - best[:, 1:] > 2.0 ** -41 * best[:, 1:]).all(1)
            assert clear.sum() >= 40
            assert np.float32(best[:, 0]).max() == np.float32(best[:, 8]).min()  # one value in fp32
            for i in np.flatnonzero(clear):
                check(ids[i:i + 1], w[i:i + 1], l[i:i + 1], rule, f"{experts} {groups} row {i}")


def special_logits(experts):
    rng = np.random.default_rng(experts)
    l = (rng.standard_normal((24, experts)) * 1.5).astype(np.float32)
    inf, nan = np.inf, np.nan
    l[0, ::2] = -inf                       # masked experts
    l[1, 1:] = -inf                        # one expert left
    l[2] = -inf                            # none left
    l[3, 5 % experts] = nan
    l[4] = nan
    l[5, 2 % experts] = inf
    l[6, ::3], l[6, 1::3] = -inf, inf
    l[7, ::3], l[7, 1::3] = nan, -inf
    l[8] = np.finfo(np.float32).min        # masks of the type's lowest value
    l[9, 1:] = np.finfo(np.float32).min
    l[10, ::2] = np.finfo(np.float32).min
    l[11] = 3e38
    l[12] = np.where(np.arange(experts) % 2, 1e-45, -1e-45)  # subnormals
    l[13] = l[13] * 1e-40
    l[14] = l[14] * 1e4
    l[15] = -100 + l[15]                   # sigmoids below the normals
    l[16] = 100 + l[16]                    # sigmoids of 1
    l[17, : experts // 2] = -inf           # whole groups masked
    l[18, : experts // 2] = nan
    l[19, experts // 4:] = nan
    l[20, experts // 4:] = -inf
    return l


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,topk_groups,group_score", [(1, 1, "max"), (4, 2, "max"), (4, 2, "top2")])
@pytest.mark.parametrize("experts", [8, 60, 256, 1024])
def test_route_masked_and_bad_logits(experts, groups, topk_groups, group_score, scoring):
    import gemm_exl3_linear_amd as X
    l = special_logits(experts)
    rng = np.random.default_rng(1)
    for b in (None, rng.standard_normal(experts) * 0.1):
        keep = np.ones(len(l), dtype=bool)
        if scoring == "sigmoid" and b is None and group_score == "top2":
            keep[[15, 16]] = False  # sums of scores that round to each other in 64 bits
        if scoring == "softmax" and (b is not None or group_score == "top2"):
            keep[14] = False        # scores that fall below 2^-1074
        for renormalize in (False, True):
            rule = rule_of(experts, 4, b, scoring=scoring, groups=groups, topk_groups=topk_groups,
                           group_score=group_score, renormalize=renormalize)
            ids, w = X.exl3_route_topk(G.to_dev(l), rule)
            got = np.sort(ids.cpu().numpy(), axis=1)
            assert (got >= 0).all() and (got < experts).all() and (np.diff(got, axis=1) > 0).all()
            if renormalize:
                keep[15] = keep[15] and scoring == "softmax"  # sums of subnormal weights keep fewer bits
                keep[7] = keep[7] and scoring == "softmax"
            for i in np.flatnonzero(keep):
                check(ids[i:i + 1], w[i:i + 1], l[i:i + 1], rule, f"row {i}")


def test_route_infinite_balance_and_none():
    import torch
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(9)
    l = rng.standard_normal((30, 96)).astype(np.float32)
    b = np.zeros(96)
    b[::3], b[1], b[5] = -np.inf, np.inf, np.nan
    for groups, tg, score in ((1, 1, "max"), (8, 3, "top2"), (8, 5, "max")):
        rule = rule_of(96, 10, b, scoring="sigmoid", groups=groups, topk_groups=tg, group_score=score)
        ids, w = X.exl3_route_topk(G.to_dev(l), rule)
        check(ids, w, l, rule)
    ids, w = X.exl3_route_topk(torch.empty((0, 96), device=G.dev()), rule)
    assert ids.shape == (0, 10) and w.shape == (0, 10)


# ---------------------------------------------------------------------------
# the router's linear
# ---------------------------------------------------------------------------
LINEAR = [(1, 8, 1), (1, 2048, 256), (2, 40, 17), (3, 5120, 256), (5, 1440, 60), (15, 264, 33), (16, 2048, 1024),
          (16, 8192, 5), (17, 2048, 256), (31, 24, 3), (32, 512, 64), (33, 1000, 100), (64, 5120, 256), (65, 72, 130),
          (100, 2880, 128), (127, 32, 31), (128, 4096, 384), (129, 1448, 257), (333, 1440, 60), (500, 2048, 16),
          (1000, 520, 1000), (1500, 7168, 256), (2049, 96, 72), (4096, 1024, 64), (5000, 256, 8)]


def router_case(t, hidden, experts, bias, seed=0):
    rng = np.random.default_rng(t * 5 + hidden + experts + seed)
    x = rng.standard_normal((t, hidden)).astype(np.float16)
    w = (rng.standard_normal((experts, hidden)) * 1.5 * hidden ** -0.5).astype(np.float16)
    c = rng.standard_normal(experts).astype(np.float32) if bias else None
    return x, w, c


def handle(w, c):
    import gemm_exl3_linear_amd as X
    return X.Exl3Router(G.to_dev(w), bias=None if c is None else G.to_dev(c))


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("t,hidden,experts", LINEAR)
def test_router_linear(t, hidden, experts, bias):
    import torch
    import gemm_exl3_linear_amd as X
    x, w, c = router_case(t, hidden, experts, bias)
    buf = torch.full((t + 1, experts + 3), 7.0, device=G.dev())
    X.exl3_router_linear(G.to_dev(x), handle(w, c), out=buf[:t, :experts])
    ref, mag = S.logits(x, w, c)
    got = buf.cpu().numpy()
    assert (np.abs(got[:t, :experts] - ref) <= logit_bound(mag, hidden)).all()
    assert (got[t:] == 7).all() and (got[:, experts:] == 7).all()


@pytest.mark.parametrize("t", [1, 16, 40, 200, 1100])
def test_router_linear_of_whole_numbers_is_exact(t):
    import torch
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(t)
    for hidden, experts, pad in ((1448, 60, 8), (5120, 256, 0), (64, 300, 16)):
        x = rng.integers(-4, 5, (t, hidden + pad)).astype(np.float16)
        w = rng.integers(-4, 5, (experts, hidden)).astype(np.float16)
        got = X.exl3_router_linear(G.to_dev(x)[:, :hidden], handle(w, None))
        np.testing.assert_array_equal(got.cpu().numpy(), x[:, :hidden].astype(np.float64) @ w.T.astype(np.float64))


@pytest.mark.parametrize("t", [1, 16, 40, 200, 1100])
def test_router_linear_bad_rows_stay_alone(t):
    import gemm_exl3_linear_amd as X
    x, w, c = router_case(t, 1000, 70, True)
    x[t // 2, 3], x[t // 3, 999] = np.nan, np.inf
    w[5, 7], w[69, 0] = np.inf, np.nan
    with np.errstate(invalid="ignore"):
        ref, mag = S.logits(x, w, c)
    got = X.exl3_router_linear(G.to_dev(x), handle(w, c)).cpu().numpy().astype(np.float64)
    fine = np.isfinite(ref)
    np.testing.assert_array_equal(got[~fine], ref[~fine])
    assert (np.abs(got[fine] - ref[fine]) <= logit_bound(mag[fine], 1000)).all()


# ---------------------------------------------------------------------------
# both in a call
# ---------------------------------------------------------------------------
ROUTER = [(1, 2048, 256, 8, 1, 1, "max"), (1, 8, 4, 4, 1, 1, "max"), (2, 1440, 60, 4, 1, 1, "max"),
          (7, 264, 33, 9, 3, 2, "top2"), (16, 5120, 256, 8, 8, 4, "top2"), (16, 2048, 1024, 16, 32, 7, "max"),
          (9, 4096, 512, 8, 1, 1, "max"), (13, 2880, 128, 4, 1, 1, "max"), (17, 2048, 256, 8, 8, 4, "top2"),
          (33, 1000, 100, 6, 1, 1, "max"), (64, 5120, 256, 8, 8, 4, "top2"), (64, 2048, 60, 4, 1, 1, "max"),
          (200, 1440, 384, 8, 1, 1, "max"), (777, 2048, 256, 8, 8, 4, "max")]


@pytest.mark.parametrize("scoring,balanced,bias", [("softmax", False, False), ("sigmoid", True, False),
                                                   ("softmax", True, True), ("sigmoid", False, True)])
@pytest.mark.parametrize("t,hidden,experts,topk,groups,topk_groups,group_score", ROUTER)
def test_router(t, hidden, experts, topk, groups, topk_groups, group_score, scoring, balanced, bias):
    import torch
    import gemm_exl3_linear_amd as X
    x, w, c = router_case(t, hidden, experts, bias, seed=11)
    rng = np.random.default_rng(experts)
    b = rng.standard_normal(experts) * (0.1 if scoring == "sigmoid" else 0.5 / experts) if balanced else None
    rule = rule_of(experts, topk, b, scoring=scoring, groups=groups, topk_groups=topk_groups, group_score=group_score,
                   scale=2.5)
    r, xd = handle(w, c), G.to_dev(x)
    logits = torch.full((t, experts + 5), 7.0, device=G.dev())
    ids, wt = X.exl3_router(xd, r, rule, logits=logits[:, :experts])
    ref, mag = S.logits(x, w, c)
    got = logits.cpu().numpy()
    assert (np.abs(got[:, :experts] - ref) <= logit_bound(mag, hidden)).all() and (got[:, experts:] == 7).all()
    check(ids, wt, got[:, :experts].astype(np.float64), rule)
    # the same without the logits, and as two calls
    ids2, wt2 = X.exl3_router(xd, r, rule)
    assert torch.equal(ids, ids2) and torch.equal(wt, wt2)
    ids3, wt3 = X.exl3_route_topk(logits[:, :experts], rule)
    assert torch.equal(ids, ids3)
    check(ids3, wt3, got[:, :experts].astype(np.float64), rule)


@pytest.mark.parametrize("t", [1, 5, 16, 40])
def test_router_bad_rows(t):
    import torch
    import gemm_exl3_linear_amd as X
    x, w, c = router_case(t, 520, 96, True)
    x[0] = np.nan
    c[7], c[20] = -np.inf, np.inf
    rule = rule_of(96, 6, None, scoring="sigmoid")
    logits = torch.empty((t, 96), device=G.dev())
    ids, wt = X.exl3_router(G.to_dev(x), handle(w, c), rule, logits=logits)
    check(ids, wt, logits.cpu().numpy().astype(np.float64), rule)
    assert (ids[1:, 0] == 20).all() and (ids[0] == torch.arange(6, device=G.dev())).all()


def test_one_workspace_serves_routers_and_sizes():
    import torch
    import gemm_exl3_linear_amd as X
    cases = [(1, 2048, 256, 8), (16, 5120, 256, 8), (3, 8192, 60, 4), (16, 2048, 1024, 16), (5, 264, 33, 9),
             (40, 1440, 60, 4), (1, 65536, 16, 2)]
    made = []
    for t, hidden, experts, topk in cases:
        x, w, _ = router_case(t, hidden, experts, False)
        made.append((G.to_dev(x), handle(w, None), rule_of(experts, topk), S.logits(x, w)))
    need = max(max(X.exl3_router_workspace_size(r, x.shape[0], False), X.exl3_router_linear_workspace_size(r, x.shape[0]))
               for x, r, _, _ in made)
    ws = torch.zeros(need, dtype=torch.uint8, device=G.dev())
    for i in (0, 1, 2, 3, 4, 5, 6, 0, 3, 6, 1, 5, 2):
        x, r, rule, (ref, mag) = made[i]
        l = X.exl3_router_linear(x, r, workspace=ws).cpu().numpy()
        assert (np.abs(l - ref) <= logit_bound(mag, x.shape[1])).all()
        ids, wt = X.exl3_router(x, r, rule, workspace=ws)
        check(ids, wt, oracle_logits(x, r, ws), rule)


def oracle_logits(x, r, ws):
    import torch
    import gemm_exl3_linear_amd as X
    l = torch.empty((x.shape[0], r.experts), device=G.dev())
    big = torch.zeros(X.exl3_router_workspace_size(r, x.shape[0]), dtype=torch.uint8, device=G.dev())
    X.exl3_router(x, r, rule_of(r.experts, 1), logits=l, workspace=big)
    return l.cpu().numpy().astype(np.float64)


@pytest.mark.parametrize("t,hidden,experts,topk", [(17, 2048, 60, 4), (24, 1000, 33, 2), (40, 264, 20, 3),
                                                   (100, 5120, 8, 2), (300, 72, 3, 1), (1024, 520, 1, 1)])
def test_router_more_tokens_than_a_tile_and_few_experts(t, hidden, experts, topk):
    """Tokens times experts as few as one tile's: the sums of every tile are whole when
    they are routed, and the workspace's counts end at zero."""
    import torch
    import gemm_exl3_linear_amd as X
    x, w, c = router_case(t, hidden, experts, True, seed=5)
    r, rule, xd = handle(w, c), rule_of(experts, topk), G.to_dev(x)
    ref, mag = S.logits(x, w, c)
    ws = torch.zeros(X.exl3_router_workspace_size(r, t), dtype=torch.uint8, device=G.dev())
    for _ in range(3):
        logits = torch.full((t, experts), float("nan"), device=G.dev())
        ids, wt = X.exl3_router(xd, r, rule, logits=logits, workspace=ws)
        got = logits.cpu().numpy()
        assert (np.abs(got - ref) <= logit_bound(mag, hidden)).all()
        check(ids, wt, got.astype(np.float64), rule)
        assert not ws[:512].any()


def test_router_refuses_a_mismatch():
    import torch
    import gemm_exl3_linear_amd as X
    x, w, _ = router_case(3, 64, 16, False)
    r, xd = handle(w, None), G.to_dev(x)
    with pytest.raises(X.Exl3Error):
        X.exl3_router(xd, r, rule_of(8, 2))
    for kw in (dict(logits=torch.empty((3, 16), dtype=torch.float16, device=G.dev())),
               dict(logits=torch.empty((2, 16), device=G.dev())), dict(logits=torch.empty((3, 16))),
               dict(topk_ids=torch.empty((3, 2), dtype=torch.int64, device=G.dev())),
               dict(topk_weights=torch.empty((3, 3), device=G.dev())),
               dict(topk_ids=torch.empty((2, 3), dtype=torch.int32, device=G.dev()).t())):
        with pytest.raises(ValueError):
            X.exl3_router(xd, r, rule_of(16, 2), **kw)
    with pytest.raises(X.Exl3Error):
        X.exl3_router(xd, r, rule_of(16, 2), workspace=torch.zeros(64, dtype=torch.uint8, device=G.dev()))


def test_router_of_rows_past_32_bits():
    import torch
    import gemm_exl3_linear_amd as X
    t, pitch = 40, 1 << 26  # the last row starts 5 GiB in
    buf = torch.zeros(t * pitch, dtype=torch.float16, device=G.dev())
    x, w, _ = router_case(t, 72, 20, False)
    xd = buf.view(t, pitch)[:, :72]
    xd.copy_(G.to_dev(x))
    logits = torch.empty((t * (1 << 26),), device=G.dev()).view(t, 1 << 26)[:, :20]
    r, rule = handle(w, None), rule_of(20, 3)
    for n in (16, t):
        ids, wt = X.exl3_router(xd[:n], r, rule, logits=logits[:n])
        ref, mag = S.logits(x[:n], w)
        got = logits[:n].cpu().numpy()
        assert (np.abs(got - ref) <= logit_bound(mag, 72)).all()
        check(ids, wt, got.astype(np.float64), rule)
        ids2, _ = X.exl3_route_topk(logits[:n], rule)
        assert torch.equal(ids, ids2)


@pytest.mark.parametrize("t,hidden,experts", [(17, 8192, 1000), (33, 5120, 512), (70, 5120, 1000), (130, 8192, 256),
                                              (450, 5120, 300), (577, 5120, 1000), (1025, 4104, 130)])
def test_router_shares_of_a_few_tiles(t, hidden, experts):
    """Row tiles that are no multiple of eight, in several shares: logits, and routed."""
    import gemm_exl3_linear_amd as X
    x, w, c = router_case(t, hidden, experts, True, seed=3)
    r, rule, xd = handle(w, c), rule_of(experts, 5), G.to_dev(x)
    ref, mag = S.logits(x, w, c)
    got = X.exl3_router_linear(xd, r).cpu().numpy()
    assert (np.abs(got - ref) <= logit_bound(mag, hidden)).all()
    logits = G.to_dev(np.full((t, experts), np.nan, dtype=np.float32))
    ids, wt = X.exl3_router(xd, r, rule, logits=logits)
    got = logits.cpu().numpy()
    assert (np.abs(got - ref) <= logit_bound(mag, hidden)).all()
    check(ids, wt, got.astype(np.float64), rule)
    ids2, wt2 = X.exl3_router(xd, r, rule)
    assert (ids == ids2).all() and (wt == wt2).all()


def test_router_many_tokens_in_shares():
    """More tokens than are else routed by a wave each, from shares of k."""
    import gemm_exl3_linear_amd as X
    x, w, c = router_case(4000, 5120, 60, True, seed=3)
    r, xd = handle(w, c), G.to_dev(x)
    rule = rule_of(60, 4, np.random.default_rng(4).standard_normal(60) * 0.1, scoring="sigmoid", groups=4,
                   topk_groups=2, group_score="top2")
    logits = G.to_dev(np.full((4000, 60), np.nan, dtype=np.float32))
    ids, wt = X.exl3_router(xd, r, rule, logits=logits)
    ref, mag = S.logits(x, w, c)
    got = logits.cpu().numpy()
    assert (np.abs(got - ref) <= logit_bound(mag, 5120)).all()
    check(ids, wt, got.astype(np.float64), rule)
