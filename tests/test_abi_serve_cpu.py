"""Refusals and workspace queries of the routing's and the adapters' entry points
(host only: none of these calls reaches a HIP API)."""
import copy
import ctypes
import pickle

import pytest

import gemm_exl3_linear_amd as X

OK, INV, WS = X.EXL3_OK, X.EXL3_E_INVALID, X.EXL3_E_WORKSPACE
F16, F32 = X.EXL3_F16, X.EXL3_F32
BIG = 1 << 60


def rule(**kw):
    a = dict(balance=0, experts=64, topk=8, scoring=X.ROUTE_SOFTMAX, groups=1, topk_groups=1, group_score=X.GROUP_MAX,
             renormalize=1, scale=1.0) | kw
    return X._RouteRule(*a.values())


BAD_RULES = [dict(experts=0), dict(experts=-1), dict(experts=1025), dict(topk=0), dict(topk=17), dict(topk=-1),
             dict(experts=4, topk=5), dict(scoring=2), dict(scoring=-1), dict(group_score=2), dict(groups=0),
             dict(groups=65, experts=650), dict(groups=3), dict(groups=4, topk_groups=0),
             dict(groups=4, topk_groups=5), dict(groups=32, topk_groups=3), dict(balance=2),
             dict(groups=64, topk_groups=32, group_score=X.GROUP_TOP2)]


def route(r=None, logits=16, dtype=F32, t=3, ldl=64, ids=16, weights=16):
    return X.lib().exl3_route_topk(ctypes.byref(r or rule()), logits, dtype, t, ldl, ids, weights, 0)


@pytest.mark.parametrize("kw", BAD_RULES)
def test_rules_are_refused(kw):
    assert route(rule(**kw), ldl=2000) == INV
    assert router(r=rule(**kw), w=weight(experts=kw.get("experts", 64)), ws=16, n=BIG) == INV


def test_route_refuses():
    for kw in (dict(dtype=2), dict(t=-1), dict(t=(1 << 24) + 1), dict(ldl=63), dict(logits=0), dict(logits=2),
               dict(logits=1, dtype=F16), dict(ids=0), dict(ids=6), dict(weights=0), dict(weights=18)):
        assert route(**kw) == INV, kw
    assert X.lib().exl3_route_topk(None, 16, F32, 1, 64, 16, 16, 0) == INV
    assert route(t=0, logits=0, ids=0, weights=0) == OK


def weight(**kw):
    a = dict(weight=16, bias=0, experts=64, hidden=2048) | kw
    return X._RouterWeight(*a.values())


BAD_WEIGHTS = [dict(weight=0), dict(weight=8), dict(bias=2), dict(experts=0), dict(experts=1025), dict(hidden=0),
               dict(hidden=-8), dict(hidden=12), dict(hidden=65544)]


def linear(w=None, x=16, t=3, ldx=2048, logits=16, ldl=64, ws=0, n=0):
    return X.lib().exl3_router_linear(ctypes.byref(w or weight()), x, t, ldx, logits, ldl, ws, n, 0)


def router(w=None, r=None, x=16, t=3, ldx=2048, logits=16, ldl=64, ids=16, weights=16, ws=0, n=0):
    return X.lib().exl3_router(ctypes.byref(w or weight()), ctypes.byref(r or rule()), x, t, ldx, logits, ldl, ids,
                               weights, ws, n, 0)


def test_router_refuses():
    for kw in BAD_WEIGHTS:
        assert linear(weight(**kw), ldx=1 << 17, ldl=2000, ws=16, n=BIG) == INV, kw
        assert router(weight(**kw), ldx=1 << 17, ldl=2000, ws=16, n=BIG) == INV, kw
        assert X.lib().exl3_router_linear_workspace_size(ctypes.byref(weight(**kw)), 1) == 0
        assert X.lib().exl3_router_workspace_size(ctypes.byref(weight(**kw)), 1, 1) == 0
    for call in (linear, router):
        for kw in (dict(t=-1), dict(t=(1 << 24) + 1), dict(ldx=2040), dict(ldx=2052), dict(x=0), dict(x=8),
                   dict(logits=2), dict(ldl=63)):
            assert call(**kw, ws=16, n=BIG) == INV, (call, kw)
        assert call(t=0, x=0) == OK
    assert linear(logits=0, ws=16, n=BIG) == INV
    for kw in (dict(ids=0), dict(ids=2), dict(weights=0), dict(weights=2), dict(r=rule(experts=32))):
        assert router(**kw, ws=16, n=BIG) == INV, kw
    assert X.lib().exl3_router_linear(None, 16, 1, 64, 16, 64, 16, BIG, 0) == INV
    assert X.lib().exl3_router(None, ctypes.byref(rule()), 16, 1, 64, 16, 64, 16, 16, 16, BIG, 0) == INV
    assert X.lib().exl3_router(ctypes.byref(weight()), None, 16, 1, 2048, 16, 64, 16, 16, 16, BIG, 0) == INV


def test_router_workspaces_are_asked_for():
    for t in (1, 7, 16, 17, 64, 333, 4096):
        for hidden in (8, 2048, 5120, 65536):
            w = weight(hidden=hidden)
            need = X.lib().exl3_router_linear_workspace_size(ctypes.byref(w), t)
            if need:
                for kw in (dict(), dict(ws=16, n=need - 1), dict(ws=24, n=need)):
                    assert linear(w, t=t, ldx=hidden, **kw) == WS
            for logits in (0, 16):
                need = X.lib().exl3_router_workspace_size(ctypes.byref(w), t, logits)
                if need:
                    for kw in (dict(), dict(ws=16, n=need - 1), dict(ws=24, n=need)):
                        assert router(w, t=t, ldx=hidden, logits=logits, **kw) == WS
    for t in (0, -1, (1 << 24) + 1):
        assert X.lib().exl3_router_linear_workspace_size(ctypes.byref(weight()), t) == 0
        assert X.lib().exl3_router_workspace_size(ctypes.byref(weight()), t, 1) == 0


def stack(**kw):
    a = dict(a=16, b=16, scales=0, ranks=0, adapters=4, rank=16, k=256, n=100) | kw
    return X._LoraStack(*a.values())


def lora(l=None, x=16, m=3, ldx=256, rows=16, base=32, ldb=100, y=32, ldy=100, dt=F16, ws=16, n=BIG):
    return X.lib().exl3_lora(ctypes.byref(l or stack()), x, m, ldx, rows, base, ldb, y, ldy, dt, ws, n, 0)


def test_lora_refuses():
    for kw in (dict(a=0), dict(a=8), dict(b=0), dict(b=24), dict(scales=2), dict(ranks=2), dict(adapters=-1),
               dict(adapters=4097), dict(rank=0), dict(rank=12), dict(rank=264), dict(rank=-8), dict(k=0), dict(k=252),
               dict(k=(1 << 20) + 8), dict(n=0), dict(n=(1 << 20) + 1), dict(n=-1)):
        assert lora(stack(**kw), ldx=1 << 21, ldy=1 << 21, ldb=1 << 21) == INV, kw
        assert X.lib().exl3_lora_workspace_size(ctypes.byref(stack(**kw)), 3) == 0
    for kw in (dict(x=0), dict(x=8), dict(m=-1), dict(m=(1 << 24) + 1), dict(ldx=248), dict(ldx=260), dict(rows=0),
               dict(rows=2), dict(base=33), dict(base=34, dt=F32), dict(ldb=99), dict(y=0), dict(y=33), dict(ldy=99),
               dict(ldy=104), dict(dt=2)):
        assert lora(**kw) == INV, kw
    assert X.lib().exl3_lora(None, 16, 1, 256, 16, 0, 0, 16, 100, F16, 16, BIG, 0) == INV
    assert lora(m=0, x=0, rows=0, base=0, y=0) == OK


def test_lora_workspace_is_asked_for():
    for m in (1, 4, 64, 333, 4096):
        for kw in (dict(), dict(rank=256, k=17408, n=5120), dict(adapters=1, rank=8), dict(adapters=0)):
            l = stack(**kw)
            need = X.lib().exl3_lora_workspace_size(ctypes.byref(l), m)
            if need:
                for bad in (dict(ws=0, n=0), dict(n=need - 1), dict(ws=24, n=need)):
                    assert lora(l, m=m, ldx=l.k, ldy=l.n, ldb=l.n, **bad) == WS
    for m in (0, -1, (1 << 24) + 1):
        assert X.lib().exl3_lora_workspace_size(ctypes.byref(stack()), m) == 0


def test_binding_refuses_before_the_library():
    torch = pytest.importorskip("torch")
    f16 = lambda *s: torch.zeros(s, dtype=torch.float16)
    f32 = lambda *s: torch.zeros(s)
    for args in ((f32(4, 64),), (f16(64),), (f16(64, 4).t(),), (f16(4, 64), f16(4)), (f16(4, 64), f32(5))):
        with pytest.raises(ValueError):
            X.Exl3Router(*args)
    for kw in (dict(scoring="top"), dict(group_score="sum"), dict(balance=f32(5)), dict(balance=f16(4))):
        with pytest.raises(ValueError):
            X.Exl3RouteRule(4, 2, **kw)
    for args in ((f32(2, 8, 64), f16(2, 5, 8)), (f16(2, 8, 64), f16(3, 5, 8)), (f16(2, 8, 64), f16(2, 5, 16)),
                 (f16(8, 64), f16(5, 8)), (f16(2, 8, 64), f16(2, 5, 8), f32(3)),
                 (f16(2, 8, 64), f16(2, 5, 8), None, f32(2)), (f16(2, 8, 64), f16(2, 8, 5).transpose(1, 2))):
        with pytest.raises(ValueError):
            X.Exl3Lora(*args)
    r, q = X.Exl3Router(f16(4, 64)), X.Exl3RouteRule(4, 2)
    l = X.Exl3Lora(f16(2, 8, 64), f16(2, 5, 8))
    assert (r.experts, r.hidden) == (4, 64) and (l.adapters, l.rank, l.k, l.n) == (2, 8, 64, 5)
    rows = torch.zeros(3, dtype=torch.int32)
    for call in (lambda: X.exl3_router(f16(3, 64), r, q), lambda: X.exl3_router_linear(f16(3, 64), r),  # on the CPU
                 lambda: X.exl3_route_topk(f32(3, 4), q), lambda: X.exl3_lora(f16(3, 64), l, rows),
                 lambda: X.exl3_router(f16(3, 56), r, q), lambda: X.exl3_route_topk(f32(3, 5), q),
                 lambda: X.exl3_lora(f32(3, 64), l, rows), lambda: X.exl3_lora(f16(3, 72), l, rows)):
        with pytest.raises(ValueError):
            call()


def test_copies_and_swapped_memory():
    torch = pytest.importorskip("torch")
    f16 = lambda *s: torch.zeros(s, dtype=torch.float16)
    r, q = X.Exl3Router(f16(4, 64), bias=torch.zeros(4)), X.Exl3RouteRule(4, 2, balance=torch.zeros(4), scale=2.5)
    l = X.Exl3Lora(f16(2, 8, 64), f16(2, 5, 8), ranks=torch.ones(2, dtype=torch.int32))
    for twin in (copy.deepcopy, lambda o: pickle.loads(pickle.dumps(o))):
        a, b, c = twin(r), twin(q), twin(l)
        assert a._record.weight == a.weight.data_ptr() != r.weight.data_ptr() and a._record.bias == a.bias.data_ptr()
        assert b._record.balance == b.balance.data_ptr() != q.balance.data_ptr() and b._record.scale == 2.5
        assert c._record.a == c.a.data_ptr() != l.a.data_ptr() and c._record.ranks == c.ranks.data_ptr()
    r.weight.data = f16(6, 128)
    with pytest.raises(ValueError):  # the bias is still of four
        X.exl3_router_linear_workspace_size(r, 1)
    r.bias.data = torch.zeros(6)
    assert r._now().experts == 6 and r._record.weight == r.weight.data_ptr()
    l.a.data = f16(2, 8, 32)
    assert l._now().k == 32 and l._record.a == l.a.data_ptr()
    q.balance.data = torch.zeros(4)
    assert q._now().balance == q.balance.data_ptr()
