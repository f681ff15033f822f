"""Refusals and workspace queries of the MXFP4 entry points (host only: none
of these calls reaches a HIP API)."""
import ctypes

import pytest

import gemm_exl3_linear_amd as X

OK, INV, WS = X.EXL3_OK, X.EXL3_E_INVALID, X.EXL3_E_WORKSPACE
F16, F32 = X.EXL3_F16, X.EXL3_F32


def mx(rows=64, k=256, codes=16, scales=16):
    return X._Mx4(codes, scales, rows, k)


@pytest.mark.parametrize("kw", [
    dict(dtype=2), dict(rows=-1), dict(rows=(1 << 24) + 1), dict(k=0), dict(k=-32), dict(k=48), dict(k=1 << 24),
    dict(ldx=224), dict(ldx=260), dict(x=0), dict(x=8), dict(codes=0), dict(codes=24), dict(scales=0),
    dict(scales=17), dict(rows=1 << 24, k=2048, ldx=2048)])
def test_quantize_refuses(kw):
    a = dict(x=16, dtype=F16, rows=4, k=256, ldx=256, codes=16, scales=16) | kw
    assert X.lib().exl3_mx4_quantize(a["x"], a["dtype"], a["rows"], a["k"], a["ldx"], a["codes"], a["scales"],
                                     0) == INV


def test_quantize_of_no_rows_is_a_no_op():
    assert X.lib().exl3_mx4_quantize(0, F16, 0, 256, 256, 0, 0, 0) == OK


@pytest.mark.parametrize("w,kw", [
    (dict(k=40), {}), (dict(codes=0), {}), (dict(scales=8), {}), (dict(rows=-1), {}), ({}, dict(out=0)),
    ({}, dict(out=8)), ({}, dict(ld=248)), ({}, dict(ld=260)), ({}, dict(dtype=3)),
    (dict(rows=1 << 24, k=2048), dict(ld=2048))])
def test_reconstruct_refuses(w, kw):
    a = dict(out=16, dtype=F16, ld=256) | kw
    assert X.lib().exl3_mx4_reconstruct(ctypes.byref(mx(**w)), a["out"], a["dtype"], a["ld"], 0) == INV
    assert X.lib().exl3_mx4_reconstruct(None, 16, F16, 256, 0) == INV


def test_reconstruct_of_no_rows_is_a_no_op():
    assert X.lib().exl3_mx4_reconstruct(ctypes.byref(mx(rows=0, codes=0, scales=0)), 0, F16, 256, 0) == OK


def matmul(a=None, b=None, bias=0, y=16, ldy=64, dt=F16, ws=0, n=0):
    a, b = a or mx(3), b or mx(64)
    return X.lib().exl3_mx4_matmul(ctypes.byref(a), ctypes.byref(b), bias, y, ldy, dt, ws, n, 0)


def test_matmul_refuses():
    assert matmul(b=mx(k=512)) == INV
    assert matmul(a=mx(k=33)) == INV
    assert matmul(a=mx(codes=4)) == INV
    assert matmul(b=mx(scales=0)) == INV
    assert matmul(ldy=63) == INV
    assert matmul(dt=5) == INV
    assert matmul(y=0) == INV
    assert matmul(y=17) == INV
    assert matmul(y=18, dt=F32) == INV
    assert matmul(bias=3) == INV
    assert X.lib().exl3_mx4_matmul(None, ctypes.byref(mx()), 0, 16, 64, F16, 0, 0, 0) == INV
    assert X.lib().exl3_mx4_matmul(ctypes.byref(mx()), None, 0, 16, 64, F16, 0, 0, 0) == INV
    # 2^20 x 2^6 output tiles: one launch does not hold them
    assert matmul(a=mx(1 << 24), b=mx(1024), ldy=1024, ws=16, n=1 << 60) == INV
    assert matmul(a=mx(0)) == OK and matmul(b=mx(0), ldy=0) == OK


def test_matmul_workspace_is_asked_for():
    q = lambda a, b: X.lib().exl3_mx4_matmul_workspace_size(ctypes.byref(a), ctypes.byref(b))
    assert q(mx(3), mx(64, k=512)) == 0 and q(mx(0), mx(64)) == 0 and q(mx(3, k=30), mx(64)) == 0
    for m in (1, 16, 64, 333, 4096):
        need = q(mx(m, 5120), mx(5120, 5120))
        if need:
            assert matmul(mx(m, 5120), mx(5120, 5120), ldy=5120) == WS
            assert matmul(mx(m, 5120), mx(5120, 5120), ldy=5120, ws=16, n=need - 1) == WS
            assert matmul(mx(m, 5120), mx(5120, 5120), ldy=5120, ws=24, n=need) == WS


def linear(w=None, bias=0, x=16, m=3, ldx=256, y=16, ldy=64, dt=F16, ws=0, n=0):
    w = w or mx(64)
    return X.lib().exl3_mx4_linear(ctypes.byref(w), bias, x, m, ldx, y, ldy, dt, ws, n, 0)


def test_linear_refuses():
    for kw in (dict(m=-1), dict(m=X.MX4_LINEAR_MAX_ROWS + 1), dict(ldx=248), dict(ldx=260), dict(x=0), dict(x=8),
               dict(y=0), dict(ldy=63), dict(dt=2), dict(bias=1), dict(w=mx(k=100)), dict(w=mx(codes=0))):
        assert linear(**kw) == INV, kw
    assert linear(m=0, x=0, y=0) == OK and linear(w=mx(0), y=0, ldy=0) == OK
    q = lambda w, m: X.lib().exl3_mx4_linear_workspace_size(ctypes.byref(w), m)
    assert q(mx(), 0) == 0 and q(mx(), 65) == 0 and q(mx(k=31), 1) == 0
    for m in (1, 16, 17, 64):
        need = q(mx(5120, 17408), m)
        if need:
            assert linear(mx(5120, 17408), m=m, ldx=17408, ldy=5120) == WS
            assert linear(mx(5120, 17408), m=m, ldx=17408, ldy=5120, ws=16, n=need - 1) == WS


def layer(**kw):
    a = dict(router=16, bias=0, scoring=0, renorm=1, scale=1.0, e=8, h=256, i=128, e2=None, dk=None, dn=None, slots=2,
             dslots=1, sh=0, si=64, sh_e=1, sh_dn=None, gate=0, codes=16) | kw
    gu = X._Mx4Experts(a["codes"], 16, a["e"], a["slots"], a["i"], a["h"])
    dn = X._Mx4Experts(16, 16, a["e2"] or a["e"], a["dslots"], a["dn"] or a["h"], a["dk"] or a["i"])
    sg, sd = X._Mx4Experts(), X._Mx4Experts()
    if a["sh"] in (1, 3):
        sg = X._Mx4Experts(16, 16, a["sh_e"], 2, a["si"], a["h"])
    if a["sh"] in (1, 2):
        sd = X._Mx4Experts(16, 16, 1, 1, a["sh_dn"] or a["h"], a["si"])
    return X._Mx4MoeLayer(a["router"], a["bias"], a["scoring"], a["renorm"], a["scale"], gu, dn, sg, sd, a["gate"])


def moe(l, x=16, t=2, ldx=256, topk=2, y=16, ldy=256, dt=F16, ids=0, w=0, ws=0, n=0):
    return X.lib().exl3_mx4_moe(ctypes.byref(l), x, t, ldx, topk, y, ldy, dt, ids, w, ws, n, 0)


@pytest.mark.parametrize("kw", [
    dict(router=0), dict(router=8), dict(bias=2), dict(scoring=2), dict(scoring=-1), dict(e=0), dict(e=1025),
    dict(e2=7), dict(h=250), dict(i=100), dict(i=0), dict(h=65568), dict(dk=64), dict(dn=128), dict(slots=1),
    dict(dslots=2), dict(codes=0), dict(codes=24), dict(sh=2), dict(sh=3), dict(sh=1, si=50), dict(sh=1, sh_e=2),
    dict(sh=1, sh_dn=128), dict(sh=1, gate=8), dict(gate=16)])
def test_moe_refuses_layers(kw):
    l = layer(**kw)
    h = kw.get("h", 256)
    assert moe(l, ldx=max(h, 256) // 8 * 8 + 8, ldy=h + 8) == INV
    assert X.lib().exl3_mx4_moe_workspace_size(ctypes.byref(l), 2, 2) == 0


def test_moe_refuses_calls():
    l = layer()
    for kw in (dict(t=-1), dict(t=X.MX4_MOE_MAX_TOKENS + 1), dict(topk=0), dict(topk=9), dict(topk=17), dict(x=0),
               dict(x=8), dict(y=0), dict(y=17), dict(y=18, dt=F32), dict(dt=2), dict(ldx=248), dict(ldx=260),
               dict(ldy=255), dict(ids=2), dict(w=2)):
        assert moe(l, **kw) == INV, kw
    assert moe(l, t=0, x=0, y=0) == OK
    q = lambda l, t, k: X.lib().exl3_mx4_moe_workspace_size(ctypes.byref(l), t, k)
    need = q(l, 2, 2)
    assert need > 0 and q(l, 0, 2) == 0 and q(l, 17, 2) == 0 and q(l, 2, 9) == 0
    assert moe(l) == WS and moe(l, ws=16, n=need - 1) == WS and moe(l, ws=8, n=need) == WS
    assert X.lib().exl3_mx4_moe(None, 16, 1, 256, 2, 16, 256, F16, 0, 0, 16, 1 << 40, 0) == INV


def test_binding_refuses_before_the_library():
    import torch
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)
    for codes, scales in ((u8(4, 24), u8(4, 1)), (u8(4, 32), u8(4, 1)), (u8(4, 32), u8(3, 2)), (u8(32), u8(2)),
                          (torch.zeros(4, 32), u8(4, 2)), (u8(32, 4).t(), u8(4, 2)), (u8(4, 0), u8(4, 0))):
        with pytest.raises(ValueError):
            X.Exl3Mx4(codes, scales)
    w = X.Exl3Mx4(u8(4, 32), u8(4, 2))
    assert (w.rows, w.k) == (4, 64)
    x = torch.zeros(2, 64, dtype=torch.float16)
    for call in (lambda: X.exl3_mx4_linear(x, w), lambda: X.exl3_mx4_quantize(x),       # tensors on the CPU
                 lambda: X.exl3_mx4_reconstruct(w), lambda: X.exl3_mx4_matmul(w, w),
                 lambda: X.exl3_mx4_quantize(x.to(torch.bfloat16)), lambda: X.exl3_mx4_linear(x[:, :32], w),
                 lambda: X.exl3_mx4_quantize(x.t())):
        with pytest.raises(ValueError):
            call()
    gu, dn = X.Exl3Mx4Arena(u8(2, 2, 32, 32), u8(2, 2, 32, 2)), X.Exl3Mx4Arena(u8(2, 1, 64, 16), u8(2, 1, 64, 1))
    r = torch.zeros(2, 64, dtype=torch.float16)
    X.Exl3Mx4Moe(X.Exl3MoeRouter(r), gu, dn)
    for router in (X.Exl3MoeRouter(r[:1]), X.Exl3MoeRouter(r.float()), X.Exl3MoeRouter(r, scoring="top"),
                   X.Exl3MoeRouter(r, bias=torch.zeros(3)), X.Exl3MoeRouter(r, bias=torch.zeros(2).half())):
        with pytest.raises(ValueError):
            X.Exl3Mx4Moe(router, gu, dn)
    with pytest.raises(ValueError):
        X.exl3_mx4_moe(x, X.Exl3Mx4Moe(X.Exl3MoeRouter(r), gu, dn), 2)


def test_copies_hold_their_own_tensors():
    import copy
    import pickle
    torch = pytest.importorskip("torch")
    a = lambda *s: torch.zeros(s, dtype=torch.uint8)
    w = X.Exl3Mx4(a(4, 64), a(4, 4))
    l = X.Exl3Mx4Moe(X.Exl3MoeRouter(torch.zeros(3, 64, dtype=torch.float16)),
                     X.Exl3Mx4Arena(a(3, 2, 32, 32), a(3, 2, 32, 2)), X.Exl3Mx4Arena(a(3, 1, 64, 16), a(3, 1, 64, 1)))
    for twin in (copy.deepcopy, lambda o: pickle.loads(pickle.dumps(o))):
        v, m = twin(w), twin(l)
        assert v.codes.data_ptr() != w.codes.data_ptr() and v._record.codes == v.codes.data_ptr()
        assert v._record.scales == v.scales.data_ptr() and (v._record.rows, v._record.k) == (4, 128)
        assert m._record.router == m.router.weight.data_ptr() != l.router.weight.data_ptr()
        assert m._record.gate_up.codes == m.gate_up.codes.data_ptr() and m._record.down.n == 64


def _swapped(t, new):
    t.data = new
    return t


def test_tensors_swapped_after_construction_are_read_anew():
    torch = pytest.importorskip("torch")
    a = lambda *s: torch.zeros(s, dtype=torch.uint8)
    w, b = X.Exl3Mx4(a(4096, 2560), a(4096, 160)), X.Exl3Mx4(a(512, 2560), a(512, 160))
    before = X.exl3_mx4_matmul_workspace_size(w, b)
    _swapped(w.codes, a(1024, 2560)), _swapped(w.scales, a(1024, 160))
    fresh = X.exl3_mx4_matmul_workspace_size(X.Exl3Mx4(w.codes, w.scales), b)
    assert before != fresh == X.exl3_mx4_matmul_workspace_size(w, b)
    assert X.exl3_mx4_linear_workspace_size(w, 40) == X.exl3_mx4_linear_workspace_size(X.Exl3Mx4(w.codes, w.scales), 40)
    w.codes.set_(a(1024, 2560))  # the shape as it was, other memory
    assert w._now() == (w.codes.data_ptr(), w.scales.data_ptr(), 1024, 5120)
    assert w._record.codes == w.codes.data_ptr() and w._record.rows == 1024
    _swapped(w.codes, a(1024, 24))
    with pytest.raises(ValueError):
        X.exl3_mx4_matmul_workspace_size(w, b)
    with pytest.raises(ValueError):
        X.exl3_mx4_linear_workspace_size(w, 1)

    f = lambda *s: torch.zeros(s, dtype=torch.float16)
    gu, dn = X.Exl3Mx4Arena(a(3, 2, 32, 32), a(3, 2, 32, 2)), X.Exl3Mx4Arena(a(3, 1, 64, 16), a(3, 1, 64, 1))
    sh = X.Exl3Mx4Shared(X.Exl3Mx4Arena(a(1, 2, 96, 32), a(1, 2, 96, 2)), X.Exl3Mx4Arena(a(1, 1, 64, 48), a(1, 1, 64, 3)),
                         gate=f(64))
    l = X.Exl3Mx4Moe(X.Exl3MoeRouter(f(3, 64), bias=torch.zeros(3)), gu, dn, sh)
    before = X.exl3_mx4_moe_workspace_size(l, 16, 2)
    _swapped(gu.codes, a(3, 2, 320, 32)), _swapped(gu.scales, a(3, 2, 320, 2))
    _swapped(dn.codes, a(3, 1, 64, 160)), _swapped(dn.scales, a(3, 1, 64, 10))
    assert before < X.exl3_mx4_moe_workspace_size(l, 16, 2)
    for t, at in ((l.router.weight, lambda r: r.router), (l.router.bias, lambda r: r.router_bias),
                  (sh.gate, lambda r: r.shared_gate), (sh.down.scales, lambda r: r.shared_down.scales),
                  (sh.gate_up.codes, lambda r: r.shared_gate_up.codes), (dn.codes, lambda r: r.down.codes)):
        _swapped(t, t.clone())
        assert at(l._now()) == t.data_ptr()
    _swapped(gu.scales, a(3, 2, 320, 1))
    with pytest.raises(ValueError):
        X.exl3_mx4_moe_workspace_size(l, 16, 2)


def test_sizes_past_a_grid_are_refused():
    # a grid holds less than 2^32 threads: 2^32 - 4 chunks of eight elements round up
    # to it, and so do 2^23 tiles of 512 threads
    quantize = lambda rows, k: X.lib().exl3_mx4_quantize(16, F16, rows, k, k, 16, 16, 0)
    k = 32 * 9 * 331
    rows = ((1 << 35) - 32) // k
    assert rows * k == (1 << 35) - 32 and quantize(rows, k) == INV
    assert quantize(1 << 24, 2048) == INV and quantize((1 << 24) - 1, 2048 + 32) == INV
    a, b = mx(1 << 24, 8192), mx(1000, 8192)
    assert X.lib().exl3_mx4_matmul_workspace_size(ctypes.byref(a), ctypes.byref(b)) == 0
    assert matmul(a, b, ldy=1000, ws=16, n=1 << 60) == INV
    # as many tiles, with scales that go through LDS, are a call that wants its workspace
    a, b = mx(1 << 24, 512), mx(1000, 512)
    assert X.lib().exl3_mx4_matmul_workspace_size(ctypes.byref(a), ctypes.byref(b)) > 0
    assert matmul(a, b, ldy=1000) == WS
