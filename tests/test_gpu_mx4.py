"""MXFP4 operators on the GPU against the float64 oracle.

Tolerances.  Quantization and reconstruction are exact by definition.  In the
products every single product is exact in fp32 (at most 11 + 2 significand
bits), so an fp32 output is off by the roundings of its sum only.  A sum over k
goes through the matrix cores in blocks of at least 32 and then through fp32
additions, at most k/32 + 64 of them in a row (blocks of a wave, its waves,
their workgroups, the bias); with the additions inside a matrix instruction
(32 products and the running sum, counted as 40 roundings) and two roundings
allowed for each step, |y - y64| <= 2 (k/32 + 104) 2^-24 sum |a||b| + 2^-149.
An fp16 output adds half a step, eps/2 of the value (2^-25 below the normals).
Sums of products that are all multiples of one power of two and stay below 2^24
times it are exact in any order."""
import numpy as np
import pytest

from oracle import mx4_oracle as M
from tests import _gpu as G

pytestmark = pytest.mark.gpu


def rand_mx(rng, *shape, lo=120, hi=130):
    """codes and scales of random MXFP4 values [..., k], scale bytes lo .. hi."""
    *lead, k = shape
    return (rng.integers(0, 256, (*lead, k // 2), dtype=np.uint8),
            rng.integers(lo, hi + 1, (*lead, k // 32)).astype(np.uint8))


def mx(q):
    import gemm_exl3_linear_amd as X
    return X.Exl3Mx4(G.to_dev(q[0]), G.to_dev(q[1]))


def arena(q):
    import gemm_exl3_linear_amd as X
    return X.Exl3Mx4Arena(G.to_dev(q[0]), G.to_dev(q[1]))


def bound(y, mag, k, f32):
    b = 2 * (k / 32 + 104) * 2.0 ** -24 * mag + 2.0 ** -149
    return b if f32 else b + np.maximum(np.abs(y) * 2.0 ** -11, 2.0 ** -25) * 1.001


def assert_within(got, ref, lim, what=""):
    got = np.asarray(got, dtype=np.float64)
    np.testing.assert_array_equal(np.isnan(got), np.isnan(ref), err_msg=f"{what} NaN pattern")
    ok = ~np.isnan(ref)
    bad = ok & ~(np.abs(got - np.where(ok, ref, 0)) <= lim)
    assert not bad.any(), (f"{what} {bad.sum()} of {bad.size} outside, first at {np.argwhere(bad)[0]}: "
                           f"{got[bad][0]!r} for {ref[bad][0]!r}, limit {np.broadcast_to(lim, got.shape)[bad][0]!r}")


# ---------------------------------------------------------------------------
# quantize, reconstruct
# ---------------------------------------------------------------------------
def specials(dtype):
    """Rows whose blocks hold what can go wrong."""
    fi = np.finfo(dtype)
    rows = [np.zeros(32), -np.zeros(32), np.full(32, fi.max), np.full(32, -fi.max), np.full(32, fi.smallest_subnormal),
            np.linspace(-8, 8, 32), np.arange(32) * 0.25, np.arange(32) * 0.125 - 2,
            np.arange(32) * float(fi.smallest_subnormal), np.full(32, fi.tiny)]
    for v in (np.nan, np.inf, -np.inf):
        for at in (0, 13, 31):
            r = np.ones(32)
            r[at] = v
            rows.append(r)
    if dtype == np.float32:
        rows += [np.linspace(1, 2, 32) * 2.0 ** e for e in (-149, -140, -130, -127, -126, -125, -124, 100, 126)]
        near = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0], dtype=np.float32)
        rows.append(np.concatenate([near, np.nextafter(near, np.float32(9)), np.nextafter(near, np.float32(0)), -near]))
    return np.stack(rows).astype(dtype)


@pytest.mark.parametrize("dtype", [np.float16, np.float32])
@pytest.mark.parametrize("rows,k,pad", [(1, 32, 0), (1, 5120, 0), (3, 96, 0), (5, 96, 8), (17, 2080, 40), (1000, 32, 0),
                                        (33, 6880, 0)])
def test_quantize_and_reconstruct_are_exact(rows, k, pad, dtype):
    import torch
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(rows * 7 + k)
    x = (rng.standard_normal((rows, k + pad)) * np.exp2(rng.integers(-12, 6, (rows, 1)))).astype(dtype)
    xd = G.to_dev(x)[:, :k]
    q = X.exl3_mx4_quantize(xd)
    codes, scales = M.quantize(x[:, :k])
    np.testing.assert_array_equal(q.scales.cpu().numpy(), scales)
    np.testing.assert_array_equal(q.codes.cpu().numpy(), codes)
    ref = M.decode(codes, scales)
    for dt in (torch.float16, torch.float32):
        buf = torch.full((rows, k + pad), 7.0, dtype=dt, device=G.dev())
        X.exl3_mx4_reconstruct(q, out=buf[:, :k])
        np.testing.assert_array_equal(buf[:, :k].double().cpu().numpy(), ref.astype(
            np.float16 if dt == torch.float16 else np.float32).astype(np.float64))
        assert (buf[:, k:] == 7.0).all()


@pytest.mark.parametrize("dtype", [np.float16, np.float32])
def test_quantize_special_blocks(dtype):
    import gemm_exl3_linear_amd as X
    x = specials(dtype)
    q = X.exl3_mx4_quantize(G.to_dev(x))
    codes, scales = M.quantize(x)
    np.testing.assert_array_equal(q.scales.cpu().numpy(), scales)
    np.testing.assert_array_equal(q.codes.cpu().numpy(), codes)


def test_reconstruct_every_code_at_every_scale():
    import torch
    import gemm_exl3_linear_amd as X
    codes = np.tile(np.arange(16, dtype=np.uint8) * 16 + np.arange(16, dtype=np.uint8)[::-1], (256, 1))
    q = (codes, np.arange(256, dtype=np.uint8)[:, None])
    with np.errstate(over="ignore"):
        for dt, nt in ((torch.float32, np.float32), (torch.float16, np.float16)):
            got = X.exl3_mx4_reconstruct(mx(q), dtype=dt).cpu().numpy()
            np.testing.assert_array_equal(got, M.decode(*q).astype(nt))


def test_quantize_empty_rows():
    import torch
    import gemm_exl3_linear_amd as X
    q = X.exl3_mx4_quantize(torch.empty((0, 64), dtype=torch.float16, device=G.dev()))
    assert q.rows == 0 and X.exl3_mx4_reconstruct(q).shape == (0, 64)


# ---------------------------------------------------------------------------
# matmul
# ---------------------------------------------------------------------------
MATMUL_SHAPES = [(1, 1, 32), (1, 17, 64), (2, 16, 96), (5, 100, 128), (16, 512, 160), (17, 33, 288), (31, 257, 512),
                 (33, 65, 2080), (64, 64, 256), (65, 1111, 1056), (1, 640, 5120), (3, 5, 17408), (129, 130, 384),
                 (257, 300, 992), (333, 1111, 2080), (520, 260, 1024), (1024, 768, 640), (1000, 1500, 544)]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("m,n,k", MATMUL_SHAPES)
def test_matmul(m, n, k, f32):
    import torch
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(m * 31 + n * 7 + k)
    a, b = rand_mx(rng, m, k), rand_mx(rng, n, k, lo=112, hi=122)
    bias = rng.standard_normal(n).astype(np.float16) if (m + n) % 2 else None
    dt = torch.float32 if f32 else torch.float16
    pad = 3
    buf = torch.full((m, n + pad), 7.0, dtype=dt, device=G.dev())
    y = X.exl3_mx4_matmul(mx(a), mx(b), bias=None if bias is None else G.to_dev(bias), out=buf[:, :n])
    ref, mag = M.product(M.decode(*a), M.decode(*b), bias)
    assert_within(y.cpu().numpy(), ref, bound(ref, mag, k, f32), f"{m}x{n}x{k}")
    assert (buf[:, n:] == 7.0).all()


@pytest.mark.parametrize("m,n,k", [(1, 48, 17408), (16, 80, 5120), (65, 190, 5120), (300, 300, 5152), (512, 512, 4096)])
def test_matmul_of_one_scale_is_exact(m, n, k):
    # products are multiples of 1/4 below 36 k < 2^20: exact in fp32 in any order
    import torch
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(k + m)
    a, b = rand_mx(rng, m, k, lo=127, hi=127), rand_mx(rng, n, k, lo=127, hi=127)
    y = X.exl3_mx4_matmul(mx(a), mx(b), out_dtype=torch.float32)
    np.testing.assert_array_equal(y.double().cpu().numpy(), M.product(M.decode(*a), M.decode(*b))[0])


@pytest.mark.parametrize("m,n,k", [(3, 40, 416), (80, 70, 416), (300, 290, 416), (520, 520, 1056)])
def test_matmul_wide_scales_and_nan_blocks(m, n, k):
    # scale bytes far apart (their products inside fp32), and one NaN block in
    # a row of either operand: it takes that row or column and nothing else
    import torch
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(9 + m)
    a, b = rand_mx(rng, m, k, lo=60, hi=150), rand_mx(rng, n, k, lo=90, hi=160)
    a[1][m // 2, k // 32 - 1] = 255
    b[1][n - 1, 0] = 255
    y = X.exl3_mx4_matmul(mx(a), mx(b), out_dtype=torch.float32).cpu().numpy()
    da, db = M.decode(*a), M.decode(*b)
    ref, _ = M.product(da, db)
    mag = M.product(np.nan_to_num(da), np.nan_to_num(db))[1]
    assert np.isnan(ref).sum() == m + n - 1
    assert_within(y, ref, bound(ref, mag, k, True))


def test_matmul_empty():
    import torch
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(1)
    a, e = mx(rand_mx(rng, 4, 64)), X.Exl3Mx4.empty(0, 64, device=G.dev())
    assert X.exl3_mx4_matmul(a, e).shape == (4, 0) and X.exl3_mx4_matmul(e, a).shape == (0, 4)


# ---------------------------------------------------------------------------
# linear
# ---------------------------------------------------------------------------
LINEAR_SHAPES = [(1, 1, 32), (1, 512, 2048), (1, 33, 5120), (2, 17, 96), (5, 130, 288), (16, 512, 1056), (17, 65, 224),
                 (31, 96, 512), (33, 260, 2080), (37, 640, 17408), (48, 48, 64), (49, 111, 800), (64, 1111, 1024),
                 (3, 17408, 512), (1, 5120, 17408), (8, 2048, 5120)]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("m,n,k", LINEAR_SHAPES)
def test_linear(m, n, k, f32):
    import torch
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(m * 131 + n + k)
    w = rand_mx(rng, n, k, lo=112, hi=122)
    x = np.full((m, k + 8), np.nan, dtype=np.float16)
    x[:, :k] = rng.standard_normal((m, k)) * np.exp2(rng.integers(-8, 4, (m, 1)))
    bias = rng.standard_normal(n).astype(np.float16) if n % 2 else None
    dt = torch.float32 if f32 else torch.float16
    buf = torch.full((m, n + 5), 7.0, dtype=dt, device=G.dev())
    y = X.exl3_mx4_linear(G.to_dev(x)[:, :k], mx(w), bias=None if bias is None else G.to_dev(bias), out=buf[:, :n])
    ref, mag = M.product(x[:, :k], M.decode(*w), bias)
    assert_within(y.cpu().numpy(), ref, bound(ref, mag, k, f32), f"{m}x{n}x{k}")
    assert (buf[:, n:] == 7.0).all()


@pytest.mark.parametrize("m", [1, 16, 33, 64])
def test_linear_of_whole_numbers_is_exact(m):
    # |x| <= 8, |w| <= 6 in halves, k = 4128: multiples of 1/2 below 2^18
    import torch
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(m)
    w = rand_mx(rng, 200, 4128, lo=127, hi=127)
    x = rng.integers(-8, 9, (m, 4128)).astype(np.float16)
    y = X.exl3_mx4_linear(G.to_dev(x), mx(w), out_dtype=torch.float32)
    np.testing.assert_array_equal(y.double().cpu().numpy(), M.product(x, M.decode(*w))[0])


@pytest.mark.parametrize("m", [1, 20, 50])
def test_linear_any_scale_byte(m):
    # every scale byte but the three highest (whose sums pass fp32's range), one
    # to a weight row, and two NaN blocks; x holds subnormal and large values
    import torch
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(12)
    n, k = 252, 288
    codes, scales = rand_mx(rng, n, k)
    scales[:] = np.arange(n, dtype=np.uint8)[:, None]
    scales[220:] = np.arange(90, 122, dtype=np.uint8)[:, None]
    scales[230, 3] = scales[251, 8] = 255
    x = (rng.standard_normal((m, k)) * np.exp2(rng.integers(-22, 10, (1, k)))).astype(np.float16)
    y = X.exl3_mx4_linear(G.to_dev(x), mx((codes, scales)), out_dtype=torch.float32).cpu().numpy()
    w = M.decode(codes, scales)
    ref, _ = M.product(x, w)
    assert_within(y, ref, bound(ref, M.product(x, np.nan_to_num(w))[1], k, True))


@pytest.mark.parametrize("m", [1, 24])
def test_linear_far_scales_inside_a_row(m):
    # a block 2^100 above its neighbours meets zeros of x: the others count alone
    import torch
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(13)
    codes, scales = rand_mx(rng, 40, 512, lo=100, hi=101)
    scales[:, 5] = 201
    x = rng.standard_normal((m, 512)).astype(np.float16)
    x[:, 160:192] = 0
    y = X.exl3_mx4_linear(G.to_dev(x), mx((codes, scales)), out_dtype=torch.float32).cpu().numpy()
    ref, mag = M.product(x, M.decode(codes, scales))
    assert_within(y, ref, bound(ref, mag, 512, True))


def test_linear_infinite_and_nan_activations_stay_in_their_rows():
    import torch
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(14)
    w = rand_mx(rng, 70, 320)
    x = rng.standard_normal((21, 320)).astype(np.float16)
    x[4, 7], x[20, 319] = np.nan, np.inf
    y = X.exl3_mx4_linear(G.to_dev(x), mx(w), out_dtype=torch.float32).cpu().numpy()
    with np.errstate(invalid="ignore"):
        ref, _ = M.product(x, M.decode(*w))
    rest = np.delete(np.arange(21), [4, 20])
    assert np.isnan(y[4]).all() and not np.isfinite(y[20]).any()
    r, mag = M.product(x[rest], M.decode(*w))
    assert_within(y[rest], r, bound(r, mag, 320, True))
    np.testing.assert_array_equal(np.isnan(y[20]), np.isnan(ref[20]))


# ---------------------------------------------------------------------------
# moe
# ---------------------------------------------------------------------------
def moe_case(seed, t, e, h, i, si=0, gate=False, scoring="softmax", renorm=True, bias=False, scale=1.0):
    rng = np.random.default_rng(seed)
    f16 = np.float16

    def weights(*shape):  # about 1 / sqrt(k): rms of a random code is about 2.9
        k = shape[-1]
        s = int(127 + np.round(np.log2(k ** -0.5 / 2.9)))
        return rand_mx(rng, *shape, lo=s - 1, hi=s + 1)
    layer = {"router": (rng.standard_normal((e, h)) * 1.5 * h ** -0.5).astype(f16),
             "gate_up": weights(e, 2, i, h), "down": weights(e, 1, h, i), "scoring": scoring, "renormalize": renorm,
             "scale": scale, "bias": rng.standard_normal(e).astype(np.float32) * 0.1 if bias else None}
    if si:
        layer["shared"] = (weights(1, 2, si, h), weights(1, 1, h, si))
        layer["shared_gate"] = (rng.standard_normal(h) * h ** -0.5).astype(f16) if gate else None
    return rng.standard_normal((t, h)).astype(f16), layer


def moe_layer(l):
    import gemm_exl3_linear_amd as X
    dev = lambda a: None if a is None else G.to_dev(a)
    shared = None
    if l.get("shared") is not None:
        shared = X.Exl3Mx4Shared(arena(l["shared"][0]), arena(l["shared"][1]), gate=dev(l.get("shared_gate")))
    return X.Exl3Mx4Moe(X.Exl3MoeRouter(dev(l["router"]), bias=dev(l.get("bias")), scoring=l["scoring"],
                                        renormalize=l["renormalize"], scale=l["scale"]),
                        arena(l["gate_up"]), arena(l["down"]), shared)


def moe_limit(x, l, topk, ref, w, f32):
    """Bound of |y - y64|.  With c the relative roundings of a sum against its
    sum of magnitudes (as for the products): g and u are off by c(h) mag_g and
    c(h) mag_u; silu is 1.1-Lipschitz; a is off by 1.1 dg |u| + |silu(g)| du and
    a few roundings (2^-21 |a|); the down sum adds c(i).  Routing weights are
    off by 2^-19 relative: a logit's error c(h) sum|x||r| is under 2e-6 here and
    exponentials and divisions add a few roundings."""
    x = x.astype(np.float64)
    lim = np.zeros_like(ref)
    c = lambda k: 2 * (k / 32 + 104) * 2.0 ** -24
    wr = 2.0 ** -19 + 8 * c(x.shape[1])

    def one(xt, gu, dn, weight):
        g, u = gu @ xt
        mg, mu = np.abs(gu) @ np.abs(xt)
        sg = g * M.sigmoid(g)
        a = np.abs(sg * u)
        da = c(xt.size) * (1.1 * mg * np.abs(u) + np.abs(sg) * mu) + 2.0 ** -21 * a
        ad = np.abs(dn)
        return abs(weight) * (ad @ (da + c(u.size) * a) + (wr + c(16)) * (ad @ a))
    ids, _ = M.route(x @ l["router"].astype(np.float64).T, topk, l["scoring"], l.get("bias"), l["renormalize"],
                     l["scale"])
    for t in range(x.shape[0]):
        for s, e in enumerate(ids[t]):
            lim[t] += one(x[t], M.decode(l["gate_up"][0][e], l["gate_up"][1][e]),
                          M.decode(l["down"][0][e, 0], l["down"][1][e, 0]), w[t, s])
        if l.get("shared") is not None:
            (gc, gs), (dc, ds) = l["shared"]
            lim[t] += one(x[t], M.decode(gc[0], gs[0]), M.decode(dc[0, 0], ds[0, 0]), 1.0)
    return lim if f32 else lim + np.maximum(np.abs(ref) * 2.0 ** -11, 2.0 ** -25) * 1.001


MOE = [
    dict(t=1, e=4, h=32, i=32, topk=1),
    dict(t=1, e=256, h=2048, i=512, topk=8),
    dict(t=3, e=8, h=128, i=96, topk=8, si=32),
    dict(t=5, e=60, h=1440, i=352, topk=4, si=736, scoring="sigmoid", bias=True),
    dict(t=16, e=64, h=512, i=160, topk=6, si=160, gate=True, bias=True),
    dict(t=16, e=16, h=288, i=64, topk=16, renorm=False, scale=2.5),
    dict(t=2, e=1024, h=256, i=32, topk=10, scoring="sigmoid", renorm=False),
    dict(t=9, e=65, h=544, i=288, topk=3, scoring="sigmoid", scale=0.5, si=96, gate=True),
    dict(t=16, e=1, h=256, i=1056, topk=1),
]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("case", MOE, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()))
def test_moe(case, f32):
    import torch
    import gemm_exl3_linear_amd as X
    c = dict(case)
    topk = c.pop("topk")
    x, l = moe_case(77 + c["t"] + c["h"], **c)
    t, h = x.shape
    layer = moe_layer(l)
    buf = torch.full((t, h + 3), 7.0, dtype=torch.float32 if f32 else torch.float16, device=G.dev())
    ids = torch.full((t, topk), -1, dtype=torch.int32, device=G.dev())
    w = torch.zeros((t, topk), dtype=torch.float32, device=G.dev())
    xp = np.full((t, h + 8), np.nan, dtype=np.float16)
    xp[:, :h] = x
    ws = torch.zeros(X.exl3_mx4_moe_workspace_size(layer, t, topk), dtype=torch.uint8, device=G.dev())
    ref, rid, rw = M.moe(x, l, topk)
    lim = moe_limit(x, l, topk, ref, rw, f32)
    first = None
    for again in range(3):  # the same workspace three times, the same bits
        X.exl3_mx4_moe(G.to_dev(xp)[:, :h], layer, topk, out=buf[:, :h], topk_ids=ids, topk_weights=w, workspace=ws)
        np.testing.assert_array_equal(ids.cpu().numpy(), rid)
        np.testing.assert_allclose(w.cpu().numpy(), rw, rtol=2.0 ** -19 + 16 * (h / 32 + 104) * 2.0 ** -24)
        assert_within(buf[:, :h].cpu().numpy(), ref, lim, f"call {again}")
        assert (buf[:, h:] == 7.0).all()
        first = buf.clone() if first is None else first
        assert torch.equal(first, buf)
    y = X.exl3_mx4_moe(G.to_dev(x), layer, topk, out_dtype=buf.dtype)  # nothing optional
    assert torch.equal(y, first[:, :h])


def test_moe_one_workspace_serves_layers_and_sizes():
    import torch
    import gemm_exl3_linear_amd as X
    cases = [(moe_case(5, 16, 32, 256, 96, si=64), 4), (moe_case(6, 2, 128, 512, 32), 8), (moe_case(7, 7, 5, 64, 160), 2)]
    built = [(G.to_dev(x), moe_layer(l), k) for (x, l), k in cases]
    ws = torch.zeros(max(X.exl3_mx4_moe_workspace_size(l, x.shape[0], k) for x, l, k in built), dtype=torch.uint8,
                     device=G.dev())
    own = [X.exl3_mx4_moe(x, l, k) for x, l, k in built]
    for order in ([0, 1, 2], [2, 0, 1], [1, 1, 0], [2, 2, 0]):
        for i in order:
            x, l, k = built[i]
            for t in (x.shape[0], 1):
                y = X.exl3_mx4_moe(x[:t], l, k, workspace=ws)
                if t == x.shape[0]:
                    assert torch.equal(y, own[i])


def test_moe_ties_go_to_the_lower_expert():
    import torch
    import gemm_exl3_linear_amd as X
    x, l = moe_case(21, 3, 70, 64, 32)
    l["router"][:] = l["router"][0]
    l["router"][40] = 0  # logit 0 among equal ones
    x[0] = np.abs(x[0]) * np.sign(l["router"][0].astype(np.float64) + 1e-9)   # the others positive
    x[1] = -x[0]                                                                # the others negative
    x[2] = 0                                                                    # all zero
    layer = moe_layer(l)
    ids = torch.empty((3, 4), dtype=torch.int32, device=G.dev())
    X.exl3_mx4_moe(G.to_dev(x), layer, 4, topk_ids=ids)
    assert ids.tolist() == [[0, 1, 2, 3], [40, 0, 1, 2], [0, 1, 2, 3]]


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_moe_masked_experts_and_bad_tokens(scoring):
    # experts masked by a bias of -inf or the type's lowest value are taken
    # last; a NaN or infinite token keeps valid ids and spoils only its own row
    import torch
    import gemm_exl3_linear_amd as X
    x, l = moe_case(33, 6, 12, 96, 64, si=32, bias=True, scoring=scoring)
    l["bias"][[1, 4]] = -np.inf
    l["bias"][7] = np.finfo(np.float32).min
    x[2, 5], x[4, 0] = np.nan, np.inf
    layer = moe_layer(l)
    ids = torch.empty((6, 9), dtype=torch.int32, device=G.dev())
    w = torch.empty((6, 9), dtype=torch.float32, device=G.dev())
    y = X.exl3_mx4_moe(G.to_dev(x), layer, 9, out_dtype=torch.float32, topk_ids=ids, topk_weights=w).cpu().numpy()
    good = [0, 1, 3, 5]
    with np.errstate(invalid="ignore"):
        ref, rid, rw = M.moe(x[good], l, 9)
    np.testing.assert_array_equal(ids.cpu().numpy()[good], rid)
    assert not np.isin(rid, [1, 4, 7]).any()
    assert_within(y[good], ref, moe_limit(x[good], l, 9, ref, rw, True))
    for t in (2, 4):
        assert sorted(set(ids[t].tolist())) == sorted(ids[t].tolist()) and 0 <= min(ids[t]) and max(ids[t]) < 12
    assert np.isnan(y[2]).all() and not np.isfinite(y[4]).any()


# ---------------------------------------------------------------------------
# together, in graphs, on streams
# ---------------------------------------------------------------------------
def test_together_a_trellis_layer_as_mxfp4():
    """A trellis tensor's weights as MXFP4, in the Hadamard domain: decode,
    quantize, and the layer around both products; against the float64 layer
    with the same quantized weights (and rows)."""
    import torch
    import gemm_exl3_linear_amd as X
    from oracle import exl3_oracle as O
    k, n, m = 512, 384, 40
    d = G.linear_case(610, m, k, n, 4)
    w = G.weight(d)
    x = G.to_dev(d["x"])
    q = X.exl3_mx4_quantize(X.exl3_reconstruct(w).t().contiguous())
    wq = M.quantize(G.decoded(610, m, k, n, 4).T)
    np.testing.assert_array_equal(q.codes.cpu().numpy(), wq[0])
    xt = X.exl3_hadamard(x, sign_before=w.suh)
    xq = X.exl3_mx4_quantize(xt)
    zero = torch.zeros(n, dtype=torch.float16, device=G.dev())
    outs = [X.exl3_mx4_linear(xt, q, out_dtype=torch.float32),
            X.exl3_mx4_matmul(xq, q, bias=zero, out_dtype=torch.float32)]
    xh = xt.double().cpu().numpy()
    refs = [xh @ M.decode(*wq).T, M.decode(*M.quantize(xt.cpu().numpy())) @ M.decode(*wq).T]
    exact = O.linear(d["x"], d["trellis"], d["suh"], d["svh"], 4)
    for y, ref, loss in zip(outs, refs, (0.2, 0.3)):
        assert O.rel_frobenius(y.cpu().numpy(), ref) < 1e-6
        z = X.exl3_hadamard(y, sign_after=w.svh).cpu().numpy()
        # 4-bit operands: each costs about 0.12 of the norm (uniform within a
        # step of up to 1/3 of the value), well under these limits
        assert O.rel_frobenius(z, exact) < loss


def _graph_runs():
    import torch
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(90)
    runs = []
    x = G.to_dev(rng.standard_normal((37, 2048)).astype(np.float16))
    q, r = X.Exl3Mx4.empty(37, 2048, device=G.dev()), torch.empty_like(x)

    def quant():
        X.exl3_mx4_quantize(x, out=q)
        X.exl3_mx4_reconstruct(q, out=r)
    runs.append((quant, [q.codes, q.scales, r]))
    for m, n, k in ((1, 5120, 2048), (37, 640, 17408), (64, 512, 2048)):
        w, xx = mx(rand_mx(rng, n, k)), G.to_dev(rng.standard_normal((m, k)).astype(np.float16))
        y = torch.empty((m, n), dtype=torch.float32, device=G.dev())
        ws = torch.zeros(X.exl3_mx4_linear_workspace_size(w, m), dtype=torch.uint8, device=G.dev())
        runs.append((lambda w=w, xx=xx, y=y, ws=ws: X.exl3_mx4_linear(xx, w, out=y, workspace=ws), [y]))
    for m, n, k in ((1, 512, 17408), (40, 640, 4096), (700, 1100, 1056)):
        a, b = mx(rand_mx(rng, m, k)), mx(rand_mx(rng, n, k))
        y = torch.empty((m, n), dtype=torch.float32, device=G.dev())
        ws = torch.zeros(X.exl3_mx4_matmul_workspace_size(a, b), dtype=torch.uint8, device=G.dev())
        runs.append((lambda a=a, b=b, y=y, ws=ws: X.exl3_mx4_matmul(a, b, out=y, workspace=ws), [y]))
    for t, topk in ((1, 8), (16, 4)):
        xm, l = moe_case(91, t, 64, 512, 160, si=96, gate=True)
        layer, xd = moe_layer(l), G.to_dev(xm)
        y = torch.empty((t, 512), dtype=torch.float32, device=G.dev())
        ids = torch.empty((t, topk), dtype=torch.int32, device=G.dev())
        ws = torch.zeros(X.exl3_mx4_moe_workspace_size(layer, t, topk), dtype=torch.uint8, device=G.dev())
        runs.append((lambda xd=xd, layer=layer, topk=topk, y=y, ids=ids, ws=ws: X.exl3_mx4_moe(
            xd, layer, topk, out=y, topk_ids=ids, workspace=ws), [y, ids]))
    return runs


def test_graph_capture_and_replay():
    import torch
    runs = _graph_runs()
    refs = []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for run, outs in runs:
            run()
            run()
    torch.cuda.synchronize()
    refs = [[o.clone() for o in outs] for _, outs in runs]
    graphs = []
    for run, _ in runs:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        graphs.append(g)
    for i in range(4):
        for (run, outs), g, ref in zip(runs, graphs, refs):
            for o in outs:
                o.zero_()
            torch.cuda.synchronize()
            g.replay()
            torch.cuda.synchronize()
            for o, r in zip(outs, ref):
                assert torch.equal(o, r), f"replay {i}"
        for run, _ in runs:  # eager calls on the same workspaces in between
            run()
        torch.cuda.synchronize()


def test_two_streams_with_their_own_workspaces():
    import torch
    runs = [_graph_runs(), _graph_runs()]
    for rs in runs:
        for run, _ in rs:
            run()
    torch.cuda.synchronize()
    refs = [[[o.clone() for o in outs] for _, outs in rs] for rs in runs]
    for rs in runs:
        for _, outs in rs:
            for o in outs:
                o.zero_()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, rs in zip(streams, runs):
            with torch.cuda.stream(s):
                for run, _ in rs:
                    run()
    torch.cuda.synchronize()
    for rs, rr in zip(runs, refs):
        for (_, outs), ref in zip(rs, rr):
            assert all(torch.equal(o, r) for o, r in zip(outs, ref))


# ---------------------------------------------------------------------------
# scales outside fp16 next to infinities
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("m,n", [(1, 40), (4, 2064), (7, 40), (8, 2064), (12, 40), (16, 2064), (20, 140), (40, 140), (64, 140)])
def test_linear_infinity_next_to_far_scales(m, n):
    # every code is 1.0 (and x positive), so an infinite x gives an infinity
    # whatever the scales of its block and of the others
    import torch
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(15)
    codes = np.full((n, 160), 0x22, dtype=np.uint8)
    scales = rng.integers(110, 130, (n, 10)).astype(np.uint8)
    scales[: n // 2, 2] = 160
    scales[n // 3:, 7] = 60
    x = np.abs(rng.standard_normal((m, 320))).astype(np.float16)
    x[0, 70] = x[m // 2, 239] = x[m - 1, 5] = np.inf
    y = X.exl3_mx4_linear(G.to_dev(x), mx((codes, scales)), out_dtype=torch.float32).cpu().numpy()
    rows = np.unique([0, m // 2, m - 1])
    assert np.isposinf(y[rows]).all()
    rest = np.delete(np.arange(m), rows)
    ref, mag = M.product(x[rest], M.decode(codes, scales))
    assert_within(y[rest], ref, bound(ref, mag, 320, True))


@pytest.mark.parametrize("t", [1, 3, 6, 16])
def test_moe_activations_past_fp32(t):
    # silu(g) u passes fp32's range for token 0 only, and stays an infinity
    import torch
    import gemm_exl3_linear_amd as X
    x, l = moe_case(41, t, 3, 64, 64)
    for k, s in (("gate_up", 190), ("down", 127)):
        l[k][0][:] = 0x22
        l[k][1][:] = s
    x[:] = 0
    x[0] = 1
    y = X.exl3_mx4_moe(G.to_dev(x), moe_layer(l), 2, out_dtype=torch.float32).cpu().numpy()
    assert np.isposinf(y[0]).all() and (y[1:] == 0).all()


@pytest.mark.parametrize("t", [1, 5, 6, 16])
def test_moe_any_scale_byte(t):
    # gate and up blocks on either side of fp16's range, a NaN block of one
    # expert, far and NaN scales of down
    import torch
    import gemm_exl3_linear_amd as X
    x, l = moe_case(43, t, 4, 288, 96, si=64)
    x = (x * np.float16(2.0 ** -3)).astype(np.float16)
    gs, ds = l["gate_up"][1], l["down"][1]
    gs[1, :, 5] = 90
    gs[2, 0, 7, 3], gs[2, 1, 7, 3] = 150, 95
    x[:, 96:128] = 0  # the block of scale 150
    ds[0, 0, 3], ds[0, 0, 4] = 60, 190
    gs[3, 0, 9, 8] = ds[3, 0, 11, 1] = 255
    y = X.exl3_mx4_moe(G.to_dev(x), moe_layer(l), 2, out_dtype=torch.float32).cpu().numpy()
    ref, ids, w = M.moe(x, l, 2)
    clean = dict(l)
    for name in ("gate_up", "down"):
        clean[name] = (l[name][0], np.where(l[name][1] == 255, 127, l[name][1]))
    lim = moe_limit(x, clean, 2, ref, w, True)
    assert_within(y, ref, lim)


# ---------------------------------------------------------------------------
# products large enough for the tiles in LDS
# ---------------------------------------------------------------------------
# 128 x 128 tiles with k shared by 28 workgroups, by two, and not; 256 x 256 tiles
TILES = [(65, 1111, 46496), (128, 1028, 26080), (700, 1290, 4128), (1000, 2602, 1312), (2040, 7700, 288), (4097, 4100, 224)]


@pytest.mark.parametrize("aligned", [False, True])
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("m,n,k", TILES)
def test_matmul_tiles(m, n, k, f32, aligned):
    import torch
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(m + n + k + aligned)
    a, b = rand_mx(rng, m, k), rand_mx(rng, n, k, lo=112, hi=122)
    a[1][m - 1, -1] = b[1][n // 2, 0] = 255
    bias = rng.standard_normal(n).astype(np.float16) if f32 == aligned else None
    dt = torch.float32 if f32 else torch.float16
    first, pitch = (8, (n + 7) // 8 * 8 + 16) if aligned else (1, n + 2)
    buf = torch.full((m, pitch), 7.0, dtype=dt, device=G.dev())
    y = X.exl3_mx4_matmul(mx(a), mx(b), bias=None if bias is None else G.to_dev(bias), out=buf[:, first:first + n])
    da, db = M.decode(*a).astype(np.float32), M.decode(*b).astype(np.float32)  # exact
    rows = np.unique(np.concatenate([np.arange(0, m, max(1, m // 90)), np.arange(max(0, m - 20), m)]))
    ref, _ = M.product(da[rows], db, bias)
    mag = M.product(np.nan_to_num(da[rows]), np.nan_to_num(db), bias)[1]
    assert_within(y.cpu().numpy()[rows], ref, bound(ref, mag, k, f32), f"{m}x{n}x{k}")
    rest = np.isnan(y.cpu().numpy())
    assert rest[:, n // 2].all() and rest[m - 1].all() and rest.sum() == m + n - 1
    assert (buf[:, :first] == 7.0).all() and (buf[:, first + n:] == 7.0).all()


def test_matmul_tiles_of_one_scale_are_exact():
    # multiples of 1/4 below 36 k < 2^20, every element, in any order
    import torch
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(3)
    for m, n, k in ((192, 900, 26080), (1300, 1500, 2080), (2048, 7680, 320)):
        a, b = rand_mx(rng, m, k, lo=127, hi=127), rand_mx(rng, n, k, lo=127, hi=127)
        y = X.exl3_mx4_matmul(mx(a), mx(b), out_dtype=torch.float32)
        np.testing.assert_array_equal(y.double().cpu().numpy(), M.product(M.decode(*a), M.decode(*b))[0])


def test_matmul_workspace_serves_other_sizes():
    # the same scratch, full of NaNs at first, for products cut differently, two in a row
    import torch
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(4)
    sizes = [(65, 1111, 46496), (700, 1290, 4128), (4097, 4100, 224), (1000, 2602, 1312), (20, 5000, 4096)]
    built = [(mx(rand_mx(rng, m, k)), mx(rand_mx(rng, n, k))) for m, n, k in sizes]
    own = [X.exl3_mx4_matmul(a, b) for a, b in built]
    ws = torch.full((max(X.exl3_mx4_matmul_workspace_size(a, b) for a, b in built),), 255, dtype=torch.uint8, device=G.dev())
    for i in (0, 1, 2, 3, 4, 2, 0, 3, 0, 0):
        assert torch.equal(X.exl3_mx4_matmul(*built[i], workspace=ws), own[i])


# the rows of a k that is not whole units, of weight rows that start at any byte of
# a dword of scales, with k shared and not, one column over a tile; and rows too far
# apart for 32-bit offsets
@pytest.mark.parametrize("m,n,k,pitch", [(17, 129, 5152, 0), (33, 257, 4160, 8), (49, 128, 2080, 8), (64, 1, 32, 0),
                                         (32, 2, 17440, 0), (48, 40000, 96, 0), (18, 33, 320, (1 << 24) + 8)])
def test_linear_shared_rows(m, n, k, pitch):
    import torch
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(m + n + k)
    w = rand_mx(rng, n, k, lo=112, hi=122)
    w[1][n - 1, -1] = 90   # outside fp16
    w[0][0, 16:32], w[1][0, 1 % (k // 32)] = (w[0][0, 16:32], w[1][0, 0]) if k == 32 else (0, 0)  # zeros at 2^-127
    x = rng.standard_normal((m, k)).astype(np.float16)
    bias = rng.standard_normal(n).astype(np.float16)
    if pitch > k:
        big = torch.empty((m - 1) * pitch + k, dtype=torch.float16, device=G.dev())
        xd = big.as_strided((m, k), (pitch, 1))
        xd.copy_(G.to_dev(x))
    else:
        xd = torch.full((m, k + pitch), float("nan"), dtype=torch.float16, device=G.dev())[:, :k]
        xd.copy_(G.to_dev(x))
    y = X.exl3_mx4_linear(xd, mx(w), bias=G.to_dev(bias), out_dtype=torch.float32)
    ref, mag = M.product(x, M.decode(*w), bias)
    assert_within(y.cpu().numpy(), ref, bound(ref, mag, k, True), f"{m}x{n}x{k}")
    ws = X.exl3_mx4_linear_workspace_size(mx(w), m)
    ws = torch.full((ws + 16,), 255, dtype=torch.uint8, device=G.dev())
    for _ in range(2):
        again = X.exl3_mx4_linear(xd, mx(w), bias=G.to_dev(bias), out_dtype=torch.float32, workspace=ws)
        assert torch.equal(again, y)


@pytest.mark.parametrize("m,n,k", [(9, 4613, 17440), (16, 17408, 4640)])
def test_linear_shared_rows_of_large_weights(m, n, k):
    import torch
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(m + n)
    w = rand_mx(rng, n, k, lo=112, hi=122)
    w[1][n // 2, 7], w[1][5, k // 32 - 1] = 90, 255
    x = rng.standard_normal((m, k)).astype(np.float16)
    y = X.exl3_mx4_linear(G.to_dev(x), mx(w), out_dtype=torch.float32).cpu().numpy()
    cols = np.unique(np.concatenate([np.arange(0, n, 37), [5, n // 2], np.arange(n - 140, n)]))
    wc = M.decode(w[0][cols], w[1][cols])
    ref, _ = M.product(x, wc)
    assert_within(y[:, cols], ref, bound(ref, M.product(x, np.nan_to_num(wc))[1], k, True))
    assert np.isnan(y).sum() == m


def test_calls_on_another_stream_take_their_memory_there():
    # outputs and workspaces that the call makes itself belong to its stream:
    # while the current stream is busy, its freed blocks are not taken over
    import torch
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(50)
    x, l = moe_case(51, 16, 32, 512, 256, si=64)
    layer, xd = moe_layer(l), G.to_dev(x)
    w = mx(rand_mx(rng, 512, 8192))
    rows = G.to_dev(rng.standard_normal((40, 8192)).astype(np.float16))
    q = X.exl3_mx4_quantize(rows)
    a, b = mx(rand_mx(rng, 700, 4128)), mx(rand_mx(rng, 1290, 4128))
    calls = [lambda s: X.exl3_mx4_moe(xd, layer, 6, stream=s), lambda s: X.exl3_mx4_linear(rows, w, stream=s),
             lambda s: X.exl3_mx4_matmul(a, b, stream=s), lambda s: X.exl3_mx4_quantize(rows, stream=s).codes,
             lambda s: X.exl3_mx4_reconstruct(q, stream=s)]
    want = [c(None) for c in calls]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    big = torch.randn(4096, 4096, device=G.dev())
    for _ in range(3):
        for c, y in zip(calls, want):
            for _ in range(4):
                junk = [torch.full((n,), 255, dtype=torch.uint8, device=G.dev()) for n in (1 << 14, 1 << 20, 1 << 22)]
                big = torch.tanh(big)
                del junk
            got = c(s)
            junk = [torch.full((n,), 255, dtype=torch.uint8, device=G.dev()) for n in (1 << 14, 1 << 20, 1 << 22)]
            s.synchronize()
            assert torch.equal(got, y)
            del junk


# every cut of a product: 16 x 16, 32 x 32 and 64 x 32 tiles at lengths with and
# without whole units, LDS tiles of a short k, and few columns, where the operands
# change places
CUTS = [(100, 50, 5152), (30, 30, 10240), (300, 300, 2048), (500, 500, 5120), (24, 2100, 2080), (17, 6000, 1024),
        (333, 1111, 2080), (500, 1000, 2048), (1500, 1400, 96), (2050, 1930, 32), (600, 1, 96), (129, 16, 2080),
        (5000, 3, 544), (4100, 16, 288), (17, 16, 64)]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("m,n,k", CUTS)
def test_matmul_cuts(m, n, k, f32):
    import torch
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(m + 3 * n + k)
    a, b = rand_mx(rng, m, k), rand_mx(rng, n, k, lo=112, hi=122)
    a[1][m // 3, 0] = b[1][n - 1, -1] = 255
    bias = rng.standard_normal(n).astype(np.float16)
    buf = torch.full((m, n + 3), 7.0, dtype=torch.float32 if f32 else torch.float16, device=G.dev())
    y = X.exl3_mx4_matmul(mx(a), mx(b), bias=G.to_dev(bias), out=buf[:, 1:n + 1])
    da, db = M.decode(*a), M.decode(*b)
    ref, _ = M.product(da, db, bias)
    mag = M.product(np.nan_to_num(da), np.nan_to_num(db), bias)[1]
    assert_within(y.cpu().numpy(), ref, bound(ref, mag, k, f32), f"{m}x{n}x{k}")
    assert (buf[:, 0] == 7.0).all() and (buf[:, n + 1:] == 7.0).all()


# rows shared through LDS: two, three and four groups of 16, k shared by many and
# whole, lengths that end inside a unit, weight rows that start at any byte of a dword
# of scales, a column over a tile, and rows too far apart for that
@pytest.mark.parametrize("m,n,k,pitch", [(17, 129, 17440, 0), (32, 2, 12320, 8), (33, 257, 13344, 8), (49, 128, 10336, 0),
                                         (64, 130, 17440, 16), (64, 5000, 2080, 0), (23, 17000, 416, 8),
                                         (18, 33, 17440, (1 << 24) + 8)])
def test_linear_long_shared_rows(m, n, k, pitch):
    import torch
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(m + n + k)
    w = rand_mx(rng, n, k, lo=112, hi=122)
    w[1][n - 1, -1], w[1][n // 2, 3] = 90, 255      # outside fp16, NaN
    w[0][0, 16:32], w[1][0, 1] = 0, 0               # zeros at 2^-127
    x = rng.standard_normal((m, k)).astype(np.float16)
    bias = rng.standard_normal(n).astype(np.float16)
    if pitch > k:
        xd = torch.empty((m - 1) * pitch + k, dtype=torch.float16, device=G.dev()).as_strided((m, k), (pitch, 1))
    else:
        xd = torch.full((m, k + pitch), float("nan"), dtype=torch.float16, device=G.dev())[:, :k]
    xd.copy_(G.to_dev(x))
    wd, bd = mx(w), G.to_dev(bias)
    y = X.exl3_mx4_linear(xd, wd, bias=bd, out_dtype=torch.float32)
    cols = np.unique(np.concatenate([np.arange(0, n, max(1, n // 200)), [0, n // 2], np.arange(max(0, n - 140), n)]))
    wc = M.decode(w[0][cols], w[1][cols])
    ref, _ = M.product(x, wc, bias[cols])
    got = y.cpu().numpy()
    assert_within(got[:, cols], ref, bound(ref, M.product(x, np.nan_to_num(wc), bias[cols])[1], k, True), f"{m}x{n}x{k}")
    assert np.isnan(got).sum() == m
    ws = torch.full((X.exl3_mx4_linear_workspace_size(wd, m) + 16,), 255, dtype=torch.uint8, device=G.dev())
    for _ in range(2):
        assert torch.equal(torch.nan_to_num(X.exl3_mx4_linear(xd, wd, bias=bd, out_dtype=torch.float32, workspace=ws)),
                           torch.nan_to_num(y))


@pytest.mark.parametrize("m,n,k", [(2, 4100, 4128), (4, 5000, 4640), (3, 70, 4128), (4, 4100, 96), (8, 4097, 288),
                                   (5, 4000, 2080), (9, 2000, 2080), (12, 9000, 544), (40, 600, 2080), (64, 8200, 288)])
def test_linear_cuts(m, n, k):
    import torch
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(m + n + k)
    w = rand_mx(rng, n, k, lo=112, hi=122)
    w[1][n - 1, -1], w[1][n // 2, 0] = 90, 255
    x = rng.standard_normal((m, k)).astype(np.float16)
    bias = rng.standard_normal(n).astype(np.float16)
    y = X.exl3_mx4_linear(G.to_dev(x), mx(w), bias=G.to_dev(bias), out_dtype=torch.float32).cpu().numpy()
    wd = M.decode(*w)
    ref, _ = M.product(x, wd, bias)
    assert_within(y, ref, bound(ref, M.product(x, np.nan_to_num(wd), bias)[1], k, True), f"{m}x{n}x{k}")


@pytest.mark.parametrize("m,n,k", [(1500, 1300, 4640), (1417, 17, 13664), (2100, 700, 7200)])
def test_matmul_long_k_shared_by_two(m, n, k):
    import torch
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(m)
    a, b = rand_mx(rng, m, k), rand_mx(rng, n, k, lo=112, hi=122)
    bias = rng.standard_normal(n).astype(np.float16)
    y = X.exl3_mx4_matmul(mx(a), mx(b), bias=G.to_dev(bias), out_dtype=torch.float32).cpu().numpy()
    rows = np.unique(np.concatenate([np.arange(0, m, 17), np.arange(m - 130, m)]))
    ref, mag = M.product(M.decode(a[0][rows], a[1][rows]), M.decode(*b), bias)
    assert_within(y[rows], ref, bound(ref, mag, k, True), f"{m}x{n}x{k}")


@pytest.mark.parametrize("dtype,rows,k,pad", [(np.float32, 3277, 5152, 0), (np.float32, 3300, 5120, 8),
                                              (np.float16, 6601, 5120, 16), (np.float16, 6701, 5024, 0)])
def test_reconstruct_past_the_caches(dtype, rows, k, pad):
    import torch
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(rows)
    q = rand_mx(rng, rows, k, lo=100, hi=140)
    q[1][rows - 1, -1] = 255
    buf = torch.full((rows, k + pad), 7.0, dtype=torch.float32 if dtype == np.float32 else torch.float16, device=G.dev())
    out = X.exl3_mx4_reconstruct(mx(q), out=buf[:, :k])
    want = M.decode(*q).astype(dtype)  # one rounding
    np.testing.assert_array_equal(out.cpu().numpy(), want)
    assert (buf[:, k:] == 7.0).all()


@pytest.mark.parametrize("f32", [False, True])
def test_matmul_output_past_the_caches(f32):
    # 64 MB and more in whole lines, ragged at the end of rows and columns
    import torch
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(60)
    m, n, k = (2100, 8090, 224) if f32 else (4099, 8250, 96)
    a, b = rand_mx(rng, m, k), rand_mx(rng, n, k, lo=112, hi=122)
    bias = rng.standard_normal(n).astype(np.float16)
    buf = torch.full((m, (n + 63) // 64 * 64), 7.0, dtype=torch.float32 if f32 else torch.float16, device=G.dev())
    y = X.exl3_mx4_matmul(mx(a), mx(b), bias=G.to_dev(bias), out=buf[:, :n]).cpu().numpy()
    rows = np.unique(np.concatenate([np.arange(0, m, 41), np.arange(m - 140, m)]))
    ref, mag = M.product(M.decode(a[0][rows], a[1][rows]), M.decode(*b), bias)
    assert_within(y[rows], ref, bound(ref, mag, k, f32))
    assert (buf[:, n:] == 7.0).all() and np.isfinite(y).all()


# ---------------------------------------------------------------------------
# offsets past 32 bits
# ---------------------------------------------------------------------------
def test_quantize_and_reconstruct_past_32_bits():
    import torch
    import gemm_exl3_linear_amd as X
    rows, k = 270000, 16384  # 4.4e9 elements
    x = torch.empty((rows, k), dtype=torch.float16, device=G.dev())
    torch.manual_seed(1)
    x.copy_(torch.randn(k, device=G.dev()))  # every row the same but for its own factor
    x *= torch.exp2((torch.arange(rows, device=G.dev()) % 9 - 4).half())[:, None]
    q = X.exl3_mx4_quantize(x)
    for first in (0, 131070, 262143, rows - 3):
        c, s = M.quantize(x[first:first + 3].cpu().numpy())
        np.testing.assert_array_equal(q.codes[first:first + 3].cpu().numpy(), c)
        np.testing.assert_array_equal(q.scales[first:first + 3].cpu().numpy(), s)
    x.zero_()
    X.exl3_mx4_reconstruct(q, out=x)
    for first in (0, 131070, 262143, rows - 3):
        want = M.decode(q.codes[first:first + 3].cpu().numpy(), q.scales[first:first + 3].cpu().numpy())
        np.testing.assert_array_equal(x[first:first + 3].cpu().numpy(), want.astype(np.float16))


@pytest.mark.parametrize("m", [1, 6, 14, 40])
def test_linear_and_matmul_of_weights_past_32_bits(m):
    import torch
    import gemm_exl3_linear_amd as X
    n, k = 540000, 16384  # 4.4 GB of codes
    torch.manual_seed(m)
    w = X.Exl3Mx4(torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, device=G.dev()),
                  torch.randint(112, 122, (n, k // 32), dtype=torch.uint8, device=G.dev()))
    x = torch.randn((m, k), device=G.dev()).half()
    cols = np.unique(np.concatenate([np.arange(20), np.arange(262134, 262154), np.arange(524278, 524298),
                                     np.arange(n - 130, n)]))
    wc = M.decode(w.codes[cols].cpu().numpy(), w.scales[cols].cpu().numpy())
    y = X.exl3_mx4_linear(x, w, out_dtype=torch.float32)[:, cols].cpu().numpy()
    ref, mag = M.product(x.cpu().numpy(), wc)
    assert_within(y, ref, bound(ref, mag, k, True))
    a = X.exl3_mx4_quantize(x)
    y = X.exl3_mx4_matmul(a, w, out_dtype=torch.float32)[:, cols].cpu().numpy()
    ref, mag = M.product(M.decode(a.codes.cpu().numpy(), a.scales.cpu().numpy()), wc)
    assert_within(y, ref, bound(ref, mag, k, True))


def test_matmul_output_past_32_bits():
    import torch
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(70)
    m, n, k = 4100, 1050000, 64  # 4.3e9 elements
    a, b = rand_mx(rng, m, k), rand_mx(rng, n, k, lo=112, hi=122)
    y = X.exl3_mx4_matmul(mx(a), mx(b))
    da, db = M.decode(*a), M.decode(*b)
    for r in (0, 2047, 4090, m - 1):
        ref, mag = M.product(da[r:r + 1], db)
        assert_within(y[r:r + 1].cpu().numpy(), ref, bound(ref, mag, k, False), f"row {r}")


@pytest.mark.parametrize("t", [1, 7])
def test_moe_of_arenas_past_32_bits(t):
    # the last four of 1024 experts are chosen; alone, they are a layer of four
    import torch
    import gemm_exl3_linear_amd as X
    h, i, e = 2048, 2112, 1024  # 4.4 GB of gate and up codes
    x, l = moe_case(80, t, 4, h, i, scoring="sigmoid", bias=True)
    big = {}
    for name, slots, n, k in (("gate_up", 2, i, h), ("down", 1, h, i)):
        codes = torch.zeros((e, slots, n, k // 2), dtype=torch.uint8, device=G.dev())
        scales = torch.full((e, slots, n, k // 32), 255, dtype=torch.uint8, device=G.dev())
        codes[e - 4:], scales[e - 4:] = G.to_dev(l[name][0]), G.to_dev(l[name][1])
        big[name] = X.Exl3Mx4Arena(codes, scales)
    router = torch.zeros((e, h), dtype=torch.float16, device=G.dev())
    router[e - 4:] = G.to_dev(l["router"])
    bias = torch.full((e,), -9.0, dtype=torch.float32, device=G.dev())
    bias[e - 4:] = G.to_dev(l["bias"])
    layer = X.Exl3Mx4Moe(X.Exl3MoeRouter(router, bias=bias, scoring="sigmoid"), big["gate_up"], big["down"])
    ids = torch.empty((t, 3), dtype=torch.int32, device=G.dev())
    y = X.exl3_mx4_moe(G.to_dev(x), layer, 3, out_dtype=torch.float32, topk_ids=ids).cpu().numpy()
    ref, rid, rw = M.moe(x, l, 3)
    np.testing.assert_array_equal(ids.cpu().numpy(), rid + e - 4)
    assert_within(y, ref, moe_limit(x, l, 3, ref, rw, True))


@pytest.mark.parametrize("m,n,k", [(5, 512, 17408), (8, 131, 17440), (7, 40, 13344)])
def test_linear_few_long_rows(m, n, k):
    import torch
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(m + n + k)
    w = rand_mx(rng, n, k, lo=112, hi=122)
    w[1][n - 1, -1], w[1][n // 2, 0] = 90, 255
    x = np.full((m, k + 8), np.nan, dtype=np.float16)
    x[:, :k] = rng.standard_normal((m, k))
    bias = rng.standard_normal(n).astype(np.float16)
    y = X.exl3_mx4_linear(G.to_dev(x)[:, :k], mx(w), bias=G.to_dev(bias), out_dtype=torch.float32).cpu().numpy()
    wd = M.decode(*w)
    ref, _ = M.product(x[:, :k], wd, bias)
    assert_within(y, ref, bound(ref, M.product(x[:, :k], np.nan_to_num(wd), bias)[1], k, True), f"{m}x{n}x{k}")
