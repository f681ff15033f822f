"""MXFP4 operators on the GPU where memory, scales and logits are at their ends,
against the float64 oracle; bounds as derived in tests/test_gpu_mx4.py."""
import numpy as np
import pytest

from oracle import mx4_oracle as M
from tests import _gpu as G
from tests import test_gpu_mx4 as B

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------------------
# what lies behind a tensor
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("m,n,k", [(17, 129, 17440), (64, 130, 17440), (33, 257, 13344), (9, 4613, 17440)])
def test_linear_whatever_follows_the_scales(m, n, k):
    """n k / 32 bytes of scales end inside a dword: what else it holds is not the
    weight's, and the same call gives the same bits over it."""
    import torch
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(m + n)
    codes, scales = B.rand_mx(rng, n, k, lo=112, hi=122)
    size = scales.size
    assert size % 4
    room = torch.zeros(size + 64, dtype=torch.uint8, device=G.dev())
    room[:size] = G.to_dev(scales).reshape(-1)
    w = X.Exl3Mx4(G.to_dev(codes), room[:size].view(n, k // 32))
    x = rng.standard_normal((m, k)).astype(np.float16)
    xd = G.to_dev(x)
    got = []
    for fill in (0, 255, 90):
        room[size:] = fill
        got.append(X.exl3_mx4_linear(xd, w, out_dtype=torch.float32))
    cols = np.unique(np.concatenate([np.arange(0, n, max(1, n // 200)), np.arange(n - 2, n)]))
    ref, mag = M.product(x, M.decode(codes[cols], scales[cols]))
    B.assert_within(got[0].cpu().numpy()[:, cols], ref, B.bound(ref, mag, k, True))
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


# ---------------------------------------------------------------------------
# the highest scale bytes
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("hidden", [288, 4128])
@pytest.mark.parametrize("t", [1, 5, 6, 16])
def test_moe_down_at_the_highest_scale_bytes(t, hidden):
    """Blocks of 2^126 and 2^127 whose values pass bf16's range, against small
    activations, next to ordinary blocks and blocks at byte 0, in routed and shared
    experts; a token of zeros gives zeros."""
    import torch
    import gemm_exl3_linear_amd as X
    x, l = B.moe_case(47, t, 4, hidden, 288, si=96)
    x = (x * np.float16(2.0 ** -3)).astype(np.float16)
    if t > 1:
        x[t - 1] = 0
    l["gate_up"][1][:, 1] -= 60  # up: activations about 2^-64
    l["shared"][0][1][:, 1] -= 60
    for s in (l["down"][1], l["shared"][1][1]):
        s[:, :, ::3, 1], s[:, :, 1::3, 2], s[:, :, ::5, 0] = 254, 253, 0
    y = X.exl3_mx4_moe(G.to_dev(x), B.moe_layer(l), 2, out_dtype=torch.float32).cpu().numpy()
    ref, ids, w = M.moe(x, l, 2)
    assert np.isfinite(ref).all() and np.abs(ref).max() > 2.0 ** 50
    B.assert_within(y, ref, B.moe_limit(x, l, 2, ref, w, True))
    if t > 1:
        assert (y[t - 1] == 0).all()


@pytest.mark.parametrize("t", [1, 5, 6, 16])
def test_moe_infinite_activations_at_the_highest_scale_bytes(t):
    # silu(g) u passes fp32's range for token 0 only, every code of down is 4.0:
    # an infinity whatever the scales of its block and of the others
    import torch
    import gemm_exl3_linear_amd as X
    x, l = B.moe_case(48, t, 3, 64, 288)
    for k, s in (("gate_up", 190), ("down", 127)):
        l[k][0][:] = 0x22
        l[k][1][:] = s
    l["down"][0][:] = 0x66  # 4.0
    l["down"][1][:, :, ::2, 1], l["down"][1][:, :, ::3, 4] = 254, 253
    x[:] = 0
    x[0] = 1
    y = X.exl3_mx4_moe(G.to_dev(x), B.moe_layer(l), 2, out_dtype=torch.float32).cpu().numpy()
    assert np.isposinf(y[0]).all() and (y[1:] == 0).all()


@pytest.mark.parametrize("m", [1, 4, 8, 16, 24, 64])
def test_linear_at_the_highest_and_lowest_scale_bytes(m):
    import torch
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(m)
    n, k = 130, 544
    codes, scales = B.rand_mx(rng, n, k)
    scales[:] = rng.choice([0, 1, 2, 3], (n, k // 32))
    scales[::2] = rng.choice([251, 252, 253, 254], (n // 2, k // 32))
    x = (rng.standard_normal((m, k)) * 2.0 ** -12).astype(np.float16)
    y = X.exl3_mx4_linear(G.to_dev(x), B.mx((codes, scales)), out_dtype=torch.float32).cpu().numpy()
    ref, mag = M.product(x, M.decode(codes, scales))
    B.assert_within(y, ref, B.bound(ref, mag, k, True) + k * 2.0 ** -149)  # products below the normals are rounded too


# products of scales at both ends (as one factor they are ordinary), near fp32's
# largest, below its normals, below its least
ENDS = [("both", (0, 3), (251, 254)), ("large", (250, 251), (118, 119)), ("subnormal", (20, 21), (88, 89)),
        ("least", (0, 1), (0, 1))]


@pytest.mark.parametrize("name,la,lb", ENDS, ids=[e[0] for e in ENDS])
@pytest.mark.parametrize("m,n,k", [(1, 40, 544), (16, 5000, 288), (300, 290, 416), (64, 64, 256), (1100, 1300, 1056)])
def test_matmul_at_the_ends_of_the_scales(m, n, k, name, la, lb):
    import torch
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(m + k)
    a, b = B.rand_mx(rng, m, k, lo=la[0], hi=la[1]), B.rand_mx(rng, n, k, lo=lb[0], hi=lb[1])
    y = X.exl3_mx4_matmul(B.mx(a), B.mx(b), out_dtype=torch.float32).cpu().numpy()
    ref, mag = M.product(M.decode(*a), M.decode(*b))
    assert np.abs(ref).max() < 2.0 ** 128
    B.assert_within(y, ref, B.bound(ref, mag, k, True) + k * 2.0 ** -149)


@pytest.mark.parametrize("m,n", [(3, 40), (300, 290), (1100, 1300)])
def test_matmul_zero_blocks_at_any_scale(m, n):
    # blocks of zeros are zeros at 2^127 and 2^-127 alike, whatever they meet
    import torch
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(m)
    a, b = B.rand_mx(rng, m, 416, lo=112, hi=122), B.rand_mx(rng, n, 416, lo=112, hi=122)
    for q, at in ((a, 2), (b, 9)):
        q[0][:, 16 * at:16 * at + 16] = 0x80
        q[1][::2, at], q[1][1::2, at] = 254, 0
    a[1][:, 9], b[1][:, 2] = 254, 254
    y = X.exl3_mx4_matmul(B.mx(a), B.mx(b), out_dtype=torch.float32).cpu().numpy()
    ref, mag = M.product(M.decode(*a), M.decode(*b))
    B.assert_within(y, ref, B.bound(ref, mag, 416, True))


# ---------------------------------------------------------------------------
# tensors whose memory is swapped after their record was made
# ---------------------------------------------------------------------------
def test_weights_swapped_or_reloaded_between_calls():
    import torch
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(5)
    one, two = B.rand_mx(rng, 96, 512), B.rand_mx(rng, 160, 512)
    x = G.to_dev(rng.standard_normal((3, 512)).astype(np.float16))
    a = X.exl3_mx4_quantize(x)
    calls = lambda w: (X.exl3_mx4_linear(x, w), X.exl3_mx4_matmul(a, w), X.exl3_mx4_reconstruct(w))
    want = calls(B.mx(two))
    w = B.mx(one)
    calls(w)
    w.codes.data, w.scales.data = G.to_dev(two[0]), G.to_dev(two[1])
    for got in (calls(w), calls(w)):
        assert all(torch.equal(g, r) for g, r in zip(got, want))
    for t, host in ((w.codes, two[0]), (w.scales, two[1])):  # offloaded, its place taken, loaded again
        t.untyped_storage().resize_(0)
    taken = [torch.full((96, 256), 0x55, dtype=torch.uint8, device=G.dev()) for _ in range(8)]
    for t, host in ((w.codes, two[0]), (w.scales, two[1])):
        t.untyped_storage().resize_(host.size)
        t.copy_(G.to_dev(host))
    assert all(torch.equal(g, r) for g, r in zip(calls(w), want))
    X.exl3_mx4_quantize(torch.zeros((160, 512), dtype=torch.float16, device=G.dev()), out=w)
    assert not w.codes.any() and all((t == 0x55).all() for t in taken)

    (xm, l), (_, m) = B.moe_case(71, 4, 6, 128, 64, si=32, gate=True, bias=True), B.moe_case(72, 4, 6, 128, 96, si=64,
                                                                                          gate=True, bias=True)
    xd, layer, other = G.to_dev(xm), B.moe_layer(l), B.moe_layer(m)
    want = X.exl3_mx4_moe(xd, other, 3)
    X.exl3_mx4_moe(xd, layer, 3)
    pairs = [(layer.router.weight, other.router.weight), (layer.router.bias, other.router.bias),
             (layer.shared.gate, other.shared.gate)]
    for u, v in ((layer.gate_up, other.gate_up), (layer.down, other.down), (layer.shared.gate_up, other.shared.gate_up),
                 (layer.shared.down, other.shared.down)):
        pairs += [(u.codes, v.codes), (u.scales, v.scales)]
    for u, v in pairs:
        u.data = v.clone()
    assert torch.equal(X.exl3_mx4_moe(xd, layer, 3), want)


# ---------------------------------------------------------------------------
# routing of tokens whose logits are not finite
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("renorm", [False, True])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_moe_weights_of_tokens_without_finite_logits(scoring, renorm):
    import torch
    import gemm_exl3_linear_amd as X
    x, l = B.moe_case(61, 7, 12, 96, 64, bias=True, scoring=scoring, renorm=renorm, scale=0.5)
    r = l["router"]
    r[:, 0] = np.where(np.arange(12) % 3 == 0, 1, -1)  # an infinite x[0]: +inf for every third expert
    r[:, 1], r[:, 2] = -1, 1                           # x[1]: all -inf; x[2]: all +inf
    r[:, 3] = 1
    r[5, 3] = 0                                        # x[3]: +inf, but NaN for expert 5
    l["bias"][[2, 8]] = -np.inf                        # -inf next to finite logits
    for t in range(4):
        x[t, t] = np.inf
    x[4, 10] = np.nan
    ids = torch.empty((7, 12), dtype=torch.int32, device=G.dev())
    w = torch.empty((7, 12), dtype=torch.float32, device=G.dev())
    for topk in (12, 5):
        i, v = ids[:, :topk].contiguous(), w[:, :topk].contiguous()
        X.exl3_mx4_moe(G.to_dev(x), B.moe_layer(l), topk, topk_ids=i, topk_weights=v)
        with np.errstate(invalid="ignore"):
            logits = x.astype(np.float64) @ r.astype(np.float64).T
            rid, rw = M.route(logits, topk, scoring, l["bias"], renorm, 0.5)
        i, v = i.cpu().numpy(), v.cpu().numpy()
        assert all(sorted(set(q)) == sorted(q) and min(q) >= 0 and max(q) < 12 for q in i.tolist())
        np.testing.assert_array_equal(i[5:], rid[5:])
        np.testing.assert_allclose(v, rw, rtol=2.0 ** -19 + 16 * 107 * 2.0 ** -24)
        if scoring == "softmax":
            assert np.isnan(v[:5]).all() and np.isfinite(v[5:]).all()
        else:
            assert np.isnan(v[4]).all() and (renorm or (v[2] == 0.5).all() and (v[1] == 0).all())


def test_moe_sigmoid_without_a_bias_chooses_by_the_logit():
    # sigmoids that round to 1 in fp32 keep the order of their logits
    import torch
    import gemm_exl3_linear_amd as X
    x, l = B.moe_case(62, 2, 9, 64, 32, scoring="sigmoid")
    l["router"][:], x[:] = 0, 0
    l["router"][:, 0] = [20, 24, 40, 22, 18, -3, 30, 30, 1]
    x[:, 0] = 1
    ids = torch.empty((2, 6), dtype=torch.int32, device=G.dev())
    w = torch.empty((2, 6), dtype=torch.float32, device=G.dev())
    X.exl3_mx4_moe(G.to_dev(x), B.moe_layer(l), 6, topk_ids=ids, topk_weights=w)
    assert ids.tolist() == [[2, 6, 7, 1, 3, 0]] * 2
    np.testing.assert_allclose(w.cpu().numpy(), 1 / 6, rtol=2.0 ** -19)


# ---------------------------------------------------------------------------
# more rows than a call takes
# ---------------------------------------------------------------------------
def test_more_tokens_and_rows_than_a_call_takes():
    import torch
    import gemm_exl3_linear_amd as X
    x, l = B.moe_case(63, 41, 12, 160, 96, si=32, gate=True)
    layer, xd, n = B.moe_layer(l), G.to_dev(x), X.MX4_MOE_MAX_TOKENS
    ws = torch.zeros(X.exl3_mx4_moe_workspace_size(layer, n, 3), dtype=torch.uint8, device=G.dev())
    y = torch.empty((41, 160), dtype=torch.float32, device=G.dev())
    for i in range(0, 41, n):
        X.exl3_mx4_moe(xd[i:i + n], layer, 3, out=y[i:i + n], workspace=ws)
    ref, _, w = M.moe(x, l, 3)
    B.assert_within(y.cpu().numpy(), ref, B.moe_limit(x, l, 3, ref, w, True))

    rng = np.random.default_rng(64)
    q, rows = B.rand_mx(rng, 300, 2080, lo=112, hi=122), rng.standard_normal((150, 2080)).astype(np.float16)
    w, xd, n = B.mx(q), G.to_dev(rows), X.MX4_LINEAR_MAX_ROWS
    y = torch.empty((150, 300), dtype=torch.float32, device=G.dev())
    for i in range(0, 150, n):
        X.exl3_mx4_linear(xd[i:i + n], w, out=y[i:i + n])
    ref, mag = M.product(rows, M.decode(*q))
    B.assert_within(y.cpu().numpy(), ref, B.bound(ref, mag, 2080, True))


# ---------------------------------------------------------------------------
# expert layers of every kernel
# ---------------------------------------------------------------------------
# hidden past 4096 (more workgroups than CUs in down) with entries of one, of two to
# five and of more tokens; 129 to 1024 experts for few and many tokens; gate and up by
# one workgroup a CU, over lengths that end in a wave's first or second unit and inside
# a unit
LAYERS = [
    dict(t=1, e=8, h=5120, i=64, topk=3),
    dict(t=3, e=8, h=5120, i=96, topk=8, si=32),
    dict(t=16, e=8, h=4608, i=320, topk=3, si=64, gate=True),
    dict(t=16, e=32, h=4128, i=288, topk=2, bias=True),
    dict(t=16, e=256, h=512, i=32, topk=8),
    dict(t=9, e=128, h=256, i=64, topk=4, scoring="sigmoid"),
    dict(t=2, e=300, h=256, i=32, topk=8),
    dict(t=16, e=300, h=288, i=32, topk=4, renorm=False),
    dict(t=2, e=512, h=256, i=32, topk=16, scoring="sigmoid", bias=True),
    dict(t=16, e=512, h=256, i=32, topk=8, si=32, gate=True),
    dict(t=16, e=600, h=288, i=32, topk=6),
    dict(t=1, e=4, h=1440, i=32, topk=2, si=32),
    dict(t=16, e=4, h=2080, i=32, topk=2, si=64, gate=True),
    dict(t=5, e=2, h=2848, i=32, topk=1),
    dict(t=16, e=4, h=1312, i=64, topk=4, si=32),
]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("case", LAYERS, ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items()))
def test_moe_layers(case, f32):
    B.test_moe(case, f32)


# ---------------------------------------------------------------------------
# NaN blocks as quantization makes them: scale byte 255, codes 0
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("m,n,k", [(1, 40, 544), (16, 5000, 288), (40, 3, 96), (64, 64, 256), (300, 290, 416),
                                   (1100, 1300, 1056)])
def test_quantized_nans_reach_the_products(m, n, k):
    import torch
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(m + n)
    x, v = rng.standard_normal((m, k)).astype(np.float16), rng.standard_normal((n, k)).astype(np.float16)
    x[m // 2, k - 1], v[n - 1, 0], v[0, k // 2] = np.nan, np.inf, -np.inf
    a, w = X.exl3_mx4_quantize(G.to_dev(x)), X.exl3_mx4_quantize(G.to_dev(v))
    assert (w.scales == 255).sum() == 2 and (a.scales == 255).sum() == 1
    y = X.exl3_mx4_matmul(a, w, out_dtype=torch.float32).cpu().numpy()
    da, dw = M.decode(*M.quantize(x)), M.decode(*M.quantize(v))
    ref, _ = M.product(da, dw)
    B.assert_within(y, ref, B.bound(ref, M.product(np.nan_to_num(da), np.nan_to_num(dw))[1], k, True))
    x[m // 2, k - 1] = 1
    for rows in (x[:64], x[:7], x[:1]):
        y = X.exl3_mx4_linear(G.to_dev(rows), w, out_dtype=torch.float32).cpu().numpy()
        ref, _ = M.product(rows, dw)
        B.assert_within(y, ref, B.bound(ref, M.product(rows, np.nan_to_num(dw))[1], k, True))


@pytest.mark.parametrize("hidden", [288, 4128])
@pytest.mark.parametrize("t", [1, 5, 6, 16])
def test_moe_nan_blocks_of_zero_codes(t, hidden):
    # in a unit of ordinary blocks, and next to a block at byte 254
    import torch
    import gemm_exl3_linear_amd as X
    x, l = B.moe_case(49, t, 4, hidden, 288, si=96)
    x = (x * np.float16(2.0 ** -3)).astype(np.float16)
    l["gate_up"][1][:, 1] -= 60
    l["shared"][0][1][:, 1] -= 60
    for e, row, b in ((0, 3, 1), (1, 17, 8), (2, hidden - 1, 0), (3, 40, 5)):
        l["down"][0][e, 0, row, 16 * b:16 * b + 16] = 0
        l["down"][1][e, 0, row, b] = 255
    l["down"][1][3, 0, 40, 2] = 254
    l["shared"][1][0][0, 0, 60, 16:32], l["shared"][1][1][0, 0, 60, 1] = 0, 255
    y = X.exl3_mx4_moe(G.to_dev(x), B.moe_layer(l), 4, out_dtype=torch.float32).cpu().numpy()
    ref, ids, w = M.moe(x, l, 4)
    assert np.isnan(ref).sum() == 5 * t
    clean = {**l, "down": (l["down"][0], np.where(l["down"][1] == 255, 127, l["down"][1])),
             "shared": (l["shared"][0], (l["shared"][1][0], np.where(l["shared"][1][1] == 255, 127, l["shared"][1][1])))}
    B.assert_within(y, ref, B.moe_limit(x, clean, 4, ref, w, True))


@pytest.mark.parametrize("t", [1, 5, 16])
def test_moe_nan_blocks_of_zero_codes_in_gate_and_up(t):
    import torch
    import gemm_exl3_linear_amd as X
    x, l = B.moe_case(50, t, 4, 288, 96)
    l["gate_up"][0][2, 1, 7, 64:80], l["gate_up"][1][2, 1, 7, 4] = 0, 255
    y = X.exl3_mx4_moe(G.to_dev(x), B.moe_layer(l), 2, out_dtype=torch.float32).cpu().numpy()
    _, ids, _ = M.moe(x, l, 2)
    np.testing.assert_array_equal(np.isnan(y).all(1), (ids == 2).any(1))
    np.testing.assert_array_equal(np.isnan(y).any(1), (ids == 2).any(1))


# ---------------------------------------------------------------------------
# captured calls that make their own outputs and workspaces, and graphs that share one
# ---------------------------------------------------------------------------
def test_captured_calls_with_their_own_memory():
    import torch
    import gemm_exl3_linear_amd as X
    rng = np.random.default_rng(81)
    xm, l = B.moe_case(82, 16, 32, 512, 160, si=96, gate=True)
    layer, xd = B.moe_layer(l), G.to_dev(xm)
    w, rows = B.mx(B.rand_mx(rng, 640, 17408)), G.to_dev(rng.standard_normal((37, 17408)).astype(np.float16))
    a, b = B.mx(B.rand_mx(rng, 700, 4128)), B.mx(B.rand_mx(rng, 1290, 4128))

    def run():
        q = X.exl3_mx4_quantize(xd)
        return [X.exl3_mx4_moe(xd, layer, 4), X.exl3_mx4_linear(rows, w), X.exl3_mx4_matmul(a, b),
                X.exl3_mx4_reconstruct(q), X.exl3_mx4_moe(X.exl3_mx4_reconstruct(q), layer, 4)]
    want = run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = run()
    for i in range(4):
        for o in got:
            o.fill_(7.0)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, r) for o, r in zip(got, want)), f"replay {i}"
        run()


def test_graphs_of_layers_that_share_a_workspace():
    # one after the other on one stream, with eager calls on the same workspace between
    import torch
    import gemm_exl3_linear_amd as X
    cases = [(B.moe_case(83, 16, 32, 256, 96, si=64), 4), (B.moe_case(84, 2, 128, 512, 32), 8)]
    built = [(G.to_dev(x), B.moe_layer(l), k) for (x, l), k in cases]
    ws = torch.zeros(max(X.exl3_mx4_moe_workspace_size(l, x.shape[0], k) for x, l, k in built), dtype=torch.uint8,
                     device=G.dev())
    want = [X.exl3_mx4_moe(x, l, k) for x, l, k in built]
    outs, graphs = [torch.empty_like(y) for y in want], []
    for (x, l, k), y in zip(built, outs):
        X.exl3_mx4_moe(x, l, k, out=y, workspace=ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            X.exl3_mx4_moe(x, l, k, out=y, workspace=ws)
        graphs.append(g)
    for order in ([0, 1], [1, 0], [1, 1, 0, 0], [0, 1, 0, 1]):
        for y in outs:
            y.zero_()
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        assert all(torch.equal(y, r) for y, r in zip(outs, want))
        x, l, k = built[order[0]]
        X.exl3_mx4_moe(x[:1], l, k, workspace=ws)
