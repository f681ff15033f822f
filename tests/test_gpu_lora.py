"""Low-rank adapters on the GPU against the float64 oracle.

Tolerances.  With H_j = sum |a_j||x|: h_j = a_j x is off by at most 2 (k/32 + 104) 2^-24
H_j (exact products, fp32 sums as in the other products of this library); h is carried on
with an error of at most 2^-22 |h_j| + 2^-38 max|h|; the sum over the rank is of exact
products again, 2 (r/16 + 104) 2^-24 sum |b_j| H_j; then the factor, and the addition to
base, a rounding of at most 2^-24 each, of values no larger than the sum of magnitudes.
An fp16 output adds half a step, 2^-11 of the value (2^-25 below the normals)."""
import numpy as np
import pytest

from oracle import serve_oracle as S
from tests import _gpu as G

pytestmark = pytest.mark.gpu


def bound(y, mag, peak, base, k, rank, f32):
    b = ((2 * (k / 32 + 104) + 2 * (rank / 16 + 104) + 16) * 2.0 ** -24 * mag + 2.0 ** -38 * peak
         + 2.0 ** -23 * (np.abs(0.0 if base is None else base) + mag) + 2.0 ** -149)
    return b if f32 else b + np.maximum(np.abs(y) * 2.0 ** -11, 2.0 ** -25) * 1.001


def case(m, k, n, rank, adapters, seed=0, f32=False, ranks=False, scales=True, none=0.2, base=True, rows=None):
    rng = np.random.default_rng(m * 3 + k + n * 7 + rank + adapters + seed)
    d = dict(x=rng.standard_normal((m, k)).astype(np.float16),
             a=(rng.standard_normal((adapters, rank, k)) * k ** -0.5).astype(np.float16),
             b=(rng.standard_normal((adapters, n, rank)) * rank ** -0.5).astype(np.float16),
             base=rng.standard_normal((m, n)).astype(np.float32 if f32 else np.float16) if base else None,
             scales=rng.uniform(0.5, 2, adapters).astype(np.float32) if scales else None,
             ranks=rng.integers(0, rank + 1, adapters).astype(np.int32) if ranks else None)
    if rows is None:
        rows = rng.integers(0, adapters, m) if adapters else np.zeros(m)
        rows = np.where(rng.random(m) < none, rng.choice([-1, adapters, adapters + 7, -(1 << 31), (1 << 31) - 1], m),
                        rows)
    d["rows"] = np.asarray(rows).astype(np.int32)
    return d


def handle(d):
    import gemm_exl3_linear_amd as X
    put = lambda v: None if v is None else G.to_dev(v)
    return X.Exl3Lora(put(d["a"]), put(d["b"]), scales=put(d["scales"]), ranks=put(d["ranks"]))


def reference(d):
    return S.lora(d["x"], d["a"], d["b"], d["rows"], d["base"], d["scales"], d["ranks"])


def check(got, d, f32, what=""):
    y, mag, peak = reference(d)
    lim = bound(y, mag, peak, d["base"], d["x"].shape[1], d["a"].shape[1], f32)
    got = got.cpu().numpy().astype(np.float64)
    np.testing.assert_array_equal(np.isnan(got), np.isnan(y), err_msg=f"{what} NaN pattern")
    odd = ~np.isfinite(y)
    np.testing.assert_array_equal(got[odd], y[odd], err_msg=f"{what} infinities")
    bad = ~odd & ~(np.abs(got - np.where(odd, 0, y)) <= np.where(odd, 0, lim))
    assert not bad.any(), (f"{what} {bad.sum()} of {bad.size} outside, first at {np.argwhere(bad)[0]}: "
                           f"{got[bad][0]!r} for {y[bad][0]!r}, limit {lim[bad][0]!r}")


def call(d, f32, **kw):
    import torch
    import gemm_exl3_linear_amd as X
    base = None if d["base"] is None else G.to_dev(d["base"])
    return X.exl3_lora(G.to_dev(d["x"]), handle(d), G.to_dev(d["rows"]), base,
                       out_dtype=torch.float32 if f32 else torch.float16, **kw)


SHAPES = [  # m, k, n, rank, adapters
    (1, 8, 1, 8, 1), (1, 2048, 512, 16, 3), (1, 5120, 1111, 64, 2), (1, 520, 300, 256, 1), (2, 64, 64, 8, 2),
    (2, 5120, 640, 16, 8), (3, 40, 17, 24, 5), (4, 2056, 257, 128, 4), (5, 136, 100, 40, 1), (8, 1024, 96, 16, 64),
    (15, 72, 33, 32, 2), (16, 264, 65, 16, 16), (17, 1448, 129, 8, 3), (33, 512, 31, 48, 1), (40, 2048, 512, 16, 40),
    (63, 96, 256, 16, 2), (64, 1000, 320, 16, 64), (65, 328, 70, 64, 9), (100, 88, 520, 256, 3), (129, 640, 48, 104, 20),
    (200, 4096, 128, 16, 1), (333, 2056, 300, 40, 7), (600, 136, 1000, 8, 4), (1000, 256, 64, 64, 100),
    (1025, 64, 257, 16, 1000), (1500, 520, 640, 72, 3), (2000, 8, 8, 128, 4), (257, 17408, 24, 16, 2),
]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("m,k,n,rank,adapters", SHAPES)
def test_lora(m, k, n, rank, adapters, f32):
    d = case(m, k, n, rank, adapters, f32=f32, ranks=bool(m % 2), scales=bool((m + rank) % 3))
    check(call(d, f32), d, f32)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("m,k,n,rank,adapters", [(1, 2048, 512, 16, 3), (3, 264, 100, 24, 2), (64, 328, 320, 16, 30),
                                                 (500, 136, 129, 64, 5)])
def test_lora_without_base_and_in_place(m, k, n, rank, adapters, f32):
    import torch
    import gemm_exl3_linear_amd as X
    d = case(m, k, n, rank, adapters, f32=f32, none=0.4)
    put = G.to_dev
    y = put(d["base"])
    X.exl3_lora(put(d["x"]), handle(d), put(d["rows"]), y, out=y)
    check(y, d, f32, "in place")
    away = (d["rows"] < 0) | (d["rows"] >= adapters)
    np.testing.assert_array_equal(y.cpu().numpy()[away], d["base"][away])
    apart = call(d, f32)
    assert torch.equal(apart, y)
    d["base"] = None
    got = call(d, f32)
    check(got, d, f32, "without base")
    assert (got.cpu().numpy()[away] == 0).all()


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("m", [1, 2, 7, 64, 300])
def test_lora_strides_and_what_lies_between(m, f32):
    import torch
    import gemm_exl3_linear_amd as X
    dt = torch.float32 if f32 else torch.float16
    for k, n, rank, xpad, bpad, ypad, yoff in ((72, 100, 16, 8, 3, 5, 1), (512, 256, 8, 24, 8, 16, 8),
                                                (264, 77, 40, 0, 1, 0, 0)):
        d = case(m, k, n, rank, 4, f32=f32)
        xb = torch.full((m, k + xpad), float("nan"), dtype=torch.float16, device=G.dev())
        xb[:, :k] = G.to_dev(d["x"])
        bb = torch.full((m, n + bpad), float("nan"), dtype=dt, device=G.dev())
        bb[:, :n] = G.to_dev(d["base"])
        yb = torch.full((m + 2, yoff + n + ypad), 7.0, dtype=dt, device=G.dev())
        X.exl3_lora(xb[:, :k], handle(d), G.to_dev(d["rows"]), bb[:, :n], out=yb[1:m + 1, yoff:yoff + n])
        check(yb[1:m + 1, yoff:yoff + n], d, f32)
        yb[1:m + 1, yoff:yoff + n] = 7.0
        assert (yb == 7.0).all()


ORDERS = {
    "one": lambda m, L: np.zeros(m),
    "last": lambda m, L: np.full(m, L - 1),
    "none": lambda m, L: np.full(m, -1),
    "runs": lambda m, L: np.arange(m) * L // m,
    "turns": lambda m, L: np.arange(m) % L,
    "back": lambda m, L: (m - 1 - np.arange(m)) * L // m,
    "few": lambda m, L: np.where(np.arange(m) % 13 == 5, L - 1, -1),
    "lonely": lambda m, L: np.where(np.arange(m) == m // 2, 0, L - 1),
}


@pytest.mark.parametrize("order", list(ORDERS))
@pytest.mark.parametrize("m", [1, 2, 16, 17, 64, 65, 130, 1024, 1100])
def test_lora_orders_of_rows(m, order):
    for L in (1, 5, 70):
        d = case(m, 72, 40, 16, L, f32=True, rows=ORDERS[order](m, L))
        check(call(d, True), d, True, f"{L}")


@pytest.mark.parametrize("m", [1, 3, 16, 64, 200, 1030])
def test_lora_of_whole_numbers_is_exact(m):
    """Sums of whole numbers below 2^22 stand for themselves at every step."""
    rng = np.random.default_rng(m)
    for k, n, rank, L in ((264, 70, 16, 6), (1000, 33, 40, 3), (64, 300, 8, 1)):
        d = case(m, k, n, rank, L, f32=True, scales=False)
        d["x"] = rng.integers(-2, 3, d["x"].shape).astype(np.float16)
        d["a"] = rng.integers(-2, 3, d["a"].shape).astype(np.float16)
        d["b"] = rng.integers(-3, 4, d["b"].shape).astype(np.float16)
        d["base"] = rng.integers(-99, 100, d["base"].shape).astype(np.float32)
        np.testing.assert_array_equal(call(d, True).cpu().numpy(), reference(d)[0])


@pytest.mark.parametrize("n", [8, 63, 200, 1111, 4096, 4101])
@pytest.mark.parametrize("rank", [8, 16, 24, 64, 72, 136, 256])
def test_lora_many_rows_of_whole_numbers_are_exact(rank, n):
    """Long segments, several tiles a workgroup, every column: each sum is a whole number
    below 2^22 in magnitude (100 * 2 * 2 by rank * 3), which fp32 and both pieces hold."""
    import torch
    import gemm_exl3_linear_amd as X
    g = torch.Generator(device=G.dev()).manual_seed(rank * 7 + n)
    whole = lambda lo, hi, *s: torch.randint(lo, hi, s, generator=g, device=G.dev())
    k = 104
    for m, L in ((600, 3), (2100, 1), (5000, 7)):
        x, a = whole(-2, 3, m, k).half(), whole(-2, 3, L, rank, k).half()
        b, rows = whole(-3, 4, L, n, rank).half(), whole(-1, L, m).int()
        lora = X.Exl3Lora(a, b)
        base = whole(-99, 100, m, n).float()
        ref = base.double()
        for i in range(L):
            mine = rows == i
            ref[mine] += (x[mine].double() @ a[i].double().T) @ b[i].double().T
        for _ in range(3):
            y = X.exl3_lora(x, lora, rows, base)
            assert torch.equal(y.double(), ref), (m, L)
        y = base.clone()
        X.exl3_lora(x, lora, rows, y, out=y)
        assert torch.equal(y.double(), ref), (m, L)
        small = whole(-9, 10, m, n).half()
        y = X.exl3_lora(x, lora, rows, small)
        ref += small.double() - base.double()
        assert torch.equal(y, ref.to(torch.float16)), (m, L)


@pytest.mark.parametrize("m", [1, 4, 40, 300])
@pytest.mark.parametrize("rank", [8, 16, 40, 256])
def test_lora_what_lies_past_a_rank_has_no_say(m, rank):
    """a and b hold NaN and infinities past each adapter's own rank, and adapters that no
    row names hold nothing else."""
    d = case(m, 136, 50, rank, 6, f32=True, ranks=True)
    d["ranks"] = np.array([rank, rank - 1, 1, 0, rank + 5, -3], dtype=np.int32)
    for i, r in enumerate(np.clip(d["ranks"], 0, rank)):
        d["a"][i, r:], d["b"][i, :, r:] = np.nan, np.inf
    d["rows"] = np.where(d["rows"] == 4, 5, d["rows"]).astype(np.int32)
    d["a"][4], d["b"][4] = np.nan, np.nan
    check(call(d, True), d, True)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("m", [2, 16, 64, 300])
def test_lora_bad_rows_stay_alone(m, f32):
    """NaN and infinities in one row's x, in one adapter and in one row's base."""
    d = case(m, 136, 50, 24, 5, f32=f32, rows=np.arange(m) % 5)
    d["x"][0, 3] = np.nan
    d["base"][m - 1, 7] = np.inf
    if m > 2:
        d["x"][5, 100] = np.inf
        d["a"][1, 20, 135], d["b"][2, 49, 3] = np.nan, np.inf
        d["b"][3, 0, 0] = np.nan
        d["base"][8, 0] = -np.inf
    check(call(d, f32), d, f32)


@pytest.mark.parametrize("m", [1, 16, 200])
def test_lora_large_and_small(m):
    """Inner sums far past fp16's range, far below it, and rows of both."""
    rng = np.random.default_rng(m)
    for xs, as_, bs in ((6e4, 6e4, 1e-7), (1e-7, 1e-7, 6e4), (6e4, 1.0, 1.0), (1e-6, 1.0, 1.0), (1.0, 1.0, 6e4)):
        d = case(m, 264, 40, 24, 3, f32=True, base=False, scales=False)
        d["x"] = (d["x"] * 0.2 * xs).astype(np.float16)
        d["a"] = np.clip(d["a"].astype(np.float64) * 4 * as_, -65504, 65504).astype(np.float16)
        d["b"] = np.clip(d["b"] * bs, -65504, 65504).astype(np.float16)
        spread = np.exp2(rng.integers(-10, 1, (3, 24, 1)))
        d["a"] = (d["a"].astype(np.float64) * spread).astype(np.float16)
        check(call(d, True), d, True, f"{xs} {as_} {bs}")


def test_lora_no_rows_no_adapters():
    import torch
    import gemm_exl3_linear_amd as X
    d = case(5, 64, 30, 8, 0, f32=True)
    got = call(d, True)
    np.testing.assert_array_equal(got.cpu().numpy(), d["base"])
    d = case(0, 64, 30, 8, 2, f32=False)
    assert call(d, False).shape == (0, 30)
    with pytest.raises(ValueError):
        X.exl3_lora(torch.zeros((2, 64), dtype=torch.float16, device=G.dev()), handle(d),
                    torch.zeros(2, dtype=torch.int64, device=G.dev()))
    with pytest.raises(ValueError):
        X.exl3_lora(torch.zeros((2, 64), dtype=torch.float16, device=G.dev()), handle(d),
                    torch.zeros(2, dtype=torch.int32, device=G.dev()),
                    torch.zeros((2, 30), dtype=torch.float32, device=G.dev()), out_dtype=torch.float16)


def test_lora_one_workspace_serves_sizes():
    import torch
    import gemm_exl3_linear_amd as X
    made = [case(*s, f32=True) for s in ((1, 2048, 512, 16, 3), (64, 1000, 320, 16, 64), (333, 520, 300, 40, 7),
                                         (3, 40, 17, 24, 5), (1500, 136, 64, 64, 3))]
    hs = [handle(d) for d in made]
    need = max(X.exl3_lora_workspace_size(h, d["x"].shape[0]) for h, d in zip(hs, made))
    ws = torch.full((need,), 255, dtype=torch.uint8, device=G.dev())
    for i in (0, 1, 2, 3, 4, 3, 2, 1, 0, 4, 0):
        check(call(made[i], True, workspace=ws), made[i], True)


@pytest.mark.parametrize("m", [1, 70])
def test_lora_past_32_bits(m):
    """Adapters, x, base and y whose last elements lie past 4 GiB."""
    import torch
    import gemm_exl3_linear_amd as X
    k, n, rank, L = 64, 40, 256, 3
    d = case(m, k, n, rank, L, f32=True, rows=np.full(m, L - 1))
    put = G.to_dev
    pitch = (1 << 32) // max(m - 1, 1) // 2 // 8 * 8 + 64
    xb = torch.zeros(max(m, 2) * pitch, dtype=torch.float16, device=G.dev()).view(-1, pitch)
    xb[:m, :k] = put(d["x"])
    wide = torch.zeros((2 * max(m, 2), pitch // 2 + 4), device=G.dev())
    base, y = wide[:m, :n], wide[max(m, 2):max(m, 2) + m, :n]
    base.copy_(put(d["base"]))
    X.exl3_lora(xb[:m, :k], handle(d), put(d["rows"]), base, out=y)
    check(y, d, True)
    del xb, wide, base, y
    # a stack of 4096 adapters of 2.1 MB in a, and of 2.1 MB in b
    k, n, rank, L = 8192, 8192, 128, 4096
    rng = np.random.default_rng(1)
    a = torch.zeros((L, rank, k), dtype=torch.float16, device=G.dev())
    b = torch.zeros((L, n, rank), dtype=torch.float16, device=G.dev())
    last = case(m, k, n, rank, 1, f32=True, rows=np.zeros(m))
    a[L - 1], b[L - 1] = put(last["a"])[0], put(last["b"])[0]
    scales = torch.ones(L, device=G.dev()) * float(last["scales"][0])
    got = X.exl3_lora(put(last["x"]), X.Exl3Lora(a, b, scales=scales),
                      torch.full((m,), L - 1, dtype=torch.int32, device=G.dev()), put(last["base"]))
    check(got, last, True)


# ---------------------------------------------------------------------------
# many rows an adapter, and more rows than registers hold
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("m", [512, 1100, 9000])
def test_lora_many_rows_strides_and_what_lies_between(m, f32):
    test_lora_strides_and_what_lies_between(m, f32)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("m,k,n,rank,adapters", [(512, 136, 129, 64, 5), (1100, 72, 65, 8, 2), (700, 264, 8, 136, 1),
                                                 (9000, 64, 70, 16, 3), (9000, 64, 30, 24, 700),
                                                 (1300, 64, 1000, 256, 90), (513, 8, 9, 8, 4096)])
def test_lora_many_rows_without_base_and_in_place(m, k, n, rank, adapters, f32):
    test_lora_without_base_and_in_place(m, k, n, rank, adapters, f32)


@pytest.mark.parametrize("order", list(ORDERS))
@pytest.mark.parametrize("m", [512, 1023, 1025, 8192, 8193])
def test_lora_many_rows_orders(m, order):
    test_lora_orders_of_rows(m, order)


@pytest.mark.parametrize("m", [512, 1100])
@pytest.mark.parametrize("rank", [8, 16, 40, 64, 136, 256])
def test_lora_many_rows_what_lies_past_a_rank_has_no_say(m, rank):
    test_lora_what_lies_past_a_rank_has_no_say(m, rank)


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("m", [512, 1100])
def test_lora_many_rows_bad_rows_stay_alone(m, f32):
    test_lora_bad_rows_stay_alone(m, f32)


@pytest.mark.parametrize("m", [600, 1100])
def test_lora_many_rows_large_and_small(m):
    test_lora_large_and_small(m)


@pytest.mark.parametrize("past", [False, True])
def test_lora_many_rows_past_32_bits(past):
    """x whose last row ends just below 2^32 bytes, and past them; base and y past."""
    import torch
    import gemm_exl3_linear_amd as X
    m, k, n, rank, L = 600, 72, 70, 40, 3
    d = case(m, k, n, rank, L, f32=True)
    put = G.to_dev
    pitch = ((1 << 31) - 1) // m // 8 * 8 + (8 if past else 0)
    xb = torch.zeros(m * pitch, dtype=torch.float16, device=G.dev()).view(m, pitch)
    xb[:, pitch - k:] = put(d["x"])
    wide = torch.zeros((2, m, pitch + 3), device=G.dev())
    base, y = wide[0, :, 1:n + 1], wide[1, :, 2:n + 2]
    base.copy_(put(d["base"]))
    X.exl3_lora(xb[:, pitch - k:], handle(d), put(d["rows"]), base, out=y)
    check(y, d, True)


@pytest.mark.parametrize("m", [300, 700, 1100])
@pytest.mark.parametrize("rank", [8, 16, 32, 64, 128, 256])
def test_lora_bad_weights_stay_in_their_columns(m, rank):
    """NaN and infinities in single elements of B, next to and 16 columns away from sound
    ones, and in single ranks of A."""
    d = case(m, 136, 150, rank, 5, f32=True, rows=np.arange(m) % 5, none=0)
    d["b"][0, 17, 0], d["b"][0, 40, rank - 1], d["b"][0, 149, 3] = np.inf, np.nan, -np.inf
    d["b"][1, 0, :], d["b"][1, 64, 5] = np.nan, np.inf
    d["b"][2, ::7, rank // 2] = np.inf
    d["a"][3, rank - 1, 135] = -np.inf
    d["a"][4, 0, 0], d["b"][4, 33, 0] = np.inf, 0
    check(call(d, True), d, True)


@pytest.mark.parametrize("m", [70, 600, 1500])
def test_lora_graphs_take_rows_as_they_are(m):
    """A captured call finds its segments anew at every replay: same bits as eager calls."""
    import torch
    import gemm_exl3_linear_amd as X
    d = case(m, 264, 200, 24, 9, f32=True)
    lora, x, rows, base = handle(d), G.to_dev(d["x"]), G.to_dev(d["rows"]), G.to_dev(d["base"])
    ws = [torch.full((X.exl3_lora_workspace_size(lora, m),), 255, dtype=torch.uint8, device=G.dev()) for _ in range(2)]
    y, z = torch.empty_like(base), torch.empty_like(base)
    X.exl3_lora(x, lora, rows, base, out=y, workspace=ws[0])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        X.exl3_lora(x, lora, rows, base, out=y, workspace=ws[0])
    rng = np.random.default_rng(m)
    for order in ("one", "turns", "none", "runs", "few", "lonely"):
        d["rows"] = ORDERS[order](m, 9).astype(np.int32)
        d["x"] = rng.standard_normal(d["x"].shape).astype(np.float16)
        rows.copy_(G.to_dev(d["rows"]))
        x.copy_(G.to_dev(d["x"]))
        y.fill_(-3)
        graph.replay()
        X.exl3_lora(x, lora, rows, base, out=z, workspace=ws[1])
        torch.cuda.synchronize()
        assert torch.equal(y, z), order
        check(y, d, True, order)
