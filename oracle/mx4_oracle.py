"""Float64 oracle of the MXFP4 operators, from the format's definition (OCP
Microscaling Formats specification 1.0: E2M1 elements, E8M0 scales, blocks of
32) and the formulas in include/exl3.h.  Plain numpy; test infrastructure."""
import numpy as np

BLOCK = 32
MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def decode(codes, scales):
    """codes uint8 [..., k/2], scales uint8 [..., k/32] -> float64 [..., k]."""
    codes = np.asarray(codes)
    nib = np.stack([codes & 15, codes >> 4], axis=-1).reshape(*codes.shape[:-1], -1)
    v = MAGNITUDES[nib & 7] * np.where(nib & 8, -1.0, 1.0)
    s = np.asarray(scales).astype(np.int64)
    factor = np.where(s == 255, np.nan, np.ldexp(1.0, s - 127))
    return v * np.repeat(factor, BLOCK, axis=-1)


def quantize(x):
    """fp16 or fp32 [rows, k] -> codes uint8 [rows, k/2], scales uint8 [rows, k/32]."""
    x = np.asarray(x).astype(np.float64)
    b = x.reshape(x.shape[0], -1, BLOCK)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    top = np.abs(b).max(-1)
    _, e = np.frexp(top)                      # top = m 2^e, m in [0.5, 1)
    exp = np.where(top > 0, np.maximum(e - 1 - 2, -127), -127)
    q = b / np.ldexp(1.0, exp)[..., None]
    dist = np.abs(np.abs(q)[..., None] - MAGNITUDES)
    code = np.zeros(q.shape, dtype=np.int64)  # nearest; on a tie the even code
    best = dist[..., 0]
    for c in range(1, 8):
        take = (dist[..., c] < best) | ((dist[..., c] == best) & (c % 2 == 0))
        code = np.where(take, c, code)
        best = np.where(take, dist[..., c], best)
    code = code | (np.signbit(b) << 3)
    code = np.where(bad[..., None], 0, code).reshape(x.shape)
    scales = np.where(bad, 255, exp + 127).astype(np.uint8)
    return (code[:, 0::2] | (code[:, 1::2] << 4)).astype(np.uint8), scales


def product(a, b, bias=None):
    """a b^T (+ bias), and sum |a| |b| (+ |bias|) for error bounds."""
    a, b = np.asarray(a, dtype=np.float64), np.asarray(b, dtype=np.float64)
    y, mag = a @ b.T, np.abs(a) @ np.abs(b).T
    if bias is not None:
        y, mag = y + bias.astype(np.float64), mag + np.abs(bias.astype(np.float64))
    return y, mag


def sigmoid(z):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-z))


def route(logits, topk, scoring="softmax", bias=None, renormalize=True, scale=1.0):
    """ids [t, topk] (best first, ties to the lower id, NaN lowest) and weights."""
    logits = np.asarray(logits, dtype=np.float64)
    b = 0.0 if bias is None else np.asarray(bias, dtype=np.float64)
    if scoring == "softmax":
        choice = logits + b
        z = np.exp(choice - choice.max(-1, keepdims=True))
        score = z / z.sum(-1, keepdims=True)
    else:
        score = sigmoid(logits)
        choice = score + b
    rank = np.where(np.isnan(choice), -np.inf, choice)
    # a NaN ranks below -inf: order by (is NaN, -choice, id)
    ids = np.stack([np.lexsort((np.arange(r.size), -r, np.isnan(c)))[:topk] for r, c in zip(rank, choice)])
    w = np.take_along_axis(score, ids, 1)
    if renormalize:
        w = w / w.sum(-1, keepdims=True)
    return ids, w * scale


def swiglu(x, gate, up, down):
    g, u = x @ gate.T, x @ up.T
    return (g * sigmoid(g) * u) @ down.T


def moe(x, layer, topk):
    """layer: dict with router [E, h], gate_up and down as (codes [E, slots, n, k/2],
    scales), and optionally bias, scoring, renormalize, scale, shared (gate_up,
    down), shared_gate.  Returns y, ids, weights."""
    x = np.asarray(x, dtype=np.float64)
    ids, w = route(x @ layer["router"].astype(np.float64).T, topk, layer.get("scoring", "softmax"),
                   layer.get("bias"), layer.get("renormalize", True), layer.get("scale", 1.0))
    y = np.zeros_like(x)
    for e in np.unique(ids):
        gu = decode(layer["gate_up"][0][e], layer["gate_up"][1][e])
        dn = decode(layer["down"][0][e, 0], layer["down"][1][e, 0])
        for t, s in np.argwhere(ids == e):
            y[t] += w[t, s] * swiglu(x[t:t + 1], gu[0], gu[1], dn)[0]
    if layer.get("shared") is not None:
        (gc, gs), (dc, ds) = layer["shared"]
        gu, dn = decode(gc[0], gs[0]), decode(dc[0, 0], ds[0, 0])
        d = swiglu(x, gu[0], gu[1], dn)
        if layer.get("shared_gate") is not None:
            d = d * sigmoid(x @ layer["shared_gate"].astype(np.float64))[:, None]
        y += d
    return y, ids, w
