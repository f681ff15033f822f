"""The MXFP4 operators on cases of real use, and what they compute in plain torch.

Microscaled 4-bit floating point (MXFP4): a row is cut into blocks of 32
consecutive elements; a block holds 32 four-bit E2M1 codes (two to a byte, the
even element in the low half) and one E8M0 scale byte s, and stands for the
values e2m1(code) * 2^(s - 127).

  quantize  rows of fp16 or fp32 -> MXFP4 -> the values it stands for
            (exl3_mx4_quantize, then exl3_mx4_reconstruct)
  matmul    y = A B^T (+ bias), both operands MXFP4 (exl3_mx4_matmul)
  linear    y = x W^T (+ bias), fp16 rows against MXFP4 weights, few rows
            (exl3_mx4_linear)
  moe       a whole mixture-of-experts layer for a few tokens: router, top-k,
            SwiGLU experts in MXFP4, a shared expert (exl3_mx4_moe)
"""
import math

import torch

own = False

BLOCK = 32
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
TYPES = {"fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one hidden row of a decode step before a product with 4-bit activations
        {"name": "quantize_1x5120", "op": "quantize", "rows": 1, "k": 5120, "type": "fp16"},
        # the hidden rows of a 4096-token prefill
        {"name": "quantize_4096x5120", "op": "quantize", "rows": 4096, "k": 5120, "type": "fp16"},
        # an fp32 master weight converted once, ragged row count and odd block count
        {"name": "quantize_f32_10007x6880", "op": "quantize", "rows": 10007, "k": 6880, "type": "fp32"},
        # one token through an up projection, 4-bit weights and activations
        {"name": "matmul_1x5120x17408", "op": "matmul", "m": 1, "k": 5120, "n": 17408, "bias": False, "type": "fp16"},
        # a short ragged chunk, odd sizes everywhere, fp32 sums kept
        {"name": "matmul_333x2080x1111", "op": "matmul", "m": 333, "k": 2080, "n": 1111, "bias": True, "type": "fp32"},
        # the same projection at a 4096-token prefill
        {"name": "matmul_4096x5120x17408", "op": "matmul", "m": 4096, "k": 5120, "n": 17408, "bias": False, "type": "fp16"},
        # the smallest call: one token through a 2048 -> 512 projection
        {"name": "linear_1x2048x512", "op": "linear", "m": 1, "k": 2048, "n": 512, "bias": False, "type": "fp16"},
        # one token through an up projection of a dense layer
        {"name": "linear_1x5120x17408", "op": "linear", "m": 1, "k": 5120, "n": 17408, "bias": False, "type": "fp16"},
        # a verify batch through a down projection, odd row count, fp32 out
        {"name": "linear_37x17408x5120", "op": "linear", "m": 37, "k": 17408, "n": 5120, "bias": True, "type": "fp32"},
        # one token through a layer of 256 experts, eight of them routed to
        {"name": "moe_1x256x2048x512", "op": "moe", "t": 1, "experts": 256, "topk": 8, "hidden": 2048, "inter": 512,
         "shared": 0, "shared_gate": False, "scoring": "softmax", "renormalize": True, "bias": False, "type": "fp16"},
        # sixteen streams through the same layer with a shared expert
        {"name": "moe_16x256x2048x512_shared", "op": "moe", "t": 16, "experts": 256, "topk": 8, "hidden": 2048,
         "inter": 512, "shared": 512, "shared_gate": True, "scoring": "softmax", "renormalize": True, "bias": False,
         "type": "fp16"},
        # a few rows, sigmoid scores with a selection bias, ragged widths, fp32 out
        {"name": "moe_5x60x1440x352_sigmoid", "op": "moe", "t": 5, "experts": 60, "topk": 4, "hidden": 1440,
         "inter": 352, "shared": 736, "shared_gate": False, "scoring": "sigmoid", "renormalize": True, "bias": True,
         "type": "fp32"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quantize", "matmul", "linear", "moe"])
    type_ = rng.choice(["fp16", "fp32"])
    if op == "quantize":
        k = BLOCK * _log(rng, 1, 544)
        rows = _log(rng, 1, max(1, min(20000, 10007 * 6880 // k)))
        return {"op": op, "rows": rows, "k": k, "type": type_}
    if op == "matmul":
        m, n = _log(rng, 1, 4096), _log(rng, 1, 17408)
        most = 4096 * 5120 * 17408 // (m * n)
        return {"op": op, "m": m, "k": BLOCK * _log(rng, 1, max(1, min(544, most // BLOCK))), "n": n,
                "bias": rng.random() < 0.5, "type": type_}
    if op == "linear":
        k = BLOCK * _log(rng, 1, 544)
        return {"op": op, "m": _log(rng, 1, 64), "k": k, "n": _log(rng, 1, min(17408, 17408 * 5120 // k)),
                "bias": rng.random() < 0.5, "type": type_}
    experts = _log(rng, 4, 256)
    topk = rng.randint(1, min(8, experts))
    hidden = BLOCK * _log(rng, 4, 160)
    inter = BLOCK * _log(rng, 1, max(1, min(48, 512 * 2048 // hidden // BLOCK)))
    shared = rng.choice([0, inter, BLOCK * _log(rng, 1, max(1, inter // BLOCK))])
    scoring = rng.choice(["softmax", "sigmoid"])
    return {"op": op, "t": rng.randint(1, 16), "experts": experts, "topk": topk, "hidden": hidden, "inter": inter,
            "shared": shared, "shared_gate": shared > 0 and rng.random() < 0.5, "scoring": scoring,
            "renormalize": rng.random() < 0.7, "bias": rng.random() < 0.5, "type": type_}


def work(case):
    """Bytes: every operand once, MXFP4 at 17/32 bytes an element.  A moe pass
    reads the experts that its tokens are expected to reach under even routing."""
    q = 0.5 + 1 / BLOCK
    out = 2 if case["type"] == "fp16" else 4
    if case["op"] == "quantize":
        n = case["rows"] * case["k"]
        return {"bytes": n * (2 * out + q), "flops": 0}
    if case["op"] in ("matmul", "linear"):
        m, n, k = case["m"], case["n"], case["k"]
        x = q if case["op"] == "matmul" else 2
        return {"bytes": m * k * x + n * k * q + m * n * out + 2 * n * case["bias"], "flops": 2 * m * n * k}
    t, e, h, i = case["t"], case["experts"], case["hidden"], case["inter"]
    reached = e * (1 - (1 - case["topk"] / e) ** t)
    weights = 3 * h * (reached * i + case["shared"]) * q
    return {"bytes": e * h * 2 + weights + t * h * (2 + out) + t * case["topk"] * 8,
            "flops": 2 * t * h * (e + 3 * (case["topk"] * i + case["shared"]))}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _pack(x):
    """fp32 [..., k] -> codes uint8 [..., k/2], scales uint8 [..., k/32]."""
    v = x.unflatten(-1, (-1, BLOCK))
    amax = v.abs().amax(-1, keepdim=True)
    e = (torch.frexp(amax).exponent - 3).clamp(min=-127)  # floor(log2 amax) - 2
    e = torch.where(amax > 0, e, -127)
    v = torch.ldexp(v, -e)
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = (torch.round(a / step) * step).clamp(max=6.0)
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = (code | (torch.signbit(v).to(torch.uint8) << 3)).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), (e.squeeze(-1) + 127).to(torch.uint8)


def _mx4(g, *shape, scale=1.0):
    return _pack(torch.randn(*shape, generator=g, device="cuda") * scale)


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + 17)
    f16 = torch.float16

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * scale
    s = {"op": case["op"], "type": TYPES[case["type"]]}
    if case["op"] == "quantize":
        s["x"] = normal(case["rows"], case["k"]).to(s["type"])
    elif case["op"] == "matmul":
        s["a"] = _mx4(g, case["m"], case["k"])
        s["b"] = _mx4(g, case["n"], case["k"], scale=case["k"] ** -0.5)
        s["bias"] = normal(case["n"], scale=0.1).to(f16) if case["bias"] else None
    elif case["op"] == "linear":
        s["x"] = normal(case["m"], case["k"]).to(f16)
        s["w"] = _mx4(g, case["n"], case["k"], scale=case["k"] ** -0.5)
        s["bias"] = normal(case["n"], scale=0.1).to(f16) if case["bias"] else None
    else:
        t, e, h, i, si = case["t"], case["experts"], case["hidden"], case["inter"], case["shared"]
        s["x"] = normal(t, h).to(f16)
        s["topk"], s["scoring"], s["renormalize"] = case["topk"], case["scoring"], case["renormalize"]
        s["router"] = normal(e, h, scale=1.5 * h ** -0.5).to(f16)
        s["router_bias"] = normal(e, scale=0.1) if case["bias"] else None
        s["gate_up"] = _mx4(g, e, 2, i, h, scale=h ** -0.5)
        s["down"] = _mx4(g, e, 1, h, i, scale=i ** -0.5)
        s["shared_gate_up"] = _mx4(g, 1, 2, si, h, scale=h ** -0.5) if si else None
        s["shared_down"] = _mx4(g, 1, 1, h, si, scale=si ** -0.5) if si else None
        s["shared_gate"] = normal(h, scale=h ** -0.5).to(f16) if case["shared_gate"] else None
    return s


def _zeros(nbytes):
    return torch.zeros(nbytes, dtype=torch.uint8, device="cuda")


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:  # the weight handles, outputs and workspaces that a program keeps
        import gemm_exl3_linear_amd as X
        if s["op"] == "quantize":
            rows, k = s["x"].shape
            s["q"] = X.Exl3Mx4.empty(rows, k, device="cuda")
            s["out"] = torch.empty_like(s["x"])
        elif s["op"] == "matmul":
            s["a"], s["b"] = X.Exl3Mx4(*s["a"]), X.Exl3Mx4(*s["b"])
            s["out"] = torch.empty((case["m"], case["n"]), dtype=s["type"], device="cuda")
            s["ws"] = _zeros(X.exl3_mx4_matmul_workspace_size(s["a"], s["b"]))
        elif s["op"] == "linear":
            s["w"] = X.Exl3Mx4(*s["w"])
            s["out"] = torch.empty((case["m"], case["n"]), dtype=s["type"], device="cuda")
            s["ws"] = _zeros(X.exl3_mx4_linear_workspace_size(s["w"], case["m"]))
        else:
            shared = None
            if s["shared_gate_up"] is not None:
                shared = X.Exl3Mx4Shared(X.Exl3Mx4Arena(*s["shared_gate_up"]), X.Exl3Mx4Arena(*s["shared_down"]),
                                         gate=s["shared_gate"])
            s["layer"] = X.Exl3Mx4Moe(X.Exl3MoeRouter(s["router"], bias=s["router_bias"], scoring=s["scoring"],
                                                      renormalize=s["renormalize"]),
                                      X.Exl3Mx4Arena(*s["gate_up"]), X.Exl3Mx4Arena(*s["down"]), shared)
            s["out"] = torch.empty((case["t"], case["hidden"]), dtype=s["type"], device="cuda")
            s["ids"] = torch.empty((case["t"], case["topk"]), dtype=torch.int32, device="cuda")
            s["weights"] = torch.empty((case["t"], case["topk"]), dtype=torch.float32, device="cuda")
            s["ws"] = _zeros(X.exl3_mx4_moe_workspace_size(s["layer"], case["t"], case["topk"]))
    return s


# ---------------------------------------------------------------------------
# plain form
# ---------------------------------------------------------------------------
def _values(q):
    """fp32 values of codes [..., k/2] and scales [..., k/32]."""
    codes, scales = q
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    v = table[torch.stack((codes & 15, codes >> 4), -1).flatten(-2).int()]
    scale = (scales.int() << 23).view(torch.float32)  # 2^(s - 127)
    return (v.unflatten(-1, (-1, BLOCK)) * scale.unsqueeze(-1)).flatten(-2)


def _plain_moe(s):
    x, k = s["x"].float(), s["topk"]
    logits = x @ s["router"].float().t()
    if s["scoring"] == "softmax":
        if s["router_bias"] is not None:
            logits = logits + s["router_bias"]
        score = torch.exp(logits - logits.amax(-1, keepdim=True))
        score = score / score.sum(-1, keepdim=True)
        choice = logits
    else:
        score = 1 / (1 + torch.exp(-logits))
        choice = score if s["router_bias"] is None else score + s["router_bias"]
    ids = torch.sort(choice, dim=-1, descending=True, stable=True).indices[:, :k]
    weights = torch.gather(score, 1, ids)
    if s["renormalize"]:
        weights = weights / weights.sum(-1, keepdim=True)
    flat = ids.flatten()
    rows = x.repeat_interleave(k, 0).unsqueeze(-1)  # [P, hidden, 1]
    gu = _values((s["gate_up"][0][flat], s["gate_up"][1][flat]))  # [P, 2, inter, hidden]
    g, u = (gu @ rows.unsqueeze(1)).squeeze(-1).unbind(1)
    act = g / (1 + torch.exp(-g)) * u
    dn = _values((s["down"][0][flat, 0], s["down"][1][flat, 0]))  # [P, hidden, inter]
    d = (dn @ act.unsqueeze(-1)).squeeze(-1).view(x.shape[0], k, -1)
    y = (d * weights.unsqueeze(-1)).sum(1)
    if s["shared_gate_up"] is not None:
        g, u = (x @ _values(s["shared_gate_up"])[0].transpose(1, 2)).unbind(0)
        d = (g / (1 + torch.exp(-g)) * u) @ _values(s["shared_down"])[0, 0].t()
        if s["shared_gate"] is not None:
            d = d / (1 + torch.exp(-(x @ s["shared_gate"].float()))).unsqueeze(-1)
        y = y + d
    return y.to(s["type"]), ids.int(), weights


def run(s):
    if own:
        import gemm_exl3_linear_amd as X
        if s["op"] == "quantize":
            X.exl3_mx4_quantize(s["x"], out=s["q"])
            return X.exl3_mx4_reconstruct(s["q"], out=s["out"])
        if s["op"] == "matmul":
            return X.exl3_mx4_matmul(s["a"], s["b"], bias=s["bias"], out=s["out"], workspace=s["ws"])
        if s["op"] == "linear":
            return X.exl3_mx4_linear(s["x"], s["w"], bias=s["bias"], out=s["out"], workspace=s["ws"])
        X.exl3_mx4_moe(s["x"], s["layer"], s["topk"], out=s["out"], topk_ids=s["ids"], topk_weights=s["weights"],
                       workspace=s["ws"])
        return s["out"], s["ids"], s["weights"]
    if s["op"] == "quantize":
        return _values(_pack(s["x"].float())).to(s["type"])
    if s["op"] == "moe":
        return _plain_moe(s)
    x = s["x"].float() if s["op"] == "linear" else _values(s["a"])
    y = x @ _values(s["w"] if s["op"] == "linear" else s["b"]).t()
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(s["type"])


# ---------------------------------------------------------------------------
# from the definition, in 64 bits
# ---------------------------------------------------------------------------
def _decode64(q):
    codes, scales = (t.long() for t in q)
    magnitude = torch.tensor(E2M1, dtype=torch.float64, device=codes.device)
    power = torch.tensor([2.0 ** (i - 127) for i in range(255)] + [math.nan], dtype=torch.float64,
                         device=codes.device)
    out = torch.empty(*codes.shape[:-1], codes.shape[-1] * 2, dtype=torch.float64, device=codes.device)
    for half in range(2):
        nibble = (codes >> (4 * half)) % 16
        out[..., half::2] = magnitude[nibble % 8] * (1 - 2 * (nibble // 8))
    return out * power[scales].repeat_interleave(BLOCK, -1)


def _exact_quantize(x):
    x = x.double()
    blocks = x.reshape(x.shape[0], -1, BLOCK)
    top = blocks.abs().max(-1, keepdim=True).values
    unit = torch.exp2(torch.clamp(torch.floor(torch.log2(top)) - 2, min=-127))
    low, high = 2.0 ** -127, torch.finfo(torch.float64).max
    unit = torch.where((unit * 4 > top) & (top > 0), unit / 2, unit).clamp(low, high)
    v = blocks / unit
    best = torch.zeros_like(v)  # nearest value of the table, an even code where two are as near
    gap = v.abs()
    for code in range(1, 8):
        d = (v.abs() - E2M1[code]).abs()
        nearer = (d < gap) | ((d == gap) & (code % 2 == 0))
        best = torch.where(nearer, torch.full_like(v, E2M1[code]), best)
        gap = torch.minimum(gap, d)
    return (torch.copysign(best, v) * unit).reshape(x.shape)


def _exact_moe(s):
    x = s["x"].double()
    logits = x @ s["router"].double().T
    bias = 0.0 if s["router_bias"] is None else s["router_bias"].double()
    y = torch.zeros_like(x)
    all_ids, all_weights = [], []
    for t in range(x.shape[0]):
        if s["scoring"] == "softmax":
            choice = logits[t] + bias
            score = torch.exp(choice - choice.max())
            score = score / score.sum()
        else:
            score = torch.sigmoid(logits[t])
            choice = score + bias
        order = sorted(range(len(choice)), key=lambda e, c=choice.tolist(): (-c[e], e))[:s["topk"]]
        w = score[order]
        if s["renormalize"]:
            w = w / w.sum()
        for slot, e in enumerate(order):
            gate_up = _decode64((s["gate_up"][0][e], s["gate_up"][1][e]))
            g, u = gate_up[0] @ x[t], gate_up[1] @ x[t]
            y[t] += w[slot] * (_decode64((s["down"][0][e, 0], s["down"][1][e, 0])) @ (g * torch.sigmoid(g) * u))
        all_ids.append(order)
        all_weights.append(w)
    if s["shared_gate_up"] is not None:
        gate, up = _decode64(s["shared_gate_up"])[0]
        g, u = x @ gate.T, x @ up.T
        d = (g * torch.sigmoid(g) * u) @ _decode64(s["shared_down"])[0, 0].T
        if s["shared_gate"] is not None:
            d = d * torch.sigmoid(x @ s["shared_gate"].double())[:, None]
        y += d
    return y, torch.tensor(all_ids, device=x.device).int(), torch.stack(all_weights)


def exact(case, seed):
    s = _inputs(case, seed)
    if s["op"] == "quantize":
        return _exact_quantize(s["x"])
    if s["op"] == "moe":
        return _exact_moe(s)
    x = s["x"].double() if s["op"] == "linear" else _decode64(s["a"])
    y = x @ _decode64(s["w"] if s["op"] == "linear" else s["b"]).T
    return y if s["bias"] is None else y + s["bias"].double()
