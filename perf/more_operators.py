"""Routing to experts and low-rank adapters on cases of real use, and what they
compute in plain torch.

  logits  a router's logits of many tokens: l = x W^T (+ c), fp16 in, fp32 out
          (exl3_router_linear)
  route   logits to choices and weights: scores s = softmax(l) or sigmoid(l);
          choice values s + b where there is a balance b (else in l's order);
          the best groups of experts by their best choice value or by the sum
          of their two best; the top-k of those groups, best first, equal values
          to the lower expert; weights s, divided by their sum, times a factor
          (exl3_route_topk)
  router  both in one call, for few tokens (exl3_router)
  lora    y_i = base_i + scale_a B_a (A_a x_i) with a row's own adapter a, or
          base_i where it has none (exl3_lora)
"""
import math

import torch

own = False

TYPES = {"fp16": torch.float16, "fp32": torch.float32}
MAX_EXPERTS, MAX_TOPK = 1024, 16


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # a ragged chunk of a prompt through a small router whose linear has a bias
        {"name": "logits_333x1440x60_bias", "op": "logits", "t": 333, "hidden": 1440, "experts": 60, "bias": True},
        # a 4096-token prefill in front of 256 experts
        {"name": "logits_4096x5120x256", "op": "logits", "t": 4096, "hidden": 5120, "experts": 256, "bias": False},
        # the smallest call: one token's logits, eight of 256 experts
        {"name": "route_1x256_softmax", "op": "route", "t": 1, "experts": 256, "topk": 8, "scoring": "softmax",
         "groups": 1, "topk_groups": 1, "group_score": "max", "balance": False, "renormalize": True, "type": "fp32"},
        # a ragged chunk, logits held in fp16 (equal ones are common), an odd count of experts
        {"name": "route_777x60_fp16", "op": "route", "t": 777, "experts": 60, "topk": 4, "scoring": "sigmoid",
         "groups": 1, "topk_groups": 1, "group_score": "max", "balance": False, "renormalize": False,
         "type": "fp16"},
        # a 4096-token prefill
        {"name": "route_4096x256_softmax", "op": "route", "t": 4096, "experts": 256, "topk": 8, "scoring": "softmax",
         "groups": 1, "topk_groups": 1, "group_score": "max", "balance": False, "renormalize": True, "type": "fp32"},
        # several prompts at once, balanced sigmoid scores, four of eight groups
        {"name": "route_16384x256_grouped", "op": "route", "t": 16384, "experts": 256, "topk": 8,
         "scoring": "sigmoid", "groups": 8, "topk_groups": 4, "group_score": "top2", "balance": True,
         "renormalize": True, "type": "fp32"},
        # one token of a decode step, from its hidden row to its experts
        {"name": "router_1x2048x256", "op": "router", "t": 1, "hidden": 2048, "experts": 256, "topk": 8,
         "scoring": "softmax", "groups": 1, "topk_groups": 1, "group_score": "max", "balance": False,
         "renormalize": True, "bias": False},
        # sixteen streams, balanced sigmoid scores, four of eight groups
        {"name": "router_16x5120x256_grouped", "op": "router", "t": 16, "hidden": 5120, "experts": 256, "topk": 8,
         "scoring": "sigmoid", "groups": 8, "topk_groups": 4, "group_score": "top2", "balance": True,
         "renormalize": True, "bias": False},
        # one token of one request beside an up projection
        {"name": "lora_1x5120x17408_r16", "op": "lora", "m": 1, "k": 5120, "n": 17408, "rank": 16, "adapters": 8,
         "ranks": "full", "rows": "mixed", "none": 0.0, "type": "fp16"},
        # a decode batch of 64 requests, most with adapters of their own
        {"name": "lora_64x5120x17408_r16", "op": "lora", "m": 64, "k": 5120, "n": 17408, "rank": 16, "adapters": 64,
         "ranks": "full", "rows": "mixed", "none": 0.1, "type": "fp16"},
        # a ragged verify batch, ranks from 1 to 40, odd widths, fp32 sums kept
        {"name": "lora_333x2056x1111_r40", "op": "lora", "m": 333, "k": 2056, "n": 1111, "rank": 40, "adapters": 7,
         "ranks": "mixed", "rows": "mixed", "none": 0.2, "type": "fp32"},
        # a prefill of four requests' prompts, one behind the other
        {"name": "lora_4096x5120x17408_r64", "op": "lora", "m": 4096, "k": 5120, "n": 17408, "rank": 64,
         "adapters": 4, "ranks": "full", "rows": "runs", "none": 0.0, "type": "fp16"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _rule(rng, experts):
    """A rule of routing that `experts` experts allow."""
    groups = rng.choice([g for g in (1, 1, 2, 4, 8, 16) if experts % g == 0 and experts // g >= 2])
    topk_groups = rng.randint(1, groups)
    topk = rng.randint(1, min(MAX_TOPK, topk_groups * (experts // groups)))
    return {"topk": topk, "scoring": rng.choice(["softmax", "sigmoid"]), "groups": groups,
            "topk_groups": topk_groups, "group_score": rng.choice(["max", "top2"]),
            "balance": rng.random() < 0.5, "renormalize": rng.random() < 0.7}


def draw(rng):
    op = rng.choice(["logits", "route", "router", "lora"])
    if op == "lora":
        k, n = 8 * _log(rng, 8, 2176), _log(rng, 1, 17408)
        m = _log(rng, 1, max(1, min(4096, 4096 * 22528 // (k + n))))
        rank = 8 * rng.choice([1, 1, 2, 2, 3, 4, 5, 8, 16])
        most = max(1, 4096 * 4 * 64 * 22528 // (m * rank * (k + n)))
        return {"op": op, "m": m, "k": k, "n": n, "rank": rank, "adapters": _log(rng, 1, min(64, most)),
                "ranks": rng.choice(["full", "mixed"]), "rows": rng.choice(["mixed", "runs"]),
                "none": rng.choice([0.0, 0.2]), "type": rng.choice(["fp16", "fp32"])}
    experts = rng.choice([_log(rng, 4, MAX_EXPERTS), 8 * _log(rng, 1, MAX_EXPERTS // 8)])
    if op == "route":
        t = _log(rng, 1, min(16384, 16384 * 256 // experts))
        return {"op": op, "t": t, "experts": experts, **_rule(rng, experts), "type": rng.choice(["fp16", "fp32"])}
    hidden = 8 * _log(rng, 8, 1024)
    if op == "logits":
        t = _log(rng, 1, max(1, min(8192, 4096 * 5120 * 256 // (hidden * experts))))
        return {"op": op, "t": t, "hidden": hidden, "experts": experts, "bias": rng.random() < 0.5}
    return {"op": op, "t": _log(rng, 1, 64), "hidden": hidden, "experts": experts, **_rule(rng, experts),
            "bias": rng.random() < 0.5}


def work(case):
    """Bytes: every operand once.  A lora pass reads the adapters that its rows
    are expected to reach; ranks count in full."""
    if case["op"] == "lora":
        m, k, n, r = case["m"], case["k"], case["n"], case["rank"]
        out = 2 if case["type"] == "fp16" else 4
        with_one = m * (1 - case["none"])
        reached = case["adapters"] * (1 - (1 - 1 / case["adapters"]) ** with_one)
        if case["rows"] == "runs":
            reached = min(case["adapters"], with_one)
        if case["ranks"] == "mixed":
            r = (r + 1) / 2
        return {"bytes": with_one * k * 2 + 2 * m * n * out + reached * r * (k + n) * 2 + 4 * m,
                "flops": 2 * with_one * r * (k + n)}
    t, e = case["t"], case["experts"]
    nbytes, flops = 0, 0
    if case["op"] != "route":
        nbytes += (t + e) * case["hidden"] * 2 + t * e * 4 + 4 * e * case["bias"]
        flops += 2 * t * e * case["hidden"]
    else:
        nbytes += t * e * (2 if case["type"] == "fp16" else 4)
    if case["op"] != "logits":
        nbytes += t * case["topk"] * 8 + 4 * e * case["balance"]
        flops += 4 * t * e  # scores; a comparison is no operation here
    return {"bytes": nbytes, "flops": flops}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _adapters_of_rows(case, g):
    """int32 [m]: a row's adapter, -1 for none."""
    m, count = case["m"], case["adapters"]
    if case["rows"] == "runs":  # requests one behind the other, about as long as each other
        ids = torch.arange(m, device="cuda") * count // m
        drop = torch.rand(count, generator=g, device="cuda")[ids] < case["none"]
    else:
        ids = torch.randint(count, (m,), generator=g, device="cuda")
        drop = torch.rand(m, generator=g, device="cuda") < case["none"]
    return torch.where(drop, -1, ids).int()


def _inputs(case, seed):
    g = torch.Generator(device="cuda").manual_seed(int(seed) * 1000003 + 29)
    f16 = torch.float16

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device="cuda") * scale
    s = {"op": case["op"], "case": case}
    if case["op"] == "lora":
        count, r, k, n = case["adapters"], case["rank"], case["k"], case["n"]
        s["type"] = TYPES[case["type"]]
        s["x"] = normal(case["m"], k).to(f16)
        s["base"] = normal(case["m"], n).to(s["type"])
        s["a"] = normal(count, r, k, scale=k ** -0.5).to(f16)
        s["b"] = normal(count, n, r, scale=0.5 * r ** -0.5).to(f16)
        s["scales"] = 0.5 + 1.5 * torch.rand(count, generator=g, device="cuda")
        s["ranks"] = None
        if case["ranks"] == "mixed":
            s["ranks"] = torch.randint(1, r + 1, (count,), generator=g, device="cuda").int()
        s["rows"] = _adapters_of_rows(case, g)
        return s
    e = case["experts"]
    if case["op"] == "route":
        s["logits"] = normal(case["t"], e, scale=1.5).to(TYPES[case["type"]])
    else:
        h = case["hidden"]
        s["x"] = normal(case["t"], h).to(f16)
        s["weight"] = normal(e, h, scale=1.5 * h ** -0.5).to(f16)
        s["bias"] = normal(e, scale=0.1) if case["bias"] else None
    if case["op"] != "logits":
        scale = 0.1 if case["scoring"] == "sigmoid" else 0.5 / e  # beside scores of that size
        s["balance"] = normal(e, scale=scale) if case["balance"] else None
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:  # the handles, outputs and workspaces that a program keeps
        import gemm_exl3_linear_amd as X

        def new(*shape, dtype=torch.float32):
            return torch.empty(shape, dtype=dtype, device="cuda")
        if s["op"] == "lora":
            s["lora"] = X.Exl3Lora(s["a"], s["b"], scales=s["scales"], ranks=s["ranks"])
            s["out"] = torch.empty_like(s["base"])
            s["ws"] = torch.zeros(X.exl3_lora_workspace_size(s["lora"], case["m"]), dtype=torch.uint8, device="cuda")
            return s
        if s["op"] != "route":
            s["router"] = X.Exl3Router(s["weight"], bias=s["bias"])
            s["logits"] = new(case["t"], case["experts"])
            size = X.exl3_router_linear_workspace_size if s["op"] == "logits" else X.exl3_router_workspace_size
            s["ws"] = torch.zeros(size(s["router"], case["t"]), dtype=torch.uint8, device="cuda")
        if s["op"] != "logits":
            s["rule"] = X.Exl3RouteRule(case["experts"], case["topk"], scoring=case["scoring"], balance=s["balance"],
                                        groups=case["groups"], topk_groups=case["topk_groups"],
                                        group_score=case["group_score"], renormalize=case["renormalize"], scale=2.5)
            s["ids"] = new(case["t"], case["topk"], dtype=torch.int32)
            s["weights"] = new(case["t"], case["topk"])
    return s


# ---------------------------------------------------------------------------
# plain form
# ---------------------------------------------------------------------------
def _plain_route(logits, balance, case):
    """Choices in 64 bits, where values lie next to each other; weights in 32."""
    t, e = logits.shape

    def score(l):
        if case["scoring"] == "sigmoid":
            return 1 / (1 + torch.exp(-l))
        p = torch.exp(l - l.amax(-1, keepdim=True))
        return p / p.sum(-1, keepdim=True)
    value = logits.double()
    if balance is not None:
        value = score(value) + balance.double()
    if case["groups"] > 1:
        of_group = value if case["group_score"] == "max" or balance is not None else score(value)
        of_group = of_group.view(t, case["groups"], -1)
        if case["group_score"] == "max":
            best = of_group.amax(-1)
        else:
            best = torch.sort(of_group, dim=-1, descending=True).values[..., :2].sum(-1)
        kept = torch.sort(best, dim=-1, descending=True, stable=True).indices[:, :case["topk_groups"]]
        keep = torch.zeros(t, case["groups"], dtype=torch.bool, device=value.device).scatter_(1, kept, True)
        value = torch.where(keep.repeat_interleave(e // case["groups"], 1), value, -math.inf)
    ids = torch.sort(value, dim=-1, descending=True, stable=True).indices[:, :case["topk"]]
    weights = torch.gather(score(logits.float()), 1, ids)
    if case["renormalize"]:
        weights = weights / weights.sum(-1, keepdim=True)
    return ids.int(), weights * 2.5


def _plain_lora(s):
    """Every row against every adapter's A; its own adapter's part of that, in its
    place among zeros, against the B of all."""
    m, (count, r, k) = s["x"].shape[0], s["a"].shape
    h = (s["x"].float() @ s["a"].view(count * r, k).float().t()).view(m, count, r)
    mine = s["rows"].unsqueeze(1) == torch.arange(count, device=h.device)
    factor = mine.float() * s["scales"]
    h = h * factor.unsqueeze(-1)
    if s["ranks"] is not None:
        h = h * (torch.arange(r, device=h.device) < s["ranks"].unsqueeze(1))
    delta = h.view(m, count * r) @ s["b"].transpose(1, 2).reshape(count * r, -1).float()
    return (s["base"].float() + delta).to(s["type"])


def run(s):
    case = s["case"]
    if own:
        import gemm_exl3_linear_amd as X
        if s["op"] == "lora":
            return X.exl3_lora(s["x"], s["lora"], s["rows"], s["base"], out=s["out"], workspace=s["ws"])
        if s["op"] == "logits":
            return X.exl3_router_linear(s["x"], s["router"], out=s["logits"], workspace=s["ws"])
        if s["op"] == "route":
            X.exl3_route_topk(s["logits"], s["rule"], topk_ids=s["ids"], topk_weights=s["weights"])
            return s["ids"], s["weights"]
        X.exl3_router(s["x"], s["router"], s["rule"], logits=s["logits"], topk_ids=s["ids"],
                      topk_weights=s["weights"], workspace=s["ws"])
        return s["logits"], s["ids"], s["weights"]
    if s["op"] == "lora":
        return _plain_lora(s)
    if s["op"] == "route":
        return _plain_route(s["logits"], s["balance"], case)
    if s["op"] == "logits":
        logits = s["x"].float() @ s["weight"].float().t()
        return logits if s["bias"] is None else logits + s["bias"]
    logits = s["x"].double() @ s["weight"].double().t()  # in 64 bits: choices next to each other
    if s["bias"] is not None:
        logits = logits + s["bias"].double()
    return logits.float(), *_plain_route(logits, s["balance"], case)


# ---------------------------------------------------------------------------
# from the definition, in 64 bits
# ---------------------------------------------------------------------------
def _exact_route(logits, balance, case):
    e, size = case["experts"], case["experts"] // case["groups"]
    scores = torch.sigmoid(logits) if case["scoring"] == "sigmoid" else torch.softmax(logits, -1)
    value = logits if balance is None else scores + balance.double()
    allowed = torch.ones_like(logits, dtype=torch.bool)
    if case["groups"] > 1:
        top2 = case["group_score"] == "top2"
        graded = scores if top2 and balance is None else value
        grade = torch.stack([graded[:, i:i + size].topk(2 if top2 else 1, -1).values.sum(-1)
                             for i in range(0, e, size)], 1)
        for g in range(case["groups"]):  # groups ahead of g: better ones, and as good ones before it
            mine = grade[:, g:g + 1]
            ahead = (grade > mine).sum(1) + (grade[:, :g] == mine).sum(1)
            allowed[:, g * size:(g + 1) * size] = (ahead < case["topk_groups"]).unsqueeze(1)
    left = torch.where(allowed, value, -math.inf)
    index = torch.arange(e, device=logits.device)
    ids = []
    for _ in range(case["topk"]):
        best = left.max(-1, keepdim=True).values
        first = torch.where(left == best, index, e).min(-1, keepdim=True).values
        ids.append(first)
        left = left.scatter(1, first, -math.inf)
    ids = torch.cat(ids, 1)
    weights = scores.gather(1, ids)
    if case["renormalize"]:
        weights = weights / weights.sum(1, keepdim=True)
    return ids.int(), 2.5 * weights


def _exact_lora(s):
    y = s["base"].double()
    for adapter in range(s["a"].shape[0]):
        rows = (s["rows"] == adapter).nonzero().flatten()
        r = s["a"].shape[1] if s["ranks"] is None else int(s["ranks"][adapter])
        if len(rows):
            inner = s["x"][rows].double() @ s["a"][adapter, :r].double().T
            y[rows] += float(s["scales"][adapter]) * (inner @ s["b"][adapter, :, :r].double().T)
    return y


def exact(case, seed):
    s = _inputs(case, seed)
    if s["op"] == "lora":
        return _exact_lora(s)
    if s["op"] == "route":
        return _exact_route(s["logits"].double(), s["balance"], case)
    logits = s["x"].double() @ s["weight"].double().T
    if s["bias"] is not None:
        logits = logits + s["bias"].double()
    return logits if s["op"] == "logits" else (logits, *_exact_route(logits, s["balance"], case))
