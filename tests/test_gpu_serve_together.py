"""Routing and adapters as a served layer uses them: projections with the adapters of
their requests, a router in front of the experts, graphs, streams and workspaces."""
import numpy as np
import pytest

import synth
from oracle import exl3_oracle as O
from oracle import serve_oracle as S
from tests import _gpu as G
from tests import test_gpu_lora as L
from tests import test_gpu_route as R

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", [1, 3, 16, 40])
def test_a_layer_of_projection_adapters_router_and_experts(t):
    """x -> exl3_linear -> exl3_lora in place -> exl3_router -> exl3_grouped_experts, every
    step against its oracle on what the step before gave."""
    import torch
    import gemm_exl3_linear_amd as X
    hidden, inter, experts, topk, rank = 256, 128, 16, 4, 16
    d = synth.linear_inputs(77, t, hidden, hidden, 4)
    w = G.weight(d)
    x = G.to_dev(d["x"])
    h = X.exl3_linear(x, w)
    base = h.cpu().numpy()
    G.assert_parity(base, G.linear_ref(d))
    ad = L.case(t, hidden, hidden, rank, 5)
    ad["x"], ad["base"] = d["x"], base
    X.exl3_lora(x, L.handle(ad), G.to_dev(ad["rows"]), h, out=h)
    L.check(h, ad, False)
    # the norm between: without it the experts' fp16 activations are past 65504
    h = (h.float() / h.float().square().mean(-1, keepdim=True).sqrt()).half()
    _, weight, _ = R.router_case(t, hidden, experts, False)
    rng = np.random.default_rng(t)
    rule = R.rule_of(experts, topk, rng.standard_normal(experts) * 0.1, scoring="sigmoid", groups=4, topk_groups=2,
                     group_score="top2", scale=2.5)
    logits = torch.empty((t, experts), device=G.dev())
    ids, wt = X.exl3_router(h, R.handle(weight, None), rule, logits=logits)
    R.check(ids, wt, logits.cpu().numpy().astype(np.float64), rule)
    m = synth.moe_inputs(78, t, experts=experts, topk=topk, hidden=hidden, inter=inter, bits=3)
    gu, dn = X.Exl3Arena.from_numpy(m["gate_up"], G.dev()), X.Exl3Arena.from_numpy(m["down"], G.dev())
    y = X.exl3_grouped_experts(h, ids, wt, gu, dn)
    ref = O.grouped_experts(h.cpu().numpy(), ids.cpu().numpy(), wt.cpu().numpy(), m["gate_up"], m["down"])
    G.assert_parity(y.cpu().numpy(), ref)


def test_adapters_beside_an_mxfp4_projection():
    import torch
    import gemm_exl3_linear_amd as X
    t, k, n = 24, 512, 320
    d = L.case(t, k, n, 24, 6, f32=True)
    xd = G.to_dev(d["x"])
    w = X.exl3_mx4_quantize(torch.randn(n, k, device=G.dev()))
    base = X.exl3_mx4_linear(xd, w, out_dtype=torch.float32)
    d["base"] = base.cpu().numpy()
    L.check(X.exl3_lora(xd, L.handle(d), G.to_dev(d["rows"]), base), d, True)


def _calls(t, ws_of):
    """One call of each entry point on tensors of their own: (run, outputs, inputs)."""
    import torch
    import gemm_exl3_linear_amd as X
    dev = G.dev()
    x, w, c = R.router_case(t, 1448, 96, True)
    xd, r = G.to_dev(x), R.handle(w, c)
    rng = np.random.default_rng(t)
    rule = R.rule_of(96, 6, rng.standard_normal(96) * 0.1, scoring="sigmoid", groups=8, topk_groups=3,
                     group_score="top2")
    ad = L.case(t, 1448, 200, 24, 9, f32=True)
    lora, rows, base = L.handle(ad), G.to_dev(ad["rows"]), G.to_dev(ad["base"])
    out = dict(logits=torch.empty((t, 96), device=dev), l2=torch.empty((t, 96), device=dev),
               ids=torch.empty((t, 6), dtype=torch.int32, device=dev), w=torch.empty((t, 6), device=dev),
               ids2=torch.empty((t, 6), dtype=torch.int32, device=dev), w2=torch.empty((t, 6), device=dev),
               y=torch.empty((t, 200), device=dev))
    wr = ws_of("router", max(X.exl3_router_workspace_size(r, t), X.exl3_router_linear_workspace_size(r, t)))
    wl = ws_of("lora", X.exl3_lora_workspace_size(lora, t))

    def run(stream=None):
        X.exl3_router_linear(xd, r, out=out["l2"], workspace=wr, stream=stream)
        X.exl3_router(xd, r, rule, logits=out["logits"], topk_ids=out["ids"], topk_weights=out["w"], workspace=wr,
                      stream=stream)
        X.exl3_route_topk(out["l2"], rule, topk_ids=out["ids2"], topk_weights=out["w2"], stream=stream)
        X.exl3_lora(xd, lora, rows, base, out=out["y"], workspace=wl, stream=stream)
    return run, out, (xd, rows)


def _own(name, n):
    import torch
    return torch.zeros(n, dtype=torch.uint8, device=G.dev())


def _wipe(out):
    for v in out.values():
        v.fill_(-3)


@pytest.mark.parametrize("t", [1, 3, 16, 50, 300])
def test_graphs_replayed_with_new_inputs(t):
    """Every replay gives the bits of the eager call on the same inputs."""
    import torch
    run, out, (xd, rows) = _calls(t, _own)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for i in range(4):
        xd.copy_(torch.randn(xd.shape, device=G.dev()))
        rows.copy_(torch.randint(-1, 10, rows.shape, device=G.dev()))
        _wipe(out)
        graph.replay()
        torch.cuda.synchronize()
        got = {k: v.clone() for k, v in out.items()}
        _wipe(out)
        run()
        torch.cuda.synchronize()
        for k in out:
            assert torch.equal(got[k], out[k]), (i, k)


def test_graphs_that_share_workspaces():
    import torch
    shared = {}

    def ws_of(name, n):
        if name not in shared:
            shared[name] = torch.zeros(64 << 20, dtype=torch.uint8, device=G.dev())
        assert n <= shared[name].numel()
        return shared[name]
    made = [_calls(t, ws_of) for t in (1, 16, 2, 60, 300)]
    graphs = []
    for run, _, _ in made:
        run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        graphs.append(g)
    want = []
    for run, out, _ in made:
        run()
        torch.cuda.synchronize()
        want.append({k: v.clone() for k, v in out.items()})
    for order in ((0, 1, 2, 3, 4), (4, 3, 2, 1, 0), (3, 1, 4, 0, 2)):
        for i in order:
            _wipe(made[i][1])
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in order:
            for k, v in made[i][1].items():
                assert torch.equal(v, want[i][k]), (order, i, k)


def test_captured_calls_that_make_their_own_memory():
    import torch
    import gemm_exl3_linear_amd as X
    for t in (1, 16, 40):
        x, w, _ = R.router_case(t, 520, 64, False)
        xd, r, rule = G.to_dev(x), R.handle(w, None), R.rule_of(64, 4)
        ad = L.case(t, 520, 72, 16, 3, f32=True)
        lora, rows, base = L.handle(ad), G.to_dev(ad["rows"]), G.to_dev(ad["base"])

        def run():
            ids, wt = X.exl3_router(xd, r, rule)
            l = X.exl3_router_linear(xd, r)
            return ids, wt, l, *X.exl3_route_topk(l, rule), X.exl3_lora(xd, lora, rows, base)
        run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = run()
        for _ in range(3):
            xd.copy_(torch.randn(xd.shape, device=G.dev()))
            g.replay()
            torch.cuda.synchronize()
            for a, b in zip(got, run()):
                assert torch.equal(a, b)


def test_two_streams_with_their_own_workspaces():
    import torch
    made = [_calls(t, _own) for t in (16, 5, 300, 1)]
    want = []
    for run, out, _ in made:
        run()
        torch.cuda.synchronize()
        want.append({k: v.clone() for k, v in out.items()})
        _wipe(out)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in made]
    for _ in range(10):
        for (run, _, _), s in zip(made, streams):
            run(s)
    torch.cuda.synchronize()
    for (_, out, _), ref in zip(made, want):
        for k in out:
            assert torch.equal(out[k], ref[k]), k


def test_calls_on_another_stream_take_their_memory_there():
    """Outputs and workspaces that a call makes are of the stream it runs on."""
    import torch
    import gemm_exl3_linear_amd as X
    x, w, _ = R.router_case(8, 520, 64, False)
    xd, r, rule = G.to_dev(x), R.handle(w, None), R.rule_of(64, 4)
    ad = L.case(8, 520, 72, 16, 3, f32=True)
    lora, rows, base = L.handle(ad), G.to_dev(ad["rows"]), G.to_dev(ad["base"])
    want = (*X.exl3_router(xd, r, rule), X.exl3_lora(xd, lora, rows, base), X.exl3_router_linear(xd, r))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for _ in range(5):
        junk = torch.full((1 << 20,), float("nan"), device=G.dev())  # the default stream's memory, soon free
        del junk
        got = (*X.exl3_router(xd, r, rule, stream=s), X.exl3_lora(xd, lora, rows, base, stream=s),
               X.exl3_router_linear(xd, r, stream=s))
        torch.full((1 << 20,), float("nan"), device=G.dev())
        s.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    with pytest.raises(ValueError):
        X.exl3_lora(xd, lora, rows.cpu(), base)


def test_the_same_bits_on_every_run():
    import torch
    for t in (1, 16, 64, 500):
        run, out, _ = _calls(t, _own)
        run()
        torch.cuda.synchronize()
        first = {k: v.clone() for k, v in out.items()}
        for _ in range(20):
            _wipe(out)
            run()
            torch.cuda.synchronize()
            for k in out:
                assert torch.equal(out[k], first[k]), (t, k)
