"""moe_layer_forward_lora and moe_grouped_ffn_lora: the layer with low-rank
adapters of many requests beside its expert projections, against the float64
layer, from one token to batches of several tiles per expert."""
import dataclasses

import numpy as np
import pytest
import torch

from mixture_experts_layer_bias_b200 import ops
from mixture_experts_layer_bias_b200 import synthetic as syn
from mixture_experts_layer_bias_b200.layer import MoELayer

from adapters import make_adapters, make_ids, reference_layer, rows_rel, tol
from parity import MARGIN, np64, oracle_routing as reference_layer_routing, rel_l2, run_layer

pytestmark = pytest.mark.gpu

BASE = syn.LayerConfig("adapters", S=1, d=512, E=8, K=2, h=512, router_offset_var=0.5)
E4 = dataclasses.replace(BASE, weight_dtype=syn.E4M3)
GELU = dataclasses.replace(BASE, activation=syn.GELU)


def _c(base, **kw):
    return dataclasses.replace(base, **kw)


def runs(S, n, seed=0):
    """Runs of tokens of one request each, as prompts one after another."""
    g = torch.Generator().manual_seed(seed)
    at = torch.sort(torch.randint(0, 3 * n, (S,), generator=g)).values
    return torch.randint(-1, n, (3 * n,), generator=g, dtype=torch.int32)[at].cuda().contiguous()


# (layer, adapters, rank, ids: "mixed" per token or "runs")
CASES = [
    (_c(BASE, S=1), 1, 8, "mixed"), (_c(BASE, S=3), 2, 16, "mixed"), (_c(BASE, S=65, d=264, h=200), 5, 16, "mixed"),
    (_c(BASE, S=333), 16, 8, "mixed"), (_c(BASE, S=333), 4, 40, "runs"), (_c(BASE, S=700, num_shared=1), 6, 64, "runs"),
    (_c(BASE, S=515, E=64, K=8, d=256, h=264), 12, 32, "runs"), (_c(BASE, S=257, d=1032, h=136), 3, 128, "runs"),
    (_c(BASE, S=2500, d=256, h=256), 5, 16, "runs"),  # above the rows that split the products' length
    (_c(BASE, S=200, capacity=20), 4, 16, "runs"),
    (_c(GELU, S=333, d=1000, h=1352), 16, 8, "mixed"), (_c(GELU, S=70, num_shared=1), 3, 24, "runs"),
    (_c(E4, S=5), 2, 16, "mixed"), (_c(E4, S=400, num_shared=1), 6, 32, "runs"),
    (_c(E4, S=600, E=16, K=4, capacity=100), 6, 8, "mixed"), (_c(E4, S=130, d=264, h=520), 3, 16, "runs"),
]


def _id(c):
    cfg, n, r, kind = c
    return f"{'gelu' if cfg.activation == syn.GELU else 'swiglu'}-{('f32', 'bf16', 'e4m3')[cfg.weight_dtype]}" \
           f"-S{cfg.S}-d{cfg.d}-h{cfg.h}-E{cfg.E}-n{n}-r{r}-{kind}" + (f"-cap{cfg.capacity}" if cfg.capacity else "")


def _ids(cfg, n, kind):
    ids = runs(cfg.S, n) if kind == "runs" else make_ids(cfg.S, n)
    if cfg.S == 1:
        ids.zero_()
    return ids


@pytest.mark.parametrize("case", CASES, ids=_id)
def test_layer_matches_float64(case):
    cfg, n, rank, kind = case
    inp = syn.make_inputs(cfg, "cuda", seed=21)
    ad = make_adapters(cfg, n, rank, seed=3)
    ids = _ids(cfg, n, kind)
    layer = MoELayer(cfg, inp, adapters=ad)
    y = layer.forward(inp["x"], adapter_ids=ids)
    torch.cuda.synchronize()
    assert layer.status()[1] == 0
    ref, idx, _, margin = reference_layer(inp, cfg, ad, ids)
    keep = margin >= MARGIN
    assert (layer.topk_idx.cpu().numpy()[keep] == idx[keep]).all()
    # roundings to bf16: the adapters' inner products and their share (up and down, each smaller than the sums they
    # are added to: counted as one), the hidden rows, the experts' outputs, y; with E4M3 weights the two row codes
    k = 6 if cfg.weight_dtype == syn.E4M3 else 4
    assert rel_l2(np64(y)[keep], ref[keep]) <= tol(k)
    assert rows_rel(np64(y)[keep], ref[keep]) <= 1.5 * tol(k)


@pytest.mark.parametrize("pairs", [("gate",), ("up",), ("down",), ("gate", "down")])
def test_some_projections_without_adapters(pairs):
    cfg = _c(BASE, S=150)
    inp = syn.make_inputs(cfg, "cuda", seed=22)
    ad = make_adapters(cfg, 3, 16, pairs=pairs)
    ids = runs(150, 3)
    layer = MoELayer(cfg, inp, adapters=ad)
    y = layer.forward(inp["x"], adapter_ids=ids)
    ref, *_ , margin = reference_layer(inp, cfg, ad, ids)
    keep = margin >= MARGIN
    assert rel_l2(np64(y)[keep], ref[keep]) <= tol(4)


def test_without_adapters_equals_the_layer():
    for base in (BASE, E4, GELU):
        cfg = _c(base, S=130)
        inp = syn.make_inputs(cfg, "cuda", seed=23)
        want = run_layer(inp, cfg)["y"]
        layer = MoELayer(cfg, inp, adapters=make_adapters(cfg, 2, 16))
        none = torch.full((130,), -1, dtype=torch.int32, device="cuda")
        y = layer.forward(inp["x"], adapter_ids=none).clone()
        torch.cuda.synchronize()
        # the gates are made from fp64 logits here and from fp32 ones there: they differ by a few 2^-24, which moves a
        # few elements of y across a rounding border, a whole bf16 step (2^-7 relative at most) each
        assert (y != want).float().mean() <= 0.01
        assert rel_l2(np64(y), np64(want)) <= 0.1 * 2.0 ** -7
        none[5] = 2
        again = layer.forward(inp["x"], adapter_ids=none)
        assert layer.status()[1] == ops.MOE_STATUS_BAD_ADAPTER
        assert torch.equal(y, again)


@pytest.mark.parametrize("base", [BASE, _c(E4, num_shared=1), _c(BASE, capacity=30)], ids=("bf16", "e4m3", "capacity"))
def test_stage_call_equals_the_layer(base):
    """permute -> moe_grouped_ffn_lora -> combine of the layer's own selection gives its outputs."""
    cfg = _c(base, S=180)
    S = cfg.S
    inp = syn.make_inputs(cfg, "cuda", seed=24)
    ad = make_adapters(cfg, 4, 16)
    ids = runs(S, 4)
    layer = MoELayer(cfg, inp, adapters=ad)
    want = layer.forward(inp["x"], adapter_ids=ids).clone()
    desc, w, lora = layer.desc, layer.weights, layer.lora
    ws = torch.empty(ops.moe_lora_workspace_size(desc, lora), dtype=torch.uint8, device="cuda")
    ops.moe_workspace_init(ws)
    R = ops.moe_routed_rows(desc)
    i32 = dict(dtype=torch.int32, device="cuda")
    idx, gw = layer.topk_idx.clone(), layer.topk_w.clone()
    counts = torch.empty((cfg.E,), **i32)
    offsets, ros, tor = torch.empty((2 * (cfg.E + 1),), **i32), torch.empty((S * cfg.K,), **i32), torch.empty((R,), **i32)
    xp = torch.zeros((R, cfg.d), dtype=torch.bfloat16, device="cuda")
    yp = torch.zeros((R + cfg.num_shared * S, cfg.d), dtype=torch.bfloat16, device="cuda")
    y = torch.empty((S, cfg.d), dtype=torch.bfloat16, device="cuda")
    ops.moe_permute(desc, inp["x"], idx, counts, offsets, ros, tor, xp, ws)
    ops.moe_grouped_ffn_lora(desc, w, lora, ids, xp, offsets, tor, inp["x"], yp, ws)
    ops.moe_combine(desc, yp, ros, gw, y, ws)
    torch.cuda.synchronize()
    assert ops.moe_get_status(ws)[1] == 0
    assert torch.equal(y, want)


@pytest.mark.parametrize("base,offsets", [
    (BASE, [0, 64, 0, 64, 0, 64, 0, 64, 0]),                     # four groups claim all rows: twice the lists' room
    (_c(BASE, num_shared=1), [0, 8, 16, 24, 32, 40, 48, 118, 138]),  # the last one runs into the shared expert's rows
    (_c(BASE, capacity=64), list(range(0, 513, 64)) + [0] * 9),   # every expert full: more rows than S * K
], ids=("overlap", "past-the-routed-rows", "full"))
def test_offsets_that_claim_too_many_rows_leave_groups_without_adapters(base, offsets):
    """Groups whose rows the adapters' lists have no room for go without adapters and are reported."""
    cfg = _c(base, S=64)
    inp = syn.make_inputs(cfg, "cuda", seed=26)
    layer = MoELayer(cfg, inp, adapters=make_adapters(cfg, 4, 16))
    R = ops.moe_routed_rows(layer.desc)
    assert max(offsets) <= R + cfg.num_shared * 64
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    tor = (torch.arange(R, dtype=torch.int32) % 64).cuda()
    ids = torch.arange(64, dtype=torch.int32, device="cuda") % 4
    xp = torch.zeros((R, cfg.d), dtype=torch.bfloat16, device="cuda")
    xp[:] = inp["x"][tor.long()]
    yp = torch.full((R + cfg.num_shared * 64 + 1, cfg.d), 7.0, dtype=torch.bfloat16, device="cuda")
    ops.moe_grouped_ffn_lora(layer.desc, layer.weights, layer.lora, ids, xp, off, tor, inp["x"], yp, layer.ws)
    torch.cuda.synchronize()
    assert layer.status()[1] & ops.MOE_STATUS_BAD_GROUP
    assert (yp[-1] == 7.0).all()
    # a good call on the same workspace
    ops.moe_workspace_init(layer.ws)
    ref = MoELayer(cfg, inp, adapters=make_adapters(cfg, 4, 16))
    assert torch.equal(layer.forward(inp["x"], adapter_ids=ids), ref.forward(inp["x"], adapter_ids=ids))
    assert layer.status()[1] == 0


def test_calls_on_two_streams_at_once():
    cfg = _c(BASE, S=200, num_shared=1)
    inp = syn.make_inputs(cfg, "cuda", seed=27)
    ad, ids = make_adapters(cfg, 6, 24), runs(200, 6)
    want = MoELayer(cfg, inp, adapters=ad).forward(inp["x"], adapter_ids=ids).clone()
    layers = [MoELayer(cfg, inp, adapters=ad) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(6):
        for layer, st in zip(layers, streams):
            layer.forward(inp["x"], stream=st, adapter_ids=ids)
    torch.cuda.synchronize()
    for layer in layers:
        assert torch.equal(layer.y, want) and layer.status()[1] == 0


@pytest.mark.parametrize("cfg,n,rank", [
    (_c(BASE, S=200, E=2, K=2), 1, 128), (_c(BASE, S=90, d=8, h=8), 3, 8), (_c(BASE, S=150, E=64, K=32, d=256, h=128), 4096, 8),
    (_c(E4, S=77, d=16, h=16), 2, 8), (_c(E4, S=130, E=1, K=1, num_shared=1), 130, 128),
], ids=("one-adapter", "narrow", "most-adapters", "narrow-e4m3", "an-adapter-each"))
def test_adapters_at_the_edges_of_their_range(cfg, n, rank):
    inp = syn.make_inputs(cfg, "cuda", seed=28)
    ad = make_adapters(cfg, n, rank, seed=3, pairs=("up", "down") if n < 4096 else ("up",))
    ids = (torch.arange(cfg.S, dtype=torch.int32) % n).cuda()
    ids[0] = n - 1
    layer = MoELayer(cfg, inp, adapters=ad)
    y = layer.forward(inp["x"], adapter_ids=ids)
    torch.cuda.synchronize()
    assert layer.status()[1] == 0
    ref, idx, _, margin = reference_layer(inp, cfg, ad, ids)
    keep = margin >= MARGIN
    assert (layer.topk_idx.cpu().numpy()[keep] == idx[keep]).all()
    # roundings: hidden rows, expert outputs, y, the inner products and the deltas of the two stages (each of a part of
    # the sum), the codes; over narrow rows a rounding need not be better than half a step
    k = 9 if cfg.weight_dtype == syn.E4M3 else 7
    assert rel_l2(np64(y)[keep], ref[keep]) <= tol(k) * (3 ** 0.5 if cfg.d < 64 else 1)


def test_decode_and_prefill_of_the_same_requests():
    """As a server uses them: a prompt batch through forward, then the same
    requests' next tokens through decode, one set of adapters."""
    pre = _c(BASE, S=96)
    inp = syn.make_inputs(pre, "cuda", seed=25)
    ad = make_adapters(pre, 6, 16)
    ids = runs(96, 6)
    first = MoELayer(pre, inp, adapters=ad)
    y0 = first.forward(inp["x"], adapter_ids=ids)
    steps = 24
    dec = _c(BASE, S=steps)
    sub = dict(inp, x=inp["x"][-steps:].contiguous())
    tail = ids[-steps:].contiguous()
    second = MoELayer(dec, sub, adapters=ad)
    y1 = second.decode(sub["x"], adapter_ids=tail)
    torch.cuda.synchronize()
    assert torch.equal(second.topk_idx, first.topk_idx[-steps:])
    assert rel_l2(np64(y1), np64(y0[-steps:])) <= tol(6)  # decode's two roundings, forward's four
    assert first.status()[1] == 0 and second.status()[1] == 0


def test_repeats_bit_identically_and_replays():
    cfg = _c(BASE, S=300)
    inp = syn.make_inputs(cfg, "cuda", seed=26)
    ids = runs(300, 5)
    layer = MoELayer(cfg, inp, adapters=make_adapters(cfg, 5, 32))
    first = layer.forward(inp["x"], adapter_ids=ids).clone()
    assert torch.equal(layer.forward(inp["x"], adapter_ids=ids), first)
    y = torch.empty_like(first)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.forward(inp["x"], y=y, adapter_ids=ids)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, first)
    ids.copy_(ids.flip(0))
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, layer.forward(inp["x"], adapter_ids=ids))


def test_experts_closer_than_fp32_tells_apart_are_picked_by_their_exact_keys():
    """Router rows that differ in one element by one bf16 step, met by tokens
    whose element there is tiny: the logits differ by about 2^-30 of their size,
    far below fp32's steps, and the exact order still decides, in both calls and
    on both sides of the 32 experts above which the tensor-core logits come
    first."""
    for E in (8, 32, 40, 64):
        cfg = _c(BASE, S=64, E=E, K=2, d=1024, h=128, router_offset_var=0.0)
        inp = syn.make_inputs(cfg, "cpu", seed=28)
        g = torch.Generator().manual_seed(5)
        base = torch.randn(1024, generator=g) / 8
        w = inp["w_router"].float() * 0.05
        w[2:E:3] = base  # a third of the experts, far ahead of the others for half of the tokens
        w = w.bfloat16()
        cols = torch.randperm(1024, generator=g)[:E]
        for e in range(2, E, 3):
            w[e, cols[e]] = torch.nextafter(w[e, cols[e]], torch.tensor(9.0, dtype=torch.bfloat16))
        x = inp["x"].float()
        x[:, cols] = (torch.randn((64, E), generator=g) * 2.0 ** -18)
        x = x.bfloat16()
        inp["x"], inp["w_router"] = x, w
        logits = x.double() @ w.double().T
        top, order = torch.sort(logits, dim=1, descending=True, stable=True)
        want = order[:, :2].int()
        gap = torch.minimum(top[:, 0] - top[:, 1], top[:, 1] - top[:, 2])
        assert (gap < 2.0 ** -22).sum() >= 16  # such tokens are there
        clear = gap > 2.0 ** -44  # fp64 sums of 1024 products of this size are good to about 2^-47
        assert clear.sum() >= 48
        dev = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in inp.items()}
        layer = MoELayer(cfg, dev, adapters=make_adapters(cfg, 2, 8))
        ids = make_ids(64, 2)
        layer.forward(dev["x"], adapter_ids=ids)
        assert torch.equal(layer.topk_idx.cpu()[clear], want[clear]), E
        layer.topk_idx.zero_()
        layer.decode(dev["x"], adapter_ids=ids)
        assert torch.equal(layer.topk_idx.cpu()[clear], want[clear]), E
        assert layer.status()[1] == 0


@pytest.mark.parametrize("over", [dict(E=64, K=8, num_groups=8, topk_groups=2, score_fn=syn.SIGMOID, sel_bias_var=0.01),
                                  dict(E=256, K=8, num_groups=8, topk_groups=2, score_fn=syn.SIGMOID, num_shared=1),
                                  dict(E=128, K=4, renormalize=0), dict(E=45, K=3, temperature=0.5),
                                  dict(E=16, K=4, num_groups=4, topk_groups=2, renormalize=0, score_fn=syn.SIGMOID)])
def test_routers(over):
    cfg = _c(BASE, S=300, d=256, h=64, router_offset_var=0.0, **over)
    inp = syn.make_inputs(cfg, "cuda", seed=29)
    layer = MoELayer(cfg, inp, adapters=make_adapters(cfg, 2, 8))
    ids = make_ids(300, 2)
    layer.forward(inp["x"], adapter_ids=ids)
    torch.cuda.synchronize()
    _, idx, gates, margin = reference_layer_routing(inp, cfg)
    keep = margin >= MARGIN
    assert (layer.topk_idx.cpu().numpy()[keep] == idx[keep]).all()
    assert np.abs(np64(layer.topk_w)[keep] - gates[keep]).max() <= 4e-7  # fp64 logits: a few roundings of 2^-24
    assert layer.status()[1] == 0
    inp["x"] = inp["x"].clone()
    inp["x"][7, 3] = float("nan")
    y = layer.forward(inp["x"], adapter_ids=ids)
    code, flags, counters = layer.status()
    assert flags == ops.MOE_STATUS_NONFINITE_LOGIT and counters["nonfinite"] == 1
    assert torch.isnan(y[7].float()).all() and torch.isfinite(y[8:].float()).all()


def test_rerouted_layer_with_adapters():
    cfg = _c(BASE, S=256, E=16, K=2, capacity=40, reroute=1)
    inp = syn.make_inputs(cfg, "cuda", seed=27)
    ad = make_adapters(cfg, 3, 16)
    ids = runs(256, 3)
    layer = MoELayer(cfg, inp, adapters=ad)
    y = layer.forward(inp["x"], adapter_ids=ids)
    torch.cuda.synchronize()
    ref, idx, _, margin = reference_layer(inp, cfg, ad, ids)
    if (margin >= MARGIN).all():
        assert (layer.topk_idx.cpu().numpy() == idx).all()
        assert rel_l2(np64(y), ref) <= tol(4)
    assert layer.status()[1] == 0
