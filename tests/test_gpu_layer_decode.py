"""moe_layer_decode: the whole layer for a few tokens in one kernel, against
the float64 layer routed by the oracle, for every weight type, activation and
router it takes, with the row counts, widths and loads where it can go wrong."""
import dataclasses

import numpy as np
import pytest
import torch

from mixture_experts_layer_bias_b200 import ops
from mixture_experts_layer_bias_b200 import synthetic as syn
from mixture_experts_layer_bias_b200.layer import MoELayer

from adapters import make_adapters, make_ids, reference_layer, rows_rel, tol
from parity import FP8_REL_L2, MARGIN, compare_layer, np64, rel_l2, run_layer

pytestmark = pytest.mark.gpu

BASE = syn.LayerConfig("decode", S=1, d=512, E=8, K=2, h=512, router_offset_var=0.5)
E4 = dataclasses.replace(BASE, weight_dtype=syn.E4M3)
GELU = dataclasses.replace(BASE, activation=syn.GELU)
FINE = dataclasses.replace(BASE, d=256, E=256, K=8, h=128, score_fn=syn.SIGMOID, num_groups=8, topk_groups=2,
                           num_shared=1, sel_bias_var=0.01, router_offset_var=0.0)


def _c(base, **kw):
    return dataclasses.replace(base, **kw)


CASES = [
    _c(BASE, S=1), _c(BASE, S=2, d=264, h=200), _c(BASE, S=5, d=1000, h=1352), _c(BASE, S=16, h=1024),
    _c(BASE, S=17, d=520, h=136), _c(BASE, S=33, h=768), _c(BASE, S=48, h=256), _c(BASE, S=64, d=1024, h=264),
    _c(BASE, S=3, d=8, h=8), _c(BASE, S=1, d=16, h=4104), _c(BASE, S=7, d=4104, h=16),
    _c(BASE, S=64, E=2, K=2), _c(BASE, S=64, E=1, K=1), _c(BASE, S=31, E=64, K=32, d=256, h=128),
    _c(BASE, S=9, renormalize=0), _c(BASE, S=9, temperature=0.5), _c(BASE, S=9, num_shared=1),
    _c(BASE, S=20, E=32, K=4, capacity=1),
    _c(BASE, S=1, d=2048, h=14336, E=4),
    _c(BASE, S=6, d=256, h=128, E=60, K=6, score_fn=syn.SIGMOID),
    _c(GELU, S=1), _c(GELU, S=3, d=1000, h=1352), _c(GELU, S=64, d=264, h=136, num_shared=1),
    _c(FINE, S=1), _c(FINE, S=2), _c(FINE, S=19), _c(FINE, S=64),
    _c(E4, S=1), _c(E4, S=2, d=272, h=208), _c(E4, S=8, h=1040), _c(E4, S=17, num_shared=1), _c(E4, S=33, h=1408),
    _c(E4, S=64, d=1040, h=272), _c(E4, S=64, E=2, K=2), _c(E4, S=3, d=16, h=16), _c(E4, S=40, E=64, K=8, d=256),
    _c(E4, S=31, E=64, K=32, d=256, h=128),
]


def _id(c):
    return f"{'gelu' if c.activation == syn.GELU else 'swiglu'}-{('f32', 'bf16', 'e4m3')[c.weight_dtype]}" \
           f"-S{c.S}-d{c.d}-h{c.h}-E{c.E}-K{c.K}" + ("-sh" if c.num_shared else "") + \
           (f"-cap{c.capacity}" if c.capacity else "") + ("-w8a8" if c.act_quant else "")


def _run(cfg, inp, adapters=None, ids=None):
    layer = MoELayer(cfg, inp, adapters=adapters)
    y = layer.decode(inp["x"], adapter_ids=ids)
    torch.cuda.synchronize()
    return layer, y


@pytest.mark.parametrize("cfg", CASES, ids=_id)
def test_layer_matches_float64(cfg):
    inp = syn.make_inputs(cfg, "cuda", seed=3)
    layer, y = _run(cfg, inp)
    code, flags, _ = layer.status()
    assert flags == 0
    ref, idx, gates, margin = reference_layer(inp, cfg)
    keep = margin >= MARGIN
    assert keep.sum() >= 0.7 * cfg.S
    assert (layer.topk_idx.cpu().numpy()[keep] == idx[keep]).all()
    # gates: float32 logits and softmax, a few roundings of 2^-24 each on values of order 10
    assert np.abs(np64(layer.topk_w)[keep] - gates[keep]).max() <= 2e-5
    assert np.array_equal(layer.counts.cpu().numpy(),
                          np.bincount(layer.topk_idx.cpu().numpy().reshape(-1), minlength=cfg.E))
    # roundings to bf16: the hidden rows and y; with E4M3 weights also the two-term codes of the tokens and of the
    # hidden rows, each within half a bf16 step of the row's larger values
    n = 4 if cfg.weight_dtype == syn.E4M3 else 2
    err = rel_l2(np64(y)[keep], ref[keep])
    assert err <= tol(n), err
    if cfg.d >= 256 and cfg.h >= 128:
        assert rows_rel(np64(y)[keep], ref[keep]) <= 1.5 * tol(n)


@pytest.mark.parametrize("cfg", [_c(E4, S=1, act_quant=1), _c(E4, S=9, h=1040, act_quant=1, num_shared=1),
                                 _c(E4, S=64, d=272, h=208, act_quant=1)], ids=_id)
def test_w8a8_layer_matches_the_oracle(cfg):
    inp = syn.make_inputs(cfg, "cuda", seed=4)
    layer, y = _run(cfg, inp)
    gpu = dict(y=y, idx=layer.topk_idx)
    rep = compare_layer(gpu, inp, cfg, tol=FP8_REL_L2)
    assert rep["ok"], rep
    assert layer.status()[1] == 0


@pytest.mark.parametrize("cfg", [_c(BASE, S=5), _c(GELU, S=12), _c(FINE, S=16), _c(E4, S=30, d=1040)], ids=_id)
def test_agrees_with_the_staged_layer(cfg):
    inp = syn.make_inputs(cfg, "cuda", seed=5)
    layer, y = _run(cfg, inp)
    staged = run_layer(inp, cfg)
    assert torch.equal(layer.topk_idx, staged["idx"])
    assert torch.equal(layer.counts, staged["counts"])
    assert (layer.topk_w - staged["w"]).abs().max() <= 4e-6
    # the staged layer also rounds every expert's output to bf16; both round the hidden rows and y
    assert rel_l2(np64(y), np64(staged["y"])) <= tol(5)


@pytest.mark.parametrize("cfg", [_c(BASE, S=1, d=1024, h=2048), _c(E4, S=33), _c(FINE, S=7)], ids=_id)
def test_repeats_bit_identically_and_replays(cfg):
    inp = syn.make_inputs(cfg, "cuda", seed=6)
    layer = MoELayer(cfg, inp)
    first = layer.decode(inp["x"]).clone()
    for _ in range(3):
        assert torch.equal(layer.decode(inp["x"]), first)
    # captured twice: two graphs on one workspace, replayed in turn
    graphs = []
    for _ in range(2):
        y = torch.empty_like(first)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            layer.decode(inp["x"], y=y)
        graphs.append((g, y))
    for _ in range(3):
        for g, y in graphs:
            y.zero_()
            g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(y, first) for _, y in graphs)
    # new tokens in the captured buffer
    inp["x"].copy_(torch.randn_like(inp["x"]))
    graphs[0][0].replay()
    torch.cuda.synchronize()
    again = graphs[0][1].clone()
    assert torch.equal(layer.decode(inp["x"]), again) and not torch.equal(again, first)
    assert layer.status()[1] == 0


def test_one_workspace_serves_several_batch_sizes_and_leaves_other_rows():
    base = _c(BASE, S=64, h=768)
    inp = syn.make_inputs(base, "cuda", seed=7)
    w = ops.make_weights(inp)
    n = max(ops.moe_decode_workspace_size(ops.make_desc(**syn.desc_dict(base, S))) for S in (1, 64))
    ws = torch.empty(n, dtype=torch.uint8, device="cuda")
    ops.moe_workspace_init(ws)
    for S in (64, 1, 17, 64, 3):
        desc = ops.make_desc(**syn.desc_dict(base, S))
        y = torch.full((64 + 1, base.d), 7.0, dtype=torch.bfloat16, device="cuda")
        idx = torch.full((65, base.K), -5, dtype=torch.int32, device="cuda")
        ops.moe_layer_decode(desc, w, None, None, inp["x"], y, idx, None, None, ws)
        one = _c(base, S=S)
        sub = dict(inp, x=inp["x"][:S])
        _, ref = _run(one, sub)
        assert torch.equal(y[:S], ref), S
        assert (y[S:] == 7.0).all() and (idx[S:] == -5).all() and (idx[:S] >= 0).all()
    assert ops.moe_get_status(ws)[1] == 0


def test_calls_on_two_streams_at_once():
    cfg = _c(BASE, S=12, d=1024, h=2048)
    inp = syn.make_inputs(cfg, "cuda", seed=8)
    _, want = _run(cfg, inp)
    layers = [MoELayer(cfg, inp) for _ in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(8):
        for layer, st in zip(layers, streams):
            layer.decode(inp["x"], stream=st)
    torch.cuda.synchronize()
    for layer in layers:
        assert torch.equal(layer.y, want) and layer.status()[1] == 0


@pytest.mark.parametrize("base", [BASE, E4], ids=("bf16", "e4m3"))
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_bad_token_spoils_only_its_own_row(base, bad):
    cfg = _c(base, S=9, num_shared=1)
    inp = syn.make_inputs(cfg, "cuda", seed=9)
    _, want = _run(cfg, inp)
    want = want.clone()
    inp["x"] = inp["x"].clone()
    inp["x"][4, 100] = bad
    layer, y = _run(cfg, inp)
    assert layer.status()[1] == ops.MOE_STATUS_NONFINITE_LOGIT
    rest = [t for t in range(9) if t != 4]
    assert torch.isnan(y[4].float()).all()
    assert torch.isfinite(y[rest].float()).all()
    # the other rows' sums may meet other neighbours in their tiles, never other values
    assert rel_l2(np64(y[rest]), np64(want[rest])) <= tol(2)


def test_skewed_router_sends_every_token_to_the_same_experts():
    for S in (1, 15, 64):
        cfg = _c(BASE, S=S, E=16, K=4)
        inp = syn.make_inputs(cfg, "cuda", seed=10)
        inp["router_bias"] = torch.zeros(16, device="cuda")
        inp["router_bias"][[3, 7, 8, 15]] = 100.0
        layer, y = _run(cfg, inp)
        assert layer.counts[[3, 7, 8, 15]].eq(S).all() and layer.counts.sum() == 4 * S
        ref, *_ = reference_layer(inp, cfg)
        assert rel_l2(np64(y), ref) <= tol(2)


ADAPTED = [
    (_c(BASE, S=1), 1, 8, None), (_c(BASE, S=16, d=264, h=200), 5, 16, None), (_c(BASE, S=64, h=768), 32, 64, None),
    (_c(BASE, S=33, num_shared=1), 7, 40, None), (_c(BASE, S=12), 3, 128, None),
    (_c(BASE, S=12), 3, 16, ("gate",)), (_c(BASE, S=12), 3, 16, ("up",)), (_c(BASE, S=12), 3, 16, ("down",)),
    (_c(GELU, S=13, d=1000, h=136), 4, 24, None), (_c(FINE, S=21), 6, 8, None),
    (_c(E4, S=1), 2, 16, None), (_c(E4, S=33, h=1408), 9, 32, None), (_c(E4, S=64, d=272, h=208, num_shared=1), 64, 8, None),
]


@pytest.mark.parametrize("cfg,n,rank,pairs", ADAPTED, ids=[f"{_id(c)}-n{n}-r{r}-{p or 'all'}" for c, n, r, p in ADAPTED])
def test_adapters_match_float64(cfg, n, rank, pairs):
    inp = syn.make_inputs(cfg, "cuda", seed=11)
    ad = make_adapters(cfg, n, rank, seed=1, pairs=pairs or ("gate", "up", "down"))
    ids = make_ids(cfg.S, n, seed=2)
    if cfg.S == 1:
        ids.zero_()
    layer, y = _run(cfg, inp, ad, ids)
    assert layer.status()[1] == 0
    ref, idx, _, margin = reference_layer(inp, cfg, ad, ids)
    plain, *_ = reference_layer(inp, cfg)
    keep = margin >= MARGIN
    assert (layer.topk_idx.cpu().numpy()[keep] == idx[keep]).all()
    assert rel_l2(plain[keep], ref[keep]) > 0.05  # the adapters matter
    k = 4 if cfg.weight_dtype == syn.E4M3 else 2
    assert rel_l2(np64(y)[keep], ref[keep]) <= tol(k)
    assert rows_rel(np64(y)[keep], ref[keep]) <= 1.5 * tol(k)


EDGES = [
    (_c(BASE, S=3, d=8, h=8), 2, 8, None), (_c(E4, S=5, d=16, h=16), 2, 8, None),
    (_c(BASE, S=64, E=2, K=2), 1, 128, None),             # every token: the same adapter, the same experts
    (_c(BASE, S=64, E=1, K=1, num_shared=1), 64, 128, None),
    (_c(GELU, S=17, num_shared=1), 3, 16, ("down",)), (_c(GELU, S=17, num_shared=1), 3, 16, ("up",)),
    (_c(E4, S=17, num_shared=1), 3, 16, ("gate", "down")), (_c(BASE, S=31, E=64, K=32, d=256, h=128), 4096, 8, ("up",)),
]


@pytest.mark.parametrize("cfg,n,rank,pairs", EDGES, ids=[f"{_id(c)}-n{n}-r{r}-{p or 'all'}" for c, n, r, p in EDGES])
def test_adapters_at_the_edges_of_their_range(cfg, n, rank, pairs):
    inp = syn.make_inputs(cfg, "cuda", seed=14)
    ad = make_adapters(cfg, n, rank, seed=3, pairs=pairs or ("gate", "up", "down"))
    ids = make_ids(cfg.S, n, seed=4) if n > 1 else torch.zeros(cfg.S, dtype=torch.int32, device="cuda")
    ids[0] = n - 1
    layer, y = _run(cfg, inp, ad, ids)
    assert layer.status()[1] == 0
    ref, idx, _, margin = reference_layer(inp, cfg, ad, ids)
    keep = margin >= MARGIN
    assert (layer.topk_idx.cpu().numpy()[keep] == idx[keep]).all()
    # as above; over a handful of elements a rounding need not be better than half a step, sqrt(3) times its root mean square
    k = 4 if cfg.weight_dtype == syn.E4M3 else 2
    assert rel_l2(np64(y)[keep], ref[keep]) <= tol(k) * (3 ** 0.5 if cfg.d < 64 else 1)


@pytest.mark.parametrize("cfg", [_c(BASE, S=1, d=1024, h=2048), _c(E4, S=33), _c(FINE, S=40)], ids=_id)
def test_adapters_repeat_bit_identically_and_replay_on_another_stream(cfg):
    inp = syn.make_inputs(cfg, "cuda", seed=15)
    ad = make_adapters(cfg, 5, 16)
    ids = make_ids(cfg.S, 5)
    layer = MoELayer(cfg, inp, adapters=ad)
    first = layer.decode(inp["x"], adapter_ids=ids).clone()
    graphs = []
    for _ in range(2):
        y = torch.empty_like(first)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            layer.decode(inp["x"], y=y, adapter_ids=ids)
        graphs.append((g, y))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for _ in range(3):
            for g, y in graphs:
                y.zero_()
                g.replay()
            assert torch.equal(layer.decode(inp["x"], adapter_ids=ids), first)
    torch.cuda.synchronize()
    assert all(torch.equal(y, first) for _, y in graphs)
    # other adapters in the captured buffer
    ids.copy_((ids + 2) % 5)
    graphs[0][0].replay()
    torch.cuda.synchronize()
    other = graphs[0][1].clone()
    assert torch.equal(layer.decode(inp["x"], adapter_ids=ids), other) and not torch.equal(other, first)
    assert layer.status()[1] == 0


def test_tokens_without_adapter_and_bad_ids():
    cfg = _c(BASE, S=20)
    inp = syn.make_inputs(cfg, "cuda", seed=12)
    _, want = _run(cfg, inp)
    want = want.clone()
    ad = make_adapters(cfg, 4, 16)
    none = torch.full((20,), -1, dtype=torch.int32, device="cuda")
    layer, y = _run(cfg, inp, ad, none)
    assert torch.equal(y, want) and layer.status()[1] == 0
    bad = none.clone()
    bad[3], bad[4] = 4, -2
    layer, y = _run(cfg, inp, ad, bad)
    assert torch.equal(y, want)
    assert layer.status()[1] == ops.MOE_STATUS_BAD_ADAPTER


def test_refusals():
    cfg = _c(BASE, S=4)
    inp = syn.make_inputs(cfg, "cuda", seed=13)
    layer = MoELayer(cfg, inp)
    with pytest.raises(ValueError):
        layer.decode(inp["x"], adapter_ids=make_ids(4, 2))
    adapted = MoELayer(cfg, inp, adapters=make_adapters(cfg, 2, 8))
    with pytest.raises(ValueError):
        adapted.decode(inp["x"])
    with pytest.raises(ValueError):
        adapted.decode(inp["x"], adapter_ids=make_ids(5, 2))
    x = inp["x"]
    for bad in (x[:3], x.float(), x.t().contiguous().t(), x.cpu()):
        with pytest.raises(ValueError):
            layer.decode(bad)
        with pytest.raises(ValueError):
            adapted.forward(bad, adapter_ids=make_ids(4, 2))
    with pytest.raises(ValueError):
        layer.decode(x, y=torch.empty((5, cfg.d), dtype=x.dtype, device="cuda"))
    with pytest.raises(ValueError):
        adapted.decode(x, adapter_ids=make_ids(4, 2, device="cpu"))
