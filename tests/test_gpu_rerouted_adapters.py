"""Re-routing beside adapters: picks, gates and outputs of every token."""
import dataclasses

import numpy as np
import pytest
import torch

from mixture_experts_layer_bias_b200 import synthetic as syn
from mixture_experts_layer_bias_b200.layer import MoELayer

from adapters import make_adapters, make_ids, reference_layer, tol
from parity import np64, oracle_routing, rel_l2

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("capacity,num_shared", [(40, 0), (33, 1)])
def test_rerouted_layer_with_adapters_matches_float64(capacity, num_shared):
    cfg = syn.LayerConfig("rerouted", S=256, d=512, E=16, K=2, h=512, router_offset_var=0.5, capacity=capacity, reroute=1,
                          num_shared=num_shared)
    inp = syn.make_inputs(cfg, "cpu", seed=29)
    # re-routing compares any two keys of a token: with these inputs (drawn on the CPU: the same everywhere) none is
    # closer than the fp32 keys that it works on can tell
    logits = np.sort(np64(inp["x"]) @ np64(inp["w_router"]).T + np64(inp["router_bias"]), axis=1)
    assert np.diff(logits, axis=1).min() > 1e-4
    first = oracle_routing(inp, dataclasses.replace(cfg, reroute=0))[1]
    dev = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in inp.items()}
    ad, ids = make_adapters(cfg, 3, 16), make_ids(256, 3, seed=1)
    layer = MoELayer(cfg, dev, adapters=ad)
    y = layer.forward(dev["x"], adapter_ids=ids)
    torch.cuda.synchronize()
    ref, idx, gates, _ = reference_layer(dev, cfg, ad, ids)
    moved = int((idx != first).any(1).sum())
    assert moved > 0
    code, flags, counters = layer.status()
    assert flags == 0 and counters["rerouted"] >= moved
    assert (layer.topk_idx.cpu().numpy() == idx).all()
    assert np.abs(np64(layer.topk_w) - gates).max() <= 2e-5  # from fp32 logits of order 10
    assert rel_l2(np64(y), ref) <= tol(4)
