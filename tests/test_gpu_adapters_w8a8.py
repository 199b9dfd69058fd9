"""W8A8 layers with adapters, in the few-token call and in the call for any
number of tokens: the base products take E4M3 rows, the adapters the bf16 rows
they were made from."""
import dataclasses

import numpy as np
import pytest
import torch

from mixture_experts_layer_bias_b200 import synthetic as syn
from mixture_experts_layer_bias_b200.layer import MoELayer
from oracle import moe_oracle as O

from adapters import make_adapters, make_ids, tol
from parity import FP8_REL_L2, MARGIN, np64, oracle_routing, rel_l2

pytestmark = pytest.mark.gpu

BASE = syn.LayerConfig("w8a8", S=1, d=512, E=8, K=2, h=512, router_offset_var=0.5, weight_dtype=syn.E4M3, act_quant=1)


def _c(**kw):
    return dataclasses.replace(BASE, **kw)


def _quantised(rows):
    q, s = O.quantize_rows_e4m3(rows.astype(np.float32))
    return O.e4m3_bits_to_f64(q) * s[:, None].astype(np.float64)


def reference(inp, cfg, ad, ids):
    """The layer in float64 over the rows' codes, hidden rows rounded to bf16."""
    x, idx, gates, margin = oracle_routing(inp, cfg)
    ids = ids.cpu().numpy()
    y = np.zeros((cfg.S, cfg.d))

    def project(name, e, rows, tokens):
        w = O.e4m3_bits_to_f64(inp["w_" + name][e].cpu().numpy()) * np64(inp["s_" + name][e])[:, None]
        out = _quantised(rows) @ w.T
        for a in range(ad["scale"].numel()):
            m = ids[tokens] == a
            if m.any() and "a_" + name in ad:
                u = rows[m] @ np64(ad["a_" + name][a, e]).T
                out[m] += u @ np64(ad["b_" + name][a, e]).T * float(ad["scale"][a])
        return out

    for e in range(cfg.E + cfg.num_shared):
        tokens, k = np.nonzero(idx == e) if e < cfg.E else (np.arange(cfg.S), None)
        if not len(tokens):
            continue
        hid = O.silu(project("gate", e, x[tokens], tokens)) * project("up", e, x[tokens], tokens)
        hid = O.bf16_bits_to_f64(O.f64_to_bf16_bits_fast(hid))
        out = project("down", e, hid, tokens)
        y[tokens] += out if k is None else out * gates[tokens, k][:, None]
    return y, idx, margin


def _case(cfg, n, rank, pairs=("gate", "up", "down")):
    inp = syn.make_inputs(cfg, "cuda", seed=31)
    ad = make_adapters(cfg, n, rank, seed=5, pairs=pairs)
    ids = make_ids(cfg.S, n, seed=6)
    ids[0] = n - 1
    ref, idx, margin = reference(inp, cfg, ad, ids)
    keep = margin >= MARGIN
    assert keep.mean() >= 0.7
    none = reference(inp, cfg, ad, torch.full_like(ids, -1))[0]
    assert rel_l2(none[keep], ref[keep]) > 3 * FP8_REL_L2  # the adapters matter
    return inp, ad, ids, ref, idx, keep


@pytest.mark.parametrize("cfg,n,rank,pairs", [
    (_c(S=1), 1, 8, None), (_c(S=9, h=1040, num_shared=1), 3, 16, None), (_c(S=16), 4, 128, None),
    (_c(S=17, d=272, h=208), 5, 40, None), (_c(S=64, h=768), 32, 64, None), (_c(S=21), 2, 16, ("down",)),
    (_c(S=21), 2, 16, ("gate",)), (_c(S=31, E=64, K=8, d=256, h=128, num_shared=1), 6, 24, None),
], ids=lambda v: f"S{v.S}-d{v.d}-h{v.h}-E{v.E}" if isinstance(v, syn.LayerConfig) else None)
def test_decode_matches_float64(cfg, n, rank, pairs):
    inp, ad, ids, ref, idx, keep = _case(cfg, n, rank, pairs or ("gate", "up", "down"))
    layer = MoELayer(cfg, inp, adapters=ad)
    y = layer.decode(inp["x"], adapter_ids=ids)
    torch.cuda.synchronize()
    assert layer.status()[1] == 0
    assert (layer.topk_idx.cpu().numpy()[keep] == idx[keep]).all()
    # Rounding to steps s a value that is off by t moves the result by s with probability t / s: sqrt(t s) root mean
    # square.  fp32 sums of up to 1040 products are off by less than 2^-16 of a hidden value, its bf16 step is at most
    # 2^-7 of it, that of its E4M3 code 2^-3: sqrt(sqrt(2^-16 2^-7) 2^-3) = 6.6e-3, beside y's own rounding.
    assert rel_l2(np64(y)[keep], ref[keep]) <= (6.6e-3 ** 2 + tol(1) ** 2) ** 0.5


@pytest.mark.parametrize("cfg,n,rank,pairs", [
    (_c(S=5), 2, 16, None), (_c(S=130, num_shared=1), 3, 16, None), (_c(S=400, d=272, h=208), 6, 40, None),
    (_c(S=333, E=64, K=8, d=256, h=144), 12, 32, None), (_c(S=600, E=16, K=4, capacity=100), 6, 8, None),
    (_c(S=200), 3, 128, ("up", "down")),
], ids=lambda v: f"S{v.S}-d{v.d}-h{v.h}-E{v.E}" if isinstance(v, syn.LayerConfig) else None)
def test_forward_matches_float64(cfg, n, rank, pairs):
    inp, ad, ids, ref, idx, keep = _case(cfg, n, rank, pairs or ("gate", "up", "down"))
    layer = MoELayer(cfg, inp, adapters=ad)
    y = layer.forward(inp["x"], adapter_ids=ids)
    torch.cuda.synchronize()
    assert layer.status()[1] == 0
    assert (layer.topk_idx.cpu().numpy()[keep] == idx[keep]).all()
    # as above, with the adapters' inner products and shares of the hidden sums rounded to bf16, each a part of a sum:
    # t = tol(2) = 3.2e-3 of a hidden value's size, sqrt(3.2e-3 2^-3) = 2.0e-2; the down pair's two roundings, the
    # expert rows' and y's add tol(4) = 4.5e-3: 2.1e-2, within the 8-bit path's contract
    assert rel_l2(np64(y)[keep], ref[keep]) <= FP8_REL_L2
