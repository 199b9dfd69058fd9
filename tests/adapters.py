"""Helpers of the tests of the few-token layer and of the adapters: seeded
adapters and the layer with adapters in float64, expert by expert, routed by
the oracle."""
from __future__ import annotations

import math

import numpy as np
import torch

from mixture_experts_layer_bias_b200 import synthetic as syn
from oracle import moe_oracle as O

from parity import np64, oracle_routing

# One rounding to bf16 is off by at most half a step, 2^-8 relative; over many
# independent elements its root mean square is at most 2^-8 / sqrt(3).  n such
# roundings on the way to y (hidden rows, expert outputs, y, ...) therefore give
# a relative L2 error of at most sqrt(n) times that.
HALF_STEP = torch.finfo(torch.bfloat16).eps / 2


def tol(n: int) -> float:
    return math.sqrt(n) * HALF_STEP / math.sqrt(3)


def rows_rel(a, b) -> float:
    """Largest relative L2 error of a row."""
    a, b = np.asarray(a, np.float64), np.asarray(b, np.float64)
    return float(np.max(np.linalg.norm(a - b, axis=-1) / np.maximum(np.linalg.norm(b, axis=-1), 1e-300)))


def make_adapters(cfg, n, rank, seed=0, device="cuda", share=0.5, pairs=("gate", "up", "down")):
    """n adapters whose share of a projection's sums has about `share` times
    their size (rows of unit variance)."""
    g = torch.Generator().manual_seed(1000 + seed)
    slabs = cfg.E + cfg.num_shared
    out = dict(scale=(torch.rand(n, generator=g) + 0.5).to(device))
    for name, o, i in (("gate", cfg.h, cfg.d), ("up", cfg.h, cfg.d), ("down", cfg.d, cfg.h)):
        if name not in pairs or (name == "gate" and cfg.activation == syn.GELU):
            continue
        a = torch.randn((n, slabs, rank, i), generator=g) / math.sqrt(i)
        b = torch.randn((n, slabs, o, rank), generator=g) * share / math.sqrt(rank)
        out["a_" + name], out["b_" + name] = a.bfloat16().to(device), b.bfloat16().to(device)
    return out


def make_ids(S, n, seed=0, device="cuda"):
    g = torch.Generator().manual_seed(2000 + seed)
    return torch.randint(-1, n, (S,), generator=g, dtype=torch.int32).to(device)


def reference_layer(inp, cfg, adapters=None, ids=None):
    """y [S][d], indices and gates of the layer (with adapters) in float64."""
    x, idx, gates, margin = oracle_routing(inp, cfg)
    ids = None if ids is None else ids.cpu().numpy()
    y = np.zeros((cfg.S, cfg.d))

    def weight(name, e):
        t = inp[name][e]
        if t.dtype == torch.uint8:
            return O.e4m3_bits_to_f64(t.cpu().numpy()) * np64(inp["s_" + name[2:]][e])[:, None]
        return np64(t)

    def project(name, pair, e, rows, tokens):
        out = rows @ weight(name, e).T
        if adapters is None or "a_" + pair not in adapters:
            return out
        for a in range(adapters["scale"].numel()):
            m = ids[tokens] == a
            if m.any():
                u = rows[m] @ np64(adapters["a_" + pair][a, e]).T
                out[m] += u @ np64(adapters["b_" + pair][a, e]).T * float(adapters["scale"][a])
        return out

    for e in range(cfg.E + cfg.num_shared):
        tokens, k = np.nonzero(idx == e) if e < cfg.E else (np.arange(cfg.S), None)
        if not len(tokens):
            continue
        rows = x[tokens]
        if cfg.activation == syn.GELU:
            z = project("w1", "up", e, rows, tokens) + np64(inp["b1"][e])
            hid = O.gelu_erf(z)
            out = project("w2", "down", e, hid, tokens) + np64(inp["b2"][e])
        else:
            gate = project("w_gate", "gate", e, rows, tokens)
            hid = O.silu(gate) * project("w_up", "up", e, rows, tokens)
            out = project("w_down", "down", e, hid, tokens)
        y[tokens] += out if k is None else out * gates[tokens, k][:, None]
    return y, idx, gates, margin
