"""The few-token layer's gates come from 64-bit logits."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_bias_b200 import synthetic as syn
from mixture_experts_layer_bias_b200.layer import MoELayer

from parity import np64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("K,renormalize", [(2, 1), (8, 1), (4, 0)])
def test_decode_gates_of_logits_that_fp32_sums_lose(K, renormalize):
    """Products of +-2^14 cancel in every logit: fp32 sums of them are off by
    about 2^-10, the gates must not be."""
    rng = np.random.default_rng(K)
    d = 1024
    cfg = syn.LayerConfig("gates", S=16, d=d, E=8, K=K, h=64, renormalize=renormalize)
    inp = syn.make_inputs(cfg, "cpu", seed=2)
    x, w = inp["x"].float(), inp["w_router"].float()
    x[:, 0::128], x[:, 64::128] = 2.0 ** 10, 2.0 ** 10
    w[:, 0::128], w[:, 64::128] = 2.0 ** 4, -(2.0 ** 4)
    inp["x"], inp["w_router"] = x.bfloat16(), w.bfloat16()
    logits = np64(inp["x"]) @ np64(inp["w_router"]).T
    dev = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in inp.items()}
    layer = MoELayer(cfg, dev)
    layer.decode(dev["x"])
    torch.cuda.synchronize()
    idx = np.argsort(-logits, axis=1, kind="stable")[:, :K]
    assert (layer.topk_idx.cpu().numpy() == idx).all()
    picked = np.take_along_axis(logits, idx, 1)
    base = picked if renormalize else logits
    top = base.max(1, keepdims=True)
    want = np.exp(picked - top) / np.exp(base - top).sum(1, keepdims=True)
    # g = e / sum e, e = exp(z), z <= 0 rounded to fp32: |z| e^z 2^-24 <= 2^-25.4 absolute, the exponential two units,
    # 2^-22 relative (both for the numerator and for the sum), the sum's 8 additions and the division 2^-24 each
    limit = 2 * 2.0 ** -22 + 2 * 2.0 ** -25.4 + 9 * 2.0 ** -24
    assert np.abs(np64(layer.topk_w) - want).max() <= limit
