"""Selection by moe_layer_forward_lora where fp32 sums or fp32 keys cannot
tell two experts apart: the picks are those of the exact keys, in 64 bits.

Every case makes sums or keys whose fp32 roundings are as large as the gaps
between the experts, in another way each: a dominant element in front of many
products near the sum's last bit, large products that cancel, the same at
scales whose squares leave fp32's range, and biases that cancel a large logit
or score."""
import dataclasses

import numpy as np
import pytest
import torch

from mixture_experts_layer_bias_b200 import synthetic as syn
from mixture_experts_layer_bias_b200.layer import MoELayer

from adapters import make_adapters
from parity import np64

pytestmark = pytest.mark.gpu

BASE = syn.LayerConfig("router", S=64, d=1024, E=8, K=2, h=8)


def _bf16(a):
    return torch.as_tensor(np.asarray(a, np.float64)).bfloat16()


def _check(cfg, x, w, router_bias=None, sel_bias=None, close=0.0):
    """Picks of forward against the order of the keys in 64 bits, for tokens
    whose K + 1 best keys lie further apart than 64-bit sums are off; `close`
    of those keys' gaps at least must be as small as fp32 steps of what they
    are made of (so that the case tests what it says)."""
    inp = syn.make_inputs(dataclasses.replace(cfg, router_offset_var=0.0, sel_bias_var=0.0), "cpu", seed=1)
    inp.update(x=x, w_router=w, router_bias=router_bias, sel_bias=sel_bias)
    xd, wd = np64(x), np64(w)
    logits = xd @ wd.T
    scale = (np.abs(xd) @ np.abs(wd).T).max()
    if router_bias is not None:
        logits = logits + np64(router_bias)
        scale = scale + np.abs(np64(router_bias)).max()
    if cfg.score_fn == syn.SIGMOID:
        keys, slope = 1 / (1 + np.exp(-logits)), 1.0
    else:
        keys, slope = logits / (cfg.temperature or 1.0), 1 / (cfg.temperature or 1.0)
    most = max(scale * slope, np.abs(keys).max())
    if sel_bias is not None:
        keys = keys + np64(sel_bias)
    order = np.argsort(-keys, axis=1, kind="stable")
    top = np.take_along_axis(keys, order, 1)[:, :cfg.K + 1]
    gap = (top[:, :-1] - top[:, 1:]).min(1)
    clear = gap > most * cfg.d * 2.0 ** -52  # an upper bound of what 64-bit sums of d products are off by
    assert clear.mean() >= 0.9
    assert (gap[clear] < most * 2.0 ** -20).mean() >= close
    dev = {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in inp.items()}
    layer = MoELayer(cfg, dev, adapters=make_adapters(cfg, 1, 8, pairs=("up",)))
    layer.forward(dev["x"], adapter_ids=torch.full((cfg.S,), -1, dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert layer.status()[1] == 0
    picks = layer.topk_idx.cpu().numpy()
    wrong = (picks[clear] != order[clear, :cfg.K]).any(1)
    assert not wrong.any(), f"{int(wrong.sum())} of {int(clear.sum())} tokens"


@pytest.mark.parametrize("d", [1024, 8192])
@pytest.mark.parametrize("step", [23, 24, 25, 26])
def test_products_near_the_last_bit_of_a_dominant_one(d, step):
    """Expert 0's small products are each just below 2^-step of the dominant
    product, which every expert has; expert 1 has nearly their sum in a single
    product, a little less, and the others are far behind."""
    rng = np.random.default_rng(step)
    x, w = np.zeros((64, d)), np.zeros((8, d))
    x[:, 1:] = 2.0 ** -12
    w[0, 1:] = 2.0 ** (12 - step) * (1 - 2.0 ** -7)
    small = (d - 1) * 2.0 ** -12 * w[0, 1]
    at = rng.integers(0, 32, 64)  # the dominant element's column, in the first piece
    x[np.arange(64), at] = 1.0
    w[:, :32] = 1.0
    w[2:, :32] = 0.5
    # one column of expert 1 alone carries the small products' sum times 1 - 2^-2 .. 1 - 2^-8, by token
    lone = d - 1
    w[0, lone], w[1, lone] = 0.0, 2.0 ** -4
    less = 1 - 2.0 ** -(2 + np.arange(64) % 7)
    x[:, lone] = small * less / 2.0 ** -4
    _check(dataclasses.replace(BASE, d=d, K=1), _bf16(x), _bf16(w))


def test_sums_that_lose_every_product_in_opposite_directions():
    """Eight stretches of columns each start with a product of 1; expert 0 adds
    products below a sum's last bit to it, expert 1 subtracts some, and three
    further columns give expert 1 all of that back but for a tiny rest: at
    65,536 columns a sum that drops the small products is off by more than
    2^-12 of its size."""
    d, unit = 65536, 2.0 ** -24
    x, w = np.zeros((64, d)), np.zeros((8, d))
    x[:, 256:] = 2.0 ** -12
    near, far = 2.0 ** -13 * (1 - 2.0 ** -7), 2.0 ** -11 * (1 - 2.0 ** -7)  # products of half a unit and of two units
    w[0, 256:], w[1, 256:] = near, -near
    w[0, 256::32], w[0, 260::32] = far, far
    x[:, 0:256:32] = 1.0
    w[:, 0:256:32] = 1.0
    w[2:, 0:256:32] = 0.5
    both = 2.0 ** -12 * (w[0, 256:].sum() - w[1, 256:].sum())
    for t in range(64):
        rest = both - (1 + t) * 12 * unit  # expert 0 leads by 12 to 768 units
        for c in (1, 2, 3):
            x[t, c] = float(_bf16(rest / 2.0 ** -4))
            rest -= 2.0 ** -4 * x[t, c]
    w[1, 1:4] = 2.0 ** -4
    _check(dataclasses.replace(BASE, d=d, K=1), _bf16(x), _bf16(w), close=0.0)


def _cancelling(scale, d=4096):
    """x and w whose products hold +512 and -512 (times the scale) far apart
    in one stretch of columns and, between them, products of a few fp32 steps
    of 512."""
    rng = np.random.default_rng(7)
    x, w = np.zeros((64, d)), np.zeros((8, d))
    first, last = 0, d - 256
    x[:, [first, last]] = 64.0
    w[:, first], w[:, last] = 8.0, -8.0
    cols = np.arange(256, last, 256)  # 32 columns of every 256 meet in one sum: these do, one after another
    x[:, cols] = rng.normal(size=(64, len(cols)))
    w[:, cols] = rng.normal(size=(8, len(cols))) * 2.0 ** -14
    return _bf16(x * scale), _bf16(w)


def test_large_products_that_cancel():
    x, w = _cancelling(1.0)
    _check(dataclasses.replace(BASE, d=4096), x, w, close=0.5)


@pytest.mark.parametrize("exponent", [-40, -90, 40, 60])
def test_large_products_that_cancel_at_any_scale(exponent):
    x, w = _cancelling(2.0 ** exponent)
    _check(dataclasses.replace(BASE, d=4096), x, w, close=0.5)


def test_cancelling_products_of_small_rows_and_small_router_weights():
    """x and w at scales whose lengths' product still is a normal number but whose squares' product is not."""
    x, w = _cancelling(2.0 ** -45)
    _check(dataclasses.replace(BASE, d=4096), x, (w.float() * 2.0 ** -40).bfloat16(), close=0.5)


def test_a_selection_bias_that_cancels_a_large_tempered_score():
    """score = (x w + router bias) / tau around 10^5, the selection bias takes
    all but 1024 x w of it away: the score's fp32 steps are larger than the gaps."""
    rng = np.random.default_rng(8)
    d = 256
    x, w = np.zeros((64, d)), np.zeros((8, d))
    x[:, :8] = rng.normal(size=(64, 8))
    w[:, :8] = rng.normal(size=(8, 8)) * 8e-6
    rb = torch.tensor(2.0 ** (4 + 4 * rng.random(8)), dtype=torch.float32)  # of several sizes: steps of several sizes
    sb = rb * -1024.0  # exact
    _check(dataclasses.replace(BASE, d=d, temperature=2.0 ** -10), _bf16(x), _bf16(w), rb, sb, close=0.5)


def test_a_selection_bias_that_cancels_sigmoid_scores():
    """Scores around 1/2 whose differences of about 1e-7 the selection bias lays bare."""
    rng = np.random.default_rng(9)
    d = 256
    x, w = np.zeros((64, d)), np.zeros((8, d))
    x[:, :8] = rng.normal(size=(64, 8))
    w[:, :8] = rng.normal(size=(8, 8)) * 4e-7
    rb = torch.tensor(0.02 * rng.random(8) - 0.01, dtype=torch.float32)
    sb = torch.tensor(-1 / (1 + np.exp(-np64(rb))), dtype=torch.float32)
    _check(dataclasses.replace(BASE, d=d, score_fn=syn.SIGMOID), _bf16(x), _bf16(w), rb, sb, close=0.5)
