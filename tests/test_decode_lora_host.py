"""Host-side checks of moe_layer_decode and of the calls that take adapters:
sizes, refusals and the binding's own checks.  No GPU: none of these calls
reaches a CUDA API."""
import ctypes

import pytest
import torch

from mixture_experts_layer_bias_b200 import build as B
from mixture_experts_layer_bias_b200 import ops
from mixture_experts_layer_bias_b200 import synthetic as syn

from adapters import make_adapters


@pytest.fixture(scope="module", autouse=True)
def built_library():
    B.build()
    return ops.lib()


P = ctypes.c_void_p(0x10000)
WS = ctypes.c_void_p(0x100000)


def _desc(name="mixtral_decode", **over):
    cfg = syn.CONFIGS[name] if name in syn.CONFIGS else syn.VARIANTS[name]
    return ops.make_desc(**dict(syn.desc_dict(cfg), **over))


def _weights(e4m3=False, gelu=False):
    names = ["w_router"] + (["w1", "w2", "b1", "b2"] if gelu else ["w_gate", "w_up", "w_down"])
    if e4m3:
        names += ["s_gate", "s_up", "s_down"]
    return ops.make_weights({n: 0x20000 for n in names})


def _lora(**over):
    lora = ops.MoeLora()
    lora.num_adapters, lora.rank = 4, 16
    for f in ops.LORA_FIELDS:
        setattr(lora, f, 0x30000)
    for k, v in over.items():
        setattr(lora, k, v)
    return lora


def _decode(desc, w, lora, ids, x=P, y=P, ws=WS, n=None):
    size = ctypes.c_size_t(0)
    if n is None:
        ops.lib().moe_decode_workspace_size(ctypes.byref(desc), ops._byref(lora), ctypes.byref(size))
        n = size.value
    return ops.lib().moe_layer_decode(ctypes.byref(desc), None if w is None else ctypes.byref(w), ops._byref(lora), ids,
                                      x, y, None, None, None, ws, n, None)


def _size_code(desc, lora=None):
    n = ctypes.c_size_t(0)
    return ops.lib().moe_decode_workspace_size(ctypes.byref(desc), ops._byref(lora), ctypes.byref(n))


def test_decode_takes_few_tokens_of_bf16_layers():
    for S in (0, 1, 64):
        assert _size_code(_desc(num_tokens=S)) == ops.MOE_OK
        assert _size_code(_desc("mixtral_decode_e4m3", num_tokens=S)) == ops.MOE_OK
        assert _size_code(_desc("mixtral_decode_e4m3", num_tokens=S, act_quant=1)) == ops.MOE_OK
    assert _size_code(_desc(num_tokens=65)) == ops.MOE_ERR_INVALID_ARG
    assert _size_code(_desc("tiny_f32")) == ops.MOE_ERR_UNSUPPORTED
    assert _size_code(_desc("fp8_skew_capacity_reroute", num_tokens=8)) == ops.MOE_ERR_UNSUPPORTED
    assert _size_code(_desc("mixtral_decode_e4m3", d_model=4104)) == ops.MOE_ERR_UNSUPPORTED
    assert _size_code(_desc("mixtral_decode_e4m3", d_ff=14344)) == ops.MOE_ERR_UNSUPPORTED
    assert _size_code(_desc(top_k=9)) == ops.MOE_ERR_INVALID_ARG


def test_decode_refuses_layers_its_tables_cannot_hold():
    # 256 experts' tiles of 256 columns at two bytes a tile have to fit beside the weight ring's shared memory
    big = dict(num_tokens=64, num_experts=256, top_k=8, d_ff=512)
    assert _size_code(_desc(d_model=79872, **big)) == ops.MOE_OK
    assert _size_code(_desc(d_model=131072, **big)) == ops.MOE_ERR_UNSUPPORTED
    assert _size_code(_desc(d_model=131072, **dict(big, num_tokens=1))) == ops.MOE_OK  # 8 experts at most
    # more than 2^30 steps
    assert _size_code(_desc(num_tokens=1, num_experts=8, top_k=8, d_model=1 << 20, d_ff=1 << 21)) == ops.MOE_ERR_UNSUPPORTED
    d, w = _desc(d_model=131072, **big), _weights()
    assert _decode(d, w, None, None, n=1 << 40) == ops.MOE_ERR_UNSUPPORTED


def test_decode_workspace_grows_with_the_batch_and_the_rank():
    one, all_ = (ops.moe_decode_workspace_size(_desc(num_tokens=S)) for S in (1, 64))
    assert one % 256 == 0 and all_ > one
    assert all_ >= 64 * 2 * 14336 * 2                     # the hidden rows
    lora = _lora()
    assert ops.moe_decode_workspace_size(_desc(num_tokens=64), lora) >= all_ + 64 * 2 * 3 * 16 * 4  # inner products


def test_decode_refusals():
    d, w = _desc(num_tokens=4), _weights()
    assert _decode(d, w, None, None, ws=None) == ops.MOE_ERR_WORKSPACE
    assert _decode(d, w, None, None, ws=ctypes.c_void_p(0x100010)) == ops.MOE_ERR_WORKSPACE
    assert _decode(d, w, None, None, n=256) == ops.MOE_ERR_WORKSPACE
    assert _decode(d, w, None, None, x=None) == ops.MOE_ERR_INVALID_ARG
    assert _decode(d, w, None, None, y=None) == ops.MOE_ERR_INVALID_ARG
    assert _decode(d, w, None, None, x=ctypes.c_void_p(0x10004)) == ops.MOE_ERR_INVALID_ARG
    assert _decode(d, None, None, None) == ops.MOE_ERR_INVALID_ARG
    assert _decode(d, ops.MoeWeights(), None, None) == ops.MOE_ERR_INVALID_ARG
    assert _decode(_desc("mixtral_decode_e4m3", num_tokens=4), w, None, None) == ops.MOE_ERR_INVALID_ARG  # no scales
    # adapters and their ids go together
    assert _decode(d, w, _lora(), None) == ops.MOE_ERR_INVALID_ARG
    assert _decode(d, w, None, P) == ops.MOE_ERR_INVALID_ARG
    # no tokens: nothing to do
    assert _decode(_desc(num_tokens=0), None, None, None, x=None, y=None) == ops.MOE_OK


BAD_LORA = [dict(num_adapters=0), dict(num_adapters=4097), dict(num_adapters=-1), dict(rank=0), dict(rank=12), dict(rank=136), dict(rank=-8)]
BAD_POINTERS = [dict(b_gate=None), dict(a_up=None), dict(scale=None), dict(scale=0x30002), dict(a_down=0x30008),
                dict(a_gate=None, b_gate=None, a_up=None, b_up=None, a_down=None, b_down=None)]


@pytest.mark.parametrize("over", BAD_LORA)
def test_bad_adapter_shapes(over):
    d, lora = _desc(num_tokens=4), _lora(**over)
    n = ctypes.c_size_t(0)
    L = ops.lib()
    assert _size_code(d, lora) == ops.MOE_ERR_INVALID_ARG
    assert L.moe_lora_workspace_size(ctypes.byref(d), ctypes.byref(lora), ctypes.byref(n)) == ops.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("over", BAD_POINTERS)
def test_bad_adapter_pointers(over):
    d, w, lora = _desc(num_tokens=4), _weights(), _lora(**over)
    L = ops.lib()
    big = 1 << 40
    assert _decode(d, w, lora, P) == ops.MOE_ERR_INVALID_ARG
    assert L.moe_layer_forward_lora(ctypes.byref(d), ctypes.byref(w), ctypes.byref(lora), P, P, P, None, None, None, WS,
                                    big, None) == ops.MOE_ERR_INVALID_ARG
    assert L.moe_grouped_ffn_lora(ctypes.byref(d), ctypes.byref(w), ctypes.byref(lora), P, P, P, P, P, P, WS, big,
                                  None) == ops.MOE_ERR_INVALID_ARG


def test_adapters_of_the_staged_calls():
    L = ops.lib()
    d, w, lora = _desc("mixtral_prefill"), _weights(), _lora()
    n = ops.moe_lora_workspace_size(d, lora)
    assert n >= ops.moe_workspace_size(d) + 4096 * 2 * 2 * 14336 * 2  # the adapters' share of gate and up
    args = (ctypes.byref(d), ctypes.byref(w), ctypes.byref(lora), P, P, P, None, None, None, WS)
    assert L.moe_layer_forward_lora(*args, n - 256, None) == ops.MOE_ERR_WORKSPACE
    assert L.moe_layer_forward_lora(ctypes.byref(d), ctypes.byref(w), None, P, P, P, None, None, None, WS, n,
                                    None) == ops.MOE_ERR_INVALID_ARG
    assert L.moe_layer_forward_lora(ctypes.byref(d), ctypes.byref(w), ctypes.byref(lora), None, P, P, None, None, None,
                                    WS, n, None) == ops.MOE_ERR_INVALID_ARG
    # the stage call needs the permutation's token map
    assert L.moe_grouped_ffn_lora(ctypes.byref(d), ctypes.byref(w), ctypes.byref(lora), P, P, P, None, P, P, WS, n,
                                  None) == ops.MOE_ERR_INVALID_ARG
    f = _desc("tiny_f32")
    size = ctypes.c_size_t(0)
    assert L.moe_lora_workspace_size(ctypes.byref(f), ctypes.byref(lora), ctypes.byref(size)) == ops.MOE_ERR_UNSUPPORTED
    # a GeLU layer has no gate projection
    g = _desc(num_tokens=4, activation=0)
    assert _decode(g, _weights(gelu=True), lora, P) == ops.MOE_ERR_INVALID_ARG
    empty = _desc("mixtral_prefill", num_tokens=0)
    assert L.moe_layer_forward_lora(ctypes.byref(empty), ctypes.byref(w), ctypes.byref(lora), None, None, None, None,
                                    None, None, WS, ops.moe_lora_workspace_size(empty, lora), None) == ops.MOE_OK


def test_make_lora_checks_types_and_shapes():
    cfg = syn.scaled(syn.CONFIGS["mixtral_decode"], S=2, d=64, h=32, E=4)
    ad = make_adapters(cfg, 3, 8, device="cpu")
    lora = ops.make_lora(ad)
    assert (lora.num_adapters, lora.rank) == (3, 8) and lora.a_gate == ad["a_gate"].data_ptr()
    part = ops.make_lora({k: ad[k] for k in ("a_up", "b_up", "scale")})
    assert part.a_gate is None and part.b_down is None
    for bad in (dict(scale=ad["scale"].half()), dict(a_up=ad["a_up"].float()), dict(b_up=ad["b_up"][:2]),
                dict(b_down=ad["b_down"].transpose(2, 3)), dict(b_gate=ad["b_gate"][..., :4].contiguous()),
                dict(a_down=ad["a_down"][:, :3].contiguous())):
        with pytest.raises(ValueError):
            ops.make_lora(dict(ad, **bad))
    with pytest.raises(ValueError):
        ops.make_lora(dict(scale=ad["scale"]))


def test_layer_refuses_adapters_of_another_layer():
    from mixture_experts_layer_bias_b200.layer import MoELayer
    cfg = syn.scaled(syn.CONFIGS["mixtral_decode"], S=2, d=64, h=32, E=4)
    for other in (dict(d=32), dict(h=64), dict(E=8)):
        with pytest.raises(ValueError):
            MoELayer(cfg, {}, adapters=make_adapters(syn.scaled(cfg, S=2, **dict(dict(d=64, h=32, E=4), **other)), 3, 8,
                                                     device="cpu"))


def test_adapters_on_another_device_are_refused():
    """Their addresses go to the kernels as they are, so this is refused before anything is made or launched."""
    from mixture_experts_layer_bias_b200.layer import MoELayer
    cfg = syn.scaled(syn.CONFIGS["mixtral_decode"], S=2, d=64, h=32, E=4)
    ad = make_adapters(cfg, 3, 8, device="cpu")
    with pytest.raises(ValueError, match="device"):
        MoELayer(cfg, {}, adapters=ad)  # on the GPU by default
    for f in ("scale", "b_up", "a_down"):
        with pytest.raises(ValueError, match=f"{f} lies on"):
            ops.make_lora(dict(ad, **{f: ad[f].to("meta")}))
    with pytest.raises(ValueError):
        ops.make_lora(dict(ad, a_gate=ad["a_gate"][0]))
    with pytest.raises(ValueError):
        ops.make_lora(dict(ad, b_down=ad["b_down"][0]))
    with pytest.raises(ValueError):
        ops.make_lora(dict(ad, scale=ad["scale"][:, None]))


def test_decode_takes_every_width_that_its_header_promises():
    """moe.h: min(E, S * K) + num_shared experts of up to so many million / that many columns of d always fit."""
    import os
    import re
    text = open(os.path.join(B.INCLUDE, "moe.h")).read()
    promised = int(re.search(r"up to (\d+) M / that many", re.sub(r"[\s*]+", " ", text)).group(1)) * 1_000_000
    refused = []
    for over in (dict(), dict(weight_dtype=syn.E4M3), dict(weight_dtype=syn.E4M3, act_quant=1)):
        for E in (8, 32, 256):
            for ns in (0, 1):
                for S in range(1, 65):
                    for K in (1, 2, 8, 24, 29, 30, 31, 32):
                        if K > E:
                            continue
                        d = promised // (min(E, S * K) + ns) // 16 * 16
                        desc = _desc(num_tokens=S, num_experts=E, top_k=K, num_shared=ns, d_model=d, d_ff=16, **over)
                        if _size_code(desc) != ops.MOE_OK:
                            refused.append((over, E, ns, S, K, d))
    assert not refused, (len(refused), refused[:4])


def test_adapters_workspace_holds_the_slices_that_are_used():
    """The inner products lie there by slice of their length: eight of them in small batches, one in large ones."""
    def bytes_per_rank(**over):
        d = _desc("mixtral_prefill", **over)
        return (ops.moe_lora_workspace_size(d, _lora(rank=128)) - ops.moe_lora_workspace_size(d, _lora(rank=64))) / 64
    rows = 16384 * 8
    assert bytes_per_rank(num_tokens=16384, num_experts=64, top_k=8) == rows * 2 * 4
    assert bytes_per_rank(num_tokens=64, top_k=2) == 8 * 64 * 2 * 2 * 4
    # a hidden width of 512 has two slices of 256, its one pair half as many products a slice as gate and up have
    assert bytes_per_rank(num_tokens=64, top_k=2, d_model=256, d_ff=512) == 64 * 2 * 2 * 4
