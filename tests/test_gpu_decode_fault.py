"""Failure detection of the few-token layer on the GPU without a GPU fault.

Every wait of its kernel is bounded in time.  A test hook, present only in the
test build of the library (moe_test_stall_decode(1)), makes the next launch run
with a producer that delivers no tile -- a flag nothing sets -- so that the
waits of every CTA give up, MOE_STATUS_TIMEOUT is raised and the kernel leaves
with its copies landed and its counters set back.  After moe_workspace_init the
same context and workspace must give a right layer.  The test build is loaded
in a child process of its own.
"""
import json
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CHILD = r"""
import json, sys
sys.path.insert(0, {root!r}); sys.path.insert(0, {tests!r})
import torch
from mixture_experts_layer_bias_b200 import ops, synthetic as syn
from mixture_experts_layer_bias_b200.build import TEST_HOOKS_LIB
ops._LIB_PATH = TEST_HOOKS_LIB
from adapters import make_adapters, make_ids
from mixture_experts_layer_bias_b200.layer import MoELayer
name = "mixtral_decode_e4m3" if {e4m3!r} else "mixtral_decode"
cfg = syn.scaled(syn.CONFIGS[name] if name in syn.CONFIGS else syn.VARIANTS[name], S=9, d=512, h=768)
inp = syn.make_inputs(cfg, "cuda", seed=0)
adapters = ids = None
if {lora!r}:
    adapters, ids = make_adapters(cfg, 3, 16), make_ids(cfg.S, 3)
layer = MoELayer(cfg, inp, adapters=adapters)
good = layer.decode(inp["x"], adapter_ids=ids).clone()
code0, flags0, _ = layer.status()
ops.lib().moe_test_stall_decode(1)
layer.decode(inp["x"], adapter_ids=ids)
code1, flags1, cnt1 = layer.status()
ops.moe_workspace_init(layer.ws)
again = layer.decode(inp["x"], adapter_ids=ids)
code2, flags2, _ = layer.status()
torch.cuda.synchronize()
print("RESULT " + json.dumps(dict(code0=code0, code1=code1, flags1=flags1, timeouts=cnt1["timeout"], code2=code2,
                                  flags2=flags2, same=bool(torch.equal(good, again)))))
"""


@pytest.mark.parametrize("e4m3,lora", [(False, False), (True, False), (False, True)])
def test_bounded_waits_give_up_and_context_survives(e4m3, lora):
    code = CHILD.format(root=ROOT, tests=os.path.join(ROOT, "tests"), e4m3=e4m3, lora=lora)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-3000:]
    line = [l for l in r.stdout.splitlines() if l.startswith("RESULT ")][-1]
    res = json.loads(line[len("RESULT "):])
    assert res["code0"] == 0, res
    assert res["flags1"] & 0x4, res          # MOE_STATUS_TIMEOUT
    assert res["timeouts"] > 0 and res["code1"] == 5, res
    assert res["flags2"] == 0 and res["code2"] == 0 and res["same"], res
