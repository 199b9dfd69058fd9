"""moe_route with computed logits for expert counts above 32 that are not a
multiple of 4: the logits GEMM stores four columns at a time, so these take
the CUDA-core logits kernel."""
import numpy as np
import pytest
import torch

from mixture_experts_layer_bias_b200 import ops
from oracle import moe_oracle as O

from parity import MARGIN, assert_status_clean, new_ws, np64

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("E,S", [(33, 5), (37, 130), (62, 64), (255, 33), (36, 50)])
def test_wide_routers_of_any_width(E, S):
    g = torch.Generator().manual_seed(E)
    d, K = 264, 4
    x = torch.randn((S, d), generator=g).bfloat16()
    w = (torch.randn((E, d), generator=g) / d ** 0.5).bfloat16()
    desc = ops.make_desc(num_tokens=S, d_model=d, num_experts=E, top_k=K, d_ff=64)
    ws = new_ws(desc)
    idx = torch.empty((S, K), dtype=torch.int32, device="cuda")
    gw = torch.empty((S, K), dtype=torch.float32, device="cuda")
    wr = w.cuda()
    ops.moe_route(desc, ops.make_weights(dict(w_router=wr)), x.cuda(), None, idx, gw, ws)
    torch.cuda.synchronize()
    assert_status_clean(ws)
    logits = O.router_logits(np64(x), np64(w), None)
    ridx, rw = O.select_experts(logits, K, "softmax", True)
    keep = O.selection_margin(logits, K, "softmax") >= MARGIN
    assert keep.mean() > 0.9
    np.testing.assert_array_equal(idx.cpu().numpy()[keep], ridx[keep])
    assert np.abs(np64(gw)[keep] - rw[keep]).max() <= 2e-5
