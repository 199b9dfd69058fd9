"""A buffer-owning wrapper around moe_layer_forward and moe_layer_decode.

``MoELayer`` keeps the descriptor, the weight pointers, optional adapters and a
workspace sized by the library, so a forward pass is one C-ABI call on the
current stream.  Torch only provides the device memory and the stream.
"""
from __future__ import annotations

import torch

from . import ops
from .synthetic import LayerConfig, desc_dict


class MoELayer:
    def __init__(self, cfg: LayerConfig, weights: dict, device="cuda", S=None, with_outputs=True, adapters: dict = None):
        """adapters: the tensors of ops.make_lora; forward and decode then take
        adapter_ids, int32 [S], the adapter of each token (-1: none)."""
        self.cfg = cfg
        self.S = cfg.S if S is None else S
        self.device = torch.device(device)
        self.desc = ops.make_desc(**desc_dict(cfg, self.S))
        self.tensors = weights
        self.weights = ops.make_weights(weights)
        self.adapter_tensors = adapters
        self.lora = None if adapters is None else ops.make_lora(adapters)
        if adapters is not None:
            for f, (rows, cols) in dict(a_gate=(None, cfg.d), a_up=(None, cfg.d), a_down=(None, cfg.h), b_gate=(cfg.h, None),
                                        b_up=(cfg.h, None), b_down=(cfg.d, None)).items():
                t = adapters.get(f)
                if t is not None and (t.shape[1] != cfg.E + cfg.num_shared or (rows or t.shape[2]) != t.shape[2]
                                      or (cols or t.shape[3]) != t.shape[3]):
                    raise ValueError(f"{f} is not of this layer's experts, width or hidden width")
            # the library takes their addresses as they are: memory of another device would fault
            for f in ops.LORA_FIELDS:
                t = adapters.get(f)
                if t is not None and not self._holds(t):
                    raise ValueError(f"{f} lies on {t.device}, not on the layer's device")
        if self.lora is None:
            nbytes = ops.moe_workspace_size(self.desc)
        else:
            nbytes = ops.moe_lora_workspace_size(self.desc, self.lora)
        try:
            nbytes = max(nbytes, ops.moe_decode_workspace_size(self.desc, self.lora))
        except ops.MoeError:
            pass  # not a layer that moe_layer_decode takes: decode() will say so
        self.ws = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=self.device)
        ops.moe_workspace_init(self.ws)
        adt = torch.float32 if cfg.act_dtype == 0 else torch.bfloat16
        self.y = torch.empty((self.S, cfg.d), dtype=adt, device=self.device)
        self.topk_idx = self.topk_w = self.counts = None
        if with_outputs:
            self.topk_idx = torch.empty((self.S, cfg.K), dtype=torch.int32, device=self.device)
            self.topk_w = torch.empty((self.S, cfg.K), dtype=torch.float32, device=self.device)
            self.counts = torch.empty((cfg.E,), dtype=torch.int32, device=self.device)

    def _holds(self, t):
        if t.device.type != "cuda" or self.device.type != "cuda":
            return t.device == self.device
        return t.device.index == (torch.cuda.current_device() if self.device.index is None else self.device.index)

    def _ids(self, adapter_ids):
        if (adapter_ids is None) != (self.lora is None):
            raise ValueError("adapter_ids go with a layer made with adapters")
        if adapter_ids is not None and (adapter_ids.dtype != torch.int32 or tuple(adapter_ids.shape) != (self.S,)
                                        or not adapter_ids.is_contiguous()):
            raise ValueError("adapter_ids must be a contiguous int32 tensor [S]")
        return adapter_ids

    def _checked(self, x, out, ids):
        for t in (x, out):
            if t.dtype != self.y.dtype or tuple(t.shape) != tuple(self.y.shape) or not t.is_contiguous() \
                    or t.device != self.y.device:
                raise ValueError("x and y must be contiguous tensors [S][d] of the layer's type on its device")
        if ids is not None and ids.device != self.y.device:
            raise ValueError("adapter_ids must lie on the layer's device")

    def decode(self, x: torch.Tensor, y: torch.Tensor = None, stream=None, adapter_ids=None) -> torch.Tensor:
        """The layer for a few tokens (S <= ops.MOE_DECODE_MAX_TOKENS) in one kernel."""
        out = self.y if y is None else y
        self._checked(x, out, self._ids(adapter_ids))
        ops.moe_layer_decode(self.desc, self.weights, self.lora, adapter_ids, x, out, self.topk_idx, self.topk_w,
                             self.counts, self.ws, stream)
        return out

    def forward(self, x: torch.Tensor, y: torch.Tensor = None, stream=None, adapter_ids=None) -> torch.Tensor:
        out = self.y if y is None else y
        if self._ids(adapter_ids) is not None:
            self._checked(x, out, adapter_ids)
            ops.moe_layer_forward_lora(self.desc, self.weights, self.lora, adapter_ids, x, out, self.topk_idx,
                                       self.topk_w, self.counts, self.ws, stream)
            return out
        ops.moe_layer_forward(self.desc, self.weights, x, out, self.topk_idx, self.topk_w, self.counts, self.ws,
                              stream)
        return out

    def status(self):
        return ops.moe_get_status(self.ws)
