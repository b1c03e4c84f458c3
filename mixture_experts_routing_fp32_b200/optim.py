"""AdamW over a layer's weights and the vectors around it: owns the states
(allocated once, stable pointers, so a step can be captured in a CUDA graph)
and issues moe_adamw on the current stream.  No host synchronisation.
"""
from __future__ import annotations

import torch

from . import api
from ._lib import MOE_ADAMW_BLOCK, MoEError


class MoEAdamW:
    """params, grads: lists of contiguous CUDA tensors (fp32 or bf16), e.g. the
    weights given to MoELayer and its dw_r, dw13, dw_down; the gradients'
    buffers are read at every step.

    state    "fp32", or "fp8": e4m3 with a scale for every 256 elements
    masters  keep an fp32 copy of every bf16 parameter and update that
    no_decay indices into params of those that weight decay leaves out
    """

    def __init__(self, params, grads, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01,
                 state="fp32", masters=False, no_decay=()):
        params, grads = list(params), list(grads)
        if len(params) != len(grads):
            raise MoEError("MoEAdamW: %d parameters, %d gradients" % (len(params), len(grads)))
        if state not in ("fp32", "fp8"):
            raise MoEError("MoEAdamW: state is 'fp32' or 'fp8', not %r" % (state,))
        no_decay = set(no_decay)
        if not no_decay <= set(range(len(params))):
            raise MoEError("MoEAdamW: no_decay names parameters that are not there: %r"
                           % (sorted(no_decay - set(range(len(params))), key=repr),))
        self.cfg = api.make_adamw_config(lr, betas[0], betas[1], eps, weight_decay)
        self.entries = []
        for i, (p, g) in enumerate(zip(params, grads)):
            e = {"param": p, "grad": g, "decay": i not in no_decay}
            if masters and p.dtype == torch.bfloat16:
                e["master"] = p.float()
            if state == "fp32":
                for k in ("m", "v"):
                    e[k] = torch.zeros(p.shape, dtype=torch.float32, device=p.device)
            else:
                nb = -(-p.numel() // MOE_ADAMW_BLOCK)
                for k in ("m", "v"):
                    e[k] = torch.zeros(p.numel(), dtype=torch.uint8,
                                       device=p.device).view(torch.float8_e4m3fn)
                    e[k + "_scale"] = torch.zeros(nb, dtype=torch.float32, device=p.device)
            self.entries.append(e)
        self.table = api.adamw_table(self.entries)
        self.count = torch.zeros(2, dtype=torch.int32, device=self.table.device or "cuda")

    def step(self, lr=None, grad_scale=None):
        """One step on the gradients in their buffers.  lr, grad_scale: fp32
        device tensors of one element (read when the step runs) or None."""
        api.moe_adamw(self.cfg, self.table, self.count, lr, grad_scale)
