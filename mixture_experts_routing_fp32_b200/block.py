"""A block around the layer: norm, MoE layer, norm, gate, residual sum.

  x     = N(r) w_pre + b_pre                 (or handed on by the block before)
  y     = layer(x)
  r_out = r + alpha gate (N(y) w_post + b_post)
  x'    = N(r_out) w_next + b_next           (the next block's x, same pass)

The block owns the norms' buffers and a MoELayer, all allocated once with
stable pointers, so a step can be captured in a CUDA graph.  Parameters of a
forward call that are None are left out (no post norm, gate, biases, next
norm).  A forward keeps references to its inputs: backward needs them as they
were.  No host synchronisation happens inside forward or backward.
"""
from __future__ import annotations

import torch

from . import api
from ._lib import MoEError
from .layer import MoELayer


def _overlap(a, b):
    lo, at = a.data_ptr(), b.data_ptr()
    return lo < at + b.numel() * b.element_size() and at < lo + a.numel() * a.element_size()


class MoEBlock:
    """cfg: the layer's configuration; norm, eps, alpha, resid as in
    make_norm_config; gate_len: tokens that share a row of `gate` (0: no
    gate); layer_kw: MoELayer's."""

    def __init__(self, cfg, norm="rms", eps=1e-5, alpha=1.0, gate_len=0, resid=None,
                 device="cuda", **layer_kw):
        if cfg.n_local_experts:
            raise MoEError("MoEBlock: the outputs of expert shards are sums to be formed before "
                           "the norm; use moe_block_norm after the exchange")
        self.layer = MoELayer(cfg, device=device, **layer_kw)
        c = self.layer.cfg
        act = self.layer.act_dtype
        kinds = {None: act, "bf16": torch.bfloat16, "fp32": torch.float32}
        if resid not in kinds:
            raise MoEError("MoEBlock: resid is 'bf16' or 'fp32', not %r" % (resid,))
        self.resid_dtype = kinds[resid]
        make = lambda L: api.make_norm_config(  # noqa: E731
            c.T, c.D, norm=norm, dtype=act, resid=self.resid_dtype, eps=eps, alpha=alpha,
            gate_len=L)
        self.pre, self.post = make(0), make(gate_len)
        ws = max(api.moe_block_norm_ws_bytes(self.pre), api.moe_block_norm_ws_bytes(self.post))
        dev = self.device = self.layer.device
        e = lambda dt, *shape: torch.empty(shape, dtype=dt, device=dev)  # noqa: E731
        T, D, f32 = c.T, c.D, torch.float32
        self.x, self.x_next = e(act, T, D), e(act, T, D)
        self.r_out = e(self.resid_dtype, T, D)
        self.stats_pre, self.stats = e(f32, T, 4), e(f32, T, 4)
        self._ws_bytes = ws
        self._grads_ready = False
        self._saved = None

    def forward(self, r, weights, w_pre=None, b_pre=None, w_post=None, b_post=None, gate=None,
                w_next=None, b_next=None, x=None, **layer_inputs):
        """(r_out, x'), x' None without w_next.  weights: MoELayer.forward's
        (w_r, w13, w_down[, w13_s, w_down_s]); layer_inputs: its other
        arguments.  Either x (normalised by the block before) or w_pre.

        r may be this block's own r_out, and x its x_next (a block applied
        again): the outputs are right, but what a backward pass needs is
        overwritten, so that backward refuses.  The block's other buffers are
        refused as inputs."""
        if (x is None) == (w_pre is None):
            raise MoEError("MoEBlock.forward: either x or w_pre")
        if r is None:
            raise MoEError("MoEBlock.forward: no r")
        # the layer's entry points take their sizes from cfg alone
        n = self.layer.cfg.T * self.layer.cfg.D
        api._args("MoEBlock.forward", None, ("r", r, self.resid_dtype, n),
                  ("x", x, self.layer.act_dtype, n))
        # what is written before r, x are read for the last time
        early = [("layer.y", self.layer.y)] + ([("x", self.x)] if x is None else [])
        if w_next is not None:
            early.append(("x_next", self.x_next))
        for name, t in early:
            if _overlap(r, t):
                raise MoEError("MoEBlock.forward: r shares memory with the block's %s" % name)
        if r.data_ptr() != self.r_out.data_ptr() and _overlap(r, self.r_out):
            raise MoEError("MoEBlock.forward: r shares memory with a part of the block's r_out")
        if x is not None and _overlap(x, self.layer.y):
            raise MoEError("MoEBlock.forward: x shares memory with the block's layer.y")
        # backward reads x (the layer) or, with w_pre, r (the norm before it)
        kept = r if x is None else x
        lost = _overlap(kept, self.r_out) or (w_next is not None and _overlap(kept, self.x_next))
        self._saved = None      # a call that fails from here on leaves no forward
        if x is None:
            api.moe_block_norm(self.pre, r, None, None, None, None, w_pre, b_pre, None, self.x,
                               self.stats_pre)
            own_x = self.x
        else:
            own_x = x
        y = self.layer.forward(own_x, *weights, **layer_inputs)
        x_next = None if w_next is None else self.x_next
        api.moe_block_norm(self.post, r, y, w_post, b_post, gate, w_next, b_next, self.r_out,
                           x_next, self.stats)
        self._saved = dict(r=r, y=y, lost=lost, x_given=x is not None, w_pre=w_pre, b_pre=b_pre,
                           w_post=w_post, b_post=b_post, gate=gate, w_next=w_next, b_next=b_next)
        return self.r_out, x_next

    def _alloc_grads(self):
        if self._grads_ready:
            return
        c, dev = self.layer.cfg, self.device
        f32 = torch.float32
        self.dy = torch.empty(c.T, c.D, dtype=self.layer.act_dtype, device=dev)
        self.dr = torch.empty(c.T, c.D, dtype=self.resid_dtype, device=dev)
        v = lambda: torch.empty(c.D, dtype=f32, device=dev)  # noqa: E731
        self.dw_pre, self.db_pre, self.dw_post, self.db_post = v(), v(), v(), v()
        self.dw_next, self.db_next = v(), v()
        L = self.post.gate_len
        self.dgate = torch.empty(-(-c.T // L), c.D, dtype=f32, device=dev) if L else None
        self.ws = torch.empty(self._ws_bytes, dtype=torch.uint8, device=dev)
        self._grads_ready = True

    def backward(self, dr_out, dx_next=None):
        """(dr, dx): the gradient of r and, when x was given, that of x (for
        the block before, as its dx_next; else None).  dx_next: the gradient
        of x' (required with w_next).  The parameters' gradients are in
        dw_post, db_post, dgate, dw_next, db_next, dw_pre, db_pre (of those
        that were given) and in the layer's own buffers."""
        s = self._saved
        if s is None:
            raise MoEError("MoEBlock.backward: no forward before")
        if s["lost"]:
            raise MoEError("MoEBlock.backward: the forward overwrote its input (the block's own "
                           "r_out or x_next); give it a copy")
        if (dx_next is None) != (s["w_next"] is None):
            raise MoEError("MoEBlock.backward: dx_next goes with w_next")
        self._alloc_grads()
        want = lambda p, g: None if s[p] is None else g  # noqa: E731
        api.moe_block_norm_backward(
            self.post, self.r_out, s["y"], s["w_post"], s["b_post"], s["gate"], s["w_next"],
            self.stats, dx_next, dr_out, self.dy, self.dr, want("w_post", self.dw_post),
            want("b_post", self.db_post), want("gate", self.dgate),
            want("w_next", self.dw_next), want("b_next", self.db_next), self.ws)
        dx = self.layer.backward(self.dy)
        if s["x_given"]:
            return self.dr, dx
        api.moe_block_norm_backward(
            self.pre, s["r"], None, None, None, None, s["w_pre"], self.stats_pre, dx, self.dr,
            None, self.dr, None, None, None, self.dw_pre, want("b_pre", self.db_pre), self.ws)
        return self.dr, None
