"""The serving form of a MoE layer: forward only, expert weights in 8-bit
integers with a scale per output channel, activations quantised per token.

  forward : moe_router -> experts
  experts : moe_dispatch (layout only) -> moe_expert_ffn_i8 -> moe_combine

The layer owns its buffers (stable pointers, so a step can be captured in a
CUDA graph) and keeps nothing for a backward pass.  No host synchronisation.
"""
from __future__ import annotations

import ctypes

import torch

from . import api
from ._lib import MOE_GEMM_AUTO, MOE_GEMM_I8, MoEError, MoeConfig, check, lib


class MoEInt8Layer:
    def __init__(self, cfg, device="cuda"):
        c = self.cfg = MoeConfig.from_buffer_copy(cfg)
        if c.gemm_impl == MOE_GEMM_AUTO:
            c.gemm_impl = MOE_GEMM_I8
        self.ws_bytes = api.moe_expert_ffn_i8_ws_bytes(c)     # refuses what it cannot serve
        z = self.sizes = api.moe_get_sizes(c)
        dev = self.device = torch.device(device)
        T, D, E, K = c.T, c.D, c.E, c.K
        El = self.n_local = c.n_local_experts or E
        R = int(z.rows_max)
        f32, i32 = torch.float32, torch.int32
        e = lambda shape, dt: torch.empty(shape, dtype=dt, device=dev)  # noqa: E731
        self.logits, self.probs, self.lse = e((T, E), f32), e((T, E), f32), e((T,), f32)
        self.topk_idx, self.topk_w, self.near_ties = e((T, K), i32), e((T, K), f32), e((1,), i32)
        self.counts, self.kept, self.offsets = e((E,), i32), e((El,), i32), e((El + 2,), i32)
        self.slot_row, self.row_slot = e((T * K,), i32), e((R,), i32)
        self.tile_expert, self.stats = e((int(z.tiles_max),), i32), e((4,), i32)
        self.o, self.y = e((R, D), torch.bfloat16), e((T, D), torch.bfloat16)
        self.ws = e((max(int(z.ws_bytes), 256),), torch.uint8)
        self.ws_i8 = e((self.ws_bytes,), torch.uint8)
        self.weights = None
        # arguments that stay the same from call to call, marshalled once
        P = api._p
        self._cfg_p = ctypes.byref(c)
        self._layout = [P(t) for t in (self.counts, self.kept, self.offsets, self.slot_row,
                                       self.row_slot, self.tile_expert, self.stats)]
        self._map = [P(t) for t in (self.offsets, self.slot_row, self.row_slot, self.tile_expert,
                                    self.stats)]
        self._o, self._y, self._off = P(self.o), P(self.y), P(self.offsets)
        self._slots, self._ws, self._ws_i8 = P(self.slot_row), P(self.ws), P(self.ws_i8)

    def _shapes(self):
        c, El = self.cfg, self.n_local
        s = {"w13": (El, 2 * c.F, c.D), "w_down": (El, c.D, c.F)}
        if c.n_shared:
            s.update(w13_s=(2 * c.F, c.D), w_down_s=(c.D, c.F))
        return s

    def set_weights(self, w13, w13_scale, w_down, w_down_scale, w13_s=None, w13_s_scale=None,
                    w_down_s=None, w_down_s_scale=None):
        """8-bit weights [.., channels, inputs] (int8) and their scales [..,
        channels] (fp32), used where they are: the layer keeps references."""
        given = dict(w13=(w13, w13_scale), w_down=(w_down, w_down_scale),
                     w13_s=(w13_s, w13_s_scale), w_down_s=(w_down_s, w_down_s_scale))
        shapes = self._shapes()
        kept = []
        for k, (q, s) in given.items():
            shape = shapes.get(k)
            if shape is None:
                if q is not None or s is not None:
                    raise MoEError("set_weights: %s without a shared expert" % k)
                kept += [None, None]
                continue
            for t, want, dt in ((q, shape, torch.int8), (s, shape[:-1], torch.float32)):
                if (t is None or tuple(t.shape) != want or t.dtype != dt or not t.is_contiguous()
                        or t.device != self.y.device):
                    raise MoEError("set_weights: %s is not a contiguous tensor of %s %s on %s"
                                   % (k, want, dt, self.y.device))
            kept += [q, s]
        self.weights = tuple(kept)
        self._w = [api._p(t) for t in kept]

    def quantize(self, w13, w_down, w13_s=None, w_down_s=None):
        """Quantises fp32 or bf16 weights (MoELayer's) and takes them."""
        out = []
        for k, w in dict(w13=w13, w_down=w_down, w13_s=w13_s, w_down_s=w_down_s).items():
            if w is None:
                out += [None, None]
                continue
            q = torch.empty(w.shape, dtype=torch.int8, device=w.device)
            s = torch.empty(w.shape[:-1], dtype=torch.float32, device=w.device)
            api.moe_quant_i8(w, q, s)
            out += [q, s]
        self.set_weights(*out)

    def _inputs(self, x, *specs):
        """Pointers of x and the other inputs, and the stream; refuses what
        does not fit the layer."""
        if self.weights is None:
            raise MoEError("MoEInt8Layer: no weights (set_weights or quantize first)")
        if x is None:
            raise MoEError("MoEInt8Layer: no x")
        c = self.cfg
        out = api._args("MoEInt8Layer", None, ("x", x, torch.bfloat16, c.T * c.D), *specs)
        if self.y.get_device() != x.get_device():
            raise MoEError("MoEInt8Layer: the layer is on %s, x on %s" % (self.device, x.device))
        return out

    def experts(self, x, topk_idx, topk_w, sentinel_mask=None):
        """y [T, D] for given picks (topk_idx [T, K] int32, -1: none; topk_w
        [T, K] fp32): the layer's own buffer, rewritten by the next call."""
        c, L = self.cfg, lib()
        xp, idx, w, mask, s = self._inputs(
            x, ("topk_idx", topk_idx, torch.int32, c.T * c.K),
            ("topk_w", topk_w, torch.float32, c.T * c.K),
            ("sentinel_mask", sentinel_mask, torch.uint8, c.T * c.K))
        check(L.moe_dispatch(self._cfg_p, idx, mask, xp, *self._layout, None, self._ws, s),
              "moe_dispatch")
        check(L.moe_expert_ffn_i8(self._cfg_p, xp, *self._map, *self._w, self._o, self._ws_i8, s),
              "moe_expert_ffn_i8")
        check(L.moe_combine(self._cfg_p, self._o, self._slots, w, self._off, self._y, s),
              "moe_combine")
        return self.y

    def forward(self, x, w_r, logit_offset=None, sel_bias=None, sentinel_mask=None):
        """Router (fp32, as MoELayer's) and experts."""
        c = self.cfg
        # the router's entry point takes its sizes from cfg alone
        self._inputs(x, ("w_r", w_r, torch.float32, c.E * c.D),
                     ("logit_offset", logit_offset, torch.float32, c.E),
                     ("sel_bias", sel_bias, torch.float32, c.E),
                     ("sentinel_mask", sentinel_mask, torch.uint8, c.T * c.K))
        api.moe_router(self.cfg, x, w_r, logit_offset, sel_bias, self.logits, self.probs,
                       self.lse, self.topk_idx, self.topk_w, self.near_ties, self.ws)
        return self.experts(x, self.topk_idx, self.topk_w, sentinel_mask)
