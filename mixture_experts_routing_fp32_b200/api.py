"""Python binding of the C ABI with the same entry-point names.

Each function takes torch tensors (device memory owned by the caller),
passes their data pointers and the current CUDA stream to libmoe.so and
raises MoEError on a non-zero status.  Nothing is computed here.
"""
from __future__ import annotations

import ctypes

import torch

from ._lib import (AdamwConfig, AdamwTensor, MoeConfig, MoeSizes, MoEError, NormConfig, check,
                   lib)
from . import _lib as C


def _p(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _s(stream=None):
    """The stream's handle (by default the current stream's, asked for
    directly: building torch's Stream object takes 3 us)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream


def _args(what, stream, *specs):
    """Pointers of (name, tensor, dtype, elements) and the stream's handle.
    Refuses tensors that are not what a kernel would read: other types or
    sizes, strided ones, ones that are not on the current device."""
    dev = torch._C._cuda_getDevice()
    out = []
    for name, t, dt, n in specs:
        if t is None:
            out.append(None)
            continue
        if t.dtype != dt or t.numel() != n or not t.is_contiguous() or t.get_device() != dev:
            raise MoEError(
                "%s: %s is not a contiguous tensor of %d x %s on the current device (cuda:%d): "
                "%s x %s on %s" % (what, name, n, dt, dev, tuple(t.shape), t.dtype, t.device))
        out.append(t.data_ptr())
    out.append(torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream)
    return out


def make_config(T, D, E, K, F, *, n_shared=0, dtype="bf16", score_fn=0,
                renorm=1, n_groups=1, topk_groups=1, group_score=0,
                capacity_factor=0.0, min_capacity=0, route_scale=1.0,
                aux_alpha=0.0, z_lambda=0.0, gemm_impl=0, seq_len=0,
                expert_choice=0, loss_tokens=0, expert_base=0,
                n_local_experts=0) -> MoeConfig:
    return MoeConfig(
        T=T, D=D, E=E, K=K, F=F, n_shared=n_shared,
        dtype=C.MOE_BF16 if dtype in ("bf16", torch.bfloat16) else C.MOE_FP32,
        score_fn=score_fn, renorm=renorm, n_groups=n_groups,
        topk_groups=topk_groups, group_score=group_score,
        capacity_factor=capacity_factor, min_capacity=min_capacity,
        route_scale=route_scale, aux_alpha=aux_alpha, z_lambda=z_lambda,
        gemm_impl=gemm_impl, seq_len=seq_len, expert_choice=expert_choice,
        loss_tokens=loss_tokens, expert_base=expert_base, n_local_experts=n_local_experts)


def config_from(obj, **over) -> MoeConfig:
    """MoeConfig from any object carrying the layer fields by name."""
    names = ("n_shared", "dtype", "score_fn", "renorm", "n_groups",
             "topk_groups", "group_score", "capacity_factor", "min_capacity",
             "route_scale", "aux_alpha", "z_lambda", "seq_len", "expert_choice",
             "loss_tokens", "expert_base", "n_local_experts")
    kw = {n: getattr(obj, n) for n in names if hasattr(obj, n)}
    kw.update(over)
    return make_config(obj.T, obj.D, obj.E, obj.K, obj.F, **kw)


def moe_get_sizes(cfg: MoeConfig) -> MoeSizes:
    out = MoeSizes()
    check(lib().moe_get_sizes(ctypes.byref(cfg), ctypes.byref(out)), "moe_get_sizes")
    return out


def moe_router(cfg, x, w_r, logit_offset, sel_bias, logits, probs, lse,
               topk_idx, topk_w, near_ties, ws, stream=None):
    check(lib().moe_router(ctypes.byref(cfg), _p(x), _p(w_r), _p(logit_offset),
                           _p(sel_bias), _p(logits), _p(probs), _p(lse),
                           _p(topk_idx), _p(topk_w), _p(near_ties), _p(ws),
                           _s(stream)), "moe_router")


def moe_dispatch(cfg, topk_idx, sentinel_mask, x, counts, kept, offsets,
                 slot_row, row_slot, tile_expert, stats, x_perm, ws, stream=None):
    check(lib().moe_dispatch(ctypes.byref(cfg), _p(topk_idx), _p(sentinel_mask),
                             _p(x), _p(counts), _p(kept), _p(offsets),
                             _p(slot_row), _p(row_slot), _p(tile_expert),
                             _p(stats), _p(x_perm), _p(ws), _s(stream)),
          "moe_dispatch")


def moe_dispatch_static(cfg, topk_idx, sentinel_mask, x, counts, kept, offsets,
                        slot_row, row_slot, tile_expert, stats, x_perm, stream=None):
    """moe_dispatch without a workspace, for callers that cannot allocate
    device memory (see include/moe.h): scratch is the library's static
    device array, so overlapping calls race."""
    check(lib().moe_dispatch_static(ctypes.byref(cfg), _p(topk_idx), _p(sentinel_mask),
                                    _p(x), _p(counts), _p(kept), _p(offsets),
                                    _p(slot_row), _p(row_slot), _p(tile_expert),
                                    _p(stats), _p(x_perm), _s(stream)),
          "moe_dispatch_static")


def moe_route_expert_choice(cfg, x, w_r, logit_offset, logits, probs, lse, topk_idx, topk_w,
                            sentinel_mask, near_ties, ws, stream=None):
    check(lib().moe_route_expert_choice(
        ctypes.byref(cfg), _p(x), _p(w_r), _p(logit_offset), _p(logits), _p(probs), _p(lse),
        _p(topk_idx), _p(topk_w), _p(sentinel_mask), _p(near_ties), _p(ws), _s(stream)),
        "moe_route_expert_choice")


def moe_aux_loss_seq(cfg, probs, lse, topk_idx, slot_row, losses, ws, stream=None):
    check(lib().moe_aux_loss_seq(ctypes.byref(cfg), _p(probs), _p(lse), _p(topk_idx),
                                 _p(slot_row), _p(losses), _p(ws), _s(stream)),
          "moe_aux_loss_seq")


def moe_bias_update(cfg, counts, sel_bias, gamma, stream=None):
    check(lib().moe_bias_update(ctypes.byref(cfg), _p(counts), _p(sel_bias),
                                ctypes.c_float(gamma), _s(stream)), "moe_bias_update")


def moe_aux_loss(cfg, probs, lse, counts, losses, ws, stream=None):
    check(lib().moe_aux_loss(ctypes.byref(cfg), _p(probs), _p(lse), _p(counts),
                             _p(losses), _p(ws), _s(stream)), "moe_aux_loss")


def moe_aux_stats(cfg, probs, lse, sums, ws, stream=None):
    """This batch's load statistics (sums [E+1]) for globally scoped losses."""
    check(lib().moe_aux_stats(ctypes.byref(cfg), _p(probs), _p(lse), _p(sums), _p(ws),
                              _s(stream)), "moe_aux_stats")


def moe_aux_loss_global(cfg, counts, sums, losses, stream=None):
    """Aux and z losses from all-reduced counts and sums (cfg.loss_tokens tokens)."""
    check(lib().moe_aux_loss_global(ctypes.byref(cfg), _p(counts), _p(sums), _p(losses),
                                    _s(stream)), "moe_aux_loss_global")


def moe_set_backward_streams(streams=None):
    """Caller-owned side streams (three torch.cuda.Stream) for moe_backward on
    this thread, or None for the library's own."""
    if streams is None:
        check(lib().moe_set_backward_streams(None), "moe_set_backward_streams")
        return
    arr = (ctypes.c_void_p * 3)(*[s.cuda_stream for s in streams])
    check(lib().moe_set_backward_streams(arr), "moe_set_backward_streams")


def moe_expert_ffn(cfg, x_perm, offsets, tile_expert, stats, w13, w_down,
                   w13_s, w_down_s, a13, h, o, ws, stream=None):
    check(lib().moe_expert_ffn(ctypes.byref(cfg), _p(x_perm), _p(offsets),
                               _p(tile_expert), _p(stats), _p(w13), _p(w_down),
                               _p(w13_s), _p(w_down_s), _p(a13), _p(h), _p(o),
                               _p(ws), _s(stream)), "moe_expert_ffn")


def moe_expert_ffn_gather(cfg, x, row_slot, offsets, tile_expert, stats, w13, w_down,
                          w13_s, w_down_s, a13, h, o, ws, stream=None):
    check(lib().moe_expert_ffn_gather(ctypes.byref(cfg), _p(x), _p(row_slot), _p(offsets),
                                      _p(tile_expert), _p(stats), _p(w13), _p(w_down),
                                      _p(w13_s), _p(w_down_s), _p(a13), _p(h), _p(o),
                                      _p(ws), _s(stream)), "moe_expert_ffn_gather")


def moe_expert_ffn_combine(cfg, x, x_perm, offsets, slot_row, row_slot, topk_w, tile_expert,
                           stats, w13, w_down, w13_s, w_down_s, a13, h, o, y, ws, stream=None):
    check(lib().moe_expert_ffn_combine(
        ctypes.byref(cfg), _p(x), _p(x_perm), _p(offsets), _p(slot_row), _p(row_slot),
        _p(topk_w), _p(tile_expert), _p(stats), _p(w13), _p(w_down), _p(w13_s), _p(w_down_s),
        _p(a13), _p(h), _p(o), _p(y), _p(ws), _s(stream)), "moe_expert_ffn_combine")


def moe_combine(cfg, o, slot_row, topk_w, offsets, y, stream=None):
    check(lib().moe_combine(ctypes.byref(cfg), _p(o), _p(slot_row), _p(topk_w),
                            _p(offsets), _p(y), _s(stream)), "moe_combine")


def moe_backward(cfg, x, w_r, logits, probs, lse, topk_idx, topk_w, counts,
                 kept, offsets, slot_row, row_slot, tile_expert, stats, x_perm,
                 a13, h, o, w13, w_down, w13_s, w_down_s, dy, dx, dw_r, dw13,
                 dw_down, dw13_s, dw_down_s, dg_out, dlogits_out, ws,
                 stream=None):
    check(lib().moe_backward(
        ctypes.byref(cfg), _p(x), _p(w_r), _p(logits), _p(probs), _p(lse),
        _p(topk_idx), _p(topk_w), _p(counts), _p(kept), _p(offsets),
        _p(slot_row), _p(row_slot), _p(tile_expert), _p(stats), _p(x_perm),
        _p(a13), _p(h), _p(o), _p(w13), _p(w_down), _p(w13_s), _p(w_down_s),
        _p(dy), _p(dx), _p(dw_r), _p(dw13), _p(dw_down), _p(dw13_s),
        _p(dw_down_s), _p(dg_out), _p(dlogits_out), _p(ws), _s(stream)),
        "moe_backward")


def _dtype(name) -> int:
    return C.MOE_BF16 if name in ("bf16", torch.bfloat16) else C.MOE_FP32


def make_norm_config(T, D, *, norm="rms", dtype="bf16", resid=None, eps=1e-5, alpha=1.0,
                     gate_len=0) -> NormConfig:
    """Norm before / after a block (norm: "rms" or "layer"; resid: type of the
    residual stream, that of the activations by default)."""
    kinds = {"rms": C.MOE_RMSNORM, "layer": C.MOE_LAYERNORM}
    if norm not in kinds:
        raise MoEError("norm is 'rms' or 'layer', not %r" % (norm,))
    return NormConfig(T=T, D=D, norm=kinds[norm], dtype=_dtype(dtype),
                      resid=_dtype(dtype if resid is None else resid), gate_len=gate_len,
                      eps=eps, alpha=alpha)


_TYPES = {C.MOE_FP32: torch.float32, C.MOE_BF16: torch.bfloat16}


def moe_block_norm(cfg, r, y, w_post, b_post, gate, w_pre, b_pre, r_out, x, stats,
                   stream=None):
    """r_out = r + alpha gate N(y); x = N(r_out) (y None: x = N(r) alone)."""
    T, D, L, f32 = cfg.T, cfg.D, cfg.gate_len, torch.float32
    n, act, res = T * D, _TYPES[cfg.dtype], _TYPES[cfg.resid]
    check(lib().moe_block_norm(ctypes.byref(cfg), *_args(
        "moe_block_norm", stream, ("r", r, res, n), ("y", y, act, n),
        ("w_post", w_post, f32, D), ("b_post", b_post, f32, D),
        ("gate", gate, f32, -(-T // L) * D if L > 0 else 0), ("w_pre", w_pre, f32, D),
        ("b_pre", b_pre, f32, D), ("r_out", r_out, res, n), ("x", x, act, n),
        ("stats", stats, f32, 4 * T))), "moe_block_norm")


_norm_ws = {}      # workspace bytes by _norm_key, of up to _NORM_WS_MAX configurations
_NORM_WS_MAX = 256


def _norm_key(cfg):
    return cfg.T, cfg.D, cfg.gate_len, cfg.norm, cfg.dtype, cfg.resid


def moe_block_norm_ws_bytes(cfg) -> int:
    """Workspace of moe_block_norm_backward."""
    n = int(lib().moe_block_norm_ws_bytes(ctypes.byref(cfg)))
    if n <= 0:
        check(C.MOE_ERR_ARG, "moe_block_norm_ws_bytes")
    if len(_norm_ws) >= _NORM_WS_MAX:
        _norm_ws.clear()
    _norm_ws[_norm_key(cfg)] = n
    return n


def moe_block_norm_backward(cfg, r_out, y, w_post, b_post, gate, w_pre, stats, dx, dr_out, dy,
                            dr, dw_post, db_post, dgate, dw_pre, db_pre, ws, stream=None):
    T, D, L, f32 = cfg.T, cfg.D, cfg.gate_len, torch.float32
    n, act, res = T * D, _TYPES[cfg.dtype], _TYPES[cfg.resid]
    g = -(-T // L) * D if L > 0 else 0
    need = _norm_ws.get(_norm_key(cfg)) or moe_block_norm_ws_bytes(cfg)
    if ws is not None and ws.numel() < need:
        raise MoEError("moe_block_norm_backward: the workspace is too small")
    check(lib().moe_block_norm_backward(ctypes.byref(cfg), *_args(
        "moe_block_norm_backward", stream, ("r_out", r_out, res, n), ("y", y, act, n),
        ("w_post", w_post, f32, D), ("b_post", b_post, f32, D), ("gate", gate, f32, g),
        ("w_pre", w_pre, f32, D), ("stats", stats, f32, 4 * T), ("dx", dx, act, n),
        ("dr_out", dr_out, res, n), ("dy", dy, act, n), ("dr", dr, res, n),
        ("dw_post", dw_post, f32, D), ("db_post", db_post, f32, D), ("dgate", dgate, f32, g),
        ("dw_pre", dw_pre, f32, D), ("db_pre", db_pre, f32, D),
        ("ws", ws, torch.uint8, 0 if ws is None else ws.numel()))), "moe_block_norm_backward")


def make_adamw_config(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8,
                      weight_decay=0.01) -> AdamwConfig:
    return AdamwConfig(lr=lr, beta1=beta1, beta2=beta2, eps=eps, weight_decay=weight_decay)


class AdamwTable:
    """The tensors of an optimizer step, described once (it keeps them alive)."""

    def __init__(self, array, count, device, tensors):
        self.array, self.count, self.device, self.tensors = array, count, device, tensors


def adamw_table(entries) -> AdamwTable:
    """Describes the tensors of an AdamW step.  Each entry is a mapping with
    `param`, `grad`, `m`, `v` (contiguous CUDA tensors of the same length;
    m and v fp32, or float8_e4m3fn with `m_scale` and `v_scale`, fp32 with
    one element per 256) and, if wanted, `master` (fp32), `lr_mult` (1.0)
    and `decay` (True).  What a step writes overlaps nothing else."""
    types = {torch.float32: C.MOE_FP32, torch.bfloat16: C.MOE_BF16}
    entries = [dict(e) for e in entries]
    arr = (AdamwTensor * max(1, len(entries)))()
    device, ranges = None, []
    for a, e in zip(arr, entries):
        p, m = e["param"], e["m"]
        n, fp8 = p.numel(), m.dtype == torch.float8_e4m3fn
        nb = -(-n // C.MOE_ADAMW_BLOCK)
        scale = (torch.float32, nb) if fp8 else (None, 0)
        state = (m.dtype if fp8 else torch.float32, n)
        wants = {"param": (p.dtype, n), "grad": (e["grad"].dtype, n), "m": state, "v": state,
                 "master": (torch.float32, n), "m_scale": scale, "v_scale": scale}
        for k, (dt, count) in wants.items():
            t = e.get(k)
            if t is None:
                if k == "master" or (k.endswith("_scale") and not fp8):
                    continue
                raise MoEError("adamw_table: %s is missing" % k)
            if k in ("param", "grad") and t.dtype not in types:
                raise MoEError("adamw_table: %s is fp32 or bf16, not %s" % (k, t.dtype))
            if t.dtype != dt or t.numel() != count or not t.is_contiguous() or not t.is_cuda:
                raise MoEError("adamw_table: %s is not a contiguous CUDA tensor of %d x %s"
                               % (k, count, dt))
            device = t.device if device is None else device
            if t.device != device:
                raise MoEError("adamw_table: tensors on %s and %s" % (device, t.device))
            setattr(a, k, t.data_ptr())
            if count:
                ranges.append((t.data_ptr(), t.data_ptr() + count * t.element_size(), k))
        a.n, a.dtype, a.grad_dtype = n, types[p.dtype], types[e["grad"].dtype]
        a.state = C.MOE_STATE_FP8 if fp8 else C.MOE_STATE_FP32
        a.decay, a.lr_mult, a.reserved = int(bool(e.get("decay", True))), e.get("lr_mult", 1.0), 0
    end, written = 0, 0           # of all ranges so far, of the written ones
    for lo, hi, k in sorted(ranges):
        if lo < (written if k == "grad" else end):
            raise MoEError("adamw_table: %s overlaps another tensor of the step" % k)
        end = max(end, hi)
        written = written if k == "grad" else max(written, hi)
    return AdamwTable(arr, len(entries), device, entries)


def moe_adamw(cfg, table, step, lr=None, grad_scale=None, stream=None):
    """One AdamW step over an adamw_table; step: int32 [2] device tensor (the
    count of steps taken, and a word of the kernel's own that starts at 0)."""
    dev = torch._C._cuda_getDevice()
    if table.device is not None and table.device.index != dev:
        raise MoEError("moe_adamw: the tensors are on %s, the current device is cuda:%d"
                       % (table.device, dev))
    *p, s = _args("moe_adamw", stream, ("step", step, torch.int32, 2),
                  ("lr", lr, torch.float32, 1), ("grad_scale", grad_scale, torch.float32, 1))
    check(lib().moe_adamw(ctypes.byref(cfg), table.array, table.count, *p, s), "moe_adamw")


def moe_quant_i8(x, q, scale, stream=None):
    """Rows of x (the last dimension; fp32 or bf16) to 8 bits with a scale
    each.  x may be a row-strided matrix; more dimensions are contiguous."""
    cols = x.shape[-1]
    rows = x.numel() // cols if cols else 0
    if x.dim() == 2 and x.stride(1) == 1:
        ld = x.stride(0) if rows > 1 else cols
    elif x.is_contiguous():
        ld = cols
    else:
        raise MoEError("moe_quant_i8: x is not made of contiguous rows")
    if x.dtype not in (torch.float32, torch.bfloat16):
        raise MoEError("moe_quant_i8: x is fp32 or bf16, not %s" % x.dtype)
    if (q.dtype != torch.int8 or q.shape != x.shape or not q.is_contiguous()
            or scale.dtype != torch.float32 or scale.shape != x.shape[:-1]
            or not scale.is_contiguous()):
        raise MoEError("moe_quant_i8: q is int8 like x, scale fp32 with a value per row")
    pq, ps, s = _args("moe_quant_i8", stream, ("q", q, torch.int8, rows * cols),
                      ("scale", scale, torch.float32, rows))
    if x.get_device() != q.get_device():
        raise MoEError("moe_quant_i8: x is on %s, q on %s" % (x.device, q.device))
    check(lib().moe_quant_i8(x.data_ptr(), _dtype(x.dtype), rows, cols, ld, pq, ps, s),
          "moe_quant_i8")


def moe_expert_ffn_i8_ws_bytes(cfg) -> int:
    """Workspace of moe_expert_ffn_i8."""
    n = int(lib().moe_expert_ffn_i8_ws_bytes(ctypes.byref(cfg)))
    if n <= 0:
        check(C.MOE_ERR_ARG, "moe_expert_ffn_i8_ws_bytes")
    return n


def moe_expert_ffn_i8(cfg, x, offsets, slot_row, row_slot, tile_expert, stats, w13, w13_scale,
                      w_down, w_down_scale, w13_s, w13_s_scale, w_down_s, w_down_s_scale, o, ws,
                      stream=None):
    T, D, K, F = cfg.T, cfg.D, cfg.K, cfg.F
    E = cfg.n_local_experts or cfg.E
    z = moe_get_sizes(cfg)
    R, i32, i8, f32, bf16 = (int(z.rows_max), torch.int32, torch.int8, torch.float32,
                             torch.bfloat16)
    if ws is not None and ws.numel() < moe_expert_ffn_i8_ws_bytes(cfg):
        raise MoEError("moe_expert_ffn_i8: the workspace is too small")
    check(lib().moe_expert_ffn_i8(ctypes.byref(cfg), *_args(
        "moe_expert_ffn_i8", stream, ("x", x, bf16, T * D), ("offsets", offsets, i32, E + 2),
        ("slot_row", slot_row, i32, T * K), ("row_slot", row_slot, i32, R),
        ("tile_expert", tile_expert, i32, int(z.tiles_max)), ("stats", stats, i32, 4),
        ("w13", w13, i8, E * 2 * F * D), ("w13_scale", w13_scale, f32, E * 2 * F),
        ("w_down", w_down, i8, E * D * F), ("w_down_scale", w_down_scale, f32, E * D),
        ("w13_s", w13_s, i8, 2 * F * D), ("w13_s_scale", w13_s_scale, f32, 2 * F),
        ("w_down_s", w_down_s, i8, D * F), ("w_down_s_scale", w_down_s_scale, f32, D),
        ("o", o, bf16, R * D), ("ws", ws, torch.uint8, 0 if ws is None else ws.numel()))),
        "moe_expert_ffn_i8")


def moe_check_status(stream=None) -> int:
    bits = ctypes.c_uint32(0)
    rc = lib().moe_check_status(_s(stream), ctypes.byref(bits))
    if rc == C.MOE_ERR_DEVICE:
        raise MoEError("device error word set: 0x%x" % bits.value)
    check(rc, "moe_check_status")
    return bits.value


def moe_launch_count(reset: bool = False) -> int:
    return int(lib().moe_launch_count(1 if reset else 0))


def moe_set_side_streams(enable: bool) -> bool:
    """Side streams inside moe_backward for this thread; returns the previous setting."""
    return bool(lib().moe_set_side_streams(1 if enable else 0))


class LaunchProfile:
    """Per-launch CUDA-event timing of this thread's library launches."""

    def __init__(self, max_launches: int = 128):
        self.max = max_launches
        check(lib().moe_profile_enable(max_launches), "moe_profile_enable")

    def reset(self):
        lib().moe_profile_reset()

    def read(self):
        """[(kernel name, ms, on_side_stream)] of the launches since reset
        (the caller has synchronised)."""
        buf = (ctypes.c_float * self.max)()
        n = lib().moe_profile_read(buf, self.max)
        if n < 0:
            check(n, "moe_profile_read")
        return [(lib().moe_profile_name(i).decode(), float(buf[i]),
                 lib().moe_profile_side(i) == 1) for i in range(n)]

    def starts(self):
        """Start of each launch since reset, in ms after the first one."""
        buf = (ctypes.c_float * self.max)()
        n = lib().moe_profile_starts(buf, self.max)
        if n < 0:
            check(n, "moe_profile_starts")
        return [float(buf[i]) for i in range(n)]

    def close(self):
        lib().moe_profile_disable()


__all__ = ["LaunchProfile", "MoEError", "MoeConfig", "MoeSizes", "make_config", "config_from",
           "moe_get_sizes", "moe_router", "moe_dispatch", "moe_dispatch_static",
           "moe_aux_loss",
           "moe_expert_ffn", "moe_combine", "moe_backward", "moe_check_status",
           "moe_launch_count", "moe_set_side_streams", "moe_aux_loss_seq",
           "moe_bias_update", "moe_route_expert_choice", "moe_expert_ffn_gather",
           "moe_expert_ffn_combine", "moe_aux_stats", "moe_aux_loss_global",
           "moe_set_backward_streams", "NormConfig", "make_norm_config", "moe_block_norm",
           "moe_block_norm_ws_bytes", "moe_block_norm_backward", "AdamwConfig", "AdamwTable",
           "make_adamw_config", "adamw_table", "moe_adamw", "moe_quant_i8",
           "moe_expert_ffn_i8", "moe_expert_ffn_i8_ws_bytes"]
