"""The norms around a block: host-side refusals, the workspace's size and the
reference's own gradients (against differences).  No GPU needed."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest

from mixture_experts_routing_fp32_b200 import _lib as C
from mixture_experts_routing_fp32_b200 import api
from mixture_experts_routing_fp32_b200.build import build
from tests import norm_ref as R


@pytest.fixture(scope="module")
def lib():
    build()
    return C.lib()


GOOD = dict(T=4, D=64, norm="rms", dtype="bf16", gate_len=0)
A, B = ctypes.c_void_p(4096), ctypes.c_void_p(4104)     # aligned / misaligned, never read


@pytest.mark.parametrize("bad", [
    dict(T=0), dict(D=0), dict(D=12), dict(D=8200), dict(gate_len=-1), dict(eps=0.0),
    dict(eps=float("nan")), dict(alpha=float("nan")), dict(dtype="fp32", resid="bf16"),
])
def test_bad_configs_are_refused(lib, bad):
    nc = api.make_norm_config(**{**GOOD, **bad})
    with pytest.raises(C.MoEError):
        api.moe_block_norm_ws_bytes(nc)
    args = [A, A, None, None, None, A, None, A, A, None, None]
    assert lib.moe_block_norm(ctypes.byref(nc), *args) == C.MOE_ERR_ARG


def test_unknown_norm_is_refused():
    with pytest.raises(C.MoEError):
        api.make_norm_config(4, 64, norm="batch")


# r, y, w_post, b_post, gate, w_pre, b_pre, r_out, x, stats
@pytest.mark.parametrize("args", [
    [None, A, None, None, None, A, None, A, A, None],      # no r
    [A, None, None, None, None, None, None, None, None, None],   # nothing to do
    [A, None, A, None, None, A, None, None, A, None],      # w_post without y
    [A, None, None, None, None, A, None, A, A, None],      # r_out without y
    [A, A, None, None, None, A, None, None, A, None],      # y without r_out
    [A, A, None, A, None, A, None, A, A, None],            # b_post without w_post
    [A, A, None, None, A, A, None, A, A, None],            # gate with gate_len = 0
    [A, A, None, None, None, None, A, A, None, None],      # b_pre without w_pre
    [A, A, None, None, None, A, None, A, None, None],      # w_pre without x
    [A, A, None, None, None, None, None, A, A, None],      # x without w_pre
    [B, A, None, None, None, A, None, A, A, None],         # misaligned
    [A, A, None, None, None, B, None, A, A, None],
    [A, A, None, None, None, A, None, A, A, B],
])
def test_bad_forward_arguments_are_refused(lib, args):
    nc = api.make_norm_config(**GOOD)
    assert lib.moe_block_norm(ctypes.byref(nc), *args, None) == C.MOE_ERR_ARG


# r_out, y, w_post, b_post, gate, w_pre, stats, dx, dr_out, dy, dr,
# dw_post, db_post, dgate, dw_pre, db_pre, ws
@pytest.mark.parametrize("change", [
    {0: None}, {6: None}, {10: None}, {16: None},     # r_out, stats, dr, ws
    {1: None}, {9: None},                             # y without dy, dy without y
    {5: None}, {7: None},                             # w_pre without dx, dx without w_pre
    {1: None, 9: None},                               # w_post without y
    {3: A, 2: None, 11: None}, {2: None},             # b_post / dw_post without w_post
    {13: A}, {4: A},                                  # dgate, gate without gate_len
    {0: B}, {8: B}, {9: B}, {16: B},
])
def test_bad_backward_arguments_are_refused(lib, change):
    nc = api.make_norm_config(**GOOD)
    args = [A, A, A, None, None, A, A, A, A, A, A, A, None, None, A, None, A]
    for k, v in change.items():
        args[k] = v
    assert lib.moe_block_norm_backward(ctypes.byref(nc), *args, None) == C.MOE_ERR_ARG


def test_workspace_grows_with_gate_rows(lib):
    one = api.moe_block_norm_ws_bytes(api.make_norm_config(512, 256, gate_len=512))
    many = api.moe_block_norm_ws_bytes(api.make_norm_config(512, 256, gate_len=100))
    assert many == 2 * one > 0


def test_workspaces_of_other_norms_and_types_are_not_mixed_up(lib):
    """Norm, type and shape each have their say in the workspace: one that
    fits one configuration is refused for another that needs more."""
    import torch
    kinds = [("rms", "bf16"), ("layer", "bf16"), ("layer", "fp32")]
    for D in (2048, 2816, 4096):
        configs = [api.make_norm_config(16384, D, norm=n, dtype=d) for n, d in kinds]
        sizes = [api.moe_block_norm_ws_bytes(c) for c in configs]
        for c, size in zip(configs, sizes):
            ws = torch.empty(size - 1, dtype=torch.uint8)
            with pytest.raises(C.MoEError, match="workspace"):
                api.moe_block_norm_backward(c, *[None] * 16, ws)
    assert len(set(sizes)) > 1


@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("post,gate_len,y", [(True, 2, True), (False, 0, True), (True, 5, False)])
def test_reference_gradients_against_differences(norm, post, gate_len, y):
    """The 64-bit reference that the GPU tests use: each gradient against
    central differences of <x, dx> + <r_out, dr_out> (step 1e-5: truncation
    and rounding both stay below 1e-8 of values of order one)."""
    rng = np.random.default_rng(3)
    c = dict(T=5, D=8, norm=norm, eps=1e-5, alpha=0.7, gate_len=gate_len if y else 0)
    p = R.draw_inputs(rng, c, post=post, bias=True, y=y)
    dx, dr_out = rng.normal(size=(5, 8)), rng.normal(size=(5, 8))

    def value(q):
        out = R.forward(c, **q)
        return (out["x"] * dx).sum() + ((out["r_out"] * dr_out).sum() if y
                                        else (q["r"] * dr_out).sum())

    f = R.forward(c, **p)
    grads = R.backward(c, p, f["r_out"] if y else p["r"], dx, dr_out)
    names = {"r": "dr", "y": "dy", "w_post": "dw_post", "b_post": "db_post", "gate": "dgate",
             "w_pre": "dw_pre", "b_pre": "db_pre"}
    for k, name in names.items():
        if p[k] is None:
            continue
        for i in range(p[k].size):
            e = np.zeros_like(p[k])
            e.flat[i] = 1e-5
            d = (value({**p, k: p[k] + e}) - value({**p, k: p[k] - e})) / 2e-5
            assert abs(d - grads[name].flat[i]) < 1e-6 * max(1.0, abs(d)), (k, i)


def test_workspace_sizes_of_many_configurations_are_not_all_kept(lib):
    """A batch of another length each step does not make the table grow."""
    api._norm_ws.clear()
    sizes = {}
    for T in range(1, 1500):
        sizes[T] = api.moe_block_norm_ws_bytes(api.make_norm_config(T, 64, gate_len=7))
        assert len(api._norm_ws) <= 256
    for T in (1, 700, 1499):
        nc = api.make_norm_config(T, 64, gate_len=7)
        assert api.moe_block_norm_ws_bytes(nc) == sizes[T] == api._norm_ws[api._norm_key(nc)]
