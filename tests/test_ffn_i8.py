"""The 8-bit experts' host-side refusals (no GPU needed: the addresses below
are never read)."""
from __future__ import annotations

import ctypes

import pytest
import torch

from mixture_experts_routing_fp32_b200 import _lib as C
from mixture_experts_routing_fp32_b200 import api
from mixture_experts_routing_fp32_b200.build import build

A = 4096


@pytest.fixture(scope="module")
def lib():
    build()
    return C.lib()


GOOD = dict(T=5, D=128, E=4, K=2, F=256)


@pytest.mark.parametrize("bad", [
    dict(D=136), dict(F=200), dict(dtype="fp32"), dict(gemm_impl=1), dict(K=5), dict(T=0),
    dict(D=128 * 513), dict(F=128 * 513),
    dict(expert_choice=1, K=4, capacity_factor=1.0, renorm=0),
])
def test_layers_it_cannot_serve_are_refused(lib, bad):
    cfg = api.make_config(**{**GOOD, **bad})
    with pytest.raises(C.MoEError):
        api.moe_expert_ffn_i8_ws_bytes(cfg)
    with pytest.raises(C.MoEError):
        from mixture_experts_routing_fp32_b200 import MoEInt8Layer
        MoEInt8Layer(cfg, device="cpu")
    assert lib.moe_expert_ffn_i8(ctypes.byref(cfg), *([A] * 16), None) == C.MOE_ERR_ARG


@pytest.mark.parametrize("at,value", [(i, None) for i in (0, 1, 2, 3, 4, 5, 6, 7, 8, 9, 14, 15)]
                         + [(0, A + 8), (6, A + 8), (7, A + 4), (8, A + 1), (14, A + 8),
                            (15, A + 16)])
def test_bad_pointers_are_refused(lib, at, value):
    cfg = api.make_config(**GOOD)
    args = [A] * 10 + [None] * 4 + [A, A]
    args[at] = value
    assert lib.moe_expert_ffn_i8(ctypes.byref(cfg), *args, None) == C.MOE_ERR_ARG


def test_a_shared_expert_needs_its_weights(lib):
    cfg = api.make_config(**GOOD, n_shared=1)
    assert lib.moe_expert_ffn_i8(ctypes.byref(cfg), *([A] * 10 + [None] * 4 + [A, A]),
                                 None) == C.MOE_ERR_ARG


@pytest.mark.parametrize("bad", [
    dict(x=None), dict(q=None), dict(scale=None), dict(dtype=2), dict(rows=-1), dict(cols=0),
    dict(cols=12), dict(cols=65544, ld=65544), dict(ld=56), dict(ld=68), dict(x=A + 8),
    dict(q=A + 4), dict(scale=A + 2),
])
def test_bad_quantisations_are_refused(lib, bad):
    a = dict(x=A, dtype=1, rows=3, cols=64, ld=64, q=A, scale=A)
    a.update(bad)
    assert lib.moe_quant_i8(a["x"], a["dtype"], a["rows"], a["cols"], a["ld"], a["q"], a["scale"],
                            None) == C.MOE_ERR_ARG


def test_no_rows_is_no_work(lib):
    assert lib.moe_quant_i8(None, 1, 0, 64, 64, None, None, None) == C.MOE_OK


def test_tensors_of_other_shapes_are_refused():
    x = torch.zeros(4, 64)
    q, s = torch.zeros(4, 64, dtype=torch.int8), torch.zeros(4)
    for args in ((x, q[:3], s), (x, q, s[:3]), (x, q.float(), s), (x.double(), q, s),
                 (x.t(), q.t(), torch.zeros(64))):
        with pytest.raises(C.MoEError):
            api.moe_quant_i8(*args)


def test_rows_are_aligned_for_pairs_sooner(lib):
    """MOE_GEMM_I8: segments of 256 rows from 512 rows per expert on (1536
    otherwise); other values of gemm_impl are refused."""
    for T, impl, align in ((2048, C.MOE_GEMM_I8, 256), (2047, C.MOE_GEMM_I8, 128),
                           (2048, C.MOE_GEMM_AUTO, 128), (6144, C.MOE_GEMM_AUTO, 256)):
        cfg = api.make_config(T, 128, 8, 2, 128, gemm_impl=impl)
        assert api.moe_get_sizes(cfg).row_align == align, (T, impl)
    with pytest.raises(C.MoEError):
        api.moe_get_sizes(api.make_config(64, 128, 8, 2, 128, gemm_impl=3))


def test_blocks_refuse_shards_and_unknown_types():
    from mixture_experts_routing_fp32_b200 import MoEBlock
    shard = api.make_config(64, 128, 8, 2, 128, expert_base=0, n_local_experts=4)
    with pytest.raises(C.MoEError, match="shards"):
        MoEBlock(shard, device="cpu")
    with pytest.raises(C.MoEError, match="resid"):
        MoEBlock(api.make_config(64, 128, 8, 2, 128), resid="fp8", device="cpu")


@pytest.mark.parametrize("bad", [
    dict(x=(4, 128)), dict(x=torch.zeros(5, 128)), dict(w_r=(3, 128)),
    dict(w_r=torch.zeros(4, 128, dtype=torch.bfloat16)), dict(w_r=torch.zeros(128, 4).t()),
    dict(logit_offset=(3,)), dict(sel_bias=(5, 4)), dict(sel_bias=torch.zeros(4).double()),
    dict(sentinel_mask=torch.zeros(5, 2)), dict(sentinel_mask=torch.zeros(4, 2, dtype=torch.uint8)),
])
def test_a_layer_checks_its_inputs_before_the_router_runs(monkeypatch, bad):
    """The router takes its sizes from the configuration: a batch of fewer
    tokens would be read past its end.  (CPU tensors stand for the current
    device's here, and nothing is launched.)"""
    from mixture_experts_routing_fp32_b200 import MoEInt8Layer
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: -1, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    ran = []
    monkeypatch.setattr(api, "moe_router", lambda *a: ran.append("router"))
    layer = MoEInt8Layer(api.make_config(**GOOD), device="cpu")
    monkeypatch.setattr(layer, "experts", lambda *a: ran.append("experts"))
    good = dict(x=torch.zeros(5, 128, dtype=torch.bfloat16), w_r=torch.zeros(4, 128))
    with pytest.raises(C.MoEError, match="no weights"):
        layer.forward(**good)
    layer.weights = ()
    with pytest.raises(C.MoEError, match=next(iter(bad)) + " is not"):
        layer.forward(**{**good, **{k: torch.zeros(v, dtype=good.get(k, good["w_r"]).dtype)
                                    if isinstance(v, tuple) else v for k, v in bad.items()}})
    assert not ran
    layer.forward(**good, sel_bias=torch.zeros(4), logit_offset=torch.zeros(4),
                  sentinel_mask=torch.zeros(5, 2, dtype=torch.uint8))
    assert ran == ["router", "experts"]
