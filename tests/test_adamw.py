"""The AdamW step's host-side refusals (no GPU needed: the addresses below are
never read)."""
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


def call(lib, cfg=None, step=A, lr=None, scale=None, count=1, **fields):
    cfg = api.make_adamw_config() if cfg is None else cfg
    t = dict(param=A, grad=A, m=A, v=A, n=64, dtype=C.MOE_FP32, grad_dtype=C.MOE_FP32,
             state=C.MOE_STATE_FP32, decay=1, lr_mult=1.0)
    t.update(fields)
    arr = (C.AdamwTensor * 1)()
    for k, v in t.items():
        setattr(arr[0], k, v)
    return lib.moe_adamw(ctypes.byref(cfg), arr, count, step, lr, scale, None)


def test_struct_layout_matches_header():
    assert ctypes.sizeof(C.AdamwConfig) == 40 and ctypes.sizeof(C.AdamwTensor) == 88
    assert ctypes.sizeof(C.NormConfig) == 32


@pytest.mark.parametrize("bad", [
    dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=1.0), dict(beta2=float("nan")), dict(eps=0.0),
    dict(eps=1e-39), dict(eps=2e-38, beta1=0.9),
    dict(lr=float("inf")), dict(weight_decay=float("nan")),
])
def test_bad_hyper_parameters_are_refused(lib, bad):
    assert call(lib, cfg=api.make_adamw_config(**bad)) == C.MOE_ERR_ARG


@pytest.mark.parametrize("bad", [
    dict(param=None), dict(grad=None), dict(m=None), dict(v=None), dict(n=-1), dict(n=1 << 41),
    dict(dtype=2), dict(grad_dtype=-1), dict(state=2), dict(decay=2), dict(reserved=1),
    dict(lr_mult=float("nan")),
    dict(master=A),                                   # fp32 parameters are their own master
    dict(m_scale=A), dict(v_scale=A),                 # scales of 32-bit states
    dict(state=1), dict(state=1, m_scale=A),          # 8-bit states without scales
    dict(param=A + 2), dict(grad=A + 1), dict(m=A + 2), dict(v=A + 2),
    dict(dtype=1, param=A + 1), dict(dtype=1, master=A + 2),
    dict(state=1, m_scale=A + 2, v_scale=A),
])
def test_bad_tensors_are_refused(lib, bad):
    assert call(lib, **bad) == C.MOE_ERR_ARG


def test_bad_calls_are_refused(lib):
    assert call(lib, step=None) == C.MOE_ERR_ARG
    assert call(lib, step=A + 2) == C.MOE_ERR_ARG
    assert call(lib, lr=A + 1) == C.MOE_ERR_ARG
    assert call(lib, scale=A + 1) == C.MOE_ERR_ARG
    assert call(lib, count=-1) == C.MOE_ERR_ARG
    cfg = api.make_adamw_config()
    assert lib.moe_adamw(ctypes.byref(cfg), None, 1, A, None, None, None) == C.MOE_ERR_ARG


def test_tables_refuse_what_a_step_cannot_take():
    f = torch.zeros(8)
    with pytest.raises(C.MoEError, match="CUDA"):
        api.adamw_table([{"param": f, "grad": f, "m": f, "v": f}])
    from mixture_experts_routing_fp32_b200 import MoEAdamW
    with pytest.raises(C.MoEError):
        MoEAdamW([f], [f, f])
    with pytest.raises(C.MoEError):
        MoEAdamW([f], [f], state="int4")



@pytest.fixture
def no_gpu_table(monkeypatch):
    """MoEAdamW on CPU tensors: the table is not described to the library."""
    monkeypatch.setattr(api, "adamw_table", lambda entries: api.AdamwTable(
        None, len(entries), torch.device("cpu"), entries))


@pytest.mark.parametrize("given", [(1, 3), [3, 1, 1], {1, 3}, "generator"])
def test_parameters_without_decay(no_gpu_table, given):
    """no_decay may be any iterable, one that can be read only once too."""
    from mixture_experts_routing_fp32_b200 import MoEAdamW
    p = [torch.zeros(4) for _ in range(5)]
    opt = MoEAdamW(p, p, no_decay=(i for i in (1, 3)) if given == "generator" else given)
    assert [e["decay"] for e in opt.entries] == [True, False, True, False, True]


@pytest.mark.parametrize("bad", [(-1,), (5,), (0, 7), ("w",), (1.5,)])
def test_no_decay_of_parameters_that_are_not_there_is_refused(no_gpu_table, bad):
    from mixture_experts_routing_fp32_b200 import MoEAdamW
    p = [torch.zeros(4) for _ in range(5)]
    with pytest.raises(C.MoEError, match="no_decay"):
        MoEAdamW(p, p, no_decay=bad)
