"""MoEBlock's checks of its inputs (no GPU needed: the block's buffers are CPU
tensors and the library's calls are left out)."""
from __future__ import annotations

import pytest
import torch

from mixture_experts_routing_fp32_b200 import MoEBlock, MoEError, api

T, D = 8, 128


@pytest.fixture
def block(monkeypatch):
    # CPU tensors stand for the current device's
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: -1, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 0, raising=False)
    called = []
    monkeypatch.setattr(api, "moe_block_norm", lambda *a: called.append("norm"))
    monkeypatch.setattr(api, "moe_block_norm_backward", lambda *a: called.append("back"))
    b = MoEBlock(api.make_config(T, D, 4, 2, 128), device="cpu")
    b.layer.forward = lambda *a, **k: b.layer.y
    b.layer.backward = lambda dy: dy
    b.called = called
    return b


ONE = torch.ones(D)


def rows():
    return torch.zeros(T, D, dtype=torch.bfloat16)


def test_a_block_on_its_own_output_has_no_backward(block):
    """r = r_out and x = x_next are read before they are written, but not what
    the backward pass needs of them."""
    g = rows()
    for kw, r in ((dict(w_pre=ONE), block.r_out), (dict(x=block.r_out), rows()),
                  (dict(x=block.x_next, w_next=ONE), rows())):
        block.forward(r, (), **kw)
        block.called.clear()
        with pytest.raises(MoEError, match="overwrote"):
            block.backward(g, g if "w_next" in kw else None)
        assert not block.called
    # neither is written here, or not needed
    for kw, r in ((dict(x=rows()), block.r_out), (dict(x=block.x_next), rows()),
                  (dict(x=block.x), rows()), (dict(w_pre=ONE), block.x_next),
                  (dict(w_pre=ONE, w_next=ONE), rows())):
        block.forward(r, (), **kw)
        block.backward(g, g if "w_next" in kw else None)


def test_buffers_that_are_written_too_early_are_refused(block):
    for kw, r in ((dict(w_pre=ONE), block.x), (dict(w_pre=ONE), block.layer.y),
                  (dict(x=rows()), block.layer.y), (dict(x=block.layer.y), rows()),
                  (dict(w_pre=ONE, w_next=ONE), block.x_next)):
        with pytest.raises(MoEError, match="shares memory"):
            block.forward(r, (), **kw)
    whole = torch.zeros(T + 1, D, dtype=torch.bfloat16)
    block.r_out = whole[:T]
    with pytest.raises(MoEError, match="a part of"):
        block.forward(whole[1:], (), w_pre=ONE)
    assert not block.called


def test_a_forward_that_fails_half_way_leaves_no_forward(block, monkeypatch):
    """Its first launches have rewritten what the forward before it left."""
    block.forward(rows(), (), w_pre=ONE)

    def refuse(*a, **k):
        raise MoEError("refused")

    for at in ("layer", "post"):
        with monkeypatch.context() as m:
            if at == "layer":
                m.setattr(block.layer, "forward", refuse)
            else:
                m.setattr(api, "moe_block_norm", lambda nc, *a: nc is block.post and refuse())
            with pytest.raises(MoEError, match="refused"):
                block.forward(rows(), (), w_pre=ONE)
        with pytest.raises(MoEError, match="no forward"):
            block.backward(rows())
        block.forward(rows(), (), w_pre=ONE)
        block.backward(rows())


@pytest.mark.parametrize("bad", [
    torch.zeros(T - 1, D, dtype=torch.bfloat16), torch.zeros(T, D),
    torch.zeros(D, T, dtype=torch.bfloat16).t(), torch.zeros(T, D, dtype=torch.float16),
])
def test_inputs_that_do_not_fit_are_refused_before_the_layer_runs(block, bad):
    """x goes to the layer, which would read a shorter one past its end."""
    block.layer.forward = lambda *a, **k: block.called.append("layer")
    for name, r, kw in (("x", rows(), dict(x=bad)), ("r", bad, dict(x=rows())),
                        ("r", bad, dict(w_pre=ONE))):
        with pytest.raises(MoEError, match=name + " is not"):
            block.forward(r, (), **kw)
    assert not block.called


def test_a_missing_input_is_refused_by_name(block):
    from mixture_experts_routing_fp32_b200 import MoEInt8Layer
    for kw in (dict(w_pre=ONE), dict(x=rows())):
        with pytest.raises(MoEError, match="no r"):
            block.forward(None, (), **kw)
    layer = MoEInt8Layer(api.make_config(T, D, 4, 2, 128), device="cpu")
    layer.weights = ()
    for call in (lambda: layer.forward(None, torch.zeros(4, D)),
                 lambda: layer.experts(None, None, None)):
        with pytest.raises(MoEError, match="no x"):
            call()
