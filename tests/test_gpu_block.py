"""Two blocks in a row (MoEBlock): norms, layers, gates and residual sums,
forward and backward, against the norms' float64 formulas around the layers'
own outputs and gradients (which their own tests check), then an optimizer
step over both blocks' weights.

Tolerances: every bf16 tensor is rounded once on the way out of the kernel
that writes it (2^-8 of a value at most, so less in the 2-norm), with fp32
arithmetic before; the first block's dr is rounded twice (after the norm
behind the layer, after the one before it).  fp32 column sums of at most 300
tokens: 96 * 2^-24 of the terms' magnitudes, which their cancellation leaves
at most a hundred times the sum.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

import workloads as W
from tests import norm_ref as R
from tests.test_gpu_block_norm import down, up

pytestmark = pytest.mark.gpu
HALF = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mixture_experts_routing_fp32_b200.build import build
    build()


def near(got, ref, tol, what):
    got = down(got)
    rel = np.linalg.norm(got - ref) / np.linalg.norm(ref)
    assert np.isfinite(got).all() and rel <= tol, (what, rel)


@pytest.mark.parametrize("norm,resid,gate_len", [("rms", "bf16", 0), ("layer", "fp32", 100)])
def test_two_blocks(norm, resid, gate_len):
    import mixture_experts_routing_fp32_b200 as moe
    cfg = W.REDUCED["olmoe"].replace(T=300, sentinel_frac=0.0)
    T, D = cfg.T, cfg.D
    rng = np.random.default_rng(2)
    c = dict(T=T, D=D, norm=norm, eps=1e-5, alpha=0.5, gate_len=gate_len)
    bias = norm == "layer"
    w = [W.make_input(cfg, n, "cuda") for n in ("w_r", "w13", "w_down")]
    blocks = [moe.MoEBlock(moe.config_from(cfg), norm=norm, alpha=0.5, gate_len=gate_len,
                           resid=resid) for _ in range(2)]
    vec = lambda mean: up(rng.normal(mean, 0.2, size=D))  # noqa: E731
    r0 = up(rng.normal(0, 2, size=(T, D)), torch.bfloat16 if resid == "bf16" else torch.float32)
    dr2 = up(rng.normal(size=(T, D)), r0.dtype)
    gate = up(rng.normal(0.5, 0.5, size=(-(-T // gate_len), D))) if gate_len else None
    pre, nxt, post = vec(1), vec(1), [vec(1), vec(1)]
    b_pre, b_nxt, b_post = (vec(0), vec(0), vec(0)) if bias else (None,) * 3

    r1, x1 = blocks[0].forward(r0, w, w_pre=pre, b_pre=b_pre, w_post=post[0], b_post=b_post,
                               gate=gate, w_next=nxt, b_next=b_nxt)
    r2, x2 = blocks[1].forward(r1, w, x=x1, w_post=post[1], gate=gate)
    assert x2 is None
    d = [down(t) if t is not None else None for t in (r0, r1, r2, pre, nxt, gate, b_pre, b_nxt,
                                                      b_post)]
    r0n, r1n, r2n, pren, nxtn, gaten, b_pren, b_nxtn, b_postn = d
    none = dict(y=None, w_post=None, b_post=None, gate=None)
    near(blocks[0].x, R.forward(c, r=r0n, w_pre=pren, b_pre=b_pren, **none)["x"], HALF, "x0")
    y = [down(b.layer.y) for b in blocks]
    p0 = dict(r=r0n, y=y[0], w_post=down(post[0]), b_post=b_postn, gate=gaten, w_pre=nxtn,
              b_pre=b_nxtn)
    f = R.forward(c, **p0, stream=r1n)
    near(r1, f["r_out"], HALF, "r1")
    near(x1, f["x"], HALF, "x1")
    p1 = dict(r=r1n, y=y[1], w_post=down(post[1]), b_post=None, gate=gaten, w_pre=None, b_pre=None)
    near(r2, R.forward(c, **p1)["r_out"], HALF, "r2")

    dr1, dx1 = blocks[1].backward(dr2)
    g1 = R.backward(c, p1, r2n, None, down(dr2))
    near(dr1, g1["dr"], HALF, "dr1")
    near(blocks[1].dy, g1["dy"], HALF, "dy1")
    near(blocks[1].dw_post, g1["dw_post"], 1e-4, "dw_post1")
    assert dx1 is blocks[1].layer.dx
    dr0, dx0 = blocks[0].backward(dr1, dx1)
    assert dx0 is None
    g0 = R.backward(c, p0, r1n, down(dx1), down(dr1))
    near(blocks[0].dy, g0["dy"], HALF, "dy0")
    near(blocks[0].dw_post, g0["dw_post"], 1e-4, "dw_post0")
    near(blocks[0].dw_next, g0["dw_pre"], 1e-4, "dw_next")
    if gate_len:
        near(blocks[0].dgate, g0["dgate"], 1e-4, "dgate0")
        near(blocks[1].dgate, g1["dgate"], 1e-4, "dgate1")
    if bias:
        near(blocks[0].db_next, g0["db_pre"], 1e-4, "db_next")
        near(blocks[0].db_post, g0["db_post"], 1e-4, "db_post")
    gp = R.backward(c, dict(r=r0n, y=None, w_post=None, b_post=None, gate=None, w_pre=pren,
                            b_pre=b_pren), r0n, down(blocks[0].layer.dx), g0["dr"])
    near(dr0, gp["dr"], 2 * HALF, "dr0")
    near(blocks[0].dw_pre, gp["dw_pre"], 1e-4, "dw_pre")
    assert moe.moe_check_status() == 0

    # one optimizer step over the first block's weights, expert weights with
    # fp32 masters: every parameter changes, by at most a little over lr
    lay = blocks[0].layer
    params = [pre, nxt, post[0], *w]
    grads = [blocks[0].dw_pre, blocks[0].dw_next, blocks[0].dw_post, lay.dw_r, lay.dw13, lay.dw_down]
    before = [t.float().clone() for t in params]
    opt = moe.MoEAdamW(params, grads, lr=1e-3, weight_decay=0.0, masters=True)
    opt.step()
    for e, b in zip(opt.entries, before):
        moved = (e.get("master", e["param"]).float() - b).abs()
        assert float(moved.max()) <= 1.001e-3 and float(moved.max()) > 0.5e-3


def test_blocks_refuse_what_does_not_fit():
    import mixture_experts_routing_fp32_b200 as moe
    cfg = W.REDUCED["mm_b"].replace(T=64)
    block = moe.MoEBlock(moe.config_from(cfg))
    r = torch.zeros(64, cfg.D, dtype=torch.bfloat16, device="cuda")
    one = torch.ones(cfg.D, device="cuda")
    w = [W.make_input(cfg, n, "cuda") for n in ("w_r", "w13", "w_down")]
    with pytest.raises(moe.MoEError, match="no forward"):
        block.backward(r)
    with pytest.raises(moe.MoEError, match="either"):
        block.forward(r, w)
    with pytest.raises(moe.MoEError, match="either"):
        block.forward(r, w, w_pre=one, x=r)
    with pytest.raises(moe.MoEError, match="gate"):
        block.forward(r, w, w_pre=one, gate=one)
    for bad in (r.float(), r[:32], r.t(), r.cpu(), torch.zeros(64, 2 * cfg.D, device="cuda",
                                                              dtype=torch.bfloat16)[:, ::2]):
        with pytest.raises(moe.MoEError, match="r is not"):
            block.forward(bad, w, w_pre=one)
    block.forward(r, w, w_pre=one)
    with pytest.raises(moe.MoEError, match="dx_next"):
        block.backward(r, r)


def test_a_block_applied_to_its_own_output():
    """The outputs of a block that reads its own r_out and x_next are those of
    copies; its backward, whose inputs are gone, is refused."""
    import mixture_experts_routing_fp32_b200 as moe
    cfg = W.REDUCED["mm_b"].replace(T=64)
    block = moe.MoEBlock(moe.config_from(cfg), alpha=0.5)
    g = torch.Generator("cuda").manual_seed(1)
    r = torch.randn(64, cfg.D, generator=g, device="cuda").to(torch.bfloat16)
    one = torch.ones(cfg.D, device="cuda")
    w = [W.make_input(cfg, n, "cuda") for n in ("w_r", "w13", "w_down")]
    first = [t.clone() for t in block.forward(r, w, w_pre=one, w_post=one, w_next=one)]
    want = [t.clone() for t in block.forward(first[0].clone(), w, x=first[1].clone(), w_post=one,
                                             w_next=one)]
    again = [t.clone() for t in block.forward(first[0].clone(), w, w_pre=one, w_post=one)[:1]]
    block.forward(r, w, w_pre=one, w_post=one, w_next=one)
    got = block.forward(block.r_out, w, x=block.x_next, w_post=one, w_next=one)
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    with pytest.raises(moe.MoEError, match="overwrote"):
        block.backward(r, r)
    block.forward(r, w, w_pre=one, w_post=one)
    got = block.forward(block.r_out, w, w_pre=one, w_post=one)[0]
    assert torch.equal(got, again[0])
    with pytest.raises(moe.MoEError, match="overwrote"):
        block.backward(r)
    assert moe.moe_check_status() == 0


def test_a_block_and_its_served_form_in_graphs():
    """Forward and backward of a block, and the 8-bit layer with its router,
    captured once and replayed on other inputs: the bits of eager calls."""
    import mixture_experts_routing_fp32_b200 as moe
    cfg = W.REDUCED["olmoe"].replace(T=300, sentinel_frac=0.0)
    T, D = cfg.T, cfg.D
    w = [W.make_input(cfg, n, "cuda") for n in ("w_r", "w13", "w_down")]
    g = torch.Generator("cuda").manual_seed(3)
    rand = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    vec = {k: 1 + 0.2 * rand(D) for k in ("w_pre", "w_post", "w_next")}
    vec.update(b_pre=rand(D), b_post=rand(D), b_next=rand(D), gate=rand(-(-T // 70), D))
    rows = lambda: rand(T, D).to(torch.bfloat16)  # noqa: E731
    r, dr, dx = rows(), rows(), rows()
    block = moe.MoEBlock(moe.config_from(cfg), norm="layer", alpha=0.5, gate_len=70)
    served = moe.MoEInt8Layer(moe.config_from(cfg))
    served.quantize(w[1], w[2])

    def step():
        block.forward(r, w, **vec)
        block.backward(dr, dx)
        served.forward(block.x, w[0])

    def results():
        b = block
        return [t.clone() for t in (
            b.r_out, b.x_next, b.dr, b.dy, b.dw_pre, b.db_pre, b.dw_post, b.db_post, b.dw_next,
            b.db_next, b.dgate, b.layer.dw_r, b.layer.dw13, b.layer.dw_down, served.y)]

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step()
    for t in (r, dr, dx):
        t.copy_(rows())
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    got = results()
    step()
    torch.cuda.synchronize()
    for a, b in zip(got, results()):
        assert bool(torch.isfinite(a.float()).all()) and torch.equal(a, b)
    assert moe.moe_check_status() == 0
