"""The experts in 8-bit integers on the GPU against their definition in float64.

Tolerances, U = 2^-24.  The integer sums are exact; a and b then take 4
roundings.  The sigmoid uses the fast exponential, within 2^-21 + |a| 2^-23
relative, so for |a| < 40 h is within 128 U of its own value and its row
maximum too.  A value of h whose quotient lies that close to a tie (127 * 256 U
of a step) may round to either side: one step of s(h) in that column of the
second product, which the tests add up exactly.  Otherwise o is 8 U off and
rounded to bf16 (2^-8 of the value); the combine adds K values in fp32 and
rounds once more, each term off by what its o is off times its weight.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mixture_experts_routing_fp32_b200.build import build
    build()


# ---------------------------------------------------------------------------
# row quantisation
# ---------------------------------------------------------------------------
def check_rows(x, q, s, exact_ties):
    """q and s of finite rows against the definition."""
    v = x.double()
    big = v.abs().amax(-1, keepdim=True)
    at = torch.where(big > 0, 127.0 * v / big.clamp_min(1e-300), torch.zeros_like(v))
    want = torch.round(at)
    # fp32: 127 v and the quotient are rounded, so a quotient within
    # 127 * 2 U of a tie may go either way
    near = ((at - at.floor()) - 0.5).abs() < (0.0 if exact_ties else 127 * 4 * U)
    off = (q.double() - want).abs()
    assert bool(((off == 0) | (near & (off == 1))).all())
    assert bool(((s.double() - big[..., 0] / 127.0).abs() <= U * big[..., 0] / 127.0
                 + 1.5e-45).all())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,cols", [(1, 8), (3, 64), (5, 2048), (7, 2056), (300, 1032),
                                       (2, 8192), (3, 8200), (2, 65536), (2500, 128)])
def test_rows(rows, cols, dtype):
    import mixture_experts_routing_fp32_b200 as moe
    g = torch.Generator("cuda").manual_seed(rows * cols)
    x = torch.randn(rows, cols, generator=g, device="cuda", dtype=torch.float32).to(dtype)
    q = torch.empty(rows, cols, dtype=torch.int8, device="cuda")
    s = torch.full((rows + 2,), 7.0, device="cuda")
    moe.moe_quant_i8(x, q, s[:rows])
    check_rows(x, q, s[:rows], dtype == torch.bfloat16)
    assert s[rows:].tolist() == [7.0, 7.0]
    # rows inside a wider matrix
    wide = torch.full((rows, cols + 24), 1e9, device="cuda").to(dtype)
    wide[:, 8:cols + 8] = x
    if (wide[:, 8:].data_ptr() & 15) == 0:
        q2, s2 = torch.empty_like(q), torch.empty(rows, device="cuda")
        moe.moe_quant_i8(wide[:, 8:cols + 8], q2, s2)
        assert torch.equal(q, q2) and torch.equal(s[:rows], s2)


def test_ties_extremes_and_non_finite_rows():
    import mixture_experts_routing_fp32_b200 as moe
    x = torch.zeros(12, 64, dtype=torch.float32)
    x[0, :4] = torch.tensor([2.0, 1.0, -1.0, 0.5])            # 63.5: a tie, to even 64
    x[1, :3] = torch.tensor([254.0, 1.0, 3.0])                # 0.5 -> 0, 1.5 -> 2
    x[3, 5], x[3, 6] = 3.3e38, -1.6e38                        # 127 v would overflow
    x[4, 5], x[4, 6] = 1e-38, 4e-39
    x[5, 5] = float("nan")
    x[6, 5] = float("inf")
    x[7, 5], x[7, 6] = float("-inf"), float("nan")
    x[8] = -1.0
    x[9, 63] = 1e-45
    for dt in (torch.float32, torch.bfloat16):
        v = x.to(dt).cuda()
        q = torch.empty(12, 64, dtype=torch.int8, device="cuda")
        s = torch.empty(12, device="cuda")
        moe.moe_quant_i8(v, q, s)
        ok = [0, 1, 2, 3, 4, 8, 10, 11]
        check_rows(v[ok], q[ok], s[ok], True)
        assert q[0, :4].tolist() == [127, 64, -64, 32] and q[1, :3].tolist() == [127, 0, 2]
        assert bool(s[[5, 6, 7]].isnan().all()) and bool((q[[5, 6, 7]] == 0).all())
        assert bool((q[8] == -127).all())


# ---------------------------------------------------------------------------
# experts
# ---------------------------------------------------------------------------
def quantise(v):
    big = v.abs().amax(1, keepdim=True)
    at = 127.0 * v / big.clamp_min(1e-300)
    return at, big / 127.0


def expert(x, w13, s13, wd, sd):
    """(o, how far an output may be from it); the integer sums are exact here
    too (a sum that cancels is a zero on both sides)"""
    at, s = quantise(x)
    a = torch.round(at) @ w13.double().T * s * s13.double()
    g, u = a.chunk(2, 1)
    assert float(g.abs().max()) < 40.0
    h = g / (1 + torch.exp(-g)) * u
    at, s = quantise(h)
    near = ((at - at.floor()) - 0.5).abs() < 127 * 256 * U
    o = torch.round(at) @ wd.double().T * s * sd.double()
    # 16 U: the scales, the conversion of the sum; 128 U: s(h) itself
    tol = near.double() @ wd.double().abs().T * s * sd.double() + 160 * U * o.abs()
    return o, tol + 2.0 ** -8 * o.abs()


class Case:
    def __init__(self, T, D, E, K, F, shared=False, holes=0.0, seed=0, hot=0.0, **cfg):
        import mixture_experts_routing_fp32_b200 as moe
        g = torch.Generator("cuda").manual_seed(seed)
        self.T, self.E, self.K, self.shared = T, E, K, shared
        self.x = torch.randn(T, D, generator=g, device="cuda").to(torch.bfloat16)
        score = torch.randn(T, E, generator=g, device="cuda")
        score[:, 0] += hot
        top = score.topk(K, 1)
        self.idx, self.w = top.indices.to(torch.int32), torch.softmax(top.values, 1)
        if holes:
            self.idx[torch.rand(T, K, generator=g, device="cuda") < holes] = -1

        def weight(*shape):
            q = torch.randint(-127, 128, shape, generator=g, device="cuda", dtype=torch.int8)
            s = torch.rand(shape[:-1], generator=g, device="cuda") + 0.5
            return q, s / (73.0 * shape[-1] ** 0.5)

        self.cfg = moe.make_config(T, D, E, K, F, n_shared=int(shared), **cfg)
        n = cfg.get("n_local_experts", 0) or E
        self.base = cfg.get("expert_base", 0)
        self.n = n
        self.w13, self.wd = weight(n, 2 * F, D), weight(n, D, F)
        self.w13s, self.wds = (weight(2 * F, D), weight(D, F)) if shared else ((None, None),) * 2
        self.layer = moe.MoEInt8Layer(self.cfg)
        self.layer.set_weights(*self.w13, *self.wd, *self.w13s, *self.wds)

    def run(self):
        y = self.layer.experts(self.x, self.idx, self.w)
        import mixture_experts_routing_fp32_b200 as moe
        assert moe.moe_check_status() == 0
        return y

    def check(self, y):
        x = self.x.double()
        ref, tol = torch.zeros_like(x), torch.zeros_like(x)
        kept = self.layer.slot_row.reshape(self.T, self.K) >= 0
        for e in range(self.n):
            tok, slot = torch.nonzero((self.idx == e + self.base) & kept, as_tuple=True)
            if not tok.numel():
                continue
            o, t = expert(x[tok], self.w13[0][e], self.w13[1][e], self.wd[0][e], self.wd[1][e])
            w = self.w.double()[tok, slot][:, None]
            ref.index_add_(0, tok, o * w)
            tol.index_add_(0, tok, t * w + 4 * U * (o * w).abs())
        if self.shared:
            o, t = expert(x, *self.w13s, *self.wds)
            ref, tol = ref + o, tol + t
        tol = tol * (1 + 2.0 ** -7) + 2.0 ** -8 * ref.abs()
        err = (y.double() - ref).abs()
        assert bool(torch.isfinite(y.float()).all())
        assert bool((err <= tol).all()), "error %g, %g above its tolerance" % (
            float(err.max()), float((err - tol).max()))
        # and on the whole no worse than its roundings: 2^-8 of each o and
        # of y, evenly spread, is below 2^-8 in the 2-norm; the near ties add
        # what the tolerances say at most
        assert float(err.norm()) <= 2.0 ** -8 * 2 * float(ref.norm()) + float(
            (tol - 2.0 ** -7 * 1.02 * ref.abs()).clamp_min(0).norm())


CASES = [
    dict(T=1, D=128, E=4, K=1, F=128), dict(T=1, D=256, E=64, K=8, F=128, shared=True),
    dict(T=3, D=384, E=8, K=2, F=640), dict(T=16, D=512, E=8, K=2, F=1792),
    dict(T=37, D=128, E=5, K=3, F=384, shared=True, holes=0.3),
    # few rows per expert: 16, 32 and 64 columns of tokens, turns (one expert
    # picked by all 150 tokens), an odd number of k blocks, the shared expert
    dict(T=7, D=384, E=16, K=2, F=128, shared=True), dict(T=29, D=640, E=16, K=4, F=384, shared=True),
    dict(T=60, D=256, E=32, K=4, F=640, holes=0.2), dict(T=150, D=384, E=64, K=2, F=256, hot=9.0),
    dict(T=32, D=128, E=64, K=8, F=128, hot=9.0, capacity_factor=2.0),
    dict(T=130, D=256, E=4, K=4, F=256, hot=3.0),                 # select all
    dict(T=333, D=1024, E=32, K=4, F=512, shared=True, holes=0.1),
    dict(T=400, D=256, E=16, K=6, F=128, capacity_factor=0.7),    # drops
    dict(T=2500, D=1280, E=8, K=4, F=640),                        # 256-wide single tiles
    dict(T=4100, D=256, E=2, K=1, F=256),                         # CTA pairs
    dict(T=3300, D=384, E=4, K=2, F=384, shared=True, hot=1.0),   # pairs, 128-wide down
    dict(T=300, D=2560, E=4, K=2, F=128),                         # wide rows
    dict(T=65, D=8320, E=2, K=1, F=128),                          # rows read twice
    dict(T=200, D=256, E=16, K=4, F=256, expert_base=4, n_local_experts=8),
]


@pytest.mark.parametrize("kw", CASES, ids=lambda k: "-".join("%s" % v for v in k.values()))
def test_experts(kw):
    case = Case(**kw)
    y = case.run().clone()
    case.check(y)
    # the same bits again, whatever the workspaces hold
    case.layer.ws_i8.fill_(255)
    case.layer.o.fill_(float("nan"))
    assert torch.equal(case.run(), y)


def test_tokens_without_experts_and_bad_tokens():
    case = Case(40, 256, 8, 2, 128, seed=3)
    case.idx[7] = -1
    y = case.run().clone()
    case.check(y)
    assert bool((y[7] == 0).all())
    for bad in (float("nan"), float("inf")):
        case.x[11, 3] = bad
        z = case.run()
        keep = [i for i in range(40) if i != 11]
        assert torch.equal(z[keep], y[keep]) and bool(z[11].isnan().all())
    case.x[11] = 0.0
    assert bool((case.run()[11] == 0).all())
    case.idx.fill_(-1)
    assert bool((case.run() == 0).all())


def test_graphs_streams_and_two_layers_at_once():
    a, b = Case(64, 512, 8, 2, 256, seed=4), Case(48, 256, 16, 4, 384, seed=5, shared=True)
    want = [c.run().clone() for c in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs = []
    for c, s in zip((a, b), streams):
        with torch.cuda.stream(s):
            c.layer.experts(c.x, c.idx, c.w)
            s.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                c.layer.experts(c.x, c.idx, c.w)
            graphs.append(g)
    for _ in range(5):
        for c in (a, b):
            c.layer.y.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for c, w in zip((a, b), want):
            assert torch.equal(c.layer.y, w)
    new = Case(64, 512, 8, 2, 256, seed=6)
    ref = new.run().clone()
    for k in ("x", "idx", "w"):
        getattr(a, k).copy_(getattr(new, k))
    for i in range(2):
        a.w13[i].copy_(new.w13[i])
        a.wd[i].copy_(new.wd[i])
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(a.layer.y, ref)


def test_a_block_served_in_8_bits():
    """Norm, 8-bit layer (weights quantised from a layer's own), norm and
    residual sum: near the bf16 layer's block, on the same picks."""
    import mixture_experts_routing_fp32_b200 as moe
    import workloads as W
    cfg = W.REDUCED["ds3"]
    inp = {n: W.make_input(cfg, n, "cuda") for n in ("x", "w_r", "w13", "w_down", "w13_s",
                                                     "w_down_s", "sel_bias")}
    mc = moe.config_from(cfg)
    full, small = moe.MoELayer(mc), moe.MoEInt8Layer(mc)
    small.quantize(inp["w13"], inp["w_down"], inp["w13_s"], inp["w_down_s"])
    T, D = cfg.T, cfg.D
    nc = moe.make_norm_config(T, D, norm="rms")
    w = torch.ones(D, device="cuda")
    h = torch.empty_like(inp["x"])
    moe.moe_block_norm(nc, inp["x"], None, None, None, None, w, None, None, h, None)
    bias = inp["sel_bias"].float()
    ya = full.forward(h, inp["w_r"], inp["w13"], inp["w_down"], inp["w13_s"], inp["w_down_s"],
                      sel_bias=bias)
    yb = small.forward(h, inp["w_r"], sel_bias=bias)
    assert torch.equal(full.topk_idx, small.topk_idx) and torch.equal(full.topk_w, small.topk_w)
    outs = []
    for y in (ya, yb):
        r_out, x2 = torch.empty_like(h), torch.empty_like(h)
        moe.moe_block_norm(nc, inp["x"], y, w, None, None, w, None, r_out, x2, None)
        outs.append(r_out.double() - inp["x"].double())
    moe.moe_check_status()
    a, b = outs
    # one step of 8 bits is 1 / 127 of a row's largest value, about 4 spreads:
    # x, h and both weights are each off by 4 / 127 / sqrt(12) = 0.9% of
    # their spread (h, a product of two, by up to three times that): under 5%
    assert float((a - b).norm() / a.norm()) < 0.05


@pytest.mark.parametrize("T", [1, 200])
@pytest.mark.parametrize("c", [61, 15])
def test_h_is_quantised_as_rows_are(T, c):
    """q(h) is moe_quant_i8's, ties included.  The layer is built so that h is
    known exactly: gates of 128 (whose sigmoid is 1 in fp32) times integers,
    h = 128 (2 k + 1) c beside a largest value of 128 * 254 c, so that every
    quotient 127 h / max = k + 1/2 is a tie, and the outputs read q(h) back:
    one weight of 1 per output, a scale of 1 / s(h)."""
    import mixture_experts_routing_fp32_b200 as moe
    D = F = 128
    k = torch.randperm(127, generator=torch.Generator().manual_seed(c)).double()
    b = torch.cat([torch.tensor([254.0 * c], dtype=torch.float64), (2 * k + 1) * c])
    b[1::2] *= -1
    x = torch.zeros(T, D, dtype=torch.bfloat16, device="cuda")
    x[:, 0], x[:, 1] = 127.0, 1.0                     # s(x) = 1, q(x) = x
    w13 = torch.zeros(2, 2 * F, D, dtype=torch.int8)
    w13[:, :F, :2] = 1                                # a = 128
    hi = torch.round(b / 127)
    w13[:, F:, 0], w13[:, F:, 1] = hi.to(torch.int8), (b - 127 * hi).to(torch.int8)
    wd = torch.eye(F, dtype=torch.int8).repeat(2, 1, 1)
    layer = moe.MoEInt8Layer(moe.make_config(T, D, 2, 1, F))
    layer.set_weights(w13.cuda(), torch.ones(2, 2 * F, device="cuda"), wd.cuda(),
                      torch.full((2, D), 1.0 / (256.0 * c), device="cuda"))
    idx = (torch.arange(T, device="cuda", dtype=torch.int32) % 2)[:, None].contiguous()
    y = layer.experts(x, idx, torch.ones(T, 1, device="cuda"))
    h = (128.0 * b).float().cuda()[None].contiguous()
    q, s = torch.empty(1, F, dtype=torch.int8, device="cuda"), torch.empty(1, device="cuda")
    moe.moe_quant_i8(h, q, s)
    want = torch.round(127.0 * b / (254.0 * c))       # ties to even
    assert torch.equal(q[0].double().cpu(), want) and float(s) == 256.0 * c
    assert torch.equal(y, q.to(torch.bfloat16).expand(T, F))


@pytest.mark.parametrize("kw", [CASES[4], CASES[7], CASES[11], CASES[15]],
                         ids=lambda k: "%d-%d" % (k["T"], k["D"]))
def test_rows_are_rounded_once_and_sums_once(kw):
    """Of the roundings to bf16 there are two: each row of o, and y, the fp32
    sum of the rows as they are stored (K + 1 products and sums)."""
    case = Case(**kw)
    y = case.run().double()
    rows = case.layer.slot_row.reshape(case.T, case.K).long()
    o = case.layer.o.double()
    x = case.x.double()
    total, size = torch.zeros_like(x), torch.zeros_like(x)
    for e in range(case.n):
        tok, slot = torch.nonzero((case.idx == e + case.base) & (rows >= 0), as_tuple=True)
        if not tok.numel():
            continue
        ref, tol = expert(x[tok], case.w13[0][e], case.w13[1][e], case.wd[0][e], case.wd[1][e])
        got = o[rows[tok, slot]]
        assert bool(((got - ref).abs() <= tol * (1 + 2.0 ** -7)).all())
        part = got * case.w.double()[tok, slot][:, None]
        total.index_add_(0, tok, part)
        size.index_add_(0, tok, part.abs())
    if case.shared:
        at = int(case.layer.offsets[case.n])
        got = o[at:at + case.T]
        ref, tol = expert(x, *case.w13s, *case.wds)
        assert bool(((got - ref).abs() <= tol * (1 + 2.0 ** -7)).all())
        total, size = total + got, size + got.abs()
    tol = 2.0 ** -8 * total.abs() + 2 * (case.K + 1) * U * size
    assert bool(((y - total).abs() <= tol).all())


@pytest.mark.parametrize("T,E", [(1, 64), (16, 64), (16, 4), (300, 8)])
def test_an_expert_picked_twice_by_a_token(T, E):
    """Picks need not differ: the token's rows are computed and added twice
    (more rows of an expert than tokens, in turns where rows are few)."""
    case = Case(T, 256, E, 4, 128, seed=T)
    case.idx[:, 1] = case.idx[:, 0]
    case.idx[:, 3] = case.idx[:, 0]
    case.check(case.run())
    case.idx[:] = 1
    case.check(case.run())
