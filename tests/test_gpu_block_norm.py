"""The block norms on the GPU against their formulas in float64.

Tolerances.  A stored value is off by half a step of its type (eps / 2
relative).  Before that the fp32 arithmetic of a value takes fewer than 16
roundings of 2^-24 each, and the sums over a row add at most 8 values in
sequence and then join 10 levels, so every intermediate is within 32 * 2^-24
of the sum of its terms' magnitudes; 64 * 2^-24 of the row's largest term
covers the value and its statistics together.  Column sums add up to 1003
tokens: at most 4 rows in sequence per block and row group here, then up to
10 partials and 5 levels, 32 * 2^-24 of the terms' magnitudes, plus what the
terms are off themselves (the same 64 * 2^-24).
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

from tests import norm_ref as R

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
GUARD = 7.0


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mixture_experts_routing_fp32_b200.build import build
    build()


def half_step(t):
    return torch.finfo(t).eps / 2


def up(a, dtype=torch.float32):
    return None if a is None else torch.tensor(a, dtype=torch.float64).to(dtype).cuda()


def down(t):
    return None if t is None else t.double().cpu().numpy()


def guarded(shape, dtype):
    """A tensor with two guard rows behind its last one."""
    full = torch.full((shape[0] + 2, *shape[1:]), GUARD, dtype=dtype, device="cuda")
    return full[:shape[0]], full[shape[0]:]


def close(got, ref, tol, what):
    err = np.abs(down(got) - ref)
    worst = (err - tol).max()
    assert np.isfinite(err).all() and worst <= 0, "%s: %g above the tolerance (error %g)" % (
        what, worst, err.max())


class Case:
    def __init__(self, T, D, norm="rms", dtype="bf16", resid=None, gate_len=0, post=True,
                 bias=False, y=True, alpha=0.7, seed=0, inputs=None):
        self.c = dict(T=T, D=D, norm=norm, eps=1e-5, alpha=alpha, gate_len=gate_len)
        self.ta, self.tr = DT[dtype], DT[resid or dtype]
        rng = np.random.default_rng(seed + 1000 * T + D)
        p = R.draw_inputs(rng, self.c, post, bias, y)
        p.update(inputs or {})
        self.t = {k: up(v, {"r": self.tr, "y": self.ta}.get(k, torch.float32)) for k, v in p.items()}
        self.p = {k: down(v) for k, v in self.t.items()}
        self.dx, self.dr_out = up(rng.normal(size=(T, D)), self.ta), up(rng.normal(size=(T, D)),
                                                                      self.tr)
        from mixture_experts_routing_fp32_b200 import make_norm_config
        self.nc = make_norm_config(T, D, norm=norm, dtype=dtype, resid=resid, eps=1e-5,
                                   alpha=alpha, gate_len=gate_len)

    def forward(self, in_place=False, pre=True):
        from mixture_experts_routing_fp32_b200 import moe_block_norm
        t, T, D = self.t, self.c["T"], self.c["D"]
        x, gx = guarded((T, D), self.ta)
        stats, gs = guarded((T, 4), torch.float32)
        r_out = g_r = None
        r = t["r"]
        if t["y"] is not None:
            r_out, g_r = guarded((T, D), self.tr)
            if in_place:
                r_out.copy_(r)
                r = r_out
        moe_block_norm(self.nc, r, t["y"], t["w_post"], t["b_post"], t["gate"],
                       t["w_pre"] if pre else None, t["b_pre"] if pre else None, r_out,
                       x if pre else None, stats)
        torch.cuda.synchronize()
        for g in (gx, gs, g_r):
            assert g is None or bool((g == GUARD).all())
        return r_out, x if pre else None, stats

    def check_forward(self, r_out, x):
        stream = None if r_out is None else down(r_out)
        p = dict(self.p)
        if x is None:
            p["w_pre"] = p["b_pre"] = None
        ref = R.forward(self.c, **p, stream=stream)
        if r_out is not None:
            big = np.abs(self.p["r"]) + np.abs(ref["r_out"] - self.p["r"]).max(1, keepdims=True)
            close(r_out, ref["r_out"],
                  half_step(self.tr) * np.abs(ref["r_out"]) + 64 * U * big, "r_out")
        if x is not None:
            big = np.abs(ref["x"]).max(1, keepdims=True)
            v = self.p["r"] if stream is None else stream
            # a mean far above the spread: the centred values carry the
            # mean's rounding
            m, s = R.moments(self.c, v)
            big = big + np.abs(m) * s * np.abs(p["w_pre"]).max()
            close(x, ref["x"], half_step(self.ta) * np.abs(ref["x"]) + 64 * U * big, "x")

    def backward(self, r_out, stats, in_place=False, dr_out=True, only=None, ws=None):
        import mixture_experts_routing_fp32_b200 as moe
        t, T, D = self.t, self.c["T"], self.c["D"]
        new = lambda k: None if t[k] is None or (only and k not in only) else torch.full_like(  # noqa: E731
            t[k], GUARD)
        o = {"dw_post": new("w_post"), "db_post": new("b_post"), "dgate": new("gate"),
             "dw_pre": new("w_pre"), "db_pre": new("b_pre")}
        o["dr"], g1 = guarded((T, D), self.tr)
        o["dy"], g2 = guarded((T, D), self.ta) if t["y"] is not None else (None, None)
        src = self.dr_out if dr_out else None
        if in_place:
            o["dr"].copy_(src)
            src = o["dr"]
        if ws is None:
            ws = torch.full((moe.moe_block_norm_ws_bytes(self.nc),), 255, dtype=torch.uint8,
                            device="cuda")
        moe.moe_block_norm_backward(
            self.nc, r_out if r_out is not None else t["r"], t["y"], t["w_post"], t["b_post"],
            t["gate"], t["w_pre"], stats, self.dx, src, o["dy"], o["dr"], o["dw_post"],
            o["db_post"], o["dgate"], o["dw_pre"], o["db_pre"], ws)
        torch.cuda.synchronize()
        for g in (g1, g2):
            assert g is None or bool((g == GUARD).all())
        return o

    def check_backward(self, r_out, o, dr_out=True):
        v = self.p["r"] if r_out is None else down(r_out)
        ref = R.backward(self.c, self.p, v, down(self.dx), down(self.dr_out) if dr_out else None)
        m, s = R.moments(self.c, v)
        # rows: the largest term of the row
        u = np.abs(down(self.dx) * self.p["w_pre"]).max(1, keepdims=True) * s
        rh = np.abs((v - m) * s).max(1, keepdims=True)
        big = (np.abs(down(self.dr_out)).max(1, keepdims=True) if dr_out else 0) + u * (1 + rh)
        close(o["dr"], ref["dr"], half_step(self.tr) * np.abs(ref["dr"]) + 64 * U * big, "dr")
        if o["dy"] is not None:
            yh, _, sy = R.post(self.c, self.p["y"], self.p["w_post"], self.p["b_post"])
            scale = self.c["alpha"] * np.abs(R.gate_rows(self.c, self.p["gate"])) * np.ones_like(v)
            if self.p["w_post"] is not None:
                scale = scale * np.abs(self.p["w_post"]) * sy * (
                    1 + np.abs(yh).max(1, keepdims=True))
            bigy = scale.max(1, keepdims=True) * big
            close(o["dy"], ref["dy"], half_step(self.ta) * np.abs(ref["dy"]) + 64 * U * bigy, "dy")
        n_in = {"dw_post": None, "db_post": None, "dgate": None, "dw_pre": None, "db_pre": None}
        for k in n_in:
            if o[k] is None:
                continue
            # the terms' own errors: d carries 64 U of the row's largest term
            loose = 1.0
            if k in ("dw_post", "db_post", "dgate"):
                loose += float((big / np.abs(ref["dr"]).mean(1, keepdims=True)).max())
            mean_abs = ref["abs_" + k]
            close(o[k], ref[k], 96 * U * loose * (mean_abs + mean_abs.mean()), k)


CASES = [
    dict(T=1, D=8), dict(T=1, D=7168, gate_len=1), dict(T=2, D=64, norm="layer", bias=True),
    dict(T=3, D=200, dtype="fp32", norm="layer", gate_len=1, bias=True),
    dict(T=37, D=256, gate_len=37), dict(T=300, D=768, norm="layer", bias=True, gate_len=7),
    dict(T=300, D=768, resid="fp32", gate_len=100), dict(T=299, D=1032, dtype="fp32", post=False),
    dict(T=1003, D=264, dtype="fp32", norm="layer", gate_len=100, bias=True),
    dict(T=1003, D=2048, resid="fp32", norm="layer", gate_len=50, bias=True),
    dict(T=613, D=40, gate_len=300, bias=True), dict(T=401, D=4096, gate_len=401, norm="layer"),
    dict(T=160, D=7168, gate_len=3, bias=True), dict(T=155, D=8192, dtype="fp32", gate_len=60,
                                                     norm="layer", bias=True),
    dict(T=150, D=8192, dtype="fp32"), dict(T=64, D=520, post=False, gate_len=9),
    dict(T=2, D=4096, gate_len=2, norm="layer", bias=True), dict(T=16, D=256, bias=True),
    dict(T=17, D=256, gate_len=17, bias=True), dict(T=8, D=264, y=False, bias=True),
    dict(T=10, D=768, resid="fp32", gate_len=10), dict(T=31, D=64, post=False, gate_len=40),
    dict(T=129, D=512, y=False), dict(T=70, D=1536, y=False, norm="layer", bias=True,
                                      dtype="fp32"),
]


@pytest.mark.parametrize("kw", CASES, ids=lambda k: "-".join("%s" % v for v in k.values()))
def test_forward_and_backward(kw):
    case = Case(**kw)
    r_out, x, stats = case.forward()
    case.check_forward(r_out, x)
    case.check_backward(r_out, case.backward(r_out, stats))


@pytest.mark.parametrize("kw", [CASES[5], CASES[9], CASES[13]], ids=lambda k: str(k["D"]))
def test_in_place_repeated_and_partial_calls(kw):
    """r_out over r and dr over dr_out give the same bits, and so does a
    second call on a workspace with anything in it; gradients that are not
    asked for do not change the others."""
    case = Case(**kw)
    r_out, x, stats = case.forward()
    for a, b in zip((r_out, x, stats), case.forward(in_place=True)):
        assert torch.equal(a, b)
    o = case.backward(r_out, stats)
    for again in (case.backward(r_out, stats, in_place=True), case.backward(r_out, stats)):
        for k in o:
            assert o[k] is None or torch.equal(o[k], again[k]), k
    some = case.backward(r_out, stats, only=("w_pre",))
    for k in ("dr", "dy", "dw_pre"):
        assert torch.equal(o[k], some[k]), k
    none = case.backward(r_out, stats, dr_out=False)
    case.check_backward(r_out, none, dr_out=False)
    alone, _, _ = case.forward(pre=False)
    assert torch.equal(alone, r_out)


def test_zero_rows_large_means_and_nan_rows():
    """A row of zeros normalises to zeros; a mean of 1000 spreads costs no
    more digits than the mean itself carries; a NaN stays in its row."""
    T, D = 9, 776
    rng = np.random.default_rng(5)
    y = rng.normal(1000.0, 1.0, size=(T, D))
    r = rng.normal(0.0, 1.0, size=(T, D))
    y[3] = 0.0
    r[3] = 0.0
    case = Case(T, D, norm="layer", dtype="fp32", inputs={"y": y, "r": r}, post=False)
    r_out, x, _ = case.forward()
    case.check_forward(r_out, x)
    assert bool((x[3] == 0).all())
    y[5, 17] = np.nan
    bad = Case(T, D, norm="layer", dtype="fp32", inputs={"y": y, "r": r}, post=False)
    r2, x2, _ = bad.forward()
    keep = [i for i in range(T) if i != 5]
    assert torch.equal(x2[keep], x[keep]) and bool(x2[5].isnan().all())


def test_graphs_and_streams():
    """Forward and backward captured once, replayed on new inputs, on a
    stream other than the one that made the tensors."""
    case = Case(300, 768, norm="layer", bias=True, gate_len=70)
    import mixture_experts_routing_fp32_b200 as moe
    t = case.t
    T, D = 300, 768
    e = lambda like: torch.empty_like(like)  # noqa: E731
    r_out, x, stats = e(t["r"]), e(t["y"]), torch.empty(T, 4, device="cuda")
    o = {k: e(t[v]) for k, v in (("dw_post", "w_post"), ("db_post", "b_post"), ("dgate", "gate"),
                                 ("dw_pre", "w_pre"), ("db_pre", "b_pre"), ("dy", "y"),
                                 ("dr", "r"))}
    ws = torch.empty(moe.moe_block_norm_ws_bytes(case.nc), dtype=torch.uint8, device="cuda")

    def step():
        moe.moe_block_norm(case.nc, t["r"], t["y"], t["w_post"], t["b_post"], t["gate"],
                           t["w_pre"], t["b_pre"], r_out, x, stats)
        moe.moe_block_norm_backward(case.nc, r_out, t["y"], t["w_post"], t["b_post"], t["gate"],
                                    t["w_pre"], stats, case.dx, case.dr_out, o["dy"], o["dr"],
                                    o["dw_post"], o["db_post"], o["dgate"], o["dw_pre"],
                                    o["db_pre"], ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step()
    other = Case(300, 768, norm="layer", bias=True, gate_len=70, seed=9)
    for k in t:
        t[k].copy_(other.t[k])
    case.dx.copy_(other.dx)
    case.dr_out.copy_(other.dr_out)
    graph.replay()
    torch.cuda.synchronize()
    want_r, want_x, want_s = other.forward()
    want = other.backward(want_r, want_s)
    assert torch.equal(r_out, want_r) and torch.equal(x, want_x)
    for k in o:
        assert torch.equal(o[k], want[k]), k

# Each register budget of the general backward, one to three CTAs an SM.  Up
# to 7 rows in sequence per block here: 7 roundings, 10 partials and 5 levels
# stay below the 32 that the column sums' tolerance counts.
@pytest.mark.parametrize("kw", [
    dict(T=900, D=2048, norm="layer", bias=True), dict(T=900, D=2304, norm="layer", gate_len=30),
    dict(T=1000, D=2312, bias=True), dict(T=900, D=6152, norm="layer", gate_len=1000),
    dict(T=500, D=6152, norm="layer", bias=True, resid="fp32", gate_len=9),
    dict(T=500, D=6152, norm="layer", bias=True, dtype="fp32"),
    dict(T=300, D=7176, norm="layer", bias=True), dict(T=1000, D=1000, dtype="fp32", bias=True),
    dict(T=2000, D=72, norm="layer", bias=True, gate_len=4),
], ids=lambda k: "-".join("%s" % v for v in k.values()))
def test_the_backwards_block_shapes(kw):
    case = Case(**kw)
    r_out, x, stats = case.forward()
    case.check_forward(r_out, x)
    case.check_backward(r_out, case.backward(r_out, stats))


@pytest.mark.parametrize("D", [264, 4096])
def test_rows_aligned_to_16_bytes_only(D):
    """Tensors that start 16 bytes behind a 32-byte boundary: the same bits."""
    import mixture_experts_routing_fp32_b200 as moe
    T = 67
    case = Case(T, D, dtype="fp32", gate_len=T)
    t = case.t

    def step(off):
        def at(like):
            flat = torch.full((like.numel() + 8,), GUARD, device="cuda")
            view = flat[off:off + like.numel()].view_as(like)
            assert view.data_ptr() % 32 == (16 if off == 4 else 0)
            return view, flat

        (r_out, f0), (x, f1), (dy, f2), (dr, f3) = (at(t[k]) for k in ("r", "y", "y", "r"))
        y, _ = at(t["y"])
        y.copy_(t["y"])
        stats = torch.empty(T, 4, device="cuda")
        moe.moe_block_norm(case.nc, t["r"], y, t["w_post"], None, t["gate"], t["w_pre"], None,
                           r_out, x, stats)
        ws = torch.empty(moe.moe_block_norm_ws_bytes(case.nc), dtype=torch.uint8, device="cuda")
        moe.moe_block_norm_backward(case.nc, r_out, y, t["w_post"], None, t["gate"], t["w_pre"],
                                    stats, case.dx, case.dr_out, dy, dr, None, None, None, None,
                                    None, ws)
        torch.cuda.synchronize()
        for f in (f0, f1, f2, f3):
            assert bool((f[:off] == GUARD).all()) and bool((f[off + T * D:] == GUARD).all())
        return r_out, x, dy, dr

    for a, b in zip(step(0), step(4)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype,resid", [("fp32", "fp32"), ("bf16", "fp32"), ("bf16", "bf16")])
@pytest.mark.parametrize("D", [264, 768, 4096, 7168])
def test_layer_norm_of_rows_with_a_large_mean(D, dtype, resid):
    """Rows of integers whose sum is exact in fp32 (below 2^24) and divides
    by D: their mean is exact, and so are the values behind it.  A constant
    row normalises to zeros, exactly, so that x = b_pre, r_out = r + alpha
    gate b_post and the products with the normalised row vanish.  Rows of
    c +- 1 (as many of each) have variance 1: rstd is within 5 U (1 / D, the
    sum with eps, its root within 2 units), the value then takes two products
    and a sum: 16 U of |rstd w| + |b| covers it, whatever the mean is."""
    import mixture_experts_routing_fp32_b200 as moe
    big = 128.0 if dtype == "bf16" else 1000.0           # c +- 1 is a bf16 value
    rows = np.array([[big, big], [-big, -big], [big + 1, big - 1], [-big - 1, 1 - big],
                     [3.0, 3.0], [1.0, -1.0]])
    y = np.tile(rows, (1, D // 2))
    const, T = np.array([0, 1, 4]), len(rows)
    case = Case(T, D, norm="layer", dtype=dtype, resid=resid, gate_len=2, bias=True,
                inputs={"y": y, "r": y})
    t, p, a = case.t, case.p, case.c["alpha"]
    mean = y.mean(1, keepdims=True)
    rstd = 1.0 / np.sqrt(y.var(1, keepdims=True) + 1e-5)
    hat = (y - mean) * rstd
    # x = N(r) alone
    x, stats = torch.empty_like(t["y"]), torch.empty(T, 4, device="cuda")
    nc = moe.make_norm_config(T, D, norm="layer", dtype=dtype, resid=resid, eps=1e-5)
    moe.moe_block_norm(nc, t["r"], None, None, None, None, t["w_pre"], t["b_pre"], None, x, stats)
    assert np.array_equal(down(stats[:, 2]), mean[:, 0])
    assert torch.equal(x[const], t["b_pre"].to(x.dtype).expand(3, D))
    ref = hat * p["w_pre"] + p["b_pre"]
    terms = 16 * U * (rstd * np.abs(p["w_pre"]) + np.abs(p["b_pre"]))
    terms[const] = 0.0
    close(x, ref, half_step(x.dtype) * np.abs(ref) * (1 + 2.0 ** -7) + terms, "x")
    # the norm behind a block (alpha gate rounds once more, the sum with r too)
    r_out, _, st = case.forward(pre=False)
    assert np.array_equal(down(st[:, 0]), mean[:, 0])
    e = a * R.gate_rows(case.c, p["gate"])
    ref = p["r"] + e * (hat * p["w_post"] + p["b_post"])
    spread = np.where(np.isin(np.arange(T), const)[:, None], 0.0, rstd)
    terms = 16 * U * np.abs(e) * (spread * np.abs(p["w_post"]) + np.abs(p["b_post"]))
    close(r_out, ref, (half_step(r_out.dtype) * (1 + 2.0 ** -7) + 2 * U) * np.abs(ref)
          + 2 * U * np.abs(p["r"]) + terms, "r_out")
    # constant rows alone: nothing but the biases' gradients has a column sum
    keep = torch.tensor(const, device="cuda")
    few = moe.make_norm_config(3, D, norm="layer", dtype=dtype, resid=resid, eps=1e-5, alpha=a)
    o = {k: torch.full((D,), GUARD, device="cuda") for k in ("dw_post", "db_post", "dw_pre",
                                                             "db_pre")}
    dy, dr = torch.empty_like(t["y"][:3]), torch.empty_like(t["r"][:3])
    stats = torch.cat([stats[keep][:, 2:]] * 2, 1)
    dx, dr_out = case.dx[:3].contiguous(), case.dr_out[:3].contiguous()
    ws = torch.empty(moe.moe_block_norm_ws_bytes(few), dtype=torch.uint8, device="cuda")
    moe.moe_block_norm_backward(few, t["r"][keep], t["y"][keep], t["w_post"], t["b_post"], None,
                                t["w_pre"], stats, dx, dr_out, dy, dr, o["dw_post"],
                                o["db_post"], None, o["dw_pre"], o["db_pre"], ws)
    assert not o["dw_pre"].any() and not o["dw_post"].any()
    u = down(dx) * p["w_pre"]
    s = 1e-5 ** -0.5
    d = down(dr_out) + s * (u - u.mean(1, keepdims=True))
    big_d = np.abs(down(dr_out)).max(1, keepdims=True) + 2 * s * np.abs(u).max(1, keepdims=True)
    close(dr, d, half_step(dr.dtype) * np.abs(d) * (1 + 2.0 ** -7) + 64 * U * big_d, "dr")
    dz = a * d * p["w_post"]
    ref = s * (dz - dz.mean(1, keepdims=True))
    big_y = s * a * np.abs(p["w_post"]).max() * 2 * big_d
    close(dy, ref, half_step(dy.dtype) * np.abs(ref) * (1 + 2.0 ** -7) + 64 * U * big_y, "dy")
