"""The AdamW step on the GPU against its formulas in float64.

Tolerances, with U = 2^-24: g, m' and v' take at most 4 roundings each of
terms whose magnitudes are summed below.  The update m'/c1 / (sqrt(v'/c2) +
eps) takes 3 + 3 of those, the corrections c1, c2 (t ln b rounded twice, expm1
and rsqrt within 2 units each) and 5 operations: 32 U covers it; the sum with
p rounds twice more.  Stored in bf16, half a step (2^-8 of the value) on top.
8-bit states: half a step of e4m3 is 2^-4 of the value, and 2^-10 of the
block's scale where it is subnormal (a whole step, 2^-9, where a positive root
is lifted to the smallest positive value); the scale itself carries 8 U.
"""
from __future__ import annotations

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HP = dict(lr=1e-2, beta1=0.9, beta2=0.99, eps=1e-6, weight_decay=0.1)
BLOCK = 256


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mixture_experts_routing_fp32_b200.build import build
    build()


def down(t):
    return t.double().cpu().numpy().reshape(-1)


def within(got, ref, tol, what):
    err = np.abs(down(got) - ref)
    assert np.isfinite(err).all() and (err <= tol).all(), "%s: error %g, %g above" % (
        what, err.max(), (err - tol).max())


def make(rng, n, dtype="fp32", grad="fp32", state="fp32", master=False, offset=0, fresh=False,
         **more):
    """One tensor's entry; `offset` elements into buffers that end 3 elements
    behind it (to see writes past the end)."""
    dt = {"fp32": torch.float32, "bf16": torch.bfloat16}

    def place(values, dtype):
        full = torch.full((offset + len(values) + 3,), 9.0, device="cuda").to(dtype)
        full[offset:offset + len(values)] = torch.tensor(values).to(dtype)
        return full[offset:offset + len(values)], full

    e, whole = {}, {}

    def put(k, values, dtype):
        e[k], whole[k] = place(values, dtype)

    p = rng.normal(0, 0.5, size=n)
    put("param", p, dt[dtype])
    put("grad", rng.normal(0, 0.01, size=n) * 10.0 ** rng.integers(-3, 1, size=n), dt[grad])
    if master:
        put("master", p, torch.float32)
    if state == "fp32":
        put("m", rng.normal(0, 0.01, size=n) * (not fresh), torch.float32)
        put("v", rng.normal(0, 0.02, size=n) ** 2 * (not fresh), torch.float32)
    else:
        nb = -(-n // BLOCK)
        put("m", np.clip(rng.normal(0, 100, size=n), -448, 448) * (not fresh),
            torch.float8_e4m3fn)
        put("v", np.clip(np.abs(rng.normal(0, 100, size=n)), 0.01, 448) * (not fresh),
            torch.float8_e4m3fn)
        put("m_scale", np.abs(rng.normal(0, 1e-4, size=nb)) * (not fresh), torch.float32)
        put("v_scale", np.abs(rng.normal(0, 2e-4, size=nb)) * (not fresh), torch.float32)
    e.update(more)
    return e, whole


def expected(e, t, gs=1.0, lr=None, hp=HP):
    """float64 results of step t from the entry as it is now."""
    n = e["param"].numel()
    p = down(e.get("master", e["param"]))
    g = down(e["grad"]) * gs
    m, v = down(e["m"].float()), down(e["v"].float())
    if "m_scale" in e:
        rep = lambda k: np.repeat(down(e[k]), BLOCK)[:n]  # noqa: E731
        m, v = m * rep("m_scale"), (v * rep("v_scale")) ** 2
    b1, b2 = hp["beta1"], hp["beta2"]
    am = np.abs(b1 * m) + np.abs((1 - b1) * g)
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    lr = (hp["lr"] if lr is None else lr) * e.get("lr_mult", 1.0)
    wd = hp["weight_decay"] if e.get("decay", True) else 0.0
    den = (1 - b1 ** t) * (np.sqrt(v / (1 - b2 ** t)) + hp["eps"])
    new = p - lr * (m / den + wd * p)
    tol_p = 32 * U * lr * (am / den + wd * np.abs(p)) + 2 * U * (np.abs(p) + np.abs(new))
    return dict(p=new, m=m, v=v, tol_p=tol_p, tol_m=4 * U * am, tol_v=4 * U * v)


def check(e, want, what=""):
    p_tol = want["tol_p"]
    if "master" in e:
        within(e["master"], want["p"], p_tol, what + " master")
    half = torch.finfo(e["param"].dtype).eps / 2 if e["param"].dtype == torch.bfloat16 else 0.0
    within(e["param"], want["p"], p_tol + half * (np.abs(want["p"]) + p_tol), what + " param")
    if "m_scale" not in e:
        within(e["m"], want["m"], want["tol_m"] + 1e-45, what + " m")
        within(e["v"], want["v"], want["tol_v"] + 1e-45, what + " v")
        return
    n = e["param"].numel()
    nb = -(-n // BLOCK)
    for k, val, least in (("m", want["m"], 2.0 ** -10), ("v", np.sqrt(want["v"]), 2.0 ** -9)):
        pad = np.zeros(nb * BLOCK)
        pad[:n] = np.abs(val)
        top = pad.reshape(nb, BLOCK).max(1)
        within(e[k + "_scale"], top / 448, 8 * U * top / 448 + want["tol_m"].max() * (k == "m"),
               what + " %s scale" % k)
        scale = np.repeat(down(e[k + "_scale"]), BLOCK)[:n]
        got = down(e[k].float()) * scale
        tol = (2.0 ** -4 + 16 * U) * np.abs(val) + least * scale * (1 + 2.0 ** -20) + (
            want["tol_m"] if k == "m" else 0.0)
        err = np.abs(got - val)
        assert (err <= tol).all(), (what, k, (err - tol).max())
        if k == "v":
            assert ((got > 0) == (val > 0)).all()


def untouched(e, whole, offset=0):
    for k, full in whole.items():
        n = e[k].numel()
        rest = torch.cat([full[:offset], full[offset + n:]]).float()
        assert bool((rest == torch.tensor(9.0).to(full.dtype).float().item()).all()), k


def run(entries, step, hp=HP, **kw):
    import mixture_experts_routing_fp32_b200 as moe
    moe.moe_adamw(moe.make_adamw_config(**hp), moe.adamw_table(entries), step, **kw)
    torch.cuda.synchronize()


SIZES = [1, 7, 8, 255, 256, 257, 2047, 2048, 2049, 6001]
KINDS = [dict(), dict(dtype="bf16", grad="bf16"), dict(dtype="bf16", grad="bf16", master=True),
         dict(dtype="bf16", grad="fp32"), dict(state="fp8"),
         dict(dtype="bf16", grad="bf16", state="fp8", master=True)]


@pytest.mark.parametrize("kind", KINDS, ids=lambda k: "-".join(map(str, k.values())) or "fp32")
@pytest.mark.parametrize("offset", [0, 1, 8])
def test_every_size_and_alignment(kind, offset):
    rng = np.random.default_rng(7)
    made = [make(rng, n, offset=offset, fresh=(i % 3 == 2), decay=i % 2 == 0,
                 lr_mult=1.0 + 0.5 * (i % 2), **kind) for i, n in enumerate(SIZES)]
    entries = [e for e, _ in made]
    step = torch.tensor([4, 0], dtype=torch.int32, device="cuda")
    for t in (5, 6):
        want = [expected(e, t, gs=0.25) for e in entries]
        run(entries, step, grad_scale=torch.full((1,), 0.25, device="cuda"))
        assert step.tolist() == [t, 0]
        for (e, whole), w in zip(made, want):
            check(e, w, "n = %d" % e["param"].numel())
            untouched(e, whole, offset)


def test_many_tensors_empty_ones_and_mixed_kinds():
    """More tensors than one launch takes, empty ones between and at the end."""
    rng = np.random.default_rng(8)
    made = [make(rng, 0 if i % 9 == 4 else 1 + 37 * i, **KINDS[i % len(KINDS)]) for i in range(95)]
    made += [make(rng, 0), make(rng, 0)]
    entries = [e for e, _ in made]
    step = torch.zeros(2, dtype=torch.int32, device="cuda")
    want = [expected(e, 1) for e in entries]
    run(entries, step)
    assert step.tolist() == [1, 0]
    for (e, whole), w in zip(made, want):
        if e["param"].numel():
            check(e, w, "n = %d" % e["param"].numel())
        untouched(e, whole)
    run([], step)
    assert step.tolist() == [2, 0]


def test_zero_gradients_and_tiny_states():
    """Nothing divides by zero: fresh states with zero gradients only decay,
    and 8-bit blocks below the smallest kept scale hold zeros."""
    rng = np.random.default_rng(9)
    for kind in (dict(), dict(state="fp8")):
        e, _ = make(rng, 600, fresh=True, **kind)
        e["grad"].zero_()
        e["grad"][300:] = 1e-33
        want = expected(e, 1)
        run([e], torch.zeros(2, dtype=torch.int32, device="cuda"))
        within(e["param"], want["p"], want["tol_p"] + 1e-12, "param")
        if kind:
            assert down(e["m"].float())[:256].tolist() == [0.0] * 256
            assert float(e["m_scale"][1]) == 0.0 and float(e["v_scale"][0]) == 0.0


def test_a_nan_stays_in_its_block():
    rng = np.random.default_rng(10)
    for kind in (dict(), dict(state="fp8")):
        for bad in (float("nan"), float("inf")):
            e, _ = make(rng, 1024, **kind)
            clean = {k: v.clone() if torch.is_tensor(v) else v for k, v in e.items()}
            e["grad"][300] = bad
            step = lambda: torch.zeros(2, dtype=torch.int32, device="cuda")  # noqa: E731
            run([clean], step())
            run([e], step())
            keep = torch.arange(1024, device="cuda") != 300
            assert torch.equal(e["param"][keep], clean["param"][keep])
            assert not bool(torch.isfinite(e["param"][300]))
            if kind:
                m = e["m"].float() * e["m_scale"].repeat_interleave(BLOCK)
                v = e["v"].float() * e["v_scale"].repeat_interleave(BLOCK)
                for s in (m, v):
                    assert bool(s[256:512].isnan().all()) and bool(
                        torch.isfinite(torch.cat([s[:256], s[512:]])).all())


def test_8_bit_states_are_those_of_plain_operations():
    """The 8-bit roundings fall as for plain fp32 operations in the formulas'
    order (each product and sum rounded), bit for bit over several steps: a
    rounding that fell the other way would stay in the state."""
    rng = np.random.default_rng(12)
    e, _ = make(rng, 256 * 400 + 77, dtype="bf16", grad="bf16", state="fp8", master=True)
    step = torch.zeros(2, dtype=torch.int32, device="cuda")
    n = e["param"].numel()
    m8, v8, ms, vs = (e[k].clone() for k in ("m", "v", "m_scale", "v_scale"))
    blocks = lambda t: torch.cat([t, t.new_zeros(-n % BLOCK)]).reshape(-1, BLOCK)  # noqa: E731
    for t in range(3):
        e["grad"].copy_(torch.tensor(rng.normal(0, 0.01, size=n)))
        g = e["grad"].float() * 0.3
        m = (blocks(m8.float()) * ms[:, None]).reshape(-1)[:n]
        v = (blocks(v8.float()) * vs[:, None]).square().reshape(-1)[:n]
        m = 0.9 * m + (1 - 0.9) * g
        r = (0.99 * v + (1 - 0.99) * g * g).sqrt()
        run([e], step, grad_scale=torch.full((1,), 0.3, device="cuda"))
        for k, val in (("m", m), ("v", r)):
            b = blocks(val)
            top = b.abs().amax(1)
            q = b * (top.reciprocal() * 448.0)[:, None]
            if k == "v":
                q = torch.where((q > 0) & (q < 2.0 ** -9), 2.0 ** -9, q)
            q = q.reshape(-1)[:n].to(torch.float8_e4m3fn)
            sc = top * (torch.ones_like(top) / 448.0)
            assert torch.equal(e[k].view(torch.uint8), q.view(torch.uint8)), (t, k)
            assert torch.equal(e[k + "_scale"], sc), (t, k)
        m8, v8, ms, vs = (e[k].clone() for k in ("m", "v", "m_scale", "v_scale"))


def test_steps_of_an_optimizer_in_a_graph():
    """MoEAdamW over 6 steps, 4 of them replays of a captured step with the
    learning rate read from the device, against the float64 recursion."""
    import mixture_experts_routing_fp32_b200 as moe
    rng = np.random.default_rng(11)
    p = [torch.tensor(rng.normal(size=s), dtype=torch.float32, device="cuda")
         for s in ((4, 32), (3, 100), (5,))]
    g = [torch.zeros_like(t) for t in p]
    opt = moe.MoEAdamW(p, g, lr=123.0, betas=(0.9, 0.99), eps=1e-6, weight_decay=0.1,
                       no_decay=(2,))
    lr = torch.zeros(1, device="cuda")
    ref = [dict(p=down(t), m=0.0, v=0.0) for t in p]
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    for t in range(1, 7):
        lr.fill_(0.01 * t)
        for a in g:
            a.copy_(torch.tensor(rng.normal(0, 0.1, size=a.shape)))
        torch.cuda.synchronize()
        if t == 1:
            opt.step(lr=lr)
        elif t == 2:
            with torch.cuda.stream(side):
                opt.step(lr=lr)
                side.synchronize()
                with torch.cuda.graph(graph, stream=side):
                    opt.step(lr=lr)
        else:
            graph.replay()
        torch.cuda.synchronize()
        for i, (r, a) in enumerate(zip(ref, g)):
            q = down(a)
            rate = float(lr.double())
            r["m"] = 0.9 * r["m"] + (1 - 0.9) * q
            r["v"] = 0.99 * r["v"] + (1 - 0.99) * q * q
            up = r["m"] / (1 - 0.9 ** t) / (np.sqrt(r["v"] / (1 - 0.99 ** t)) + 1e-6)
            r["p"] = r["p"] - rate * (up + (0.1 if i != 2 else 0.0) * r["p"])
    assert opt.count.tolist() == [6, 0]
    for r, t in zip(ref, p):
        # 6 steps of at most 64 U of an update (its terms do not cancel below
        # a hundredth) and 2 U of the parameter
        within(t, r["p"], 6 * (100 * 64 * U * 0.06 + 4 * U * np.abs(r["p"])), "param")


def test_training_step_of_a_layer():
    """The layer's weights and its own gradient buffers, 8-bit states: the
    step moves every weight against its gradient."""
    import mixture_experts_routing_fp32_b200 as moe
    import workloads as W
    cfg = W.REDUCED["mm_b"]
    inp = {n: W.make_input(cfg, n, "cuda") for n in ("x", "w_r", "w13", "w_down", "dy")}
    layer = moe.MoELayer(moe.config_from(cfg))
    w = [inp["w_r"], inp["w13"], inp["w_down"]]
    layer.forward(inp["x"], *w)
    layer.backward(inp["dy"])
    opt = moe.MoEAdamW(w, [layer.dw_r, layer.dw13, layer.dw_down], lr=1e-2, weight_decay=0.0,
                       state="fp8", masters=True)
    before = [e.get("master", e["param"]).clone() for e in opt.entries]
    opt.step()
    torch.cuda.synchronize()
    for e, b in zip(opt.entries, before):
        moved = e.get("master", e["param"]).float() - b.float()
        g = e["grad"].float()
        big = g.abs() > 1e-3 * g.abs().max()
        # the first step moves by lr against the sign of the gradient
        assert bool((moved[big] * g[big] < 0).all())


def test_tensors_that_overlap_are_refused():
    """What a step writes may be no other tensor of it, nor a part of one;
    gradients may share memory with one another."""
    import mixture_experts_routing_fp32_b200 as moe
    pool = torch.zeros(4096, device="cuda")
    names = ("param", "grad", "m", "v")
    at = lambda *starts: {k: pool[s:s + 512] for k, s in zip(names, starts)}  # noqa: E731
    ok = [at(0, 512, 1024, 1536), at(2048, 512, 2560, 3200)]
    moe.moe_adamw(moe.make_adamw_config(), moe.adamw_table(ok),
                  torch.zeros(2, dtype=torch.int32, device="cuda"))
    for bad in ([ok[0], ok[0]], [at(0, 512, 1024, 1024)], [at(0, 0, 1024, 1536)],
                [at(0, 512, 1024, 1280)], [ok[0], at(2048, 3584, 2560, 100)],
                [ok[0], at(2048, 1500, 2560, 3200)]):
        with pytest.raises(moe.MoEError, match="overlaps"):
            moe.adamw_table(bad)
    torch.cuda.synchronize()


@pytest.mark.parametrize("kind", [dict(), dict(state="fp8"), dict(dtype="bf16", master=True)],
                         ids=lambda k: "-".join(map(str, k.values())) or "fp32")
def test_small_eps_and_small_gradients(kind):
    """eps far below the smallest normal root (2^-63), gradients around and
    below it: the step still is one of about lr.  v' is subnormal there, so
    its terms are off by half of 2^-149 each (at most three of them), which
    the root halves: up to 2^-149 / v' of the update."""
    rng = np.random.default_rng(13)
    hp = dict(HP, eps=1e-25)
    for size in (1e-17, 3e-18, 1e-18, 1e-19, 1e-20):
        e, _ = make(rng, 700, fresh=True, **kind)
        e["grad"].copy_(torch.tensor(size * rng.choice([-1, 1], size=700)
                                     * rng.uniform(0.5, 1.0, size=700)))
        step = torch.zeros(2, dtype=torch.int32, device="cuda")
        want = expected(e, 1, hp=hp)
        run([e], step, hp=hp)
        update = np.abs(want["m"]) / 0.1 / (np.sqrt(want["v"] / (1 - 0.99)) + 1e-25)
        assert (np.abs(update - 1.0) < 1e-3).all()
        tol = want["tol_p"] + HP["lr"] * update * 2.0 ** -149 / want["v"]
        within(e["master"] if "master" in e else e["param"], want["p"], tol, "size %g" % size)


def test_8_bit_codes_against_the_quotient():
    """Codes and scales come from a rounded reciprocal and a product (3 U with
    the product by the value, 2 U for a scale) where the definition has one
    quotient: a code is that of 448 v / largest, or of a value 3 U away."""
    rng = np.random.default_rng(14)
    n = 256 * 1000
    e, _ = make(rng, n, dtype="bf16", grad="bf16", state="fp8", fresh=True, master=True)
    run([e], torch.zeros(2, dtype=torch.int32, device="cuda"))
    g = e["grad"].float()
    # fresh states: single fp32 operations in the formulas' order
    for k, val in (("m", (1 - 0.9) * g), ("v", ((1 - 0.99) * g * g).sqrt())):
        b = val.double().reshape(-1, BLOCK)
        top = b.abs().amax(1, keepdim=True)
        err = (e[k + "_scale"].double() - top[:, 0] / 448).abs()
        assert bool((err <= 2.01 * U * top[:, 0] / 448).all())
        at = (448 * b / top).reshape(-1)
        if k == "v":
            at = torch.where((at > 0) & (at < 2.0 ** -9), 2.0 ** -9, at)
        # (the bounds' own rounding to fp32, U more)
        ends = torch.stack([(at * f).float().to(torch.float8_e4m3fn).float()
                            for f in (1 - 4.1 * U, 1 + 4.1 * U)])
        got = e[k].float()
        assert bool(((ends.amin(0) <= got) & (got <= ends.amax(0))).all())
