"""The cases that the block operators are measured on: the norms around a
layer (forward and backward), the AdamW step over a layer's weights, and the
experts' products in 8-bit integers.

`listed()` and `draw()` say which calls; `prepare()` makes what a program has
in hand before one; `run()` makes it, in plain torch operations in 32 bits
(`own` false) or through the framework's entry points (`own` true);
`exact()` computes the same from the definitions in 64 bits; `work()` counts
the bytes and operations that a call cannot do without.
"""
from __future__ import annotations

import math

import torch

own = False

BLOCK = 256          # elements that share a scale of an 8-bit optimizer state
E4M3_MAX = 448.0     # largest e4m3 value: a block's largest state maps to it
STATE_MIN = 2.0 ** -100   # blocks whose largest state is below are held as zeros
BETA1, BETA2, ADAM_EPS, LR, DECAY = 0.9, 0.95, 1e-8, 3e-4, 0.1
NORM_EPS = 1e-5


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _norm(name, op, T, D, norm, dtype, resid, gate_len, alpha, post, bias):
    return {"name": name, "op": op, "T": T, "D": D, "norm": norm, "dtype": dtype,
            "resid": resid, "gate_len": gate_len, "alpha": alpha, "post": post, "bias": bias}


def _adamw(name, state, weights, master, E, D, F, extra):
    return {"name": name, "op": "adamw", "state": state, "weights": weights, "master": master,
            "E": E, "D": D, "F": F, "extra": extra}


def _i8(name, T, D, E, K, F, shared, empty):
    return {"name": name, "op": "ffn_i8", "T": T, "D": D, "E": E, "K": K, "F": F,
            "shared": shared, "empty": empty}


def listed():
    return [
        # one token through the widest model's block: decoding, latency only
        _norm("norm_fwd_token", "norm_fwd", 1, 7168, "rms", "bf16", "bf16", 0, 1.0, True, False),
        # a training batch of the Mixtral-shaped block (half its tokens)
        _norm("norm_fwd_mix", "norm_fwd", 16384, 4096, "rms", "bf16", "bf16", 0, 0.5, True, False),
        # ragged sequences with a gate row each, fp32 activations, LayerNorm
        _norm("norm_bwd_ragged", "norm_bwd", 1003, 768, "layer", "fp32", "fp32", 100, 0.7, True,
              True),
        # a training batch of the DeepSeek-V3-shaped block
        _norm("norm_bwd_ds3", "norm_bwd", 8192, 7168, "rms", "bf16", "bf16", 8192, 1.0, True,
              False),
        # the tiny fp32 layer's weights: many small tensors in one call
        _adamw("adamw32_tiny", "fp32", "fp32", False, 4, 32, 64, 24),
        # the MiniMind-shaped layer, bf16 weights with fp32 master copies
        _adamw("adamw32_mm", "fp32", "bf16", True, 4, 768, 2048, 3),
        # 8-bit states over tensors of odd sizes
        _adamw("adamw8_odd", "fp8", "bf16", False, 3, 136, 200, 11),
        # 8-bit states of the OLMoE-shaped layer's weights
        _adamw("adamw8_olmoe", "fp8", "bf16", False, 64, 2048, 1024, 2),
        # one token through the OLMoE-shaped experts: decoding
        _i8("i8_token", 1, 2048, 64, 8, 1024, False, 0.0),
        # a batch of decoded tokens through the Mixtral-shaped experts
        _i8("i8_decode_mix", 16, 4096, 8, 2, 14336, False, 0.0),
        # a ragged prompt with a shared expert and slots without an expert
        _i8("i8_shared_ragged", 333, 1024, 32, 4, 512, True, 0.1),
        # prompts through the OLMoE-shaped experts
        _i8("i8_olmoe", 8192, 2048, 64, 8, 1024, False, 0.0),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["norm_fwd", "norm_bwd", "adamw", "ffn_i8"])
    if op in ("norm_fwd", "norm_bwd"):
        D = 8 * _log_int(rng, 8, 1024)
        T = _log_int(rng, 1, min(16384, 16384 * 4096 // D))
        norm = rng.choice(["rms", "layer"])
        dtype, resid = rng.choice([("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")])
        gate_len = rng.choice([0, T, _log_int(rng, 1, T)])
        return _norm("", op, T, D, norm, dtype, resid, gate_len, rng.choice([1.0, 0.5, 0.22]),
                     rng.random() < 0.8, norm == "layer" and rng.random() < 0.7)
    if op == "adamw":
        state = rng.choice(["fp32", "fp8"])
        weights = rng.choice(["bf16", "fp32"])
        E = _log_int(rng, 2, 64)
        D = 8 * _log_int(rng, 2, 256)
        most = 64 * 2048 * 1024 // (4 if state == "fp32" else 1)
        F = 8 * _log_int(rng, 2, max(2, min(256, most // (E * D * 8))))
        return _adamw("", state, weights, weights == "bf16" and rng.random() < 0.5, E, D, F,
                      rng.randrange(0, 40))
    E = rng.choice([4, 8, 16, 32, 64])
    K = rng.choice([k for k in (1, 2, 4, 8) if k <= E])
    D = 128 * _log_int(rng, 2, 32)
    F = 128 * _log_int(rng, 1, min(112, 8 * 4096 * 14336 // (E * D * 128)))
    most = int(8192 * 8 * 2048 * 1024 // (K * D * F))
    T = _log_int(rng, 1, max(1, min(8192, most)))
    return _i8("", T, D, E, K, F, rng.random() < 0.4, rng.choice([0.0, 0.1]))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _dt(name):
    return torch.bfloat16 if name == "bf16" else torch.float32


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)

    def randn(*shape, dtype=torch.float32, std=1.0, mean=0.0):
        t = torch.empty(shape, dtype=dtype, device="cuda")
        return t.normal_(mean, std, generator=g)

    s = {"case": case}
    if case["op"] in ("norm_fwd", "norm_bwd"):
        T, D = case["T"], case["D"]
        act, res = _dt(case["dtype"]), _dt(case["resid"])
        # the residual stream of a deep model is wider than one block's output
        s["r"] = randn(T, D, dtype=res, std=3.0, mean=0.2)
        s["y"] = randn(T, D, dtype=act, std=0.8, mean=0.1)
        s["w_post"] = randn(D, std=0.1, mean=1.0) if case["post"] else None
        s["b_post"] = randn(D, std=0.1) if case["post"] and case["bias"] else None
        s["w_pre"] = randn(D, std=0.1, mean=1.0)
        s["b_pre"] = randn(D, std=0.1) if case["bias"] else None
        L = case["gate_len"]
        s["gate"] = randn(-(-T // L), D, std=0.5, mean=0.5) if L else None
        if case["op"] == "norm_bwd":
            # what the forward leaves: here s["r"] is the stream after the
            # block, with the statistics of both norms
            s["dx"] = randn(T, D, dtype=act)
            s["dr_out"] = randn(T, D, dtype=res)
            st = torch.zeros(T, 4, device="cuda")
            for k, v in ((0, s["y"]), (2, s["r"])):
                v = v.double()
                mean = v.mean(1) if case["norm"] == "layer" else torch.zeros(T, device="cuda",
                                                                            dtype=torch.float64)
                st[:, k] = mean
                st[:, k + 1] = ((v - mean[:, None]).square().mean(1) + NORM_EPS).rsqrt()
            if not case["post"]:
                st[:, 0], st[:, 1] = 0.0, 1.0
            s["stats"] = st
    elif case["op"] == "adamw":
        E, D, F = case["E"], case["D"], case["F"]
        # router, experts' projections, and the block's vectors (norms,
        # gates, biases) of uneven lengths
        shapes = [(E, D), (E, 2 * F, D), (E, D, F)]
        shapes += [(D + 7 * i + (i % 3),) for i in range(case["extra"])]
        s["tensors"] = []
        for i, shape in enumerate(shapes):
            wt = torch.float32 if i == 0 or len(shape) == 1 else _dt(case["weights"])
            t = {"param": randn(*shape, dtype=wt, std=0.02)}
            t["grad"] = randn(*shape, dtype=wt, std=1e-3)
            t["master"] = t["param"].float() if case["master"] and wt == torch.bfloat16 else None
            n = t["param"].numel()
            if case["state"] == "fp32":
                t["m"], t["v"] = randn(*shape, std=5e-4), randn(*shape, std=1e-3).square_()
                t["m_scale"] = t["v_scale"] = None
            else:
                nb = -(-n // BLOCK)
                t["m"] = (randn(n, std=100.0).clamp_(-448, 448)).to(torch.float8_e4m3fn)
                t["v"] = (randn(n, std=150.0).abs_().clamp_(0.01, 448)).to(torch.float8_e4m3fn)
                t["m_scale"] = randn(nb, std=1e-6).abs_().add_(1e-6)
                t["v_scale"] = randn(nb, std=2e-6).abs_().add_(3e-6)
            t["decay"] = len(shape) > 1
            s["tensors"].append(t)
        # steps taken so far (the second word belongs to the step's kernel)
        s["step"] = torch.tensor([10 + seed % 90, 0], dtype=torch.int32, device="cuda")
        s["grad_scale"] = torch.full((1,), 0.5, device="cuda")
    else:
        T, D, E, K, F = (case[k] for k in ("T", "D", "E", "K", "F"))
        s["x"] = randn(T, D, dtype=torch.bfloat16)
        # a router's picks: distinct experts per token, uneven loads
        score = randn(T, E) + 0.5 * randn(E)
        top = score.topk(K, 1)
        s["topk_idx"] = top.indices.to(torch.int32)
        s["topk_w"] = torch.softmax(top.values, 1)
        if case["empty"]:
            hole = torch.rand(T, K, generator=g, device="cuda") < case["empty"]
            s["topk_idx"][hole] = -1

        def weight(*shape):
            q = torch.empty(shape, dtype=torch.int8, device="cuda").random_(-127, 128, generator=g)
            sc = torch.empty(shape[:-1], device="cuda").uniform_(0.5, 1.5, generator=g)
            return q, sc * (1.0 / (73.0 * math.sqrt(shape[-1])))

        s["w13"], s["w13_scale"] = weight(E, 2 * F, D)
        s["w_down"], s["w_down_scale"] = weight(E, D, F)
        s["w13_s"] = s["w13_s_scale"] = s["w_down_s"] = s["w_down_s_scale"] = None
        if case["shared"]:
            s["w13_s"], s["w13_s_scale"] = weight(2 * F, D)
            s["w_down_s"], s["w_down_s_scale"] = weight(D, F)
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm_fwd": _own_norm_fwd, "norm_bwd": _own_norm_bwd, "adamw": _own_adamw,
                "ffn_i8": _own_ffn_i8}[op](state)
    return {"norm_fwd": _plain_norm_fwd, "norm_bwd": _plain_norm_bwd, "adamw": _plain_adamw,
            "ffn_i8": _plain_ffn_i8}[op](state)


# --- the framework's calls --------------------------------------------------
def _handle(state, make):
    """What a program keeps between calls: output buffers, workspace, tables."""
    if "handle" not in state:
        import mixture_experts_routing_fp32_b200 as moe
        state["handle"] = make(moe)
    return state["handle"]


def _norm_config(moe, c):
    return moe.make_norm_config(c["T"], c["D"], norm=c["norm"], dtype=c["dtype"],
                                resid=c["resid"], eps=NORM_EPS, alpha=c["alpha"],
                                gate_len=c["gate_len"])


def _own_norm_fwd(s):
    c = s["case"]

    def make(moe):
        return (moe, _norm_config(moe, c), torch.empty_like(s["r"]), torch.empty_like(s["y"]),
                torch.empty(c["T"], 4, device="cuda"))

    moe, nc, r_out, x, stats = _handle(s, make)
    moe.moe_block_norm(nc, s["r"], s["y"], s["w_post"], s["b_post"], s["gate"], s["w_pre"],
                       s["b_pre"], r_out, x, stats)
    return {"r_out": r_out, "x": x, "stats": stats}


def _own_norm_bwd(s):
    c = s["case"]

    def make(moe):
        nc = _norm_config(moe, c)
        like = lambda t: None if t is None else torch.empty_like(t)  # noqa: E731
        out = {"dy": like(s["y"]), "dr": like(s["r"]), "dw_post": like(s["w_post"]),
               "db_post": like(s["b_post"]), "dgate": like(s["gate"]),
               "dw_pre": like(s["w_pre"]), "db_pre": like(s["b_pre"])}
        ws = torch.empty(moe.moe_block_norm_ws_bytes(nc), dtype=torch.uint8, device="cuda")
        return moe, nc, out, ws

    moe, nc, o, ws = _handle(s, make)
    moe.moe_block_norm_backward(nc, s["r"], s["y"], s["w_post"], s["b_post"], s["gate"],
                                s["w_pre"], s["stats"], s["dx"], s["dr_out"], o["dy"], o["dr"],
                                o["dw_post"], o["db_post"], o["dgate"], o["dw_pre"], o["db_pre"],
                                ws)
    return o


def _own_adamw(s):
    def make(moe):
        hp = moe.make_adamw_config(lr=LR, beta1=BETA1, beta2=BETA2, eps=ADAM_EPS,
                                   weight_decay=DECAY)
        return moe, hp, moe.adamw_table(s["tensors"])

    moe, hp, table = _handle(s, make)
    moe.moe_adamw(hp, table, s["step"], grad_scale=s["grad_scale"])
    return _adamw_out(s)


def _own_ffn_i8(s):
    c = s["case"]

    def make(moe):
        cfg = moe.make_config(c["T"], c["D"], c["E"], c["K"], c["F"], n_shared=int(c["shared"]))
        layer = moe.MoEInt8Layer(cfg)
        layer.set_weights(s["w13"], s["w13_scale"], s["w_down"], s["w_down_scale"], s["w13_s"],
                          s["w13_s_scale"], s["w_down_s"], s["w_down_s_scale"])
        return layer

    return _handle(s, make).experts(s["x"], s["topk_idx"], s["topk_w"])


# --- plain forms --------------------------------------------------------------
def _moments(v, layer):
    mean = v.mean(1, keepdim=True) if layer else torch.zeros_like(v[:, :1])
    return mean, ((v - mean).square().mean(1, keepdim=True) + NORM_EPS).rsqrt()


def _gate_rows(s):
    """The gate of every token ([T, D] or a scalar 1)."""
    c = s["case"]
    if s["gate"] is None:
        return 1.0
    return s["gate"][torch.arange(c["T"], device="cuda") // c["gate_len"]]


def _plain_norm_fwd(s):
    c = s["case"]
    layer = c["norm"] == "layer"
    z = s["y"].float()
    my, ry = torch.zeros_like(z[:, :1]), torch.ones_like(z[:, :1])
    if c["post"]:
        my, ry = _moments(z, layer)
        z = (z - my) * ry * s["w_post"]
        if s["b_post"] is not None:
            z = z + s["b_post"]
    r_out = (s["r"].float() + c["alpha"] * (_gate_rows(s) * z)).to(s["r"].dtype)
    v = r_out.float()
    mr, rr = _moments(v, layer)
    x = (v - mr) * rr * s["w_pre"]
    if s["b_pre"] is not None:
        x = x + s["b_pre"]
    return {"r_out": r_out, "x": x.to(s["y"].dtype), "stats": torch.cat([my, ry, mr, rr], 1)}


def _norm_grad(dhat, hat, rstd, layer):
    d = dhat - hat * (dhat * hat).mean(1, keepdim=True)
    if layer:
        d = d - dhat.mean(1, keepdim=True)
    return d * rstd


def _by_gate_row(t, L):
    """Sums of consecutive groups of L rows."""
    G = -(-t.shape[0] // L)
    pad = torch.zeros(G * L - t.shape[0], t.shape[1], device=t.device)
    return torch.cat([t, pad]).reshape(G, L, -1).sum(1)


def _plain_norm_bwd(s):
    c = s["case"]
    layer = c["norm"] == "layer"
    my, ry, mr, rr = s["stats"].split(1, 1)
    dx = s["dx"].float()
    rhat = (s["r"].float() - mr) * rr
    d = s["dr_out"].float() + _norm_grad(dx * s["w_pre"], rhat, rr, layer)
    y = s["y"].float()
    yhat = (y - my) * ry if c["post"] else y
    z = yhat
    if c["post"]:
        z = yhat * s["w_post"]
        if s["b_post"] is not None:
            z = z + s["b_post"]
    da = c["alpha"] * d
    dz = da * _gate_rows(s)
    dy = _norm_grad(dz * s["w_post"], yhat, ry, layer) if c["post"] else dz
    return {"dy": dy.to(s["y"].dtype), "dr": d.to(s["r"].dtype),
            "dw_post": (dz * yhat).sum(0) if c["post"] else None,
            "db_post": dz.sum(0) if s["b_post"] is not None else None,
            "dgate": _by_gate_row(da * z, c["gate_len"]) if s["gate"] is not None else None,
            "dw_pre": (dx * rhat).sum(0),
            "db_pre": dx.sum(0) if s["b_pre"] is not None else None}


def _adamw_out(s):
    keys = ("param", "master", "m", "v", "m_scale", "v_scale")
    ts = s["tensors"]
    # the three weight tensors whole, then the small vectors joined
    out = {"step": s["step"][:1]}
    for i, t in enumerate(ts[:3]):
        out["t%d" % i] = {k: t[k] for k in keys}
    if len(ts) > 3:
        for k in keys:
            if ts[3][k] is not None:
                out["vectors_" + k] = torch.cat([t[k].reshape(-1) for t in ts[3:]])
    return out


def _blocks(flat):
    nb = -(-flat.numel() // BLOCK)
    pad = torch.zeros(nb * BLOCK - flat.numel(), device=flat.device)
    return torch.cat([flat, pad]).reshape(nb, BLOCK)


def _unpack8(q, scale):
    return (_blocks(q.float()) * scale[:, None]).reshape(-1)[:q.numel()]


def _pack8(val, keep_positive):
    """(e4m3 values, block scales) of a flat state; a positive value that
    rounds to zero becomes the smallest positive code if keep_positive."""
    b = _blocks(val)
    big = b.abs().amax(1)
    there = big >= STATE_MIN
    inv = torch.where(there, E4M3_MAX / big, torch.zeros_like(big))
    scaled = b * inv[:, None]
    if keep_positive:
        least = 2.0 ** -9
        scaled = torch.where((scaled > 0) & (scaled < least), torch.full_like(scaled, least),
                             scaled)
    q = scaled.reshape(-1)[:val.numel()].to(torch.float8_e4m3fn)
    return q, torch.where(there, big / E4M3_MAX, torch.zeros_like(big))


def _plain_adamw(s):
    s["step"][0] += 1
    t = s["step"][0].double()
    bc1, bc2 = (1 - BETA1 ** t).float(), (1 - BETA2 ** t).float()
    for w in s["tensors"]:
        p = (w["param"] if w["master"] is None else w["master"]).float().reshape(-1)
        g = w["grad"].float().reshape(-1) * s["grad_scale"]
        if w["m_scale"] is None:
            m, v = w["m"].reshape(-1), w["v"].reshape(-1)
        else:
            m = _unpack8(w["m"], w["m_scale"])
            v = _unpack8(w["v"], w["v_scale"]).square()
        m = BETA1 * m + (1 - BETA1) * g
        v = BETA2 * v + (1 - BETA2) * g * g
        p = p - LR * ((m / bc1) / ((v / bc2).sqrt() + ADAM_EPS) + (DECAY * w["decay"]) * p)
        w["param"].copy_(p.reshape(w["param"].shape))
        if w["master"] is not None:
            w["master"].copy_(p.reshape(w["master"].shape))
        if w["m_scale"] is None:
            w["m"].copy_(m.reshape(w["m"].shape))
            w["v"].copy_(v.reshape(w["v"].shape))
        else:
            for k, val, pos in (("m", m, False), ("v", v.sqrt(), True)):
                q, sc = _pack8(val, pos)
                w[k].copy_(q)
                w[k + "_scale"].copy_(sc)
    return _adamw_out(s)


def _quant_rows(v):
    """int8 values (held in 32 bits) and the scale of each row.  127 v is
    exact for bf16 v, so the quotient falls on a tie exactly when it is one."""
    big = v.abs().amax(-1, keepdim=True)
    return (v * 127.0 / torch.where(big > 0, big, torch.ones_like(big))).round(), big / 127.0


def _product(q, sc, w, w_scale):
    return torch.matmul(q, w.float().transpose(-1, -2)) * sc * w_scale.unsqueeze(-2)


def _swiglu_i8(q, sc, w13, w13_scale, w_down, w_down_scale):
    a = _product(q, sc, w13, w13_scale)
    F = a.shape[-1] // 2
    h = a[..., :F] * torch.sigmoid(a[..., :F]) * a[..., F:]
    return _product(*_quant_rows(h), w_down, w_down_scale)


def _plain_ffn_i8(s):
    c = s["case"]
    T, D, E, K = (c[k] for k in ("T", "D", "E", "K"))
    x = s["x"].float()
    q, sc = _quant_rows(x)
    # slots sorted by expert (those without one last), each expert's rows in
    # a padded batch
    e = s["topk_idx"].reshape(-1).long()
    e = torch.where(e < 0, E, e)
    order = torch.argsort(e, stable=True)
    counts = torch.bincount(e, minlength=E + 1)
    start = counts.cumsum(0) - counts
    rows = max(1, int(counts[:E].max()))
    es = e[order]
    at = torch.arange(T * K, device="cuda") - start[es]
    held = es < E
    es, at, tok = es[held], at[held], (order // K)[held]
    qb, sb = torch.zeros(E, rows, D, device="cuda"), torch.zeros(E, rows, 1, device="cuda")
    qb[es, at], sb[es, at] = q[tok], sc[tok]
    o = _swiglu_i8(qb, sb, s["w13"], s["w13_scale"], s["w_down"], s["w_down_scale"])
    per_slot = torch.zeros(T * K, D, device="cuda")
    per_slot[order[held]] = o[es, at]
    y = (per_slot.reshape(T, K, D) * s["topk_w"][:, :, None]).sum(1)
    if c["shared"]:
        y = y + _swiglu_i8(q, sc, s["w13_s"], s["w13_s_scale"], s["w_down_s"],
                           s["w_down_s_scale"])
    return y.to(torch.bfloat16)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    f = lambda t: None if t is None else t.double()  # noqa: E731
    if case["op"] in ("norm_fwd", "norm_bwd"):
        return _exact_norm(case, s, f)
    if case["op"] == "adamw":
        return _exact_adamw(s, f)
    return _exact_ffn_i8(case, s, f)


def _exact_norm(case, s, f):
    T, layer, L = case["T"], case["norm"] == "layer", case["gate_len"]
    gate = f(s["gate"]).repeat_interleave(L, 0)[:T] if L else torch.ones(1, 1, device="cuda",
                                                                        dtype=torch.float64)
    y, r = f(s["y"]), f(s["r"])
    w, b, wp, bp = f(s["w_post"]), f(s["b_post"]), f(s["w_pre"]), f(s["b_pre"])

    def moments(v):
        mu = v.mean(1, keepdim=True) * (1.0 if layer else 0.0)
        return mu, 1.0 / torch.sqrt(((v - mu) ** 2).mean(1, keepdim=True) + NORM_EPS)

    mu, rs = moments(y)
    if not case["post"]:
        mu, rs = torch.zeros_like(mu), torch.ones_like(rs)
    yh = (y - mu) * rs
    z = yh if w is None else yh * w + (0.0 if b is None else b)
    if case["op"] == "norm_fwd":
        # the norm reads the stream as it is stored
        r_out = r + case["alpha"] * gate * z
        kept = r_out.to(s["r"].dtype).double()
        mv, rv = moments(kept)
        x = (kept - mv) * rv * wp + (0.0 if bp is None else bp)
        return {"r_out": r_out, "x": x, "stats": torch.cat([mu, rs, mv, rv], 1)}
    # the statistics are inputs here, as the forward left them
    mu, rs, mv, rv = f(s["stats"]).split(1, 1)
    yh = (y - mu) * rs
    z = yh if w is None else yh * w + (0.0 if b is None else b)
    rh, dx = (r - mv) * rv, f(s["dx"])

    def back(dh, h, rstd):
        mean = dh.mean(1, keepdim=True) if layer else 0.0
        return rstd * (dh - mean - h * (dh * h).mean(1, keepdim=True))

    d = f(s["dr_out"]) + back(dx * wp, rh, rv)
    dz = case["alpha"] * gate * d
    dgate = None
    if L:
        G = s["gate"].shape[0]
        rows = torch.arange(T, device="cuda") // L
        dgate = torch.zeros(G, case["D"], dtype=torch.float64, device="cuda")
        dgate.index_add_(0, rows, case["alpha"] * d * z)
    return {"dy": dz if w is None else back(dz * w, yh, rs), "dr": d,
            "dw_post": None if w is None else (dz * yh).sum(0),
            "db_post": None if b is None else dz.sum(0), "dgate": dgate,
            "dw_pre": (dx * rh).sum(0), "db_pre": None if bp is None else dx.sum(0)}


def _exact_adamw(s, f):
    n = int(s["step"][0]) + 1
    c1, c2 = 1.0 - BETA1 ** n, 1.0 - BETA2 ** n
    scale = float(s["grad_scale"])
    done = []
    for w in s["tensors"]:
        shape, flat = w["param"].shape, w["param"].numel()
        p = f(w["param"] if w["master"] is None else w["master"]).reshape(-1)
        g = f(w["grad"]).reshape(-1) * scale
        m, v = f(w["m"].float()).reshape(-1), f(w["v"].float()).reshape(-1)
        if w["m_scale"] is not None:
            m = m * f(w["m_scale"]).repeat_interleave(BLOCK)[:flat]
            v = (v * f(w["v_scale"]).repeat_interleave(BLOCK)[:flat]) ** 2
        m = BETA1 * m + (1.0 - BETA1) * g
        v = BETA2 * v + (1.0 - BETA2) * g ** 2
        wd = DECAY if w["decay"] else 0.0
        p = p * (1.0 - LR * wd) - LR * (m / c1) / (torch.sqrt(v / c2) + ADAM_EPS)
        t = {"param": p.reshape(shape), "master": None if w["master"] is None else p.reshape(shape),
             "m": None, "v": None, "m_scale": None, "v_scale": None}
        if w["m_scale"] is None:
            t["m"], t["v"] = m.reshape(shape), v.reshape(shape)
        else:
            def top(u):
                short = -flat % BLOCK
                u = torch.cat([u.abs(), u.new_zeros(short)]).reshape(-1, BLOCK).amax(1)
                return torch.where(u >= STATE_MIN, u / E4M3_MAX, torch.zeros_like(u))
            # the 8-bit values are roundings, which have no 64-bit value
            t["m_scale"], t["v_scale"] = top(m), top(torch.sqrt(v))
        done.append(t)
    out = {"step": None}
    for i, t in enumerate(done[:3]):
        out["t%d" % i] = t
    if len(done) > 3:
        for k in done[3]:
            if s["tensors"][3][k] is not None:
                out["vectors_" + k] = (None if done[3][k] is None
                                       else torch.cat([t[k].reshape(-1) for t in done[3:]]))
    return out


def _exact_ffn_i8(case, s, f):
    def quantised(v):
        big = v.abs().amax(1, keepdim=True)
        return torch.round(127.0 * v / big.clamp_min(1e-300)) * (big / 127.0)

    def expert(v, w13, s13, wd, sd):
        a = quantised(v) @ (f(w13) * f(s13)[:, None]).T
        g, u = a.chunk(2, 1)
        return quantised(g / (1.0 + torch.exp(-g)) * u) @ (f(wd) * f(sd)[:, None]).T

    x = f(s["x"])
    y = torch.zeros_like(x)
    for e in range(case["E"]):
        tok, slot = torch.nonzero(s["topk_idx"] == e, as_tuple=True)
        if tok.numel():
            o = expert(x[tok], s["w13"][e], s["w13_scale"][e], s["w_down"][e],
                       s["w_down_scale"][e])
            y.index_add_(0, tok, o * f(s["topk_w"])[tok, slot][:, None])
    if case["shared"]:
        y = y + expert(x, s["w13_s"], s["w13_s_scale"], s["w_down_s"], s["w_down_s_scale"])
    return y


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(case):
    if case["op"] in ("norm_fwd", "norm_bwd"):
        T, D = case["T"], case["D"]
        a, r = (2 if case["dtype"] == "bf16" else 4), (2 if case["resid"] == "bf16" else 4)
        G = -(-T // case["gate_len"]) if case["gate_len"] else 0
        vectors = 4 * D * (1 + G + int(case["post"]) + int(case["bias"]) * (1 + int(case["post"])))
        if case["op"] == "norm_fwd":
            return {"bytes": 2 * T * D * (a + r) + vectors + 16 * T, "flops": 12 * T * D}
        return {"bytes": 3 * T * D * (a + r) + 2 * vectors + 16 * T, "flops": 30 * T * D}
    if case["op"] == "adamw":
        E, D, F = case["E"], case["D"], case["F"]
        vec = sum(D + 7 * i + (i % 3) for i in range(case["extra"]))
        wide, n = E * D + vec, 3 * E * D * F
        total = wide + n
        w = 2 if case["weights"] == "bf16" else 4
        b = wide * 12 + n * (3 * w + (8 if case["master"] else 0) - (w if case["master"] else 0))
        b += total * 16 if case["state"] == "fp32" else total * 4 + 16 * (total // BLOCK + 1)
        return {"bytes": b, "flops": 15 * total}
    T, D, E, K, F = (case[k] for k in ("T", "D", "E", "K", "F"))
    # experts that some token picks, if tokens picked evenly
    used = E * (1.0 - (1.0 - K * (1.0 - case["empty"]) / E) ** T) + int(case["shared"])
    slots = T * (K * (1.0 - case["empty"]) + int(case["shared"]))
    return {"bytes": used * (3 * D * F + 4 * (2 * F + D)) + 4 * T * D + 8 * T * K,
            "flops": 6 * slots * D * F}
