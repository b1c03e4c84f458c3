"""The block norms in float64 numpy, from their formulas (test oracle)."""
from __future__ import annotations

import numpy as np


def draw_inputs(rng, c, post, bias, y=True, several=3.0):
    T, D, L = c["T"], c["D"], c["gate_len"]
    n = rng.normal
    return dict(
        r=n(0.2, several, size=(T, D)), y=n(0.1, 0.8, size=(T, D)) if y else None,
        w_post=n(1.0, 0.2, size=D) if post and y else None,
        b_post=n(0.0, 0.2, size=D) if post and bias and y else None,
        gate=n(0.5, 0.5, size=(-(-T // L), D)) if L and y else None,
        w_pre=n(1.0, 0.2, size=D), b_pre=n(0.0, 0.2, size=D) if bias else None)


def moments(c, v):
    mean = v.mean(1, keepdims=True) if c["norm"] == "layer" else np.zeros((len(v), 1))
    return mean, 1.0 / np.sqrt(((v - mean) ** 2).mean(1, keepdims=True) + c["eps"])


def gate_rows(c, gate):
    return 1.0 if gate is None else gate[np.arange(c["T"]) // c["gate_len"]]


def post(c, y, w_post, b_post):
    """(yh, z, rstd)"""
    if w_post is None:
        return y, y, np.ones((len(y), 1))
    m, s = moments(c, y)
    yh = (y - m) * s
    return yh, yh * w_post + (0.0 if b_post is None else b_post), s


def forward(c, r, y, w_post, b_post, gate, w_pre, b_pre, stream=None):
    """stream: the stored r_out that the second norm reads (else the exact one)."""
    r_out = None
    v = r
    if y is not None:
        r_out = r + c["alpha"] * gate_rows(c, gate) * post(c, y, w_post, b_post)[1]
        v = r_out if stream is None else stream
    x = None
    if w_pre is not None:
        m, s = moments(c, v)
        x = (v - m) * s * w_pre + (0.0 if b_pre is None else b_pre)
    return {"r_out": r_out, "x": x}


def norm_back(c, dh, h, rstd):
    layer = 1.0 if c["norm"] == "layer" else 0.0
    return rstd * (dh - layer * dh.mean(1, keepdims=True) - h * (dh * h).mean(1, keepdims=True))


def backward(c, p, r_out, dx, dr_out):
    """Gradients, and under "abs_..." the sums of the absolute terms that the
    column sums add (their rounding errors are relative to those)."""
    out = {}
    d = np.zeros_like(r_out) if dr_out is None else dr_out.copy()
    if p["w_pre"] is not None:
        m, s = moments(c, r_out)
        rh = (r_out - m) * s
        d = d + norm_back(c, dx * p["w_pre"], rh, s)
        out["dw_pre"], out["db_pre"] = (dx * rh).sum(0), dx.sum(0)
        out["abs_dw_pre"], out["abs_db_pre"] = np.abs(dx * rh).sum(0), np.abs(dx).sum(0)
    out["dr"] = d
    if p["y"] is None:
        return out
    yh, z, s = post(c, p["y"], p["w_post"], p["b_post"])
    da = c["alpha"] * d
    dz = da * gate_rows(c, p["gate"])
    out["dy"] = dz
    if p["w_post"] is not None:
        out["dy"] = norm_back(c, dz * p["w_post"], yh, s)
        out["dw_post"], out["db_post"] = (dz * yh).sum(0), dz.sum(0)
        out["abs_dw_post"], out["abs_db_post"] = np.abs(dz * yh).sum(0), np.abs(dz).sum(0)
    if p["gate"] is not None:
        rows = np.arange(c["T"]) // c["gate_len"]
        for name, term in (("dgate", da * z), ("abs_dgate", np.abs(da) * (
                np.abs(yh) * np.abs(1.0 if p["w_post"] is None else p["w_post"])
                + np.abs(0.0 if p["b_post"] is None else p["b_post"])))):
            out[name] = np.zeros_like(p["gate"])
            np.add.at(out[name], rows, term)
    return out
