"""The operators around the layer where element offsets pass 32 bits, and
batches of any size: a row's (a token's, an element's) result has the same
bits in a large call as in a small one of its own.
"""
from __future__ import annotations

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from mixture_experts_routing_fp32_b200.build import build
    build()


def test_norm_rows_behind_two_to_the_31():
    import mixture_experts_routing_fp32_b200 as moe
    T, D, n = 270000, 8192, 5                         # 2.2e9 elements a tensor
    g = torch.Generator("cuda").manual_seed(0)
    new = lambda rows: torch.empty(rows, D, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    r, y, dx = (new(T).normal_(generator=g) for _ in range(3))
    w = torch.randn(D, generator=g, device="cuda")

    def step(r, y, dx):
        rows = r.shape[0]
        nc = moe.make_norm_config(rows, D, norm="layer", gate_len=0)
        r_out, x, dy, dr = (new(rows) for _ in range(4))
        stats = torch.empty(rows, 4, device="cuda")
        moe.moe_block_norm(nc, r, y, w, None, None, w, None, r_out, x, stats)
        ws = torch.empty(moe.moe_block_norm_ws_bytes(nc), dtype=torch.uint8, device="cuda")
        moe.moe_block_norm_backward(nc, r_out, y, w, None, None, w, stats, dx, None, dy, dr, None,
                                    None, None, None, None, ws)
        return r_out, x, dy, dr

    big = step(r, y, dx)
    small = step(r[-n:].clone(), y[-n:].clone(), dx[-n:].clone())
    for a, b in zip(big, small):
        assert torch.equal(a[-n:], b)


def test_adamw_elements_behind_two_to_the_31():
    import mixture_experts_routing_fp32_b200 as moe
    n, k = (1 << 31) + 256 * 9 + 17, 256 * 4 + 17     # the last blocks, one cut
    g = torch.Generator("cuda").manual_seed(1)

    def entry(n):
        f8 = lambda: torch.zeros(n, dtype=torch.uint8, device="cuda").view(  # noqa: E731
            torch.float8_e4m3fn)
        nb = -(-n // 256)
        e = {"param": torch.zeros(n, dtype=torch.bfloat16, device="cuda"), "m": f8(), "v": f8(),
             "grad": torch.zeros(n, dtype=torch.bfloat16, device="cuda")}
        e["m_scale"], e["v_scale"] = torch.zeros(nb, device="cuda"), torch.zeros(nb, device="cuda")
        return e

    big, small = entry(n), entry(k)
    for key, std in (("param", 1.0), ("grad", 0.1)):
        small[key].normal_(0, std, generator=g)
        big[key][n - k:] = small[key]
    for e in (big, small):
        step = torch.zeros(2, dtype=torch.int32, device="cuda")
        for _ in range(2):
            moe.moe_adamw(moe.make_adamw_config(lr=0.1), moe.adamw_table([e]), step)
    for key in ("param", "m", "v"):
        a, b = (e[key].view(torch.uint8) if key != "param" else e[key] for e in (big, small))
        assert torch.equal(a[n - k:], b), key
        assert not bool(a[:n - k].any()), key
    for key in ("m_scale", "v_scale"):
        assert torch.equal(big[key][-5:], small[key]), key


def test_quantised_rows_behind_two_to_the_31():
    import mixture_experts_routing_fp32_b200 as moe
    rows, cols = 33000, 65536
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_()
    q = torch.empty(rows, cols, dtype=torch.int8, device="cuda")
    s = torch.empty(rows, device="cuda")
    moe.moe_quant_i8(x, q, s)
    q1, s1 = torch.empty_like(q[:3]), torch.empty_like(s[:3])
    moe.moe_quant_i8(x[-3:], q1, s1)
    assert torch.equal(q[-3:], q1) and torch.equal(s[-3:], s1)


def _experts(T, D, E, K, F, seed, weights=None, x=None, picks=None):
    import mixture_experts_routing_fp32_b200 as moe
    g = torch.Generator("cuda").manual_seed(seed)
    if weights is None:
        weights = []
        for shape in ((E, 2 * F, D), (E, D, F)):
            weights.append(torch.empty(shape, dtype=torch.int8, device="cuda").random_(
                -127, 128, generator=g))
            weights.append((torch.rand(shape[:-1], generator=g, device="cuda") + 0.5)
                           / (73.0 * shape[-1] ** 0.5))
    if x is None:
        x = torch.empty(T, D, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
        top = torch.rand(T, E, generator=g, device="cuda").topk(K, 1)
        picks = top.indices.to(torch.int32), torch.softmax(top.values, 1)
    layer = moe.MoEInt8Layer(moe.make_config(T, D, E, K, F))
    layer.set_weights(*weights)
    y = layer.experts(x, *picks).clone()
    assert moe.moe_check_status() == 0
    return y, weights, x, picks


@pytest.mark.parametrize("T,D,E,K,F", [(5000, 384, 8, 4, 256),    # many-block dispatch, pairs
                                       (700, 256, 16, 2, 384),    # single tiles
                                       (60, 512, 16, 4, 128)])    # the few-row form
def test_a_token_does_not_depend_on_its_batch(T, D, E, K, F):
    """Every form of the products gives a token the same bits: integer sums
    are exact and the rest is done per row in one order."""
    y, weights, x, (idx, w) = _experts(T, D, E, K, F, 2)
    for rows in ([0], [T // 2], list(range(T - 40, T))):
        n = len(rows)
        part = _experts(n, D, E, K, F, 0, weights, x[rows].contiguous(),
                        (idx[rows].contiguous(), w[rows].contiguous()))[0]
        assert torch.equal(part, y[rows]), rows[:1]


def test_expert_rows_behind_two_to_the_31():
    """h of 2.3e9 elements: the last tokens as in a call of their own."""
    T, D, E, K, F = 80000, 256, 8, 2, 14336
    y, weights, x, (idx, w) = _experts(T, D, E, K, F, 3)
    rows = list(range(T - 20, T))
    part = _experts(20, D, E, K, F, 0, weights, x[rows].contiguous(),
                    (idx[rows].contiguous(), w[rows].contiguous()))[0]
    assert torch.equal(part, y[rows])
