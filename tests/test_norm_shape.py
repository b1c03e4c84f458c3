"""The launch shape of the block norms' forward (csrc/norm_shape.h, compiled
here by itself; no GPU needed): every block fits, with the others of its SM."""
from __future__ import annotations

import ctypes
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mixture_experts_routing_fp32_b200", "csrc")
SM_SMEM, STATIC, SYSTEM, BLOCK_LIMIT = 228 * 1024, 8 * 1024, 1024, 227 * 1024
FIELDS = ("R", "threads", "per_sm", "stages", "grid", "smem", "small", "bias_smem")


@pytest.fixture(scope="module")
def shape(tmp_path_factory):
    d = tmp_path_factory.mktemp("norm_shape")
    (d / "s.cpp").write_text(
        '#include "norm_shape.h"\n'
        'extern "C" void shape(int T, int D, int sms, int piece, int bias, long long* o) {\n'
        "  const auto f = moe::norm_shape::forward(T, D, sms, piece, bias != 0);\n"
        "  const long long v[] = {f.R, f.threads, f.per_sm, f.stages, f.grid, f.smem, f.small,\n"
        "                         f.bias_smem};\n"
        "  for (int i = 0; i < 8; ++i) o[i] = v[i];\n"
        "}\n")
    subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, str(d / "s.cpp"),
                    "-o", str(d / "s.so")], check=True)
    lib, out = ctypes.CDLL(str(d / "s.so")), (ctypes.c_longlong * 8)()

    def of(*a):
        lib.shape(*a, out)
        return dict(zip(FIELDS, out))

    return of


@pytest.mark.parametrize("piece", [32, 48, 64])        # bf16, bf16 with an fp32 stream, fp32
def test_blocks_fit_their_sm(shape, piece):
    for T in (1, 2, 100, 148, 149, 300, 591, 592, 593, 1183, 1200, 5000, 16384, 1 << 30):
        for D in range(8, 8193, 8):
            for bias in (0, 1):
                f = shape(T, D, 148, piece, bias)
                at = (T, D, piece, bias, f)
                row = -(-D // 256) * 32
                assert f["threads"] == f["R"] * row <= 1024, at
                assert 1 <= f["stages"] <= 4, at
                vectors = f["threads"] * 32 * (4 if f["bias_smem"] else 2)
                assert f["smem"] == f["stages"] * piece * f["threads"] + vectors, at
                assert f["smem"] + STATIC <= BLOCK_LIMIT, at
                # what shares an SM: blocks, threads, shared memory
                assert 1 <= f["per_sm"] <= 32, at
                assert f["per_sm"] * f["threads"] <= (1168 if f["small"] else 1024), at
                assert f["per_sm"] * (f["smem"] + STATIC + SYSTEM) <= SM_SMEM, at
                assert 1 <= f["grid"] <= 148 * f["per_sm"] and f["grid"] <= T, at


def test_few_narrow_rows_keep_their_ring(shape):
    """A row per SM: nothing else shares it, whatever the row's width."""
    for T in (1, 148):
        for D in (8, 256, 264, 512, 768, 1280):
            for bias in (0, 1):
                f = shape(T, D, 148, 64, bias)
                assert f["per_sm"] == 1 and f["stages"] == 4 and f["bias_smem"] == bias, (T, D, f)
