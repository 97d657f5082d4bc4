"""moe_swiglu_fp8 at gates where 1 / (1 + exp(-g)) leaves float32: every finite bf16 gate, float32 gates from
where silu falls below the smallest normal number to the lowest one, infinities and NaN."""
import numpy as np
import pytest
import torch

import combine_topk_ids_gb300 as moe
from oracle import grouped as og
from oracle.block import E4M3, EPS32
from test_grouped_gpu import BF, F32, F8, built, f64, within  # noqa: F401

pytestmark = pytest.mark.gpu

# silu(g) is below 2^-119 where 1 / (1 + exp(-g)) is below the smallest normal float32, 2^-126 (g < -87.3):
# it may be 0 there
TINY = 2.0 ** -119


def each_beside(gates, up=1.0):
    """Rows of one block: a gate each in column 0 (its up: `up`), and 127 gates of 1 with up 2^-10."""
    x = torch.ones((len(gates), 256), dtype=gates.dtype, device="cuda")
    x[:, 0], x[:, 128:], x[:, 128] = gates.cuda(), 2.0 ** -10, up
    codes, scales = torch.empty((len(x), 128), dtype=F8, device="cuda"), torch.empty((len(x), 1), device="cuda")
    moe.moe_swiglu_fp8(x, codes, scales)
    with np.errstate(invalid="ignore", over="ignore"):
        v, rel = og.swiglu(f64(x))
    return v, rel, f64(codes.float()), f64(scales)


def check(gates, up=1.0):
    v, rel, codes, scales = each_beside(gates, up)
    top = np.maximum(np.abs(v).max(1, keepdims=True), 2.0 ** -100)
    within(scales, top / 448, (rel + EPS32) * top / 448 + TINY * abs(up), "scales")
    # half a code in the normal range, half the smallest step (2^-10) below it
    within(codes * scales, v, (E4M3 + 2 * rel) * np.abs(v) + 2.0 ** -10 * 1.001 * scales + TINY * abs(up), "codes")


def test_every_finite_bf16_gate():
    bits = torch.arange(1 << 16, dtype=torch.int32)
    gates = (bits << 16).view(F32)
    gates = gates[gates.isfinite()].to(BF)
    assert len(gates) == 2 * 255 * 128
    check(gates)


@pytest.mark.parametrize("up", [1.0, -3.0])
def test_float32_gates_far_out(up):
    far = -torch.logspace(np.log10(80.0), np.log10(3.4028e38), 4000, dtype=torch.float64).float()
    low = torch.tensor([-87.0, -87.3, -87.34, -87.4, -88.0, -88.7, -88.72, -88.73, -88.8, -89.0, -103.0, -104.0, -1e3, -1e10, -1e20,
                        -1e30, -1e35, -1e38, -2.3e38, -2.4e38, -3e38, torch.finfo(F32).min])
    # positive ones with a product that stays finite (3 * 1e38 < 3.4e38)
    high = torch.cat([torch.logspace(np.log10(80.0), 38, 400, dtype=torch.float64).float(), -low[low > -1.1e38]])
    check(torch.cat([far, low]), up)
    check(high, up)
    if up == 1.0:
        check(torch.tensor([2.3e38, 2.36e38, 2.4e38, 3e38, torch.finfo(F32).max]))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_infinite_gates_and_nan(dtype):
    """-inf / (1 + exp(inf)) is not a number: it marks its own code.  +inf stays, and its block becomes NaN."""
    low, nan, high = [each_beside(torch.tensor([g], dtype=dtype)) for g in (-float("inf"), float("nan"), float("inf"))]
    for v, rel, codes, scales in (low, nan):
        assert np.isnan(codes[0, 0]) and np.isfinite(codes[0, 1:]).all()
        within(codes[0, 1:] * scales[0], v[0, 1:], (E4M3 + 2 * rel) * np.abs(v[0, 1:]) + 2.0 ** -10 * 1.001 * scales[0], "beside")
    with np.errstate(invalid="ignore"):      # codes of 0 by an infinite scale
        assert np.isnan(high[2] * high[3]).all()
