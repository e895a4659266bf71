"""CPU replay, in fp32 as on the GPU, of the ends of the software exp2 of the dense attention's tile kernel: what a score
far below the reference, -infinity, one above it and NaN give."""
import re

import numpy as np
import torch

from tests.test_exp2_poly import ROOT, coefficients


def replay(x):
    src = open(f"{ROOT}/block_sparse_online_b200/csrc/ptx_sm100.cuh").read()
    body = src[src.index("exp2_poly_nan_x2(float"):]
    low, high = re.search(r'"f"\((-[0-9.]+)f\), "f"\(([0-9.]+)f\)', body).groups()
    f = np.float32
    c0, c1, c2, c3 = coefficients()
    x = np.asarray(x, dtype=f)
    a = np.where(np.isnan(x), x, np.minimum(np.maximum(x, f(low)), f(high)))  # the clamps hand a NaN through
    shift = f(12582912.0)
    t = a + shift
    fr = a - (t - shift)
    p = ((c3 * fr + c2) * fr + c1) * fr + c0
    with np.errstate(over="ignore"):
        nan = np.int32(0x7fffffff)  # the NaN that the GPU's 32-bit arithmetic gives
        pb, tb = (np.where(np.isnan(v), nan, v.view(np.int32)) for v in (p, t))
        bits = (pb + (tb << 23)).astype(np.int32)
    return bits.view(f)


def test_no_weight_at_minus_infinity():
    y = replay([-np.inf, -1e30, -200.0, -127.0])
    assert (y >= 0).all() and (y < 2.0 ** -134).all()
    for t in (torch.bfloat16, torch.float16):  # what the product sees
        assert (torch.from_numpy(y.copy()).to(t) == 0).all()


def test_exact_down_to_the_normal_range_and_never_above_it_below():
    # (up to 1e-4 above -126 the cubic is below 1 and its sum a subnormal that holds 2 p - 1: twice the error)
    x = np.linspace(-125.9998, 0.0, 400_001, dtype=np.float32)
    true = np.exp2(x.astype(np.float64))
    assert (np.abs(replay(x) / true - 1) <= 7.6e-5).all()
    x = np.linspace(-130.0, -125.9998, 100_001, dtype=np.float32)
    y = replay(x).astype(np.float64)
    assert (y >= 0).all() and (np.diff(y) >= -2.0 ** -140).all()
    assert (np.abs(y - np.exp2(x.astype(np.float64))) <= 2.0 ** -127).all()


def test_large_scores_and_nan_show_in_the_sum():
    x = np.array([20.0, 100.0, 126.0, 1000.0, np.inf], dtype=np.float32)
    y = replay(x)
    assert (y[:3] / np.exp2(x[:3].astype(np.float64)) - 1 < 1e-4).all() and (y[3:] > 2.0 ** 125).all()
    assert replay([np.nan])[0] > 2.0 ** 127
