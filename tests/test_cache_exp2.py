"""The FMA-pipe 2^x of the cached attention at d = 64 (exp2_poly3_any_x2 in
gla_cache_frame.cuh), emulated in numpy float32 / int32.  That kernel computes the
weights of 64 keys before it knows their maximum and takes the maximum when their
sum reaches 2^15: whatever the argument, an exponential that should be 2^15 or more
has to come out so (or as infinity or NaN), and the others as 2^x."""

import os
import re

import numpy as np

from test_exp2_poly import coeffs, exp2_poly3

HDR = os.path.join(os.path.dirname(__file__), "..", "gated_linear_attention_frame_b200", "csrc",
                   "gla_cache_frame.cuh")


def bounded(x):
    text = open(HDR).read()
    top = np.float32(re.search(r"kExp2Top = ([0-9.]+)f;", text).group(1))
    with np.errstate(over="ignore"):
        return exp2_poly3(np.minimum(np.asarray(x, dtype=np.float32), top))


def test_small_arguments_are_the_same():
    x = np.linspace(-200.0, 120.0, 100001, dtype=np.float32)
    assert np.array_equal(bounded(x), exp2_poly3(x))


def test_large_arguments_stay_large():
    x = np.concatenate([np.linspace(15.01, 700.0, 400001, dtype=np.float32),
                        np.array([1e4, 1e9, 3e38, np.inf], dtype=np.float32)])
    assert np.all(bounded(x) >= 32768.0) and np.all(np.isfinite(bounded(x)))
    # without the bound the exponent runs into the sign bit
    assert np.min(exp2_poly3(np.linspace(129.5, 300.0, 1001, dtype=np.float32))) < 0


def test_the_sum_of_a_pair_of_large_ones_is_seen():
    """0 <= x below the bound: 2^x within 1e-4, so a sum below 2^15 holds no such key."""
    x = np.linspace(8.0, 126.9, 100001, dtype=np.float32)
    want = np.exp2(x.astype(np.float64))
    assert np.max(np.abs(bounded(x) - want) / want) < 1e-4


def scaled(x):
    """Step by step as the kernel does: bounds that hand NaN on, 2^n multiplied in."""
    c0, c1, c2, c3 = coeffs()
    text = open(HDR).read()
    top = np.float32(re.search(r"kExp2Top = ([0-9.]+)f;", text).group(1))
    magic = np.float32(12582912.0)
    x = np.asarray(x, dtype=np.float32)
    x = np.maximum(np.minimum(x, top), np.float32(-126.0))  # numpy's hand NaN on too
    t = (x + magic).astype(np.float32)
    r = (x - (t - magic)).astype(np.float32)
    p = (((c3 * r + c2) * r + c1) * r + c0).astype(np.float32)
    e = (t.view(np.int32) << np.int32(23)) + np.int32(0x3F800000)
    return p * e.view(np.float32)


def test_the_product_is_the_exponent_sum():
    x = np.concatenate([np.linspace(-125.4, 127.0, 200001, dtype=np.float32),
                        np.array([200.0, 1e9, np.inf], dtype=np.float32)])
    assert np.array_equal(scaled(x), bounded(x))
    low = scaled(np.array([-np.inf, -1e30, -200.0, -126.0, -125.7], dtype=np.float32))
    assert np.all(low >= 0) and np.all(low < 1e-37)


def test_nan_stays_nan():
    x = np.array([np.nan, 1.0, -np.nan, np.inf], dtype=np.float32)
    assert np.array_equal(np.isnan(scaled(x)), [True, False, True, False])
