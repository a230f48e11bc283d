"""Pins of the rollout-cache oracle (CPU): the e4m3 rounding against torch's
conversion, the page scale at its borders, the plan's page bookkeeping over a
whole rollout, and the cached attention against the anchor layer's oracle."""

import math
import random

import numpy as np
import pytest
import torch

import oracle


def test_e4m3_round_matches_the_format():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    vals = np.unique(codes[np.isfinite(codes)])
    assert vals.max() == 448.0
    assert np.array_equal(oracle.e4m3_round(vals), vals)
    mid = (vals[1:] + vals[:-1]) / 2  # ties go to the even code
    x = np.concatenate([mid, mid * (1 + 1e-7), mid * (1 - 1e-7), [500.0, -1e30, 1e-12]])
    ref = torch.tensor(x).clamp(-448, 448).to(torch.float8_e4m3fn).double().numpy()
    # torch converts through fp32: leave out what that rounding moves onto a tie
    keep = np.float32(x).astype(np.float64) == x
    assert keep.sum() >= mid.size
    assert np.array_equal(oracle.e4m3_round(x)[keep], ref[keep])


def test_page_scale_borders():
    assert oracle.page_scale(448.0) == 1.0
    assert oracle.page_scale(math.nextafter(448.0, 1e9)) == 2.0
    assert oracle.page_scale(224.0) == 0.5
    assert oracle.page_scale(0.0) == 2.0 ** -60
    assert oracle.page_scale(1e38) == 2.0 ** 60


@pytest.mark.parametrize("P,F,W,sink", [(16, 1, 0, 0), (16, 40, 2, 20), (32, 7, 3, 0),
                                        (64, 1, 100, 5)])
def test_plan_never_loses_or_doubles_a_page(P, F, W, sink):
    rng = random.Random(P * 100 + F)
    R, pages, width = 5, 120, 60
    st = dict(lens=[0] * R, held=[0] * R, free_count=pages, table=[[-1] * width for _ in range(R)],
              stack=list(range(pages)))
    for _ in range(40):
        new = [rng.choice([0, 1, F, rng.randint(0, 30), -1 if rng.random() < 0.2 else 1])
               for _ in range(R)]
        o = oracle.cache_plan(st["lens"], st["held"], new, st["stack"], st["free_count"],
                              st["table"], pages, P, 400, F, W, sink)
        if o["status"]:
            assert o["status"] in (1, 4, 5)
            st["lens"] = st["lens"][:]
            new = [-1] * R  # start again
            o = oracle.cache_plan(st["lens"], st["held"], new, st["stack"], st["free_count"],
                                  st["table"], pages, P, 400, F, W, sink)
        assert o["status"] == 0
        sp = -(-sink // P)
        used = []
        for r in range(R):
            have = -(-o["lens"][r] // P)
            used += [o["table"][r][j] for j in range(have) if j < sp or j >= o["held"][r]]
            # the window of the step's first query is still there
            if new[r] > 0 and W:
                lo = max(0, ((o["lens"][r] - new[r]) // F - W + 1) * F)
                assert all(j >= o["held"][r] for j in range(max(sp, lo // P), have))
        assert len(set(used)) == len(used)
        assert sorted(used + o["stack"][:o["free_count"]]) == list(range(pages))
        st = o


def test_attention_equals_the_anchor_layer_on_exact_codes():
    """Keys and values that e4m3 holds exactly: the cached attention of a frame
    is the anchor layer's for that frame."""
    rng = np.random.default_rng(3)
    T, frames, W, sink, P, d = 10, 4, 2, 13, 16, 8
    n = T * frames
    q = rng.standard_normal((n, d))
    k = oracle.e4m3_round(rng.standard_normal((n, d)))
    v = oracle.e4m3_round(rng.standard_normal((n, d)))
    ref = oracle.softmax_anchor_head(q, k, v, T, W, sink)
    pages = -(-n // P)
    order = list(rng.permutation(pages))
    kc, vc = np.zeros((pages, 1, P, d)), np.zeros((pages, 1, P, d))
    for s in range(n):
        kc[order[s // P], 0, s % P], vc[order[s // P], 0, s % P] = k[s], v[s]
    one = np.ones((pages, 1))
    for f in range(frames):
        got, mag = oracle.cache_attention(q[f * T:(f + 1) * T, None], kc, vc, one, one, [order],
                                          [(f + 1) * T], [0, T], P, T, W, sink)
        assert np.allclose(got[:, 0], ref[f * T:(f + 1) * T], rtol=1e-12, atol=1e-12)
        assert np.all(mag >= np.abs(got) - 1e-12)


def test_store_grows_a_page_and_keeps_its_tokens():
    P, d = 16, 4
    codes, scales = np.zeros((2, 1, P, d)), np.ones((2, 1))
    a = np.full((3, 1, d), 1.0)
    oracle.cache_store(a, [16, 17, 18], [0, 3], codes, scales, P)
    assert scales[1, 0] == 2.0 ** -8 and np.all(codes[1, 0, :3] == 256.0)
    oracle.cache_store(np.full((1, 1, d), 100.0), [19], [0, 1], codes, scales, P)
    assert scales[1, 0] == 0.25 and np.all(codes[1, 0, :3] * 0.25 == 1.0)
    assert np.all(codes[1, 0, 3] == 384.0)  # 400 lies between 12 * 32 and 13 * 32: the even one
    x = np.full((1, 1, d), np.nan)
    x[0, 0, 0] = np.inf
    oracle.cache_store(x, [20], [0, 1], codes, scales, P)
    assert scales[1, 0] == 0.25
    assert list(codes[1, 0, 4]) == [448.0, 0.0, 0.0, 0.0]
