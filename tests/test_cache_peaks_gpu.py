"""Peaked scores in the cached attention: keys that exceed what a row has seen
before by far, at every place of a tile, so that the row's reference has to be
replaced (csrc/gla_cache_frame.cuh), in both kernels and at both widths.

The bound, per element, beside those of test_cache_gpu.py (2^-8 |ref| for the
rounding of out, 2^-10 sum p |v| for the weights, 2^-20 max |v|): a score is a
sum of d products in fp32, off by at most (d + 2) 2^-24 of sum |q k| scale, and
its reference shift by 2^-23 of its size; a weight's relative error is the
difference of two of those, and here sum |q k| scale <= 1.5 max |score|:
  2 * (1.5 (d + 2) + 2) 2^-24 max |score|  of  sum p |v|
"""

import numpy as np
import pytest
import torch

import oracle
from test_cache_gpu import Cache, bf, gla, ints  # noqa: F401

pytestmark = pytest.mark.gpu

FRAME, TOKEN = 1 << 20, 1  # the hint that picks each kernel


def compare(gla, c, new, q, max_new, scale, top):  # noqa: F811
    """q [sum(new), H, d] against the oracle; `top`: largest |score| in nats."""
    pages, Hkv, P, d = c.shape
    N, H = q.shape[:2]
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    out = torch.full(q.shape, 55.0, dtype=torch.bfloat16, device="cuda")
    table = c.tables()
    gla.gla_cache_attention(q.cuda(), c.k8, c.v8, c.ks, c.vs, table, ints(c.lens), ints(cu), None,
                            out, len(new), N, max_new, H, Hkv, d, pages, P, c.width, 1, 0, 0,
                            scale)
    ref, mag = oracle.cache_attention(q.double().numpy(), *(np.nan_to_num(x) for x in c.ref + c.sc),
                                      table.tolist(), c.lens, cu, P, scale=scale)
    vmax = np.nanmax(np.abs(c.ref[1]) * c.sc[1][:, :, None, None])
    weights = 2.0 ** -10 + 2 * (1.5 * (d + 2) + 2) * 2.0 ** -24 * top
    bound = 2.0 ** -8 * np.abs(ref) + weights * mag + 2.0 ** -20 * vmax
    err = np.abs(out.double().cpu().numpy() - ref)
    bad = np.argwhere(~(err <= bound))
    assert not len(bad), "row %s off by %.3g, bound %.3g" % (
        bad[0], err[tuple(bad[0])], bound[tuple(bad[0])])


def peaked(lib, d, places, gaps, P, len_, new):
    """A cache of one sequence for each (place, gap), of len_ tokens: unit normal
    keys of score scale 1 / sqrt(d) for queries of 4, but for one key of all c at
    the place, whose score is the gap (log2 units)."""
    R = len(places) * len(gaps)
    pages = -(-len_ // P)
    c = Cache(R * pages, 1, P, d, pages, range(R * pages))
    for _ in range(R):
        c.add(0)
    k, v = bf((R * len_, 1, d), d), bf((R * len_, 1, d), d + 1)
    k = k.float() * 0.25  # ordinary scores: |.| about 1 nat, at most about 5
    for i, (at, gap) in enumerate((a, b) for a in places for b in gaps):
        k[i * len_ + at] = gap / 1.4427 / (4 * d ** 0.5)
    c.step(lib, [len_] * R, k.bfloat16(), v)
    q = torch.full((R * new, 1, d), 4.0).bfloat16()
    return c, [new] * R, q


GAPS = [20.0, 100.0, 130.0, 150.0, 270.0, 400.0, 600.0]


@pytest.mark.parametrize("max_new", [FRAME, TOKEN])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("first", [64, 128, 200])
def test_one_key_far_above_the_rest(gla, d, max_new, first):  # noqa: F811
    """At each place of eight neighbouring keys: in the second half of the first
    tile, at the start of the second tile and inside it."""
    c, new, q = peaked(gla, d, range(first, first + 8), GAPS, 16, 270, 4)
    compare(gla, c, new, q, max_new, d ** -0.5, 430.0)


@pytest.mark.parametrize("max_new", [FRAME, TOKEN])
@pytest.mark.parametrize("d", [64, 128])
def test_scores_that_climb_from_tile_to_tile(gla, d, max_new):  # noqa: F811
    """Every key above all keys before it: the reference moves in each half of
    each tile, by 64 keys at a time (steps of up to about 460 in all)."""
    P, n = 32, 320
    c = Cache(2 * n // P, 1, P, d, n // P, range(2 * n // P))
    c.add(0)
    c.add(0)
    k = torch.arange(n).float()[:, None, None] * torch.tensor([0.03, 0.005])[None, :, None]
    k = k.permute(1, 0, 2).reshape(2 * n, 1, 1).expand(-1, -1, d) / (d ** 0.5 / 8)
    c.step(gla, [n, n], k.bfloat16(), bf((2 * n, 1, d), 5))
    q = torch.full((2 * 70, 1, d), 4.0).bfloat16()
    compare(gla, c, [70, 70], q, max_new, d ** -0.5, 320.0)


@pytest.mark.parametrize("max_new", [FRAME, TOKEN])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("gap", [0.0, 40.0, 80.0, 120.0])
def test_a_reference_from_values_that_are_all_zero(gla, d, max_new, gap):  # noqa: F811
    """128 tokens with values of 0 (the least scale, 2^-60), and rows whose only
    keys behind them are the first one or two of the next tile; 32 heads share the
    keys, so that whole warps hold such rows alone."""
    P = 16
    c = Cache(36, 1, P, d, 9, range(36))
    new = [1, 2, 1, 2]
    for _ in new:
        c.add(0)
    k, v = bf((4 * 128, 1, d), 7).float() * 0.25, torch.zeros(4 * 128, 1, d)
    c.step(gla, [128] * 4, k.bfloat16(), v.bfloat16())
    k = torch.full((6, 1, d), gap / 1.4427 / (4 * d ** 0.5))
    c.step(gla, new, k.bfloat16(), bf((6, 1, d), 8))
    q = torch.full((6, 32, d), 4.0).bfloat16()
    compare(gla, c, new, q, max_new, d ** -0.5, 90.0)
