"""Query rows that hold NaN or infinity, at both widths and in both kernels: the
row's result is not finite however few keys it sees, and the other rows' results
do not change beyond a rounding."""

import pytest
import torch

from test_cache_gpu import Cache, bf, gla, ints  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("max_new", [1, 1 << 20])
@pytest.mark.parametrize("d", [64, 128])
def test_broken_rows_that_see_few_keys(gla, d, max_new, value):  # noqa: F811
    """Causal rows from the first token on: row 0 sees one key, row 1 two, and so on;
    rows 64 and 65 are the first of the second 64 keys."""
    P, H, n = 32, 2, 150
    c = Cache(8, 1, P, d, 8, range(8))
    c.add(0)
    k = bf((n, 1, d), 1)
    k[:, :, 5] = 1.0 if value > 0 else -1.0  # an infinite query's scores are +inf
    c.step(gla, [n], k, bf((n, 1, d), 2))
    q = bf((n, H, d), 3).cuda()
    args = (c.k8, c.v8, c.ks, c.vs, c.tables(), ints(c.lens), ints([0, n]), None)
    tail = (1, n, max_new, H, 1, d, 8, P, 8, 1, 0, 0, d ** -0.5)
    good, out = torch.empty_like(q), torch.empty_like(q)
    gla.gla_cache_attention(q, *args, good, *tail)
    rows = torch.ones(n, H, dtype=torch.bool, device="cuda")
    for t, h in ((0, 0), (1, 1), (9, 0), (64, 1), (65, 0), (128, 0), (129, 1), (140, 1)):
        q[t, h, 5] = value
        rows[t, h] = False
    gla.gla_cache_attention(q, *args, out, *tail)
    assert torch.isfinite(good).all() and torch.isfinite(out[rows]).all()
    # the reference that a broken row makes its neighbours take again moves them by a
    # rounding: both are within 2^-8 of themselves and 2^-10 sum p |v| of the truth
    assert torch.allclose(out[rows].float(), good[rows].float(), rtol=2 ** -6, atol=2 ** -7)
    assert not torch.isfinite(out[~rows]).any()
