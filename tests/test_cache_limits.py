"""Limits of the cached attention's arguments: score scales that fp32 cannot hold in
base 2 are refused (CPU), scores up to the documented magnitude are answered (GPU)."""

import pytest
import torch

from test_cache_abi import attend, lib  # noqa: F401
from test_cache_gpu import Cache, bf, gla  # noqa: F401
from test_cache_peaks_gpu import FRAME, TOKEN, compare


@pytest.mark.parametrize("scale,fits", [(3.4e38, False), (2.4e38, False), (2.3e38, True),
                                        (1e-45, True), (0.0, False)])
def test_scales_beyond_base_two(lib, scale, fits):  # noqa: F811
    import gated_linear_attention_frame_b200 as g

    # (a scale that fits goes on to the next check, of the misaligned q)
    want = g.GLA_ERR_ALIGN if fits else g.GLA_ERR_SHAPE
    assert attend(lib, scale=scale, q=(1 << 20) + 8) == want


@pytest.mark.gpu
@pytest.mark.parametrize("top", [2.0 ** 16, 2.0 ** 20, 2.0 ** 22])
@pytest.mark.parametrize("sign", [1.0, -1.0])
@pytest.mark.parametrize("max_new", [FRAME, TOKEN])
@pytest.mark.parametrize("d", [64, 128])
def test_large_scores(gla, d, max_new, sign, top):  # noqa: F811
    """Pages of 16 equal keys that grow (or fall, for negative queries) by 1/15 or
    more of themselves: the largest page a row sees has all its weight, in equal
    parts (equal scores), whatever the scores' own rounding."""
    P, n = 16, 300
    c = Cache(20, 1, P, d, 19, range(20))
    c.add(0)
    j = torch.arange(n) // P
    k = ((8 + j % 8) * torch.exp2((j // 8).float()))[:, None, None].expand(-1, -1, d)
    c.step(gla, [n], k.bfloat16(), bf((n, 1, d), 2))
    q = torch.full((150, 1, d), sign).bfloat16()
    # the largest |score| is top, in log2 units
    compare(gla, c, [150], q, max_new, top / 1.4427 / (float(k.max()) * d), 0.0)
