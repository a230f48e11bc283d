"""Offsets beyond 32 bits: pages behind the first 4 GB of a pool, and rows behind the
first 2^31 elements of the packed arrays."""

import pytest
import torch

from test_cache_gpu import bf, gla, ints  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("max_new", [1, 1 << 20])
def test_pages_behind_four_gigabytes(gla, max_new):  # noqa: F811
    """The same steps in the last pages of a pool of 4.4 GB a tensor and in a small pool:
    the same codes and, the schedule being the same, the same bits."""
    H, d, P = 24, 128, 64
    outs, codes = [], []
    for pages in (22500, 16):
        assert pages == 16 or pages * H * P * d > 1 << 32
        cache = gla.rollout_cache(2, pages, H, d, 8, page_tokens=P)
        cache.free_pages.copy_(torch.arange(pages, dtype=torch.int32))  # the last page first
        for n in (130, 70):
            plan = gla.cache_plan(cache, ints([n, n]), 2 * n)
            k, v, q = (bf((2 * n, H, d), n + i).cuda() for i in range(3))
            gla.cache_store(cache, plan, k, v)
            out = gla.cache_attention(cache, plan, q, max_new=max_new)
        assert plan.status.item() == 0
        outs.append(out)
        codes.append([x[-16:].clone() for x in (cache.k.view(torch.uint8), cache.v_scale)])
        del cache
    assert torch.equal(*outs)
    assert all(torch.equal(a, b) for a, b in zip(*codes))


@pytest.mark.parametrize("max_new", [1, 1 << 20])
def test_rows_behind_two_to_the_31_elements(gla, max_new):  # noqa: F811
    """A long prompt under a short window, and a second sequence behind it whose rows
    are compared with those of a call of its own."""
    H, Hkv, d, P, long, n = 64, 8, 128, 64, 263000, 90
    N = long + n
    assert long * H * d > 1 << 31
    cache = gla.rollout_cache(2, -(-long // P) + 2, Hkv, d, -(-long // P), page_tokens=P,
                              window_frames=64)
    plan = gla.cache_plan(cache, ints([long, n]), N)
    g = torch.Generator(device="cuda").manual_seed(5)
    k, v, q = (torch.randn(N, h, d, generator=g, device="cuda", dtype=torch.bfloat16)
               for h in (Hkv, Hkv, H))
    gla.cache_store(cache, plan, k, v)
    out = gla.cache_attention(cache, plan, q, max_new=max_new)
    assert plan.status.item() == 0
    small = gla.rollout_cache(1, 2, Hkv, d, 2, page_tokens=P, window_frames=64)
    tail = gla.cache_plan(small, ints([n]), n)
    gla.cache_store(small, tail, k[long:].contiguous(), v[long:].contiguous())
    one = gla.cache_attention(small, tail, q[long:].contiguous(), max_new=max_new)
    # each is off by 2^-8 of itself and 2^-10 sum p |v|, |v| < 8
    assert torch.allclose(out[long:].float(), one.float(), rtol=2 ** -7, atol=2 ** -6)
    assert one.abs().sum() > 0 and torch.isfinite(out[long - 1000:]).all()
    # the first row sees one key, which is itself
    val = cache.v[cache.block_table[0, 0].long(), :, 0].float()
    val = val * cache.v_scale[cache.block_table[0, 0].long()][:, None]
    want = val.repeat_interleave(H // Hkv, 0)
    assert torch.allclose(out[0].float(), want, rtol=2 ** -7, atol=2 ** -8)
