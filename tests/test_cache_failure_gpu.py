"""A bounded wait of the cached attention of many queries runs out, without a GPU
fault: the wait limit is lowered to a few milliseconds and the first CTA withholds the
codes of one tile (gla_inject_stall), so that nothing ever arrives on that tile's
barrier.  Every role of the kernel must give up, its copies land and its tensor
memory go back; bit 8 of the fault word says so, and the next calls, on the same SMs,
give the right bits with no fault."""

import pytest
import torch

from test_cache_gpu import bf, gla, ints  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture
def hooks(gla):  # noqa: F811
    yield gla
    gla.gla_set_wait_limit_ns(0)
    gla.gla_inject_stall(-1)


# 128 heads x 3 units of 256 rows over 6, 8 and 10 tiles of keys, 384 units on (at most)
# 148 CTAs: the first CTA has the first unit and most of the second (tile 9 is in it)
@pytest.mark.parametrize("tile", [0, 1, 9])
@pytest.mark.parametrize("d", [64, 128])
def test_a_wait_that_runs_out_is_reported_and_recovered(hooks, d, tile):
    H, old, n = 128, 500, 700
    cache = hooks.rollout_cache(1, 24, H, d, 24, page_tokens=64)
    for m in (old, n):
        plan = hooks.cache_plan(cache, ints([m]), m)
        k, v = (bf((m, H, d), d + m + i).cuda() for i in range(2))
        hooks.cache_store(cache, plan, k, v)
    q = bf((n, H, d), 9).cuda()
    good = hooks.cache_attention(cache, plan, q)
    torch.cuda.synchronize()
    assert hooks.gla_device_fault() == 0
    hooks.gla_set_wait_limit_ns(5_000_000)  # 5 ms
    hooks.gla_inject_stall(tile)
    hooks.cache_attention(cache, plan, q)
    torch.cuda.synchronize()  # the call's kernels returned
    fault = hooks.gla_device_fault()
    hooks.gla_set_wait_limit_ns(0)
    assert fault == 256, "the kernel did not report its wait (fault word %#x)" % fault
    for _ in range(2):
        assert torch.equal(hooks.cache_attention(cache, plan, q), good)
    assert hooks.gla_device_fault() == 0
