"""What cache_plan and cache_attention allocate themselves: the memory belongs to the
stream that the kernels run on."""

import pytest
import torch

from test_cache_gpu import bf, gla, ints  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["stream", "address"])
def test_memory_comes_from_the_stream_of_the_call(gla, kind):  # noqa: F811
    """What the current stream gave back may still be in use there: a call on another
    stream does not write to it."""
    d, H, n = 64, 2, 100
    cache = gla.rollout_cache(1, 8, H, d, 8, page_tokens=32)
    k, v, q = (bf((n, H, d), 3 + i).cuda() for i in range(3))
    new = ints([n])
    side = torch.cuda.Stream()
    stream = side if kind == "stream" else side.cuda_stream
    torch.cuda.synchronize()
    old = [torch.empty_like(q) for _ in range(3)]
    old += [torch.empty(m, dtype=torch.int32, device="cuda") for m in (1, 2, n) for _ in range(3)]
    given = {x.data_ptr() for x in old}
    del old
    plan = gla.cache_plan(cache, new, n, stream=stream)
    gla.cache_store(cache, plan, k, v, stream=stream)
    out = gla.cache_attention(cache, plan, q, stream=stream)
    torch.cuda.synchronize()
    assert plan.status.item() == 0 and cache.lens.tolist() == [n]
    for x in (plan.cu_tokens, plan.slots, plan.status, out):
        assert x.data_ptr() not in given
    # and the same bits as a call on the current stream, or on the default one by address
    for s in (None, 0):
        again = torch.empty_like(q)
        assert gla.cache_attention(cache, plan, q, out=again, stream=s) is again
        assert torch.equal(again, out)
        assert torch.equal(gla.cache_attention(cache, plan, q, stream=s), out)
