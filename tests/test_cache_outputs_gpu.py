"""What cache_plan and cache_attention allocate themselves: the memory belongs to the
stream that the kernels run on, and every row of a result holds something."""

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


def leave_garbage(shape):
    """The allocator's next block of this size holds NaN."""
    x = torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    del x


@pytest.mark.parametrize("max_new", [1, 1 << 20])
def test_rows_of_no_sequence_are_zero(gla, max_new):  # noqa: F811
    """Rows behind the last sequence, and all rows of a step that does not fit."""
    d, H, N = 64, 4, 200
    cache = gla.rollout_cache(2, 8, 2, d, 4, page_tokens=32)
    k, v, q = (bf((N, h, d), 3 + i).cuda() for i, h in enumerate((2, 2, H)))
    plan = gla.cache_plan(cache, ints([50, 70]), N)
    gla.cache_store(cache, plan, k, v)
    leave_garbage(q.shape)
    out = gla.cache_attention(cache, plan, q, max_new=max_new)
    assert plan.status.item() == 0
    assert out[:120].abs().sum() > 0 and torch.isfinite(out[:120]).all()
    assert out[120:].eq(0).all()
    # the second sequence would need a fifth page: nothing is attended
    plan = gla.cache_plan(cache, ints([1, 60]), N)
    gla.cache_store(cache, plan, k, v)
    leave_garbage(q.shape)
    out = gla.cache_attention(cache, plan, q, max_new=max_new)
    assert plan.status.item() == 4 and out.eq(0).all()
    # a caller's own rows stay as they are
    own = torch.full_like(q, 3.0)
    assert gla.cache_attention(cache, plan, q, out=own, max_new=max_new) is own
    assert own.eq(3).all()
