"""Refusals of the rollout-cache entry points, on the CPU: the library rejects
bad arguments before any CUDA call, the wrappers reject tensors that do not fit
the sizes they are passed with."""

import pytest
import torch

FAKE = 1 << 20  # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    from gated_linear_attention_frame_b200.build import build

    build()
    import gated_linear_attention_frame_b200 as g

    return g.load_library()


PLAN = ["lens", "held", "new_lens", "free_count", "free_pages", "block_table", "lens_out",
        "held_out", "free_count_out", "cu_tokens", "slots", "status"]
STORE = ["k", "v", "lens", "cu_tokens", "slots", "k_cache", "v_cache", "k_scale", "v_scale",
         "nonfinite"]
ATT = ["q", "k_cache", "v_cache", "k_scale", "v_scale", "block_table", "lens", "cu_tokens",
       "gate_z", "out"]


def plan(lib, R=2, max_pages=4, pages=8, P=16, tokens=8, F=1, W=0, sink=0, **kw):
    return lib.gla_cache_plan(*[kw.get(n, FAKE) for n in PLAN], R, max_pages, pages, P, tokens, F,
                              W, sink, None)


def store(lib, R=2, tokens=8, H=2, d=128, pages=8, P=16, **kw):
    kw.setdefault("nonfinite", None)
    return lib.gla_cache_store(*[kw.get(n, FAKE) for n in STORE], R, tokens, H, d, pages, P, None)


def attend(lib, R=2, tokens=8, max_new=4, H=4, Hkv=2, d=128, pages=8, P=16, max_pages=4, F=1, W=0,
           sink=0, scale=0.1, **kw):
    kw.setdefault("gate_z", None)
    return lib.gla_cache_attention(*[kw.get(n, FAKE) for n in ATT], R, tokens, max_new, H, Hkv, d,
                                   pages, P, max_pages, F, W, sink, scale, None)


def test_plan_refusals(lib):
    import gated_linear_attention_frame_b200 as g

    for bad in (dict(R=-1), dict(R=8193), dict(tokens=-1), dict(pages=-1), dict(max_pages=-1),
                dict(P=8), dict(P=48), dict(P=256), dict(F=0), dict(W=-1), dict(sink=-1),
                dict(pages=1 << 27), dict(max_pages=1 << 27), dict(tokens=(1 << 30) + 1)):
        assert plan(lib, **bad) == g.GLA_ERR_SHAPE, bad
    for name in PLAN:
        assert plan(lib, **{name: None}) == g.GLA_ERR_NULL, name
        assert plan(lib, **{name: FAKE + 2}) == g.GLA_ERR_ALIGN, name


def test_store_refusals(lib):
    import gated_linear_attention_frame_b200 as g

    for bad in (dict(R=-1), dict(R=8193), dict(tokens=-1), dict(pages=-1), dict(P=24),
                dict(H=-1), dict(H=1 << 17), dict(pages=1 << 27)):
        assert store(lib, **bad) == g.GLA_ERR_SHAPE, bad
    for d in (32, 96, 256, 0):
        assert store(lib, d=d) == g.GLA_ERR_UNSUPPORTED_D
    for name in STORE[:-1]:
        assert store(lib, **{name: None}) == g.GLA_ERR_NULL, name
    for name in ("k", "v", "k_cache", "v_cache"):
        assert store(lib, **{name: FAKE + 8}) == g.GLA_ERR_ALIGN, name
    for name in ("lens", "cu_tokens", "slots", "k_scale", "v_scale", "nonfinite"):
        assert store(lib, **{name: FAKE + 2}) == g.GLA_ERR_ALIGN, name
    for nothing in (dict(R=0), dict(tokens=0), dict(H=0), dict(pages=0)):
        assert store(lib, k=None, **nothing) == g.GLA_OK, nothing


def test_attention_refusals(lib):
    import gated_linear_attention_frame_b200 as g

    for bad in (dict(R=-1), dict(R=8193), dict(tokens=-1), dict(pages=-1), dict(P=0),
                dict(max_new=-1), dict(H=-4), dict(Hkv=0), dict(Hkv=3), dict(H=129, Hkv=1),
                dict(max_pages=-1), dict(max_pages=1 << 27), dict(F=0), dict(W=-2), dict(sink=-1),
                dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
                dict(scale=float("inf"))):
        assert attend(lib, **bad) == g.GLA_ERR_SHAPE, bad
    for d in (32, 96, 256, 0):
        assert attend(lib, d=d) == g.GLA_ERR_UNSUPPORTED_D
    for name in ATT:
        if name != "gate_z":
            assert attend(lib, **{name: None}) == g.GLA_ERR_NULL, name
    for name in ("q", "k_cache", "v_cache", "gate_z", "out"):
        assert attend(lib, **{name: FAKE + 8}) == g.GLA_ERR_ALIGN, name
    for name in ("k_scale", "v_scale", "block_table", "lens", "cu_tokens"):
        assert attend(lib, **{name: FAKE + 2}) == g.GLA_ERR_ALIGN, name
    for nothing in (dict(R=0), dict(tokens=0), dict(H=0, Hkv=0)):
        assert attend(lib, q=None, **nothing) == g.GLA_OK, nothing


def test_wrappers_check_kind_and_size(lib):
    import gated_linear_attention_frame_b200 as g

    x = torch.zeros(8, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA device"):
        g.gla_cache_store(x, x, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, 2, 8, 2, 128, 8, 16)
    with pytest.raises(TypeError, match="bfloat16"):
        g.gla_cache_store(x.float(), x, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, 2, 8, 2,
                          128, 8, 16)
    with pytest.raises(TypeError, match="int address"):
        g.gla_cache_store([1], x, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, 2, 8, 2, 128, 8,
                          16)
    with pytest.raises(g.GLAError) as e:
        g.gla_cache_attention(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, FAKE, 2, 8, 4,
                              4, 3, 128, 8, 16, 4, 1, 0, 0, 0.1)
    assert e.value.status == g.GLA_ERR_SHAPE and "gla_cache_attention" in str(e.value)
    with pytest.raises(ValueError, match="page_tokens"):
        g.rollout_cache(1, 1, 1, 128, 1, page_tokens=48, device="cpu")
    with pytest.raises(ValueError, match="d must be"):
        g.rollout_cache(1, 1, 1, 32, 1, device="cpu")
    c = g.rollout_cache(2, 6, 1, 64, 3, page_tokens=16, device="cpu")
    assert c.free_pages.tolist() == [5, 4, 3, 2, 1, 0] and c.free_count.tolist() == [6]
    assert c.block_table.eq(-1).all() and c.page_tokens == 16
    two = c.layer()
    assert two.lens is c.lens and two.k is not c.k and two.k.shape == c.k.shape
    p = g.CachePlan(torch.zeros(3, dtype=torch.int32), torch.zeros(5, dtype=torch.int32), None)
    with pytest.raises(ValueError, match="k, v must be"):
        g.cache_store(c, p, torch.zeros(4, 1, 64), torch.zeros(4, 1, 64))
    with pytest.raises(ValueError, match="q must be"):
        g.cache_attention(c, p, torch.zeros(4, 1, 64))
