"""ctypes binding of the paged 8-bit rollout cache (gla_cache_plan,
gla_cache_store, gla_cache_attention; include/gla.h) and a small container for
its tensors.

As in _binding, only argument marshalling happens here.  Beside the library's
own checks the wrappers compare dtypes and element counts with the sizes that
are passed, and run on the device of the tensors, whichever device is current.
Tensors that a call with `stream` allocates belong to that stream, as those made
under torch.cuda.stream() do.

    cache = gla.rollout_cache(sequences=8, pages=4096, kv_heads=24, d=128,
                              max_pages=512, page_tokens=64, frame_tokens=3680,
                              window_frames=4, n_sink=256)
    plan = gla.cache_plan(cache, new_lens, tokens)      # once a step
    gla.cache_store(cache, plan, k, v)                  # each layer (its own pools)
    out = gla.cache_attention(cache, plan, q, max_new=3680)

max_pages bounds the tokens of a whole rollout, not of its window: a block table has
an entry for every page a sequence has had (here 512 * 64 tokens, eight frames).  A
step that does not fit is refused as a whole: plan.status, on the GPU.
"""

from __future__ import annotations

import contextlib
import math
from dataclasses import dataclass

import torch

from . import _binding as _b

_I32, _F32, _BF16, _FP8, _U8 = (torch.int32, torch.float32, torch.bfloat16, torch.float8_e4m3fn,
                                torch.uint8)


_BF, _CODE, _INT, _FLT = (_BF16,), (_FP8, _U8), (_I32,), (_F32,)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _pointers(where, specs):
    """Device pointers of (name, tensor, dtypes, least element count) tuples and
    the one device they are on (None: no tensor among them).  None -> NULL, an
    int is taken as an address.  One loop, few calls: at the smallest sizes
    this is most of a call's time."""
    device = None
    out = []
    for name, x, dtypes, count in specs:
        if x is None or type(x) is int:
            out.append(x)
            continue
        if not isinstance(x, torch.Tensor):
            raise TypeError("%s: %s must be a torch.Tensor, an int address or None, got %r"
                            % (where, name, type(x)))
        if x.dtype not in dtypes:
            raise TypeError("%s: %s must be %s, got %s"
                            % (where, name, " or ".join(str(d) for d in dtypes), x.dtype))
        i = x.get_device()
        if i != device:
            if i < 0:
                raise ValueError("%s: %s must be on a CUDA device (got %s)"
                                 % (where, name, x.device))
            if device is not None:
                raise ValueError("%s: %s is on cuda:%d, other tensors are on cuda:%d"
                                 % (where, name, i, device))
            device = i
        if not x.is_contiguous():
            raise ValueError("%s: %s must be contiguous" % (where, name))
        if x.numel() < count:
            raise ValueError("%s: %s holds %d elements, the sizes ask for %d"
                             % (where, name, x.numel(), count))
        out.append(x.data_ptr() or None)
    return out, device


def _run(where, fn, pointers, device, sizes, stream):
    """fn(*pointers, *sizes, stream) on the tensors' device; a nonzero status
    raises.  stream None: that device's current stream."""
    if device is None or device == torch.cuda.current_device():
        if stream is None and device is not None and _raw_stream is not None:
            stream = _raw_stream(device)
        st = fn(*pointers, *sizes, _b._stream(stream))
    else:
        with torch.cuda.device(device):
            st = fn(*pointers, *sizes, _b._stream(stream))
    if st != _b.GLA_OK:
        raise _b.GLAError(st, where)


def gla_cache_plan(lens, held, new_lens, free_count, free_pages, block_table, lens_out, held_out,
                   free_count_out, cu_tokens, slots, status, R, max_pages, pages, page_tokens,
                   tokens, frame_tokens, window_frames, n_sink, stream=None) -> None:
    """Lengths, pages and slots of one step (see include/gla.h).  All arrays
    int32; raises GLAError on a nonzero return code.  Whether the step was
    admitted is in status[0] on the GPU."""
    ptr, dev = _pointers("gla_cache_plan", (
        ("lens", lens, _INT, R), ("held", held, _INT, R), ("new_lens", new_lens, _INT, R),
        ("free_count", free_count, _INT, 1), ("free_pages", free_pages, _INT, pages),
        ("block_table", block_table, _INT, R * max_pages), ("lens_out", lens_out, _INT, R),
        ("held_out", held_out, _INT, R), ("free_count_out", free_count_out, _INT, 1),
        ("cu_tokens", cu_tokens, _INT, R + 1), ("slots", slots, _INT, tokens),
        ("status", status, _INT, 1)))
    _run("gla_cache_plan", _b.load_library().gla_cache_plan, ptr, dev,
         (R, max_pages, pages, page_tokens, tokens, frame_tokens, window_frames, n_sink), stream)


def gla_cache_store(k, v, lens, cu_tokens, slots, k_cache, v_cache, k_scale, v_scale, nonfinite,
                    R, tokens, Hkv, d, pages, page_tokens, stream=None) -> None:
    """Quantise the new tokens' keys and values into the cache (see
    include/gla.h).  `nonfinite`: int32 counter tensor or None."""
    new, code, blocks = tokens * Hkv * d, pages * Hkv * page_tokens * d, pages * Hkv
    ptr, dev = _pointers("gla_cache_store", (
        ("k", k, _BF, new), ("v", v, _BF, new), ("lens", lens, _INT, R),
        ("cu_tokens", cu_tokens, _INT, R + 1), ("slots", slots, _INT, tokens),
        ("k_cache", k_cache, _CODE, code), ("v_cache", v_cache, _CODE, code),
        ("k_scale", k_scale, _FLT, blocks), ("v_scale", v_scale, _FLT, blocks),
        ("nonfinite", nonfinite, _INT, 1)))
    _run("gla_cache_store", _b.load_library().gla_cache_store, ptr, dev,
         (R, tokens, Hkv, d, pages, page_tokens), stream)


def gla_cache_attention(q, k_cache, v_cache, k_scale, v_scale, block_table, lens, cu_tokens,
                        gate_z, out, R, tokens, max_new, H, Hkv, d, pages, page_tokens, max_pages,
                        frame_tokens, window_frames, n_sink, scale, stream=None) -> None:
    """Attention of the new tokens over the cache (see include/gla.h)."""
    new, code, blocks = tokens * H * d, pages * Hkv * page_tokens * d, pages * Hkv
    ptr, dev = _pointers("gla_cache_attention", (
        ("q", q, _BF, new), ("k_cache", k_cache, _CODE, code), ("v_cache", v_cache, _CODE, code),
        ("k_scale", k_scale, _FLT, blocks), ("v_scale", v_scale, _FLT, blocks),
        ("block_table", block_table, _INT, R * max_pages), ("lens", lens, _INT, R),
        ("cu_tokens", cu_tokens, _INT, R + 1), ("gate_z", gate_z, _BF, new),
        ("out", out, _BF, new)))
    _run("gla_cache_attention", _b.load_library().gla_cache_attention, ptr, dev,
         (R, tokens, max_new, H, Hkv, d, pages, page_tokens, max_pages, frame_tokens,
          window_frames, n_sink, scale), stream)


def _allocating_for(stream, device):
    """The context to allocate a call's tensors in: memory that the current stream
    gave back may still be in use there, so a call on another stream takes its own."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(_b._stream(stream), device=device)
    return torch.cuda.stream(stream)


@dataclass
class RolloutCache:
    """The tensors of a paged rollout cache and its mask.  k, v and their
    scales belong to one layer: layers share the lengths and tables, so further
    layers are `cache.layer()`s of the first."""

    k: torch.Tensor            # float8_e4m3fn [pages, kv_heads, page_tokens, d]
    v: torch.Tensor
    k_scale: torch.Tensor      # fp32 [pages, kv_heads]
    v_scale: torch.Tensor
    lens: torch.Tensor         # int32 [sequences]: tokens held
    held: torch.Tensor         # int32 [sequences]: first page behind the sinks still held
    block_table: torch.Tensor  # int32 [sequences, max_pages]
    free_pages: torch.Tensor   # int32 [pages]: stack of free pages
    free_count: torch.Tensor   # int32 [1]
    frame_tokens: int = 1
    window_frames: int = 0
    n_sink: int = 0

    @property
    def page_tokens(self) -> int:
        return self.k.shape[2]

    def layer(self) -> "RolloutCache":
        """The cache of another layer: pools of its own, the same tables."""
        return RolloutCache(torch.zeros_like(self.k), torch.zeros_like(self.v),
                            torch.ones_like(self.k_scale), torch.ones_like(self.v_scale),
                            self.lens, self.held, self.block_table, self.free_pages,
                            self.free_count, self.frame_tokens, self.window_frames, self.n_sink)


@dataclass
class CachePlan:
    """What one step adds: row ranges and slots of the new tokens."""

    cu_tokens: torch.Tensor  # int32 [sequences + 1]
    slots: torch.Tensor      # int32 [tokens]
    status: torch.Tensor     # int32 [1]; 0: admitted (see gla_cache_plan)


def rollout_cache(sequences: int, pages: int, kv_heads: int, d: int, max_pages: int,
                  page_tokens: int = 64, frame_tokens: int = 1, window_frames: int = 0,
                  n_sink: int = 0, device="cuda") -> RolloutCache:
    """An empty cache: every page free, every sequence of length 0."""
    if page_tokens not in (16, 32, 64, 128):
        raise ValueError("page_tokens must be 16, 32, 64 or 128, got %d" % page_tokens)
    if d not in (64, 128):
        raise ValueError("d must be 64 or 128, got %d" % d)
    shape = (pages, kv_heads, page_tokens, d)
    codes = [torch.zeros(shape, dtype=_U8, device=device).view(_FP8) for _ in range(2)]
    scales = [torch.ones(pages, kv_heads, dtype=_F32, device=device) for _ in range(2)]
    ints = lambda *s: torch.zeros(*s, dtype=_I32, device=device)  # noqa: E731
    # the stack's top is its last entry: pages come out in ascending order
    free = torch.arange(pages - 1, -1, -1, dtype=_I32, device=device)
    return RolloutCache(codes[0], codes[1], scales[0], scales[1], ints(sequences),
                        ints(sequences), ints(sequences, max_pages) - 1, free, ints(1) + pages,
                        frame_tokens, window_frames, n_sink)


def cache_plan(cache: RolloutCache, new_lens, tokens: int, stream=None) -> CachePlan:
    """Plan one step in place: `new_lens` int32 [sequences] on the GPU (negative:
    the sequence has ended), `tokens` rows of the packed arrays (their sum, or
    more).  Updates the cache's lengths, tables and free pages."""
    R, max_pages = cache.block_table.shape
    dev = cache.lens.device
    with _allocating_for(stream, dev):
        plan = CachePlan(torch.empty(R + 1, dtype=_I32, device=dev),
                         torch.empty(tokens, dtype=_I32, device=dev),
                         torch.empty(1, dtype=_I32, device=dev))
    gla_cache_plan(cache.lens, cache.held, new_lens, cache.free_count, cache.free_pages,
                   cache.block_table, cache.lens, cache.held, cache.free_count, plan.cu_tokens,
                   plan.slots, plan.status, R, max_pages, cache.k.shape[0], cache.page_tokens,
                   tokens, cache.frame_tokens, cache.window_frames, cache.n_sink, stream)
    return plan


def cache_store(cache: RolloutCache, plan: CachePlan, k, v, nonfinite=None, stream=None) -> None:
    """Quantise k, v [tokens, kv_heads, d] of the step into the cache."""
    pages, H, P, d = cache.k.shape
    if k.shape != (plan.slots.numel(), H, d) or v.shape != k.shape:
        raise ValueError("k, v must be [%d, %d, %d], got %s and %s"
                         % (plan.slots.numel(), H, d, tuple(k.shape), tuple(v.shape)))
    gla_cache_store(k, v, cache.lens, plan.cu_tokens, plan.slots, cache.k, cache.v, cache.k_scale,
                    cache.v_scale, nonfinite, cache.lens.numel(), k.shape[0], H, d, pages, P,
                    stream)


def cache_attention(cache: RolloutCache, plan: CachePlan, q, gate_z=None, scale=None, out=None,
                    max_new=None, stream=None):
    """Attention of the step's queries q [tokens, H, d] over the cache (which
    already holds the step's keys and values); returns out.  Rows that belong to no
    sequence (behind the last one, or all of them when the plan refused the step:
    plan.status) are 0, or as they were in the caller's `out`.  `max_new`:
    the most new tokens of one sequence, as far as the host knows.  It picks the
    kernel of the whole call; both give the definition's result (include/gla.h
    has their precision), the wrong one slowly.  The default, the mean tokens /
    sequences, suits steps in which all sequences get about the same; a ragged
    step (a prompt among single tokens) or one with many rows of no sequence
    should pass it."""
    pages, Hkv, P, d = cache.k.shape
    R, max_pages = cache.block_table.shape
    N, H = q.shape[0], q.shape[1]
    if q.shape != (plan.slots.numel(), H, d):
        raise ValueError("q must be [%d, H, %d], got %s" % (plan.slots.numel(), d, tuple(q.shape)))
    if gate_z is not None and gate_z.shape != q.shape:
        raise ValueError("gate_z must have q's shape, got %s" % (tuple(gate_z.shape),))
    if out is None:
        with _allocating_for(stream, q.device):
            out = torch.zeros_like(q)  # the kernels leave rows of no sequence alone
    elif out.shape != q.shape:
        raise ValueError("out must have q's shape, got %s" % (tuple(out.shape),))
    if max_new is None:
        max_new = -(-N // max(R, 1))
    gla_cache_attention(q, cache.k, cache.v, cache.k_scale, cache.v_scale, cache.block_table,
                        cache.lens, plan.cu_tokens, gate_z, out, R, N, max_new, H, Hkv, d, pages,
                        P, max_pages, cache.frame_tokens, cache.window_frames, cache.n_sink,
                        1.0 / math.sqrt(d) if scale is None else scale, stream)
    return out
