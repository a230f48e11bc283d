"""The paged 8-bit rollout cache on the GPU against its fp64 oracle.

Plan and store are exact: whole numbers, e4m3 codes and power-of-two scales are
compared bit for bit.  The attention's bound is derived, per element:
  out is rounded once to bf16: half a step, 2^-8 |ref|
  the weights are rounded to fp16 (2^-11) and may come from a polynomial
  exponential (2^-13.7); an fp32 score is off by less than 2^-13 here (|score| <
  64, 128 products): together below 2^-10 of sum p |v| sigmoid(z)
  weights below 2^-33 of the largest vanish: 2^-33 * keys * max|v| < 2^-20 max|v|
"""

import math
import random

import numpy as np
import pytest
import torch

import oracle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gla():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from gated_linear_attention_frame_b200.build import build

    build()
    import gated_linear_attention_frame_b200 as g

    g.load_library()
    g.gla_device_fault()
    yield g
    assert g.gla_device_fault() == 0


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


# -------------------------------------------------------------------- plan

def run_plan(gla, st, new, pages, P, tokens, F, W, sink, inplace):
    R, width = len(st["lens"]), len(st["table"][0]) if st["lens"] else 0
    lens, held, fc = ints(st["lens"]), ints(st["held"]), ints([st["free_count"]])
    stack, table = ints(st["stack"]), ints(st["table"]).reshape(R, width)
    lo, ho, fo = (lens, held, fc) if inplace else (torch.full_like(lens, 77),
                                                   torch.full_like(held, 77),
                                                   torch.full_like(fc, 77))
    cu, slots, status = ints([77] * (R + 1)), ints([77] * tokens), ints([77])
    gla.gla_cache_plan(lens, held, ints(new), fc, stack, table, lo, ho, fo, cu, slots, status, R,
                       width, pages, P, tokens, F, W, sink)
    return dict(lens=lo.tolist(), held=ho.tolist(), free_count=fo.item(), cu=cu.tolist(),
                slots=slots.tolist(), status=status.item(), table=table.tolist(),
                stack=stack.tolist())


@pytest.mark.parametrize("R,pages,width,P,tokens,F,W,sink,steps", [
    (1, 40, 30, 16, 60, 1, 0, 0, 12),
    (5, 120, 60, 16, 401, 40, 2, 20, 12),
    (7, 300, 40, 64, 403, 7, 3, 0, 8),
    (33, 900, 30, 32, 1000, 1, 100, 5, 8),
    (3, 700, 400, 16, 9001, 1560, 2, 64, 6),     # more than 8192 rows: the cluster launch
    (1500, 4000, 8, 16, 3001, 1, 20, 3, 5),      # more sequences than threads
])
def test_plan_follows_the_oracle(gla, R, pages, width, P, tokens, F, W, sink, steps):
    rng = random.Random(R * 31 + tokens)
    st = dict(lens=[0] * R, held=[0] * R, free_count=pages,
              table=[[-5] * width for _ in range(R)], stack=rng.sample(range(pages), pages))
    statuses = set()
    for step in range(steps):
        most = max(1, tokens // R)
        new = [rng.choice([0, 1, min(F, most), rng.randint(0, most), -1]) for _ in range(R)]
        args = (st["lens"], st["held"], new, st["stack"], st["free_count"], st["table"], pages, P,
                tokens, F, W, sink)
        ref = oracle.cache_plan(*args)
        got = run_plan(gla, st, new, pages, P, tokens, F, W, sink, inplace=step % 2 == 1)
        assert got == ref
        statuses.add(ref["status"])
        st = ref
        st["stack"], st["table"] = ref["stack"], ref["table"]
    assert 0 in statuses


def test_plan_refuses_a_step_as_a_whole(gla):
    st = dict(lens=[20, 30], held=[0, 1], free_count=2, table=[[3, 4, -1], [7, 5, -1]],
              stack=[0, 1, 2, 6, 8, 9, 10, 11])
    for new, tokens, fc, status in (([28, 3], 40, 1, 1), ([9, 3], 11, 2, 2), ([0, 31], 40, 2, 4),
                                    ([1, 1], 40, -1, 9), ([-1, 1], 40, 8, 8), ([90, 90], 40, 2, 7)):
        s = dict(st, free_count=fc)
        ref = oracle.cache_plan(s["lens"], s["held"], new, s["stack"], fc, s["table"], 8, 16,
                                tokens)
        assert ref["status"] == status
        assert run_plan(gla, s, new, 8, 16, tokens, 1, 0, 0, inplace=True) == ref
    # no sequences: the row counts are still written
    got = run_plan(gla, dict(lens=[], held=[], free_count=2, table=[], stack=[0, 1]), [], 2, 16, 5,
                   1, 0, 0, inplace=False)
    assert got["cu"] == [0] and got["slots"] == [-1] * 5 and got["status"] == 0


# ------------------------------------------------------------------- store

class Cache:
    """A cache built token by token through the store, beside the oracle's."""

    def __init__(self, pages, Hkv, P, d, width, order):
        self.P, self.shape = P, (pages, Hkv, P, d)
        # slots that hold nothing: the NaN code, scales NaN
        self.k8 = torch.full(self.shape, 0x7F, dtype=torch.uint8, device="cuda")
        self.v8 = self.k8.clone()
        self.ks = torch.full((pages, Hkv), float("nan"), device="cuda")
        self.vs = self.ks.clone()
        self.ref = [np.full(self.shape, np.nan) for _ in range(2)]
        self.sc = [np.full((pages, Hkv), np.nan) for _ in range(2)]
        self.order, self.width = list(order), width
        self.lens, self.table = [], []

    def add(self, n):
        self.lens.append(n)
        self.table.append([])

    def step(self, gla, new, k, v, pad=0, nonfinite=None):
        """Append new[r] tokens to each sequence; k, v bf16 CPU [sum + pad, H, d]."""
        P = self.P
        slots, cu = [], [0]
        for r, n in enumerate(new):
            for pos in range(self.lens[r], self.lens[r] + n):
                if pos // P == len(self.table[r]):
                    self.table[r].append(self.order.pop())
                slots.append(self.table[r][pos // P] * P + pos % P)
            self.lens[r] += n
            cu.append(len(slots))
        N = len(slots) + pad
        pages, H, _, d = self.shape
        gla.gla_cache_store(k.cuda(), v.cuda(), ints(self.lens), ints(cu),
                            ints(slots + [-1] * pad), self.k8, self.v8, self.ks, self.vs,
                            nonfinite, len(new), N, H, d, pages, P)
        for x, c, s in ((k, self.ref[0], self.sc[0]), (v, self.ref[1], self.sc[1])):
            oracle.cache_store(x.double().numpy(), slots, cu, c, s, P)
        return cu

    def check(self):
        for got, ref in ((self.k8, self.ref[0]), (self.v8, self.ref[1])):
            g = got.view(torch.float8_e4m3fn).float().cpu().double().numpy()
            assert np.array_equal(g, ref, equal_nan=True)
        for got, ref in ((self.ks, self.sc[0]), (self.vs, self.sc[1])):
            assert np.array_equal(got.cpu().double().numpy(), ref, equal_nan=True)

    def tables(self, fill=-1):
        return ints([t + [fill] * (self.width - len(t)) for t in self.table])


def bf(shape, seed, spread=0.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(shape, generator=g)
    if spread:  # tokens of very different size: scales grow within a page
        x = x * torch.exp2(torch.randint(-int(spread), int(spread) + 1, (shape[0], shape[1], 1),
                                         generator=g).float())
    return x.bfloat16()


@pytest.mark.parametrize("P", [16, 32, 64, 128])
@pytest.mark.parametrize("d", [64, 128])
def test_store_follows_the_oracle(gla, P, d):
    H, R = 3, 4
    c = Cache(40, H, P, d, 12, random.Random(P + d).sample(range(40), 40))
    for _ in range(R):
        c.add(0)
    for step, new in enumerate(([5, 1, 0, P], [1, 1, 1, 1], [P - 6, 2 * P + 3, 1, 0],
                                [1, 0, 2 * P - 1, P + 1], [0, 0, 0, 1])):
        n = sum(new)
        k, v = bf((n + 3, H, d), 10 * step + P, 6), bf((n + 3, H, d), 10 * step + P + 5, 12)
        k[-3:], v[-3:] = float("nan"), float("inf")  # rows behind the last token
        c.step(gla, new, k, v, pad=3)
        c.check()


def test_store_ranges_and_nonfinite(gla):
    H, d, P = 2, 64, 16
    c = Cache(6, H, P, d, 3, range(6))
    c.add(0)
    c.add(0)
    k, v = bf((8, H, d), 1), bf((8, H, d), 2)
    k[0], k[1] = 0.0, 1e-30        # a tiny page keeps the least scale
    k[2, 1], k[3, 0, :5] = 3e38, float("nan")
    v[0] = 2.0 ** -130             # subnormal bf16
    v[1, 0, 3], v[1, 1, 7] = float("inf"), float("-inf")
    v[5] = 448.0
    v[6] = 450.0
    count = ints([10])
    c.step(gla, [4, 4], k, v, nonfinite=count)
    c.check()
    assert count.item() == 10 + 5 + 2
    z = torch.zeros(2, H, d).bfloat16()
    c.step(gla, [1, 1], z, z, nonfinite=count)  # zeros never change a scale
    c.check()
    assert count.item() == 17


def test_store_skips_slots_outside_the_cache(gla):
    H, d, P, pages = 2, 64, 16, 4
    k8 = torch.full((pages, H, P, d), 9, dtype=torch.uint8, device="cuda")
    v8, ks = k8.clone(), torch.full((pages, H), 3.0, device="cuda")
    vs = ks.clone()
    x = bf((6, H, d), 3).cuda()
    gla.gla_cache_store(x, x, ints([2, 2, 2]), ints([0, 2, 4, 6]),
                        ints([-1, -1, pages * P, pages * P + 1, 2**31 - 16, 2**31 - 15]), k8, v8,
                        ks, vs, None, 3, 6, H, d, pages, P)
    assert k8.eq(9).all() and v8.eq(9).all() and ks.eq(3).all() and vs.eq(3).all()


# --------------------------------------------------------------- attention

def check_attention(gla, c, new, H, F, W, sink, gate, seed, max_new=None, qscale=1.0, fill=-1,
                    scale=None, pad=2):
    pages, Hkv, P, d = c.shape
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    N = cu[-1] + pad
    q = (bf((N, H, d), seed) * qscale).bfloat16()
    z = bf((N, H, d), seed + 1) if gate else None
    out = torch.full((N, H, d), 55.0, dtype=torch.bfloat16, device="cuda")
    scale = d ** -0.5 if scale is None else scale
    table = c.tables(fill)
    gla.gla_cache_attention(q.cuda(), c.k8, c.v8, c.ks, c.vs, table, ints(c.lens), ints(cu),
                            None if z is None else z.cuda(), out, len(new), N,
                            max(new) if max_new is None else max_new, H, Hkv, d, pages, P,
                            c.width, F, W, sink, scale)
    got = out.double().cpu().numpy()
    assert np.all(got[cu[-1]:] == 55.0)  # rows behind the last sequence stay
    if not cu[-1]:
        return out
    ref, mag = oracle.cache_attention(
        q[:cu[-1]].double().numpy(), np.nan_to_num(c.ref[0]), np.nan_to_num(c.ref[1]),
        np.nan_to_num(c.sc[0]), np.nan_to_num(c.sc[1]), table.tolist(), c.lens, cu, P, F, W, sink,
        scale, None if z is None else z[:cu[-1]].double().numpy())
    vmax = np.nanmax(np.abs(c.ref[1]) * c.sc[1][:, :, None, None])
    bound = 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * mag + 2.0 ** -20 * vmax
    err = np.abs(got[:cu[-1]] - ref)
    assert np.all(err <= bound), "worst %.3g of its bound" % (err / bound).max()
    return out


CASES = [
    # lens before, new, P, Hkv, G, d, F, W, sink, gate
    ([0], [1], 16, 1, 1, 128, 1, 0, 0, False),                   # one token, one key
    ([0], [1], 128, 1, 1, 64, 1, 0, 0, True),
    ([31, 32, 33, 0, 7], [1, 1, 1, 1, 0], 32, 2, 3, 128, 1, 0, 0, True),
    ([700, 5, 333], [1, 1, 1], 64, 3, 8, 64, 1, 0, 0, False),
    ([500, 64, 257], [1, 1, 1], 16, 2, 1, 128, 1, 100, 20, False),  # window and sinks
    ([130, 90], [5, 3], 32, 2, 4, 128, 1, 40, 3, True),          # a few tokens, causal
    ([60, 120], [20, 20], 16, 2, 1, 128, 20, 2, 10, True),       # frames
    ([0, 300, 150], [150, 150, 150], 64, 2, 1, 128, 150, 2, 64, True),
    ([0, 17, 400], [300, 260, 1], 16, 2, 2, 64, 1, 0, 0, False),  # ragged prompts
    ([200], [300], 128, 1, 5, 128, 1, 130, 7, True),             # odd group, window inside
    ([45, 90], [45, 45], 32, 1, 3, 64, 45, 1, 45, False),        # one frame sees itself and sinks
    ([3, 290], [129, 128], 64, 1, 1, 128, 1, 0, 0, False),
    ([10], [40], 16, 1, 128, 64, 1, 0, 0, False),                # all heads share one
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_attention_follows_the_oracle(gla, case):
    old, new, P, Hkv, G, d, F, W, sink, gate = CASES[case]
    width = max(-(-(o + n) // P) for o, n in zip(old, new)) + 2
    pages = sum(-(-(o + n) // P) for o, n in zip(old, new)) + 3
    c = Cache(pages, Hkv, P, d, width, random.Random(case).sample(range(pages), pages))
    for _ in old:
        c.add(0)
    if sum(old):
        c.step(gla, old, bf((sum(old), Hkv, d), case, 1), bf((sum(old), Hkv, d), case + 50, 2))
    c.step(gla, new, bf((sum(new), Hkv, d), case + 7, 1), bf((sum(new), Hkv, d), case + 77, 2))
    outs = [check_attention(gla, c, new, Hkv * G, F, W, sink, gate, 900 + case, max_new=m)
            for m in (max(new), 1 << 20, 1, -(-9 // G))]  # the hint picks the kernel: each of them
    for o in outs[1:]:
        assert torch.allclose(outs[0].float(), o.float(), rtol=2 ** -6, atol=2 ** -6)


def test_attention_rows_that_see_nothing(gla):
    P, d = 16, 128
    c = Cache(8, 1, P, d, 4, range(8))
    c.add(0)
    c.add(0)
    c.step(gla, [40, 20], bf((60, 1, d), 1), bf((60, 1, d), 2))
    keep = list(c.lens)
    # no keys yet: an attention before any store
    c.lens = [0, 20]
    out = check_attention(gla, c, [1, 1], 2, 1, 0, 0, True, 5)
    assert out[0].eq(0).all()
    # table entries that name no page hide their keys; with all of them gone a row is 0
    c.lens, full = keep, [list(t) for t in c.table]
    c.table = [[-1, full[0][1], 8], full[1]]
    check_attention(gla, c, [2, 1], 2, 1, 0, 0, False, 6)
    c.table = [[-1, 99, -7], full[1]]
    out = check_attention(gla, c, [2, 1], 2, 1, 0, 0, False, 7)
    assert out[:2].eq(0).all()
    # pages that left the window: their entries may name another sequence's page or none
    c.table = [[full[1][1], full[0][1], full[0][2]], full[1]]
    check_attention(gla, c, [1, 1], 2, 1, 20, 0, False, 8)


def test_attention_extreme_values(gla):
    """Huge and tiny queries, values whose scales differ between the pages."""
    P, d = 16, 64
    c = Cache(12, 2, P, d, 6, range(12))
    c.add(0)
    k = bf((90, 2, d), 1)
    v = (bf((90, 2, d), 2).float() * torch.exp2((torch.arange(90) // P * 9 - 20).float())[:, None, None]).bfloat16()
    c.step(gla, [90], k, v)
    check_attention(gla, c, [1], 4, 1, 0, 0, False, 3)
    check_attention(gla, c, [7], 4, 1, 0, 0, False, 4, qscale=2.0 ** -60)
    check_attention(gla, c, [90], 4, 1, 0, 0, False, 5, qscale=2.0 ** 40, scale=2.0 ** -43)
    check_attention(gla, c, [3], 4, 1, 0, 0, False, 6, qscale=0.0)
    check_attention(gla, c, [2], 4, 1, 0, 0, False, 7, qscale=4.0)


def test_long_sequences_split_over_the_gpu(gla):
    """One sequence over many CTAs, and a mix of lengths; d = 128 and 64."""
    for d, P, Hkv, G, lens in ((128, 64, 1, 2, [20001]), (64, 32, 2, 1, [9000, 1, 4097, 33])):
        pages = sum(-(-n // P) for n in lens)
        c = Cache(pages, Hkv, P, d, max(-(-n // P) for n in lens), range(pages))
        for _ in lens:
            c.add(0)
        c.step(gla, lens, bf((sum(lens), Hkv, d), d), bf((sum(lens), Hkv, d), d + 1))
        check_attention(gla, c, [1] * len(lens), Hkv * G, 1, 0, 0, False, 11)
        check_attention(gla, c, [2] * len(lens), Hkv * G, 1, 5000, 40, True, 12)
        if d == 128:
            check_attention(gla, c, [40], Hkv * G, 1, 0, 0, True, 13)


# ---------------------------------------------------------------- together

def test_a_rollout_runs_plan_store_and_attention_together(gla):
    """Frames and single tokens through the package's calls, two layers sharing
    one plan, pages going round; every step against the oracle."""
    T, W, sink, P, d, Hkv, H = 24, 2, 10, 16, 128, 2, 4
    R, pages, width = 3, 14, 16
    cache = gla.rollout_cache(R, pages, Hkv, d, width, page_tokens=P, frame_tokens=T,
                              window_frames=W, n_sink=sink)
    second = cache.layer()
    ref = dict(lens=[0] * R, held=[0] * R, free_count=pages, table=[[-1] * width] * R,
               stack=cache.free_pages.tolist())
    code = [[np.zeros((pages, Hkv, P, d)) for _ in range(2)] for _ in range(2)]
    sc = [[np.ones((pages, Hkv)) for _ in range(2)] for _ in range(2)]
    steps = [[T, T, 0], [T, 0, T], [T, T, T], [T, T, T], [-1, T, T], [T, T, -1], [0, T, T],
             [T, T, T]]
    for i, new in enumerate(steps):
        N = 3 * T
        plan = gla.cache_plan(cache, ints(new), N)
        ref = oracle.cache_plan(ref["lens"], ref["held"], new, ref["stack"], ref["free_count"],
                                ref["table"], pages, P, N, T, W, sink)
        assert ref["status"] == 0 and plan.status.item() == 0
        assert plan.slots.tolist() == ref["slots"] and cache.lens.tolist() == ref["lens"]
        for y, layer in enumerate((cache, second)):
            k, v, q, z = (bf((N, h, d), 100 * i + 10 * y + e) for e, h in enumerate((Hkv, Hkv, H, H)))
            gla.cache_store(layer, plan, k.cuda(), v.cuda())
            out = gla.cache_attention(layer, plan, q.cuda(), gate_z=z.cuda(), max_new=T)
            n = ref["cu"][-1]
            for x, a, b in ((k, code[y][0], sc[y][0]), (v, code[y][1], sc[y][1])):
                oracle.cache_store(x.double().numpy(), ref["slots"], ref["cu"], a, b, P)
            want, mag = oracle.cache_attention(q[:n].double().numpy(), code[y][0], code[y][1],
                                               sc[y][0], sc[y][1], ref["table"], ref["lens"],
                                               ref["cu"], P, T, W, sink,
                                               gate_z=z[:n].double().numpy())
            err = np.abs(out[:n].double().cpu().numpy() - want)
            assert np.all(err <= 2.0 ** -8 * np.abs(want) + 2.0 ** -10 * mag + 2.0 ** -16)
    assert ref["free_count"] < 4  # the pool is nearly used up, and pages were reused


def test_cached_frames_stay_near_the_bf16_anchor(gla):
    """The same rollout through the anchor step's bf16 caches: what e4m3 loses
    (2^-4 relative an element) is all that differs."""
    T, W, sink, H, d, frames = 130, 2, 64, 2, 128, 3
    g = torch.Generator().manual_seed(4)
    q, k, v = (torch.randn(1, frames * T, H, d, generator=g).bfloat16().cuda() for _ in range(3))
    whole = gla.softmax_anchor(q, k, v, frames, W, sink)
    cache = gla.rollout_cache(1, 16, H, d, 16, page_tokens=32, frame_tokens=T, window_frames=W,
                              n_sink=sink)
    for f in range(frames):
        rows = slice(f * T, (f + 1) * T)
        plan = gla.cache_plan(cache, ints([T]), T)
        gla.cache_store(cache, plan, k[0, rows].contiguous(), v[0, rows].contiguous())
        out = gla.cache_attention(cache, plan, q[0, rows].contiguous())
        ref = whole[0, rows].float()
        # each value is off by at most 2^-4 of itself, each score by 2^-4 |q||k| /
        # sqrt(d) at the worst: the mean of T such terms stays well inside 10%
        assert (out.float() - ref).norm() <= 0.1 * ref.norm()


def test_streams_graphs_and_repeats(gla):
    """Bit for bit the same: on another stream, twice at once on two streams,
    captured and replayed with other lengths than at capture."""
    P, d, Hkv, H, width, pages = 32, 128, 2, 4, 40, 64
    mk = lambda: gla.rollout_cache(2, pages, Hkv, d, width, page_tokens=P)  # noqa: E731
    steps = [[37, 500], [1, 1], [1, 1], [1, 1], [64, 3], [1, 1]]
    data = []
    for i, new in enumerate(steps):
        N = sum(new)
        data.append([bf((N, h, d), 40 * i + h + e).cuda() for e, h in enumerate((Hkv, Hkv, H))])

    def run(stream=None):
        c, outs = mk(), []
        for new, (k, v, q) in zip(steps, data):
            plan = gla.cache_plan(c, ints(new), k.shape[0], stream=stream)
            gla.cache_store(c, plan, k, v, stream=stream)
            outs.append(gla.cache_attention(c, plan, q, max_new=max(new), stream=stream))
        return outs

    first = run()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for s in (s1, s2):
        with torch.cuda.stream(s):
            outs.append(run())
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(first, o))
    # graph of one decoding step, replayed as the lengths move on
    c = mk()
    k, v, q = (torch.empty_like(x) for x in data[1])
    new = ints([1, 1])
    out = torch.empty_like(q)
    plan0 = gla.cache_plan(c, ints(steps[0]), sum(steps[0]))
    gla.cache_store(c, plan0, data[0][0], data[0][1])
    keep = [t.clone() for t in (c.lens, c.held, c.block_table, c.free_pages, c.free_count)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):  # warm-up, then put the state back
        p = gla.cache_plan(c, new, 2)
        gla.cache_store(c, p, k.zero_(), v.zero_())
        gla.cache_attention(c, p, q.zero_(), out=out, max_new=1)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p = gla.cache_plan(c, new, 2)
        gla.cache_store(c, p, k, v)
        gla.cache_attention(c, p, q, out=out, max_new=1)
    for t, x in zip((c.lens, c.held, c.block_table, c.free_pages, c.free_count), keep):
        t.copy_(x)
    for i in (1, 2, 3):
        for a, b in zip((k, v, q), data[i]):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert p.status.item() == 0
        assert torch.equal(out, first[i])


def test_alloc_failure_is_reported(gla):
    c = gla.rollout_cache(1, 4, 1, 128, 4)
    plan = gla.cache_plan(c, ints([3]), 3)
    x = bf((3, 1, 128), 1).cuda()
    gla.cache_store(c, plan, x, x)
    out = torch.full((3, 1, 128), 9.0, dtype=torch.bfloat16, device="cuda")
    gla.gla_inject_alloc_failure(1)
    with pytest.raises(gla.GLAError) as e:
        gla.cache_attention(c, plan, x, out=out)
    assert e.value.status == gla.GLA_ERR_ALLOC
    assert out.eq(9.0).all()
    gla.cache_attention(c, plan, x, out=out)
    assert not out.eq(9.0).any()


def test_wrappers_refuse_on_the_gpu(gla):
    c = gla.rollout_cache(2, 4, 1, 64, 4)
    plan = gla.cache_plan(c, ints([1, 1]), 2)
    x = bf((2, 1, 64), 1).cuda()
    with pytest.raises(ValueError, match="holds"):
        gla.gla_cache_store(x, x, c.lens, plan.cu_tokens, plan.slots, c.k, c.v, c.k_scale,
                            c.v_scale, None, 2, 3, 1, 64, 4, 64)
    with pytest.raises(ValueError, match="contiguous"):
        gla.cache_store(c, plan, bf((2, 1, 128), 1).cuda()[:, :, :64], x)
    with pytest.raises(TypeError, match="int32"):
        gla.cache_plan(c, torch.ones(2, dtype=torch.int64, device="cuda"), 2)
    with pytest.raises(ValueError, match="out must"):
        gla.cache_attention(c, plan, x, out=x[:1])


@pytest.mark.parametrize("max_new", [1, 1 << 20])
def test_a_broken_query_row_stays_alone(gla, max_new):
    """NaN or infinity in one query row: that row alone is not finite."""
    P, d, H = 32, 128, 2
    c = Cache(8, 1, P, d, 8, range(8))
    c.add(0)
    c.step(gla, [200], bf((200, 1, d), 1), bf((200, 1, d), 2))
    q = bf((40, H, d), 3).cuda()
    args = (c.k8, c.v8, c.ks, c.vs, c.tables(), ints(c.lens), ints([0, 40]), None)
    tail = (1, 40, max_new, H, 1, d, 8, P, 8, 1, 0, 0, d ** -0.5)
    good, out = torch.empty_like(q), torch.empty_like(q)
    gla.gla_cache_attention(q, *args, good, *tail)
    q[7, 1, 5], q[20, 0, 9] = float("nan"), float("inf")
    gla.gla_cache_attention(q, *args, out, *tail)
    rows = torch.ones(40, H, dtype=torch.bool, device="cuda")
    rows[7, 1] = rows[20, 0] = False
    assert torch.isfinite(good).all() and torch.isfinite(out[rows]).all()
    # a rescale that the broken row sets off may move the others by a rounding
    assert torch.allclose(out[rows].float(), good[rows].float(), rtol=2 ** -6, atol=2 ** -8)
    assert not torch.isfinite(out[7, 1]).any()


def test_neighbouring_pages_of_different_scale(gla):
    """Keys and values of pages whose scales differ by up to 2^12 within 128
    keys: the tile's common scale is exact."""
    P, d = 16, 128
    c = Cache(16, 1, P, d, 16, range(16))
    c.add(0)
    step = torch.exp2(-((torch.arange(230) // P * 5) % 13).float())[:, None, None]
    c.step(gla, [230], (bf((230, 1, d), 1).float() * step).bfloat16(),
           (bf((230, 1, d), 2).float() * step.flip(0)).bfloat16())
    for m in (1, 9, 1 << 20):
        check_attention(gla, c, [100], 1, 1, 0, 0, False, 3, max_new=m, qscale=4.0)


def test_frames_in_two_graphs_at_once(gla):
    """Whole frame steps (plan, store, attention with split units) captured
    twice; the replays run together on two streams and give the eager bits."""
    P, d, Hkv, H, T, pages = 64, 128, 2, 4, 4100, 300
    data = [bf((2 * T, h, d), 5 + e).cuda() for e, h in enumerate((Hkv, Hkv, H))]
    mk = lambda: gla.rollout_cache(2, pages, Hkv, d, 200, page_tokens=P, frame_tokens=T,  # noqa: E731
                                   window_frames=2, n_sink=100)

    def step(c, new, k, v, q, out):
        plan = gla.cache_plan(c, new, 2 * T)  # above 8192 rows: two launches
        gla.cache_store(c, plan, k, v)
        gla.cache_attention(c, plan, q, out=out, max_new=T)
        return plan

    new = ints([T, T])
    c = mk()
    want = []
    for _ in range(2):
        want.append(torch.empty_like(data[2]))
        step(c, new, *data, want[-1])
    torch.cuda.synchronize()
    runs = []
    for _ in range(2):
        c, out = mk(), torch.empty_like(data[2])
        keep = [t.clone() for t in (c.lens, c.held, c.block_table, c.free_pages, c.free_count)]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step(c, new, *data, out)
        side.synchronize()
        for t, x in zip((c.lens, c.held, c.block_table, c.free_pages, c.free_count), keep):
            t.copy_(x)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            plan = step(c, new, *data, out)
        for t, x in zip((c.lens, c.held, c.block_table, c.free_pages, c.free_count), keep):
            t.copy_(x)
        runs.append((g, out, plan, torch.cuda.Stream(), c))
    torch.cuda.synchronize()
    for i in range(2):
        for g, _, _, s, _ in runs:
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for _, out, plan, _, _ in runs:
            assert plan.status.item() == 0
            assert torch.equal(out, want[i])


def test_many_tiny_sequences_and_wide_groups(gla):
    """More sequences than CTAs, most of them idle; 128 and 20 heads a group."""
    rng = random.Random(5)
    P, d = 16, 64
    lens = [rng.choice([0, 1, 5, 17]) for _ in range(700)]
    new = [min(n, rng.choice([0, 0, 1])) for n in lens]
    pages = sum(-(-n // P) for n in lens) + 1
    c = Cache(pages, 1, P, d, 2, range(pages))
    for _ in lens:
        c.add(0)
    n = sum(lens)
    c.step(gla, lens, bf((n, 1, d), 1), bf((n, 1, d), 2))
    for G in (1, 20, 128):
        for m in (1, 1 << 20):
            check_attention(gla, c, new, G, 1, 0, 0, False, G, max_new=m)


@pytest.mark.parametrize("max_new", [1, 1 << 20])
def test_tiny_queries_on_keys_that_are_all_zero(gla, max_new):
    """Row and key scales whose product is below the fp32 range, on rows with a
    mask: every visible key weighs the same."""
    P, d = 32, 128
    c = Cache(8, 1, P, d, 8, range(8))
    c.add(0)
    c.step(gla, [150], torch.zeros(150, 1, d).bfloat16(), bf((150, 1, d), 2))
    out = check_attention(gla, c, [100], 2, 1, 0, 0, False, 3, max_new=max_new, qscale=2.0 ** -100)
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("max_new", [1, 1 << 20])
def test_more_rows_than_tokens_held(gla, max_new):
    """New rows beyond a sequence's length stand before its first token: 0."""
    P, d = 16, 64
    c = Cache(8, 1, P, d, 8, range(8))
    c.add(0)
    c.step(gla, [70], bf((70, 1, d), 1), bf((70, 1, d), 2))
    q = bf((100, 1, d), 3).cuda()
    out = torch.full_like(q, 7.0)
    args = (c.k8, c.v8, c.ks, c.vs, c.tables(), ints(c.lens), ints([0, 100]), None, out)
    gla.gla_cache_attention(q, *args, 1, 100, max_new, 1, 1, d, 8, P, 8, 1, 0, 0, d ** -0.5)
    assert out[:30].eq(0).all() and out[30:].abs().sum() > 0
    tail = check_attention(gla, c, [70], 1, 1, 0, 0, False, 3, max_new=max_new, pad=0)
    assert tail.shape == (70, 1, d)


@pytest.mark.parametrize("max_new", [1, 1 << 20])
def test_row_ranges_that_descend_stay_in_bounds(gla, max_new):
    """Offsets that go up and down give each second sequence all the rows: more
    units than the host's bound.  The arrays' neighbours and a later call are as
    they should be."""
    P, d, R, N, pages = 16, 64, 64, 1100, 70
    c = Cache(pages, 1, P, d, pages, range(pages))
    c.add(0)
    c.step(gla, [N], bf((N, 1, d), 1), bf((N, 1, d), 2))
    lens, cu = ints([N] * R), ints([0, N] * (R // 2) + [0])
    tables = c.tables().expand(R, -1).contiguous()
    q, guard = bf((N, 1, d), 3).cuda(), torch.full((3 * N, 1, d), 5.0, dtype=torch.bfloat16).cuda()
    gla.gla_cache_attention(q, c.k8, c.v8, c.ks, c.vs, tables, lens, cu, None, guard[N:2 * N], R, N,
                            max_new, 1, 1, d, pages, P, pages, 1, 0, 0, d ** -0.5)
    assert guard[:N].eq(5).all() and guard[2 * N:].eq(5).all()
    before = [t.clone() for t in (c.k8, c.v8, c.ks, c.vs)]
    gla.gla_cache_store(q, q, lens, cu, torch.arange(N, dtype=torch.int32, device="cuda"), *before,
                        None, R, N, 1, d, pages, P)
    torch.cuda.synchronize()
    check_attention(gla, c, [N], 1, 1, 0, 0, False, 3, max_new=max_new)


def test_a_prefix_that_two_sequences_share(gla):
    """Two rows of the table with the same first pages."""
    P, d = 32, 128
    c = Cache(12, 2, P, d, 6, range(12))
    c.add(0)
    c.step(gla, [96], bf((96, 2, d), 1), bf((96, 2, d), 2))
    table = c.tables().expand(2, -1).contiguous()
    q = bf((2, 4, d), 3).cuda()
    out = torch.empty_like(q)
    gla.gla_cache_attention(q, c.k8, c.v8, c.ks, c.vs, table, ints([96, 96]), ints([0, 1, 2]), None,
                            out, 2, 2, 1, 4, 2, d, 12, P, 6, 1, 0, 0, d ** -0.5)
    one = torch.empty_like(q[:1])
    for r in range(2):
        gla.gla_cache_attention(q[r:r + 1].contiguous(), c.k8, c.v8, c.ks, c.vs, table[:1], ints([96]),
                                ints([0, 1]), None, one, 1, 1, 1, 4, 2, d, 12, P, 6, 1, 0, 0,
                                d ** -0.5)
        # each is off by 2^-8 of itself and 2^-10 sum p |v|, |v| < 8
        assert torch.allclose(one.float(), out[r:r + 1].float(), rtol=2 ** -7, atol=2 ** -6)


def test_more_units_than_shared_memory_holds(gla):
    """22 thousand units of two tokens: the schedule's sums lie in the workspace.
    Both kernels against each other, and the first rows against the oracle."""
    P, d, G, R, T, W = 64, 64, 128, 4, 11000, 64
    pages = R * -(-T // P)
    c = gla.rollout_cache(R, pages, 1, d, pages // R, page_tokens=P, window_frames=W)
    k, v, q = (bf((R * T, h, d), 60 + h + e).cuda() for e, h in enumerate((1, 1, G)))
    plan = gla.cache_plan(c, ints([T] * R), R * T)
    gla.cache_store(c, plan, k, v)
    a = gla.cache_attention(c, plan, q, max_new=T)
    b = gla.cache_attention(c, plan, q, max_new=0)
    assert plan.status.item() == 0
    # each is off by 2^-8 of itself and 2^-10 sum p |v|, |v| < 8
    for i in range(0, R * T, 4000):
        assert torch.allclose(a[i:i + 4000].float(), b[i:i + 4000].float(), rtol=2 ** -7,
                              atol=2 ** -6)
    n = 128  # two pages; the window leaves the first token behind at 64
    x, y = (oracle_values(t[:n, 0], P) for t in (k, v))
    s = q[:n].double().cpu().numpy() @ x.T * d ** -0.5
    at = np.arange(n)
    seen = (at[None, :] <= at[:, None]) & (at[None, :] > at[:, None] - W)
    s = np.where(seen[:, None, :], s, -np.inf)
    p = np.exp(s - s.max(-1, keepdims=True))
    ref, mag = ((p @ t) / p.sum(-1, keepdims=True) for t in (y, np.abs(y)))
    err = np.abs(a[:n].double().cpu().numpy() - ref)
    assert np.all(err <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * mag + 2.0 ** -20 * np.abs(y).max())


def oracle_values(x, P):
    """What the cache holds of one head's rows, written page by page: e4m3 with
    the smallest power of two that takes each page's largest value."""
    x = x.double().cpu()
    out = torch.empty_like(x)
    for i in range(0, x.shape[0], P):
        step = 2.0 ** math.ceil(math.log2(x[i:i + P].abs().max().item() / 448))
        out[i:i + P] = (x[i:i + P] / step).float().to(torch.float8_e4m3fn).double() * step
    return out.numpy()
