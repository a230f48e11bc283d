"""fp64 CPU oracle of the paged 8-bit rollout cache: plan, store and attention.

TEST INFRASTRUCTURE ONLY (like gla_oracle.py): used by the tests, never by the
library; imports nothing from the library.  Plain loops over sequences, pages
and heads, written from the definitions in include/gla.h:

  plan       pages of each sequence that fell out of the window go back to the
             stack, new pages come from it, every new token gets a slot
  store      code = e4m3(x / scale), scale the smallest power of two that fits
             the page's largest magnitude, never shrinking while a page fills
  attention  softmax over min(len, frame end) keys, above the window's lower
             end or among the sinks; a query that sees nothing gives 0
"""

from __future__ import annotations

import math

import numpy as np

__all__ = ["cache_plan", "cache_store", "cache_attention", "e4m3_round", "page_scale"]


def cache_plan(lens, held, new_lens, free_pages, free_count, table, pages, P, tokens, F=1, W=0,
               n_sink=0):
    """All arguments Python ints / lists (table: list of lists); returns a dict
    of the outputs, with the stack and the table after the step."""
    R = len(lens)
    width = len(table[0]) if R else 0
    sp = -(-n_sink // P)
    stack, tab = list(free_pages), [list(t) for t in table]
    out = dict(lens=list(lens), held=list(held), free_count=free_count, cu=[0] * (R + 1),
               slots=[-1] * tokens, status=0, table=tab, stack=stack)
    back, new_held, need, total, wide = [], [], 0, 0, False
    for r in range(R):
        have = -(-lens[r] // P)
        if new_lens[r] < 0:
            back += [(r, j) for j in range(have) if j < sp or j >= held[r]]
            new_held.append(0)
            wide |= have > width
            continue
        w_lo = max(0, (lens[r] // F - W + 1) * F) if W else 0
        upto = max(held[r], w_lo // P)
        back += [(r, j) for j in range(max(sp, held[r]), upto)]
        new_held.append(upto)
        after = -(-(lens[r] + new_lens[r]) // P)
        need += after - have
        total += new_lens[r]
        wide |= after > width
    if free_count + len(back) < need:
        out["status"] |= 1
    if total > tokens:
        out["status"] |= 2
    if wide:
        out["status"] |= 4
    if free_count < 0 or free_count + len(back) > pages:
        out["status"] |= 8
    if out["status"]:
        return out
    n = free_count
    for r, j in back:
        stack[n] = tab[r][j]
        n += 1
    row = 0
    for r in range(R):
        out["cu"][r] = row
        if new_lens[r] < 0:
            out["lens"][r] = out["held"][r] = 0
            continue
        for pos in range(lens[r], lens[r] + new_lens[r]):
            if pos % P == 0:
                n -= 1
                tab[r][pos // P] = stack[n]
            out["slots"][row] = tab[r][pos // P] * P + pos % P
            row += 1
        out["lens"][r] = lens[r] + new_lens[r]
        out["held"][r] = new_held[r]
    out["cu"][R] = row
    out["free_count"] = n
    return out


def e4m3_round(x):
    """x (fp64) rounded to the nearest e4m3 value, ties to even, saturating."""
    x = np.asarray(x, dtype=np.float64)
    _, e = np.frexp(x)
    step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
    return np.clip(np.rint(x / step) * step, -448.0, 448.0)


def page_scale(amax):
    """Smallest power of two s in 2^-60 .. 2^60 with amax <= 448 s."""
    for e in range(-60, 60):
        if amax <= math.ldexp(448.0, e):
            return math.ldexp(1.0, e)
    return math.ldexp(1.0, 60)


def cache_store(x, slots, cu, codes, scales, P):
    """x [tokens, H, d] fp64 into codes [pages, H, P, d] (values of the codes)
    and scales [pages, H], both changed in place.  Runs of one sequence inside
    one page are written together."""
    x = np.asarray(x, dtype=np.float64)
    for r in range(len(cu) - 1):
        i = cu[r]
        while i < cu[r + 1]:
            page, at = divmod(int(slots[i]), P)
            m = min(P - at, cu[r + 1] - i)
            for h in range(x.shape[1]):
                y = x[i:i + m, h]
                fin = np.abs(y[np.isfinite(y)])
                s = page_scale(fin.max() if fin.size else 0.0)
                if at:
                    old = scales[page, h]
                    s = max(s, old)
                    if s != old:
                        codes[page, h, :at] = e4m3_round(codes[page, h, :at] * (old / s))
                y = np.where(np.isnan(y), 0.0, y)
                codes[page, h, at:at + m] = e4m3_round(y / s)
                scales[page, h] = s
            i += m


def cache_attention(q, kc, vc, ks, vs, table, lens, cu, P, F=1, W=0, n_sink=0, scale=None,
                    gate_z=None):
    """q [tokens, H, d]; kc, vc [pages, Hkv, P, d] values of the codes; ks, vs
    [pages, Hkv].  Returns (out, mag), both [tokens, H, d]: the output and the
    same sum over |v| (the scale of a rounding error of the weights)."""
    q = np.asarray(q, dtype=np.float64)
    N, H, d = q.shape
    pages, Hkv = ks.shape
    G = H // Hkv
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    out, mag = np.zeros((N, H, d)), np.zeros((N, H, d))
    for r in range(len(lens)):
        L = int(lens[r])
        n = int(cu[r + 1]) - int(cu[r])
        for i in range(n):
            pos = L - n + i
            if pos < 0:
                continue
            f = pos // F
            seen = [s for s in range(min(L, (f + 1) * F))
                    if (W == 0 or s >= (f - W + 1) * F or s < n_sink)
                    and s // P < len(table[r]) and 0 <= table[r][s // P] < pages]
            if not seen:
                continue
            seen = np.asarray(seen)
            pg = np.asarray([table[r][s // P] for s in seen])
            at = seen % P
            for h in range(Hkv):
                K = kc[pg, h, at] * ks[pg, h][:, None]
                V = vc[pg, h, at] * vs[pg, h][:, None]
                for x in range(h * G, (h + 1) * G):
                    a = K @ q[cu[r] + i, x] * scale
                    w = np.exp(a - a.max())
                    w /= w.sum()
                    out[cu[r] + i, x] = w @ V
                    mag[cu[r] + i, x] = w @ np.abs(V)
    if gate_z is not None:
        g = 1.0 / (1.0 + np.exp(-np.asarray(gate_z, dtype=np.float64)))
        out, mag = out * g, mag * g
    return out, mag
