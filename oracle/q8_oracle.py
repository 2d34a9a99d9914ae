"""Plain fp64 CPU oracle of the page plan and of the paged cache in 8-bit codes.

TEST INFRASTRUCTURE ONLY, like the rest of this package: nothing on the
product path may import it.

The cache holds, for every page and KV head, one power-of-two scale and one
code a row element, which stands for code * scale.  Codes are kept here as the
numbers they are (e4m3 values or whole numbers).  Everything else about the
cache is the paged cache of ``paged_oracle``, applied to the values.
"""
from __future__ import annotations

import math

import numpy as np

from .paged_oracle import decode_paged

__all__ = ["QMAX", "nearest_code", "q8_scale", "q8_values", "page_plan", "append_paged_q8",
           "decode_paged_q8"]

QMAX = {"e4m3": 448.0, "i8": 127.0}


def nearest_code(y, fmt: str) -> np.ndarray:
    """The code nearest to each y (|y| <= QMAX), ties to even."""
    y = np.asarray(y, dtype=np.float64)
    if fmt == "i8":
        return np.rint(y)
    # e4m3: 3 fraction bits above 2^-6, steps of 2^-9 below
    _, e = np.frexp(np.maximum(np.abs(y), 2.0 ** -6))
    step = np.ldexp(1.0, e - 4)
    return np.rint(y / step) * step


def q8_scale(amax: float, fmt: str) -> float:
    """The least 2^e, e >= -126, with amax <= QMAX 2^e."""
    e = -126
    if amax > 0:
        e = max(e, math.frexp(amax / QMAX[fmt])[1] - 2)
    while amax > QMAX[fmt] * 2.0 ** e:
        e += 1
    return 2.0 ** e


def q8_values(P, Ps) -> np.ndarray:
    """The values ``[num_pages, Hkv, B, d]`` that codes and scales stand for."""
    return np.asarray(P, np.float64) * np.asarray(Ps, np.float64)[:, :, None, None]


def page_plan(have, want, keep, table, ring, pool, B: int, max_new: int):
    """Row by row: returns ``(got, cu, slots, pool, table, ring)`` (new arrays)."""
    table, ring = np.array(table, np.int64), np.array(ring, np.int64)
    n, mb = table.shape
    pages = len(ring)
    head, count = (int(x) for x in pool)
    free = [int(ring[(head + i) % pages]) for i in range(count)]
    got, cu, slots = np.array(have, np.int64), [0], np.full(max_new, -1, np.int64)
    tokens = asked = taken = 0
    back = []
    for b in range(n):
        h, w = int(have[b]), int(want[b])
        if not (0 <= h <= mb * B and 0 <= w <= mb * B):
            cu.append(min(tokens, max_new))
            continue
        hb, wb = -(-h // B), -(-w // B)
        new, need = max(w - h, 0), max(wb - hb, 0)
        first, start = asked, tokens
        tokens, asked = tokens + new, asked + need
        if new and tokens <= max_new and (need == 0 or asked <= count):
            got[b] = w
            for i in range(need):
                table[b, hb + i] = free[first + i]
            taken += need
            for i in range(new):
                slots[start + i] = table[b, (h + i) // B] * B + (h + i) % B
        elif w < h:
            got[b] = w
            k = 0 if keep is None else int(keep[b])
            back += [int(p) for p in table[b, max(wb, min(max(k, 0), hb)):hb]]
        cu.append(min(tokens, max_new))
    back = back[: pages - count]
    for i, p in enumerate(back):
        ring[(head + count + i) % pages] = p
    return (got, np.array(cu), slots, np.array([(head + taken) % pages, count - taken + len(back)]),
            table, ring)


def append_paged_q8(K, Ks, V, Vs, S, slots, cu, seqlens, k_new, v_new, B: int, fmt: str):
    """Block by block: returns new ``(K, Ks, V, Vs, S)``; S may be None."""
    K, Ks, V, Vs = (np.array(x, np.float64) for x in (K, Ks, V, Vs))
    S = None if S is None else np.array(S, np.float64)
    for b in range(len(seqlens)):
        c0, c1, L = int(cu[b]), int(cu[b + 1]), int(seqlens[b])
        p0 = L - (c1 - c0)
        pos = p0
        while pos < L:
            j, r0 = pos // B, pos % B
            r1 = min(B, L - j * B)
            t0 = c0 + pos - p0
            pos = j * B + r1
            if slots[t0] < 0:
                continue
            page = int(slots[t0]) // B
            for P, Ps, x in ((K, Ks, k_new), (V, Vs, v_new)):
                for g in range(P.shape[1]):
                    rows = np.asarray(x[t0:t0 + r1 - r0, g], np.float64)
                    amax = np.max(np.abs(rows))
                    old = Ps[page, g] if r0 else 0.0
                    if not np.isfinite(amax) or np.isnan(old):
                        Ps[page, g] = np.nan
                        P[page, g, r0:r1] = 0
                        continue
                    sc = max(old, q8_scale(float(amax), fmt))
                    if r0 and sc > old:
                        P[page, g, :r0] = nearest_code(P[page, g, :r0] * (old / sc), fmt)
                    P[page, g, r0:r1] = nearest_code(rows / sc, fmt)
                    Ps[page, g] = sc
            if r1 == B and S is not None:
                S[b, :, j] = q8_values(K[page:page + 1], Ks[page:page + 1])[0].mean(axis=1)
    return K, Ks, V, Vs, S


def decode_paged_q8(q, K, Ks, V, Vs, page_table, seqlens, B: int, topk: int, S=None,
                    scale: float | None = None):
    """``decode_paged`` of the values that the codes stand for."""
    return decode_paged(q, q8_values(K, Ks), q8_values(V, Vs), page_table, seqlens, B, topk, S=S,
                        scale=scale)
