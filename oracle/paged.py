"""The 8-bit paged K/V cache in float64: codes, append, attention, evict.

Codes are decoded and encoded from their definition (sign, exponent and
mantissa fields), by tables of all 256 values; nothing here uses a library's
8-bit type.  Arrays: pages [P, Hkv, ps, d] uint8, scale [P, Hkv], table [B, T],
lens [B].  Attention is the plain definition (P3 section 3.1: scores, softmax,
weighted sum) over the slots in order.
"""
from __future__ import annotations

import numpy as np

# kind -> (exponent bits, mantissa bits, bias)
_FIELDS = {"e4m3": (4, 3, 7), "e5m2": (5, 2, 15)}
LARGEST = {"e4m3": 448.0, "e5m2": 57344.0}


def code_values(kind):
    """The value of each of the 256 codes (NaN and, for e5m2, infinities among them)."""
    ebits, mbits, bias = _FIELDS[kind]
    out = np.empty(256)
    for c in range(256):
        sign = -1.0 if c & 0x80 else 1.0
        e, m = (c >> mbits) & ((1 << ebits) - 1), c & ((1 << mbits) - 1)
        if kind == "e5m2" and e == 31:
            out[c] = sign * np.inf if m == 0 else np.nan
        elif kind == "e4m3" and (c & 0x7F) == 0x7F:
            out[c] = np.nan
        elif e == 0:
            out[c] = sign * m * 2.0 ** (1 - bias - mbits)
        else:
            out[c] = sign * (1.0 + m / (1 << mbits)) * 2.0 ** (e - bias)
    return out


def encode(x, kind):
    """Nearest code of each value, ties to the even mantissa; values beyond the largest code give the largest;
    infinities and NaN give those of the type (e4m3 has NaN only)."""
    x = np.asarray(x, dtype=np.float64)
    vals = code_values(kind)[:128]
    n = int(np.isfinite(vals).sum())
    grid = vals[:n]  # codes 0 .. n-1 ascend
    mag = np.abs(np.where(np.isfinite(x), x, 0.0))
    hi = np.clip(np.searchsorted(grid, mag), 1, n - 1)
    lo = hi - 1
    dlo, dhi = mag - grid[lo], grid[hi] - mag
    pick = np.where(dlo < dhi, lo, np.where(dhi < dlo, hi, np.where(lo % 2 == 0, lo, hi)))
    pick = np.where(mag >= grid[-1], n - 1, pick)
    code = pick | np.where(np.signbit(x), 0x80, 0)
    if kind == "e5m2":
        code = np.where(np.isinf(x), np.where(x < 0, 0xFC, 0x7C), code)
    else:
        code = np.where(np.isinf(x), 0x7F, code)
    return np.where(np.isnan(x), 0x7F, code).astype(np.uint8)


def slots(pages, scale, table_row, n, h, kind):
    """Values of slots 0 .. n-1 of one sequence and head, [n, d]; slots on a page outside the pool are NaN."""
    ps = pages.shape[2]
    out = np.full((n, pages.shape[3]), np.nan)
    vals = code_values(kind)
    for t in range((n + ps - 1) // ps):
        p = int(table_row[t])
        if 0 <= p < pages.shape[0]:
            rows = min(ps, n - t * ps)
            out[t * ps:t * ps + rows] = vals[pages[p, h, :rows]] * float(scale[p, h])
    return out


def attention(q, cache, kind, table, lens, scale, causal):
    """(O, LSE, weights, mass) of q [B, Hq, Nq, d]; cache = (k_pages, v_pages, k_scale, v_scale).  weights
    [B, Hkv, T * ps]: attention weight of each slot summed over the rows of its head; mass [B, Hq, Nq, d]: sum_j p_j |v_j|."""
    kp, vp, ks, vs = cache
    B, Hq, Nq, d = q.shape
    Hkv, ps = kp.shape[1], kp.shape[2]
    g = Hq // Hkv
    o, mass = np.zeros((B, Hq, Nq, d)), np.zeros((B, Hq, Nq, d))
    lse = np.full((B, Hq, Nq), -np.inf)
    weights = np.zeros((B, Hkv, table.shape[1] * ps))
    for b in range(B):
        n = int(lens[b])
        for h in range(Hkv):
            if n == 0:
                continue
            k, v = (slots(x, s, table[b], n, h, kind) for x, s in ((kp, ks), (vp, vs)))
            bad = np.isnan(k).all(axis=1) & np.isnan(v).all(axis=1)
            v = np.where(bad[:, None], 0.0, v)
            for hq in range(h * g, (h + 1) * g):
                s = scale * (q[b, hq] @ np.where(bad[:, None], 0.0, k).T)
                j = np.arange(n)
                hidden = bad[None] | ((j[None] > n - Nq + np.arange(Nq)[:, None]) if causal else False)
                s = np.where(hidden, -np.inf, s)
                top = s.max(axis=1, keepdims=True)
                seen = np.isfinite(top[:, 0])
                if not seen.any():
                    continue
                e = np.exp(s[seen] - top[seen])
                l = e.sum(axis=1, keepdims=True)
                p = e / l
                o[b, hq][seen] = p @ v
                mass[b, hq][seen] = p @ np.abs(v)
                lse[b, hq][seen] = (top[seen] + np.log(l))[:, 0]
                weights[b, h, :n] += p.sum(axis=0)
    return o, lse, weights, mass


def append_scale(amax, kind):
    """The smallest power of two s >= 2^-100 with amax <= LARGEST * s."""
    e = -100
    while amax > LARGEST[kind] * 2.0 ** e:
        e += 1
    return 2.0 ** e


def append(pages, scale, kind, table, x, lens, counts):
    """Append x [B, Hkv, N, d] (counts[b] tokens each), in place on copies: returns (pages, scale)."""
    pages, scale = pages.copy(), scale.astype(np.float64).copy()
    vals, ps = code_values(kind), pages.shape[2]
    for b in range(x.shape[0]):
        n, c = int(lens[b]), int(counts[b])
        for t in range(n // ps, (n + c + ps - 1) // ps if c else 0):
            lo, hi = max(n, t * ps), min(n + c, t * ps + ps)
            p = int(table[b, t])
            for h in range(pages.shape[1]):
                new = x[b, h, lo - n:hi - n].astype(np.float64)
                fin = np.abs(new[np.isfinite(new)])
                s = append_scale(float(fin.max()) if fin.size else 0.0, kind)
                if lo > t * ps:
                    was = scale[p, h]
                    s = max(s, was)
                    if s != was:
                        ratio = np.float32(was) / np.float32(s)  # one float32 rounding, then the product's
                        old = vals[pages[p, h, :lo - t * ps]].astype(np.float32) * ratio
                        pages[p, h, :lo - t * ps] = encode(old, kind)
                # a scale that was not a power of two: the quotient is rounded to float32 first
                pages[p, h, lo - t * ps:hi - t * ps] = encode((new.astype(np.float32) / np.float32(s)), kind)
                scale[p, h] = s
    return pages, scale.astype(np.float32)


def evict_plan(weight, position, n, keep, recent):
    """(holes, movers) of one sequence and head: slots below min(n, keep) that leave, slots behind that stay."""
    m = min(n, keep)
    w, pos = np.asarray(weight[:n], dtype=np.float64), np.asarray(position[:n], dtype=np.int64)
    if m == n:
        return [], []
    protected = pos > pos.max() - recent
    # protected first, NaN next, then the weight; equal ones by slot
    order = sorted(range(n), key=lambda j: (0 if protected[j] else 1 if np.isnan(w[j]) else 2,
                                            0.0 if protected[j] or np.isnan(w[j]) else -w[j], j))
    kept = set(order[:m])
    return [j for j in range(m) if j not in kept], [j for j in range(m, n) if j in kept]


def evict(cache, kind, table, weight, position, lens, keep, recent):
    """Returns (k_pages, v_pages, k_scale, v_scale, weight, position, new_lens), all copies."""
    kp, vp, ks, vs = (x.copy() for x in cache)
    weight, position = weight.copy(), position.copy()
    vals, ps = code_values(kind), kp.shape[2]
    new_lens = np.minimum(lens, keep)
    for b in range(table.shape[0]):
        for h in range(kp.shape[1]):
            holes, movers = evict_plan(weight[b, h], position[b, h], int(lens[b]), keep, recent)
            m = int(new_lens[b])
            src_of = dict(zip(holes, movers))
            for pages, scale, src_pages, src_scale in ((kp, ks, cache[0], cache[2]), (vp, vs, cache[1], cache[3])):
                for t in sorted({j // ps for j in holes}):
                    p = int(table[b, t])
                    here = range(t * ps, min(m, t * ps + ps))
                    at = {j: src_of.get(j, j) for j in here}
                    scales = {j: src_scale[table[b, s // ps], h] for j, s in at.items()}
                    now = max(scales.values())
                    for j, s in at.items():
                        code = src_pages[table[b, s // ps], h, s % ps]
                        if scales[j] != now:
                            code = encode(vals[code].astype(np.float32) * (np.float32(scales[j]) / np.float32(now)), kind)
                        pages[p, h, j % ps] = code
                    scale[p, h] = now
            for j, s in src_of.items():
                weight[b, h, j], position[b, h, j] = weight[b, h, s], position[b, h, s]
    return kp, vp, ks, vs, weight, position, new_lens
