"""64-bit restatements of the scored router and of the block-scaled 8-bit
operators, and their error bounds, for the tests.

Plain NumPy loops over the definitions in include/moe_decode.h; no code is
shared with the library."""
import math

import numpy as np

BLOCK = 128
E4M3 = np.array(sorted({s * m * 2.0 ** e for s in (1, -1) for e, m in
                        [(-9, j) for j in range(8)] +                       # subnormals: j * 2^-9
                        [(x - 10, 8 + j) for x in range(1, 16) for j in range(8) if (x, j) != (15, 7)]}))


def e4m3_decode(b):
    """Values of e4m3 bytes."""
    b = np.asarray(b, np.uint8).astype(np.int64)
    s, x, m = b >> 7, (b >> 3) & 15, b & 7
    v = np.where(x == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (x - 10.0))
    v = np.where((x == 15) & (m == 7), np.nan, v)
    return np.where(s == 1, -v, v)


def e4m3_round(v):
    """Nearest e4m3 value, ties to even, |v| <= 448."""
    v = np.asarray(v, np.float64)
    e = np.frexp(v)[1] - 1.0
    step = 2.0 ** (np.maximum(e, -6.0) - 3.0)
    return np.round(v / step) * step  # np.round: half to even


def scale_of(top):
    """Smallest power of two s >= 2^-120 with top <= 448 s; 1 for zeros."""
    top = np.asarray(top, np.float64)
    s = np.ones_like(top)
    for i in np.ndindex(top.shape):
        if top[i] > 0:
            e = math.frexp(top[i] / 448.0)
            s[i] = 2.0 ** max(-120, e[1] - 1 if e[0] == 0.5 else e[1])
    return s


def quantize(x, block_rows=1):
    """(e4m3 values, scales) of x[rows][cols]."""
    x = np.asarray(x, np.float64)
    r, c = x.shape
    rb, cb = -(-r // block_rows), -(-c // BLOCK)
    top = np.zeros((rb, cb))
    for i in range(rb):
        for j in range(cb):
            b = x[i * block_rows:(i + 1) * block_rows, j * BLOCK:(j + 1) * BLOCK]
            top[i, j] = np.abs(b).max()
    s = scale_of(top)
    full = spread(s, r, c, block_rows)
    return e4m3_round(x / full), s


def spread(s, r, c, block_rows):
    return np.repeat(np.repeat(s, block_rows, 0)[:r], BLOCK, 1)[:, :c]


def route(logits, k, sigmoid, bias=None, groups=1, top_groups=1, best=1, renorm=True, scale=1.0):
    """(sel[B][k], w[B][k]) by the definition, token by token."""
    B, E = logits.shape
    sel, w = np.full((B, k), -1, np.int32), np.zeros((B, k))
    per = E // groups
    for t in range(B):
        l = np.asarray(logits[t], np.float64)
        l = np.where(np.isnan(l), -np.inf, np.minimum(l, float(np.finfo(np.float32).max)))
        pool = [e for e in range(E) if l[e] > -np.inf]
        if not pool:
            continue
        if sigmoid:
            s = {e: 1.0 / (1.0 + math.exp(-l[e])) if l[e] > -700 else math.exp(max(l[e], -1e4)) for e in pool}
        else:
            m = max(l[e] for e in pool)
            z = math.fsum(math.exp(l[e] - m) for e in pool)
            s = {e: math.exp(l[e] - m) / z for e in pool}
        c = {e: s[e] + (float(bias[e]) if bias is not None else 0.0) for e in pool}
        if groups > 1:
            value = {}
            for g in range(groups):
                m = sorted((c[e] for e in pool if e // per == g), reverse=True)[:best]
                if m:
                    value[g] = math.fsum(m)
            kept = sorted(value, key=lambda g: (-value[g], g))[:top_groups]
            pool = [e for e in pool if e // per in kept]
        chosen = sorted(pool, key=lambda e: (-c[e], e))[:k]
        total = math.fsum(s[e] for e in chosen) if renorm else 1.0
        for j, e in enumerate(chosen):
            sel[t, j] = e
            w[t, j] = s[e] / total * scale if total > 0 else 0.0
    return sel, w


def lists_of(sel, w, E):
    """Per-expert lists of a choice, as the header describes moe_lists_t."""
    B, k = sel.shape
    per = {}
    for t in range(B):
        for j in range(k):
            if sel[t, j] >= 0:
                per.setdefault(int(sel[t, j]), []).append((t, w[t, j]))
    active = np.full(E, -1, np.int32)
    offsets = np.zeros(E + 1, np.int32)
    tok, lw = np.full(B * k, -1, np.int32), np.zeros(B * k, np.float64)
    n = 0
    for i, e in enumerate(sorted(per)):
        active[i], offsets[i] = e, n
        for t, x in per[e]:
            tok[n], lw[n] = t, x
            n += 1
    offsets[len(per):] = n
    return {"n_active": len(per), "active": active, "offsets": offsets, "tok": tok, "w": lw}


def entries(lists):
    """(slot, expert, first, end) of every active expert."""
    return [(i, int(lists["active"][i]), int(lists["offsets"][i]), int(lists["offsets"][i + 1]))
            for i in range(int(lists["n_active"]))]


# A product of two e4m3 values is exact in fp32.  Adding n of them in fp32,
# in any order, with each addition off by at most one unit in the last place
# (a tensor core may truncate) is off by at most n 2^-23 times the sum of the
# magnitudes; the scale products and their additions add 3 per block.
def sum_bound(n, magnitudes):
    return (n + 3 * -(-n // BLOCK) + 4) * 2.0 ** -23 * magnitudes


HALF_STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}


def ffn(x, weights, lists, B):
    """(y, bound) of the block-scaled expert FFN; weights: 64-bit matrices
    (Wgate, Wup, Wdown).  The bound counts the fp32 sums, and the rounding of
    h where the error of the value before it can change the result."""
    Wg, Wu, Wd = weights
    d = x.shape[1]
    q, s = quantize(x)
    xv = q * spread(s, B, d, 1)
    y, bound = np.zeros((B, d)), np.zeros((B, d))
    for _, e, lo, hi in entries(lists):
        tok = lists["tok"][lo:hi]
        a = xv[tok]
        g, u = a @ Wg[e].T, a @ Wu[e].T
        eg, eu = (sum_bound(d, np.abs(a) @ np.abs(W[e]).T) for W in (Wg, Wu))
        z = 1.0 / (1.0 + np.exp(-g))
        h = g * z * u
        # |d silu / dg| <= 1.1; exp, the division and two products round, and a
        # fast exp(-g) = 2^(-g log2 e) also turns the rounding of its argument
        # (|g| log2 e 2^-24) into a relative error of |g| 2^-24
        eh = 1.1 * eg * np.abs(u) + np.abs(g * z) * eu + 1.1 * eg * eu + (8 + np.abs(g)) * 2.0 ** -23 * np.abs(h)
        hq, hs = quantize(h)
        n, F = h.shape
        full = spread(hs, n, F, 1)
        top = np.abs(h)
        # a block whose largest magnitude could fall on the other side of its
        # scale's border may take twice or half the scale: a step more each way
        lo_v = e4m3_round(np.clip((h - eh) / full, -448, 448)) * full
        hi_v = e4m3_round(np.clip((h + eh) / full, -448, 448)) * full
        dh = hi_v - lo_v
        for j in range(hs.shape[1]):
            b = slice(j * BLOCK, (j + 1) * BLOCK)
            i = np.argmax(top[:, b], 1)
            r = np.arange(n)
            m, em = top[:, b][r, i], eh[:, b][r, i]
            unsure = (scale_of(m + em) != scale_of(np.maximum(m - em, 0))) & (m > 0)
            dh[:, b] = np.where(unsure[:, None], 2.0 ** -3 * top[:, b] + hs[:, j:j + 1] * 2.0 ** -8, dh[:, b])
        hv = hq * full
        w = lists["w"][lo:hi][:, None]
        part = hv @ Wd[e].T
        mag = np.abs(hv) @ np.abs(Wd[e]).T
        np.add.at(y, tok, w * part)
        np.add.at(bound, tok, np.abs(w) * (dh @ np.abs(Wd[e]).T + sum_bound(F, mag) + 16 * 2.0 ** -24 * np.abs(part)))
    return y, bound
