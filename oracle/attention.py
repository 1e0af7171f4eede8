"""fp64 definitions of grouped attention (numpy, CPU; shares no code with the kernels).

Packed tokens [T, heads, D]; query head h reads key head h // (Hq // Hk).  Sequence b has the
query rows cu_q[b] .. cu_q[b + 1] - 1 and the keys cu_k[b] .. cu_k[b + 1] - 1; row i of lq
sees the keys up to lk - lq + i.  A row that sees nothing gives 0 and a log-sum of -inf.
"""
from __future__ import annotations

import numpy as np

from .latent import f64, ints, softmax_rows

BLOCK = 16   # tokens that share a scale


# --- prologue -------------------------------------------------------------------

def turn(x, inv_freq, pos, back=False):
    """Channel pairs (i, i + R / 2) of x [T, H, D] turned by pos * inv_freq[i] (or back)."""
    if inv_freq is None:
        return x
    f = f64(inv_freq)
    h = len(f)
    a = np.outer(f64(pos), f)[:, None]
    c, s = np.cos(a), np.sin(-a if back else a)
    y = x.copy()
    y[..., :h] = x[..., :h] * c - x[..., h:2 * h] * s
    y[..., h:2 * h] = x[..., h:2 * h] * c + x[..., :h] * s
    return y


def prologue(x, w, inv_freq, pos, eps):
    """Norm over the channels of every head, then the rotation."""
    x = f64(x)
    return turn(x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * f64(w), inv_freq, pos)


def prologue_backward(x, w, inv_freq, pos, dy, eps):
    """dx, dw."""
    x, w = f64(x), f64(w)
    r = 1 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    z = turn(f64(dy), inv_freq, pos, back=True)
    return r * (w * z - x * r * (w * z * x * r).mean(-1, keepdims=True)), (z * x * r).sum((0, 1))


# --- whole sequences ------------------------------------------------------------

def sequences(cu_q, cu_k):
    cu_q = ints(cu_q)
    cu_k = cu_q if cu_k is None else ints(cu_k)
    return zip(cu_q, cu_q[1:], cu_k, cu_k[1:])


def visible(lq, lk):
    """[lq, lk] booleans."""
    return np.arange(lk)[None] <= (np.arange(lq) + lk - lq)[:, None]


def heads(x, a, b, G=1):
    """Rows a .. b - 1 as [H, rows, D], repeated for the G heads that share them."""
    return np.repeat(np.swapaxes(f64(x[a:b]), 0, 1), G, 0)


def forward(q, k, v, cu_q, cu_k, scale):
    """o [Tq, Hq, D], lse [Tq, Hq]; NaN in rows of no sequence."""
    G = q.shape[1] // k.shape[1]
    o, lse = np.full(q.shape, np.nan), np.full(q.shape[:2], np.nan)
    for a, b, c, e in sequences(cu_q, cu_k):
        if a == b:
            continue
        p, l = softmax_rows(heads(q, a, b) @ np.swapaxes(heads(k, c, e, G), 1, 2) * scale, visible(b - a, e - c))
        o[a:b], lse[a:b] = np.swapaxes(p @ heads(v, c, e, G), 0, 1), l.T
    return o, lse


def backward(q, k, v, o, lse, d_o, cu_q, cu_k, scale):
    """dq, dk, dv by the formulas, from the forward's o and lse as given; NaN in rows of no sequence."""
    Hk = k.shape[1]
    G = q.shape[1] // Hk
    dq, dk, dv = np.full(q.shape, np.nan), np.full(k.shape, np.nan), np.full(k.shape, np.nan)
    for a, b, c, e in sequences(cu_q, cu_k):
        Q, K, V, dO, O = heads(q, a, b), heads(k, c, e, G), heads(v, c, e, G), heads(d_o, a, b), heads(o, a, b)
        with np.errstate(over="ignore", invalid="ignore"):
            p = np.where(visible(b - a, e - c), np.exp(Q @ np.swapaxes(K, 1, 2) * scale - f64(lse[a:b]).T[..., None]), 0.0)
        ds = p * (dO @ np.swapaxes(V, 1, 2) - (dO * O).sum(-1, keepdims=True)) * scale
        shared = lambda x: np.swapaxes(x.reshape(Hk, G, *x.shape[1:]).sum(1), 0, 1)  # noqa: E731
        dq[a:b] = np.swapaxes(ds @ K, 0, 1)
        dk[c:e], dv[c:e] = shared(np.swapaxes(ds, 1, 2) @ Q), shared(np.swapaxes(p, 1, 2) @ dO)
    return dq, dk, dv


# --- the cache ------------------------------------------------------------------

def e4m3_values():
    """The value of each of the 256 bytes: sign, four exponent bits (bias 7), three of fraction."""
    out = np.zeros(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = np.nan if e == 15 and m == 7 else (8 + m) * 2.0 ** (e - 10) if e else m * 2.0 ** -9
        out[b] = -x if b & 128 else x
    return out


VALUES = e4m3_values()


def e4m3_round(x):
    """The nearest e4m3 value, ties to the even fraction (|x| at most 448; NaN stays)."""
    x = np.asarray(x, np.float64)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.floor(np.log2(np.abs(x)))
    step = 2.0 ** (np.maximum(np.where(np.isfinite(e), e, -9), -6) - 3)
    return np.round(x / step) * step


def scale_of(amax):
    """The smallest power of two, 2^-126 or more, that takes amax to 448 or less."""
    e = -126
    while amax > 448 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def append(k, v, cu, kc, vc, ks, vs, table, lens):
    """In place: kc, vc values / scale [pages, Hk, page, D] and [pages, Hk, page / 16, D, 16] as
    fp64, ks, vs their scales."""
    table, lens = ints(table), ints(lens)
    pages, Hk, page, D = kc.shape
    N, width = table.shape
    cu = np.arange(N + 1) if cu is None else ints(cu)
    for x, cache, scale in ((f64(k), kc.reshape(pages, Hk, page // BLOCK, BLOCK, D), ks), (f64(v), np.swapaxes(vc, 3, 4), vs)):
        for n in range(N):
            first = max(int(lens[n]), 0) - (cu[n + 1] - cu[n])
            for b in range(max(first, 0) // BLOCK, -(-min(int(lens[n]), width * page) // BLOCK)):
                lo, hi = max(first, b * BLOCK, 0), min(int(lens[n]), (b + 1) * BLOCK, width * page)
                p, j = table[n, b * BLOCK // page], b * BLOCK % page // BLOCK
                if lo >= hi or not 0 <= p < pages:
                    continue
                for h in range(Hk):
                    new = x[cu[n] + lo - first:cu[n] + hi - first, h]
                    s = scale_of(np.abs(new[np.isfinite(new)]).max(initial=0))
                    if lo > b * BLOCK:
                        s = max(s, scale[p, h, j])
                        if s != scale[p, h, j]:
                            old = cache[p, h, j, :lo - b * BLOCK]
                            old[...] = e4m3_round(old * (scale[p, h, j] / s))
                    scale[p, h, j] = s
                    cache[p, h, j, lo - b * BLOCK:hi - b * BLOCK] = e4m3_round(np.where(np.isfinite(new), new, np.nan) / s)


def cached(kc, vc, ks, vs, table, length, n):
    """Keys and values [Hk, tokens, D] of sequence n's cached tokens, and whether each is there."""
    table = ints(table)
    pages, Hk, page, D = kc.shape
    length = min(max(int(length), 0), table.shape[1] * page) if pages else 0
    at = np.arange(length)
    ids = table[n, at // page] if length else at
    there = (ids >= 0) & (ids < pages)
    p, b, t = np.where(there, ids, 0), at % page // BLOCK, at % BLOCK
    k = kc.reshape(pages, Hk, page // BLOCK, BLOCK, D)[p, :, b, t] * ks[p, :, b][..., None] if length else np.zeros((0, Hk, D))
    v = np.swapaxes(vc, 3, 4)[p, :, b, t] * vs[p, :, b][..., None] if length else np.zeros((0, Hk, D))
    live = there[:, None, None]
    return np.swapaxes(np.where(live, k, 0), 0, 1), np.swapaxes(np.where(live, v, 0), 0, 1), there


def step(q, kc, vc, ks, vs, table, lens, scale, weigh_abs=False):
    """o [N, Hq, D] and lse [N, Hq].  weigh_abs: the weights times |values| in place of o."""
    Q = f64(q)
    o, lse = np.zeros(Q.shape), np.zeros(Q.shape[:2])
    G = Q.shape[1] // kc.shape[1]
    for n in range(Q.shape[0]):
        k, v, there = cached(kc, vc, ks, vs, table, lens[n], n)
        for h in range(Q.shape[1]):
            p, l = softmax_rows(Q[n, h:h + 1] @ k[h // G].T * scale, there[None])
            o[n, h], lse[n, h] = (p @ (np.abs(v[h // G]) if weigh_abs else v[h // G]))[0], l[0]
    return o, lse
