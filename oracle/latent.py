"""fp64 definitions of latent attention (numpy, CPU; shares no code with the kernels).

Expanded form: keys of head h are [kv[..., h, :dn] | k_rope], values kv[..., h, dn:];
query i sits at position Tk - Tq + i and sees the keys at or before it that are below
the sequence's live length.  Absorbed form: a cache row [c | k_rope] is the key, its
first r columns the value.  A row that sees nothing gives 0 and a log-sum of -inf.
"""
from __future__ import annotations

import numpy as np


def f64(x):
    return None if x is None else np.asarray(x.detach().double().cpu() if hasattr(x, "detach") else x, np.float64)


def ints(x):
    return None if x is None else np.asarray(x.detach().cpu() if hasattr(x, "detach") else x).astype(np.int64)


def softmax_rows(s, see):
    """Weights over the last axis of the visible scores, and the log of their sum."""
    s = np.where(see, s, -np.inf)
    top = s.max(-1, keepdims=True, initial=-np.inf)
    w = np.exp(s - np.where(np.isfinite(top), top, 0.0))
    tot = w.sum(-1, keepdims=True)
    with np.errstate(divide="ignore"):
        lse = (np.where(np.isfinite(top), top, 0.0) + np.log(tot))[..., 0]
    return w / np.where(tot > 0, tot, 1.0), lse


def heads(q, kv, k_rope):
    """q, k [B, H, T, dn + dr] and v [B, H, T, dv]."""
    q, kv, kr = f64(q), f64(kv), f64(k_rope)
    dn = q.shape[-1] - kr.shape[-1]
    k = np.concatenate([kv[..., :dn], np.broadcast_to(kr[:, :, None], (*kv.shape[:3], kr.shape[-1]))], -1)
    t = lambda x: np.swapaxes(x, 1, 2)  # noqa: E731
    return t(q), t(k), t(kv[..., dn:])


def visible(B, Tq, Tk, lens=None):
    """[B, 1, Tq, Tk] booleans."""
    pos, key = np.arange(Tq)[:, None] + Tk - Tq, np.arange(Tk)[None]
    n = (np.full(B, Tk) if lens is None else np.clip(ints(lens), 0, Tk))[:, None, None]
    return ((key <= pos)[None] & (key < n) & (pos[None] < n))[:, None]


def forward(q, kv, k_rope, lens, scale):
    """o [B, Tq, H, dv], lse [B, Tq, H]."""
    Q, K, V = heads(q, kv, k_rope)
    see = visible(Q.shape[0], Q.shape[2], K.shape[2], lens)
    V = np.where(see.any(2)[..., None], V, 0.0)   # what no row sees may hold anything
    K = np.where(see.any(2)[..., None], K, 0.0)
    p, lse = softmax_rows(Q @ np.swapaxes(K, 2, 3) * scale, see)
    return np.swapaxes(p @ V, 1, 2), np.swapaxes(lse, 1, 2)


def backward(q, kv, k_rope, lens, o, lse, d_o, scale):
    """dq, dkv, dk_rope by the formulas, from the forward's o and lse as given."""
    Q, K, V = heads(q, kv, k_rope)
    see = visible(Q.shape[0], Q.shape[2], K.shape[2], lens)
    t = lambda x: np.swapaxes(f64(x), 1, 2)  # noqa: E731
    O, dO, L = t(o), t(d_o), t(lse)[..., None]
    with np.errstate(over="ignore", invalid="ignore"):
        p = np.where(see, np.exp(Q @ np.swapaxes(K, 2, 3) * scale - L), 0.0)
    ds = p * (dO @ np.swapaxes(V, 2, 3) - (dO * O).sum(-1, keepdims=True)) * scale
    dq, dk, dv = ds @ K, np.swapaxes(ds, 2, 3) @ Q, np.swapaxes(p, 2, 3) @ dO
    dn = V.shape[-1] and Q.shape[-1] - f64(k_rope).shape[-1]
    dkv = np.concatenate([dk[..., :dn], dv], -1)
    return np.swapaxes(dq, 1, 2), np.swapaxes(dkv, 1, 2), dk[..., dn:].sum(1)


def rows_of(cache, table, length, n):
    """The rows of sequence n's cached tokens and whether each is there (its page exists)."""
    pages, page = cache.shape[:2]
    length = min(max(int(length), 0), table.shape[1] * page)
    at = np.arange(length)
    ids = table[n, at // page]
    there = (ids >= 0) & (ids < pages)
    if not pages:
        return np.zeros((length, cache.shape[2])), there
    rows = np.where(there, ids, 0) * page + at % page
    x = cache.reshape(-1, cache.shape[2])[rows]   # only the rows in use are widened
    return np.where(there[:, None], f64(x), 0.0), there


def absorbed(q, cache, table, lens, scale, r, draft=None, tree=None, weigh_abs=False):
    """o [N, M, H, r] and lse [N, M, H] for q [N, M, H, r + dr]; tree: int64 bits [N, M], or
    None for a chain.  weigh_abs: the weights times |values| in place of o."""
    Q, table, lens, tree = f64(q), ints(table), ints(lens), ints(tree)
    N, M, H, D = Q.shape
    o, lse = np.zeros((N, M, H, r)), np.zeros((N, M, H))
    for n in range(N):
        x, there = rows_of(cache, table, lens[n], n)
        see = np.broadcast_to(there, (M, len(there)))
        if draft is not None:
            x = np.concatenate([x, f64(draft[n])])
            own = np.tril(np.ones((M, M), bool)) if tree is None else \
                np.array([[(int(tree[n, i]) >> j) & 1 == 1 for j in range(M)] for i in range(M)]).reshape(M, M)
            see = np.concatenate([see, own], 1)
        p, l = softmax_rows(Q[n] @ x.T * scale, see[:, None])
        o[n], lse[n] = p @ (np.abs(x[:, :r]) if weigh_abs else x[:, :r]), l
    return o, lse
