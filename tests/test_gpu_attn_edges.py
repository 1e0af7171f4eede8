"""Grouped attention at its edges: rows of one key, peaked rows, calls whose offsets and lengths
change while workgroups share the work, guarded workspaces of every form, and strided inputs at
the largest step, against the fp64 oracle and its own gradients (tolerances as in test_gpu_attn.py,
u = 2^-8 or 2^-24, e = 2^-24)."""
import numpy as np
import pytest
import torch

import attn_plans
import gated_deltanet_layer_amd as gdn
from oracle import attention as ref
from test_gpu_attn import DEV, DT, E, U, _bwd_tol, _close, _fwd_tol, _on, _packed, _parts, _say

pytestmark = pytest.mark.gpu


# --- rows of one key ------------------------------------------------------------

ONE_KEY = [
    ([1], None, 1, 1), ([1, 1, 0, 1], None, 56, 8), ([1, 1], None, 64, 1), ([1] * 70, None, 6, 2), ([1, 2, 64, 1, 300], None, 12, 3),
    ([1, 5], [1, 2], 64, 1), ([140, 3], [1, 3], 4, 2), ([9, 70, 2], [4, 1, 5], 33, 1), ([1100], None, 4, 2)]


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lq,lk,Hq,Hk", ONE_KEY)
def test_rows_of_one_key(lq, lk, Hq, Hk, D, dt):
    """Their weight is 1 whatever the score, so the gradients of the score are exactly 0: dq of
    such rows, and dk of a key that only they see.  dv of that key is the sum of d_o, times
    weights of 1 that are off by the score's and the lse's roundings as in test_gpu_attn.py."""
    _say(f"one key lq {lq[:6]} lk {lk} Hq{Hq} Hk{Hk} D{D} {dt}")
    d = _packed(lq, lk, Hq, Hk, D, dt, seed=51, before=2, behind=1)
    x = _on(d)
    o, lse = gdn.attn_fwd(x["q"], x["k"], x["v"], x["cu_q"], x["cu_k"])
    g = gdn.attn_bwd(x["q"], x["k"], x["v"], o, lse, x["d_o"], x["cu_q"], x["cu_k"])
    torch.cuda.synchronize()
    G, scale, u = Hq // Hk, D ** -0.5, U[dt]
    found = 0
    for a, b, c, e in ref.sequences(d["cu_q"], d["cu_k"]):
        row = a + (b - a) - (e - c)   # whose position is 0
        if e == c or not a <= row < b:
            continue
        found += 1
        assert (g["dq"][row] == 0).all(), (row, g["dq"][row].abs().max())
        if e - c == 1:
            assert (g["dk"][c] == 0).all(), (c, g["dk"][c].abs().max())
            dO = np.abs(ref.f64(d["d_o"][row])).reshape(Hk, G, D)
            want = ref.f64(d["d_o"][row]).reshape(Hk, G, D).sum(1)
            s = scale * (np.abs(ref.f64(d["q"][row])).reshape(Hk, G, D) * np.abs(ref.f64(d["k"][c]))[:, None]).sum(-1, keepdims=True)
            off = (D + 4) * E * s + 4 * E * s + 8 * E   # |lse| <= s
            _close("dv", g["dv"][c], want, ((u + off + (G + 8) * E) * dO).sum(1) + u * np.abs(want) + 1e-37)
    assert found


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_rows_of_one_key_where_keys_are_cut(dt):
    """The same where dq is added up from pieces."""
    assert attn_plans.bwd(dt, 2, 1101, 1101, 4, 2)["kp"] > 1
    d = _on(_packed([1100, 1], None, 4, 2, 64, dt, seed=52))
    o, lse = gdn.attn_fwd(d["q"], d["k"], d["v"], d["cu_q"])
    g = gdn.attn_bwd(d["q"], d["k"], d["v"], o, lse, d["d_o"], d["cu_q"])
    assert (g["dq"][[0, 1100]] == 0).all() and (g["dk"][1100] == 0).all()
    assert (g["dq"][1:1100] != 0).any(-1).all() and (g["dk"][:1100] != 0).any(-1).all()


# --- sizes ----------------------------------------------------------------------

def test_a_million_sequences_of_which_most_are_empty():
    """1000 single tokens among 1,100,000 sequences, 8 heads: more than 2^23 row tiles, which the
    forward takes with 256 threads each.  o is v (a weight of 1 over a sum of 1, each to 16 e, and
    the rounding), dv is d_o, the gradients of the score are 0."""
    B, T, H, D = 1_100_000, 1000, 8, 64
    p = attn_plans.fwd("bf16", B, T, T, H, H)
    assert p["form"] == "whole" and 1 << 23 < p["tiles"] * H < 1 << 24
    g = torch.Generator().manual_seed(3)
    one = torch.zeros(B, dtype=torch.int32)
    one[torch.randperm(B, generator=g)[:T]] = 1
    cu = torch.cat((torch.zeros(1, dtype=torch.int32), one.cumsum(0).to(torch.int32))).to(DEV)
    q, k, v, d_o = (torch.randn(T, H, D, generator=g).to(torch.bfloat16).to(DEV) for _ in range(4))
    o, lse = gdn.attn_fwd(q, k, v, cu)
    assert ((o.double() - v.double()).abs() <= 2 * U["bf16"] * v.double().abs()).all()
    s, most = (f(q.double() * k.double()).sum(-1) * D ** -0.5 for f in (lambda x: x, torch.abs))
    assert ((lse.double() - s).abs() <= (D + 4) * E * most + 16 * E + 4 * E * s.abs()).all()
    grads = gdn.attn_bwd(q, k, v, o, lse, d_o, cu)
    assert (grads["dq"] == 0).all() and (grads["dk"] == 0).all()
    assert ((grads["dv"].double() - d_o.double()).abs() <= 2 * U["bf16"] * d_o.double().abs()).all()


# --- the gradients of the formula -----------------------------------------------

def _check_gradients(d, dt, scale):
    """Forward and backward in a row, against the formulas with o and lse as the forward gave them
    and against the gradients in 64 bits, with the oracle's own.  To what the backward may be off
    by with o and lse as given (_bwd_tol) comes what those are off by: lse by tl, which is a factor
    1 + tl of every weight, and o by to, its rounding among it, which is |d_o| . to in D, in every
    dS = scale P (dP - D) of the row.

    The hardware's exponential gives 0 for results below the normal range, so a weight may also be
    off by 2^-126.  That is 2^-126 |d_o| of a row in dv and 2^-126 scale |dP - D| in its dS; with
    scores of hundreds, keys at a distance have no other weights, and their gradients of 10^-37
    are of such terms: 900 rows, scale 2, |dP - D| up to 40 and |q| up to 4 give 2^-126 * 320 =
    4e-36 a row.
    """
    x = _on(d)
    o, lse = gdn.attn_fwd(x["q"], x["k"], x["v"], x["cu_q"], x["cu_k"], scale=scale)
    g = gdn.attn_bwd(x["q"], x["k"], x["v"], o, lse, x["d_o"], x["cu_q"], x["cu_k"], scale=scale)
    torch.cuda.synchronize()
    u, Hk = U[dt], d["k"].shape[1]
    G = d["q"].shape[1] // Hk
    o64, l64 = ref.forward(d["q"], d["k"], d["v"], d["cu_q"], d["cu_k"], scale)
    to, tl = _fwd_tol(d, scale, u)
    to, tl = to + u * np.abs(o64), tl + 4 * E * np.abs(np.where(np.isfinite(l64), l64, 0))
    for o1, l1, eo, el in ((o.cpu(), lse.cpu(), 0 * to, 0 * tl), (o64, l64, to, tl)):
        want = ref.backward(d["q"], d["k"], d["v"], o1, l1, d["d_o"], d["cu_q"], d["cu_k"], scale)
        tols = _bwd_tol(d, o1, l1, scale, u)
        for a, b, c, e, Q, K, V, see in _parts(d):
            dO, O = ref.heads(d["d_o"], a, b), ref.heads(o1, a, b)
            p, _ = ref.softmax_rows(Q @ K.swapaxes(1, 2) * scale, see)
            off = np.where(see, p * np.swapaxes(el[a:b], 0, 1)[..., None] + 2.0 ** -126, 0)
            D = (np.abs(dO) * np.swapaxes(eo[a:b], 0, 1)).sum(-1, keepdims=True)
            dS = scale * (off * np.abs(dO @ V.swapaxes(1, 2) - (dO * O).sum(-1, keepdims=True)) + p * D)
            shared = lambda x: np.swapaxes(x.reshape(Hk, G, *x.shape[1:]).sum(1), 0, 1)  # noqa: E731
            tols[0][a:b] += np.swapaxes(dS @ np.abs(K), 0, 1)
            tols[1][c:e] += shared(dS.swapaxes(1, 2) @ np.abs(Q))
            tols[2][c:e] += shared(off.swapaxes(1, 2) @ np.abs(dO))
        for n, w, t in zip(("dq", "dk", "dv"), want, tols):
            _close(n, g[n], w, t + u * np.abs(w) + 1e-37)


def _peaked(T, D, dt, seed=5):
    """Scores of some hundreds (scale 2): one key has nearly all weight of most rows."""
    d = _packed([T], None, 4, 2, D, dt, seed=seed)
    d["k"] = (d["k"].float() * torch.linspace(0.2, 3.0, T)[:, None, None]).to(DT[dt])
    return d


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("lq,lk,Hq,Hk,D", [
    ([1, 2, 64, 300, 65], None, 12, 3, 64), ([700, 0, 1], None, 4, 1, 128), ([40, 129], [500, 100], 8, 2, 128), ([3, 1], [900, 130], 5, 5, 64)])
def test_gradients_of_the_formula(lq, lk, Hq, Hk, D, dt):
    _say(f"gradients lq {lq} lk {lk} Hq{Hq} Hk{Hk} D{D} {dt}")
    _check_gradients(_packed(lq, lk, Hq, Hk, D, dt, seed=61), dt, D ** -0.5)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("T,D", [(100, 64), (400, 64), (300, 128), (900, 128)])
def test_gradients_of_peaked_rows(T, D, dt):
    """Rows of up to 128 keys, whose D is of P and dP in bf16, and of more, whose D is do . o."""
    _say(f"peaked T{T} D{D} {dt}")
    _check_gradients(_peaked(T, D, dt), dt, 2.0)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("scale", [1e-3, 0.7, 5.0])
def test_backward_of_other_scales(scale, dt):
    _check_gradients(_packed([330, 1, 70], None, 6, 2, 64, dt, seed=63), dt, scale)
