"""GPU parity of the grouped-attention entry points against the fp64 oracle.

Tolerances are elementwise and follow from the roundings of the computation, u being
half a step of the storage type (bf16 2^-8, fp32 2^-24) and e = 2^-24:

 * a score is an fp32 sum of D products: off by at most ds = (D + 4) e scale |q||k| (the
   largest sum of absolute products of the row), so a weight by a factor 1 + 2 ds + 8 e
   (the row's normaliser moves with it; 8 e for the exponential, the division and the
   base change);
 * weights and dS are rounded to the storage type (u), sums run over L terms in fp32
   (L e), the result is rounded (u).

Hence |o - ref| <= u |ref| + (u + 2 ds + (L + 8) e) sum_j P_ij |v_j|, and likewise for
the gradients with the absolute values of their terms.
"""
import math

import numpy as np
import pytest
import torch

import gated_deltanet_layer_amd as gdn
from oracle import attention as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
U = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}


def _say(*a):
    print("[attn]", *a, flush=True)


def _close(name, x, want, tol):
    """Within the tolerance where the oracle has a value (it has NaN in rows of no sequence)."""
    x = x.detach().double().cpu().numpy()
    assert x.shape == want.shape, (name, x.shape, want.shape)
    skip = (np.isneginf(x) & np.isneginf(want)) | np.isnan(want)
    assert np.isfinite(x[~skip]).all(), f"{name}: not finite"
    d = np.where(skip, 0.0, np.abs(np.where(skip, 0, x) - np.where(skip, 0, want)))
    tol = np.where(skip, 0.0, tol)
    if d.size:
        i = np.unravel_index(np.argmax(d - tol), d.shape)
        assert d[i] <= tol[i], f"{name}: off by {d[i]:.3e} at {i}, allowed {tol[i]:.3e}"
        _say(f"{name}: largest share of the tolerance {float(np.max(d / np.maximum(tol, 1e-300))):.2f}")


def _dev(d):
    return {k: v.to(DEV) if isinstance(v, torch.Tensor) else v for k, v in d.items()}


# --- prologue -------------------------------------------------------------------

def _raw(T, Hq, Hk, D, R, dt, seed=0, far=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    fused = r(T, Hq + 2 * Hk, D).to(DT[dt])
    return dict(fused=fused, w_q=1 + r(D) / 4, w_k=1 + r(D) / 4, inv_freq=10000.0 ** (-torch.arange(0, R, 2) / R) if R else None,
                pos=torch.randint(-5, 600, (T,), generator=g, dtype=torch.int32) + far,
                d_q=r(T, Hq, D).to(DT[dt]), d_k=r(T, Hk, D).to(DT[dt]))


def _split(d, Hq, Hk):
    return d["fused"][:, :Hq], d["fused"][:, Hq:Hq + Hk]


def _partners(x, R):
    """The sum of the absolute values of a channel and its partner in the rotation."""
    y = np.abs(x)
    if R:
        h = R // 2
        y = np.concatenate([y[..., :h] + y[..., h:R], y[..., :h] + y[..., h:R], y[..., R:]], -1)
    return y


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("T,Hq,Hk,D,R,far", [
    (1, 1, 1, 64, 64, 0), (3, 4, 2, 128, 128, 0), (17, 5, 1, 64, 16, 1000000), (300, 3, 3, 128, 96, 262144), (5, 40, 8, 128, 0, 0),
    (4, 7, 1, 64, 32, 2 ** 31 - 1000), (4099, 2, 1, 64, 64, 0), (4096, 1, 1, 128, 64, -2 ** 31 + 10)])
def test_prologue(T, Hq, Hk, D, R, far, dt):
    """Norm and rotation, from slices of one projection; gradients against the formulas.

    r = 1 / sqrt(mean + eps) is off by (D + 8) e of itself, a product by e; the angle's
    fraction is rounded to fp32 (pi 2^-25 in radians), and sincospi is good to 4 ulp: cos
    and sin to 6 e, 9 e with the products around them.
    """
    _say(f"prologue T{T} Hq{Hq} Hk{Hk} D{D} R{R} far {far} {dt}")
    d = _raw(T, Hq, Hk, D, R, dt, seed=T + D, far=far)
    x = _dev(d)
    eps = 1e-5
    args = [*_split(x, Hq, Hk), x["w_q"], x["w_k"], x["inv_freq"], x["pos"]]
    out = gdn.attn_prologue(*args, eps=eps)
    grads = gdn.attn_prologue_bwd(*args, x["d_q"], x["d_k"], eps=eps)
    torch.cuda.synchronize()
    for n, raw, y, H in (("q", _split(d, Hq, Hk)[0], out[0], Hq), ("k", _split(d, Hq, Hk)[1], out[1], Hk)):
        w, dy = d["w_" + n], d["d_" + n]
        want = ref.prologue(raw, w, d["inv_freq"], d["pos"], eps)
        X, W = ref.f64(raw), ref.f64(w)
        rr = 1 / np.sqrt((X * X).mean(-1, keepdims=True) + eps)
        _close(n, y, want, U[dt] * np.abs(want) + (D + 20) * E * _partners(X * rr * W, R) + 1e-37)
        dx, dw = ref.prologue_backward(raw, w, d["inv_freq"], d["pos"], dy, eps)
        A = _partners(ref.f64(dy), R)
        terms = rr * (np.abs(W) * A + np.abs(X) * rr * (np.abs(W) * A * np.abs(X) * rr).mean(-1, keepdims=True))
        _close(f"d{n}_raw", grads[f"d{n}_raw"], dx, U[dt] * np.abs(dx) + (3 * D + 40) * E * terms + 1e-37)
        _close("dw_" + n, grads["dw_" + n], dw, (T * H + D + 40) * E * (A * np.abs(X) * rr).sum((0, 1)) + 1e-37)


def test_prologue_gradients_into_slices():
    """Gradients written into slices of one tensor, whose other columns stay as they were."""
    T, Hq, Hk, D = 50, 4, 2, 64
    d = _dev(_raw(T, Hq, Hk, D, 64, "bf16", seed=3))
    q, k = _split(d, Hq, Hk)
    g = gdn.attn_prologue_bwd(q, k, d["w_q"], d["w_k"], d["inv_freq"], d["pos"], d["d_q"], d["d_k"])
    out = torch.full_like(d["fused"], 7.0)
    ws = torch.empty(gdn.gdn_attn_prologue_bwd_workspace_size(T, Hq, Hk, D, 64, torch.bfloat16), dtype=torch.uint8, device=DEV)
    dw = [torch.empty(D, device=DEV) for _ in range(2)]
    gdn.gdn_attn_prologue_bwd(q, k, d["w_q"], d["w_k"], d["inv_freq"], d["pos"], d["d_q"], d["d_k"], out[:, :Hq], out[:, Hq:Hq + Hk],
                              *dw, ws, 1e-6)
    assert torch.equal(out[:, :Hq], g["dq_raw"]) and torch.equal(out[:, Hq:Hq + Hk], g["dk_raw"])
    assert torch.equal(dw[0], g["dw_q"]) and torch.equal(dw[1], g["dw_k"]) and (out[:, Hq + Hk:] == 7).all()


def test_prologue_without_tokens():
    e = lambda *s: torch.empty(*s, device=DEV)  # noqa: E731
    w = torch.ones(64, device=DEV)
    q, k = gdn.attn_prologue(e(0, 4, 64), e(0, 2, 64), w, w, None, None)
    assert q.shape == (0, 4, 64) and k.shape == (0, 2, 64)
    g = gdn.attn_prologue_bwd(e(0, 4, 64), e(0, 2, 64), w, w, None, None, q, k)
    assert (g["dw_q"] == 0).all() and (g["dw_k"] == 0).all()


# --- whole sequences ------------------------------------------------------------

def _cu(lens, first=0):
    return torch.tensor([first + sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32)


def _packed(lq, lk, Hq, Hk, D, dt, seed=0, before=0, behind=0):
    """Packed sequences with `before` and `behind` rows of none around them."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).to(DT[dt])  # noqa: E731
    Tq, Tk = before + sum(lq) + behind, before + sum(lk or lq) + behind
    fused = r(Tk, Hq + 2 * Hk, D) if lk is None else None
    q, k, v = (r(Tq, Hq, D), r(Tk, Hk, D), r(Tk, Hk, D)) if lk else (fused[:, :Hq], fused[:, Hq:Hq + Hk], fused[:, Hq + Hk:])
    return dict(q=q, k=k, v=v, d_o=r(Tq, Hq, D), cu_q=_cu(lq, before), cu_k=_cu(lk, before) if lk else None)


def _on(d):
    """On the device, with q, k and v still slices of one tensor where they are."""
    x = _dev(d)
    if d["cu_k"] is None:
        Hq, Hk = d["q"].shape[1], d["k"].shape[1]
        fused = torch.cat((d["q"], d["k"], d["v"]), 1).to(DEV)
        x.update(q=fused[:, :Hq], k=fused[:, Hq:Hq + Hk], v=fused[:, Hq + Hk:])
    return x


def _parts(d):
    for a, b, c, e in ref.sequences(d["cu_q"], d["cu_k"]):
        G = d["q"].shape[1] // d["k"].shape[1]
        yield a, b, c, e, ref.heads(d["q"], a, b), ref.heads(d["k"], c, e, G), ref.heads(d["v"], c, e, G), ref.visible(b - a, e - c)


def _fwd_tol(d, scale, u):
    to, tl = np.zeros(d["q"].shape), np.zeros(d["q"].shape[:2])
    for a, b, c, e, Q, K, V, see in _parts(d):
        p, _ = ref.softmax_rows(Q @ K.swapaxes(1, 2) * scale, see)
        ds = (Q.shape[-1] + 4) * E * scale * np.where(see, np.abs(Q) @ np.abs(K).swapaxes(1, 2), 0).max(-1, keepdims=True, initial=0)
        L = see.sum(-1)[None, :, None]
        to[a:b] = np.swapaxes((u + 2 * ds + (L + 8) * E) * (p @ np.abs(V)), 0, 1)
        tl[a:b] = (ds + (L + 16) * E)[..., 0].T
    return to, tl


def _check_fwd(d, dt, scale=None):
    scale = 1 / math.sqrt(d["q"].shape[-1]) if scale is None else scale
    x = _on(d)
    o, lse = torch.full(d["q"].shape, 5.0, dtype=DT[dt], device=DEV), torch.full(d["q"].shape[:2], 5.0, device=DEV)
    B, Tq, Tk = len(d["cu_q"]) - 1, d["q"].shape[0], d["k"].shape[0]
    n = gdn.gdn_attn_fwd_workspace_size(B, Tq, Tk, d["q"].shape[1], *d["k"].shape[1:], DT[dt])
    ws = torch.full((n,), 255, dtype=torch.uint8, device=DEV) if n else None   # NaN
    gdn.gdn_attn_fwd(x["q"], x["k"], x["v"], x["cu_q"], x["cu_k"], o, lse, ws, scale)
    torch.cuda.synchronize()
    ro, rl = ref.forward(d["q"], d["k"], d["v"], d["cu_q"], d["cu_k"], scale)
    to, tl = _fwd_tol(d, scale, U[dt])
    _close("o", o, ro, to + U[dt] * np.abs(ro) + 1e-37)
    _close("lse", lse, rl, tl + 4 * E * np.abs(np.where(np.isfinite(rl), rl, 0)) + 1e-37)
    none = torch.from_numpy(np.isnan(rl)).to(DEV)   # rows of no sequence: as they were
    assert (o[none] == 5).all() and (lse[none] == 5).all()
    return o, lse


def _bwd_tol(d, o, lse, scale, u):
    """The terms' absolute values times what each may be off.  P: 2 ds + 8 e (and the
    rounding u in dv; for bf16 in dk half a step of fp16, 2^-11, of 4096 P, or of its
    subnormals, 2^-25 / 4096); dP - D: (D + 4) e sums of absolute products, and in D
    u |do| |o|, by which do . o of the rounded o may be off the sum of P dP, which the
    kernel takes for the first rows; dS: u."""
    Hk = d["k"].shape[1]
    G = d["q"].shape[1] // Hk
    tq, tk, tv = np.zeros(d["q"].shape), np.zeros(d["k"].shape), np.zeros(d["k"].shape)
    for a, b, c, e, Q, K, V, see in _parts(d):
        O, dO, L = ref.heads(o, a, b), ref.heads(d["d_o"], a, b), np.swapaxes(ref.f64(lse[a:b]), 0, 1)[..., None]
        L = np.where(np.isfinite(L), L, 0)
        D = Q.shape[-1]
        p = np.where(see, np.exp(np.where(see, Q @ K.swapaxes(1, 2) * scale - L, 0)), 0)
        ds = (D + 4) * E * scale * np.where(see, np.abs(Q) @ np.abs(K).swapaxes(1, 2), 0) + 4 * E * np.abs(L) + 8 * E
        dp, Dv = dO @ V.swapaxes(1, 2), (dO * O).sum(-1, keepdims=True)
        A = (np.abs(dO) * np.abs(O)).sum(-1, keepdims=True)
        off = (D + 4) * E * (np.abs(dO) @ np.abs(V).swapaxes(1, 2) + A) + u * A
        S = scale * p * np.abs(dp - Dv)
        eS = scale * p * ((u + ds + 4 * E) * np.abs(dp - Dv) + off)
        nq, nk = (e - c + 8) * E, ((b - a) * G + 8) * E
        hand = scale * np.where(see, p * 2.0 ** -11 + 2.0 ** -37, 0) * np.abs(dp - Dv) if u > E else 0
        shared = lambda x: np.swapaxes(x.reshape(Hk, G, *x.shape[1:]).sum(1), 0, 1)  # noqa: E731
        tq[a:b] = np.swapaxes((eS + nq * S) @ np.abs(K), 0, 1)
        tk[c:e] = shared((eS + hand + nk * S).swapaxes(1, 2) @ np.abs(Q))
        tv[c:e] = shared((p * (u + ds + nk)).swapaxes(1, 2) @ np.abs(dO))
    return tq, tk, tv


def _check_bwd(d, dt, scale=None):
    scale = 1 / math.sqrt(d["q"].shape[-1]) if scale is None else scale
    x = _on(d)
    o, lse = gdn.attn_fwd(x["q"], x["k"], x["v"], x["cu_q"], x["cu_k"], scale=scale)
    B, Tq, Tk, Hq, Hk, D = len(d["cu_q"]) - 1, d["q"].shape[0], d["k"].shape[0], *d["q"].shape[1:2], *d["k"].shape[1:]
    # gradients into slices of one tensor each, with another column behind
    g = {n: torch.full((T, H + 1, D), 5.0, dtype=DT[dt], device=DEV) for n, T, H in (("dq", Tq, Hq), ("dk", Tk, Hk), ("dv", Tk, Hk))}
    ws = torch.full((gdn.gdn_attn_bwd_workspace_size(B, Tq, Tk, Hq, Hk, D, DT[dt]),), 255, dtype=torch.uint8, device=DEV)
    gdn.gdn_attn_bwd(x["q"], x["k"], x["v"], x["cu_q"], x["cu_k"], o, lse, x["d_o"], g["dq"][:, :Hq], g["dk"][:, :Hk], g["dv"][:, :Hk],
                     ws, scale)
    torch.cuda.synchronize()
    want = ref.backward(d["q"], d["k"], d["v"], o, lse, d["d_o"], d["cu_q"], d["cu_k"], scale)
    for (n, got), w, t in zip(g.items(), want, _bwd_tol(d, o, lse, scale, U[dt])):
        assert (got[:, -1] == 5).all()
        _close(n, got[:, :-1], w, t + U[dt] * np.abs(w) + 1e-37)
        assert (got[:, :-1][torch.from_numpy(np.isnan(w[:, 0, 0]))] == 5).all()
    # the convenience: the same values
    h = gdn.attn_bwd(x["q"], x["k"], x["v"], o, lse, x["d_o"], x["cu_q"], x["cu_k"], scale=scale)
    for (n, got), w in zip(g.items(), want):
        live = torch.from_numpy(~np.isnan(w[:, 0, 0]))
        assert torch.equal(got[:, :-1][live], h[n][live]), n
    return h


BATCHES = [
    ([1], None, 1, 1), ([3, 1], None, 3, 3), ([63], None, 4, 2), ([64, 0, 65], None, 8, 1), ([130, 1, 77], None, 6, 2),
    ([0], None, 2, 1), ([5, 0, 0, 9, 1, 1], None, 5, 1), ([200, 31], None, 7, 1), ([40], None, 64, 1), ([33, 2], None, 48, 1),
    # other numbers of keys than of rows: more, fewer (rows that see nothing), none
    ([1, 17], [300, 500], 5, 5), ([20, 7, 4], [9, 7, 0], 4, 2), ([129, 64], [257, 40], 4, 1), ([0, 3], [8, 130], 2, 2),
    ([70, 200], [3, 90], 8, 2)]


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lq,lk,Hq,Hk", BATCHES)
def test_forward_and_backward(lq, lk, Hq, Hk, D, dt):
    _say(f"lq {lq} lk {lk} Hq{Hq} Hk{Hk} D{D} {dt}")
    d = _packed(lq, lk, Hq, Hk, D, dt, seed=sum(lq) + D, before=2, behind=3)
    _check_fwd(d, dt)
    _check_bwd(d, dt)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("lq,lk,Hq,Hk", [
    ([1100], None, 3, 1), ([5], [3001], 8, 2), ([700, 0, 90, 1, 401], None, 4, 2), ([600, 100], [1700, 1100], 4, 4), ([900], None, 14, 2),
    ([513, 513], [200, 1025], 2, 2)])
def test_longer(lq, lk, Hq, Hk, dt):
    """Few workgroups and long walks: keys and rows are cut, in forms that the sizes choose."""
    _say(f"longer lq {lq} lk {lk} Hq{Hq} Hk{Hk} {dt}")
    d = _packed(lq, lk, Hq, Hk, 128, dt, seed=13)
    _check_fwd(d, dt)
    _check_bwd(d, dt)


@pytest.mark.parametrize("lq,lk,Hq,Hk,D,dt", [
    ([2500, 0, 300, 1, 64], None, 4, 2, 128, "bf16"), ([200, 7], [2900, 3000], 16, 2, 64, "bf16"), ([1500, 900], None, 8, 4, 64, "fp32"),
    ([4000], [700], 4, 2, 64, "bf16"), ([33] * 100, None, 3, 1, 64, "bf16"), ([2049], None, 12, 12, 64, "bf16"),
    ([3] * 70 + [2700] + [1] * 70, None, 4, 1, 64, "bf16")])
def test_forward_in_shares(lq, lk, Hq, Hk, D, dt):
    """Sizes with which workgroups share the keys of all row tiles, or just do not."""
    _say(f"shares lq {lq[:6]} lk {lk} Hq{Hq} Hk{Hk} D{D} {dt}")
    d = _packed(lq, lk, Hq, Hk, D, dt, seed=29)
    o, lse = _check_fwd(d, dt)
    x = _on(d)
    o2, lse2 = gdn.attn_fwd(x["q"], x["k"], x["v"], x["cu_q"], x["cu_k"])
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_large_scores(dt):
    """Scores of some hundreds: one key takes nearly all of a row, and the running maximum
    rises often."""
    d = _packed([200], None, 4, 2, 64, dt, seed=5)
    ramp = torch.linspace(0.2, 3.0, 200)[:, None, None]
    d["k"] = (d["k"].float() * ramp).to(DT[dt])
    _check_fwd(d, dt, scale=2.0)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_other_sequences_are_not_touched(dt):
    """NaN and infinities in rows of no sequence, and in another sequence, change nothing."""
    d = _packed([37, 64, 50], None, 4, 2, 64, dt, seed=7, before=9, behind=30)
    x = _on(d)
    o, lse = gdn.attn_fwd(x["q"], x["k"], x["v"], x["cu_q"])
    g = gdn.attn_bwd(x["q"], x["k"], x["v"], o, lse, x["d_o"], x["cu_q"])
    bad = {n: x[n].clone() for n in ("q", "k", "v", "d_o")}
    for t in bad.values():
        t[:9], t[46:110], t[160:] = float("nan"), float("inf"), float("nan")
    o2, lse2 = gdn.attn_fwd(bad["q"], bad["k"], bad["v"], x["cu_q"])
    g2 = gdn.attn_bwd(bad["q"], bad["k"], bad["v"], o2, lse2, bad["d_o"], x["cu_q"])
    for rows in (slice(9, 46), slice(110, 160)):
        assert torch.equal(o[rows], o2[rows]) and torch.equal(lse[rows], lse2[rows])
        for n in g:
            assert torch.equal(g[n][rows], g2[n][rows]), n


def test_a_live_nan_shows():
    d = _packed([90], None, 2, 1, 64, "bf16", seed=8)
    d["k"][40] = float("nan")
    x = _on(d)
    o, lse = gdn.attn_fwd(x["q"], x["k"], x["v"], x["cu_q"])
    assert torch.isfinite(o[:40]).all() and torch.isnan(o[40:]).all() and torch.isnan(lse[40:]).all()


def test_offsets_out_of_range_stay_inside():
    """Offsets that fall, or lie outside, give no row outside the outputs: what is behind
    and before them stays as it was."""
    d = _on(_packed([100], None, 4, 2, 64, "bf16", seed=9))
    cu = torch.tensor([-5, 70, 30, 1000, 100], dtype=torch.int32, device=DEV)
    room = torch.full((3, 100, 4, 64), 5.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full((3, 100, 4), 5.0, device=DEV)
    q, k, v = (d[n].contiguous() for n in "qkv")
    ws = torch.empty(1 << 24, dtype=torch.uint8, device=DEV)
    gdn.gdn_attn_fwd(q, k, v, cu, None, room[1], lse[1], ws, 0.1)
    kv = torch.full((2, 3, 100, 2, 64), 5.0, dtype=torch.bfloat16, device=DEV)
    dq = torch.full((3, 100, 4, 64), 5.0, dtype=torch.bfloat16, device=DEV)
    gdn.gdn_attn_bwd(q, k, v, cu, None, room[1], lse[1], d["d_o"].contiguous(), dq[1], kv[0, 1], kv[1, 1], ws, 0.1)
    torch.cuda.synchronize()
    for t in (room[0], room[2], lse[0], lse[2], dq[0], dq[2], kv[:, 0], kv[:, 2]):
        assert (t == 5).all()


# --- the cache ------------------------------------------------------------------

def _cache(N, width, page, Hk, D, seed=0, extra=3):
    """A cache of random bytes (NaN among them), random scales, and a table."""
    g = torch.Generator().manual_seed(seed)
    pages = N * width + extra
    byte = lambda *s: torch.randint(0, 256, s, generator=g, dtype=torch.uint8)  # noqa: E731
    exp = lambda: torch.exp2(torch.randint(-9, -2, (pages, Hk, page // 16), generator=g).float())  # noqa: E731
    return dict(k_cache=byte(pages, Hk, page, D), v_cache=byte(pages, Hk, page // 16, D, 16), k_scale=exp(), v_scale=exp(),
                table=torch.randperm(pages, generator=g)[:N * width].reshape(N, width).to(torch.int32))


def _live(c):
    """No NaN among the bytes."""
    for n in ("k_cache", "v_cache"):
        c[n][(c[n] & 127) == 127] = 0x35
    return c


def _values(c):
    return [ref.VALUES[c["k_cache"].numpy()], ref.VALUES[c["v_cache"].numpy()], c["k_scale"].double().numpy(), c["v_scale"].double().numpy()]


def _append_args(c):
    return c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"], c["table"]


APPENDS = [  # lens with the new tokens, new tokens
    ([1], None), ([17, 16, 1, 33, 300], None), ([5, 40, 100], [5, 33, 1]), ([300, 0, 16, 31, 64], [300, 0, 16, 15, 48]),
    ([200, 37], [37, 20]), ([3], [0])]


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("Hk,D,page", [(1, 64, 16), (3, 128, 48), (2, 128, 256), (5, 64, 32)])
@pytest.mark.parametrize("lens,new", APPENDS)
def test_append(lens, new, Hk, D, page, dt):
    """Bit for bit: scales, stored values, and every other slot as it was."""
    _say(f"append lens {lens} new {new} Hk{Hk} D{D} page {page} {dt}")
    N, width = len(lens), -(-max(lens) // page)
    c = _live(_cache(N, width, page, Hk, D, seed=sum(lens)))
    news = new or [1] * N
    g = torch.Generator().manual_seed(7)
    kv = torch.randn(sum(news), 2 * Hk, D, generator=g)
    kv = (kv * torch.exp2(torch.randint(-12, 6, (sum(news), 2 * Hk, 1), generator=g))).to(DT[dt])
    x, before = _dev(c), {k: v.clone() for k, v in c.items()}
    n = torch.tensor(lens, dtype=torch.int32)
    cu = _cu(new) if new else None
    kvd = kv.to(DEV)
    for _ in range(2):   # a second time changes nothing
        gdn.attn_append_(kvd[:, :Hk], kvd[:, Hk:], *_append_args(x), n.to(DEV), cu=None if cu is None else cu.to(DEV))
        torch.cuda.synchronize()
    want = _values(before)
    ref.append(kv[:, :Hk], kv[:, Hk:], cu, *want, before["table"], n)
    got = _values({k: v.cpu() for k, v in x.items()})
    for name, a, b in zip(("k_cache", "v_cache", "k_scale", "v_scale"), got, want):
        assert np.array_equal(a, b), (name, np.argwhere(a != b)[:5])


def test_append_of_special_values():
    """Zeros, values that are not finite, the largest and the smallest, and a scale that
    grows over stored values down to e4m3's subnormals."""
    Hk, D = 1, 64
    c = _cache(4, 1, 16, Hk, D)
    c["k_cache"][:], c["v_cache"][:] = 0, 0
    x = _dev(c)
    rows = torch.zeros(4, 3, Hk, D)
    rows[0, 1] = torch.tensor([float("inf"), float("-inf"), float("nan"), 1.0] * 16)
    rows[1, 0] = torch.finfo(torch.float32).max
    rows[1, 1] = -torch.finfo(torch.float32).tiny
    rows[2, 0] = torch.logspace(-40, 0, 64, base=2.0)
    rows[2, 2] = 2.0 ** 9 * 1.75
    rows[3] = 1e-45
    for t in range(3):
        r = rows[:, t].to(DEV)
        gdn.attn_append_(r, -r, *_append_args(x), torch.full((4,), t + 1, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    want = _values(c)
    for t in range(3):
        ref.append(rows[:, t], -rows[:, t], None, *want, c["table"], torch.full((4,), t + 1))
    got = _values({k: v.cpu() for k, v in x.items()})
    for name, a, b in zip(("k_cache", "v_cache", "k_scale", "v_scale"), got, want):
        assert np.array_equal(a, b, equal_nan=True), (name, np.argwhere(a != b)[:5])
    p = int(c["table"][2, 0])
    assert got[2][p, 0, 0] == 2.0 and got[0][p, 0, 2, 0] == 448


def test_append_where_there_is_no_room():
    """Pages outside the cache, positions behind the table, and before the first: not stored."""
    c = _live(_cache(4, 2, 16, 2, 64, seed=4))
    c["table"][1, 0], c["table"][2, 1] = -1, 10 ** 6
    lens, cu = torch.tensor([40, 20, 20, 3], dtype=torch.int32), _cu([12, 20, 20, 9])
    g = torch.Generator().manual_seed(1)
    k, v = torch.randn(61, 2, 64, generator=g), torch.randn(61, 2, 64, generator=g)
    x = _dev(c)
    gdn.attn_append_(k.to(DEV), v.to(DEV), *_append_args(x), lens.to(DEV), cu=cu.to(DEV))
    torch.cuda.synchronize()
    want = _values(c)
    ref.append(k, v, cu, *want, c["table"], lens)
    got = _values({k: v.cpu() for k, v in x.items()})
    for a, b in zip(got, want):
        assert np.array_equal(a, b)


def _check_step(c, q, lens, dt, scale=None, want_lse=True):
    scale = 1 / math.sqrt(q.shape[-1]) if scale is None else scale
    x = _dev(c)
    n = torch.tensor(lens, dtype=torch.int32)
    o, lse = gdn.attn_step(q.to(DEV), *_append_args(x), n.to(DEV), scale=scale, want_lse=True)
    torch.cuda.synchronize()
    vals = _values(c)
    with np.errstate(invalid="ignore"):
        ro, rl = ref.step(q, *vals, c["table"], n, scale)
        A, _ = ref.step(q, *vals, c["table"], n, scale, weigh_abs=True)
    ds, L = np.zeros(ro.shape[:2]), np.zeros((len(lens), 1))
    G = q.shape[1] // vals[0].shape[1]
    D, u = q.shape[2], U[dt]
    for i in range(len(lens)):
        k, _, there = ref.cached(*vals, c["table"], n[i], i)
        L[i] = there.sum()
        for h in range(q.shape[1]):   # three products for one in fp32, with a residue of 2^-24
            ds[i, h] = (3 * D + 8) * E * scale * (np.abs(ref.f64(q[i, h])) @ np.abs(k[h // G]).T * there).max(initial=0)
    tol = (u + 2 * ds + (3 * L + 8) * E)[..., None] * A + u * np.abs(ro) + 1e-37
    _close("o", o, ro, tol)
    _close("lse", lse, rl, ds + (L + 16) * E + 4 * E * np.abs(np.where(np.isfinite(rl), rl, 0)) + 1e-37)
    return o, lse


def _blank(c, lens, page):
    """NaN bytes and NaN scales wherever no token of a sequence stands; none among the live."""
    live_k, live_v = torch.zeros(c["k_cache"].shape[0], page, dtype=torch.bool), None
    for i, n in enumerate(lens):
        for t in range(min(max(n, 0), c["table"].shape[1] * page)):
            live_k[c["table"][i, t // page], t % page] = True
    live_v = live_k.reshape(live_k.shape[0], -1, 16)
    _live(c)
    c["k_cache"][~live_k[:, None, :, None].expand_as(c["k_cache"])] = 0x7f
    c["v_cache"][~live_v[:, None, :, None].expand_as(c["v_cache"])] = 0xff
    for s in ("k_scale", "v_scale"):
        c[s][~live_v.any(-1)[:, None].expand_as(c[s])] = float("nan")
    return c


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("lens,Hq,Hk,D,page", [
    ([1], 1, 1, 64, 16), ([0, 5], 4, 2, 128, 16), ([300], 32, 8, 128, 64), ([17, 64, 65, 128, 1], 12, 3, 64, 48),
    ([1000, 30], 40, 1, 128, 16), ([1025, 0, 900], 64, 1, 64, 32), ([3000, 10, 700], 7, 1, 128, 256), ([2047], 6, 6, 64, 16),
    ([40] * 90, 2, 1, 64, 16), ([1300, 5] * 40, 4, 2, 64, 16)])
def test_step(lens, Hq, Hk, D, page, dt):
    _say(f"step lens {lens[:6]} Hq{Hq} Hk{Hk} D{D} page {page} {dt}")
    N = len(lens)
    c = _blank(_cache(N, -(-max(lens) // page) + 1, page, Hk, D, seed=N), lens, page)
    g = torch.Generator().manual_seed(3)
    q = (torch.randn(N, Hq, D, generator=g) * 0.2).to(DT[dt])
    _check_step(c, q, lens, dt)


@pytest.mark.parametrize("width", [3, 200])
def test_step_with_pages_that_are_none(width):
    """Entries outside the cache hold no tokens, whole sequences of them among these; what the
    entries behind a sequence say does not matter.  Both forms: with and without pieces."""
    c = _live(_cache(4, width, 16, 2, 64, seed=5))
    lens = [33, 48, 16, 40]
    c["table"][0, 1], c["table"][1], c["table"][3, 0] = -7, 2 ** 31 - 1, len(c["k_cache"])
    c["table"][2, 1:], c["table"][0, 3:] = -2 ** 31, 2 ** 30
    g = torch.Generator().manual_seed(3)
    q = torch.randn(4, 6, 64, generator=g) * 0.2
    o, lse = _check_step(c, q, lens, "fp32")
    assert (o[1] == 0).all() and torch.isneginf(lse[1]).all()


def test_step_lengths_are_clamped():
    c = _live(_cache(2, 2, 16, 1, 64, seed=6))
    q = (torch.randn(2, 2, 64, generator=torch.Generator().manual_seed(3)) * 0.2).to(torch.bfloat16)
    x = _dev(c)
    run = lambda n: gdn.attn_step(q.to(DEV), *_append_args(x), torch.tensor(n, dtype=torch.int32, device=DEV))  # noqa: E731
    assert torch.equal(run([2 ** 31 - 1, -5]), run([32, 0]))


def test_step_of_large_scores():
    c = _live(_cache(2, 40, 16, 2, 64, seed=8))
    q = torch.randn(2, 8, 64, generator=torch.Generator().manual_seed(3))
    _check_step(c, q, [640, 333], "fp32", scale=1.0)


# --- together -------------------------------------------------------------------

def test_prompt_then_tokens():
    """A layer as a model runs it: prompts through the prologue, the forward and the append,
    then single tokens through the prologue, the append and the step, against attention over
    the cache's values in 64 bits."""
    Hq, Hk, D, R, page, eps = 8, 2, 64, 32, 32, 1e-6
    prompts, more = [70, 5, 33], 20
    N, width = 3, 4
    g = torch.Generator(device=DEV).manual_seed(11)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV, dtype=torch.bfloat16)  # noqa: E731
    w_q, w_k = 1 + r(D).float() / 4, 1 + r(D).float() / 4
    inv = (10000.0 ** (-torch.arange(0, R, 2) / R)).to(DEV)
    table = torch.randperm(N * width, generator=g, device=DEV).reshape(N, width).to(torch.int32)
    cache = [torch.zeros(N * width, Hk, page, D, dtype=torch.float8_e4m3fn, device=DEV),
             torch.zeros(N * width, Hk, page // 16, D, 16, dtype=torch.float8_e4m3fn, device=DEV),
             torch.zeros(N * width, Hk, page // 16, device=DEV), torch.zeros(N * width, Hk, page // 16, device=DEV)]
    cu = _cu(prompts).to(DEV)
    lens = torch.tensor(prompts, dtype=torch.int32, device=DEV)
    fused = r(sum(prompts), Hq + 2 * Hk, D)
    pos = torch.cat([torch.arange(n) for n in prompts]).to(torch.int32).to(DEV)
    q, k = gdn.attn_prologue(fused[:, :Hq], fused[:, Hq:Hq + Hk], w_q, w_k, inv, pos, eps=eps)
    v = fused[:, Hq + Hk:]
    o, _ = gdn.attn_fwd(q, k, v, cu)
    gdn.attn_append_(k, v, *cache, table, lens, cu=cu)
    ro, _ = ref.forward(q.cpu(), k.cpu(), v.cpu(), cu.cpu(), None, D ** -0.5)
    assert np.abs(o.double().cpu().numpy() - ro).max() < 0.02 * np.abs(ro).max()
    kept = [[k[a:b], v[a:b]] for a, b in zip(cu.tolist(), cu.tolist()[1:])]
    for t in range(more):
        fused = r(N, Hq + 2 * Hk, D) * (1 + t)   # values grow: scales of shared blocks do too
        q, k = gdn.attn_prologue(fused[:, :Hq], fused[:, Hq:Hq + Hk], w_q, w_k, inv, lens, eps=eps)
        lens += 1
        v = fused[:, Hq + Hk:]
        gdn.attn_append_(k, v, *cache, table, lens)
        o = gdn.attn_step(q, *cache, table, lens)
        for i in range(N):
            kept[i] = [torch.cat((kept[i][0], k[i:i + 1])), torch.cat((kept[i][1], v[i:i + 1]))]
        vals = [ref.VALUES[cache[0].view(torch.uint8).cpu().numpy()], ref.VALUES[cache[1].view(torch.uint8).cpu().numpy()],
                cache[2].double().cpu().numpy(), cache[3].double().cpu().numpy()]
        ro, _ = ref.step(q.cpu(), *vals, table.cpu(), lens.cpu(), D ** -0.5)
        A, _ = ref.step(q.cpu(), *vals, table.cpu(), lens.cpu(), D ** -0.5, weigh_abs=True)
        assert (np.abs(o.double().cpu().numpy() - ro) <= 2.0 ** -8 * (np.abs(ro) + 1.1 * A) + 1e-6).all()
        for i in range(N):   # a value is off by half a step of e4m3, or of its subnormals at the block's scale
            ck, cv, _ = ref.cached(*vals, table.cpu(), lens[i], i)
            for held, x, sc in ((ck, kept[i][0], vals[2]), (cv, kept[i][1], vals[3])):
                x = np.swapaxes(ref.f64(x), 0, 1)
                top = max(s for s in sc[ref.ints(table[i])].ravel())
                # each time the scale of a block grows, a subnormal may be rounded again
                assert (np.abs(held - x) <= 2.0 ** -4 * np.abs(x) + 6 * 2.0 ** -10 * top).all()


def test_gradients_of_the_layer():
    """Prologue and attention forward and backward in a chain, against differences of the loss
    in 64 bits along a random direction of every input."""
    Hq, Hk, D, R = 4, 2, 64, 64
    d = _raw(45, Hq, Hk, D, R, "fp32", seed=17)
    cu = _cu([30, 0, 15])
    x = _dev(d)
    (qr, kr), v = _split(x, Hq, Hk), x["fused"][:, Hq + Hk:]
    args = (qr, kr, x["w_q"], x["w_k"], x["inv_freq"], x["pos"])
    q, k = gdn.attn_prologue(*args)
    cud = cu.to(DEV)
    o, lse = gdn.attn_fwd(q, k, v, cud)
    g = gdn.attn_bwd(q, k, v, o, lse, x["d_q"], cud)
    gp = gdn.attn_prologue_bwd(*args, g["dq"], g["dk"])
    grads = dict(fused=torch.cat((gp["dq_raw"], gp["dk_raw"], g["dv"]), 1), w_q=gp["dw_q"], w_k=gp["dw_k"])

    def loss(fused, w_q, w_k):
        q = ref.prologue(fused[:, :Hq], w_q, d["inv_freq"], d["pos"], 1e-6)
        k = ref.prologue(fused[:, Hq:Hq + Hk], w_k, d["inv_freq"], d["pos"], 1e-6)
        return (ref.forward(q, k, fused[:, Hq + Hk:], cu, None, D ** -0.5)[0] * ref.f64(d["d_q"])).sum()

    at = {n: ref.f64(d[n]) for n in grads}
    rng = np.random.default_rng(0)
    for n in grads:
        way = rng.standard_normal(at[n].shape)
        h = 1e-5
        up, down = loss(**{**at, n: at[n] + h * way}), loss(**{**at, n: at[n] - h * way})
        want, got = (up - down) / (2 * h), float((ref.f64(grads[n]) * way).sum())
        size = float((np.abs(ref.f64(grads[n])) * np.abs(way)).sum())
        assert abs(got - want) <= 1e-5 * size, (n, got, want)


@pytest.mark.parametrize("long", [False, True])
def test_captured_with_lengths_that_change(long):
    """Forward, backward, append and step in a graph; offsets, lengths and tables change between
    replays, with eager calls and synchronisations in between."""
    Hq, Hk, D, page = (4, 1, 128, 16) if long else (4, 2, 64, 32)
    T, width = (1800, 130) if long else (90, 3)
    d = _on(_packed([T], None, Hq, Hk, D, "bf16", seed=31))
    q, k, v, d_o = (d[n].contiguous() for n in ("q", "k", "v", "d_o"))
    cu, lens = torch.zeros(4, dtype=torch.int32, device=DEV), torch.zeros(3, dtype=torch.int32, device=DEV)
    c = _dev(_live(_cache(3, width, page, Hk, D)))
    qs = q[:3].clone()

    def work():
        o, lse = gdn.attn_fwd(q, k, v, cu)
        g = gdn.attn_bwd(q, k, v, o, lse, d_o, cu)
        gdn.attn_append_(k, v, *_append_args(c), lens, cu=cu)
        return [o, lse, *g.values(), gdn.attn_step(qs, *_append_args(c), lens)]

    def fill(splits):
        cu.copy_(torch.tensor([0, *splits, T], dtype=torch.int32))
        lens.copy_(cu[1:] - cu[:-1])

    fill([10, 50])
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for splits in ([10, 50], [0, T], [T // 2, T // 2 + 1], [1, 2], [10, 50]):
        fill(splits)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out] + [t.clone() for t in _append_args(c)]
        want = work() + list(_append_args(c))
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), (splits, i)


def test_on_another_stream():
    d = _on(_packed([60, 9], None, 4, 2, 64, "bf16", seed=37))
    o, lse = gdn.attn_fwd(d["q"], d["k"], d["v"], d["cu_q"])
    g = gdn.attn_bwd(d["q"], d["k"], d["v"], o, lse, d["d_o"], d["cu_q"])
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    o2, lse2 = gdn.attn_fwd(d["q"], d["k"], d["v"], d["cu_q"], stream=s)
    g2 = gdn.attn_bwd(d["q"], d["k"], d["v"], o2, lse2, d["d_o"], d["cu_q"], stream=s)
    s.synchronize()
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and all(torch.equal(g[n], g2[n]) for n in g)
