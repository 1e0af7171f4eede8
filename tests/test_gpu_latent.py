"""GPU parity of the latent-attention entry points against the fp64 oracle.

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
from oracle import latent as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
E = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
U = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}


def _say(*a):
    print("[latent]", *a, flush=True)


def _close(name, x, want, tol):
    x = x.detach().double().cpu().numpy()
    assert x.shape == want.shape, (name, x.shape, want.shape)
    both = np.isneginf(x) & np.isneginf(want)
    assert np.isfinite(x[~both]).all(), f"{name}: not finite"
    d = np.where(both, 0.0, np.abs(np.where(both, 0, x) - np.where(both, 0, want)))
    over = d - tol
    i = np.unravel_index(np.argmax(over), over.shape) if d.size else None
    assert not d.size or over[i] <= 0, f"{name}: off by {d[i]:.3e} at {i}, allowed {np.broadcast_to(tol, d.shape)[i]:.3e}"
    if d.size:
        _say(f"{name}: largest share of the tolerance {float(np.max(d / np.maximum(tol, 1e-300))):.2f}")


def _expanded(B, Tq, Tk, H, dn, dv, dt, seed=0, lens=None):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).to(DT[dt])  # noqa: E731
    d = dict(q=r(B, Tq, H, dn + 64), kv=r(B, Tk, H, dn + dv), k_rope=r(B, Tk, 64), d_o=r(B, Tq, H, dv))
    d["lens"] = None if lens is None else torch.tensor(lens, dtype=torch.int32)
    return d


def _dev(d):
    return {k: None if v is None else v.to(DEV) for k, v in d.items()}


def _fwd_tol(d, scale, u):
    Q, K, V = ref.heads(d["q"], d["kv"], d["k_rope"])
    B, H, Tq, D = Q.shape
    see = ref.visible(B, Tq, K.shape[2], d["lens"])
    live = see.any(2)[..., None]
    K, V = np.where(live, K, 0), np.where(live, V, 0)
    p, _ = ref.softmax_rows(Q @ K.swapaxes(2, 3) * scale, see)
    ds = (D + 4) * E * scale * np.where(see, np.abs(Q) @ np.abs(K).swapaxes(2, 3), 0).max(-1, keepdims=True, initial=0)
    A = p @ np.abs(V)
    L = see.sum(-1, keepdims=True)
    return ((u + 2 * ds + (L + 8) * E) * A).swapaxes(1, 2), ((ds + (L + 16) * E)[..., 0]).swapaxes(1, 2)


def _check_fwd(d, dt, scale=None):
    scale = 1 / math.sqrt(d["q"].shape[-1]) if scale is None else scale
    x = _dev(d)
    o, lse = gdn.latent_fwd(x["q"], x["kv"], x["k_rope"], lens=x["lens"], scale=scale)
    torch.cuda.synchronize()
    ro, rl = ref.forward(d["q"], d["kv"], d["k_rope"], d["lens"], scale)
    to, tl = _fwd_tol(d, scale, U[dt])
    _close("o", o, ro, to + U[dt] * np.abs(ro) + 1e-37)
    _close("lse", lse, rl, tl + 4 * E * np.abs(np.where(np.isfinite(rl), rl, 0)) + 1e-37)
    return o, lse


DIMS = [(128, 128), (64, 64), (128, 64), (64, 128)]


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("dn,dv", DIMS)
@pytest.mark.parametrize("B,Tq,Tk,H,lens", [
    (1, 1, 1, 1, None), (2, 3, 3, 3, [1, 3]), (1, 63, 63, 2, None), (2, 64, 64, 1, [64, 0]), (1, 65, 129, 3, None),
    (3, 130, 130, 2, [130, 77, 64]), (1, 1, 300, 5, None), (2, 17, 500, 2, [500, 490]), (1, 300, 300, 8, [257])])
def test_forward(B, Tq, Tk, H, dn, dv, dt, lens):
    _say(f"fwd B{B} Tq{Tq} Tk{Tk} H{H} dn{dn} dv{dv} {dt} lens {lens}")
    _check_fwd(_expanded(B, Tq, Tk, H, dn, dv, dt, lens=lens), dt)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("B,Tq,Tk,H", [(1, 1100, 1100, 3), (1, 5, 3001, 2), (1, 200, 2500, 4), (2, 129, 1030, 16)])
def test_forward_longer(B, Tq, Tk, H, dt):
    _say(f"fwd long B{B} Tq{Tq} Tk{Tk} H{H} {dt}")
    _check_fwd(_expanded(B, Tq, Tk, H, 128, 128, dt, seed=3), dt)


@pytest.mark.parametrize("B,Tq,Tk,H,dn,dv,dt,lens", [
    (1, 2048, 2048, 10, 128, 128, "bf16", [2011]), (4, 1000, 3000, 2, 64, 128, "bf16", [3000, 0, 2100, 2999]),
    (3, 1000, 1000, 8, 64, 64, "fp32", [1000, 1, 640]), (2, 600, 1700, 4, 128, 128, "fp32", [1100, 1700]),
    (100, 64, 1400, 2, 128, 64, "bf16", [(37 * i) % 1500 for i in range(100)])])
def test_forward_in_shares(B, Tq, Tk, H, dn, dv, dt, lens):
    """Grids small enough, and rows long enough, for workgroups that share all key tiles:
    some or all sequences padded, empty ones between."""
    _say(f"fwd shares B{B} Tq{Tq} Tk{Tk} H{H} dn{dn} dv{dv} {dt}")
    d = _expanded(B, Tq, Tk, H, dn, dv, dt, lens=lens, seed=29)
    o, lse = _check_fwd(d, dt)
    x = _dev(d)
    o2, lse2 = gdn.latent_fwd(x["q"], x["kv"], x["k_rope"], lens=x["lens"])
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_forward_large_scores(dt):
    """Scores of some hundreds: one key takes nearly all of a row, and the running
    maximum rises often."""
    d = _expanded(1, 200, 200, 2, 64, 64, dt, seed=5)
    ramp = torch.linspace(0.2, 3.0, 200)[None, :, None, None]
    d["kv"] = (d["kv"].float() * ramp).to(DT[dt])
    _check_fwd(d, dt, scale=2.0)


def test_forward_all_scores_equal():
    d = _expanded(1, 150, 150, 2, 64, 64, "bf16", seed=6)
    d["q"].zero_()
    _check_fwd(d, "bf16")


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_what_lies_behind_a_sequence_is_not_touched(dt):
    """NaN and infinities behind the live lengths, in every input and gradient."""
    d = _expanded(2, 100, 100, 2, 64, 128, dt, lens=[37, 64], seed=7)
    for b, n in enumerate([37, 64]):
        for k in ("q", "kv", "k_rope", "d_o"):
            d[k][b, n:] = float("nan") if b else float("inf")
    o, lse = _check_fwd(d, dt)
    x = _dev(d)
    g = gdn.latent_bwd(x["q"], x["kv"], x["k_rope"], o, lse, x["d_o"], lens=x["lens"])
    clean = {k: (torch.where(torch.isfinite(v), v, torch.zeros_like(v)) if v.is_floating_point() else v) for k, v in x.items()}
    o2, lse2 = gdn.latent_fwd(clean["q"], clean["kv"], clean["k_rope"], lens=x["lens"])
    g2 = gdn.latent_bwd(clean["q"], clean["kv"], clean["k_rope"], o2, lse2, clean["d_o"], lens=x["lens"])
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    for k in g:
        assert torch.equal(g[k], g2[k]), k
        for b, n in enumerate([37, 64]):
            assert (g[k][b, n:] == 0).all(), k


def _bwd_tol(d, o, lse, scale, u):
    """Tolerances of dq, dkv, dk_rope: the terms' absolute values times what each may
    be off.  P: 2 ds + 8 e (and the rounding u in dv; for bf16 in dk half a step of fp16,
    2^-11, of 4096 P, or of its subnormals, 2^-25 / 4096); dP - D: (DV + 2) e sums of
    absolute products, and in D u |do| |o|, by which do . o of the rounded o may be off
    the sum of P dP, which the kernel takes for the first rows; dS: u."""
    Q, K, V = ref.heads(d["q"], d["kv"], d["k_rope"])
    B, H, Tq, D = Q.shape
    Tk = K.shape[2]
    see = ref.visible(B, Tq, Tk, d["lens"])
    live = see.any(2)[..., None]
    K, V = np.where(live, K, 0), np.where(live, V, 0)
    rows = see.any(3)[..., None]
    Q = np.where(rows, Q, 0)
    t = lambda x: np.where(rows, np.swapaxes(ref.f64(x), 1, 2), 0)  # noqa: E731
    O, dO, L = t(o), t(d["d_o"]), t(lse[..., None])
    p = np.where(see, np.exp(np.where(see, Q @ K.swapaxes(2, 3) * scale - L, 0)), 0)
    ds = (D + 4) * E * scale * np.where(see, np.abs(Q) @ np.abs(K).swapaxes(2, 3), 0) + 4 * E * np.abs(L) + 8 * E
    dp, Dv = dO @ V.swapaxes(2, 3), (dO * O).sum(-1, keepdims=True)
    off = (V.shape[-1] + 4) * E * (np.abs(dO) @ np.abs(V).swapaxes(2, 3) + (np.abs(dO) * np.abs(O)).sum(-1, keepdims=True))
    off = off + u * (np.abs(dO) * np.abs(O)).sum(-1, keepdims=True)
    eS = scale * p * ((u + ds + 4 * E) * np.abs(dp - Dv) + off)   # error of dS
    S = scale * p * np.abs(dp - Dv)
    nq, nk = (Tk + 8) * E, (Tq * 1 + 8) * E
    dq = (eS + nq * S) @ np.abs(K)
    hand = scale * np.where(see, p * 2.0 ** -11 + 2.0 ** -37, 0) * np.abs(dp - Dv) if u > E else 0
    dk = (eS + hand + nk * S).swapaxes(2, 3) @ np.abs(Q)
    dv = (p * (u + ds + nk)).swapaxes(2, 3) @ np.abs(dO)
    dn = D - 64
    rope = (dk[..., dn:] + H * E * (S.swapaxes(2, 3) @ np.abs(Q))[..., dn:]).sum(1)
    return dq.swapaxes(1, 2), np.concatenate([dk[..., :dn], dv], -1).swapaxes(1, 2), rope


def _check_bwd(d, dt):
    scale = 1 / math.sqrt(d["q"].shape[-1])
    x = _dev(d)
    o, lse = gdn.latent_fwd(x["q"], x["kv"], x["k_rope"], lens=x["lens"])
    g = gdn.latent_bwd(x["q"], x["kv"], x["k_rope"], o, lse, x["d_o"], lens=x["lens"])
    torch.cuda.synchronize()
    want = ref.backward(d["q"], d["kv"], d["k_rope"], d["lens"], o, lse, d["d_o"], scale)
    tol = _bwd_tol(d, o, lse, scale, U[dt])
    for name, w, t in zip(("dq", "dkv", "dk_rope"), want, tol):
        _close(name, g[name], w, t + U[dt] * np.abs(w) + 1e-37)
    return g


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("dn,dv", DIMS)
@pytest.mark.parametrize("B,Tq,Tk,H,lens", [
    (1, 1, 1, 1, None), (2, 3, 3, 3, [1, 3]), (1, 65, 65, 2, None), (2, 64, 128, 1, [128, 100]), (1, 40, 129, 3, None),
    (3, 130, 130, 2, [130, 77, 0]), (1, 1, 300, 5, None), (1, 200, 200, 7, [150])])
def test_backward(B, Tq, Tk, H, dn, dv, dt, lens):
    _say(f"bwd B{B} Tq{Tq} Tk{Tk} H{H} dn{dn} dv{dv} {dt} lens {lens}")
    _check_bwd(_expanded(B, Tq, Tk, H, dn, dv, dt, lens=lens, seed=11), dt)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("B,Tq,Tk,H", [(1, 900, 900, 2), (1, 33, 1500, 3)])
def test_backward_longer(B, Tq, Tk, H, dt):
    _say(f"bwd long B{B} Tq{Tq} Tk{Tk} H{H} {dt}")
    _check_bwd(_expanded(B, Tq, Tk, H, 128, 128, dt, seed=13), dt)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("dn,dv", [(64, 128), (128, 64)])
@pytest.mark.parametrize("B,Tq,Tk,H,lens", [
    (3, 700, 700, 2, [700, 70, 0]), (2, 300, 1200, 1, [1200, 930]), (2, 513, 1025, 2, [1025, 513]), (1, 640, 640, 3, None)])
def test_calls_cut_into_pieces(B, Tq, Tk, H, dn, dv, dt, lens):
    """Few workgroups and long walks: keys (fwd, dq) and query rows (dkv) are cut; ragged
    lengths end inside a piece, before one, and before every row."""
    _say(f"pieces B{B} Tq{Tq} Tk{Tk} H{H} dn{dn} dv{dv} {dt} lens {lens}")
    assert gdn.gdn_latent_fwd_workspace_size(B, Tq, Tk, H, dn, 64, dv, DT[dt]) > 0
    d = _expanded(B, Tq, Tk, H, dn, dv, dt, lens=lens, seed=23)
    _check_fwd(d, dt)
    _check_bwd(d, dt)


def test_backward_without_queries_writes_zeros():
    kv, kr = torch.randn(1, 5, 2, 128, device=DEV), torch.randn(1, 5, 64, device=DEV)
    q = torch.zeros(1, 0, 2, 128, device=DEV)
    o, lse = gdn.latent_fwd(q, kv, kr)
    g = gdn.latent_bwd(q, kv, kr, o, lse, torch.empty_like(o))
    torch.cuda.synchronize()
    assert g["dq"].numel() == 0 and (g["dkv"] == 0).all() and (g["dk_rope"] == 0).all()


def test_backward_equals_differences_of_the_forward():
    """fp32 gradients along a random direction of every input, against central
    differences of the fp64 forward (h^2 / 6 of a third derivative of order 1e2 and
    2^-52 / h: both below 1e-7 at h = 1e-5), to the fp32 tolerance of the gradients:
    their sums of about 3e4 terms of order 1 are right to 1e-5 of sqrt(terms)."""
    d = _expanded(2, 70, 90, 2, 64, 64, "fp32", lens=[90, 61], seed=17)
    g = _check_bwd(d, "fp32")
    scale = 1 / math.sqrt(128)
    args = {k: ref.f64(d[k]) for k in ("q", "kv", "k_rope")}
    rng = np.random.default_rng(0)
    for name, grad in (("q", "dq"), ("kv", "dkv"), ("k_rope", "dk_rope")):
        v = rng.standard_normal(args[name].shape)
        f = [(ref.forward(**{**args, name: args[name] + s * 1e-5 * v}, lens=d["lens"], scale=scale)[0] * ref.f64(d["d_o"])).sum()
             for s in (1, -1)]
        num, got = (f[0] - f[1]) / 2e-5, float((ref.f64(g[grad]) * v).sum())
        size = float(np.sqrt((ref.f64(g[grad]) ** 2 * v ** 2).sum()))
        _say(f"{grad}: along a direction {got:.6f}, differences {num:.6f}")
        assert abs(num - got) <= 1e-5 * size + 1e-6


def test_gradients_are_the_same_on_every_call():
    d = _dev(_expanded(2, 300, 300, 5, 64, 128, "bf16", lens=[300, 211], seed=19))
    o, lse = gdn.latent_fwd(d["q"], d["kv"], d["k_rope"], lens=d["lens"])
    a = gdn.latent_bwd(d["q"], d["kv"], d["k_rope"], o, lse, d["d_o"], lens=d["lens"])
    b = gdn.latent_bwd(d["q"], d["kv"], d["k_rope"], o, lse, d["d_o"], lens=d["lens"])
    for k in a:
        assert torch.equal(a[k], b[k]), k


# --- absorbed form ---------------------------------------------------------------
def _paged(lens, H, r, page, dt, M=None, seed=0, width=None, spare=2):
    g = torch.Generator().manual_seed(seed)
    R = lambda *s: torch.randn(*s, generator=g).to(DT[dt])  # noqa: E731
    N = len(lens)
    need = max(-(-n // page) for n in lens) if lens else 0
    width = need if width is None else width
    pages = N * width + spare
    d = dict(cache=R(pages, page, r + 64), table=torch.randperm(pages, generator=g)[:N * width].reshape(N, width).to(torch.int32),
             lens=torch.tensor(lens, dtype=torch.int32), q=R(*((N, H) if M is None else (N, M, H)), r + 64), draft=None, tree=None)
    if M is not None:
        d["draft"] = R(N, M, r + 64)
        parent = torch.stack([torch.randint(-1, i, (N,), generator=g) if i else torch.full((N,), -1) for i in range(M)], 1)
        tree = [[0] * M for _ in range(N)]
        for n in range(N):
            for i in range(M):
                p = int(parent[n, i])
                tree[n][i] = (tree[n][p] if p >= 0 else 0) | 1 << i
        d["tree"] = torch.tensor([[b - (1 << 64) if b >= 1 << 63 else b for b in row] for row in tree], dtype=torch.int64)
    return d


def _run(x, scale, **kw):
    if x["draft"] is None:
        return gdn.latent_step(x["q"], x["cache"], x["table"], x["lens"], scale, want_lse=True, **kw)
    return gdn.latent_steps(x["q"], x["draft"], x["tree"], x["cache"], x["table"], x["lens"], scale, want_lse=True, **kw)


def _check_absorbed(d, dt, scale=None, **kw):
    r = d["q"].shape[-1] - 64
    scale = 1 / math.sqrt(192) if scale is None else scale
    o, lse = _run(_dev(d), scale, **kw)
    torch.cuda.synchronize()
    q = d["q"] if d["draft"] is not None else d["q"][:, None]
    args = (q, d["cache"], d["table"], d["lens"], scale, r, d["draft"], d["tree"])
    ro, rl = ref.absorbed(*args)
    A, _ = ref.absorbed(*args, weigh_abs=True)
    keys = float(np.abs(ref.f64(torch.nan_to_num(d["cache"].float(), 0, 0, 0))).max()) if d["cache"].numel() else 0.0
    if d["draft"] is not None and d["draft"].numel():
        keys = max(keys, float(d["draft"].float().abs().max()))
    # the largest |key| stands for every key: sum |q||k| <= max|k| sum |q|
    ds = (r + 68) * E * scale * keys * np.abs(ref.f64(q)).sum(-1, keepdims=True)
    L = d["table"].shape[1] * d["cache"].shape[1] + 64
    # pieces joined from the workspace add a few fp32 roundings: 16 e
    to = U[dt] * np.abs(ro) + (U[dt] + 2 * ds + (L + 24) * E) * A + 1e-37
    tl = ds[..., 0] + (L + 24) * E + 4 * E * np.abs(np.where(np.isfinite(rl), rl, 0))
    _close("o", o.reshape(ro.shape), ro, to)
    _close("lse", lse.reshape(rl.shape), rl, tl)
    return o, lse


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("r", [512, 256])
@pytest.mark.parametrize("lens,H,page", [
    ([1], 1, 1), ([5, 0, 3], 3, 4), ([64], 16, 64), ([63, 65, 129], 16, 17), ([300, 1, 1000], 17, 100), ([777, 40], 40, 16),
    ([130] * 9, 33, 32), ([2000], 128, 256)])
def test_step(lens, H, page, r, dt):
    _say(f"step lens {lens} H{H} r{r} page {page} {dt}")
    _check_absorbed(_paged(lens, H, r, page, dt, seed=1), dt)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("r", [512, 256])
@pytest.mark.parametrize("lens,M,H,page", [
    ([0], 1, 1, 4), ([0, 7], 5, 3, 4), ([64], 8, 16, 64), ([63, 65, 0, 200], 3, 5, 17), ([500], 64, 4, 100),
    ([130, 1], 33, 8, 16), ([61], 6, 11, 8)])
def test_steps(lens, M, H, page, r, dt):
    _say(f"steps lens {lens} M{M} H{H} r{r} page {page} {dt}")
    d = _paged(lens, H, r, page, dt, M=M, seed=2)
    _check_absorbed(d, dt)
    d["tree"] = None   # a chain
    _check_absorbed(d, dt)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_many_ragged_sequences(dt):
    """More sequences than workgroups, some empty, and a few that many workgroups share."""
    g = torch.Generator().manual_seed(3)
    lens = [int(x) for x in torch.randint(0, 70, (600,), generator=g)]
    lens[0], lens[5], lens[599] = 0, 3000, 0
    _check_absorbed(_paged(lens, 2, 256, 16, dt, seed=4, width=188), dt)


@pytest.mark.parametrize("r", [512, 256])
def test_many_ragged_trees(r):
    """The same for 64 rows a workgroup, with drafts on their own in empty sequences."""
    g = torch.Generator().manual_seed(23)
    lens = [int(x) for x in torch.randint(0, 70, (300,), generator=g)]
    lens[0], lens[5], lens[299] = 0, 2000, 0
    _check_absorbed(_paged(lens, 5, r, 16, "bf16", M=7, seed=24, width=125), "bf16")
    _check_absorbed(_paged(lens, 70, r, 16, "bf16", seed=25, width=125), "bf16")


def test_one_long_sequence_among_empty_ones():
    _check_absorbed(_paged([0] * 40 + [9000] + [0] * 40, 16, 512, 64, "bf16", seed=5, width=141), "bf16")


def test_sequences_without_any_token_or_page():
    d = _paged([0, 0], 4, 512, 16, "bf16", seed=6, width=0)
    o, lse = _run(_dev(d), 0.1)
    assert (o == 0).all() and torch.isneginf(lse).all()
    d = _paged([0, 0], 4, 512, 16, "bf16", M=2, seed=6, width=3)
    d["tree"] = torch.tensor([[0, 0], [1, 0]])   # rows that see nothing beside one that sees itself
    o, lse = _check_absorbed(d, "bf16")
    assert (o[0] == 0).all() and (o[1, 1] == 0).all() and torch.isfinite(lse[1, 0]).all()


def test_lengths_are_clamped_to_the_table():
    d = _paged([40, 40], 4, 256, 16, "fp32", seed=7, width=3)
    d["lens"] = torch.tensor([1000, -5], dtype=torch.int32)
    _check_absorbed(d, "fp32")


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_pages_outside_the_cache_hold_no_tokens(dt):
    d = _paged([100, 70, 33], 5, 512, 16, dt, seed=8)
    d["table"][0, 2], d["table"][1, 0], d["table"][1, 4] = -1, d["cache"].shape[0], 1 << 30
    d["table"][2, :] = -7
    _check_absorbed(d, dt)


@pytest.mark.parametrize("M", [None, 3])
def test_slots_behind_a_sequence_are_not_touched(M):
    """NaN in every slot that holds no live token, and table entries behind the last page
    that name no page."""
    d = _paged([37, 1, 64], 4, 512, 16, "bf16", M=M, seed=9, width=6)
    live = torch.zeros(d["cache"].shape[:2], dtype=torch.bool)
    for n, k in enumerate(d["lens"].tolist()):
        for t in range(k):
            live[d["table"][n, t // 16], t % 16] = True
        d["table"][n, -(-k // 16):] = 1 << 29
    d["cache"][~live] = float("nan")
    _check_absorbed(d, "bf16")


def test_sequences_may_share_pages():
    d = _paged([90, 90], 16, 512, 16, "bf16", seed=10)
    d["table"][1] = d["table"][0]
    d["q"][1] = d["q"][0]
    o, _ = _check_absorbed(d, "bf16")
    assert torch.equal(o[0], o[1])


def test_steps_ignore_bits_from_m_on():
    d = _dev(_paged([50], 4, 512, 16, "bf16", M=3, seed=11))
    o, lse = _run(d, 0.1)
    d["tree"] = d["tree"] | ~0b111
    o2, lse2 = _run(d, 0.1)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("H,M,r", [(1, 6, 512), (4, 6, 256), (16, 6, 512), (16, 6, 256), (3, 64, 512)])
def test_unused_drafts_may_hold_anything(H, M, r, dt):
    """A batch of chains padded to M drafts: what the rows of the used drafts do not see
    (NaN, infinities) leaves no trace in them, and a row that sees it is a NaN."""
    lens, used = [61, 0, 130], [4, M - 1, 1]
    d = _paged(lens, H, r, 16, dt, M=M, seed=17)
    d["tree"] = None
    want, wl = _run(_dev(d), 0.1)
    for n, k in enumerate(used):
        d["draft"][n, k:] = float("nan")
        if n:
            d["draft"][n, k] = 0
            d["draft"][n, k, 3] = float("inf")
    got, gl = _run(_dev(d), 0.1)
    for n, k in enumerate(used):
        assert torch.equal(got[n, :k], want[n, :k]) and torch.equal(gl[n, :k], wl[n, :k])
        assert torch.isnan(got[n, k + 1:]).all()


def test_a_nan_in_a_live_token_shows():
    """In the step, and in the forward in pieces: NaN, never the zeros of an empty row."""
    for lens in ([5], [3000]):
        d = _paged(lens, 4, 512, 16, "bf16", seed=18)
        d["cache"][d["table"][0, 0], 2] = float("nan")
        o, lse = _run(_dev(d), 0.1)
        assert torch.isnan(o).all() and torch.isnan(lse).all()
    d = _dev(_expanded(1, 5, 3001, 2, 128, 128, "bf16", seed=18))
    d["q"].fill_(float("nan"))
    o, lse = gdn.latent_fwd(d["q"], d["kv"], d["k_rope"])
    assert torch.isnan(o).all() and torch.isnan(lse).all()


def test_a_long_cache_passes_32_bit_offsets():
    """Rows beyond 2^31 bytes and 2^31 elements into the cache."""
    page, D = 64, 576
    pages = (1 << 31) // (page * D) + 50
    cache = torch.empty(pages, page, D, dtype=torch.bfloat16, device=DEV)
    table = torch.tensor([[pages - 1, pages - 20, 0]], dtype=torch.int32)
    g = torch.Generator().manual_seed(0)
    small = torch.randn(3, page, D, generator=g).bfloat16()
    for i, p in enumerate(table[0].tolist()):
        cache[p] = small[i].to(DEV)
    q = torch.randn(1, 16, D, generator=g).bfloat16()
    n = torch.tensor([170], dtype=torch.int32, device=DEV)
    far = gdn.latent_step(q.to(DEV), cache, table.to(DEV), n, 0.07)
    near = gdn.latent_step(q.to(DEV), small.to(DEV), torch.tensor([[0, 1, 2]], dtype=torch.int32, device=DEV), n, 0.07)
    assert torch.equal(far, near)


# --- together, streams, graphs ----------------------------------------------------
def test_prefill_then_steps_then_a_tree():
    """The use as a whole, fp32: a prompt by the expanded forward, its latents put in
    pages; the next token by the absorbed step equals the expanded form's row; then a
    tree of drafts, whose accepted path, once appended, gives the same as the tree did."""
    g = torch.Generator().manual_seed(21)
    B, T, H, dn, dv, r, page = 2, 45, 3, 64, 64, 256, 16
    R = lambda *s: torch.randn(*s, generator=g).to(DEV)  # noqa: E731
    c, kr, q = R(B, T, r), R(B, T, 64), R(B, T, H, dn + 64)
    Wk, Wv = R(H, dn, r) / 16, R(H, dv, r) / 16
    up = lambda W: (c.reshape(B * T, r) @ W.reshape(-1, r).t().contiguous()).reshape(B, T, H, -1)  # noqa: E731
    kv = torch.cat((up(Wk), up(Wv)), -1)
    scale = 1 / math.sqrt(dn + 64)
    o, lse = gdn.latent_fwd(q, kv, kr)
    rows = torch.cat((c, kr), -1)
    cache, table = torch.zeros(9, page, r + 64, device=DEV), torch.tensor([[4, 0, 7, 5], [2, 8, 1, 3]], dtype=torch.int32, device=DEV)
    slots = (table.long()[:, :3, None] * page + torch.arange(page, device=DEV)).reshape(B, -1)[:, :T]
    cache.view(-1, r + 64)[slots.reshape(-1)] = rows.reshape(-1, r + 64)

    def absorb(x):   # [.., H, dn + 64] -> [.., H, r + 64]
        return torch.cat((torch.stack([x[..., h, :dn] @ Wk[h] for h in range(H)], -2), x[..., dn:]), -1).contiguous()

    def out(y):
        return torch.stack([y[..., h, :] @ Wv[h].t().contiguous() for h in range(H)], -2)

    n = torch.full((B,), T, dtype=torch.int32, device=DEV)
    y, ly = gdn.latent_step(absorb(q[:, -1]), cache, table, n, scale, want_lse=True)
    # fp32 throughout; the folded products differ by their order: 2 r e of terms of order 1
    torch.testing.assert_close(out(y), o[:, -1], rtol=1e-4, atol=1e-4)
    torch.testing.assert_close(ly, lse[:, -1], rtol=1e-4, atol=1e-4)

    M = 5   # 0 - 1 - 3, 0 - 2, 4 beside 0
    tree = torch.tensor([[1, 3, 5, 11, 16]] * B, device=DEV)
    draft, qd = R(B, M, r + 64), R(B, M, H, r + 64)
    t = gdn.latent_steps(qd, draft, tree, cache, table, n, scale)
    path = [0, 1, 3]
    full = (table.long()[:, :, None] * page + torch.arange(page, device=DEV)).reshape(B, -1)
    for i, m in enumerate(path):
        cache.view(-1, r + 64)[full[:, T + i]] = draft[:, m]
        one = gdn.latent_step(qd[:, m].contiguous(), cache, table, n + i + 1, scale)
        torch.testing.assert_close(one, t[:, m], rtol=1e-5, atol=1e-5)


@pytest.mark.parametrize("T", [200, 1000, 3100])   # in pieces, 3100: the forward in shares
@pytest.mark.parametrize("other", ["object", "handle"])
def test_another_stream(other, T):
    s = torch.cuda.Stream(DEV)
    d = _dev(_paged([700, 20], 16, 512, 16, "bf16", seed=12))
    e = _dev(_expanded(1, T, T, 4, 64, 64, "bf16", seed=12))
    assert (gdn.gdn_latent_fwd_workspace_size(1, T, T, 4, 64, 64, 64, torch.bfloat16) > 0) == (T >= 1000)
    want = _run(d, 0.1)
    ow = gdn.latent_fwd(e["q"], e["kv"], e["k_rope"])
    gw = gdn.latent_bwd(e["q"], e["kv"], e["k_rope"], *ow, e["d_o"])
    torch.cuda.synchronize()
    on = s if other == "object" else s.cuda_stream
    got = _run(d, 0.1, stream=on)
    og = gdn.latent_fwd(e["q"], e["kv"], e["k_rope"], stream=on)
    gg = gdn.latent_bwd(e["q"], e["kv"], e["k_rope"], *og, e["d_o"], stream=on)
    s.synchronize()
    for a, b in zip(want + ow + tuple(gw.values()), got + og + tuple(gg.values())):
        assert torch.equal(a, b)


def test_two_calls_at_once_with_their_own_workspaces():
    d = [_dev(_paged([3000, 100], 16, 512, 16, "bf16", seed=s)) for s in (13, 14)]
    want = [_run(x, 0.1)[0] for x in d]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(DEV) for _ in d]
    for _ in range(5):
        got = [_run(x, 0.1, stream=s)[0] for x, s in zip(d, streams)]
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b)


@pytest.mark.parametrize("T,M,dt", [(150, 4, "bf16"), (700, 8, "bf16"), (300, 2, "fp32"), (2500, 3, "bf16")])   # in pieces, 2500: shares
def test_captured_and_replayed(T, M, dt):
    """The calls in a graph, replayed with new inputs and lengths in place and eager work
    between."""
    d = _dev(_paged([400, 33], 16, 512, 16, dt, M=M, seed=15))
    e = _dev(_expanded(2, T, T, 3, 64, 64, dt, lens=[T, T], seed=15))

    def work():
        o, lse = gdn.latent_fwd(e["q"], e["kv"], e["k_rope"], lens=e["lens"])
        g = gdn.latent_bwd(e["q"], e["kv"], e["k_rope"], o, lse, e["d_o"], lens=e["lens"])
        return [*_run(d, 0.1), gdn.latent_step(d["q"][:, 0].contiguous(), d["cache"], d["table"], d["lens"], 0.1), o, lse, *g.values()]

    s = torch.cuda.Stream(DEV)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        work()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work()
    for i in range(4):
        g = torch.Generator().manual_seed(100 + i)
        for x in (d["q"], d["cache"], d["draft"], e["q"], e["kv"], e["d_o"]):
            x.copy_(torch.randn(x.shape, generator=g).to(x.dtype))
        d["lens"].copy_(torch.tensor([400 - 50 * i, 33 + i], dtype=torch.int32))
        e["lens"].copy_(torch.tensor([T - 70 * i % T, i * T // 3], dtype=torch.int32))
        want = [x.clone() for x in work()]
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(want, got):
            assert torch.equal(a, b), i


def test_outputs_stay_inside_their_buffers():
    """Low-level calls into views of larger buffers: nothing around them changes."""
    d = _dev(_paged([100, 7], 3, 512, 16, "bf16", seed=16))
    e = _dev(_expanded(1, 70, 70, 3, 64, 64, "bf16", seed=16))
    n = gdn.gdn_latent_steps_workspace_size(2, 1, 3, 512, 64, torch.bfloat16)
    big = torch.full((n + 8192,), 77, dtype=torch.uint8, device=DEV)
    ob = torch.full((2 * 3 * 512 + 512,), 5.0, dtype=torch.bfloat16, device=DEV)
    gdn.gdn_latent_step(d["q"], d["cache"], d["table"], d["lens"], ob[256:-256].view(2, 3, 512), None, big[4096:-4096], 0.1)
    assert (ob[:256] == 5).all() and (ob[-256:] == 5).all() and (big[:4096] == 77).all() and (big[-4096:] == 77).all()
    f = _dev(_expanded(1, 70, 1000, 3, 64, 64, "bf16", seed=16))   # in pieces
    n = gdn.gdn_latent_fwd_workspace_size(1, 70, 1000, 3, 64, 64, 64, torch.bfloat16)
    big, ob = torch.full((n + 8192,), 77, dtype=torch.uint8, device=DEV), torch.full((70 * 3 * 64 + 512,), 5.0, dtype=torch.bfloat16, device=DEV)
    lb = torch.full((70 * 3 + 64,), 5.0, device=DEV)
    gdn.gdn_latent_fwd(f["q"], f["kv"], f["k_rope"], None, ob[256:-256].view(1, 70, 3, 64), lb[32:-32].view(1, 70, 3), big[4096:-4096], 0.1)
    want = gdn.latent_fwd(f["q"], f["kv"], f["k_rope"], scale=0.1)
    assert n > 0 and torch.equal(ob[256:-256].view(1, 70, 3, 64), want[0]) and torch.equal(lb[32:-32].view(1, 70, 3), want[1])
    assert (ob[:256] == 5).all() and (ob[-256:] == 5).all() and (big[:4096] == 77).all() and (big[-4096:] == 77).all()
    assert (lb[:32] == 5).all() and (lb[-32:] == 5).all()
    o, lse = gdn.latent_fwd(e["q"], e["kv"], e["k_rope"])
    n = gdn.gdn_latent_bwd_workspace_size(1, 70, 70, 3, 64, 64, 64, torch.bfloat16)
    big = torch.full((n + 8192,), 77, dtype=torch.uint8, device=DEV)
    outs = {k: torch.full((e[s].numel() + 512,), 5.0, dtype=torch.bfloat16, device=DEV) for k, s in (("dq", "q"), ("dkv", "kv"), ("dk_rope", "k_rope"))}
    v = {k: x[256:-256].view(e[s].shape) for (k, x), s in zip(outs.items(), ("q", "kv", "k_rope"))}
    gdn.gdn_latent_bwd(e["q"], e["kv"], e["k_rope"], None, o, lse, e["d_o"], v["dq"], v["dkv"], v["dk_rope"], big[4096:-4096], 1 / math.sqrt(128))
    want = gdn.latent_bwd(e["q"], e["kv"], e["k_rope"], o, lse, e["d_o"])
    for k in v:
        assert torch.equal(v[k], want[k]) and (outs[k][:256] == 5).all() and (outs[k][-256:] == 5).all(), k
    assert (big[:4096] == 77).all() and (big[-4096:] == 77).all()
