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
from test_gpu_attn import (DEV, DT, E, U, _append_args, _bwd_tol, _cache, _check_step, _close, _dev, _fwd_tol, _live, _on, _packed,
                           _parts, _say)

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


# --- work that is shared and cut ------------------------------------------------

def _shared(dt, B, Tq, Tk, Hq, Hk):
    """Sizes whose forward is in shares and whose backward is cut: both have workspaces that the
    offsets fill."""
    assert attn_plans.fwd(dt, B, Tq, Tk, Hq, Hk)["form"] == "shares" and attn_plans.bwd(dt, B, Tq, Tk, Hq, Hk)["kp"] > 1


class _Guarded:
    """Tensors with 0x5a bytes in front of them and behind."""
    def __init__(self):
        self.all = []

    def __call__(self, shape, dtype):
        t = torch.full((2048 + torch.empty(shape, dtype=dtype, device="meta").nbytes,), 0x5a, dtype=torch.uint8, device=DEV)
        self.all.append(t)
        return t[1024:-1024].view(dtype).view(shape)

    def check(self):
        torch.cuda.synchronize()
        for i, t in enumerate(self.all):
            assert (t[:1024] == 0x5a).all() and (t[-1024:] == 0x5a).all(), i


def _all_guarded(d, cu_q, cu_k, dt, scale=0.1):
    """Forward and backward with outputs and workspaces, of just the size that is asked for, in guards."""
    Tq, Hq, D = d["q"].shape
    Tk, Hk, _ = d["k"].shape
    room, sizes, t = _Guarded(), (len(cu_q) - 1, Tq, Tk, Hq, Hk, D, DT[dt]), DT[dt]
    o, lse = room((Tq, Hq, D), t), room((Tq, Hq), torch.float32)
    ws = room((gdn.gdn_attn_fwd_workspace_size(*sizes),), torch.uint8)
    gdn.gdn_attn_fwd(d["q"], d["k"], d["v"], cu_q, cu_k, o, lse, ws, scale)
    g = dict(dq=room((Tq, Hq, D), t), dk=room((Tk, Hk, D), t), dv=room((Tk, Hk, D), t))
    ws = room((gdn.gdn_attn_bwd_workspace_size(*sizes),), torch.uint8)
    gdn.gdn_attn_bwd(d["q"], d["k"], d["v"], cu_q, cu_k, o, lse, d["d_o"].contiguous(), *g.values(), ws, scale)
    room.check()
    return o, lse, g


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("lq,lk,Hq,Hk,D", [
    ([90, 1], [6000, 900], 4, 2, 64), ([64], [4001], 8, 2, 128), ([5, 0, 3], [3100, 7, 4000], 17, 1, 64), ([2500], [2500], 4, 1, 128),
    ([1], [20000], 64, 1, 64)])
def test_shared_work_stays_inside_its_buffers(lq, lk, Hq, Hk, D, dt):
    _say(f"guards lq {lq} lk {lk} Hq{Hq} Hk{Hk} D{D} {dt}")
    _shared(dt, len(lq), sum(lq), sum(lk), Hq, Hk)
    d = _on(_packed(lq, lk, Hq, Hk, D, dt, seed=71))
    o, lse, g = _all_guarded(d, d["cu_q"], d["cu_k"], dt)
    o2, lse2 = gdn.attn_fwd(d["q"], d["k"], d["v"], d["cu_q"], d["cu_k"], scale=0.1)
    g2 = gdn.attn_bwd(d["q"], d["k"], d["v"], o2, lse2, d["d_o"], d["cu_q"], d["cu_k"], scale=0.1)
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and all(torch.equal(g[n], g2[n]) for n in g)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("cq,ck", [([-5, 70, 30, 1000, 100], [10, 9000, 2000, -7, 6500]), ([100, 0, 100, 0, 100], [7000, 0, 7000, 0, 7000]),
                                   ([0, 100, 0, 100, 50], [0, 7000, 0, 7000, 1]), ([2 ** 31 - 1, -2 ** 31, 2 ** 31 - 1, 0, 3], [-2 ** 31, 2 ** 31 - 1, 5, 4, 6])])
def test_offsets_out_of_range_in_shared_work_stay_inside(cq, ck, dt):
    """Offsets that fall or lie outside, sequences over each other among them."""
    _shared(dt, 4, 100, 7000, 4, 2)
    d = _on(_packed([100], [7000], 4, 2, 64, dt, seed=72))
    cu_q, cu_k = (torch.tensor(c, dtype=torch.int32, device=DEV) for c in (cq, ck))
    _all_guarded(d, cu_q, cu_k, dt)


def test_shared_work_side_by_side():
    """Two calls at once on two streams give what they give alone."""
    _shared("bf16", 2, 73, 5000, 4, 2)
    ds = [_on(_packed([70, 3], [4100, 900], 4, 2, 64, "bf16", seed=s)) for s in (1, 2)]

    def both(d, s=None):
        o, lse = gdn.attn_fwd(d["q"], d["k"], d["v"], d["cu_q"], d["cu_k"], stream=s)
        return o, lse, *gdn.attn_bwd(d["q"], d["k"], d["v"], o, lse, d["d_o"], d["cu_q"], d["cu_k"], stream=s).values()

    alone = [both(d) for d in ds]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ds]
    for _ in range(3):
        got = [both(d, s) for d, s in zip(ds, streams)]
        torch.cuda.synchronize()
        for a, b in zip(got, alone):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_shared_work_captured_with_offsets_that_change(dt):
    """Forward and backward in a graph, with eager calls and synchronisations between the replays."""
    Tq, Tk = 120, 7000
    _shared(dt, 3, Tq, Tk, 4, 2)
    d = _on(_packed([Tq], [Tk], 4, 2, 64, dt, seed=73))
    cu_q, cu_k = torch.zeros(4, dtype=torch.int32, device=DEV), torch.zeros(4, dtype=torch.int32, device=DEV)

    def work():
        o, lse = gdn.attn_fwd(d["q"], d["k"], d["v"], cu_q, cu_k)
        return [o, lse, *gdn.attn_bwd(d["q"], d["k"], d["v"], o, lse, d["d_o"], cu_q, cu_k).values()]

    def fill(q, k):
        cu_q.copy_(torch.tensor([0, *q, Tq], dtype=torch.int32))
        cu_k.copy_(torch.tensor([0, *k, Tk], dtype=torch.int32))

    splits = [((40, 80), (2000, 5000)), ((0, 120), (0, 7000)), ((1, 1), (6000, 6100)), ((60, 110), (30, 6900)), ((40, 80), (2000, 5000))]
    fill(*splits[0])
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for q, k in splits:
        fill(q, k)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = work()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), (q, k, i)


# --- the prologue's sums ---------------------------------------------------------

@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("T,Hq,Hk,D", [(16384, 8, 2, 64), (9001, 16, 3, 128), (1000, 32, 8, 128)])
def test_norm_weight_gradients_of_long_calls(T, Hq, Hk, D, dt):
    """dw is a sum of T H terms in 32 bits, but not one after the other: a lane adds up the heads
    of its tokens, the workgroup its 256 / (D / 8) groups, then 64 runs of up to 1024 workgroups
    are added up, and the runs.  Its rounding goes by the longest chain of these, n additions, so
    it is off by (n + D + 40) e of the sum of absolute terms (D + 40: each term's own)."""
    g = torch.Generator().manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    raw, dy, w = r(T, Hq + Hk, D).to(DT[dt]), r(T, Hq + Hk, D).to(DT[dt]), 1 + r(D) / 4
    inv, pos = 10000.0 ** (-torch.arange(0, D, 2) / D), torch.arange(T, dtype=torch.int32)
    x, y, wd = raw.to(DEV), dy.to(DEV), w.to(DEV)
    got = gdn.attn_prologue_bwd(x[:, :Hq], x[:, Hq:], wd, wd, inv.to(DEV), pos.to(DEV), y[:, :Hq].contiguous(), y[:, Hq:].contiguous())
    groups = 256 // (D // 8)
    for n, a, b in (("dw_q", 0, Hq), ("dw_k", Hq, Hq + Hk)):
        X, Z = ref.f64(raw[:, a:b]), ref.turn(ref.f64(dy[:, a:b]), inv, pos, back=True)
        X = X / np.sqrt((X * X).mean(-1, keepdims=True) + 1e-6)
        A = np.abs(ref.f64(dy[:, a:b]))
        A = np.concatenate([A[..., :D // 2] + A[..., D // 2:]] * 2, -1)
        # one token at a time or four: the chain of four in groups / 4 is as long or longer
        chain = -(-T // 1024) * -(-(b - a) // (groups // 4)) + groups + 16 + 64
        _close(n, got[n], (Z * X).sum((0, 1)), (chain + D + 40) * E * (A * np.abs(X)).sum((0, 1)))


# --- strides --------------------------------------------------------------------

@pytest.mark.parametrize("dt,T,step", [("bf16", 2100, 1 << 20), ("bf16", 1100, 1 << 21), ("fp32", 300, 1 << 21)])
def test_inputs_and_gradients_at_large_steps(dt, T, step):
    """q, k and v from slices of a tensor of more than 2^31 bytes, and gradients into others, up to
    the largest step from token to token: the same bits as from contiguous tensors."""
    Hq, Hk, D = 4, 2, 64
    H = Hq + 2 * Hk
    _say(f"steps of {step}, {T} tokens, {dt}")
    big = torch.empty(T, step, dtype=DT[dt], device=DEV)
    assert big.nbytes > 1 << 31
    x, y = (big.as_strided((T, H, D), (step, D, 1), at) for at in (0, 2048))   # gradients beside the values
    x.copy_(torch.randn(T, H, D, generator=torch.Generator().manual_seed(1)))
    far = x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:]
    near = [t.contiguous() for t in far]
    cu = torch.tensor([0, T - 200, T], dtype=torch.int32, device=DEV)
    d_o = torch.randn(T, Hq, D, generator=torch.Generator().manual_seed(2)).to(DT[dt]).to(DEV)
    o, lse = gdn.attn_fwd(*near, cu)
    o2, lse2 = gdn.attn_fwd(*far, cu)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    want = gdn.attn_bwd(*near, o, lse, d_o, cu)
    got = gdn.attn_bwd(*far, o, lse, d_o, cu)
    assert all(torch.equal(got[n], want[n]) for n in want)
    ws = torch.empty(gdn.gdn_attn_bwd_workspace_size(2, T, T, Hq, Hk, D, DT[dt]), dtype=torch.uint8, device=DEV)
    into = y[:, :Hq], y[:, Hq:Hq + Hk], y[:, Hq + Hk:]
    gdn.gdn_attn_bwd(*far, cu, None, o, lse, d_o, *into, ws, D ** -0.5)
    assert all(torch.equal(t, want[n]) for n, t in zip(("dq", "dk", "dv"), into))
    w = torch.linspace(0.5, 1.5, D, device=DEV)
    args = w, w, torch.rand(D // 2, generator=torch.Generator().manual_seed(3)).to(DEV), torch.arange(T, dtype=torch.int32, device=DEV)
    q, k = gdn.attn_prologue(*near[:2], *args)
    assert all(torch.equal(a, b) for a, b in zip((q, k), gdn.attn_prologue(*far[:2], *args)))
    want = gdn.attn_prologue_bwd(*near[:2], *args, q, k)
    got = gdn.attn_prologue_bwd(*far[:2], *args, q, k)
    assert all(torch.equal(got[n], want[n]) for n in want)
    ws = torch.empty(gdn.gdn_attn_prologue_bwd_workspace_size(T, Hq, Hk, D, D, DT[dt]), dtype=torch.uint8, device=DEV)
    dw = torch.empty(2, D, device=DEV)
    gdn.gdn_attn_prologue_bwd(*far[:2], *args, q, k, *into[:2], dw[0], dw[1], ws, 1e-6)
    assert all(torch.equal(a, want[n]) for n, a in zip(("dq_raw", "dk_raw", "dw_q", "dw_k"), (*into[:2], *dw)))


def test_append_at_large_steps():
    """New tokens from slices at the largest step: the same bytes as from contiguous tensors."""
    T, Hk, D, page, step = 1100, 2, 64, 16, 1 << 21
    big = torch.empty(T, step, dtype=torch.bfloat16, device=DEV)
    x = big.as_strided((T, 2 * Hk, D), (step, D, 1), 0)
    x.copy_(torch.randn(T, 2 * Hk, D, generator=torch.Generator().manual_seed(1)))
    table = torch.randperm(70, generator=torch.Generator().manual_seed(2)).to(torch.int32).to(DEV)[None]
    lens, cu, out = torch.tensor([T + 3], dtype=torch.int32, device=DEV), torch.tensor([0, T], dtype=torch.int32, device=DEV), []
    for k, v in ((x[:, :Hk], x[:, Hk:]), (x[:, :Hk].contiguous(), x[:, Hk:].contiguous())):
        c = [torch.zeros(70, Hk, page, D, dtype=torch.uint8, device=DEV), torch.zeros(70, Hk, 1, D, 16, dtype=torch.uint8, device=DEV),
             torch.zeros(70, Hk, 1, device=DEV), torch.zeros(70, Hk, 1, device=DEV)]
        gdn.attn_append_(k, v, *c, table, lens, cu=cu)
        out.append(c)
    assert (out[0][0] != 0).any() and all(torch.equal(a, b) for a, b in zip(*out))


# --- one token ------------------------------------------------------------------

@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("N,Hq,Hk,D,longest", [(1, 1, 1, 64, 20000), (300, 3, 1, 64, 9000), (70, 34, 2, 64, 6000), (1000, 8, 8, 64, 4000), (64, 20, 4, 128, 2500),
                                               (5, 64, 1, 128, 5000)])
def test_cut_steps_stay_inside_their_workspace(N, Hq, Hk, D, longest, dt):
    """A few long sequences in pieces among many short, whole and empty ones, with a workspace of
    just the size that is asked for."""
    _say(f"cut step N{N} Hq{Hq} Hk{Hk} D{D} {dt}")
    g, page = torch.Generator().manual_seed(N), 16
    width = longest // page
    c = _live(_cache(5, 40, page, Hk, D, seed=N))
    c["table"] = torch.randint(0, len(c["k_cache"]), (N, width), generator=g).to(torch.int32)   # pages shared
    long = {N - 1: longest, N // 2: longest // 2 + 3, 3: longest - 1}
    lens = [long.get(i, (37 * i) % 90) for i in range(N)]
    q = (torch.randn(N, Hq, D, generator=g) * 0.2).to(DT[dt])
    o, lse = _check_step(c, q, lens, dt)
    x, room = _dev(c), _Guarded()
    o2, lse2 = room((N, Hq, D), DT[dt]), room((N, Hq), torch.float32)
    size = gdn.gdn_attn_step_workspace_size(N, Hq, Hk, D, page, width)
    assert size > 0
    gdn.gdn_attn_step(q.to(DEV), *_append_args(x), torch.tensor(lens, dtype=torch.int32, device=DEV), o2, lse2, room((size,), torch.uint8),
                      D ** -0.5)
    room.check()
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


# --- calls that a user may make -------------------------------------------------

@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("Hq,Hk,T", [(4, 0, 5), (0, 3, 5), (0, 2, 1), (6, 0, 5000), (0, 0, 7)])
def test_prologue_of_queries_or_keys_alone(Hq, Hk, T, dt):
    """No heads on one side: the other is as with both, the norm weight's gradient of none is 0."""
    D, g = 64, torch.Generator().manual_seed(T)
    both = torch.randn(T, 9, D, generator=g).to(DT[dt]).to(DEV)
    w, inv, pos = torch.rand(2, D, generator=g).to(DEV), torch.rand(16, generator=g).to(DEV), torch.arange(T, dtype=torch.int32, device=DEV)
    args = w[0], w[1], inv, pos
    full = gdn.attn_prologue(both[:, :6], both[:, 6:], *args)
    q, k = gdn.attn_prologue(both[:, :Hq], both[:, 6:6 + Hk], *args)
    assert torch.equal(q, full[0][:, :Hq]) and torch.equal(k, full[1][:, :Hk])
    want = gdn.attn_prologue_bwd(both[:, :6], both[:, 6:], *args, *full)
    got = gdn.attn_prologue_bwd(both[:, :Hq], both[:, 6:6 + Hk], *args, q, k)
    assert torch.equal(got["dq_raw"], want["dq_raw"][:, :Hq]) and torch.equal(got["dk_raw"], want["dk_raw"][:, :Hk])
    assert (Hq or (got["dw_q"] == 0).all()) and (Hk or (got["dw_k"] == 0).all())


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("lq,lk,form", [([600] * 5, None, "whole"), ([65, 1], [90, 70], "halves"), ([60, 3], [6300, 900], "shares")])
def test_forward_without_lse(lq, lk, form, dt):
    Hq, Hk = (64, 16) if form == "whole" else (4, 2)
    assert attn_plans.fwd(dt, len(lq), sum(lq), sum(lk or lq), Hq, Hk)["form"] == form
    d = _on(_packed(lq, lk, Hq, Hk, 64, dt, seed=81))
    o, _ = gdn.attn_fwd(d["q"], d["k"], d["v"], d["cu_q"], d["cu_k"], scale=0.1)
    n = gdn.gdn_attn_fwd_workspace_size(len(lq), sum(lq), sum(lk or lq), Hq, Hk, 64, DT[dt])
    o2, ws = torch.empty_like(o), torch.empty(n, dtype=torch.uint8, device=DEV) if n else None
    gdn.gdn_attn_fwd(d["q"], d["k"], d["v"], d["cu_q"], d["cu_k"], o2, None, ws, 0.1)
    assert torch.equal(o, o2)


def test_idle_sequences_of_a_serving_batch():
    """Sequences of no tokens among those of a decoding batch: one new row each, of which theirs is
    not stored, whatever their table says, and their token is 0; the others are as without them."""
    N, Hq, Hk, D, page, width = 7, 8, 2, 64, 32, 3
    idle = [0, 3, 6]
    live = [i for i in range(N) if i not in idle]
    g = torch.Generator().manual_seed(4)
    c = _live(_cache(N, width, page, Hk, D, seed=9))
    lens = torch.tensor([0 if i in idle else 17 * i for i in range(N)], dtype=torch.int32)
    q, k, v = (torch.randn(N, H, D, generator=g).to(torch.bfloat16).to(DEV) for H in (Hq, Hk, Hk))
    one, few = _dev(c), _dev({n: t.clone() for n, t in c.items()})
    few["table"] = few["table"][live].contiguous()
    one["table"][idle] = one["table"][live[0]].clone()   # another's pages
    gdn.attn_append_(k, v, *_append_args(one), lens.to(DEV))
    gdn.attn_append_(k[live], v[live], *_append_args(few), lens[live].to(DEV))
    for n in ("k_cache", "v_cache", "k_scale", "v_scale"):
        assert torch.equal(one[n], few[n]), n
    o, lse = gdn.attn_step(q, *_append_args(one), lens.to(DEV), want_lse=True)
    o2, lse2 = gdn.attn_step(q[live], *_append_args(few), lens[live].to(DEV), want_lse=True)
    assert torch.equal(o[live], o2) and torch.equal(lse[live], lse2)
    assert (o[idle] == 0).all() and torch.isneginf(lse[idle]).all()


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_prologue_captured(dt):
    """The prologue and its gradients in a graph; positions and rows change between replays."""
    T, Hq, Hk, D = 700, 4, 2, 64
    raw, d_q, d_k = (torch.randn(T, H, D, generator=torch.Generator().manual_seed(H), dtype=torch.float32).to(DT[dt]).to(DEV)
                     for H in (Hq + Hk, Hq, Hk))
    w, inv, pos = torch.rand(2, D).to(DEV), torch.rand(D // 2).to(DEV), torch.zeros(T, dtype=torch.int32, device=DEV)
    work = lambda: [*gdn.attn_prologue(raw[:, :Hq], raw[:, Hq:], w[0], w[1], inv, pos),  # noqa: E731
                    *gdn.attn_prologue_bwd(raw[:, :Hq], raw[:, Hq:], w[0], w[1], inv, pos, d_q, d_k).values()]
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        work()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = work()
    for i in range(4):
        pos.add_(1000 * i + 1)
        raw.mul_(0.75)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        assert all(torch.equal(a, b) for a, b in zip(got, work())), i
        torch.cuda.synchronize()


def test_one_tensor_as_keys_and_values():
    d = _on(_packed([130, 5], None, 4, 2, 64, "bf16", seed=83))
    k = d["k"].contiguous()
    o, lse = gdn.attn_fwd(d["q"], k, k, d["cu_q"])
    o2, lse2 = gdn.attn_fwd(d["q"], k, k.clone(), d["cu_q"])
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    g, g2 = (gdn.attn_bwd(d["q"], k, x, o, lse, d["d_o"], d["cu_q"]) for x in (k, k.clone()))
    assert all(torch.equal(g[n], g2[n]) for n in g)
