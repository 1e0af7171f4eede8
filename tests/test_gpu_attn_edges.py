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
from test_gpu_attn import DEV, E, U, _close, _on, _packed, _say

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
