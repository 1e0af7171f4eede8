"""Latent attention on the paths that large calls take, against the fp64 oracle: two row
groups a wave, uncut backward passes and long pieces, many key tiles a share.  Each test
asks the launchers' own rules whether its sizes take that path.  Tolerances are those of
test_gpu_latent.py; heads and sequences are independent, so a few stand for all."""
import math

import numpy as np
import pytest
import torch

import gated_deltanet_layer_amd as gdn
from oracle import latent as ref
from tests import latent_plans as plans
from tests.test_gpu_latent import DIMS, DT, E, U, _bwd_tol, _check_absorbed, _close, _dev, _expanded, _fwd_tol, _paged, _say

pytestmark = pytest.mark.gpu


def _part(d, seqs, heads):
    """Some sequences and heads of a call's tensors."""
    out = {}
    for k, x in d.items():
        if x is not None:
            x = x[seqs]
            out[k] = x[:, :, heads].contiguous() if x.dim() == 4 or k == "lse" else x
    return {"lens": None, **out}


def _fwd_parts(d, dt, seqs, heads, scale=None):
    scale = 1 / math.sqrt(d["q"].shape[-1]) if scale is None else scale
    x = _dev(d)
    o, lse = gdn.latent_fwd(x["q"], x["kv"], x["k_rope"], lens=x["lens"], scale=scale)
    torch.cuda.synchronize()
    p = _part(d, seqs, heads)
    ro, rl = ref.forward(p["q"], p["kv"], p["k_rope"], p["lens"], scale)
    to, tl = _fwd_tol(p, scale, U[dt])
    _close("o", o[seqs][:, :, heads], ro, to + U[dt] * np.abs(ro) + 1e-37)
    _close("lse", lse[seqs][:, :, heads], rl, tl + 4 * E * np.abs(np.where(np.isfinite(rl), rl, 0)) + 1e-37)
    return o, lse


@pytest.mark.parametrize("dn,dv", DIMS)
@pytest.mark.parametrize("B,Tq,Tk,H,lens,cut", [
    (4, 520, 520, 32, [520, 513, 130, 0], "whole"), (2, 600, 1100, 64, [1100, 850], "whole"),
    (8, 130, 130, 32, [130, 129, 128, 65, 64, 1, 0, 130], "whole"), (1, 2100, 2100, 32, None, "whole"),
    (1, 530, 530, 64, [517], "pieces"), (2, 500, 700, 32, [700, 431], "pieces")])
def test_forward_two_row_groups(B, Tq, Tk, H, dn, dv, lens, cut):
    assert plans.fwd("bf16", B, Tq, Tk, H) == (2, cut)
    _say(f"fwd two groups B{B} Tq{Tq} Tk{Tk} H{H} dn{dn} dv{dv} {cut}")
    d = _expanded(B, Tq, Tk, H, dn, dv, "bf16", seed=31, lens=lens)
    o, lse = _fwd_parts(d, "bf16", list(range(min(B, 4))), [0, H // 2 + 1, H - 1])
    if lens is not None:
        for b, n in enumerate(lens):   # padding, of every head
            row = max(0, n - (Tk - Tq))
            assert (o[b, row:] == 0).all() and torch.isneginf(lse[b, row:]).all()


def test_forward_two_row_groups_with_a_rising_maximum():
    """Scores that grow along the keys, so that every tile rescales what came before."""
    B, T, H = 4, 520, 32
    assert plans.fwd("bf16", B, T, T, H) == (2, "whole")
    d = _expanded(B, T, T, H, 64, 64, "bf16", seed=32)
    d["kv"] = (d["kv"].float() * torch.linspace(0.2, 3.0, T)[None, :, None, None]).bfloat16()
    _fwd_parts(d, "bf16", [0, 3], [1, 30], scale=2.0)


@pytest.mark.parametrize("dn,dv", DIMS)
def test_forward_fp32_whole(dn, dv):
    assert plans.fwd("fp32", 2, 260, 260, 64) == (1, "whole")
    _fwd_parts(_expanded(2, 260, 260, 64, dn, dv, "fp32", seed=33, lens=[260, 201]), "fp32", [0, 1], [0, 40, 63])


def _bwd_parts(d, dt, seqs):
    """All heads of some sequences (the rotary gradient adds them up)."""
    scale = 1 / math.sqrt(d["q"].shape[-1])
    x = _dev(d)
    o, lse = gdn.latent_fwd(x["q"], x["kv"], x["k_rope"], lens=x["lens"])
    g = gdn.latent_bwd(x["q"], x["kv"], x["k_rope"], o, lse, x["d_o"], lens=x["lens"])
    torch.cuda.synchronize()
    H = d["q"].shape[2]
    for b in seqs:
        p = _part(dict(d, o=o.cpu(), lse=lse.cpu()), [b], list(range(H)))
        want = ref.backward(p["q"], p["kv"], p["k_rope"], p["lens"], p["o"], p["lse"], p["d_o"], scale)
        tol = _bwd_tol(p, p["o"], p["lse"], scale, U[dt])
        for name, w, t in zip(("dq", "dkv", "dk_rope"), want, tol):
            _close(f"{name}[{b}]", g[name][b:b + 1], w, t + U[dt] * np.abs(w) + 1e-37)
    if d["lens"] is not None:
        off = d["kv"].shape[1] - d["q"].shape[1]
        for b, n in enumerate(d["lens"].tolist()):
            assert (g["dq"][b, max(0, n - off):] == 0).all() and (g["dkv"][b, n:] == 0).all() and (g["dk_rope"][b, n:] == 0).all()
    return g


@pytest.mark.parametrize("dn,dv", DIMS)
@pytest.mark.parametrize("B,Tq,Tk,H,lens,seqs", [
    (5, 520, 520, 32, [520, 517, 130, 0, 389], [1, 4]), (8, 300, 420, 32, [420, 300, 121, 120, 119, 0, 257, 419], [0, 2, 7])])
def test_backward_uncut(B, Tq, Tk, H, dn, dv, lens, seqs):
    """Both kernels walk every tile of their rows themselves, three buffers over and over."""
    (kp, _), (qp, _) = plans.bwd("bf16", B, Tq, Tk, H)
    assert kp == 1 and qp == 1 and Tk // 64 >= 6
    _say(f"bwd uncut B{B} Tq{Tq} Tk{Tk} H{H} dn{dn} dv{dv}")
    _bwd_parts(_expanded(B, Tq, Tk, H, dn, dv, "bf16", seed=34, lens=lens), "bf16", seqs)


@pytest.mark.parametrize("dn,dv", DIMS)
def test_backward_fp32_uncut(dn, dv):
    (kp, _), (qp, _) = plans.bwd("fp32", 4, 260, 260, 32)
    assert kp == 1 and qp == 1
    _bwd_parts(_expanded(4, 260, 260, 32, dn, dv, "fp32", seed=35, lens=[260, 259, 0, 97]), "fp32", [1, 3])


@pytest.mark.parametrize("dn,dv", [(128, 128), (64, 128)])
@pytest.mark.parametrize("B,T,H,lens,keys,rows,seqs", [
    (2, 900, 10, [900, 833], False, True, [1]), (4, 900, 10, [900, 833, 500, 700], True, False, [1, 2])])
def test_backward_in_long_pieces(B, T, H, dn, dv, lens, keys, rows, seqs):
    """Pieces of eight tiles, of the query rows (dk, dv) and of the keys (dq)."""
    (kp, kt), (qp, qt) = plans.bwd("bf16", B, T, T, H)
    assert (not keys or (kp > 1 and kt >= 8)) and (not rows or (qp > 1 and qt >= 8)) and (rows or qp == 1)
    _bwd_parts(_expanded(B, T, T, H, dn, dv, "bf16", seed=36, lens=lens), "bf16", seqs)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_backward_of_peaked_rows(dt):
    """Scores of a standard deviation of 8: most rows give nearly all their weight to one key,
    and D, by the stored o, carries that key's rounding.  Also says how far the gradients
    are from those of the forward in 64 bits, whose o is not rounded."""
    B, T, H = 2, 400, 5
    scale = 1 / math.sqrt(192)
    d = _expanded(B, T, T, H, 128, 128, dt, seed=42)
    d["q"] = (d["q"].float() * 8).to(DT[dt])
    g = _bwd_parts(d, dt, [0, 1])
    o, lse = ref.forward(d["q"], d["kv"], d["k_rope"], None, scale)
    want = ref.backward(d["q"], d["kv"], d["k_rope"], None, o, lse, d["d_o"], scale)
    for name, w in zip(("dq", "dkv", "dk_rope"), want):
        _say(f"{name} {dt}: off by {np.linalg.norm(ref.f64(g[name]) - w) / np.linalg.norm(w):.2e} of its norm")


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("B,Tq,Tk,H,lens", [(1, 1, 5000, 1, None), (2, 7, 4200, 2, [4200, 4194])])
def test_backward_of_few_rows_over_many_keys(B, Tq, Tk, H, lens, dt):
    (kp, _), (qp, _) = plans.bwd(dt, B, Tq, Tk, H)
    assert 20 <= kp <= 32 and qp == 1
    _bwd_parts(_expanded(B, Tq, Tk, H, 128, 64, dt, seed=41, lens=lens), dt, list(range(B)))


def test_backward_without_heads_writes_zeros():
    """No head, but keys: the rotary gradient, a sum over no heads, is written."""
    x = [torch.randn(s, device="cuda") for s in ((2, 5, 0, 128), (2, 5, 0, 128), (2, 5, 64))]
    o, lse = gdn.latent_fwd(*x)
    g = gdn.latent_bwd(*x, o, lse, torch.empty_like(o))
    assert o.shape == (2, 5, 0, 64) and g["dq"].numel() == 0 and g["dkv"].numel() == 0
    assert g["dk_rope"].shape == (2, 5, 64) and (g["dk_rope"] == 0).all()


def test_keys_beyond_32_bit_offsets():
    """kv and its gradient of more than 2^31 values: the first and the last head."""
    Tq, Tk, H, heads = 64, 66000, 256, [0, 255]
    assert Tk * H * 128 > 1 << 31
    gen = torch.Generator("cuda").manual_seed(43)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=torch.bfloat16)  # noqa: E731
    x = dict(q=r(1, Tq, H, 128), kv=r(1, Tk, H, 128), k_rope=r(1, Tk, 64), d_o=r(1, Tq, H, 64))
    o, lse = gdn.latent_fwd(x["q"], x["kv"], x["k_rope"])
    g = gdn.latent_bwd(x["q"], x["kv"], x["k_rope"], o, lse, x["d_o"])
    p = {k: v.cpu() for k, v in _part({**x, "o": o, "lse": lse}, [0], heads).items() if v is not None}
    scale = 1 / math.sqrt(128)
    ro, rl = ref.forward(p["q"], p["kv"], p["k_rope"], None, scale)
    to, tl = _fwd_tol({**p, "lens": None}, scale, U["bf16"])
    _close("o", p["o"], ro, to + U["bf16"] * np.abs(ro) + 1e-37)
    _close("lse", p["lse"], rl, tl + 4 * E * np.abs(rl))
    want = ref.backward(p["q"], p["kv"], p["k_rope"], None, p["o"], p["lse"], p["d_o"], scale)
    tol = _bwd_tol({**p, "lens": None}, p["o"], p["lse"], scale, U["bf16"])
    for name, w, t in list(zip(("dq", "dkv"), want, tol)):
        _close(name, g[name][:, :, heads], w, t + U["bf16"] * np.abs(w) + 1e-37)


def _tiles_a_share(dt, lens, rows, drafts):
    rt, shares = plans.step(dt, rows)
    kt = 64 if dt == "bf16" and rt <= 32 else 32
    return rt, sum(-(-(n + drafts) // kt) for n in lens) / shares


LENS = [4600 - 37 * i for i in range(40)]   # 155,000 tokens


@pytest.mark.parametrize("r", [512, 256])
@pytest.mark.parametrize("H,rt,page", [(13, 16, 17), (31, 32, 100)])
def test_step_with_long_shares(H, rt, page, r):
    got, tiles = _tiles_a_share("bf16", LENS, H, 0)
    assert got == rt and tiles >= 9
    _say(f"step long shares H{H} r{r} page {page}: {tiles:.1f} tiles a share")
    _check_absorbed(_paged(LENS, H, r, page, "bf16", seed=37), "bf16")


@pytest.mark.parametrize("r", [512, 256])
@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_step_of_many_heads_with_long_shares(dt, r):
    lens = [4501, 1, 2999, 0, 5000]
    rt, tiles = _tiles_a_share(dt, lens, 500 if dt == "bf16" else 125, 0)
    assert rt == (64 if dt == "bf16" else 16) and tiles >= 10
    _check_absorbed(_paged(lens, 500 if dt == "bf16" else 125, r, 17, dt, seed=38), dt)


@pytest.mark.parametrize("r", [512, 256])
@pytest.mark.parametrize("page", [17, 64])
def test_trees_with_long_shares(page, r):
    lens = [4501, 0, 2999, 5003]
    rt, tiles = _tiles_a_share("bf16", lens, 17 * 30, 17)
    assert rt == 64 and tiles >= 10
    _check_absorbed(_paged(lens, 30, r, page, "bf16", M=17, seed=39), "bf16")


@pytest.mark.parametrize("H,M", [(16, None), (32, None), (30, 17)])
def test_long_shares_with_a_rising_maximum(H, M):
    """Scores that grow along the cache, so that every tile rescales what came before."""
    lens = [5003, 2999, 4501] if M else LENS
    rt, tiles = _tiles_a_share("bf16", lens, H * (M or 1), M or 0)
    assert tiles >= 9
    d = _paged(lens, H, 512, 16, "bf16", M=M, seed=40)
    c = d["cache"].view(-1, 576)
    for n, k in enumerate(lens):
        at = torch.arange(k)
        slots = d["table"][n].long()[at // 16] * 16 + at % 16
        c[slots] = (c[slots].float() * (0.2 + 3.0 * at / k)[:, None]).bfloat16()
    _check_absorbed(d, "bf16", scale=0.15)
