"""How calls of the grouped-attention kernels are cut (CPU): bounds that the kernels' grids
and workspaces rest on, and the form that typical sizes take."""
import random

import pytest

import attn_plans


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_grids_cover_every_split_of_the_rows(dt):
    """The row tiles of any packing of Tq rows into B sequences fit the grid."""
    rng = random.Random(0)
    for _ in range(400):
        B, G, Hk = rng.choice((1, 2, 7, 64, 300)), rng.choice((1, 2, 3, 5, 8, 16, 33, 64)), rng.choice((1, 2, 8))
        lens = [rng.choice((0, 0, 0, 1, 2, 3, 17, 64, 65, 400)[:rng.choice((4, 10))]) for _ in range(B)]
        T = sum(lens)
        f, b = attn_plans.fwd(dt, B, T, T, G * Hk, Hk), attn_plans.bwd(dt, B, T, T, G * Hk, Hk)
        for tokens, tiles in ((f["tokens"], f["tiles"]), (b["tokens"], b["qtiles"])):
            assert tokens >= 1 and sum(-(-n // tokens) for n in lens) <= tiles
            if B > 64:   # tile t of sequence b is number start / tokens + b + t
                starts = [sum(lens[:b]) // tokens + b for b in range(B + 1)]
                assert all(a + -(-n // tokens) <= e for a, e, n in zip(starts, starts[1:], lens)) and starts[-1] <= tiles
        assert f["tokens"] * G <= 64 * f["nr"] and b["tokens"] * G <= (128 if dt == "bf16" else 64)
        assert b["shares"] % 8 == 0 and 8 <= b["shares"] <= 256
        st = 64 if dt == "bf16" else 32
        assert b["kp"] == 1 or b["kstep"] % st == 0 and b["kstep"] > 0
        assert f["shares"] in (0, 512) and not (f["shares"] and f["halves"])


@pytest.mark.parametrize("dt,B,Tq,Tk,Hq,Hk,form", [
    ("bf16", 1, 333, 333, 32, 8, "halves"), ("bf16", 7, 8192, 8192, 32, 8, "whole"), ("bf16", 1, 4096, 4096, 8, 2, "shares"),
    ("bf16", 1, 2048, 2048, 8, 2, "halves"), ("bf16", 4, 4000, 4000, 8, 2, "whole"), ("bf16", 1, 5, 3001, 8, 2, "shares"),
    ("fp32", 1, 1000, 1000, 8, 2, "shares"), ("fp32", 5, 613, 613, 8, 2, "halves"), ("bf16", 0, 0, 0, 8, 2, "whole")])
def test_form_of_the_forward(dt, B, Tq, Tk, Hq, Hk, form):
    p = attn_plans.fwd(dt, B, Tq, Tk, Hq, Hk)
    assert p["form"] == form or (Tq == 0 and not p["shares"])


@pytest.mark.parametrize("dt,B,T,Hq,Hk,kp", [("bf16", 1, 333, 16, 4, 1), ("bf16", 1, 1000, 8, 2, 4), ("bf16", 8, 2400, 8, 2, 1),
                                             ("bf16", 7, 8192, 16, 4, 1), ("fp32", 1, 300, 4, 4, 10)])
def test_pieces_of_the_backward(dt, B, T, Hq, Hk, kp):
    assert attn_plans.bwd(dt, B, T, T, Hq, Hk)["kp"] == kp
