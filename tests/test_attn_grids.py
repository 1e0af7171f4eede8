"""Grids of the grouped-attention kernels (CPU): every size that the entry points accept gives
launches of less than 2^32 threads, the most that a launch takes."""
import os
import random

import pytest
import torch

import attn_plans
import gated_deltanet_layer_amd as gdn

DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not os.path.exists(gdn.LIB_PATH):
        from gated_deltanet_layer_amd import build
        build.build()


def _accepted(query, *args):
    try:
        query(*args)
    except gdn.GDNError as e:
        assert e.status == gdn.GDN_ENOTSUP
        return False
    return True


def _threads(dt, B, Tq, Tk, Hq, Hk, D):
    """Threads of the launches whose number of workgroups grows with the sizes."""
    f, b = attn_plans.fwd(dt, B, Tq, Tk, Hq, Hk), attn_plans.bwd(dt, B, Tq, Tk, Hq, Hk)
    run = 4 if Tk * Hk >= 4 * 4096 else 1
    return dict(fwd=512 * 256 if f["shares"] else f["tiles"] * Hk * (512 if f["halves"] else 256),
                join=Tq * Hq * 256 if f["shares"] and Tq * Hq <= 2048 else f["shares"] and Tq * Hq * D // 4,
                bwd_q=b["qtiles"] * Hk * b["kp"] * 256, bwd_kv=b["shares"] * 512,
                bwd_sum=(Tq * Hq * D // 4 if b["kp"] > 1 else 0) + -(-Tk // run) * Hk * 2 * D // 4 + 512)


MANY = [("bf16", 1_100_000, 1000, 1000, 8, 8), ("fp32", 9_000_000, 1000, 1000, 1, 1), ("bf16", 9_000_000, 100, 100, 64, 1),
        ("bf16", (1 << 24) - 1, 1, 1, 1, 1), ("bf16", 1 << 21, 500, 500, 4, 4), ("bf16", (1 << 23) - 20, 1000, 1000, 1, 1)]


@pytest.mark.parametrize("dt,B,Tq,Tk,Hq,Hk", MANY)
@pytest.mark.parametrize("D", [64, 128])
def test_many_sequences_of_few_tokens(dt, B, Tq, Tk, Hq, Hk, D):
    if _accepted(gdn.gdn_attn_fwd_workspace_size, B, Tq, Tk, Hq, Hk, D, DT[dt]):
        t = _threads(dt, B, Tq, Tk, Hq, Hk, D)
        assert max(t.values()) < 1 << 32, t


def test_sizes_over_the_whole_range():
    rng = random.Random(0)
    log = lambda hi: int(2 ** rng.uniform(0, hi))  # noqa: E731
    seen = 0
    for _ in range(20000):
        dt, Hk, G, D = rng.choice(("bf16", "fp32")), log(14), rng.choice((1, 2, 3, 5, 8, 16, 64)), rng.choice((64, 128))
        B, Tq, Tk = log(24.2), log(28), log(26)
        if rng.random() < 0.5:
            Tq = Tk
        if not _accepted(gdn.gdn_attn_fwd_workspace_size, B, Tq, Tk, Hk * G, Hk, D, DT[dt]):
            continue
        seen += 1
        t = _threads(dt, B, Tq, Tk, Hk * G, Hk, D)
        assert max(t.values()) < 1 << 32, (dt, B, Tq, Tk, G, Hk, t)
    assert seen > 2000


def test_form_without_sequences():
    assert attn_plans.fwd("bf16", 0, 0, 0, 8, 2)["form"] == "halves"
    assert gdn.gdn_attn_fwd_workspace_size(0, 0, 0, 8, 2, 64, torch.bfloat16) == 0


@pytest.mark.parametrize("N,Hq,Hk,D,page,width", [(1024, 32, 32, 128, 64, 100), (4096, 64, 64, 128, 64, 100), (100_000, 64, 1, 128, 64, 100),
                                                  (1, 32, 8, 128, 64, 2048)])
def test_step_workspace_grows_with_what_is_shared(N, Hq, Hk, D, page, width):
    """512 to 768 workgroups share the tiles, a sequence is cut into fewer than twice its part of
    them, and a piece has rows for 16 heads; and four bytes a sequence."""
    assert gdn.gdn_attn_step_workspace_size(N, Hq, Hk, D, page, width) <= 2 * 768 * 16 * (D + 1) * 4 + 4 * (N + 1) + 512
