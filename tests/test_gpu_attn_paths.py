"""The paths that calls of the grouped-attention kernels take by their sizes, against the fp64
oracle (tolerances as in test_gpu_attn.py): every form of the forward and the backward, many
sequences, offsets beyond 2^31 values, other streams and devices, and calls side by side."""
import math

import numpy as np
import pytest
import torch

import attn_plans
import gated_deltanet_layer_amd as gdn
import test_gpu_attn
from oracle import attention as ref
from test_gpu_attn import (DEV, DT, _append_args, _cache, _check_bwd, _check_fwd, _check_step, _cu, _dev, _live, _on, _packed,
                           _say, _values)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form,lq,lk,Hq,Hk,D,dt", [
    ("whole", [600] * 5, None, 16, 4, 64, "bf16"), ("halves", [65, 700, 1, 64, 128], None, 4, 1, 64, "bf16"),
    ("halves", [200, 3], [450, 64], 6, 2, 128, "bf16"), ("halves", [70, 33], None, 4, 4, 128, "fp32"), ("shares", [4700, 31], None, 2, 1, 128, "bf16"),
    ("shares", [60, 61], [3000, 1900], 10, 2, 64, "bf16"), ("shares", [1900, 0, 100], None, 6, 2, 64, "fp32"),
    ("shares", [3200], [2500], 4, 2, 64, "bf16"), ("shares", [2400, 200], None, 17, 1, 64, "bf16")])
def test_forms_of_the_forward(form, lq, lk, Hq, Hk, D, dt):
    _say(f"{form} lq {lq} lk {lk} Hq{Hq} Hk{Hk} D{D} {dt}")
    assert attn_plans.fwd(dt, len(lq), sum(lq), sum(lk or lq), Hq, Hk)["form"] == form
    d = _packed(lq, lk, Hq, Hk, D, dt, seed=41)
    o, lse = _check_fwd(d, dt)
    x = _on(d)
    o2, lse2 = gdn.attn_fwd(x["q"], x["k"], x["v"], x["cu_q"], x["cu_k"])
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


@pytest.mark.parametrize("cut,lq,lk,Hq,Hk,D,dt", [
    (True, [1100], None, 4, 2, 64, "bf16"), (True, [300, 40], [1500, 2000], 6, 2, 128, "bf16"), (False, [300] * 8, None, 4, 1, 64, "bf16"),
    (True, [333, 0, 100], None, 3, 3, 64, "fp32"), (True, [700, 650], [1200, 10], 4, 2, 64, "bf16"), (False, [900] * 4, None, 32, 8, 64, "bf16"),
    # a longer sequence among those that the rule is made for: the last piece has the rest
    (True, [2600, 1, 1, 1], None, 4, 2, 64, "bf16")])
def test_forms_of_the_backward(cut, lq, lk, Hq, Hk, D, dt):
    _say(f"cut {cut} lq {lq} lk {lk} Hq{Hq} Hk{Hk} D{D} {dt}")
    assert (attn_plans.bwd(dt, len(lq), sum(lq), sum(lk or lq), Hq, Hk)["kp"] > 1) == cut
    _check_bwd(_packed(lq, lk, Hq, Hk, D, dt, seed=43), dt)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_many_sequences(dt):
    """More than 64, and more than 64^2, sequences: empty ones, single tokens, and longer ones."""
    for B in (65, 700, 4200):
        lens = [(37 * i * i) % 11 if i % 50 else 90 for i in range(B)]
        if B == 4200:
            lens = [n // 8 for n in lens]
        _say(f"{B} sequences, {sum(lens)} tokens, {dt}")
        d = _packed(lens, None, 4, 2, 64, dt, seed=B, before=3, behind=5)
        _check_fwd(d, dt)
        _check_bwd(d, dt)


def test_many_sequences_appended():
    B, Hk, D, page = 4200, 2, 64, 16
    lens = torch.tensor([(53 * i) % 33 for i in range(B)], dtype=torch.int32)
    new = [min(int(n), (7 * i) % 20) for i, n in enumerate(lens)]
    c = _live(_cache(B, 3, page, Hk, D, seed=3))
    kv = torch.randn(sum(new), 2 * Hk, D, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16)
    x, cu = _dev(c), _cu(new)
    kvd = kv.to(DEV)
    gdn.attn_append_(kvd[:, :Hk], kvd[:, Hk:], *_append_args(x), lens.to(DEV), cu=cu.to(DEV))
    torch.cuda.synchronize()
    want = _values(c)
    ref.append(kv[:, :Hk], kv[:, Hk:], cu, *want, c["table"], lens)
    for a, b in zip(_values({k: v.cpu() for k, v in x.items()}), want):
        assert np.array_equal(a, b)


def test_no_queries_and_no_keys():
    e = lambda *s: torch.zeros(*s, device=DEV)  # noqa: E731
    cu0, cu5 = torch.zeros(3, dtype=torch.int32, device=DEV), torch.tensor([0, 2, 5], dtype=torch.int32, device=DEV)
    o, lse = gdn.attn_fwd(e(0, 4, 64), e(5, 2, 64), e(5, 2, 64), cu0, cu5)
    g = gdn.attn_bwd(e(0, 4, 64), e(5, 2, 64), e(5, 2, 64), o, lse, o, cu0, cu5)
    assert (g["dk"] == 0).all() and (g["dv"] == 0).all()
    o, lse = gdn.attn_fwd(e(5, 4, 64), e(0, 2, 64), e(0, 2, 64), cu5, cu0)
    assert (o == 0).all() and torch.isneginf(lse).all()
    assert (gdn.attn_bwd(e(5, 4, 64), e(0, 2, 64), e(0, 2, 64), o, lse, o, cu5, cu0)["dq"] == 0).all()


def test_rows_beyond_2_31_values():
    """Packed slices of a tensor of more than 2^32 bytes: the last rows' offsets pass 31 bits."""
    Hq, Hk, D, T, step = 4, 2, 64, 2100, 1 << 20
    big = torch.empty(T, step, dtype=torch.bfloat16, device=DEV)
    small = torch.randn(T, Hq + 2 * Hk, D, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    big[:, :(Hq + 2 * Hk) * D] = small.reshape(T, -1).to(DEV)
    x = big.as_strided((T, Hq + 2 * Hk, D), (step, D, 1))
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:]
    cu = torch.tensor([0, 1900, 2100], dtype=torch.int32, device=DEV)
    c = [t.contiguous() for t in (q, k, v)]
    o, lse = gdn.attn_fwd(q, k, v, cu)
    o2, lse2 = gdn.attn_fwd(*c, cu)
    d_o = torch.randn(T, Hq, D, device=DEV).to(torch.bfloat16)
    want = gdn.attn_bwd(*c, o2, lse2, d_o, cu)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    y = big[:, 2048:].as_strided((T, Hq + 2 * Hk, D), (step, D, 1), 2048)   # gradients beside the values
    ws = torch.empty(gdn.gdn_attn_bwd_workspace_size(2, T, T, Hq, Hk, D, torch.bfloat16), dtype=torch.uint8, device=DEV)
    gdn.gdn_attn_bwd(*c, cu, None, o2, lse2, d_o, y[:, :Hq], y[:, Hq:Hq + Hk], y[:, Hq + Hk:], ws, 1 / math.sqrt(D))
    for n, t in (("dq", y[:, :Hq]), ("dk", y[:, Hq:Hq + Hk]), ("dv", y[:, Hq + Hk:])):
        assert torch.equal(t, want[n]), n
    w, inv, pos = torch.ones(D, device=DEV), torch.ones(D // 2, device=DEV), torch.arange(T, dtype=torch.int32, device=DEV)
    for a, b in zip(gdn.attn_prologue(q, k, w, w, inv, pos), gdn.attn_prologue(c[0], c[1], w, w, inv, pos)):
        assert torch.equal(a, b)


def test_cache_beyond_2_31_bytes():
    """Pages whose bytes lie behind the first 2^31 of each cache."""
    Hk, D, page, pages = 8, 128, 64, 36000
    c = dict(k_cache=torch.zeros(pages, Hk, page, D, dtype=torch.uint8, device=DEV),
             v_cache=torch.zeros(pages, Hk, page // 16, D, 16, dtype=torch.uint8, device=DEV),
             k_scale=torch.zeros(pages, Hk, page // 16, device=DEV), v_scale=torch.zeros(pages, Hk, page // 16, device=DEV))
    assert c["k_cache"].numel() > 1 << 31
    far, near = (torch.tensor(t, dtype=torch.int32, device=DEV) for t in ([[pages - 1, 35000], [34999, 20000]], [[0, 1], [2, 3]]))
    lens, cu = torch.tensor([100, 77], dtype=torch.int32, device=DEV), torch.tensor([0, 100, 177], dtype=torch.int32, device=DEV)
    g = torch.Generator(device=DEV).manual_seed(1)
    kv = torch.randn(177, 2 * Hk, D, generator=g, device=DEV).to(torch.bfloat16)
    q = torch.randn(2, 32, D, generator=g, device=DEV).to(torch.bfloat16)
    out = []
    for table in (far, near):
        gdn.attn_append_(kv[:, :Hk], kv[:, Hk:], c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"], table, lens, cu=cu)
        out.append(gdn.attn_step(q, c["k_cache"], c["v_cache"], c["k_scale"], c["v_scale"], table, lens))
    assert torch.equal(*out)
    for n in c:
        assert torch.equal(c[n][far.long()], c[n][near.long()]), n
    ro, _ = ref.forward(q[0:1].cpu(), kv[:100, :Hk].cpu(), kv[:100, Hk:].cpu(), [0, 1], [0, 100], D ** -0.5)
    assert np.abs(out[0][0].double().cpu().numpy() - ro[0]).max() < 0.1 * np.abs(ro).max()   # the cache's 8 bits


def test_calls_side_by_side():
    """Two calls at once on two streams, each with its own workspace, give what they give alone."""
    ds = [_on(_packed([700, 33], None, 4, 2, 64, "bf16", seed=s)) for s in (1, 2)]
    alone = []
    for d in ds:
        o, lse = gdn.attn_fwd(d["q"], d["k"], d["v"], d["cu_q"])
        alone.append((o, lse, gdn.attn_bwd(d["q"], d["k"], d["v"], o, lse, d["d_o"], d["cu_q"])))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ds]
    for _ in range(3):
        got = []
        for d, s in zip(ds, streams):
            o, lse = gdn.attn_fwd(d["q"], d["k"], d["v"], d["cu_q"], stream=s)
            got.append((o, lse, gdn.attn_bwd(d["q"], d["k"], d["v"], o, lse, d["d_o"], d["cu_q"], stream=s)))
        torch.cuda.synchronize()
        for (o, lse, g), (o2, lse2, g2) in zip(got, alone):
            assert torch.equal(o, o2) and torch.equal(lse, lse2) and all(torch.equal(g[n], g2[n]) for n in g)


def test_outputs_stay_inside_their_buffers():
    """Guards in front of and behind every output and workspace."""
    lq, Hq, Hk, D, dt = [130, 1, 77], 6, 2, 64, torch.bfloat16
    d = _on(_packed(lq, None, Hq, Hk, D, "bf16", seed=3))
    T = sum(lq)
    guards = []

    def guarded(n, dtype):
        size = torch.empty(0, dtype=dtype).element_size()
        t = torch.full((n * size + 2048,), 0x5a, dtype=torch.uint8, device=DEV)
        guards.append((t, n * size))
        return t[1024:1024 + n * size].view(dtype)

    o, lse = guarded(T * Hq * D, dt).view(T, Hq, D), guarded(T * Hq, torch.float32).view(T, Hq)
    gdn.gdn_attn_fwd(d["q"], d["k"], d["v"], d["cu_q"], None, o, lse, None, 0.125)
    g = [guarded(T * H * D, dt).view(T, H, D) for H in (Hq, Hk, Hk)]
    ws = guarded(gdn.gdn_attn_bwd_workspace_size(3, T, T, Hq, Hk, D, dt), torch.uint8)
    gdn.gdn_attn_bwd(d["q"], d["k"], d["v"], d["cu_q"], None, o, lse, d["d_o"].contiguous(), *g, ws, 0.125)
    w, pos, inv = torch.ones(D, device=DEV), torch.arange(T, dtype=torch.int32, device=DEV), torch.ones(8, device=DEV)
    qk = [guarded(T * H * D, dt).view(T, H, D) for H in (Hq, Hk)]
    gdn.gdn_attn_prologue(d["q"], d["k"], w, w, inv, pos, *qk, 1e-6)
    pw = guarded(gdn.gdn_attn_prologue_bwd_workspace_size(T, Hq, Hk, D, 16, dt), torch.uint8)
    gdn.gdn_attn_prologue_bwd(d["q"], d["k"], w, w, inv, pos, *qk, *[guarded(T * H * D, dt).view(T, H, D) for H in (Hq, Hk)],
                              guarded(D, torch.float32), guarded(D, torch.float32), pw, 1e-6)
    N, width, page = 3, 80, 16
    c = _live(_cache(N, width, page, Hk, D))
    kc = guarded(c["k_cache"].numel(), torch.uint8).view(c["k_cache"].shape).copy_(c["k_cache"])
    vc = guarded(c["v_cache"].numel(), torch.uint8).view(c["v_cache"].shape).copy_(c["v_cache"])
    ks, vs = (guarded(c[n].numel(), torch.float32).view(c[n].shape).copy_(c[n]) for n in ("k_scale", "v_scale"))
    table, lens = c["table"].to(DEV), torch.tensor([1100, 1, 600], dtype=torch.int32, device=DEV)
    gdn.gdn_attn_append(d["k"], d["v"], d["cu_q"], kc, vc, ks, vs, table, torch.tensor([1280, 1, 80], dtype=torch.int32, device=DEV))
    sw = guarded(gdn.gdn_attn_step_workspace_size(N, Hq, Hk, D, page, width), torch.uint8)
    gdn.gdn_attn_step(d["q"][:N].contiguous(), kc, vc, ks, vs, table, lens, guarded(N * Hq * D, dt).view(N, Hq, D),
                      guarded(N * Hq, torch.float32).view(N, Hq), sw, 0.125)
    torch.cuda.synchronize()
    for i, (t, n) in enumerate(guards):
        assert (t[:1024] == 0x5a).all() and (t[1024 + n:] == 0x5a).all(), i


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
def test_step_over_long_and_many(dt):
    """One long sequence in many pieces, and more sequences than workgroups to share."""
    g = torch.Generator().manual_seed(5)
    for N, width, lens, Hq, Hk, page in ((1, 1100, [17000], 8, 2, 16), (300, 70, [(91 * i) % 1121 for i in range(300)], 4, 1, 16)):
        _say(f"step N{N} {dt}")
        c = _live(_cache(N, width, page, Hk, 64, seed=N))
        q = (torch.randn(N, Hq, 64, generator=g) * 0.2).to(DT[dt])
        _check_step(c, q, lens, dt)


def test_prologue_of_equal_rows_is_equal():
    """Rows with the same values and positions give the same bits, wherever they stand: in calls
    of either form, alone or among others."""
    g = torch.Generator().manual_seed(9)
    x = torch.randn(1, 6, 64, generator=g).to(torch.bfloat16).to(DEV)
    w, inv = torch.randn(64, generator=g).to(DEV), torch.rand(32, generator=g).to(DEV)
    one = gdn.attn_prologue(x[:, :4], x[:, 4:], w, w, inv, torch.tensor([77777], dtype=torch.int32, device=DEV))
    for T in (5, 5000):
        many = gdn.attn_prologue(x.expand(T, -1, -1).contiguous()[:, :4], x.expand(T, -1, -1).contiguous()[:, 4:], w, w, inv,
                                 torch.full((T,), 77777, dtype=torch.int32, device=DEV))
        for a, b in zip(one, many):
            assert (a == b).all()


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("N,Hq,Hk,D", [(257, 8, 2, 128), (9, 34, 2, 64)])
def test_step_joined_by_lanes_and_by_workgroups(N, Hq, Hk, D, dt):
    """Sequences in many pieces beside whole and empty ones, with more and fewer rows than are
    joined by a workgroup each."""
    _say(f"step joined N{N} Hq{Hq} Hk{Hk} D{D} {dt}")
    g = torch.Generator().manual_seed(N)
    c = _live(_cache(7, 40, 32, Hk, D, seed=N))
    c["table"] = torch.randint(0, 280, (N, 160), generator=g).to(torch.int32)   # pages shared
    lens = [5120 if i in (3, N - 1) else 1500 if i == 5 else (37 * i) % 130 for i in range(N)]
    q = (torch.randn(N, Hq, D, generator=g) * 0.2).to(DT[dt])
    _check_step(c, q, lens, dt)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("lq,lk,Hq,Hk,D", [([3], [9000], 8, 2, 64), ([1, 40, 0], [6000, 7, 900], 12, 1, 128),
                                           ([1, 40, 0], [6000, 7, 1900], 12, 1, 128), ([130, 2], [5000, 4000], 17, 1, 64)])
def test_few_rows_over_long_sequences(lq, lk, Hq, Hk, D, dt):
    """A few tokens, some of which see nothing, behind long sequences: rows of many parts."""
    _say(f"few rows lq {lq} lk {lk} Hq{Hq} Hk{Hk} D{D} {dt}")
    assert attn_plans.fwd(dt, len(lq), sum(lq), sum(lk), Hq, Hk)["form"] == "shares"
    _check_fwd(_packed(lq, lk, Hq, Hk, D, dt, seed=31), dt)


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("T,Hq,Hk,D", [(130, 32, 3, 128), (1024, 32, 1, 128), (1025, 64, 2, 64), (128, 3, 2, 64), (129, 3, 2, 64)])
def test_prologue_of_one_and_of_four_tokens_a_workgroup(T, Hq, Hk, D, dt):
    test_gpu_attn.test_prologue(T, Hq, Hk, D, D, 1000, dt)
