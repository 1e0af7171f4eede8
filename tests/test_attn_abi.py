"""gdn_attn_*: refusals on the host (CPU only: every call here fails a check or is an empty
no-op, so no kernel is launched), and those of the Python binding."""
import ctypes
import os

import pytest
import torch

import gated_deltanet_layer_amd as gdn

BASE, SEP = 1 << 56, 1 << 48
BIG = 1 << 34


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(gdn.LIB_PATH):
        from gated_deltanet_layer_amd import build
        build.build()
    return gdn.lib()


def _p(i):
    return BASE + i * SEP


def _call(L, name, order, a, kw):
    a = dict(a, **kw)
    assert set(a) == set(order), set(a) ^ set(order)
    return getattr(L, name)(*[a[k] for k in order], None)


PRO = dict(qr=_p(0), kr=_p(1), wq=_p(2), wk=_p(3), inv=_p(4), pos=_p(5), q=_p(6), k=_p(7), T=100, Hq=4, Hk=2, D=64, R=32, qs=512, ks=512,
           eps=1e-6, dtype=1)


def _pro(L, **kw):
    return _call(L, "gdn_attn_prologue", "qr kr wq wk inv pos q k T Hq Hk D R qs ks eps dtype".split(), PRO, kw)


def _pro_bwd(L, **kw):
    a = dict({k: v for k, v in PRO.items() if k not in ("q", "k")}, dq=_p(6), dk=_p(7), dqr=_p(8), dkr=_p(9), dwq=_p(10), dwk=_p(11),
             ws=_p(12), nb=BIG, dqs=max(512, kw.get("qs", 512)), dks=512)
    return _call(L, "gdn_attn_prologue_bwd",
                 "qr kr wq wk inv pos dq dk dqr dkr dwq dwk ws nb T Hq Hk D R qs ks dqs dks eps dtype".split(), a, kw)


SEQ = dict(q=_p(0), k=_p(1), v=_p(2), cuq=_p(3), cuk=_p(4), B=3, Tq=100, Tk=300, Hq=6, Hk=2, D=128, qs=768, ks=256, vs=256, scale=0.1,
           dtype=1)


def _fwd(L, **kw):
    return _call(L, "gdn_attn_fwd", "q k v cuq cuk o lse ws nb B Tq Tk Hq Hk D qs ks vs scale dtype".split(),
                 dict(SEQ, o=_p(5), lse=_p(6), ws=_p(7), nb=BIG), kw)


def _bwd(L, **kw):
    return _call(L, "gdn_attn_bwd",
                 "q k v cuq cuk o lse d_o dq dk dv ws nb B Tq Tk Hq Hk D qs ks vs dqs dks dvs scale dtype".split(),
                 dict(SEQ, o=_p(5), lse=_p(6), d_o=_p(7), dq=_p(8), dk=_p(9), dv=_p(10), ws=_p(11), nb=BIG, dqs=768, dks=256, dvs=256), kw)


CACHE = dict(kc=_p(3), vc=_p(4), ksc=_p(5), vsc=_p(6), table=_p(7), lens=_p(8), N=4, Hk=2, D=128, pages=40, page=48, width=9, dtype=1)


def _append(L, **kw):
    return _call(L, "gdn_attn_append", "k v cu kc vc ksc vsc table lens N T Hk D pages page width ks vs dtype".split(),
                 dict(CACHE, k=_p(0), v=_p(1), cu=_p(2), T=70, ks=256, vs=256), kw)


def _step(L, **kw):
    return _call(L, "gdn_attn_step", "q kc vc ksc vsc table lens o lse ws nb N Hq Hk D pages page width scale dtype".split(),
                 dict(CACHE, q=_p(0), o=_p(9), lse=_p(10), ws=_p(11), nb=BIG, Hq=6, scale=0.1, page=64, width=40), kw)


@pytest.mark.parametrize("call", [_pro, _pro_bwd])
@pytest.mark.parametrize("kw", [
    dict(dtype=2), dict(T=-1), dict(Hq=-1), dict(Hk=-2), dict(D=0), dict(R=-16), dict(R=80), dict(eps=-1e-6), dict(eps=float("nan")),
    dict(eps=float("inf")), dict(qs=248), dict(ks=127), dict(qs=513), dict(qr=None), dict(kr=None), dict(wq=None), dict(wk=None),
    dict(inv=None), dict(pos=None), dict(qr=_p(0) + 8), dict(wk=_p(3) + 4), dict(pos=_p(5) + 2), dict(inv=_p(4) + 1),
    dict(T=1 << 30, Hq=1 << 30, qs=1 << 40)])
def test_prologue_rejects_invalid(L, call, kw):
    assert call(L, **kw) == gdn.GDN_EINVAL


@pytest.mark.parametrize("kw", [dict(q=None), dict(k=None), dict(q=_p(6) + 8), dict(q=_p(0)), dict(k=_p(0) + 512), dict(q=_p(5)),
                                dict(k=_p(6) + 64), dict(q=_p(2) - 16)])
def test_prologue_rejects_outputs(L, kw):
    assert _pro(L, **kw) == gdn.GDN_EINVAL


@pytest.mark.parametrize("kw", [
    dict(dq=None), dict(dk=None), dict(dqr=None), dict(dkr=None), dict(dwq=None), dict(dwk=None), dict(ws=None), dict(nb=100),
    dict(ws=_p(12) + 64), dict(dqr=_p(8) + 8), dict(dwq=_p(10) + 2), dict(dqs=248), dict(dks=130),
    # overlaps: with inputs, with each other, rows that interleave but share bytes
    dict(dqr=_p(0)), dict(dqr=_p(6)), dict(dkr=_p(8) + 256), dict(dkr=_p(8), dks=500), dict(dwk=_p(10) + 16), dict(ws=_p(9)), dict(dwq=_p(2))])
def test_prologue_bwd_rejects_invalid(L, kw):
    assert _pro_bwd(L, **kw) == gdn.GDN_EINVAL


@pytest.mark.parametrize("call", [_pro, _pro_bwd])
@pytest.mark.parametrize("kw", [dict(D=96, R=32), dict(D=256, qs=1024), dict(R=8), dict(R=24), dict(Hq=(1 << 15) + 1, qs=(1 << 22) + 64),
                                dict(T=1 << 24), dict(qs=(1 << 21) + 8)])
def test_prologue_unsupported(L, call, kw):
    assert call(L, **kw) == gdn.GDN_ENOTSUP


@pytest.mark.parametrize("kw", [dict(T=0), dict(T=0, qr=None, kr=None, q=None, k=None, pos=None), dict(Hq=0, Hk=0)])
def test_prologue_empty_is_a_noop(L, kw):
    assert _pro(L, **kw) == gdn.GDN_OK


SEQ_BAD = [
    dict(dtype=2), dict(B=-1), dict(Tq=-1), dict(Tk=-1), dict(Hq=0), dict(Hk=0), dict(Hq=5), dict(D=-64), dict(scale=0.0), dict(scale=-1.0),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=3e38), dict(cuk=None), dict(cuq=None), dict(qs=760), dict(ks=255),
    dict(vs=129), dict(qs=770), dict(q=None), dict(k=None), dict(v=None), dict(o=None), dict(q=_p(0) + 8), dict(k=_p(1) + 2),
    dict(v=_p(2) + 4), dict(o=_p(5) + 8), dict(cuq=_p(3) + 1), dict(cuk=_p(4) + 2), dict(lse=_p(6) + 2), dict(ws=_p(7) + 128),
    dict(Tq=1 << 30, Hq=1 << 30, Hk=1 << 29, qs=1 << 40, ks=1 << 40, vs=1 << 40)]


@pytest.mark.parametrize("kw", SEQ_BAD + [
    dict(o=_p(0)), dict(o=_p(1) + 64), dict(o=_p(2)), dict(lse=_p(3)), dict(lse=_p(5) + 16), dict(o=_p(4) - 16),
    # long enough for a workspace
    dict(Tk=9000, ws=None), dict(Tk=9000, nb=1000), dict(Tk=9000, ws=_p(0))])
def test_fwd_rejects_invalid(L, kw):
    assert _fwd(L, **kw) == gdn.GDN_EINVAL


@pytest.mark.parametrize("kw", [kw for kw in SEQ_BAD if kw != dict(ws=_p(7) + 128)] + [
    dict(lse=None), dict(d_o=None), dict(dq=None), dict(dk=None), dict(dv=None), dict(ws=None), dict(nb=100), dict(ws=_p(11) + 64),
    dict(dq=_p(8) + 8), dict(d_o=_p(7) + 2), dict(dqs=760), dict(dks=100), dict(dvs=258), dict(dq=_p(0)), dict(dk=_p(1)), dict(dv=_p(2)),
    dict(dq=_p(7)), dict(dk=_p(8) + 64), dict(dv=_p(9)), dict(dv=_p(9) + 256, dks=512, dvs=320), dict(dv=_p(9) + 256, dks=320, dvs=320),
    dict(ws=_p(5)), dict(ws=_p(8)), dict(dk=_p(3))])
def test_bwd_rejects_invalid(L, kw):
    assert _bwd(L, **kw) == gdn.GDN_EINVAL


@pytest.mark.parametrize("call", [_fwd, _bwd])
@pytest.mark.parametrize("kw", [
    dict(D=96), dict(D=256, qs=1536, ks=512, vs=512, dqs=1536, dks=512, dvs=512), dict(Hq=130, qs=130 * 128, dqs=130 * 128),
    dict(Hq=1 << 15, Hk=1 << 15, qs=1 << 22, ks=1 << 22, vs=1 << 22, dqs=1 << 22, dks=1 << 22, dvs=1 << 22, Tq=1, Tk=1),
    dict(Tq=1 << 26), dict(Tk=1 << 25), dict(Tq=1 << 23, Tk=1 << 23, Hq=128, Hk=2, qs=1 << 14, dqs=1 << 14), dict(B=1 << 24),
    dict(qs=(1 << 21) + 8), dict(vs=1 << 22)])
def test_sequences_unsupported(L, call, kw):
    if call is _fwd:
        kw = {k: v for k, v in kw.items() if k not in ("dqs", "dks", "dvs")}
    assert call(L, **kw) == gdn.GDN_ENOTSUP


@pytest.mark.parametrize("kw", [dict(B=0), dict(Tq=0), dict(B=0, q=None, k=None, v=None, cuq=None, cuk=_p(4), o=None, lse=None, ws=None)])
def test_fwd_empty_is_a_noop(L, kw):
    assert _fwd(L, **kw) == gdn.GDN_OK


@pytest.mark.parametrize("kw", [dict(B=0), dict(Tq=0, Tk=0), dict(Tq=0, Tk=0, cuk=None)])
def test_bwd_empty_is_a_noop(L, kw):
    assert _bwd(L, **kw) == gdn.GDN_OK


CACHE_BAD = [
    dict(dtype=7), dict(N=-1), dict(Hk=0), dict(D=0), dict(pages=-1), dict(page=0), dict(width=-1), dict(kc=None), dict(vc=None),
    dict(ksc=None), dict(vsc=None), dict(table=None), dict(lens=None), dict(kc=_p(3) + 8), dict(vc=_p(4) + 1), dict(ksc=_p(5) + 2),
    dict(table=_p(7) + 2), dict(lens=_p(8) + 1)]
CACHE_WIDE = [dict(page=24), dict(page=1 << 19), dict(pages=1 << 24, page=1 << 12, width=1), dict(N=1 << 16, width=1 << 16),
              dict(page=1 << 16, pages=1, width=1 << 15), dict(N=1 << 22, width=1)]


@pytest.mark.parametrize("kw", CACHE_BAD + [
    dict(T=-1), dict(cu=None), dict(k=None), dict(v=None), dict(k=_p(0) + 8), dict(cu=_p(2) + 2), dict(ks=248), dict(vs=257),
    dict(kc=_p(0)), dict(vc=_p(3) + 16), dict(ksc=_p(4)), dict(vsc=_p(5) + 4), dict(kc=_p(7)), dict(vsc=_p(8))])
def test_append_rejects_invalid(L, kw):
    assert _append(L, **kw) == gdn.GDN_EINVAL


@pytest.mark.parametrize("kw", CACHE_WIDE + [dict(D=256, ks=512, vs=512), dict(T=1 << 28), dict(ks=(1 << 21) + 8)])
def test_append_unsupported(L, kw):
    assert _append(L, **kw) == gdn.GDN_ENOTSUP


@pytest.mark.parametrize("kw", [dict(N=0, T=0), dict(T=0), dict(pages=0), dict(width=0), dict(N=0, T=0, cu=None)])
def test_append_empty_is_a_noop(L, kw):
    assert _append(L, **kw) == gdn.GDN_OK


@pytest.mark.parametrize("kw", CACHE_BAD + [
    dict(Hq=0), dict(Hq=5), dict(scale=0.0), dict(scale=float("nan")), dict(q=None), dict(o=None), dict(ws=None), dict(nb=1000),
    dict(q=_p(0) + 4), dict(o=_p(9) + 2), dict(lse=_p(10) + 2), dict(ws=_p(11) + 16), dict(o=_p(0)), dict(o=_p(3) + 16), dict(lse=_p(9)),
    dict(ws=_p(3)), dict(o=_p(7)), dict(lse=_p(5))])
def test_step_rejects_invalid(L, kw):
    assert _step(L, **kw) == gdn.GDN_EINVAL


@pytest.mark.parametrize("kw", CACHE_WIDE + [dict(D=32), dict(Hq=130), dict(N=1 << 18, width=1, Hq=32, Hk=16)])
def test_step_unsupported(L, kw):
    assert _step(L, **kw) == gdn.GDN_ENOTSUP


def test_step_without_sequences_is_a_noop(L):
    assert _step(L, N=0) == gdn.GDN_OK


def test_slices_of_one_tensor_do_not_overlap(L):
    """Equal steps, rows that miss each other: as good as apart; checked by what comes next (an
    unsupported stride), since a call that passes would be enqueued."""
    wide = (1 << 21) + 16
    assert _bwd(L, dk=_p(9), dv=_p(9) + 512, dks=wide, dvs=wide) == gdn.GDN_ENOTSUP
    assert _bwd(L, dk=_p(9) + 512, dv=_p(9), dks=wide, dvs=wide) == gdn.GDN_ENOTSUP
    assert _bwd(L, dk=_p(9), dv=_p(9) + 496, dks=wide, dvs=wide) == gdn.GDN_EINVAL
    assert _bwd(L, dk=_p(9), dv=_p(9) + wide * 2 + 512, dks=wide, dvs=wide) == gdn.GDN_ENOTSUP


@pytest.mark.parametrize("name,args", [
    ("gdn_attn_prologue_bwd_workspace_size", (100, 4, 2, 64, 32, 1)), ("gdn_attn_fwd_workspace_size", (1, 64, 9000, 8, 2, 128, 1)),
    ("gdn_attn_bwd_workspace_size", (3, 100, 100, 8, 2, 64, 0)), ("gdn_attn_step_workspace_size", (4, 8, 2, 128, 64, 100))])
def test_workspace_queries(L, name, args):
    n = ctypes.c_size_t(0)
    f = getattr(L, name)
    assert f(*args, ctypes.byref(n)) == gdn.GDN_OK and n.value > 0
    assert f(*args, None) == gdn.GDN_EINVAL
    assert f(-1, *args[1:], ctypes.byref(n)) == gdn.GDN_EINVAL


def test_workspaces_that_are_not_needed(L):
    assert gdn.gdn_attn_fwd_workspace_size(1, 100, 100, 4, 4, 64, torch.bfloat16) == 0
    assert gdn.gdn_attn_step_workspace_size(4, 8, 2, 128, 64, 16) == 0
    assert gdn.gdn_attn_step_workspace_size(0, 8, 2, 128, 64, 100) == 0
    assert gdn.gdn_attn_bwd_workspace_size(0, 0, 0, 4, 4, 64, torch.float32) == 0


def test_binding_wants_a_gpu():
    x = torch.zeros(3, 2, 64)
    w, cu = torch.ones(64), torch.tensor([0, 3], dtype=torch.int32)
    for call in (lambda: gdn.attn_prologue(x, x, w, w, None, None), lambda: gdn.attn_fwd(x, x, x, cu),
                 lambda: gdn.attn_append_(x, x, x, x, x, x, cu, cu), lambda: gdn.attn_step(x, x, x, x, x, cu, cu)):
        with pytest.raises(ValueError, match="GPU"):
            call()


def test_binding_wants_a_known_dtype():
    x = torch.zeros(3, 2, 64, dtype=torch.float16)
    with pytest.raises(TypeError):
        gdn.attn_fwd(x, x, x, torch.tensor([0, 3], dtype=torch.int32))
