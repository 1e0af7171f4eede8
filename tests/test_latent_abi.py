"""gdn_latent_*: refusals on the host (CPU only: every call here fails a check or is
an empty no-op, so no kernel is launched)."""
import ctypes
import os

import pytest

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


def _fwd(L, **kw):
    a = dict(q=_p(0), kv=_p(1), kr=_p(2), lens=_p(3), o=_p(4), lse=_p(5), ws=_p(6), nb=BIG, B=2, Tq=100, Tk=300,
             H=3, dn=128, dr=64, dv=128, scale=0.1, dtype=1)
    a.update(kw)
    return L.gdn_latent_fwd(*[a[k] for k in ("q", "kv", "kr", "lens", "o", "lse", "ws", "nb", "B", "Tq", "Tk", "H",
                                             "dn", "dr", "dv", "scale", "dtype")], None)


def _bwd(L, **kw):
    a = dict(q=_p(0), kv=_p(1), kr=_p(2), lens=_p(3), o=_p(4), lse=_p(5), d_o=_p(6), dq=_p(7), dkv=_p(8), dkr=_p(9),
             ws=_p(10), nb=BIG, B=2, Tq=100, Tk=300, H=3, dn=128, dr=64, dv=128, scale=0.1, dtype=1)
    a.update(kw)
    return L.gdn_latent_bwd(*[a[k] for k in ("q", "kv", "kr", "lens", "o", "lse", "d_o", "dq", "dkv", "dkr", "ws", "nb",
                                             "B", "Tq", "Tk", "H", "dn", "dr", "dv", "scale", "dtype")], None)


def _steps(L, **kw):
    a = dict(q=_p(0), draft=_p(1), tree=_p(2), cache=_p(3), table=_p(4), lens=_p(5), o=_p(6), lse=_p(7), ws=_p(8),
             nb=BIG, N=4, M=5, H=3, r=512, dr=64, pages=40, page=16, width=9, scale=0.1, dtype=1)
    a.update(kw)
    return L.gdn_latent_steps(*[a[k] for k in ("q", "draft", "tree", "cache", "table", "lens", "o", "lse", "ws", "nb",
                                               "N", "M", "H", "r", "dr", "pages", "page", "width", "scale", "dtype")], None)


def _step(L, **kw):
    a = dict(q=_p(0), cache=_p(3), table=_p(4), lens=_p(5), o=_p(6), lse=_p(7), ws=_p(8),
             nb=BIG, N=4, H=3, r=512, dr=64, pages=40, page=16, width=9, scale=0.1, dtype=1)
    a.update(kw)
    return L.gdn_latent_step(*[a[k] for k in ("q", "cache", "table", "lens", "o", "lse", "ws", "nb", "N", "H", "r",
                                              "dr", "pages", "page", "width", "scale", "dtype")], None)


SIZES = [dict(dtype=2), dict(dtype=-1), dict(B=-1), dict(Tq=-1), dict(Tk=-1), dict(H=-1), dict(dn=0), dict(dv=-64),
         dict(dr=0), dict(Tq=301), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
         dict(scale=float("inf")), dict(B=1 << 30, Tk=1 << 30, H=1 << 30)]


@pytest.mark.parametrize("kw", SIZES + [
    dict(q=None), dict(kv=None), dict(kr=None), dict(o=None), dict(q=_p(0) + 8), dict(kv=_p(1) + 4), dict(kr=_p(2) + 2),
    dict(o=_p(4) + 8), dict(lens=_p(3) + 2), dict(lse=_p(5) + 1), dict(ws=_p(6) + 128),
    dict(o=_p(0)), dict(o=_p(1) + 64), dict(lse=_p(2)), dict(o=_p(3)), dict(lse=_p(4) + 16), dict(o=_p(5) - 16)])
def test_fwd_rejects_invalid(L, kw):
    assert _fwd(L, **kw) == gdn.GDN_EINVAL


@pytest.mark.parametrize("kw", SIZES + [
    dict(q=None), dict(kv=None), dict(kr=None), dict(o=None), dict(lse=None), dict(d_o=None), dict(dq=None),
    dict(dkv=None), dict(dkr=None), dict(ws=None), dict(nb=100), dict(ws=_p(10) + 64), dict(dq=_p(7) + 8),
    dict(d_o=_p(6) + 2), dict(lse=_p(5) + 2), dict(dq=_p(0)), dict(dkv=_p(1)), dict(dkr=_p(2)), dict(dq=_p(8) + 16),
    dict(dkv=_p(6)), dict(ws=_p(7)), dict(ws=_p(0)), dict(dkr=_p(3))])
def test_bwd_rejects_invalid(L, kw):
    assert _bwd(L, **kw) == gdn.GDN_EINVAL


@pytest.mark.parametrize("call", [_fwd, _bwd])
@pytest.mark.parametrize("kw", [dict(dn=96), dict(dn=256), dict(dv=32), dict(dr=32), dict(dr=128), dict(B=1 << 14, H=1 << 14),
                                dict(B=1 << 20, Tk=1 << 10, Tq=1, H=1)])
def test_expanded_unsupported(L, call, kw):
    assert call(L, **kw) == gdn.GDN_ENOTSUP


@pytest.mark.parametrize("kw", [dict(B=0), dict(Tq=0), dict(Tq=0, Tk=0), dict(H=0),
                                dict(B=0, q=None, kv=None, kr=None, o=None, lse=None, ws=None)])
def test_fwd_empty_is_a_noop(L, kw):
    assert _fwd(L, **kw) == gdn.GDN_OK


@pytest.mark.parametrize("kw", [dict(B=0), dict(Tq=0, Tk=0)])
def test_bwd_empty_is_a_noop(L, kw):
    assert _bwd(L, **kw) == gdn.GDN_OK


BOTH = [dict(dtype=3), dict(N=-1), dict(H=-1), dict(r=0), dict(dr=-1), dict(pages=-1), dict(page=0), dict(width=-1),
        dict(scale=0.0), dict(scale=float("nan")), dict(q=None), dict(cache=None), dict(table=None), dict(lens=None),
        dict(o=None), dict(ws=None), dict(nb=1000), dict(q=_p(0) + 4), dict(cache=_p(3) + 8), dict(table=_p(4) + 2),
        dict(lens=_p(5) + 1), dict(o=_p(6) + 2), dict(lse=_p(7) + 2), dict(ws=_p(8) + 16), dict(o=_p(0)),
        dict(o=_p(3) + 16), dict(lse=_p(6)), dict(ws=_p(3)), dict(o=_p(4)), dict(lse=_p(5))]
WIDE = [dict(r=128), dict(r=1024), dict(dr=32), dict(pages=1 << 20, page=1 << 12, width=1), dict(N=1 << 16, width=1 << 16),
        dict(page=1 << 16, pages=1, width=1 << 15), dict(N=1 << 24, H=4), dict(H=1 << 21)]


@pytest.mark.parametrize("call", [_step, _steps])
@pytest.mark.parametrize("kw", BOTH)
def test_absorbed_rejects_invalid(L, call, kw):
    assert call(L, **kw) == gdn.GDN_EINVAL


@pytest.mark.parametrize("kw", [dict(M=-1), dict(draft=None), dict(draft=_p(1) + 8), dict(tree=_p(2) + 4),
                                dict(o=_p(1)), dict(lse=_p(2))])
def test_steps_rejects_invalid(L, kw):
    assert _steps(L, **kw) == gdn.GDN_EINVAL


@pytest.mark.parametrize("call", [_step, _steps])
@pytest.mark.parametrize("kw", WIDE)
def test_absorbed_unsupported(L, call, kw):
    assert call(L, nb=1 << 35, **kw) == gdn.GDN_ENOTSUP


def test_fwd_in_pieces_needs_its_workspace(L):
    n = ctypes.c_size_t(0)
    a = dict(B=1, Tq=3, Tk=4096, H=2)
    assert L.gdn_latent_fwd_workspace_size(1, 3, 4096, 2, 128, 64, 128, 1, ctypes.byref(n)) == gdn.GDN_OK and n.value > 0
    assert _fwd(L, ws=None, **a) == gdn.GDN_EINVAL
    assert _fwd(L, nb=n.value - 1, **a) == gdn.GDN_EINVAL
    assert _fwd(L, ws=_p(4), **a) == gdn.GDN_EINVAL   # over o


def test_rows_too_wide_for_32_bit_offsets_are_refused(L):
    assert _fwd(L, B=1, Tq=1, Tk=1, H=(1 << 15) + 1) == gdn.GDN_ENOTSUP
    assert _bwd(L, B=1, Tq=1, Tk=1, H=(1 << 15) + 1) == gdn.GDN_ENOTSUP


@pytest.mark.parametrize("call", [_fwd, _bwd, _step, _steps])
def test_scale_beyond_base_two_is_refused(L, call):
    """scale log2(e) must be a number: a score of 0 would otherwise be 0 times infinity."""
    top = 3.4028234663852886e38   # the largest float
    for scale in (top, top * 0.7):
        assert call(L, scale=scale) == gdn.GDN_EINVAL
    if call is _fwd:
        assert call(L, scale=top * 0.69, B=0) == gdn.GDN_OK
    elif call is not _bwd:
        assert call(L, scale=top * 0.69, N=0) == gdn.GDN_OK


@pytest.mark.parametrize("dtype,keys", [(0, 64), (1, 128)])
def test_bwd_grid_of_512_threads(L, dtype, keys):
    """The key-owning kernel's workgroups times 512 threads stay below 2^32."""
    n = ctypes.c_size_t(0)
    ask = lambda **a: L.gdn_latent_bwd_workspace_size(a["B"], 1, a["Tk"], a["H"], 64, 64, 64, dtype, ctypes.byref(n))  # noqa: E731
    for Tk, H in ((1, 1 << 15), (keys, 1 << 15), (keys + 1, 1 << 14)):
        assert ask(B=256, Tk=Tk, H=H) == gdn.GDN_ENOTSUP
        assert _bwd(L, B=256, Tq=1, Tk=Tk, H=H, dn=64, dv=64, dtype=dtype) == gdn.GDN_ENOTSUP
        assert ask(B=255, Tk=Tk, H=H) == gdn.GDN_OK
    assert L.gdn_latent_fwd_workspace_size(256, 1, 1, 1 << 15, 64, 64, 64, dtype, ctypes.byref(n)) == gdn.GDN_OK


def test_steps_takes_at_most_64_drafts(L):
    assert _steps(L, M=65) == gdn.GDN_ENOTSUP


@pytest.mark.parametrize("kw", [dict(N=0), dict(H=0), dict(N=0, q=None, cache=None, table=None, lens=None, o=None, ws=None)])
def test_absorbed_empty_is_a_noop(L, kw):
    assert _step(L, **kw) == gdn.GDN_OK
    assert _steps(L, **kw) == gdn.GDN_OK
    assert _steps(L, M=0, draft=None) == gdn.GDN_OK


def test_workspace_queries(L):
    n = ctypes.c_size_t(7)
    assert L.gdn_latent_fwd_workspace_size(1, 8, 8, 4, 128, 64, 128, 1, None) == gdn.GDN_EINVAL
    assert L.gdn_latent_bwd_workspace_size(1, 8, 8, 4, 128, 64, 96, 1, ctypes.byref(n)) == gdn.GDN_ENOTSUP
    assert L.gdn_latent_steps_workspace_size(1, 65, 4, 512, 64, 1, ctypes.byref(n)) == gdn.GDN_ENOTSUP
    assert n.value == 7   # a refused query writes nothing
    import torch
    assert gdn.gdn_latent_bwd_workspace_size(2, 100, 300, 3, 128, 64, 128, torch.bfloat16) > 0
    assert gdn.gdn_latent_steps_workspace_size(4, 1, 3, 512, 64, torch.float32) > 0
    assert gdn.gdn_latent_steps_workspace_size(0, 1, 3, 512, 64, torch.bfloat16) == 0
    with pytest.raises(TypeError):
        gdn.gdn_latent_bwd_workspace_size(2, 100, 300, 3, 128, 64, 128, torch.float16)


def test_binding_refuses_cpu_tensors_and_wrong_shapes():
    import torch
    q, kv, kr = torch.zeros(1, 4, 2, 192), torch.zeros(1, 4, 2, 256), torch.zeros(1, 4, 64)
    with pytest.raises(ValueError, match="GPU"):
        gdn.latent_fwd(q, kv, kr)
    with pytest.raises(ValueError, match="value part"):
        gdn.latent_fwd(q, kv[..., :128], kr)
    with pytest.raises(ValueError, match="contiguous"):
        gdn.latent_fwd(q, kv.transpose(1, 2).contiguous().transpose(1, 2), kr)
    with pytest.raises(TypeError):
        gdn.latent_fwd(q, kv.bfloat16(), kr)
    with pytest.raises(TypeError):
        gdn.latent_fwd(q, kv, kr, lens=torch.zeros(1, dtype=torch.int64))
    c, t, n = torch.zeros(3, 4, 576), torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError, match="shape"):
        gdn.latent_step(torch.zeros(3, 2, 576), c, t, n, 0.1)
    with pytest.raises(TypeError):
        gdn.latent_steps(torch.zeros(2, 3, 2, 576), torch.zeros(2, 3, 576), torch.zeros(2, 3, dtype=torch.int32), c, t, n, 0.1)
    with pytest.raises(ValueError, match="draft"):
        gdn.latent_steps(torch.zeros(2, 3, 2, 576), None, None, c, t, n, 0.1)
