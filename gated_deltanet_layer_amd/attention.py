"""Attention of grouped heads: the binding of the ``gdn_attn_*`` entry points.

Low-level calls (outputs and workspace given, as in the C ABI):
    gdn_attn_prologue(q_raw, k_raw, w_q, w_k, inv_freq, pos, q, k, eps)
    gdn_attn_prologue_bwd(q_raw, k_raw, w_q, w_k, inv_freq, pos, d_q, d_k, dq_raw, dk_raw,
                          dw_q, dw_k, workspace, eps)
    gdn_attn_fwd(q, k, v, cu_q, cu_k, o, lse, workspace, scale)
    gdn_attn_bwd(q, k, v, cu_q, cu_k, o, lse, d_o, dq, dk, dv, workspace, scale)
    gdn_attn_append(k, v, cu, k_cache, v_cache, k_scale, v_scale, table, lens)
    gdn_attn_step(q, k_cache, v_cache, k_scale, v_scale, table, lens, o, lse, workspace, scale)
and conveniences that allocate: attn_prologue, attn_prologue_bwd, attn_fwd, attn_bwd,
attn_append_ (which writes into the cache that it is given), attn_step.

Tokens are packed: q [T, Hq, D], k and v [T, Hk, D].  q_raw, k_raw, q, k and v, and the
gradients dq_raw, dk_raw, dq, dk and dv, may be slices of a larger tensor along the heads
(the heads of a token next to each other, any step from token to token that is a multiple
of 16 bytes).  The caches are [pages, Hk, page, D] (keys) and [pages, Hk, page / 16, D, 16]
(values), of torch.float8_e4m3fn or uint8.

Tensors may live on any one GPU: the call is made on that device, on its current stream (or
on ``stream``, a stream of that device).  What the conveniences allocate, they allocate on
the stream that the call runs on.
"""
from __future__ import annotations

import functools

import torch

from . import GDN_BF16, GDN_F32, _check, lib
from .latent import _bytes, _done, _dtype, _gpu, _on as _on_slow, _ptr, _query, _scale, _workspace

__all__ = ["gdn_attn_prologue", "gdn_attn_prologue_bwd", "gdn_attn_prologue_bwd_workspace_size",
           "gdn_attn_fwd", "gdn_attn_fwd_workspace_size", "gdn_attn_bwd", "gdn_attn_bwd_workspace_size",
           "gdn_attn_append", "gdn_attn_step", "gdn_attn_step_workspace_size", "attn_prologue",
           "attn_prologue_bwd", "attn_fwd", "attn_bwd", "attn_append_", "attn_step"]

BLOCK = 16  # tokens that share a scale


@functools.lru_cache(maxsize=None)   # the loaded library keeps its entry points
def _entry(name):
    return getattr(lib(), name)


# Small calls take as long as their host side, so the checks below look at what must hold
# first, in as few steps as it takes, and say what does not hold only then.

_CODES = {torch.bfloat16: GDN_BF16, torch.float32: GDN_F32}


def _code(t) -> int:
    """The dtype code of a tensor on a GPU."""
    code = _CODES.get(t.dtype)
    if code is None:
        code = _dtype(t.dtype)
    if not t.is_cuda:
        _gpu(t)
    return code


def _need(t, name, shape, dtype, dev):
    """Check a contiguous tensor on GPU `dev`."""
    if not (t.shape == shape and t.dtype is dtype and t.get_device() == dev and t.is_contiguous()):
        _check(t, name, shape, dtype, torch.device("cuda", dev))


def _step_of(t, name, T, H, D, dtype, dev) -> int:
    """Check a packed tensor [T, H, D] on GPU `dev` that may be a slice along the heads;
    returns the elements from token to token."""
    if t.shape != (T, H, D):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(T, H, D)}")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")
    s0, s1, s2 = t.stride()
    if (s2 != 1 and D > 1) or (s1 != D and H > 1):
        raise ValueError(f"{name}: the heads of a token must be contiguous, got strides {t.stride()}")
    return s0 if T > 1 else max(H, 1) * D


def _packed(t, name):
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, D], got {tuple(t.shape)}")
    return t.shape


_like = torch.empty_like   # contiguous for slices along the heads too, and quicker than new_empty


def _space(workspace, dev):
    if workspace is not None:
        _check(workspace, "workspace", device=torch.device("cuda", dev))


_current, _raw_stream = getattr(torch._C, "_cuda_getDevice", None), getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _on(t, stream, call):
    """``call(handle)`` with t's GPU current, and the stream that the work goes to."""
    if stream is None:
        i = t.get_device()
        if i == _current():
            return call(_raw_stream(i))
    return _on_slow(t, stream, call)


# --- prologue -------------------------------------------------------------------

def _prologue_args(q_raw, k_raw, w_q, w_k, inv_freq, pos):
    """Check the inputs; returns (T, Hq, Hk, D, R), the strides and the dtype code."""
    T, Hq, D = _packed(q_raw, "q_raw")
    Hk = _packed(k_raw, "k_raw")[1]
    code = _code(q_raw)
    dt, dev = q_raw.dtype, q_raw.get_device()
    qs = _step_of(q_raw, "q_raw", T, Hq, D, dt, dev)
    ks = _step_of(k_raw, "k_raw", T, Hk, D, dt, dev)
    f = torch.float32
    if not (w_q.shape == (D,) and w_k.shape == (D,) and w_q.dtype is f and w_k.dtype is f and w_q.get_device() == dev
            and w_k.get_device() == dev and w_q.is_contiguous() and w_k.is_contiguous()):
        _need(w_q, "w_q", (D,), f, dev)
        _need(w_k, "w_k", (D,), f, dev)
    R = 0
    if inv_freq is not None:
        if inv_freq.dim() != 1:
            raise ValueError("inv_freq must be [R / 2]")
        R = 2 * inv_freq.shape[0]
        _need(inv_freq, "inv_freq", inv_freq.shape, f, dev)
        if pos is None:
            raise ValueError("pos is required for the rotation")
        _need(pos, "pos", (T,), torch.int32, dev)
    return (T, Hq, Hk, D, R), (qs, ks), code


def _prologue(q_raw, k_raw, w_q, w_k, inv_freq, pos, q, k, eps, sizes, steps, code, handle):
    _done(_entry("gdn_attn_prologue")(q_raw.data_ptr(), k_raw.data_ptr(), w_q.data_ptr(), w_k.data_ptr(), _ptr(inv_freq),
                                  _ptr(pos), q.data_ptr(), k.data_ptr(), *sizes, *steps, eps, code, handle),
          "gdn_attn_prologue")


def gdn_attn_prologue(q_raw, k_raw, w_q, w_k, inv_freq, pos, q, k, eps, stream=None) -> None:
    """RMS norm of every head and rotation by position: writes q [T,Hq,D] and k [T,Hk,D].

    q_raw [T,Hq,D] and k_raw [T,Hk,D] share a dtype (bf16 or fp32); w_q, w_k [D] fp32;
    inv_freq [R/2] fp32 rotates the channel pairs (i, i + R/2) by pos * inv_freq[i], or None
    (no rotation); pos [T] int32.
    """
    sizes, steps, code = _prologue_args(q_raw, k_raw, w_q, w_k, inv_freq, pos)
    _need(q, "q", q_raw.shape, q_raw.dtype, q_raw.get_device())
    _need(k, "k", k_raw.shape, q_raw.dtype, q_raw.get_device())
    _on(q_raw, stream, lambda handle: _prologue(q_raw, k_raw, w_q, w_k, inv_freq, pos, q, k, eps, sizes, steps, code, handle))


def attn_prologue(q_raw, k_raw, w_q, w_k, inv_freq, pos, eps=1e-6, stream=None):
    """Allocate q and k, run gdn_attn_prologue, return (q, k)."""
    sizes, steps, code = _prologue_args(q_raw, k_raw, w_q, w_k, inv_freq, pos)

    def call(handle):
        q, k = _like(q_raw), _like(k_raw)
        _prologue(q_raw, k_raw, w_q, w_k, inv_freq, pos, q, k, eps, sizes, steps, code, handle)
        return q, k

    return _on(q_raw, stream, call)


def gdn_attn_prologue_bwd_workspace_size(T, Hq, Hk, D, R, dtype) -> int:
    """Bytes of workspace gdn_attn_prologue_bwd needs."""
    return _query("gdn_attn_prologue_bwd_workspace_size", T, Hq, Hk, D, R, _dtype(dtype))


def _prologue_bwd_args(q_raw, k_raw, w_q, w_k, inv_freq, pos, d_q, d_k):
    args = _prologue_args(q_raw, k_raw, w_q, w_k, inv_freq, pos)
    _need(d_q, "d_q", q_raw.shape, q_raw.dtype, q_raw.get_device())
    _need(d_k, "d_k", k_raw.shape, q_raw.dtype, q_raw.get_device())
    return args


def _prologue_bwd(q_raw, k_raw, w_q, w_k, inv_freq, pos, d_q, d_k, dq_raw, dk_raw, dw_q, dw_k, workspace, eps, sizes, steps,
                  code, handle):
    _done(_entry("gdn_attn_prologue_bwd")(q_raw.data_ptr(), k_raw.data_ptr(), w_q.data_ptr(), w_k.data_ptr(), _ptr(inv_freq),
                                      _ptr(pos), d_q.data_ptr(), d_k.data_ptr(), dq_raw.data_ptr(), dk_raw.data_ptr(),
                                      dw_q.data_ptr(), dw_k.data_ptr(), _ptr(workspace), _bytes(workspace), *sizes, *steps,
                                      eps, code, handle), "gdn_attn_prologue_bwd")


def gdn_attn_prologue_bwd(q_raw, k_raw, w_q, w_k, inv_freq, pos, d_q, d_k, dq_raw, dk_raw, dw_q, dw_k, workspace, eps,
                          stream=None) -> None:
    """Gradients of gdn_attn_prologue: writes dq_raw, dk_raw in the shapes of q_raw, k_raw
    and dw_q, dw_k [D] fp32, from d_q and d_k, the gradients of its outputs."""
    sizes, steps, code = _prologue_bwd_args(q_raw, k_raw, w_q, w_k, inv_freq, pos, d_q, d_k)
    T, Hq, Hk, D, _ = sizes
    dt, dev = q_raw.dtype, q_raw.get_device()
    steps += (_step_of(dq_raw, "dq_raw", T, Hq, D, dt, dev), _step_of(dk_raw, "dk_raw", T, Hk, D, dt, dev))
    _need(dw_q, "dw_q", (D,), torch.float32, dev)
    _need(dw_k, "dw_k", (D,), torch.float32, dev)
    _space(workspace, dev)
    _on(q_raw, stream, lambda handle: _prologue_bwd(q_raw, k_raw, w_q, w_k, inv_freq, pos, d_q, d_k, dq_raw, dk_raw, dw_q,
                                                    dw_k, workspace, eps, sizes, steps, code, handle))


def attn_prologue_bwd(q_raw, k_raw, w_q, w_k, inv_freq, pos, d_q, d_k, eps=1e-6, workspace=None, stream=None):
    """Allocate the gradients (and the workspace unless one is given), run
    gdn_attn_prologue_bwd, return a dict with dq_raw, dk_raw, dw_q, dw_k."""
    sizes, steps, code = _prologue_bwd_args(q_raw, k_raw, w_q, w_k, inv_freq, pos, d_q, d_k)
    T, Hq, Hk, D, _ = sizes
    _space(workspace, q_raw.get_device())
    steps += (max(Hq, 1) * D, max(Hk, 1) * D)

    def call(handle):
        g = dict(dq_raw=_like(q_raw), dk_raw=_like(k_raw), dw_q=_like(w_q), dw_k=_like(w_k))
        ws = workspace if workspace is not None else \
            _workspace(_query("gdn_attn_prologue_bwd_workspace_size", *sizes, code), q_raw.device)
        _prologue_bwd(q_raw, k_raw, w_q, w_k, inv_freq, pos, d_q, d_k, g["dq_raw"], g["dk_raw"], g["dw_q"], g["dw_k"], ws,
                      eps, sizes, steps, code, handle)
        return g

    return _on(q_raw, stream, call)


# --- whole sequences ------------------------------------------------------------

def _attn_args(q, k, v, cu_q, cu_k):
    """Check the inputs; returns (B, Tq, Tk, Hq, Hk, D), the strides and the dtype code."""
    Tq, Hq, D = _packed(q, "q")
    Tk, Hk, _ = _packed(k, "k")
    code = _code(q)
    dt, dev = q.dtype, q.get_device()
    steps = (_step_of(q, "q", Tq, Hq, D, dt, dev), _step_of(k, "k", Tk, Hk, D, dt, dev), _step_of(v, "v", Tk, Hk, D, dt, dev))
    if cu_q.dim() != 1 or cu_q.shape[0] < 1:
        raise ValueError("cu_q must be [B + 1]")
    _need(cu_q, "cu_q", cu_q.shape, torch.int32, dev)
    if cu_k is not None:
        _need(cu_k, "cu_k", cu_q.shape, torch.int32, dev)
    elif Tq != Tk:
        raise ValueError(f"q has {Tq} tokens and k {Tk}: cu_k is required")
    return (cu_q.shape[0] - 1, Tq, Tk, Hq, Hk, D), steps, code


def gdn_attn_fwd_workspace_size(B, Tq, Tk, Hq, Hk, D, dtype) -> int:
    """Bytes of workspace gdn_attn_fwd needs (0: none)."""
    return _query("gdn_attn_fwd_workspace_size", B, Tq, Tk, Hq, Hk, D, _dtype(dtype))


def gdn_attn_bwd_workspace_size(B, Tq, Tk, Hq, Hk, D, dtype) -> int:
    """Bytes of workspace gdn_attn_bwd needs."""
    return _query("gdn_attn_bwd_workspace_size", B, Tq, Tk, Hq, Hk, D, _dtype(dtype))


def _fwd(q, k, v, cu_q, cu_k, o, lse, workspace, scale, sizes, steps, code, handle):
    _done(_entry("gdn_attn_fwd")(q.data_ptr(), k.data_ptr(), v.data_ptr(), cu_q.data_ptr(), _ptr(cu_k), o.data_ptr(), _ptr(lse),
                             _ptr(workspace), _bytes(workspace), *sizes, *steps, scale, code, handle), "gdn_attn_fwd")


def gdn_attn_fwd(q, k, v, cu_q, cu_k, o, lse, workspace, scale, stream=None) -> None:
    """Causal forward over packed sequences: writes o [Tq,Hq,D] and lse [Tq,Hq] fp32 (or None).

    q [Tq,Hq,D] and k, v [Tk,Hk,D] share a dtype (bf16 or fp32); cu_q [B+1] int32 are the
    sequences' first query rows, cu_k [B+1] their first keys, or None (as cu_q).  Row i of a
    sequence of lq rows and lk keys sees the keys up to lk - lq + i; a row that sees none has
    o = 0, lse = -inf.  Rows of no sequence are left as they were.
    """
    sizes, steps, code = _attn_args(q, k, v, cu_q, cu_k)
    _need(o, "o", q.shape, q.dtype, q.get_device())
    _check(lse, "lse", q.shape[:2], torch.float32, q.device)
    _space(workspace, q.get_device())
    _on(q, stream, lambda handle: _fwd(q, k, v, cu_q, cu_k, o, lse, workspace, scale, sizes, steps, code, handle))


def attn_fwd(q, k, v, cu_q, cu_k=None, scale=None, workspace=None, stream=None):
    """Allocate o and lse (and the workspace, if one is needed and none is given), run
    gdn_attn_fwd, return (o, lse).  scale: 1 / sqrt(D) unless given.  Rows of no sequence
    hold whatever the memory held."""
    sizes, steps, code = _attn_args(q, k, v, cu_q, cu_k)
    _space(workspace, q.get_device())

    def call(handle):
        o, lse = _like(q), torch.empty(q.shape[:2], dtype=torch.float32, device=q.device)
        ws = workspace if workspace is not None else _workspace(_query("gdn_attn_fwd_workspace_size", *sizes, code), q.device)
        _fwd(q, k, v, cu_q, cu_k, o, lse, ws, _scale(scale, sizes[5]), sizes, steps, code, handle)
        return o, lse

    return _on(q, stream, call)


def _bwd_args(q, k, v, o, lse, d_o, cu_q, cu_k):
    args = _attn_args(q, k, v, cu_q, cu_k)
    dev = q.get_device()
    _need(o, "o", q.shape, q.dtype, dev)
    _need(d_o, "d_o", q.shape, q.dtype, dev)
    _need(lse, "lse", q.shape[:2], torch.float32, dev)
    return args


def _bwd(q, k, v, cu_q, cu_k, o, lse, d_o, dq, dk, dv, workspace, scale, sizes, steps, code, handle):
    _done(_entry("gdn_attn_bwd")(q.data_ptr(), k.data_ptr(), v.data_ptr(), cu_q.data_ptr(), _ptr(cu_k), o.data_ptr(),
                             lse.data_ptr(), d_o.data_ptr(), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), _ptr(workspace),
                             _bytes(workspace), *sizes, *steps, scale, code, handle), "gdn_attn_bwd")


def gdn_attn_bwd(q, k, v, cu_q, cu_k, o, lse, d_o, dq, dk, dv, workspace, scale, stream=None) -> None:
    """Gradients of gdn_attn_fwd: writes dq, dk and dv in the shapes of q, k and v.  o and
    lse are the forward's outputs.  Rows of no sequence are left as they were."""
    sizes, steps, code = _bwd_args(q, k, v, o, lse, d_o, cu_q, cu_k)
    _, Tq, Tk, Hq, Hk, D = sizes
    dt, dev = q.dtype, q.get_device()
    steps += (_step_of(dq, "dq", Tq, Hq, D, dt, dev), _step_of(dk, "dk", Tk, Hk, D, dt, dev),
              _step_of(dv, "dv", Tk, Hk, D, dt, dev))
    _space(workspace, dev)
    _on(q, stream, lambda handle: _bwd(q, k, v, cu_q, cu_k, o, lse, d_o, dq, dk, dv, workspace, scale, sizes, steps, code, handle))


def attn_bwd(q, k, v, o, lse, d_o, cu_q, cu_k=None, scale=None, workspace=None, stream=None):
    """Allocate the gradients (and the workspace unless one is given), run gdn_attn_bwd,
    return a dict with dq, dk, dv.  cu_q, cu_k and scale as given to the forward.  Rows of
    no sequence hold whatever the memory held."""
    sizes, steps, code = _bwd_args(q, k, v, o, lse, d_o, cu_q, cu_k)
    _space(workspace, q.get_device())
    _, _, _, Hq, Hk, D = sizes
    steps += (Hq * D, Hk * D, Hk * D)

    def call(handle):
        dq, dk, dv = _like(q), _like(k), _like(v)
        ws = workspace if workspace is not None else _workspace(_query("gdn_attn_bwd_workspace_size", *sizes, code), q.device)
        _bwd(q, k, v, cu_q, cu_k, o, lse, d_o, dq, dk, dv, ws, _scale(scale, D), sizes, steps, code, handle)
        return dict(dq=dq, dk=dk, dv=dv)

    return _on(q, stream, call)


# --- the cache ------------------------------------------------------------------

def _cache_args(k_cache, v_cache, k_scale, v_scale, table, lens, dev):
    """Check a cache; returns (N, Hk, D, pages, page, width)."""
    if k_cache.dim() != 4 or table.dim() != 2:
        raise ValueError("k_cache must be [pages, Hk, page, D], table [N, width]")
    pages, Hk, page, D = k_cache.shape
    if page % BLOCK:
        raise ValueError(f"pages must have a multiple of {BLOCK} tokens, got {page}")
    N, width = table.shape
    dt = k_cache.dtype
    if dt is not torch.float8_e4m3fn and dt is not torch.uint8:
        raise TypeError(f"k_cache must be float8_e4m3fn or uint8, got {dt}")
    blocks = (pages, Hk, page // BLOCK)
    f, i = torch.float32, torch.int32
    if not (v_cache.shape == (*blocks, D, BLOCK) and v_cache.dtype is dt and k_scale.shape == blocks and k_scale.dtype is f
            and v_scale.shape == blocks and v_scale.dtype is f and table.dtype is i and lens.shape == (N,) and lens.dtype is i
            and k_cache.get_device() == dev and v_cache.get_device() == dev and k_scale.get_device() == dev
            and v_scale.get_device() == dev and table.get_device() == dev and lens.get_device() == dev
            and k_cache.is_contiguous() and v_cache.is_contiguous() and k_scale.is_contiguous() and v_scale.is_contiguous()
            and table.is_contiguous() and lens.is_contiguous()):
        _need(k_cache, "k_cache", k_cache.shape, dt, dev)
        _need(v_cache, "v_cache", (*blocks, D, BLOCK), dt, dev)
        _need(k_scale, "k_scale", blocks, f, dev)
        _need(v_scale, "v_scale", blocks, f, dev)
        _need(table, "table", (N, width), i, dev)
        _need(lens, "lens", (N,), i, dev)
    return N, Hk, D, pages, page, width


def gdn_attn_append(k, v, cu, k_cache, v_cache, k_scale, v_scale, table, lens, stream=None) -> None:
    """New tokens k, v [T,Hk,D] into the cache, in place.

    The rows cu[n] .. cu[n+1] - 1 (cu [N+1] int32; None: row n) become the last tokens of
    sequence n, whose lens[n] counts them.  A block of 16 tokens and head takes the smallest
    power of two as its scale that brings its largest magnitude to 448 or less; a block that
    older tokens share keeps theirs unless it has to grow.
    """
    T = _packed(k, "k")[0]
    code = _code(k)
    dt, dev = k.dtype, k.get_device()
    N, Hk, D, pages, page, width = _cache_args(k_cache, v_cache, k_scale, v_scale, table, lens, dev)
    ks, vs = _step_of(k, "k", T, Hk, D, dt, dev), _step_of(v, "v", T, Hk, D, dt, dev)
    if cu is not None:
        _need(cu, "cu", (N + 1,), torch.int32, dev)
    elif T != N:
        raise ValueError(f"{T} tokens for {N} sequences: cu is required")
    _on(k, stream, lambda handle: _done(
        _entry("gdn_attn_append")(k.data_ptr(), v.data_ptr(), _ptr(cu), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(),
                              v_scale.data_ptr(), table.data_ptr(), lens.data_ptr(), N, T, Hk, D, pages, page, width, ks, vs,
                              code, handle), "gdn_attn_append"))


def attn_append_(k, v, k_cache, v_cache, k_scale, v_scale, table, lens, cu=None, stream=None) -> None:
    """gdn_attn_append with the cache first, then how the tokens are packed."""
    gdn_attn_append(k, v, cu, k_cache, v_cache, k_scale, v_scale, table, lens, stream=stream)


def gdn_attn_step_workspace_size(N, Hq, Hk, D, page, width) -> int:
    """Bytes of workspace gdn_attn_step needs (0: none)."""
    return _query("gdn_attn_step_workspace_size", N, Hq, Hk, D, page, width)


def _step_args(q, k_cache, v_cache, k_scale, v_scale, table, lens):
    """Check the inputs; returns (N, Hq, Hk, D, pages, page, width) and the dtype code."""
    N, Hq, D = _packed(q, "q")
    code, dev = _code(q), q.get_device()
    n, Hk, d, pages, page, width = _cache_args(k_cache, v_cache, k_scale, v_scale, table, lens, dev)
    _need(q, "q", (n, Hq, d), q.dtype, dev)
    return (N, Hq, Hk, D, pages, page, width), code


def _step(q, k_cache, v_cache, k_scale, v_scale, table, lens, o, lse, workspace, scale, sizes, code, handle):
    _done(_entry("gdn_attn_step")(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                              table.data_ptr(), lens.data_ptr(), o.data_ptr(), _ptr(lse), _ptr(workspace), _bytes(workspace),
                              *sizes, scale, code, handle), "gdn_attn_step")


def gdn_attn_step(q, k_cache, v_cache, k_scale, v_scale, table, lens, o, lse, workspace, scale, stream=None) -> None:
    """One token a sequence: q [N,Hq,D] over the cache by table [N,width] int32 and lens [N]
    int32; writes o [N,Hq,D] and lse [N,Hq] fp32 (or None).  Pages outside the cache hold no
    tokens; a sequence with no token has o = 0, lse = -inf."""
    sizes, code = _step_args(q, k_cache, v_cache, k_scale, v_scale, table, lens)
    _need(o, "o", q.shape, q.dtype, q.get_device())
    _check(lse, "lse", q.shape[:2], torch.float32, q.device)
    _space(workspace, q.get_device())
    _on(q, stream, lambda handle: _step(q, k_cache, v_cache, k_scale, v_scale, table, lens, o, lse, workspace, scale, sizes,
                                        code, handle))


def attn_step(q, k_cache, v_cache, k_scale, v_scale, table, lens, scale=None, want_lse=False, workspace=None, stream=None):
    """Allocate o (and the workspace, if one is needed and none is given), run gdn_attn_step,
    return o, or (o, lse).  scale: 1 / sqrt(D) unless given."""
    sizes, code = _step_args(q, k_cache, v_cache, k_scale, v_scale, table, lens)
    _space(workspace, q.get_device())

    def call(handle):
        o = _like(q)
        lse = torch.empty(q.shape[:2], dtype=torch.float32, device=q.device) if want_lse else None
        N, Hq, Hk, D, _, page, width = sizes
        ws = workspace if workspace is not None else \
            _workspace(_query("gdn_attn_step_workspace_size", N, Hq, Hk, D, page, width), q.device)
        _step(q, k_cache, v_cache, k_scale, v_scale, table, lens, o, lse, ws, _scale(scale, D), sizes, code, handle)
        return (o, lse) if want_lse else o

    return _on(q, stream, call)
