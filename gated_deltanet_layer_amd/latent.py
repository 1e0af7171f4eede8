"""Latent attention: the binding of the ``gdn_latent_*`` entry points.

Low-level calls (outputs and workspace given, as in the C ABI):
    gdn_latent_fwd(q, kv, k_rope, lens, o, lse, workspace, scale)
    gdn_latent_bwd(q, kv, k_rope, lens, o, lse, d_o, dq, dkv, dk_rope, workspace, scale)
    gdn_latent_step(q, cache, table, lens, o, lse, workspace, scale)
    gdn_latent_steps(q, draft, tree, cache, table, lens, o, lse, workspace, scale)
and conveniences that allocate: latent_fwd, latent_bwd, latent_step, latent_steps.

Tensors may live on any one GPU: the call is made on that device, on its current
stream (or on ``stream``, a stream of that device).  What the conveniences
allocate, they allocate on the stream that the call runs on.
"""
from __future__ import annotations

import ctypes
import functools
import math

from . import GDN_BF16, GDN_F32, GDN_OK, GDNError, _check, lib

__all__ = ["gdn_latent_fwd", "gdn_latent_fwd_workspace_size", "gdn_latent_bwd",
           "gdn_latent_bwd_workspace_size", "gdn_latent_step", "gdn_latent_steps",
           "gdn_latent_steps_workspace_size", "latent_fwd", "latent_bwd", "latent_step",
           "latent_steps"]

ROPE = 64  # width of the rotary key


def _on(t, stream, call):
    """``call(handle)`` with t's GPU current, and the stream that the work goes to:
    what it allocates belongs to that stream."""
    import torch
    i = t.device.index
    if stream is None:
        if i == torch.cuda.current_device():
            return call(torch._C._cuda_getCurrentRawStream(i))
        with torch.cuda.device(i):
            return call(torch._C._cuda_getCurrentRawStream(i))
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=t.device)
    elif stream.device != t.device:
        raise ValueError(f"stream is on {stream.device}, expected {t.device}")
    with torch.cuda.device(i), torch.cuda.stream(stream):
        return call(stream.cuda_stream)


def _need(t, name, shape, dtype, device):
    """_check of a tensor that is required; quick where it holds."""
    if not (t.shape == shape and t.dtype is dtype and t.device == device and t.is_contiguous()):
        _check(t, name, shape, dtype, device)


def _dtype(dtype) -> int:
    if isinstance(dtype, int):
        return dtype
    import torch
    if dtype is torch.bfloat16:
        return GDN_BF16
    if dtype is torch.float32:
        return GDN_F32
    raise TypeError(f"q must be float32 or bfloat16, got {dtype}")


def _done(rc, what):
    if rc != GDN_OK:
        raise GDNError(rc, what)


@functools.lru_cache(maxsize=4096)   # sizes only: asked for on every call
def _query(what, *args) -> int:
    n = ctypes.c_size_t(0)
    _done(getattr(lib(), what)(*args, ctypes.byref(n)), what)
    return int(n.value)


def _bytes(workspace):
    return 0 if workspace is None else workspace.numel() * workspace.element_size()


def _scale(scale, dk):
    return 1.0 / math.sqrt(dk) if scale is None else scale


def _workspace(n, device):
    import torch
    return torch.empty(n, dtype=torch.uint8, device=device) if n > 0 else None


def _gpu(t):
    if t.device.type != "cuda":
        raise ValueError("tensors must be on a GPU")


def _expanded_args(q, kv, k_rope, lens):
    """Check the inputs of the expanded form; returns (B, Tq, Tk, H, dn, dr, dv, dtype)."""
    import torch
    if q.dim() != 4 or kv.dim() != 4 or k_rope.dim() != 3:
        raise ValueError("q and kv must be [B, T, H, D], k_rope [B, T, dr]")
    B, Tq, H, dk = q.shape
    Tk, dr = kv.shape[1], k_rope.shape[-1]
    dn, dv = dk - dr, kv.shape[-1] - (dk - dr)
    if dn <= 0 or dv <= 0:
        raise ValueError(f"q has {dk} columns, k_rope {dr} and kv {kv.shape[-1]}: no key or no value part is left")
    dt, dev = q.dtype, q.device
    _need(q, "q", q.shape, dt, dev)
    _need(kv, "kv", (B, Tk, H, dn + dv), dt, dev)
    _need(k_rope, "k_rope", (B, Tk, dr), dt, dev)
    if lens is not None:
        _need(lens, "lens", (B,), torch.int32, dev)
    code = _dtype(dt)
    _gpu(q)
    return B, Tq, Tk, H, dn, dr, dv, code


def _absorbed_args(q, draft, tree, cache, table, lens, steps):
    """Check the inputs of the absorbed form; returns (N, M, H, r, dr, pages, page, width, dtype)."""
    import torch
    if q.dim() != (4 if steps else 3) or cache.dim() != 3 or table.dim() != 2:
        raise ValueError("q must be [N, H, r + dr] ([N, M, H, r + dr] with drafts), cache "
                         "[pages, page, r + dr], table [N, width]")
    N, M, H, D = q.shape if steps else (q.shape[0], 1, *q.shape[1:])
    pages, page, _ = cache.shape
    width = table.shape[1]
    dt, dev = q.dtype, q.device
    _need(q, "q", q.shape, dt, dev)
    _need(cache, "cache", (pages, page, D), dt, dev)
    _need(table, "table", (N, width), torch.int32, dev)
    _need(lens, "lens", (N,), torch.int32, dev)
    if steps:
        if draft is None:
            raise ValueError("draft is required")
        _need(draft, "draft", (N, M, D), dt, dev)
        if tree is not None:
            _need(tree, "tree", (N, M), torch.int64, dev)
    code = _dtype(dt)
    _gpu(q)
    return N, M, H, D - ROPE, ROPE, pages, page, width, code


def gdn_latent_fwd_workspace_size(B, Tq, Tk, H, dn, dr, dv, dtype) -> int:
    """Bytes of workspace gdn_latent_fwd needs (0: none)."""
    return _query("gdn_latent_fwd_workspace_size", B, Tq, Tk, H, dn, dr, dv, _dtype(dtype))


def gdn_latent_bwd_workspace_size(B, Tq, Tk, H, dn, dr, dv, dtype) -> int:
    """Bytes of workspace gdn_latent_bwd needs."""
    return _query("gdn_latent_bwd_workspace_size", B, Tq, Tk, H, dn, dr, dv, _dtype(dtype))


def gdn_latent_steps_workspace_size(N, M, H, r, dr, dtype) -> int:
    """Bytes of workspace gdn_latent_steps (gdn_latent_step: M = 1) needs."""
    return _query("gdn_latent_steps_workspace_size", N, M, H, r, dr, _dtype(dtype))


def _ptr(t):
    return None if t is None else t.data_ptr()


def _fwd(q, kv, k_rope, lens, o, lse, workspace, scale, sizes, handle):
    _done(lib().gdn_latent_fwd(q.data_ptr(), kv.data_ptr(), k_rope.data_ptr(), _ptr(lens), o.data_ptr(),
                               _ptr(lse), _ptr(workspace), _bytes(workspace), *sizes[:-1], scale,
                               sizes[-1], handle), "gdn_latent_fwd")


def _bwd(q, kv, k_rope, lens, o, lse, d_o, dq, dkv, dk_rope, workspace, scale, sizes, handle):
    _done(lib().gdn_latent_bwd(q.data_ptr(), kv.data_ptr(), k_rope.data_ptr(), _ptr(lens), o.data_ptr(),
                               lse.data_ptr(), d_o.data_ptr(), dq.data_ptr(), dkv.data_ptr(),
                               dk_rope.data_ptr(), _ptr(workspace), _bytes(workspace), *sizes[:-1],
                               scale, sizes[-1], handle), "gdn_latent_bwd")


def _step(q, draft, tree, cache, table, lens, o, lse, workspace, scale, sizes, handle):
    N, M, H, r, dr, pages, page, width, dt = sizes
    if draft is None:
        _done(lib().gdn_latent_step(q.data_ptr(), cache.data_ptr(), table.data_ptr(), lens.data_ptr(),
                                    o.data_ptr(), _ptr(lse), _ptr(workspace), _bytes(workspace), N, H, r,
                                    dr, pages, page, width, scale, dt, handle), "gdn_latent_step")
    else:
        _done(lib().gdn_latent_steps(q.data_ptr(), draft.data_ptr(), _ptr(tree), cache.data_ptr(),
                                     table.data_ptr(), lens.data_ptr(), o.data_ptr(), _ptr(lse),
                                     _ptr(workspace), _bytes(workspace), N, M, H, r, dr, pages, page,
                                     width, scale, dt, handle), "gdn_latent_steps")


def gdn_latent_fwd(q, kv, k_rope, lens, o, lse, workspace, scale, stream=None) -> None:
    """Expanded causal forward: writes o [B,Tq,H,dv] and lse [B,Tq,H] fp32 (or None).

    q [B,Tq,H,dn+dr], kv [B,Tk,H,dn+dv] (key part and value, as the up-projection of
    the latents leaves them) and k_rope [B,Tk,dr] share a dtype (bf16 or fp32); lens
    [B] int32 live lengths or None.  Query i sits at position Tk - Tq + i; rows at or
    behind lens[b] are padding (o = 0, lse = -inf).
    """
    import torch
    sizes = B, Tq, Tk, H, dn, dr, dv, _ = _expanded_args(q, kv, k_rope, lens)
    _need(o, "o", (B, Tq, H, dv), q.dtype, q.device)
    _check(lse, "lse", (B, Tq, H), torch.float32, q.device)
    _check(workspace, "workspace", device=q.device)
    _on(q, stream, lambda handle: _fwd(q, kv, k_rope, lens, o, lse, workspace, scale, sizes, handle))


def gdn_latent_bwd(q, kv, k_rope, lens, o, lse, d_o, dq, dkv, dk_rope, workspace, scale,
                   stream=None) -> None:
    """Gradients of gdn_latent_fwd: writes dq, dkv and dk_rope (the sum over the heads)
    in the layouts of q, kv and k_rope.  o and lse are the forward's outputs."""
    sizes = _bwd_args(q, kv, k_rope, lens, o, lse, d_o)
    for t, name, like in ((dq, "dq", q), (dkv, "dkv", kv), (dk_rope, "dk_rope", k_rope)):
        _need(t, name, like.shape, q.dtype, q.device)
    _check(workspace, "workspace", device=q.device)
    _on(q, stream, lambda handle: _bwd(q, kv, k_rope, lens, o, lse, d_o, dq, dkv, dk_rope, workspace,
                                       scale, sizes, handle))


def _bwd_args(q, kv, k_rope, lens, o, lse, d_o):
    import torch
    sizes = B, Tq, Tk, H, dn, dr, dv, _ = _expanded_args(q, kv, k_rope, lens)
    for t, name in ((o, "o"), (d_o, "d_o")):
        _need(t, name, (B, Tq, H, dv), q.dtype, q.device)
    _need(lse, "lse", (B, Tq, H), torch.float32, q.device)
    return sizes


def gdn_latent_step(q, cache, table, lens, o, lse, workspace, scale, stream=None) -> None:
    """Absorbed form, one token: q [N,H,r+dr] over the cache [pages,page,r+dr] by table
    [N,width] int32 and lens [N] int32 (the new token counted); writes o [N,H,r] and lse
    [N,H] fp32 (or None).  Pages outside the cache hold no tokens."""
    _given(q, None, None, cache, table, lens, o, lse, workspace, scale, stream, False)


def gdn_latent_steps(q, draft, tree, cache, table, lens, o, lse, workspace, scale, stream=None) -> None:
    """Absorbed form, M drafted tokens: q [N,M,H,r+dr], draft [N,M,r+dr] the drafts' own
    rows (not in the cache), tree [N,M] int64 (bit j of tree[n,m]: draft m sees draft j)
    or None (a chain).  Every draft sees the lens[n] cached tokens."""
    _given(q, draft, tree, cache, table, lens, o, lse, workspace, scale, stream, True)


def _given(q, draft, tree, cache, table, lens, o, lse, workspace, scale, stream, steps):
    import torch
    sizes = _absorbed_args(q, draft, tree, cache, table, lens, steps)
    _need(o, "o", (*q.shape[:-1], sizes[3]), q.dtype, q.device)
    _check(lse, "lse", q.shape[:-1], torch.float32, q.device)
    _check(workspace, "workspace", device=q.device)
    _on(q, stream, lambda handle: _step(q, draft, tree, cache, table, lens, o, lse, workspace, scale,
                                        sizes, handle))


def latent_fwd(q, kv, k_rope, lens=None, scale=None, workspace=None, stream=None):
    """Allocate o and lse (and the workspace, if one is needed and none is given), run
    gdn_latent_fwd, return (o, lse).  scale: 1 / sqrt(dn + dr) unless given."""
    import torch
    sizes = B, Tq, Tk, H, dn, dr, dv, _ = _expanded_args(q, kv, k_rope, lens)
    _check(workspace, "workspace", device=q.device)

    def call(handle):
        o = torch.empty((B, Tq, H, dv), dtype=q.dtype, device=q.device)
        lse = torch.empty((B, Tq, H), dtype=torch.float32, device=q.device)
        ws = workspace if workspace is not None else _workspace(_query("gdn_latent_fwd_workspace_size", *sizes), q.device)
        _fwd(q, kv, k_rope, lens, o, lse, ws, _scale(scale, dn + dr), sizes, handle)
        return o, lse

    return _on(q, stream, call)


def latent_bwd(q, kv, k_rope, o, lse, d_o, lens=None, scale=None, workspace=None, stream=None):
    """Allocate the gradients (and the workspace unless one is given), run gdn_latent_bwd,
    return a dict with dq, dkv, dk_rope.  lens and scale as given to the forward."""
    import torch
    sizes = _bwd_args(q, kv, k_rope, lens, o, lse, d_o)
    _check(workspace, "workspace", device=q.device)

    def call(handle):
        g = dict(dq=torch.empty_like(q), dkv=torch.empty_like(kv), dk_rope=torch.empty_like(k_rope))
        ws = workspace if workspace is not None else _workspace(_query("gdn_latent_bwd_workspace_size", *sizes), q.device)
        _bwd(q, kv, k_rope, lens, o, lse, d_o, g["dq"], g["dkv"], g["dk_rope"], ws,
             _scale(scale, sizes[4] + sizes[5]), sizes, handle)
        return g

    return _on(q, stream, call)


def latent_step(q, cache, table, lens, scale, want_lse=False, workspace=None, stream=None):
    """Allocate o (and the workspace unless one is given), run gdn_latent_step, return o,
    or (o, lse)."""
    return _allocated(q, None, None, cache, table, lens, scale, want_lse, workspace, stream, False)


def latent_steps(q, draft, tree, cache, table, lens, scale, want_lse=False, workspace=None, stream=None):
    """Allocate o (and the workspace unless one is given), run gdn_latent_steps, return o,
    or (o, lse)."""
    return _allocated(q, draft, tree, cache, table, lens, scale, want_lse, workspace, stream, True)


def _allocated(q, draft, tree, cache, table, lens, scale, want_lse, workspace, stream, steps):
    import torch
    sizes = N, M, H, r, dr, _, _, _, dt = _absorbed_args(q, draft, tree, cache, table, lens, steps)
    _check(workspace, "workspace", device=q.device)

    def call(handle):
        o = torch.empty((*q.shape[:-1], r), dtype=q.dtype, device=q.device)
        lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device) if want_lse else None
        ws = workspace if workspace is not None else \
            _workspace(_query("gdn_latent_steps_workspace_size", N, M, H, r, dr, dt), q.device)
        _step(q, draft, tree, cache, table, lens, o, lse, ws, scale, sizes, handle)
        return (o, lse) if want_lse else o

    return _on(q, stream, call)
