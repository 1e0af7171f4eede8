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

import contextlib
import ctypes
import math

from . import GDN_OK, GDNError, _check, _dtype_code, _ptr, _stream, lib

__all__ = ["gdn_latent_fwd", "gdn_latent_fwd_workspace_size", "gdn_latent_bwd",
           "gdn_latent_bwd_workspace_size", "gdn_latent_step", "gdn_latent_steps",
           "gdn_latent_steps_workspace_size", "latent_fwd", "latent_bwd", "latent_step",
           "latent_steps"]

ROPE = 64  # width of the rotary key


@contextlib.contextmanager
def _on(t, stream):
    """Make t's GPU, and the stream the call runs on, the current ones."""
    import torch
    if t.device.type != "cuda":
        raise ValueError("tensors must be on a GPU")
    with torch.cuda.device(t.device):
        if stream is None:
            yield None
        else:
            if not hasattr(stream, "cuda_stream"):
                stream = torch.cuda.ExternalStream(int(stream), device=t.device)
            elif stream.device != t.device:
                raise ValueError(f"stream is on {stream.device}, expected {t.device}")
            with torch.cuda.stream(stream):
                yield stream


def _dtype(dtype) -> int:
    if isinstance(dtype, int):
        return dtype
    import torch
    if dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"q must be float32 or bfloat16, got {dtype}")
    return 1 if dtype == torch.bfloat16 else 0


def _query(fn, what, *args) -> int:
    n = ctypes.c_size_t(0)
    rc = fn(*args, ctypes.byref(n))
    if rc != GDN_OK:
        raise GDNError(rc, what)
    return int(n.value)


def _bytes(workspace):
    return 0 if workspace is None else workspace.numel() * workspace.element_size()


def _scale(scale, dk):
    return 1.0 / math.sqrt(dk) if scale is None else scale


def _workspace(n, device):
    import torch
    return torch.empty(n, dtype=torch.uint8, device=device) if n > 0 else None


def _expanded_args(q, kv, k_rope, lens):
    """Check the inputs of the expanded form; returns (B, Tq, Tk, H, dn, dr, dv)."""
    import torch
    if q.dim() != 4 or kv.dim() != 4 or k_rope.dim() != 3:
        raise ValueError("q and kv must be [B, T, H, D], k_rope [B, T, dr]")
    B, Tq, H, dk = q.shape
    Tk, dr = kv.shape[1], k_rope.shape[-1]
    dn, dv = dk - dr, kv.shape[-1] - (dk - dr)
    if dn <= 0 or dv <= 0:
        raise ValueError(f"q has {dk} columns, k_rope {dr} and kv {kv.shape[-1]}: no key or no value part is left")
    _check(q, "q")
    _check(kv, "kv", (B, Tk, H, dn + dv), q.dtype, q.device)
    _check(k_rope, "k_rope", (B, Tk, dr), q.dtype, q.device)
    _check(lens, "lens", (B,), torch.int32, q.device)
    return B, Tq, Tk, H, dn, dr, dv


def _absorbed_args(q, draft, tree, cache, table, lens, o, lse, workspace):
    """Check the tensors of the absorbed form; returns (N, M, H, r, dr, pages, page, width)."""
    import torch
    steps = draft is not None
    if q.dim() != (4 if steps else 3) or cache.dim() != 3 or table.dim() != 2:
        raise ValueError("q must be [N, H, r + dr] ([N, M, H, r + dr] with drafts), cache "
                         "[pages, page, r + dr], table [N, width]")
    N, M, H, D = q.shape if steps else (q.shape[0], 1, *q.shape[1:])
    dev, r = q.device, D - ROPE
    _check(q, "q")
    _check(cache, "cache", (*cache.shape[:2], D), q.dtype, dev)
    _check(table, "table", (N, table.shape[1]), torch.int32, dev)
    _check(lens, "lens", (N,), torch.int32, dev)
    _check(draft, "draft", (N, M, D), q.dtype, dev)
    _check(tree, "tree", (N, M), torch.int64, dev)
    _check(o, "o", (*q.shape[:-1], r), q.dtype, dev)
    _check(lse, "lse", q.shape[:-1], torch.float32, dev)
    _check(workspace, "workspace", device=dev)
    return N, M, H, r, ROPE, cache.shape[0], cache.shape[1], table.shape[1]


def gdn_latent_fwd_workspace_size(B, Tq, Tk, H, dn, dr, dv, dtype) -> int:
    """Bytes of workspace gdn_latent_fwd needs (0: none)."""
    return _query(lib().gdn_latent_fwd_workspace_size, "gdn_latent_fwd_workspace_size",
                  B, Tq, Tk, H, dn, dr, dv, _dtype(dtype))


def gdn_latent_bwd_workspace_size(B, Tq, Tk, H, dn, dr, dv, dtype) -> int:
    """Bytes of workspace gdn_latent_bwd needs."""
    return _query(lib().gdn_latent_bwd_workspace_size, "gdn_latent_bwd_workspace_size",
                  B, Tq, Tk, H, dn, dr, dv, _dtype(dtype))


def gdn_latent_steps_workspace_size(N, M, H, r, dr, dtype) -> int:
    """Bytes of workspace gdn_latent_steps (gdn_latent_step: M = 1) needs."""
    return _query(lib().gdn_latent_steps_workspace_size, "gdn_latent_steps_workspace_size",
                  N, M, H, r, dr, _dtype(dtype))


def gdn_latent_fwd(q, kv, k_rope, lens, o, lse, workspace, scale, stream=None) -> None:
    """Expanded causal forward: writes o [B,Tq,H,dv] and lse [B,Tq,H] fp32 (or None).

    q [B,Tq,H,dn+dr], kv [B,Tk,H,dn+dv] (key part and value, as the up-projection of
    the latents leaves them) and k_rope [B,Tk,dr] share a dtype (bf16 or fp32); lens
    [B] int32 live lengths or None.  Query i sits at position Tk - Tq + i; rows at or
    behind lens[b] are padding (o = 0, lse = -inf).
    """
    import torch
    B, Tq, Tk, H, dn, dr, dv = _expanded_args(q, kv, k_rope, lens)
    _check(o, "o", (B, Tq, H, dv), q.dtype, q.device)
    _check(lse, "lse", (B, Tq, H), torch.float32, q.device)
    _check(workspace, "workspace", device=q.device)
    with _on(q, stream) as st:
        rc = lib().gdn_latent_fwd(_ptr(q), _ptr(kv), _ptr(k_rope), _ptr(lens), _ptr(o), _ptr(lse),
                                  _ptr(workspace), _bytes(workspace), B, Tq, Tk, H, dn, dr, dv,
                                  float(scale), _dtype_code(q), _stream(st))
    if rc != GDN_OK:
        raise GDNError(rc, "gdn_latent_fwd")


def gdn_latent_bwd(q, kv, k_rope, lens, o, lse, d_o, dq, dkv, dk_rope, workspace, scale,
                   stream=None) -> None:
    """Gradients of gdn_latent_fwd: writes dq, dkv and dk_rope (the sum over the heads)
    in the layouts of q, kv and k_rope.  o and lse are the forward's outputs."""
    import torch
    B, Tq, Tk, H, dn, dr, dv = _expanded_args(q, kv, k_rope, lens)
    for t, name in ((o, "o"), (d_o, "d_o")):
        _check(t, name, (B, Tq, H, dv), q.dtype, q.device)
    _check(lse, "lse", (B, Tq, H), torch.float32, q.device)
    for t, name, like in ((dq, "dq", q), (dkv, "dkv", kv), (dk_rope, "dk_rope", k_rope)):
        _check(t, name, like.shape, q.dtype, q.device)
    _check(workspace, "workspace", device=q.device)
    with _on(q, stream) as st:
        rc = lib().gdn_latent_bwd(_ptr(q), _ptr(kv), _ptr(k_rope), _ptr(lens), _ptr(o), _ptr(lse),
                                  _ptr(d_o), _ptr(dq), _ptr(dkv), _ptr(dk_rope), _ptr(workspace),
                                  _bytes(workspace), B, Tq, Tk, H, dn, dr, dv, float(scale),
                                  _dtype_code(q), _stream(st))
    if rc != GDN_OK:
        raise GDNError(rc, "gdn_latent_bwd")


def gdn_latent_step(q, cache, table, lens, o, lse, workspace, scale, stream=None) -> None:
    """Absorbed form, one token: q [N,H,r+dr] over the cache [pages,page,r+dr] by table
    [N,width] int32 and lens [N] int32 (the new token counted); writes o [N,H,r] and lse
    [N,H] fp32 (or None).  Pages outside the cache hold no tokens."""
    N, M, H, r, dr, pages, page, width = _absorbed_args(q, None, None, cache, table, lens, o, lse, workspace)
    with _on(q, stream) as st:
        rc = lib().gdn_latent_step(_ptr(q), _ptr(cache), _ptr(table), _ptr(lens), _ptr(o), _ptr(lse),
                                   _ptr(workspace), _bytes(workspace), N, H, r, dr, pages, page,
                                   width, float(scale), _dtype_code(q), _stream(st))
    if rc != GDN_OK:
        raise GDNError(rc, "gdn_latent_step")


def gdn_latent_steps(q, draft, tree, cache, table, lens, o, lse, workspace, scale, stream=None) -> None:
    """Absorbed form, M drafted tokens: q [N,M,H,r+dr], draft [N,M,r+dr] the drafts' own
    rows (not in the cache), tree [N,M] int64 (bit j of tree[n,m]: draft m sees draft j)
    or None (a chain).  Every draft sees the lens[n] cached tokens."""
    N, M, H, r, dr, pages, page, width = _absorbed_args(q, draft, tree, cache, table, lens, o, lse, workspace)
    with _on(q, stream) as st:
        rc = lib().gdn_latent_steps(_ptr(q), _ptr(draft), _ptr(tree), _ptr(cache), _ptr(table),
                                    _ptr(lens), _ptr(o), _ptr(lse), _ptr(workspace),
                                    _bytes(workspace), N, M, H, r, dr, pages, page, width,
                                    float(scale), _dtype_code(q), _stream(st))
    if rc != GDN_OK:
        raise GDNError(rc, "gdn_latent_steps")


def latent_fwd(q, kv, k_rope, lens=None, scale=None, workspace=None, stream=None):
    """Allocate o and lse (and the workspace, if one is needed and none is given), run
    gdn_latent_fwd, return (o, lse).  scale: 1 / sqrt(dn + dr) unless given."""
    import torch
    B, Tq, Tk, H, dn, dr, dv = _expanded_args(q, kv, k_rope, lens)
    with _on(q, stream):
        o = torch.empty((B, Tq, H, dv), dtype=q.dtype, device=q.device)
        lse = torch.empty((B, Tq, H), dtype=torch.float32, device=q.device)
        if workspace is None:
            workspace = _workspace(gdn_latent_fwd_workspace_size(B, Tq, Tk, H, dn, dr, dv, q.dtype), q.device)
        gdn_latent_fwd(q, kv, k_rope, lens, o, lse, workspace, _scale(scale, dn + dr))
    return o, lse


def latent_bwd(q, kv, k_rope, o, lse, d_o, lens=None, scale=None, workspace=None, stream=None):
    """Allocate the gradients (and the workspace unless one is given), run gdn_latent_bwd,
    return a dict with dq, dkv, dk_rope.  lens and scale as given to the forward."""
    import torch
    B, Tq, Tk, H, dn, dr, dv = _expanded_args(q, kv, k_rope, lens)
    with _on(q, stream):
        out = dict(dq=torch.empty_like(q), dkv=torch.empty_like(kv), dk_rope=torch.empty_like(k_rope))
        if workspace is None:
            workspace = _workspace(gdn_latent_bwd_workspace_size(B, Tq, Tk, H, dn, dr, dv, q.dtype), q.device)
        gdn_latent_bwd(q, kv, k_rope, lens, o, lse, d_o, out["dq"], out["dkv"], out["dk_rope"],
                       workspace, _scale(scale, dn + dr))
    return out


def latent_step(q, cache, table, lens, scale, want_lse=False, workspace=None, stream=None):
    """Allocate o (and the workspace unless one is given), run gdn_latent_step, return o,
    or (o, lse)."""
    return _absorbed(q, None, None, cache, table, lens, scale, want_lse, workspace, stream)


def latent_steps(q, draft, tree, cache, table, lens, scale, want_lse=False, workspace=None, stream=None):
    """Allocate o (and the workspace unless one is given), run gdn_latent_steps, return o,
    or (o, lse)."""
    if draft is None:
        raise ValueError("draft is required")
    return _absorbed(q, draft, tree, cache, table, lens, scale, want_lse, workspace, stream)


def _absorbed(q, draft, tree, cache, table, lens, scale, want_lse, workspace, stream):
    import torch
    N, M, H, r, dr, *_ = _absorbed_args(q, draft, tree, cache, table, lens, None, None, None)
    with _on(q, stream):
        o = torch.empty((*q.shape[:-1], r), dtype=q.dtype, device=q.device)
        lse = torch.empty(q.shape[:-1], dtype=torch.float32, device=q.device) if want_lse else None
        if workspace is None:
            workspace = _workspace(gdn_latent_steps_workspace_size(N, M, H, r, dr, q.dtype), q.device)
        if draft is None:
            gdn_latent_step(q, cache, table, lens, o, lse, workspace, scale)
        else:
            gdn_latent_steps(q, draft, tree, cache, table, lens, o, lse, workspace, scale)
    return (o, lse) if want_lse else o
