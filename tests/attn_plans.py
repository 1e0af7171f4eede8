"""The rules by which calls of the grouped-attention kernels are cut, as the launchers have
them: csrc/attn_plan.h, compiled for the host."""
import ctypes
import functools
import os
import subprocess
import tempfile

import gated_deltanet_layer_amd as gdn

CSRC = os.path.join(os.path.dirname(gdn.LIB_PATH), "csrc")
SHIM = """
#include "attn_plan.h"
extern "C" void fwd(int bf16, int B, int Tq, int Tk, int Hk, int G, long *out) {
    const gdn::AttnFwdPlan p = gdn::attn_fwd_plan(bf16, B, Tq, Tk, Hk, G);
    out[0] = p.nr, out[1] = p.tokens, out[2] = p.shares, out[3] = p.halves, out[4] = p.tiles;
}
extern "C" void bwd(int bf16, int B, int Tq, int Tk, int Hk, int G, long *out) {
    const gdn::AttnBwdPlan p = gdn::attn_bwd_plan(bf16, B, Tq, Tk, Hk, G);
    out[0] = p.tokens, out[1] = p.qtiles, out[2] = p.kp, out[3] = p.kstep, out[4] = p.shares;
}
"""


@functools.lru_cache(None)
def _lib():
    with tempfile.TemporaryDirectory() as d:
        src, so = os.path.join(d, "plan.cpp"), os.path.join(d, "plan.so")
        with open(src, "w") as f:
            f.write(SHIM)
        subprocess.run(["g++", "-O1", "-std=c++17", "-shared", "-fPIC", "-I", CSRC, src, "-o", so], check=True)
        return ctypes.CDLL(so)


def _ask(name, names, *args):
    out = (ctypes.c_long * 5)()
    getattr(_lib(), name)(*[int(a) for a in args], out)
    return dict(zip(names, out))


def fwd(dt, B, Tq, Tk, Hq, Hk):
    """nr, tokens, shares, halves, tiles of a forward; form: whole, halves or shares."""
    p = _ask("fwd", ("nr", "tokens", "shares", "halves", "tiles"), dt == "bf16", B, Tq, Tk, Hk, Hq // Hk)
    return dict(p, form="shares" if p["shares"] else "halves" if p["halves"] else "whole")


def bwd(dt, B, Tq, Tk, Hq, Hk):
    """tokens, qtiles, kp, kstep, shares of a backward."""
    return _ask("bwd", ("tokens", "qtiles", "kp", "kstep", "shares"), dt == "bf16", B, Tq, Tk, Hk, Hq // Hk)
