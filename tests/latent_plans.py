"""The rules by which calls of the latent-attention kernels are cut, as the launchers have
them: csrc/latent_plan.h, compiled for the host."""
import ctypes
import functools
import os
import subprocess
import tempfile

import gated_deltanet_layer_amd as gdn

CSRC = os.path.join(os.path.dirname(gdn.LIB_PATH), "csrc")
SHIM = """
#include "latent_plan.h"
extern "C" void fwd(int bf16, int B, int Tq, int Tk, int H, int *out) {
    const gdn::FwdPlan p = gdn::fwd_plan(bf16, B, Tq, Tk, H);
    out[0] = p.nr, out[1] = p.pieces, out[2] = p.each, out[3] = p.shares;
}
extern "C" void bwd(int bf16, int B, int Tq, int Tk, int H, int *out) {
    const gdn::BwdPlan p = gdn::bwd_plan(bf16, B, Tq, Tk, H);
    out[0] = p.kp, out[1] = p.qp, out[2] = p.kstep, out[3] = p.qstep;
}
extern "C" void step(int bf16, int rows, int *out) {
    out[0] = gdn::step_rt(bf16, rows);
    out[1] = gdn::step_shares((rows + out[0] - 1) / out[0]);
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


def _ask(name, n, *args):
    out = (ctypes.c_int * n)()
    getattr(_lib(), name)(*[int(a) for a in args], out)
    return list(out)


def fwd(dt, B, Tq, Tk, H):
    """(row groups a wave, how the call is cut)."""
    nr, pieces, _, shares = _ask("fwd", 4, dt == "bf16", B, Tq, Tk, H)
    return nr, "shares" if shares else "pieces" if pieces > 1 else "whole"


def bwd(dt, B, Tq, Tk, H):
    """Pieces and tiles a piece: of the keys (dq), of the query rows (dk, dv)."""
    st = 64 if dt == "bf16" else 32
    kp, qp, kstep, qstep = _ask("bwd", 4, dt == "bf16", B, Tq, Tk, H)
    return (kp, kstep // st), (qp, qstep // st)


def step(dt, rows):
    """(rows a workgroup, shares of the key tiles)."""
    return tuple(_ask("step", 2, dt == "bf16", rows))
