"""The rules by which calls of the latent-attention kernels are cut (CPU: csrc/latent_plan.h
compiled for the host)."""
import pytest

from tests import latent_plans as plans


@pytest.mark.parametrize("dt", ["bf16", "fp32"])
@pytest.mark.parametrize("B,H", [(1, 1), (1, 3), (2, 4), (1, 16), (4, 16)])
def test_backward_pieces_are_bounded(dt, B, H):
    """At most 32 pieces of a walk, whatever its length, and never more for a shorter one."""
    for Tq in (1, 33, 500):
        last = (1, 1)
        for Tk in (500, 1500, 8191, 8192, 65408, 65536, 1 << 20):
            (kp, kt), (qp, qt) = plans.bwd(dt, B, Tq, Tk, H)
            step = 64 if dt == "bf16" else 32
            assert 1 <= kp <= 32 and 1 <= qp <= 32
            assert (kp - 1) * kt * step < Tk <= kp * kt * step     # whole tiles, none empty
            assert qp == 1 or (qp - 1) * qt * step < Tq <= qp * qt * step
            if Tk >= 65408:
                assert kp >= last[0]
            last = kp, qp
