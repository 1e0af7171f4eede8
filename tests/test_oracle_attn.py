"""Pins of the fp64 grouped-attention oracle (CPU): gradients against central differences,
packed sequences against single ones, rows that see nothing, and the 8-bit cache's rounding
and scales."""
import numpy as np
import pytest
import torch

from oracle import attention as ref

R = np.random.default_rng


def _difference(f, xs, i, d, h=1e-5):
    """Central differences: h^2 / 6 of the third derivative (order 1 here) and 2^-52 / h of
    rounding, both below 1e-9 at h = 1e-5."""
    at = lambda s: f(*[y + s * h * d if j == i else y for j, y in enumerate(xs)])  # noqa: E731
    return (at(1) - at(-1)) / (2 * h)


@pytest.mark.parametrize("lq,lk", [([5], None), ([3, 0, 4], None), ([2, 3], [6, 3]), ([4, 2], [2, 0])])
def test_gradients_equal_central_differences(lq, lk):
    g = R(0)
    cq = np.cumsum([0] + lq)
    ck = None if lk is None else np.cumsum([0] + lk)
    T, Tk = sum(lq), sum(lk or lq)
    xs = [g.standard_normal((T, 4, 3)), g.standard_normal((Tk, 2, 3)), g.standard_normal((Tk, 2, 3))]
    d_o = g.standard_normal((T, 4, 3))
    o, lse = ref.forward(*xs, cq, ck, 0.5)
    grads = ref.backward(*xs, o, lse, d_o, cq, ck, 0.5)
    for i, x in enumerate(xs):
        d = g.standard_normal(x.shape)
        num = _difference(lambda *y: (ref.forward(*y, cq, ck, 0.5)[0] * d_o).sum(), xs, i, d)
        assert abs(num - (grads[i] * d).sum()) <= 1e-8 * max(1.0, abs(num))


def test_prologue_gradients_equal_central_differences():
    g = R(1)
    x, w, dy = g.standard_normal((3, 2, 8)), g.standard_normal(8), g.standard_normal((3, 2, 8))
    inv, pos = np.array([0.3, 1.7]), np.array([0, 5, -2])
    f = lambda x, w: (ref.prologue(x, w, inv, pos, 1e-3) * dy).sum()  # noqa: E731
    grads = ref.prologue_backward(x, w, inv, pos, dy, 1e-3)
    for i in range(2):
        d = g.standard_normal((x, w)[i].shape)
        num = _difference(f, [x, w], i, d)
        assert abs(num - (grads[i] * d).sum()) <= 1e-8 * max(1.0, abs(num))


def test_rotation_keeps_lengths_and_relative_angles():
    g = R(2)
    x, y = g.standard_normal((1, 1, 6)), g.standard_normal((1, 1, 6))
    inv = np.array([1.0, 0.1])
    dot = lambda a, b: float((ref.turn(x, inv, [a]) * ref.turn(y, inv, [b])).sum())  # noqa: E731
    assert np.isclose(dot(7, 3), dot(104, 100)) and not np.isclose(dot(7, 3), dot(7, 4))
    assert np.allclose(ref.turn(ref.turn(x, inv, [9]), inv, [9], back=True), x)
    assert np.array_equal(ref.turn(x, inv, [9])[..., 4:], x[..., 4:])


def test_packed_sequences_are_those_alone():
    g = R(3)
    q, k, v = g.standard_normal((9, 4, 3)), g.standard_normal((9, 2, 3)), g.standard_normal((9, 2, 3))
    o, lse = ref.forward(q, k, v, [1, 5, 5, 8], None, 0.7)
    for a, b in ((1, 5), (5, 8)):
        o1, l1 = ref.forward(q[a:b], k[a:b], v[a:b], [0, b - a], None, 0.7)
        assert np.allclose(o[a:b], o1) and np.allclose(lse[a:b], l1)
    assert np.isnan(o[[0, 8]]).all()
    # heads 0 and 1 read key head 0
    one = ref.forward(q[1:5, 1:2], k[1:5, :1], v[1:5, :1], [0, 4], None, 0.7)[0]
    assert np.allclose(o[1:5, 1:2], one)


def test_rows_that_see_nothing():
    q, k = np.ones((4, 1, 2)), np.ones((2, 1, 2))
    o, lse = ref.forward(q, k, k, [0, 4], [0, 2], 1.0)
    assert (o[:2] == 0).all() and np.isneginf(lse[:2]).all() and np.allclose(o[2:], 1) and np.allclose(lse[2:, 0], [2, 2 + np.log(2)])


def test_values_and_rounding_are_those_of_e4m3():
    assert np.array_equal(torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy(), ref.VALUES, equal_nan=True)
    x = R(4).standard_normal(20000) * 2.0 ** R(5).integers(-14, 8, 20000)
    x = np.clip(x, -448, 448).astype(np.float32)
    x = np.concatenate([x, (ref.VALUES[1:120] + ref.VALUES[2:121]) / 2])   # ties
    assert np.array_equal(torch.from_numpy(x).float().to(torch.float8_e4m3fn).double().numpy(), ref.e4m3_round(x))


def test_scales():
    for x in (448.0, 1.75, 1.0, 1e-3, 447.9, 448.1, 3e38):
        s = ref.scale_of(x)
        assert x <= 448 * s and (x > 224 * s or s == 2.0 ** -126)
    assert ref.scale_of(0.0) == 2.0 ** -126


def test_appended_tokens_are_what_a_step_reads():
    """Tokens appended in pieces, values that grow within a block: every stored value is the
    nearest at its block's scale, and the step is the attention over them."""
    g = R(6)
    Hk, D, page = 2, 4, 32
    kc, vc = np.zeros((5, Hk, page, D)), np.zeros((5, Hk, page // 16, D, 16))
    ks, vs = np.ones((5, Hk, page // 16)), np.ones((5, Hk, page // 16))
    table = np.array([[3, 1]])
    x = g.standard_normal((40, 2, Hk, D)) * 2.0 ** np.arange(40)[:, None, None, None] / 1e4
    for a, b in ((0, 5), (5, 6), (6, 30), (30, 40)):
        ref.append(x[a:b, 0], x[a:b, 1], [0, b - a], kc, vc, ks, vs, table, [b])
    k, v, there = ref.cached(kc, vc, ks, vs, table, 40, 0)
    assert there.all() and k.shape == (Hk, 40, D)
    for held, want, s in ((k, x[:, 0], ks), (v, x[:, 1], vs)):
        want = np.swapaxes(want, 0, 1)
        at = np.arange(40)
        scale = s[table[0][at // page], :, at % page // 16].T[..., None]
        # half a step of e4m3, or of its subnormals (2^-9) once for each time the scale grew
        assert (np.abs(held - want) <= 2.0 ** -4 * np.abs(want) + 16 * 2.0 ** -10 * scale).all()
    q = g.standard_normal((1, 6, D))
    o, lse = ref.step(q, kc, vc, ks, vs, table, [40], 0.3)
    for h in range(6):
        s = k[h // 3] @ q[0, h] * 0.3
        w = np.exp(s - s.max())
        assert np.allclose(o[0, h], w @ v[h // 3] / w.sum()) and np.isclose(lse[0, h], s.max() + np.log(w.sum()))
