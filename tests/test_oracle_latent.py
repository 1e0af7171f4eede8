"""Pins of the fp64 latent-attention oracle (CPU): its gradients against central
differences of its forward, the expanded form against the absorbed one, a chain of
drafts against one-token steps, and rows that see nothing."""
import numpy as np
import pytest

from oracle import latent as ref

R = np.random.default_rng


def _expanded(g, B, Tq, Tk, H, dn, dr, dv):
    return g.standard_normal((B, Tq, H, dn + dr)), g.standard_normal((B, Tk, H, dn + dv)), g.standard_normal((B, Tk, dr))


@pytest.mark.parametrize("Tq,Tk,lens", [(5, 5, None), (3, 7, [7, 5]), (6, 6, [2, 6]), (1, 1, None)])
def test_gradients_equal_central_differences(Tq, Tk, lens):
    g = R(0)
    q, kv, kr = _expanded(g, 2, Tq, Tk, 2, 3, 2, 4)
    d_o = g.standard_normal((2, Tq, 2, 4))
    o, lse = ref.forward(q, kv, kr, lens, 0.5)
    grads = ref.backward(q, kv, kr, lens, o, lse, d_o, 0.5)
    for i, x in enumerate((q, kv, kr)):
        d = g.standard_normal(x.shape)
        # central differences: h^2 / 6 of the third derivative (order 1 here) and
        # 2^-52 / h of rounding, both below 1e-9 at h = 1e-5
        h = 1e-5
        f = [ref.forward(*[y + s * h * d if j == i else y for j, y in enumerate((q, kv, kr))], lens, 0.5)[0] for s in (1, -1)]
        num = ((f[0] - f[1]) * d_o).sum() / (2 * h)
        assert abs(num - (grads[i] * d).sum()) <= 1e-8 * max(1.0, abs(num))


def test_expanded_and_absorbed_forms_agree():
    """k = W_uk c and v = W_uv c: folding W_uk into the query and W_uv into the output
    gives the expanded form's output for the last token."""
    g = R(1)
    T, H, dn, dr, dv, r, page = 11, 3, 4, 2, 5, 6, 4
    c, kr = g.standard_normal((1, T, r)), g.standard_normal((1, T, dr))
    Wk, Wv = g.standard_normal((H, dn, r)), g.standard_normal((H, dv, r))
    q = g.standard_normal((1, T, H, dn + dr))
    kv = np.concatenate([np.einsum("btr,hdr->bthd", c, Wk), np.einsum("btr,hdr->bthd", c, Wv)], -1)
    o, lse = ref.forward(q, kv, kr, None, 0.3)
    rows = np.concatenate([c, kr], -1)[0]
    cache = np.zeros((5, page, r + dr))
    table = np.array([[4, 0, 2]])
    for t in range(T):
        cache[table[0, t // page], t % page] = rows[t]
    qa = np.concatenate([np.einsum("hd,hdr->hr", q[0, -1, :, :dn], Wk), q[0, -1, :, dn:]], -1)
    oa, la = ref.absorbed(qa[None, None], cache, table, [T], 0.3, r)
    np.testing.assert_allclose(np.einsum("hr,hdr->hd", oa[0, 0], Wv), o[0, -1], rtol=1e-12)
    np.testing.assert_allclose(la[0, 0], lse[0, -1], rtol=1e-12)


def test_chain_of_drafts_equals_one_token_steps():
    g = R(2)
    r, dr, page, M = 6, 2, 3, 4
    cache, table = g.standard_normal((4, page, r + dr)), np.array([[1, 3, 0]])
    q, draft = g.standard_normal((1, M, 2, r + dr)), g.standard_normal((1, M, r + dr))
    chain, _ = ref.absorbed(q, cache, table, [5], 0.4, r, draft=draft)
    bits, _ = ref.absorbed(q, cache, table, [5], 0.4, r, draft=draft, tree=[[(2 << m) - 1 for m in range(M)]])
    assert np.array_equal(chain, bits)
    for m in range(M):
        c = cache.copy()
        for t in range(m + 1):
            c[table[0, (5 + t) // page], (5 + t) % page] = draft[0, t]
        one, _ = ref.absorbed(q[:, m:m + 1], c, table, [6 + m], 0.4, r)
        np.testing.assert_allclose(one[0, 0], chain[0, m], rtol=1e-12)


def test_rows_that_see_nothing():
    g = R(3)
    q, kv, kr = _expanded(g, 1, 4, 4, 1, 2, 2, 3)
    kv[0, 2:] = np.nan
    o, lse = ref.forward(q, kv, kr, [2], 1.0)
    assert np.isfinite(o).all() and (o[0, 2:] == 0).all() and np.isneginf(lse[0, 2:]).all()
    o, lse = ref.absorbed(g.standard_normal((1, 2, 1, 5)), np.zeros((1, 2, 5)), [[7]], [2], 1.0, 3,
                          draft=np.ones((1, 2, 5)), tree=[[0, 2]])
    assert (o[0, 0] == 0).all() and np.isneginf(lse[0, 0]).all() and (o[0, 1] == 1).all()
