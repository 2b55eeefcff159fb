"""The fp64 reference of the sequence-to-sequence operators against central
differences of its own forward, and against values that follow from the
definitions alone."""
import numpy as np
import pytest

from oracle import seq_oracle as so


def differences(f, x, idx, h=1e-5):
    out = []
    for i in idx:
        a, b = x.copy(), x.copy()
        a.reshape(-1)[i] += h
        b.reshape(-1)[i] -= h
        out.append((f(a) - f(b)) / (2 * h))
    return np.array(out)


def test_embedding_gradient_by_differences():
    rng = np.random.default_rng(0)
    V, D, scale = 7, 3, 1.7
    ids = np.array([3, 3, 0, 6, -1, 7, 3, 2])
    table, dout = rng.normal(size=(V, D)), rng.normal(size=(8, D))
    got = so.embed_grad(ids, dout, V, scale)
    num = differences(lambda t: (so.embed(ids, t, scale) * dout).sum(), table, range(V * D))
    np.testing.assert_allclose(got.reshape(-1), num, atol=1e-8)
    pad = so.embed_grad(ids, dout, V, scale, padding=3)
    assert not pad[3].any() and np.array_equal(np.delete(pad, 3, 0), np.delete(got, 3, 0))


@pytest.mark.parametrize("Hq,Hk", [(2, 2), (4, 2), (3, 1)])
def test_attention_gradients_by_differences(Hq, Hk):
    rng = np.random.default_rng(1)
    Tq, Tk, B, D, scale = 3, 5, 3, 4, 0.6
    q, do = rng.normal(size=(2, Tq, B, Hq, D))
    k, v = rng.normal(size=(2, Tk, B, Hk, D))
    length, mask = np.array([5, 3, 0]), np.array([[1, 0, 1, 1, 1], [1, 1, 1, 0, 1], [1] * 5])
    o, lse, dq, dk, dv = so.attend(q, k, v, scale, length, mask, do)
    assert not o[:, 2].any() and np.isneginf(lse[2]).all() and not dq[:, 2].any() and not dk[:, 2].any()

    def loss(q=q, k=k, v=v):
        return (so.attend(q, k, v, scale, length, mask)[0] * do).sum()

    for x, g, f in ((q, dq, lambda a: loss(q=a)), (k, dk, lambda a: loss(k=a)), (v, dv, lambda a: loss(v=a))):
        idx = rng.choice(x.size, 24, replace=False)
        np.testing.assert_allclose(g.reshape(-1)[idx], differences(f, x, idx), atol=1e-8)


def test_attention_of_equal_scores_is_the_mean():
    v = np.random.default_rng(2).normal(size=(4, 1, 1, 3))
    o, lse = so.attend(np.zeros((1, 1, 1, 3)), np.ones((4, 1, 1, 3)), v, 1.0, length=[3])
    np.testing.assert_allclose(o[0, 0, 0], v[:3, 0, 0].mean(0))
    np.testing.assert_allclose(lse[0, 0, 0], np.log(3))


def test_logprob_gradient_by_differences():
    rng = np.random.default_rng(3)
    N, V, scale, top = 4, 9, 0.7, 3
    x, t = rng.normal(size=(N, V)) * 2, np.array([2, -1, 8, 9])
    x[1, 4] = -np.inf
    dl, dh, dt = rng.normal(size=N), rng.normal(size=N), rng.normal(size=(N, top))
    r = so.logprob(x, t, scale, top, dl, dh, dt)

    def loss(a):
        q = so.logprob(a, t, scale, top)
        return (q["logp"] * dl).sum() + (q["entropy"] * dh).sum() + (q["top_logp"] * dt).sum()

    idx = [i for i in range(N * V) if np.isfinite(x.reshape(-1)[i])]
    np.testing.assert_allclose(r["dlogits"].reshape(-1)[idx], differences(loss, x, idx), atol=1e-8)
    assert r["dlogits"][1, 4] == 0


def test_logprob_of_a_uniform_row_ties_and_an_empty_row():
    x = np.array([[1.0, 1.0, 1.0, 1.0], [-np.inf] * 4, [0.0, 2.0, 2.0, -np.inf]])
    r = so.logprob(x, np.array([0, 1, 3]), 1.0, 3)
    np.testing.assert_allclose([r["logp"][0], r["entropy"][0]], [-np.log(4), np.log(4)])
    assert r["lse"][1] == r["logp"][1] == -np.inf and r["entropy"][1] == 0 and np.isneginf(r["top_logp"][1]).all()
    assert r["top_ids"].tolist() == [[0, 1, 2], [0, 1, 2], [1, 2, 0]] and r["logp"][2] == -np.inf
