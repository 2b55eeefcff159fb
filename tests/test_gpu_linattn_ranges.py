"""Linear attention in fp16 on values of very different sizes within one call:
the bounds of test_gpu_linattn.py are relative to each output's own terms, so
what is large beside it must not count."""
import numpy as np
import pytest

from seq_util import stored
from test_gpu_linattn import check, make, run

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lstm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from layer_lstm_amd import lstm as mod
    return mod


def put(c, x, name, value):
    t, x[name] = stored(torch, value, "f16")
    c[name] = t.cuda()


@pytest.mark.parametrize("T,B,Hq,Hk,D", [(70, 2, 2, 2, 64), (300, 1, 4, 2, 40), (600, 1, 2, 2, 128), (40, 64, 8, 4, 96),
                                         (100, 2, 3, 3, 200)])
def test_columns_of_different_sizes(lstm, T, B, Hq, Hk, D):
    """v and dout with columns of 1000 beside columns of 0.0001: the states are fp32 outputs, each column as exact as if it
    were alone.  (dq sums products of 1e6 over a third of the columns and some hundred steps: scale 2^-14 keeps it below
    fp16's 65504.)"""
    c, x = make("f16", T, B, Hq, Hk, D, D, decays=[-0.01, -0.3])
    size = np.where(np.arange(D) % 3 == 1, 1000.0, 0.0001)
    for n in ("v", "do"):
        put(c, x, n, x[n] * size)
    x["state"], x["dstate"] = x["state"] * 0.0001, x["dstate"] * 0.0001
    for n in ("state", "dstate"):
        t, x[n] = stored(torch, x[n], "f32")
        c[n] = t.cuda()
    _, o, S, g = run(lstm, "f16", c, scale=2.0**-14)
    check("f16", x, 2.0**-14, o, S, g)


@pytest.mark.parametrize("T", [32, 33, 96, 400])
@pytest.mark.parametrize("decay", [-1.5, -2.6])
def test_a_head_whose_terms_have_nearly_died_away(lstm, T, decay):
    """Two query heads to a state, the second's dout nothing but a step that is 31 from where its chunk's powers begin
    (e^-83 here), the first's of the order of 1000: the sum over both heads keeps the first's."""
    c, x = make("f16", T, 2, 2, 1, 32, 48, ragged=False, decays=[decay])
    do = x["do"].copy() * 1000
    do[np.arange(T) % 32 != 31, :, 1] = 0
    put(c, x, "do", do)
    _, o, S, g = run(lstm, "f16", c, scale=0.37)
    assert all(bool(torch.isfinite(i).all()) for i in (o, S, *g))
    check("f16", x, 0.37, o, S, g)


def test_steps_that_die_away_beside_large_states(lstm):
    """Steps of zeros but for the first of a chunk, strong decays (what is left, e^-48 of 1e-8, is a normal fp32 number),
    and states of 1e5 to begin with (dv = R^T k
    of 64 terms with k of 0.01 stays below 65504)."""
    T, D = 200, 64
    c, x = make("f16", T, 2, 2, 2, D, D, ragged=False, decays=[-1.5, -0.02])
    v, do = x["v"].copy(), x["do"].copy()
    v[np.arange(T) % 32 != 0] = 0
    do[np.arange(T) % 32 != 31] = 0
    put(c, x, "v", v * 1e-3), put(c, x, "do", do * 1e-3)
    for n in ("state", "dstate"):
        t, x[n] = stored(torch, x[n] * 1e5, "f32")
        c[n] = t.cuda()
    put(c, x, "q", x["q"] * 1e-3), put(c, x, "k", x["k"] * 1e-2)
    _, o, S, g = run(lstm, "f16", c, scale=0.01)
    check("f16", x, 0.01, o, S, g)
