"""Steps that are not finite, in linear attention: what depends on them by the
definition is not finite, everything else is as if they were zeros.

o_t and dq_t depend on the steps up to t, dk_t and dv_t on those from t on, the
last state's gradient and the first state's on all.  Which of the two, NaN or
an infinity, is not asked (V is multiplied in parts, whose infinities cancel)."""
import numpy as np
import pytest

from oracle import model_oracle as mo
from seq_util import TINY, U32, UNIT, host
from test_gpu_linattn import make, run

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lstm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from layer_lstm_amd import lstm as mod
    return mod


def check(lstm, dt, c, x, bad, scale=0.37):
    """bad: {name: indexes of elements, values}."""
    y = {n: None if x[n] is None else x[n].copy() for n in x}
    for n, (at, value) in bad.items():
        y[n][at], x[n][at] = value, 0.0
        c[n][at] = value
    args = lambda z: (z["q"], z["k"], z["v"], z["log_decay"], scale, z["state"], z["length"], z["do"], z["dstate"])  # noqa: E731
    with np.errstate(all="ignore"):
        there = [np.isfinite(i) for i in mo.linattn(*args(y))]
    for i in (0, 2, 3, 4):  # (zeros by definition past the end: the oracle multiplies zeros there)
        if x["length"] is not None:
            there[i] |= (np.arange(x["q"].shape[0])[:, None] >= x["length"][None])[:, :, None, None]
    want = mo.linattn(*args(x))
    mass = mo.linattn(*args({n: i if i is None or n in ("log_decay", "length") else abs(i) for n, i in x.items()}))
    m, o, S, g = run(lstm, dt, c, scale)
    T, D, Dv = x["q"].shape[0], x["q"].shape[3], x["v"].shape[3]
    low = abs(x["log_decay"][np.isfinite(x["log_decay"])]).max()
    cc = (3 * low * T + T + 2 * max(D, Dv) + 64) * U32
    u = 0.0 if dt == "f32" else 2 * UNIT[dt]
    for name, got, w, s, ok in zip(("o", "state", "dq", "dk", "dv", "dstate"), (o, S, *g), want, mass, there):
        got = host(got)
        wrong = np.argwhere(np.isfinite(got) != ok)
        assert not wrong.size, f"{name}: {len(wrong)} of {(~ok).sum()} expected, the first at {wrong[0]}"
        tol = s * (2.0**-21 + cc) + TINY["f32"] if "state" in name else s * (u + cc) + UNIT[dt] * 1.01 * abs(w) + TINY[dt]
        assert (abs(got - w)[ok] <= tol[ok]).all(), name


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,B,Hq,Hk,D,Dv", [(40, 2, 2, 2, 64, 64), (70, 2, 4, 2, 48, 80), (33, 1, 2, 2, 37, 51), (75, 2, 2, 1, 128, 128),
                                            (600, 1, 2, 1, 64, 64), (70, 32, 16, 8, 32, 32), (100, 1, 2, 2, 200, 256),
                                            (7, 2, 4, 2, 24, 40)])
@pytest.mark.parametrize("name", ["q", "k", "v", "do"])
def test_one_step(lstm, dt, T, B, Hq, Hk, D, Dv, name):
    print(f"case: not finite {name} {dt} T={T} B={B} heads {Hq}/{Hk} D={D} Dv={Dv}", flush=True)
    for t, d, value in ((0, 0, NAN), (5, 3, INF), (min(T - 1, 31), D // 2, -INF), (T // 2, 1, NAN), (T - 1, 2, INF)):
        c, x = make(dt, T, B, Hq, Hk, D, Dv, ragged=False, decays=[-0.02, -0.3, -1.0])
        check(lstm, dt, c, x, {name: ((t, B - 1, 0, d), value)})


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T", [64, 400])
def test_several_steps_and_strong_decays(lstm, dt, T):
    """Elements of three tensors, in one chunk and the next; decays whose powers fp32 does not hold or that
    are zero; a short last chunk."""
    for h in range(5):
        c, x = make(dt, T, 2, 5, 5, 40, 48, decays=[-0.1, -4.0, -40.0, float("-inf"), 0.0])
        c["length"].fill_(T - 3), x["length"].fill(T - 3)
        check(lstm, dt, c, x, {"v": ((9, 1, h, 4), INF), "k": ((35, 0, h, 11), NAN), "do": ((21, 0, h, 5), -INF)})
        c, x = make(dt, T, 2, 5, 5, 40, 48, decays=[-0.1, -4.0, -40.0, float("-inf"), 0.0])
        check(lstm, dt, c, x, {"v": (([9, 20, 20], [0, 0, 0], [h, h, h], [4, 7, 4]), INF), "q": ((3, 0, h, 39), INF)})


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_states(lstm, dt):
    """An element of the first state reaches its column of o and row of dq at all steps, and nothing else."""
    for T in (5, 40, 600):
        for name in ("state", "dstate"):
            c, x = make(dt, T, 2, 4, 2, 40, 48, ragged=False, decays=[-0.01, -0.2])
            check(lstm, dt, c, x, {name: ((1, 0, 7, 9), INF)})
