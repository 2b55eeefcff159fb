"""The bounds of linattn_bounds.py themselves, on the CPU: results rounded where
the kernels round pass, and wrong ones do not, at every tested size."""
import numpy as np
import pytest

import linattn_bounds as lb
from oracle import model_oracle as mo
from seq_util import stored

torch = pytest.importorskip("torch")

SIZES = [(9, 4, 2, 2, 8, 8), (33, 2, 4, 4, 128, 128), (65, 4, 6, 3, 80, 48), (97, 2, 8, 2, 200, 136), (100, 1, 5, 1, 37, 201),
         (300, 2, 3, 3, 129, 64), (600, 1, 2, 1, 64, 96), (191, 3, 6, 3, 41, 127), (7, 3, 4, 2, 33, 40)]


def inputs(dt, T, B, Hq, Hk, D, Dv, seed=0, ragged=True):
    """fp64 values of what the kernels are given (the names of test_gpu_linattn.make)."""
    r = np.random.default_rng(seed + T + D)
    x = {n: stored(torch, r.normal(size=s), dt)[1] for n, s in
         (("q", (T, B, Hq, D)), ("k", (T, B, Hk, D)), ("v", (T, B, Hk, Dv)), ("do", (T, B, Hq, Dv)))}
    for n in ("state", "dstate"):
        x[n] = stored(torch, r.normal(size=(B, Hk, D, Dv)), "f32")[1]
    x["log_decay"] = stored(torch, -np.exp(r.uniform(-7, 0, Hk)), "f32")[1]
    x["length"] = r.integers(1, T + 1, B) if ragged else None
    return x


def rounded_one(dt, a, k, v, ld, scale, S0, rev):
    """One run with p and the state rounded to the storage type as operands."""
    r = lambda y: stored(torch, y, dt)[1]  # noqa: E731
    lift = 2.0 ** (4 if dt == "f16" else 0)  # (fp16: a power of two keeps scores of strong decays normal)
    T = a.shape[0]
    out, S = np.zeros((T, v.shape[2])), S0.copy()
    starts = list(range(0, T, 32))
    for lo in (reversed(starts) if rev else starts):
        n = min(32, T - lo)
        i = np.arange(n)
        e = (i[None] - i[:, None]) if rev else (i[:, None] - i[None])
        w = np.where(e >= 0, np.exp(ld * np.maximum(e, 0)), 0.0) * scale
        since = np.exp(ld * (n - 1 - i)) if rev else np.exp(ld * (i + 1)) * scale
        A = a[lo : lo + n]
        for K, V in zip(k[:, lo : lo + n], v[:, lo : lo + n]):
            out[lo : lo + n] += r((A @ K.T) * w * lift) / lift @ V
        out[lo : lo + n] += since[:, None] * (A @ r(S))
        b = np.exp(ld * (i + 1)) * scale if rev else np.exp(ld * (n - 1 - i))
        S = np.exp(ld * n) * S + np.einsum("gjd,gjc,j->dc", k[:, lo : lo + n], v[:, lo : lo + n], b)
    return r(out)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("size", SIZES)
def test_bounds_pass_roundings_and_nothing_else(dt, size):
    x, scale = inputs(dt, *size), 0.37
    T, B, Hq, Hk, D, Dv = size
    want, var, fixed = lb.results(dt, x, scale)
    o, _, dq, dk, dv, _ = mo.linattn(x["q"], x["k"], x["v"], x["log_decay"], scale, x["state"], x["length"], x["do"], x["dstate"])
    for n, y in zip(("o", "dq", "dk", "dv"), (o, dq, dk, dv)):
        np.testing.assert_allclose(want[n], y, rtol=1e-9, atol=1e-11)
    got = {n: np.zeros_like(y) for n, y in want.items()}
    G = Hq // Hk
    for b in range(B):
        t = slice(0, x["length"][b])
        for h in range(Hk):
            ld, K, V = x["log_decay"][h], x["k"][t, b, h], x["v"][t, b, h]
            Q, O = (np.stack([x[i][t, b, h * G + g] for g in range(G)]) for i in ("q", "do"))
            for g in range(G):
                got["o"][t, b, h * G + g] = rounded_one(dt, Q[g], K[None], V[None], ld, scale, x["state"][b, h], False)
                got["dq"][t, b, h * G + g] = rounded_one(dt, O[g], V[None], K[None], ld, scale, x["state"][b, h].T, False)
            got["dk"][t, b, h] = rounded_one(dt, V, O, Q, ld, scale, x["dstate"][b, h].T, True)
            got["dv"][t, b, h] = rounded_one(dt, K, Q, O, ld, scale, x["dstate"][b, h], True)
    if T <= 8:
        got["o"] = stored(torch, want["o"], dt)[1]
    for n, y in got.items():
        row, total = lb.worst(dt, y, want[n], var[n], fixed[n])
        assert row <= 1 and total <= 1, (n, row, total)
        u = lb.UNIT[dt]
        for wrong in (np.zeros_like(y), -want[n], want[n] * (1 + 8 * u)):
            assert lb.worst(dt, wrong, want[n], var[n], fixed[n])[1] > 1, n
    # without the state, and without the shared heads' other terms
    less = dict(x, state=np.zeros_like(x["state"]), dstate=np.zeros_like(x["dstate"]))
    for n, y in lb.results(dt, less, scale)[0].items():
        assert lb.worst(dt, y, want[n], var[n], fixed[n])[1] > 1, n
    if G > 1:
        less = dict(x, do=x["do"].copy())
        less["do"][:, :, ::G] = 0
        for n in ("dk", "dv"):
            y = lb.results(dt, less, scale)[0][n]
            assert lb.worst(dt, y, want[n], var[n], fixed[n])[1] > 1, n
