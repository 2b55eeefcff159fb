"""The bounds of attend_bounds.py themselves, on the CPU: results rounded where
the kernels round pass, and wrong gradients do not, at every tested size."""
import numpy as np
import pytest

import attend_bounds as ab
from oracle import seq_oracle as so
from seq_util import stored

torch = pytest.importorskip("torch")

SIZES = [(1, 33, 2, 4, 2, 64), (2, 31, 3, 3, 1, 32), (1, 700, 2, 8, 1, 128), (5, 64, 1, 2, 2, 40), (33, 65, 2, 2, 1, 96),
         (40, 129, 3, 6, 3, 80), (130, 70, 1, 1, 1, 64), (9, 300, 2, 2, 2, 192), (17, 100, 1, 4, 2, 256),
         (12, 45, 2, 2, 1, 33), (7, 40, 2, 2, 2, 250), (3, 20, 2, 1, 1, 130), (1, 5000, 1, 2, 1, 64),
         (40, 5000, 1, 2, 1, 64), (34, 140, 2, 4, 4, 37)]


def inputs(dt, Tq, Tk, B, Hq, Hk, D, seed=0, dout=1.0):
    """q, k, v, dout as (tensors of the storage type, their fp64 values)."""
    rng = np.random.default_rng(seed + Tk)
    return list(zip(*(stored(torch, rng.normal(size=(T, B, H, D)) * by, dt)
                      for T, H, by in ((Tq, Hq, 1), (Tk, Hk, 1), (Tk, Hk, 1), (Tq, Hq, dout)))))


def rounded(dt, q, k, v, g, scale):
    """The results with p, o and ds rounded to the storage type, sums in fp64."""
    r = lambda x: stored(torch, x, dt)[1]  # noqa: E731
    Tq, B, Hq, D = q.shape
    G = Hq // k.shape[2]
    out = dict(o=np.zeros_like(q), dq=np.zeros_like(q), dk=np.zeros_like(k), dv=np.zeros_like(v))
    for b in range(B):
        for h in range(Hq):
            Q, O, K, V = q[:, b, h], g[:, b, h], k[:, b, h // G], v[:, b, h // G]
            s = scale * Q @ K.T
            e = np.exp(s - s.max(1, keepdims=True))
            p = e / e.sum(1, keepdims=True)
            o = r(r(e) @ V / e.sum(1, keepdims=True))
            ds = p * (O @ V.T - (O * o).sum(1, keepdims=True))
            ds = r(ds * 2.0**10) / 2.0**10
            out["o"][:, b, h], out["dq"][:, b, h] = o, scale * ds @ K
            out["dk"][:, b, h // G] += scale * ds.T @ Q
            out["dv"][:, b, h // G] += r(p * 2.0**15).T @ O / 2.0**15
    return {n: r(x) for n, x in out.items()}


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("size", SIZES)
def test_bounds_pass_roundings_and_nothing_else(dt, size):
    q, k, v, g = inputs(dt, *size)[1]
    scale = size[-1] ** -0.5
    want, var, shared = ab.results(dt, q, k, v, g, scale)
    for n, x in zip(("o", "dq", "dk", "dv"), (lambda r: (r[0], *r[2:]))(so.attend(q, k, v, scale, do=g))):
        np.testing.assert_allclose(want[n], x, rtol=1e-9, atol=1e-12)
    ab.check(dt, rounded(dt, q, k, v, g, scale), q, k, v, g, scale)
    G = size[3] // size[4]
    s = scale * np.einsum("qbhd,kbhd->bhqk", q, k.repeat(G, 2))
    p = np.exp(s - s.max(-1, keepdims=True))
    p /= p.sum(-1, keepdims=True)
    e = p * np.einsum("qbhd,kbhd->bhqk", g, v.repeat(G, 2))  # without delta
    no_delta = dict(dq=scale * np.einsum("bhqk,kbhd->qbhd", e, k.repeat(G, 2)),
                    dk=scale * np.einsum("bhqk,qbhd->kbhd", e, q).reshape(k.shape[0], k.shape[1], k.shape[2], G, -1).sum(3))
    for n in ("o", "dq", "dk", "dv"):
        wrong = [np.zeros_like(want[n]), -want[n]] + ([no_delta[n]] if n in no_delta else [])
        wrong += [want[n] * (1 + 8 * ab.UNIT[dt])] if dt != "f32" else []
        for x in wrong:
            assert ab.worst(dt, x, want[n], var[n], shared)[1] > 1, n
