"""Bounds for cross attention's results from where its roundings are, for
inputs of random numbers.

In 16 bits the operands of the second product are rounded one by one: p (for o
and dv) and ds = p (dp - delta) (for dq and dk), each by at most u of itself,
so in the square mean by at most u^2 / 3; they are independent of each other,
and so are the roundings of the results.  o is rounded before delta = dout . o
uses it, one error for all keys of a row.  Variances of the results follow:
  o:  (u^2/3) (sum p^2 v^2 + o^2)
  d:  sum_d g^2 var o                                  (delta)
  dq: scale^2 ((u^2/3) sum_k e^2 k^2 + d (sum_k p k)^2) + (u^2/3) dq^2
  dk: scale^2 ((u^2/3) sum_r e^2 q^2 + sum_r d p^2 q^2) + (u^2/3) dk^2
  dv: (u^2/3) (sum_r p^2 g^2 + dv^2)
with e = p (dp - delta).  The errors of fp32, one at its largest for each of a
row's keys, are as independent and enter the same sums: relative to p
  c = (D + 4) u32 scale sum |q k| + 4 u32 (4 + |s| + |lse|) + sqrt(n) u32
(scores, exponential, a sum of n terms), f = (D + 2) u32 sum |g v| of dp and the
same of delta.  What a whole row shares, lse's own error and in 16 bits 2^-18 of
a power of two that p's exponent carries, is relative to the result.

A row (D values) may be off by five of its standard deviations and what it
shares, the whole tensor by 1.5.  So a gradient that is zero, negated or without
delta does not pass, whatever the size."""
import numpy as np

from oracle import seq_oracle as so
from seq_util import TINY, U32, UNIT


def results(dt, q, k, v, g, scale, length=None, mask=None):
    """(wanted, variance, relative error a row shares) of o, dq, dk, dv as arrays of the results' shapes."""
    Tq, B, Hq, D = q.shape
    Tk, _, Hk, _ = k.shape
    G = Hq // Hk
    r = UNIT[dt]**2 / 3
    ok = so.valid_keys(Tk, B, length, mask)
    want = dict(o=np.zeros_like(q), dq=np.zeros_like(q), dk=np.zeros_like(k), dv=np.zeros_like(v))
    var = {n: np.zeros_like(x) for n, x in want.items()}
    shared = 0.0 if dt == "f32" else 2.0**-18
    for b in range(B):
        at = np.flatnonzero(ok[b])
        if at.size == 0:
            continue
        for h in range(Hq):
            j = h // G
            Q, O, K, V = q[:, b, h], g[:, b, h], k[at, b, j], v[at, b, j]
            s = scale * Q @ K.T
            m = s.max(1, keepdims=True)
            lse = m + np.log(np.exp(s - m).sum(1, keepdims=True))
            p = np.exp(s - lse)
            o, dp = p @ V, O @ V.T
            e = p * (dp - (p * dp).sum(1, keepdims=True))
            c = (D + 4) * U32 * scale * (np.abs(Q) @ np.abs(K).T) + 4 * U32 * (4 + np.abs(s) + np.abs(lse)) + \
                np.sqrt(max(at.size, Tq * G)) * U32
            shared = max(shared, float(c.max()) / (1 if dt == "f32" else np.sqrt(at.size)))
            c2 = r + c**2
            vo = (c2 * p**2) @ V**2 + r * o**2
            f2 = ((D + 2) * U32 * (np.abs(O) @ np.abs(V).T))**2
            vd = ((O**2) * vo).sum(1, keepdims=True) + ((D + 2) * U32 * (np.abs(O) * np.abs(o)).sum(1, keepdims=True))**2
            ve = c2 * e**2 + f2 * p**2
            want["o"][:, b, h], var["o"][:, b, h] = o, vo
            want["dq"][:, b, h] = scale * e @ K
            var["dq"][:, b, h] = scale**2 * (ve @ K**2 + vd * (p @ K)**2) + r * want["dq"][:, b, h]**2
            want["dk"][at, b, j] += scale * e.T @ Q
            var["dk"][at, b, j] += scale**2 * (ve.T @ Q**2 + (p**2).T @ (vd * Q**2))
            want["dv"][at, b, j] += p.T @ O
            var["dv"][at, b, j] += (c2 * p**2).T @ O**2
    for x in ("dk", "dv"):
        var[x] += r * want[x]**2
    return want, var, shared


def worst(dt, got, want, var, shared):
    """The largest error of a row and that of the whole tensor, each in units of its bound."""
    err = got - want
    assert np.isfinite(err).all()
    fixed = shared * np.linalg.norm(want, axis=-1) + TINY[dt] * np.sqrt(want.shape[-1])
    rows = np.linalg.norm(err, axis=-1) / np.maximum(5 * np.sqrt(var.sum(-1)) + fixed, 1e-300)
    total = 1.5 * np.sqrt(var.sum()) + np.linalg.norm(fixed)
    return float(rows.max(initial=0)), float(np.linalg.norm(err) / max(total, 1e-300))


def check(dt, got, q, k, v, g, scale, length=None, mask=None):
    """got: dict of o, dq, dk, dv in fp64."""
    want, var, shared = results(dt, q, k, v, g, scale, length, mask)
    for n, x in got.items():
        row, total = worst(dt, x, want[n], var[n], shared)
        print(f"  {n}: row {row:.2f}, tensor {total:.2f} of the bound", flush=True)
        assert row <= 1 and total <= 1, f"{n}: {row:.3g} times the bound of a row, {total:.3g} of the tensor"
