"""Bounds for linear attention's results from where its roundings are, for inputs
of random numbers in 16 bits.

The kernels go by chunks of 32 steps, and round as operands of the matrix cores,
each by at most u of itself and so in the square mean by at most u^2 / 3: each
score times its power of the decay (p, for the terms inside a chunk) and each
element of the state that a chunk begins with (S, for those before it).  These
roundings are independent of each other and of the result's own.  Where two waves
share a row's values (halves of 64, 128 or 256), each has the score of its half
and rounds that: p^2 stands for the larger of p^2 and p1^2 + p2^2 (halves that
cancel leave a row off by more than its own u, though not more on the average).
For a row a_i with keys k and values v,
  out_i = sum_j p_ij v_j + w_i a_i S,
  var   = (u^2/3) (sum_j p_ij^2 v_j^2 + w_i^2 sum_d a_id^2 S_d^2 + out_i^2),
and for heads whose terms add up the sum over them.  o has rows q, keys k, values
v and state S; dq rows dout, keys v, values k and state S^T; backwards in time, dk
has rows v, keys dout, values q, and dv rows k, keys q, values dout.  Up to 8 steps
o is computed in fp32.

What is not independent enters by its size: the sum of the terms' absolute values
times
  2^-17 in bf16, 2^-21 in fp16   (V's weighted numbers in the state)
  (T / 32 + 2 sqrt(D) + 16) u32  (decays of T / 32 chunks, sums, powers)

A row (D values) may be off by five of its standard deviations and that, the
whole tensor by 1.5."""
import numpy as np

from oracle import model_oracle as mo
from seq_util import TINY, U32, UNIT

CHUNK, FEW = 32, 8


def one(a, k, v, ld, scale, S0, rev, r, few=False):
    """(out, var) of rows a [T, D] with heads of keys and values k [G, T, D], v [G, T, Dv] and the state S0 [D, Dv] before
    (with `rev`: after) them; r: the square mean of a rounding."""
    T = a.shape[0]
    out, var = np.zeros((T, v.shape[2])), np.zeros((T, v.shape[2]))
    starts = list(range(0, T, CHUNK))
    S = S0.copy()
    half = (64 if a.shape[1] <= 64 else 128 if a.shape[1] <= 128 else 256) // 2
    for lo in (reversed(starts) if rev else starts):
        n = min(CHUNK, T - lo)
        A, K, V = a[lo : lo + n], k[:, lo : lo + n], v[:, lo : lo + n]
        i = np.arange(n)
        e = (i[None] - i[:, None]) if rev else (i[:, None] - i[None])
        w = np.where(e >= 0, np.exp(ld * np.maximum(e, 0)), 0.0) * scale
        p = np.einsum("id,gjd->gij", A, K) * w
        since = np.exp(ld * (n - 1 - i)) if rev else np.exp(ld * (i + 1)) * scale
        out[lo : lo + n] = np.einsum("gij,gjc->ic", p, V) + since[:, None] * (A @ S)
        if not few:
            parts = sum((np.einsum("id,gjd->gij", A[:, c], K[:, :, c]) * w) ** 2 for c in (slice(0, half), slice(half, None)))
            var[lo : lo + n] = r * (np.einsum("gij,gjc->ic", np.maximum(p**2, parts), V**2) + since[:, None] ** 2 * (A**2 @ S**2))
        b = np.exp(ld * (i + 1)) * scale if rev else np.exp(ld * (n - 1 - i))
        S = np.exp(ld * n) * S + np.einsum("gjd,gjc,j->dc", K, V, b)
    return out, var + r * out**2, S


def results(dt, x, scale):
    """({name: wanted}, {name: variance}, {name: sizes}) of o, dq, dk, dv; x: the fp64 values of test_gpu_linattn.make."""
    q, k, v, do, ld = (x[i] for i in ("q", "k", "v", "do", "log_decay"))
    T, B, Hq, D = q.shape
    Hk, Dv = k.shape[2], v.shape[3]
    G, r = Hq // Hk, UNIT[dt] ** 2 / 3
    n = np.full(B, T) if x["length"] is None else np.clip(x["length"], 0, T)
    want = dict(o=np.zeros((T, B, Hq, Dv)), dq=np.zeros_like(q), dk=np.zeros_like(k), dv=np.zeros_like(v))
    var = {i: np.zeros_like(j) for i, j in want.items()}
    zeros = np.zeros((B, Hk, D, Dv))
    S0, R0 = (zeros if x[i] is None else x[i] for i in ("state", "dstate"))
    for b in range(B):
        t = slice(0, n[b])
        if n[b] == 0:
            continue
        for h in range(Hk):
            l, heads = min(ld[h], 0.0), range(h * G, (h + 1) * G)
            K, V = k[t, b, h], v[t, b, h]
            Q, O = (np.stack([i[t, b, g] for g in heads]) for i in (q, do))
            for g, c in zip(heads, range(G)):
                for name, a, kk, vv, S, few in (("o", Q[c], K, V, S0[b, h], T <= FEW), ("dq", O[c], V, K, S0[b, h].T, False)):
                    want[name][t, b, g], var[name][t, b, g], _ = one(a, kk[None], vv[None], l, scale, S, False, r, few)
            want["dk"][t, b, h], var["dk"][t, b, h], _ = one(V, O, Q, l, scale, R0[b, h].T, True, r)
            want["dv"][t, b, h], var["dv"][t, b, h], _ = one(K, Q, O, l, scale, R0[b, h], True, r)
    size = mo.linattn(*(abs(i) for i in (q, k, v)), ld, abs(scale), *(i if i is None else abs(i) for i in (x["state"],)), x["length"],
                      abs(do), None if x["dstate"] is None else abs(x["dstate"]))
    c = {"bf16": 2.0**-17, "f16": 2.0**-21}[dt] + (T / 32 + 2 * np.sqrt(max(D, Dv)) + 16) * U32
    return want, var, {i: c * s for i, s in zip(("o", "state", "dq", "dk", "dv"), size)}


def worst(dt, got, want, var, fixed):
    """The largest error of a row and that of the whole tensor, each in units of its bound."""
    err = got - want
    assert np.isfinite(err).all()
    rest = np.linalg.norm(fixed, axis=-1) + TINY[dt] * np.sqrt(want.shape[-1])
    rows = np.linalg.norm(err, axis=-1) / np.maximum(5 * np.sqrt(var.sum(-1)) + rest, 1e-300)
    total = 1.5 * np.sqrt(var.sum()) + np.linalg.norm(rest)
    return float(rows.max(initial=0)), float(np.linalg.norm(err) / max(total, 1e-300))


def check(dt, got, x, scale):
    """got: dict of o, dq, dk, dv in fp64."""
    want, var, fixed = results(dt, x, scale)
    for n, y in got.items():
        row, total = worst(dt, y, want[n], var[n], fixed[n])
        print(f"  {n}: row {row:.2f}, tensor {total:.2f} of the bound", flush=True)
        assert row <= 1 and total <= 1, f"{n}: {row:.3g} times the bound of a row, {total:.3g} of the tensor"
