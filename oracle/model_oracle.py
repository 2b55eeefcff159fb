"""fp64 reference of linear attention, the logits' penalties and the AdamW step
(test infrastructure only), written from their definitions in numpy.  It shares
no code with the library.

  linear attention  S_t = a S_{t-1} + k_t v_t^T, o_t = scale q_t S_t, step by
                    step; a = exp(min(log_decay, 0)) per key head; steps past a
                    sequence's length hold the state and have o = 0.  q [T,B,Hq,D],
                    k [T,B,Hk,D], v [T,B,Hk,Dv]; query head h reads key head
                    h // (Hq / Hk)
  penalties         x > 0 ? x / r : x r where the token has been said, minus
                    presence and frequency times the count, plus the bias; -inf
                    where the mask's bit is 0
  AdamW             m, v, decoupled decay; 8-bit states as e4m3 numbers times a
                    scale per 256 values, sqrt(v) in place of v
"""
import numpy as np


def linattn(q, k, v, log_decay, scale, state=None, length=None, do=None, dstate=None):
    """o, the last state and, with do, dq, dk, dv and the first state's gradient."""
    T, B, Hq, D = q.shape
    Hk, Dv = k.shape[2], v.shape[3]
    G = Hq // Hk if Hk else 1
    a = np.exp(np.minimum(log_decay, 0.0))[None, :, None, None]
    n = np.full(B, T) if length is None else np.clip(np.asarray(length), 0, T)
    S = np.zeros((B, Hk, D, Dv)) if state is None else state.copy()
    o = np.zeros((T, B, Hq, Dv))
    states = []
    for t in range(T):
        real = (t < n)[:, None, None, None]
        kt, vt = np.where(real[..., 0], k[t], 0.0), np.where(real[..., 0], v[t], 0.0)
        S = np.where(real, a * S + kt[..., :, None] * vt[..., None, :], S)
        states.append(S)
        qt = np.where(real[..., 0], q[t], 0.0).reshape(B, Hk, G, D)
        o[t] = scale * (qt @ S).reshape(B, Hq, Dv)
    if do is None:
        return o, S
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    X = np.zeros((B, Hk, D, Dv)) if dstate is None else dstate.copy()  # the gradient of S_t by later steps
    for t in reversed(range(T)):
        real = (t < n)[:, None, None, None]
        gt = np.where(real[..., 0], do[t], 0.0).reshape(B, Hk, G, Dv)
        qt = np.where(real[..., 0], q[t], 0.0).reshape(B, Hk, G, D)
        kt, vt = np.where(real[..., 0], k[t], 0.0), np.where(real[..., 0], v[t], 0.0)
        dq[t] = scale * (gt @ states[t].swapaxes(2, 3)).reshape(B, Hq, D)
        R = X + scale * qt.swapaxes(2, 3) @ gt
        dk[t] = np.where(real[..., 0], (R @ vt[..., None])[..., 0], 0.0)
        dv[t] = np.where(real[..., 0], (kt[..., None, :] @ R)[..., 0, :], 0.0)
        X = np.where(real, a * R, X)
    return o, S, dq, dk, dv, X


def penalty(logits, history=None, length=None, repetition=None, presence=None, frequency=None, bias=None, allowed=None):
    """allowed: [N, V] of bool."""
    x = logits.copy()
    N, V = x.shape
    for n in range(N):
        if history is not None:
            said = history[n][: history.shape[1] if length is None else max(0, int(length[n]))]
            ids, count = np.unique(said[(said >= 0) & (said < V)], return_counts=True)
            old = x[n, ids]
            if repetition is not None:
                old = np.where(old > 0, old / repetition[n], old * repetition[n])
            if presence is not None:
                old = old - presence[n]
            if frequency is not None:
                old = old - frequency[n] * count
            x[n, ids] = old
        if bias is not None:
            x[n] = x[n] + (bias if bias.ndim == 1 else bias[n])
        if allowed is not None:
            x[n] = np.where(allowed[n], x[n], -np.inf)
    return x


def adamw(w, g, m, v, t, lr, beta1, beta2, eps, decay):
    """w, m, v after step t."""
    m = beta1 * m + (1 - beta1) * g
    v = beta2 * v + (1 - beta2) * g * g
    return w - lr * (decay * w + (m / (1 - beta1**t)) / (np.sqrt(v / (1 - beta2**t)) + eps)), m, v


def e4m3_values():
    """The numbers of e4m3 (bias 7, no infinities), from 0 up."""
    out = [0.0]
    for e in range(16):
        for f in range(8):
            if (e, f) == (0, 0) or (e, f) == (15, 7):
                continue
            out.append((f / 8) * 2.0**-6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7))
    return np.array(sorted(out))


def e4m3_step(x):
    """The distance between the e4m3 numbers about |x| <= 448."""
    x = np.abs(x)
    return np.where(x < 2.0**-6, 2.0**-9, 2.0 ** (np.floor(np.log2(np.maximum(x, 2.0**-6))) - 3))


def blocks(x, size=256):
    """x in rows of `size`, the last filled with zeros."""
    n = -(-x.size // size) * size
    return np.pad(x, (0, n - x.size)).reshape(-1, size)
