"""fp64 reference of the sequence-to-sequence operators (test infrastructure
only): embedding, cross attention and log probabilities with their gradients,
written from their definitions in numpy.  It shares no code with the library.

  embedding   out[n] = scale * table[ids[n]] (0 for an id outside [0, V));
              dtable[v] = scale * sum of dout[n] over ids[n] = v != padding
  attention   s = scale q.k over a sequence's valid keys, p = softmax(s),
              o = sum p v; a query with no valid key: o = 0, lse = -inf, no
              gradient.  q [Tq,B,Hq,D], k, v [Tk,B,Hk,D]; query head h reads
              key head h // (Hq / Hk)
  log prob.   z = scale * logits, lse = log sum exp z, logp = z[target] - lse
              (0 for a target outside [0, V)), entropy = -sum p log p, the
              best alternatives in descending order, ties by the lower id
"""
import numpy as np


def embed(ids, table, scale):
    ids = np.asarray(ids)
    ok = (ids >= 0) & (ids < table.shape[0])
    rows = table[np.where(ok, ids, 0)] if table.shape[0] else np.zeros((*ids.shape, table.shape[1]))
    return np.where(ok[..., None], rows, 0.0) * scale


def embed_grad(ids, dout, V, scale, padding=None):
    ids = np.asarray(ids).reshape(-1)
    dout = dout.reshape(ids.size, -1)
    ok = (ids >= 0) & (ids < V)
    if padding is not None:
        ok &= ids != padding
    out = np.zeros((V, dout.shape[1]))
    np.add.at(out, ids[ok], dout[ok])
    return out * scale


def valid_keys(Tk, B, length=None, mask=None):
    """[B, Tk] of bool."""
    ok = np.ones((B, Tk), bool)
    if length is not None:
        ok &= np.arange(Tk)[None, :] < np.asarray(length)[:, None]
    if mask is not None:
        ok &= np.asarray(mask) != 0
    return ok


def attend(q, k, v, scale, length=None, mask=None, do=None):
    """o, lse and, with do, dq, dk, dv."""
    Tq, B, Hq, D = q.shape
    Tk, _, Hk, _ = k.shape
    G = Hq // Hk
    ok = valid_keys(Tk, B, length, mask)
    o, lse = np.zeros_like(q), np.full((B, Hq, Tq), -np.inf)
    dq, dk, dv = np.zeros_like(q), np.zeros_like(k), np.zeros_like(v)
    for b in range(B):
        at = np.flatnonzero(ok[b])
        if at.size == 0:
            continue
        for h in range(Hq):
            K, X = k[at, b, h // G], v[at, b, h // G]
            s = scale * q[:, b, h] @ K.T
            top = s.max(1, keepdims=True)
            e = np.exp(s - top)
            total = e.sum(1, keepdims=True)
            p = e / total
            lse[b, h] = (top + np.log(total))[:, 0]
            o[:, b, h] = p @ X
            if do is None:
                continue
            g = do[:, b, h]
            dp = g @ X.T
            ds = scale * p * (dp - (p * dp).sum(1, keepdims=True))
            dq[:, b, h] = ds @ K
            dk[at, b, h // G] += ds.T @ q[:, b, h]
            dv[at, b, h // G] += p.T @ g
    return (o, lse) if do is None else (o, lse, dq, dk, dv)


def logprob(logits, targets, scale=1.0, top=0, dlogp=None, dentropy=None, dtop=None):
    """dict of lse, logp, entropy, top_logp, top_ids, dlogits."""
    N, V = logits.shape
    z = logits * scale
    out = dict(lse=np.full(N, -np.inf), logp=np.zeros(N), entropy=np.zeros(N), top_logp=np.zeros((N, top)),
               top_ids=np.zeros((N, top), np.int64), dlogits=np.zeros((N, V)))
    for n in range(N):
        t = int(targets[n])
        real = 0 <= t < V
        order = np.argsort(-logits[n], kind="stable")[:top]
        out["top_ids"][n] = order
        if V == 0 or z[n].max() == -np.inf:
            out["logp"][n] = -np.inf if real else 0.0
            out["top_logp"][n] = -np.inf
            continue
        m = z[n].max()
        total = np.log(np.exp(z[n] - m).sum())
        lse, lp = m + total, (z[n] - m) - total
        p = np.exp(lp)
        plp = np.where(p > 0, p * np.where(p > 0, lp, 0.0), 0.0)
        H = -plp.sum()
        out["lse"][n], out["entropy"][n] = lse, H
        out["logp"][n] = lp[t] if real else 0.0
        out["top_logp"][n] = lp[order]
        g = np.zeros(V)
        G = 0.0
        if dlogp is not None and real:
            g[t] += dlogp[n]
            G += dlogp[n]
        if dtop is not None:
            np.add.at(g, order, dtop[n])
            G += dtop[n].sum()
        g -= p * G
        if dentropy is not None:
            g -= dentropy[n] * (plp + p * H)
        out["dlogits"][n] = scale * g
    return out
