"""Cross attention on the GPU against fp64: forward, statistics, gradients.

Bounds.  fp32 storage: every product and sum in fp32; a score's error is
(D + 2) u32 sum|q k| scale, which p carries relatively, p v sums n terms; the
same along each gradient.  As 2-norms over a row (D values of one query or
key), with E = the largest score error of the call + 2^-22 (exponential, sums):
  o:  (2 E + u_s + u) max_k |v|      (p rounded to u_s for the second product)
  gradients, from dp = g v (|.| <= |g| max|v|) and ds = scale p (dp - delta):
  dq: scale 2 (2 E + 2 u_s + u32 n) 2 |g| max|v| max|k|  + u |dq|
  dk, dv: sums over the rows of the same, with p's own column of weights.
Written below in the row's own units; u is the storage type's roundoff, u_s
that of the rounded operands (u in 16 bits, u32 in fp32).  lse: E + 4 u32
(1 + |lse|)."""
import numpy as np
import pytest

from oracle import seq_oracle as so
from seq_util import TINY, U32, UNIT, code, host, stored, within

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lstm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from layer_lstm_amd import lstm as mod
    return mod


def rows_within(got, want, tol, what):
    """2-norms of the rows' errors against `tol` (one bound per row)."""
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert got.shape == want.shape and np.isfinite(got).all(), what
    err = np.linalg.norm(got - want, axis=-1)
    worst = float((err / np.maximum(tol, 1e-300)).max()) if err.size else 0.0
    assert worst <= 1.0, f"{what}: error {worst:.3g} times the bound"


def check(dt, q, k, v, do, scale, length, mask, o, lse, grads):
    """fp64 inputs as stored; o, lse, (dq, dk, dv) as fp64 host arrays."""
    want = so.attend(q, k, v, scale, length, mask, do)
    Tq, B, Hq, D = q.shape
    Tk, _, Hk, _ = k.shape
    G = Hq // Hk
    ok = so.valid_keys(Tk, B, length, mask)
    u, us = UNIT[dt], UNIT[dt]
    small = TINY[dt] * np.sqrt(D) * 2
    kz, vz = (np.where(ok.T[:, :, None, None], x, 0.0) for x in (k, v))
    nk, nv = (np.linalg.norm(x, axis=-1).max(0, initial=0).repeat(G, 1) for x in (kz, vz))  # [B, Hq]
    nq, ng = np.linalg.norm(q, axis=-1), np.linalg.norm(do, axis=-1)  # [Tq, B, Hq]
    E = (D + 2) * U32 * scale * nq * nk + 2.0**-22 * 4  # a score's error
    n = Tk * U32
    rows_within(o, want[0], (2 * E + n + us) * nv + 1.01 * u * np.linalg.norm(want[0], axis=-1) + small, "o")
    within(lse, want[1], np.moveaxis(E, 0, 2) + n + 4 * U32 * (1 + np.where(np.isfinite(want[1]), np.abs(want[1]), 0)),
           "lse")
    if grads is None:
        return
    # |error of ds| <= scale p (dp's and delta's errors + 2 (E + us) |dp - delta|), summed over keys with sum p = 1;
    # delta = g . o carries o's own rounding
    part = scale * (2 * (2 * E + us + n) + 2 * u) * 2 * ng * nv
    rows_within(grads[0], want[2], part * nk + 1.01 * u * np.linalg.norm(want[2], axis=-1) + small, "dq")
    # a key's gradient: the rows' errors weighted by p (of that key) and their own norms
    wk, wv = np.zeros((Tk, B, Hk)), np.zeros((Tk, B, Hk))
    for b in range(B):
        at = np.flatnonzero(ok[b])
        if at.size == 0:
            continue
        for h in range(Hq):
            s = scale * q[:, b, h] @ k[at, b, h // G].T
            p = np.exp(s - s.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            wk[at, b, h // G] += (part[:, b, h] * nq[:, b, h]) @ p
            wv[at, b, h // G] += ((2 * E[:, b, h] + us + Tq * G * U32) * ng[:, b, h]) @ p
    rows_within(grads[1], want[3], wk + 1.01 * u * np.linalg.norm(want[3], axis=-1) + small, "dk")
    rows_within(grads[2], want[4], wv + 1.01 * u * np.linalg.norm(want[4], axis=-1) + small, "dv")


def case(lstm, dt, Tq, Tk, B, Hq, Hk, D, length=None, mask=None, scale=None, seed=0, train=True, spread=1.0):
    print(f"case: attention {dt} Tq={Tq} Tk={Tk} B={B} heads {Hq}/{Hk} D={D} train={train}", flush=True)
    rng = np.random.default_rng(seed + Tk)
    scale = float(np.float32(D ** -0.5 if scale is None else scale))
    (q, q64), (g, g64) = (stored(torch, rng.normal(size=(Tq, B, Hq, D)) * spread, dt) for _ in range(2))
    (k, k64), (v, v64) = (stored(torch, rng.normal(size=(Tk, B, Hk, D)), dt) for _ in range(2))
    m = lstm.Attention(Tq, Tk, B, Hq, Hk, D, code(lstm, dt), scale=scale)
    m.o.fill_(float("nan")), m.lse.fill_(float("nan")), m.workspace.fill_(255)
    cl = None if length is None else torch.tensor(length, dtype=torch.int32, device="cuda")
    cm = None if mask is None else torch.from_numpy(mask).cuda()
    x = [t.cuda() for t in (q, k, v, g)]
    o, lse = m.forward(x[0], x[1], x[2], cl, cm)
    grads = None
    if train:
        m.dq = torch.full_like(x[0], float("nan"))
        m.dk, m.dv = (torch.full_like(x[1], float("nan")) for _ in range(2))
        grads = [host(t) for t in m.backward(x[3], x[0], x[1], x[2], cl, cm)]
        first = [t.clone() for t in (m.o, m.lse, m.dq, m.dk, m.dv)]
        m.forward(x[0], x[1], x[2], cl, cm), m.backward(x[3], x[0], x[1], x[2], cl, cm)
        assert all(torch.equal(a, b) for a, b in zip(first, (m.o, m.lse, m.dq, m.dk, m.dv)))
    torch.cuda.synchronize()
    check(dt, q64, k64, v64, g64, scale, length, mask, host(o), host(lse), grads)


def ragged(rng, B, Tk):
    n = rng.integers(0, Tk + 1, B)
    n[0], n[-1] = Tk, 0
    return n.tolist()


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("Tq,Tk,B,Hq,Hk,D", [
    (1, 1, 1, 1, 1, 8), (1, 1, 2, 1, 1, 1), (1, 33, 2, 4, 2, 64), (2, 31, 3, 3, 1, 32), (1, 700, 2, 8, 1, 128),
    (5, 64, 1, 2, 2, 40), (33, 65, 2, 2, 1, 96), (40, 129, 3, 6, 3, 80), (130, 70, 1, 1, 1, 64),
    (9, 300, 2, 2, 2, 192), (17, 100, 1, 4, 2, 256), (12, 45, 2, 2, 1, 33), (7, 40, 2, 2, 2, 250), (3, 20, 2, 1, 1, 130),
])
def test_sizes(lstm, dt, Tq, Tk, B, Hq, Hk, D):
    rng = np.random.default_rng(Tq)
    case(lstm, dt, Tq, Tk, B, Hq, Hk, D, length=ragged(rng, B, Tk) if B > 1 else None)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("D", [32, 64, 96, 128, 192, 256, 37])
def test_shared_tiles(lstm, dt, D):
    """Enough rows and sequences for the kernel whose waves share their tiles, in every head size it is built for."""
    B, Hk = (20, 8) if D != 37 else (16, 8)
    rng = np.random.default_rng(D)
    case(lstm, dt, 34, 140, B, Hk, Hk, D, length=ragged(rng, B, 140))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("Tq,B,Hq,Hk", [(1, 4, 4, 2), (50, 2, 2, 2), (40, 32, 8, 4)])
def test_key_masks(lstm, dt, Tq, B, Hq, Hk):
    """Holes, a sequence without a key, whole tiles masked, a mask beside lengths; bytes other than 1."""
    rng = np.random.default_rng(3)
    Tk = 260
    mask = (rng.random((B, Tk)) < 0.7).astype(np.uint8) * 255
    mask[1] = 0
    mask[0, 64:200] = 0
    case(lstm, dt, Tq, Tk, B, Hq, Hk, 64, mask=mask, length=rng.integers(1, Tk, B).tolist())
    case(lstm, dt, Tq, Tk, B, Hq, Hk, 72, mask=mask != 0)


def test_lengths_beyond_and_below(lstm):
    case(lstm, "bf16", 3, 50, 4, 2, 2, 64, length=[50, 1000, -3, 0])


@pytest.mark.parametrize("Tq", [1, 40])
def test_long_keys_split(lstm, Tq):
    case(lstm, "bf16", Tq, 5000, 1, 2, 1, 64, train=True)
    case(lstm, "f32", Tq, 3001, 2, 2, 2, 128, length=[3001, 77], train=Tq == 1)


def test_large_scores(lstm):
    """Scores in the hundreds, rising and falling along the keys: the reference moves, nothing overflows."""
    case(lstm, "f32", 40, 300, 2, 2, 2, 64, scale=4.0, spread=3.0)
    case(lstm, "bf16", 4, 300, 2, 2, 2, 64, scale=4.0, spread=3.0, train=False)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("Tq", [1, 140])
def test_what_lies_in_masked_places_is_not_read(lstm, dt, Tq):
    """NaN and infinities in the keys and values past the length and under the mask change no bit."""
    rng = np.random.default_rng(7)
    B, Tk, H, D = 2, 150, 2, 64
    k, v = (stored(torch, rng.normal(size=(Tk, B, H, D)), dt)[0].cuda() for _ in range(2))
    q, g = (stored(torch, rng.normal(size=(Tq, B, H, D)), dt)[0].cuda() for _ in range(2))
    mask = torch.from_numpy(rng.random((B, Tk)) < 0.8).cuda()
    length = torch.tensor([97, 0], dtype=torch.int32, device="cuda")
    gone = ~(mask & (torch.arange(Tk, device="cuda")[None] < length[:, None])).t()
    m = lstm.Attention(Tq, Tk, B, H, H, D, code(lstm, dt))
    runs = []
    for bad in (0.0, float("nan"), float("inf"), -float(torch.finfo(k.dtype).max)):
        kb, vb = k.clone(), v.clone()
        kb[gone], vb[gone] = bad, bad
        m.forward(q, kb, vb, length, mask)
        m.backward(g, q, kb, vb, length, mask)
        runs.append([t.clone() for t in (m.o, m.lse, m.dq, m.dk, m.dv)])
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(r, runs[0]))
    o, lse, dq, dk, dv = runs[0]
    assert not o[:, 1].any() and torch.isneginf(lse[1]).all() and not dq[:, 1].any()
    assert not dk[gone].any() and not dv[gone].any() and torch.isfinite(dq).all()


def test_strides_streams_and_broadcast_keys(lstm):
    """Heads first, rows of a wider tensor, keys shared by the batch (stride 0), a row out of line with 16 bytes."""
    rng = np.random.default_rng(8)
    Tq, Tk, B, H, D = 35, 90, 3, 2, 64
    s = torch.cuda.Stream()
    q, q64 = stored(torch, rng.normal(size=(B, H, Tq, D)), "bf16")
    g, g64 = stored(torch, rng.normal(size=(Tq, B, H, D + 8)), "bf16")
    k, k64 = stored(torch, rng.normal(size=(Tk, 1, H, D)), "bf16")
    v, v64 = stored(torch, rng.normal(size=(Tk, B, H, D + 1)), "bf16")
    m = lstm.Attention(Tq, Tk, B, H, H, D, lstm.BF16)
    qc, kc = q.cuda().permute(2, 0, 1, 3), k.cuda().expand(Tk, B, H, D)
    vc, gc = v.cuda()[..., 1:], g.cuda()[..., :D]
    torch.cuda.synchronize()
    o, lse = m.forward(qc, kc, vc, stream=s)
    grads = m.backward(gc, qc, kc, vc, stream=s)
    s.synchronize()
    check("bf16", q64.transpose(2, 0, 1, 3), np.broadcast_to(k64, (Tk, B, H, D)), v64[..., 1:], g64[..., :D],
          D ** -0.5, None, None, host(o), host(lse), [host(t) for t in grads])


def test_empty_dimensions(lstm):
    m = lstm.Attention(3, 0, 2, 2, 1, 16, lstm.F32)
    q, k = torch.randn(3, 2, 2, 16, device="cuda"), torch.empty(0, 2, 1, 16, device="cuda")
    o, lse = m.forward(q, k, k)
    dq, dk, dv = m.backward(q, q, k, k)
    assert not o.any() and torch.isneginf(lse).all() and not dq.any() and dk.shape == (0, 2, 1, 16)
    m = lstm.Attention(0, 4, 2, 2, 1, 16, lstm.F32)
    q, k = torch.empty(0, 2, 2, 16, device="cuda"), torch.randn(4, 2, 1, 16, device="cuda")
    assert m.forward(q, k, k)[0].shape == (0, 2, 2, 16)
    m.dq, m.dk, m.dv = q, torch.full_like(k, 7.0), torch.full_like(k, 7.0)
    _, dk, dv = m.backward(q, q, k, k)
    assert not dk.any() and not dv.any()
    m = lstm.Attention(2, 4, 0, 2, 1, 16, lstm.F32)
    e = torch.empty(2, 0, 2, 16, device="cuda")
    m.forward(e, torch.empty(4, 0, 1, 16, device="cuda"), torch.empty(4, 0, 1, 16, device="cuda"))


def test_graph_replays(lstm):
    T, B, H, D = 20, 4, 2, 64
    for Tq in (1, 20):
        m, ref = (lstm.Attention(Tq, 700, B, H, H, D, lstm.F16) for _ in range(2))
        q, g = (torch.randn(Tq, B, H, D, device="cuda", dtype=torch.float16) for _ in range(2))
        k, v = (torch.randn(700, B, H, D, device="cuda", dtype=torch.float16) for _ in range(2))
        n = torch.full((B,), 700, dtype=torch.int32, device="cuda")
        m.forward(q, k, v, n), m.backward(g, q, k, v, n)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            m.forward(q, k, v, n)
            m.backward(g, q, k, v, n)
        for _ in range(3):
            q.normal_(), k.normal_(), n.random_(0, 701)
            graph.replay()
            torch.cuda.synchronize()
            want = [*ref.forward(q, k, v, n), *ref.backward(g, q, k, v, n)]
            assert all(torch.equal(a, b) for a, b in zip((m.o, m.lse, m.dq, m.dk, m.dv), want))


def test_refusals(lstm):
    import ctypes
    base = dict(Tq=2, Tk=4, B=2, Hq=4, Hk=2, D=16, dtype=lstm.F32)
    for kw, rc in ((dict(Tq=-1), -2), (dict(Hk=3), -2), (dict(Hk=0), -2), (dict(D=0), -2), (dict(scale=0.0), -2),
                   (dict(scale=float("nan")), -2), (dict(dtype=9), -3), (dict(D=257), -6), (dict(Tk=1 << 26), -6)):
        with pytest.raises(lstm.LstmError) as e:
            lstm.Attention(**{**base, **kw})
        assert e.value.code == rc, kw
    m = lstm.Attention(**base)
    q, k = torch.randn(2, 2, 4, 16, device="cuda"), torch.randn(4, 2, 2, 16, device="cuda")
    n = torch.tensor([4, 4], dtype=torch.int32, device="cuda")
    for bad in ((q[:1], k, k), (q, k.half(), k), (q, k, k[:, :1]), (q.transpose(2, 3).contiguous().transpose(2, 3), k, k),
                (q, k, k, n.long()), (q, k, k, n[:1]), (q, k, k, n, torch.ones(2, 4, device="cuda")),
                (q, k, k, n, torch.ones(2, 5, device="cuda", dtype=torch.bool))):
        with pytest.raises(ValueError):
            m.forward(*bad)
    L, s, P = lstm.lib(), m.shape, lambda t: t.data_ptr()
    out, ws = torch.full_like(q, 7.0), m.workspace
    m.forward(q, k, k)
    fwd = lambda *a: L.lstm_attend_fwd(ctypes.byref(s), *a, None)  # noqa: E731
    assert fwd(None, P(k), P(k), None, None, P(ws), ws.numel(), P(out), P(m.lse)) == -1
    assert fwd(P(q), P(k), P(k), None, None, P(ws), ws.numel(), P(out), None) == -1
    assert fwd(P(q) + 2, P(k), P(k), None, None, P(ws), ws.numel(), P(out), P(m.lse)) == -4
    assert fwd(P(q), P(k), P(k), P(n) + 2, None, P(ws), ws.numel(), P(out), P(m.lse)) == -4
    bwd = lambda *a: L.lstm_attend_bwd(ctypes.byref(s), *a, None)  # noqa: E731
    assert bwd(P(q), P(q), P(k), P(k), None, None, P(m.o), P(m.lse), P(ws), 0, P(out), P(k), P(k)) == -5
    assert bwd(P(q), P(q), P(k), P(k), None, None, P(m.o), P(m.lse), P(ws) + 4, ws.numel(), P(out), P(k), P(k)) == -4
    s.o.h = 8  # overlapping rows of an output
    assert fwd(P(q), P(k), P(k), None, None, P(ws), ws.numel(), P(out), P(m.lse)) == -2
    s.o.h, s.q.t = 16, -1
    assert fwd(P(q), P(k), P(k), None, None, P(ws), ws.numel(), P(out), P(m.lse)) == -2
    torch.cuda.synchronize()
    assert (out == 7.0).all()


@pytest.mark.skip(reason="a run of this file with a variant of the fp16 backward, since taken out, faulted the GPU near "
                         "this case; the cause is not shown yet")
def test_fp16_probabilities_among_denormals(lstm):
    """p of about 2^-17 each, below fp16's normal numbers, where dv is a normal number: its error is p's rounding and
    its own, one unit each, and less than a third for the sums."""
    Tq, Tk, D = 16, 131072, 16
    rng = np.random.default_rng(3)
    q, q64 = stored(torch, rng.normal(size=(Tq, 1, 1, D)), "f16")
    k, k64 = stored(torch, rng.normal(size=(Tk, 1, 1, D)), "f16")
    v, v64 = stored(torch, rng.normal(size=(Tk, 1, 1, D)), "f16")
    g, g64 = stored(torch, 64 * rng.normal(size=(Tq, 1, 1, D)), "f16")
    m = lstm.Attention(Tq, Tk, 1, 1, 1, D, lstm.F16)
    m.forward(q, k, v)
    dv = host(m.backward(g, q, k, v)[2])
    want = so.attend(q64, k64, v64, D**-0.5, None, None, g64)[4]
    err = np.linalg.norm(dv - want) / np.linalg.norm(want)
    assert err <= 3 * UNIT["f16"], err
