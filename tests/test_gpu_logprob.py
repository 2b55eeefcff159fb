"""Log probabilities, entropy, best alternatives and the logits' gradient on
the GPU against fp64.

Bounds.  The sums: y = (x - m) scale log2 e has a relative error of 3 u32, so
2^y one of 3 |y| u32 + 2 u32; |y| <= 16 + log2 V carries weight, and V / 256
terms are added in a row per lane, a few dozen more in the joins:
  d = (V / 256 + 32 + 3 (17 + log2 V)) u32  relative, of both sums.
lse: d + 4 u32 (|m scale| + |lse| + 1).  logp, top_logp: the same once more for
x scale - lse.  entropy = log s - t / s with |t / s| <= 17 + log2 V: 3 d (18 +
log2 V).  Gradient: p carries the error e of log p and 3 u32 of the
exponential; every product 4 u32; then one rounding to the storage type."""
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


def bounds(x64, scale, r):
    V = max(x64.shape[1], 1)
    lg = np.log2(V)
    d = (V / 256 + 32 + 3 * (17 + lg)) * U32
    top = np.max(np.where(np.isfinite(x64), np.abs(x64), 0), axis=1, initial=0) * scale
    lse = np.where(np.isfinite(r["lse"]), np.abs(r["lse"]), 0)
    e = d + 4 * U32 * (top + lse + 1)
    return e, 2 * e, 3 * d * (18 + lg)


def check(lstm, dt, x, t, scale=1.0, top=0, grads=True, seed=0, ids=torch.int64 if torch else None, ld=None):
    """x: numpy [N, V]; through the class, every output and the gradient of every cotangent."""
    N, V = x.shape
    rng = np.random.default_rng(seed)
    xs, x64 = stored(torch, x, dt)
    dl, dh, dtop = rng.normal(size=N), rng.normal(size=N), rng.normal(size=(N, top))
    f32 = lambda a: np.asarray(a, np.float32).astype(np.float64)  # noqa: E731
    dl, dh, dtop = f32(dl), f32(dh), f32(dtop)
    scale = float(np.float32(scale))
    r = so.logprob(x64, t, scale, top, dl, dh, dtop)
    g = torch.zeros((N, ld or V), dtype=xs.dtype)
    g[:, :V] = xs
    logits = g.cuda()[:, :V]
    targets = torch.from_numpy(np.asarray(t)).to(ids).cuda()
    m = lstm.LogProb(N, V, code(lstm, dt), top=top, scale=scale)
    for b in (m.lse, m.logp, m.entropy, m.top_logp):
        b.fill_(float("nan"))
    out = m.forward(logits, targets)
    e, e2, eh = bounds(x64, scale, r)
    within(host(m.lse), r["lse"], e, "lse")
    within(host(out[0]), r["logp"], e2, "logp")
    within(host(out[1]), r["entropy"], eh, "entropy")
    if top:
        assert out[3].dtype == ids
        np.testing.assert_array_equal(out[3].cpu().numpy(), r["top_ids"])
        within(host(out[2]), r["top_logp"], e2[:, None], "top_logp")
    if grads:
        cu = lambda a: torch.from_numpy(a.astype(np.float32)).cuda()  # noqa: E731
        m.dlogits = torch.full((N, V), float("nan"), dtype=xs.dtype, device="cuda")
        got = m.backward(logits, targets, cu(dl), cu(dh), cu(dtop) if top else None)
        real = (np.asarray(t) >= 0) & (np.asarray(t) < V)
        with np.errstate(all="ignore"):
            z = x64 * scale - x64.max(1, keepdims=True) * scale
            lp = np.where(np.isneginf(x64) | np.isneginf(r["lse"])[:, None], -1000.0,
                          z - np.log(np.exp(z).sum(1, keepdims=True)))
        p = np.exp(lp)
        A = np.abs(dl) * real + np.abs(dtop).sum(1)
        H = r["entropy"][:, None]
        err = p * ((A[:, None] + np.abs(dh)[:, None] * (np.abs(lp) + H)) * (e2[:, None] + 12 * U32) +
                   np.abs(dh)[:, None] * (e2[:, None] + eh))
        own = np.zeros_like(p)
        own[np.arange(N)[real], np.asarray(t)[real]] = np.abs(dl[real])
        if top:
            np.add.at(own, (np.arange(N)[:, None], r["top_ids"]), np.abs(dtop))
        err = scale * (err + (top + 4) * U32 * own)
        within(host(got), r["dlogits"], err + 1.01 * UNIT[dt] * np.abs(r["dlogits"]) + TINY[dt] + 1e-37, "dlogits")
        again = got.clone()
        assert torch.equal(again, m.backward(logits, targets, cu(dl), cu(dh), cu(dtop) if top else None))
    return m, r


def targets_of(rng, N, V):
    t = rng.integers(0, V, N)
    t[::5] = -1
    t[3::7] = V
    return t


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,V,top,scale", [
    (1, 1, 1, 1.0), (1, 2, 0, 1.0), (3, 7, 7, 0.5), (2, 9, 3, 1.0), (5, 255, 32, 2.0), (4, 1025, 1, 1.0),
    (7, 10007, 5, 1.0), (1, 131072, 32, 0.8), (2, 100003, 8, 1.0), (1100, 513, 4, 1.0), (33, 4099, 20, 1.0),
])
def test_sizes(lstm, dt, N, V, top, scale):
    print(f"case: logprob {dt} N={N} V={V} top={top}", flush=True)
    rng = np.random.default_rng(V + N)
    check(lstm, dt, rng.normal(size=(N, V)) * 3, targets_of(rng, N, V), scale, top, seed=V)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("V", [300, 20000])
def test_banned_tokens_and_rows_of_nothing(lstm, dt, V):
    """-inf logits; a row of nothing else; one finite logit; the type's lowest value in place of -inf."""
    rng = np.random.default_rng(11)
    x = rng.normal(size=(6, V)) * 2
    x[0, rng.random(V) < 0.5] = -np.inf
    x[1] = -np.inf
    x[2, : V - 1] = -np.inf
    lowest = -float(torch.finfo(torch.bfloat16 if dt == "bf16" else torch.float32).max)
    x[3, rng.random(V) < 0.9] = lowest
    x[4] = lowest
    x[5, 5:] = -np.inf
    check(lstm, dt, x, np.array([3, 4, V - 1, 7, 9, V - 2]), 1.0, 8)


@pytest.mark.parametrize("V", [64, 5000, 50000])
def test_ties_go_to_the_lower_id(lstm, V):
    rng = np.random.default_rng(4)
    x = np.stack([np.zeros(V), np.round(rng.normal(size=V)), np.arange(V) * 0.01, -np.arange(V) * 0.01,
                  np.where(np.arange(V) % 2, 0.0, -0.0)])
    check(lstm, "f32", x, np.zeros(5, np.int64), 1.0, 20)


def test_growing_rows_move_the_reference(lstm):
    """Logits that rise by far more than a power of two 16 along the row, and extreme scales."""
    x = np.stack([np.linspace(-400, 400, 9000), np.linspace(400, -400, 9000), 1e4 * np.sin(np.arange(9000.0))])
    check(lstm, "f32", x, np.array([8999, 0, 5]), 1.0, 4)
    check(lstm, "f32", x, np.array([8999, 0, 5]), 1e-3, 4)


def test_nan_and_inf_stay_in_their_rows(lstm):
    x = torch.randn(4, 3000, device="cuda")
    x[1, 77], x[2, 5] = float("nan"), float("inf")
    m = lstm.LogProb(4, 3000, lstm.F32, top=4)
    t = torch.tensor([1, 2, 3, 4], device="cuda")
    ones = torch.ones(4, device="cuda")
    logp, H, tl, ids = m.forward(x, t)
    g = m.backward(x, t, ones, ones)
    for bad in (1, 2):
        assert torch.isnan(logp[bad]) and torch.isnan(H[bad]) and torch.isnan(g[bad]).any()
    for good in (0, 3):
        assert torch.isfinite(logp[good]) and torch.isfinite(H[good]) and torch.isfinite(g[good]).all()
    assert ((ids >= 0) & (ids < 3000)).all()


@pytest.mark.parametrize("dt,V,ld", [("bf16", 1000, 1003), ("f32", 999, 1024), ("f16", 4097, 4104)])
def test_strided_rows_and_int32(lstm, dt, V, ld):
    rng = np.random.default_rng(6)
    check(lstm, dt, rng.normal(size=(9, V)), targets_of(rng, 9, V), 1.0, 3, ids=torch.int32, ld=ld)


def test_gradient_in_place_and_each_cotangent_alone(lstm):
    rng = np.random.default_rng(9)
    N, V, top = 6, 30011, 3
    x, x64 = stored(torch, rng.normal(size=(N, V)), "f32")
    t = targets_of(rng, N, V)
    tg = torch.from_numpy(t).cuda()
    m = lstm.LogProb(N, V, lstm.F32, top=top)
    one, tops = torch.ones(N, device="cuda"), torch.ones(N, top, device="cuda")
    for k in range(4):
        logits = x.cuda()
        m.forward(logits, tg)
        m.dlogits = logits  # in place
        args = [one if k in (0, 3) else None, one if k in (1, 3) else None, tops if k in (2, 3) else None]
        got = host(m.backward(logits, tg, *args))
        h = [None if a is None else host(a) for a in args]
        want = so.logprob(x64, t, 1.0, top, *h)["dlogits"]
        within(got, want, 2e-5 * np.abs(want) + 1e-9, f"cotangent {k}")


def test_other_stream_graph_and_no_rows(lstm):
    N, V = 20, 40000
    m, ref = lstm.LogProb(N, V, lstm.BF16, top=6), lstm.LogProb(N, V, lstm.BF16, top=6)
    x = torch.zeros(N, V, dtype=torch.bfloat16, device="cuda")
    t = torch.zeros(N, dtype=torch.int64, device="cuda")
    one = torch.ones(N, device="cuda")
    m.forward(x, t), m.backward(x, t, one)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.forward(x, t)
        m.backward(x, t, one, one)
    s = torch.cuda.Stream()
    for k in range(3):
        x.normal_()
        t.random_(0, V)
        g.replay()
        torch.cuda.synchronize()
        out = ref.forward(x, t, stream=s)
        grad = ref.backward(x, t, one, one, stream=s)
        s.synchronize()
        for a, b in zip((m.logp, m.entropy, m.top_logp, m.top_ids, m.dlogits), (*out, grad)):
            assert torch.equal(a, b)
    e = lstm.LogProb(0, 5, lstm.F32)
    et = torch.empty(0, dtype=torch.int64, device="cuda")
    assert e.forward(torch.empty(0, 5, device="cuda"), et)[0].shape == (0,)
    z = lstm.LogProb(2, 0, lstm.F32)
    logp, H = z.forward(torch.empty(2, 0, device="cuda"), torch.tensor([0, -1], device="cuda"))
    assert not logp.any() and not H.any() and torch.isneginf(z.lse).all()


def test_refusals(lstm):
    import ctypes
    e = lstm.LstmError
    for kw in (dict(N=-1), dict(V=-1), dict(top=33), dict(top=6), dict(top=-1), dict(scale=0.0), dict(scale=-1.0),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(dtype=3)):
        with pytest.raises(e):
            lstm.LogProb(**{**dict(N=4, V=5, dtype=lstm.F32), **kw})
    m = lstm.LogProb(4, 5, lstm.F32, top=2)
    x, t = torch.zeros(4, 5, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    for bx, bt in ((x[:3], t), (x.half(), t), (x.t().contiguous().t(), t), (x, t.float()), (x, t[:2])):
        with pytest.raises(ValueError):
            m.forward(bx, bt)
    m.forward(x, t)
    with pytest.raises(ValueError):
        m.backward(x, t, torch.zeros(5, device="cuda"))
    with pytest.raises(ValueError):
        m.backward(x, t, None, None, torch.zeros(4, 3, device="cuda"))
    L, s, P = lstm.lib(), m.shape, lambda a: a.data_ptr()
    out = torch.full((4, 5), 7.0, device="cuda")
    none = [None] * 4
    assert L.lstm_logprob_fwd(ctypes.byref(s), P(x), None, None, 0, P(m.record), None, P(m.logp), None, P(m.top_logp),
                              P(m.top_ids), None) == -1
    assert L.lstm_logprob_fwd(ctypes.byref(s), P(x), P(t), None, 0, None, None, *none, None) == -1
    assert L.lstm_logprob_fwd(ctypes.byref(s), P(x) + 2, P(t), None, 0, P(m.record), None, None, None, P(m.top_logp),
                              P(m.top_ids), None) == -4
    assert L.lstm_logprob_bwd(ctypes.byref(s), P(x), P(t), P(m.record), None, None, None, P(m.lse), None, P(out),
                              None) == -1
    s.ld_grad = 4
    assert L.lstm_logprob_bwd(ctypes.byref(s), P(x), P(t), P(m.record), None, None, P(m.lse), None, None, P(out),
                              None) == -2
    big = lstm.LogprobShape(16, 131072, 131072, 131072, 1.0, 2, lstm.F32, lstm.I64)
    n = ctypes.c_size_t(0)
    assert L.lstm_logprob_query(ctypes.byref(big), ctypes.byref(n)) == 0 and n.value > 0
    assert L.lstm_logprob_fwd(ctypes.byref(big), P(x), P(t), P(out), n.value - 1, P(m.record), None, None, None, P(m.top_logp),
                              P(m.top_ids), None) in (-4, -5)
    torch.cuda.synchronize()
    assert (out == 7.0).all()
