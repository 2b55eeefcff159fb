"""The logits' gradient on the GPU from the record that it reads, within its
own roundings.

From (m, ls) = record, log p = scale (x - m) - ls in one difference and one
fused multiply-add: d = u32 (|scale (x - m)| + |log p|).  p = exp(log p), the
square of a power of two, has relative d + u32 (2 |log p| + 12).  With G the sum
of K + 1 cotangents of given tokens, A that of their sizes and gH the cotangent
of the entropy H,
  value: scale p ((A + |gH| (|log p| + H)) (that + (4 + K) u32) + |gH| d)
and where a token of its own cotangents g has p > 1/2, by 1 - p = -expm1(log p),
  scale (A ((1 - p) (8 + K) u32 + p d) + |gH| p ((|log p| + H) 8 u32 + d)
         + (3 + K) u32 (A of the other tokens)),
else that of the value and 4 u32 scale |g|; then the storage type's rounding."""
import numpy as np
import pytest

from seq_util import TINY, U32, UNIT, code, host, stored, within

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lstm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from layer_lstm_amd import lstm as mod
    return mod


def check(lstm, dt, x, t, scale=1.0, top=0, gl=None, gh=None, gt=None):
    N, V = x.shape
    xs, x64 = stored(torch, x, dt)
    m = lstm.LogProb(N, V, code(lstm, dt), top=top, scale=scale)
    logits, targets = xs.cuda(), torch.from_numpy(np.asarray(t)).cuda()
    out = m.forward(logits, targets)
    cu = lambda a: None if a is None else torch.from_numpy(np.asarray(a, np.float32)).cuda()  # noqa: E731
    got = host(m.backward(logits, targets, cu(gl), cu(gh), cu(gt)))
    f = lambda a, *s: np.zeros(s) if a is None else np.asarray(a, np.float32).astype(np.float64)  # noqa: E731
    gl, gh, gt, scale = f(gl, N), f(gh, N)[:, None], f(gt, N, top), float(np.float32(scale))
    rec, H = host(m.record), host(m.entropy)[:, None]
    z = scale * (x64 - rec[:, :1])
    lp = z - rec[:, 1:]
    p = np.exp(lp)
    g, size = np.zeros((N, V)), np.zeros((N, V))
    real = (t >= 0) & (t < V)
    ids = out[3].cpu().numpy() if top else np.zeros((N, 0), np.int64)
    for a, by in ((g, lambda v: v), (size, np.abs)):
        a[np.flatnonzero(real), t[real]] += by(gl[real])
        np.add.at(a, (np.arange(N)[:, None], ids), by(gt))
    G, A = (gl * real + gt.sum(1))[:, None], (np.abs(gl) * real + np.abs(gt).sum(1))[:, None]
    with np.errstate(invalid="ignore"):
        rest = np.where(p > 0, gh * p * (lp + H), 0.0)
        want = scale * (np.where(p > 0.5, (g - G) - G * np.expm1(lp), g - p * G) - rest)  # neither cancels in 64 bits
        d = U32 * (np.abs(z) + np.abs(lp))
        err = p * ((A + np.abs(gh) * (np.abs(lp) + H)) * (d + U32 * (2 * np.abs(lp) + 16 + top)) + np.abs(gh) * d)
        own = A * (-np.expm1(lp) * (8 + top) * U32 + p * d) + np.abs(gh) * p * ((np.abs(lp) + H) * 8 * U32 + d) + \
            (3 + top) * U32 * (A - size)
    mine = np.zeros((N, V), bool)
    mine[np.flatnonzero(real), t[real]] = True
    np.put_along_axis(mine, ids, True, 1)
    err = scale * np.where(mine & (p > 0.5), own, np.where(p > 0, err, 0.0) + 4 * U32 * np.abs(g))
    worst = within(got, want, err + 1.01 * UNIT[dt] * np.abs(want) + TINY[dt] + 1e-38, "dlogits")
    print(f"  gradient: {worst:.2f} of the bound", flush=True)
    return x64, got


def confident(rng, N, V, q, dt):
    """Rows whose target has p = 1 - q, the other logits of a usual spread."""
    x, t = rng.normal(size=(N, V)), rng.integers(0, V, N)
    e = np.exp(x)
    e[np.arange(N), t] = 0
    x[np.arange(N), t] = np.log(e.sum(1) * (1 - q) / q)
    return x, t


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("V", [100, 5003])
@pytest.mark.parametrize("q", [1e-1, 1e-3, 1e-5, 1e-7])
def test_confident_targets(lstm, dt, V, q):
    rng = np.random.default_rng(V)
    print(f"case: logprob gradient {dt} V={V} 1-p={q}", flush=True)
    x, t = confident(rng, 8, V, q, dt)
    check(lstm, dt, x, t, gl=rng.normal(size=8))
    check(lstm, dt, x, t, gl=rng.normal(size=8), gh=rng.normal(size=8) * 0.01)
    check(lstm, dt, x / 0.7, t, 0.7, 3, gl=rng.normal(size=8), gt=rng.normal(size=(8, 3)))


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,V,top,scale,spread", [(3, 7, 2, 1.0, 1.0), (5, 1000, 0, 0.3, 0.01), (9, 10007, 5, 1.0, 3.0),
                                                  (2, 70001, 8, 2.0, 10.0)])
def test_flat_and_spread_rows(lstm, dt, N, V, top, scale, spread):
    print(f"case: logprob gradient {dt} {N} x {V} top {top} spread {spread}", flush=True)
    rng = np.random.default_rng(N + V)
    check(lstm, dt, rng.normal(size=(N, V)) * spread, rng.integers(-1, V + 1, N), scale, top, gl=rng.normal(size=N),
          gh=rng.normal(size=N), gt=rng.normal(size=(N, top)) if top else None)
