"""Log probabilities and entropies near 0 on the GPU, relative to themselves.

Where one token has nearly all of p, log p = -log1p(R) and the entropy R + ...
are sums R of small terms, in which nothing cancels: each 2^y has relative
u32 (|y| + 4), weighed by its share of R, and a lane adds V / 64 terms, the
joins a dozen more; log1p, the quotient and the differences add 8 u32."""
import numpy as np
import pytest

from oracle import seq_oracle as so
from seq_util import U32, code, host, stored

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lstm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from layer_lstm_amd import lstm as mod
    return mod


def confident(rng, N, V, q):
    """Rows whose target has p = 1 - q, the other logits of a usual spread."""
    x, t = rng.normal(size=(N, V)), rng.integers(0, V, N)
    e = np.exp(x)
    e[np.arange(N), t] = 0
    x[np.arange(N), t] = np.log(e.sum(1) * (1 - q) / q)
    return x, t


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,V", [(8, 100), (8, 5003), (3, 70001), (2100, 700)])
@pytest.mark.parametrize("q", [1e-1, 1e-3, 1e-5, 1e-7])
def test_log_p_and_entropy_keep_their_digits(lstm, dt, N, V, q):
    print(f"case: confident rows {dt} {N} x {V} 1-p={q}", flush=True)
    x, t = confident(np.random.default_rng(V), N, V, q)
    xs, x64 = stored(torch, x + 3.0, dt)
    m = lstm.LogProb(N, V, code(lstm, dt), scale=1.0)
    logp, H = (host(a) for a in m.forward(xs.cuda(), torch.from_numpy(t).cuda()))
    z = x64 - x64.max(1, keepdims=True)
    e = np.exp(z)
    e[np.arange(N), t] = 0
    R = e.sum(1)
    want = -np.log1p(R)
    wantH = np.log1p(R) - (e * z).sum(1) / (1 + R)
    np.testing.assert_allclose(so.logprob(x64, t)["logp"], want, rtol=1e-6)
    d = (e * (np.abs(z) * np.log2(np.e) + 4)).sum(1) / R * U32 + (V / 64 + 12 + 8) * U32
    assert (np.argmax(x64, 1) == t).all()
    worst = (np.abs(logp - want) / (d * np.abs(want))).max(), (np.abs(H - wantH) / (d * wantH)).max()
    print("  log p %.2f, entropy %.2f of the bound" % worst, flush=True)
    assert max(worst) <= 1


@pytest.mark.parametrize("dt", ["f32", "f16"])
def test_equal_maxima(lstm, dt):
    """c equal largest logits, wherever they are, beside much smaller ones: log p = -log c - R / c."""
    rng = np.random.default_rng(1)
    for V in (3, 64, 1000, 20000):
        for c in (1, 2, 3, V // 2, V):
            x = rng.normal(size=(4, V)) - 30
            for n in range(4):
                x[n, rng.choice(V, max(c, 1), replace=False)] = 2.5
            xs, x64 = stored(torch, x, dt)
            m = lstm.LogProb(4, V, code(lstm, dt))
            t = np.argmax(x64, 1)
            logp, H = (host(a) for a in m.forward(xs.cuda(), torch.from_numpy(t).cuda()))
            r = so.logprob(x64, t)
            np.testing.assert_allclose(logp, r["logp"], rtol=2e-6 + V / 64 * U32, atol=2e-12, err_msg=f"{V} {c}")
            np.testing.assert_allclose(H, r["entropy"], rtol=2e-6 + V / 64 * U32, atol=2e-11, err_msg=f"{V} {c}")
