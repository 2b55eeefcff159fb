"""Penalties, biases and masks on logits on the GPU against fp64.

Bound, element by element: at most five fp32 operations (division or product,
product and sum of the penalties, two sums) of values up to the sum of their
sizes s, 5 u32 s, then one rounding to the storage type."""
import numpy as np
import pytest

from oracle import model_oracle as mo
from seq_util import TINY, U32, UNIT, code, host, stored, tdtype, within

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lstm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from layer_lstm_amd import lstm as mod
    return mod


def pack_mask(allowed, words):
    N, V = allowed.shape
    bits = np.zeros((N, words * 32), bool)
    bits[:, :V] = allowed
    return (bits.reshape(N, words, 32).astype(np.uint64) << np.arange(32, dtype=np.uint64)).sum(2).astype(np.uint32)


def make(N, V, L, seed=0, ids=np.int64):
    r = np.random.default_rng(seed + N + V + L)
    history = np.minimum(np.exp(r.random((N, L)) * np.log(V + 1)).astype(ids) - 1, V)  # V: outside
    if L:
        history[r.random((N, L)) < 0.05] = -1
    length = r.integers(0, L + 1, N)
    length[: min(N, 3)] = [L + 7, 0, -4][: min(N, 3)]
    f = lambda a: a.astype(np.float32)  # noqa: E731
    allowed = r.random((N, V)) < 0.4
    allowed[N // 2] = False  # a row without a token
    return dict(x=r.normal(size=(N, V)) * 3, history=history, length=length.astype(np.int32),
                repetition=f(r.uniform(0.7, 1.6, N)), presence=f(r.normal(size=N)), frequency=f(r.normal(size=N) * 0.3),
                bias=f(r.normal(size=V)), biases=f(r.normal(size=(N, V))), allowed=allowed)


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def check(got, x, d, use, dt, bias=None):
    g = {k: d[k].astype(np.float64) if k in use else None for k in ("repetition", "presence", "frequency")}
    want = mo.penalty(x, d["history"], np.maximum(d["length"], 0), bias=bias, allowed=d["allowed"] if "mask" in use else None, **g)
    c = max(1, d["history"].shape[1])
    size = abs(x) * 1.6 + abs(x) / 0.7 + abs(d["presence"])[:, None] + c * abs(d["frequency"])[:, None] + (0 if bias is None else abs(bias))
    fin = np.where(np.isfinite(want), abs(want), 0)
    within(got, want, 5 * U32 * size + UNIT[dt] * 1.01 * fin + TINY[dt], "penalised")


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,V,L", [(1, 1, 1), (1, 5, 0), (3, 31, 4), (4, 32, 9), (5, 33, 40), (2, 1000, 100), (7, 2047, 300),
                                   (7, 2049, 3000), (3, 10007, 64), (40, 8193, 257), (300, 9999, 33), (2, 131072, 500)])
def test_penalties(lstm, dt, N, V, L):
    print(f"case: penalty {dt} N={N} V={V} L={L}", flush=True)
    d = make(N, V, L)
    xs, x = stored(torch, d["x"], dt)
    m = lstm.Penalty(N, V, code(lstm, dt))
    words = (V + 31) // 32
    mask = torch.from_numpy(pack_mask(d["allowed"], words).view(np.int32)).cuda()
    hist = dev(d["history"])
    args = [dev(d[k]) for k in ("length", "repetition", "presence", "frequency")]
    got = m.forward(xs.cuda(), hist, *args, dev(d["bias"]), mask)
    check(host(got), x, d, ("repetition", "presence", "frequency", "mask"), dt, d["bias"].astype(np.float64))
    # time-major 32-bit ids, a bias a row, in place in rows further apart than they are long
    wide = torch.full((N, V + 5), 7.0, dtype=tdtype(torch, dt), device="cuda")
    wide[:, 3 : V + 3] = xs.cuda()
    view = wide[:, 3 : V + 3]
    tm = hist.to(torch.int32).t().contiguous().t()
    assert m.forward(view, tm, *args, dev(d["biases"]), out=view) is view
    check(host(view), x, d, ("repetition", "presence", "frequency"), dt, d["biases"].astype(np.float64))
    assert bool((wide[:, :3] == 7).all()) and bool((wide[:, V + 3 :] == 7).all())
    # one of them at a time, the mask's words further apart
    wmask = torch.cat([mask, torch.full((N, 2), -1, dtype=torch.int32, device="cuda")], 1)
    check(host(m.forward(xs.cuda(), hist, args[0], repetition=args[1])), x, d, ("repetition",), dt)
    check(host(m.forward(xs.cuda(), hist, args[0], presence=args[2])), x, d, ("presence",), dt)
    check(host(m.forward(xs.cuda(), hist, args[0], frequency=args[3], mask=wmask)), x, d, ("frequency", "mask"), dt)
    check(host(m.forward(xs.cuda(), mask=mask)), x, d, ("mask",), dt)
    assert torch.equal(m.forward(xs.cuda()), xs.cuda())


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_values_that_are_no_numbers(lstm, dt):
    """NaN and infinities, masked and not, said and not; the type's lowest value; -0."""
    low = torch.finfo(tdtype(torch, dt)).min
    row = torch.tensor([float("nan"), float("inf"), float("-inf"), low, -0.0, 1.0] * 2, dtype=tdtype(torch, dt), device="cuda")
    x = row.repeat(2, 1)
    said = torch.arange(6, device="cuda").repeat(2, 1)  # the first half
    two = torch.full((2,), 2.0, device="cuda")
    m = lstm.Penalty(2, 12, code(lstm, dt))
    got = m.forward(x, said, repetition=two).float().cpu()
    assert torch.isnan(got[:, 0]).all() and torch.isnan(got[:, 6]).all()
    assert (got[:, 1] == float("inf")).all() and (got[:, 2] == float("-inf")).all() and (got[:, 3] == float("-inf")).all()
    assert (got[:, 4] == 0).all() and (got[:, 5] == 0.5).all() and torch.equal(got[0, 7:], row[7:].float().cpu())
    none = torch.zeros(2, 1, dtype=torch.int32, device="cuda")
    assert (m.forward(x, said, repetition=two, mask=none) == float("-inf")).all()


def test_one_token_many_times(lstm):
    """Every count is a whole number: 200000 times the same one, next to tokens said once."""
    N, V, L = 2, 5000, 200003
    h = torch.full((N, L), 4999, dtype=torch.int64, device="cuda")
    h[:, :3] = torch.tensor([0, 2048, 4998], device="cuda")
    m = lstm.Penalty(N, V)
    f = torch.full((N,), 0.5, device="cuda")
    got = m.forward(torch.zeros(N, V, device="cuda"), h, frequency=f)
    want = torch.zeros(N, V, device="cuda")
    want[:, [0, 2048, 4998]], want[:, 4999] = -0.5, -100000.0
    assert torch.equal(got, want)


def test_offsets_past_32_bits(lstm):
    V, ld = 40, (1 << 31) + 8
    big = torch.zeros(ld + V, dtype=torch.float16, device="cuda")
    x = big.as_strided((2, V), (ld, 1))
    x.copy_(torch.randn(2, V, device="cuda"))
    keep = x.clone()
    bias = torch.randn(V, device="cuda")
    lstm.Penalty(2, V, lstm.F16).forward(x, bias=bias, out=x)
    assert torch.equal(x, (keep.float() + bias).half())


def test_streams_graphs_and_empty_calls(lstm):
    N, V, L = 6, 3001, 50
    d = make(N, V, L)
    x = torch.from_numpy(d["x"]).float().cuda()
    args = [dev(d[k]) for k in ("history", "length", "repetition", "presence", "frequency", "bias")]
    m = lstm.Penalty(N, V)
    want = m.forward(x, *args).clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    m2 = lstm.Penalty(N, V)
    got = m2.forward(x, *args, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.forward(x, *args)
    for k in range(3):
        x.mul_(-1.5)
        want = m2.forward(x, *args).clone()
        m.out.fill_(7)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(m.out, want)
    for n, v in ((0, 5), (5, 0)):
        assert lstm.Penalty(n, v).forward(torch.empty(n, v, device="cuda")).shape == (n, v)


def test_refusals(lstm):
    N, V, L = 4, 40, 6
    d = make(N, V, L)
    x = torch.from_numpy(d["x"]).float().cuda()
    args = [x] + [dev(d[k]) for k in ("history", "length", "repetition", "presence", "frequency", "bias")] + [
        torch.zeros(N, 2, dtype=torch.int32, device="cuda")]
    m = lstm.Penalty(N, V)
    m.forward(*args)
    for i in range(len(args)):
        with pytest.raises(ValueError, match="cuda:0"):
            m.forward(*(a.cpu() if j == i else a for j, a in enumerate(args)))
    import ctypes
    s, p = m.shape, x.data_ptr()
    s.ld_bias = 3
    assert lstm.lib().lstm_penalty(ctypes.byref(s), p, None, None, None, None, None, p, None, p, None) == -2
    s.ld_bias, s.ld_mask = 0, 1
    assert lstm.lib().lstm_penalty(ctypes.byref(s), p, None, None, None, None, None, None, p, p, None) == -2
    s.ld_mask, s.ld_out = 2, V + 8
    assert lstm.lib().lstm_penalty(ctypes.byref(s), p, None, None, None, None, None, None, None, p, None) == -2
    s.ld_out = V
    assert lstm.lib().lstm_penalty(ctypes.byref(s), p + 2, None, None, None, None, None, None, None, p, None) == -4
    assert lstm.lib().lstm_penalty(ctypes.byref(s), p, None, None, p, None, None, None, None, p, None) == -1
    torch.cuda.synchronize()
