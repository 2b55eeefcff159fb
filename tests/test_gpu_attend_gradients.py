"""Cross attention's results against fp64 within what their own roundings
account for (attend_bounds.py)."""
import numpy as np
import pytest

import attend_bounds as ab
from seq_util import UNIT, code, host
from test_attend_bounds import SIZES, inputs

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lstm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from layer_lstm_amd import lstm as mod
    return mod


def run(lstm, dt, size, dout=1.0, seed=0):
    print(f"case: attention gradients {dt} {size} dout {dout}", flush=True)
    Tq, Tk, B, Hq, Hk, D = size
    x, x64 = inputs(dt, *size, seed=seed, dout=dout)
    q, k, v, g = (t.cuda() for t in x)
    m = lstm.Attention(Tq, Tk, B, Hq, Hk, D, code(lstm, dt))
    o, _ = m.forward(q, k, v)
    got = dict(zip(("o", "dq", "dk", "dv"), (host(t) for t in (o, *m.backward(g, q, k, v)))))
    ab.check(dt, got, *x64, m.shape.scale)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("size", [s for s in SIZES if s[1] < 5000])
def test_gradients(lstm, dt, size):
    run(lstm, dt, size)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("D", [32, 64, 96, 128, 192, 256, 37])
def test_gradients_of_shared_tiles(lstm, dt, D):
    """Enough rows and sequences for the kernels whose waves share their tiles, in every head size."""
    run(lstm, dt, (34, 140, 20, 8, 8, D))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("size", [s for s in SIZES if s[1] >= 5000] + [(300, 4096, 2, 2, 2, 128)])
def test_gradients_over_thousands_of_keys(lstm, dt, size):
    run(lstm, dt, size)


@pytest.mark.parametrize("dt,dout", [("f32", 1.0), ("bf16", 1.0), ("f16", 1.0), ("f16", 8000.0)])
@pytest.mark.parametrize("size", [(5, 200, 4, 6, 2, 64), (40, 150, 40, 8, 4, 128), (130, 90, 3, 2, 2, 40)])
def test_gradients_of_ragged_and_masked_keys(lstm, dt, dout, size):
    """Lengths from none to all, holes, a sequence whose mask leaves nothing; NaN in every place that is no key."""
    print(f"case: attention gradients, masked, {dt} {size} dout {dout}", flush=True)
    Tq, Tk, B, Hq, Hk, D = size
    rng = np.random.default_rng(Tk)
    x, x64 = inputs(dt, *size, dout=dout)
    length, mask = rng.integers(0, Tk + 1, B), rng.random((B, Tk)) < 0.8
    length[0], length[1], mask[2] = Tk, 0, False
    gone = torch.from_numpy(~(mask & (np.arange(Tk) < length[:, None]))).T
    k, v = x[1].clone(), x[2].clone()
    k[gone], v[gone] = float("nan"), float("nan")
    q, k, v, g = (t.cuda() for t in (x[0], k, v, x[3]))
    n, holes = torch.from_numpy(length.astype(np.int32)).cuda(), torch.from_numpy(mask).cuda()
    m = lstm.Attention(Tq, Tk, B, Hq, Hk, D, code(lstm, dt))
    o, _ = m.forward(q, k, v, n, holes)
    got = dict(zip(("o", "dq", "dk", "dv"), (host(t) for t in (o, *m.backward(g, q, k, v, n, holes)))))
    ab.check(dt, got, *x64, m.shape.scale, length, mask)


@pytest.mark.parametrize("dout", [3e-4, 12000.0])
@pytest.mark.parametrize("size", [(32, 16, 1, 1, 1, 128), (60, 48, 3, 4, 2, 64), (40, 300, 20, 8, 8, 192), (34, 70, 20, 8, 8, 256),
                                  (5, 33, 2, 2, 1, 250), (600, 90, 1, 3, 3, 128)])
def test_fp16_gradients_at_the_ends_of_the_range(lstm, size, dout):
    """dout as a scaled loss brings it, so large that p (dp - delta) passes fp16's largest number where the gradients
    do not, and so small that it falls among the denormals where they do not."""
    x64 = inputs("f16", *size, dout=dout)[1]
    want = ab.results("f16", *x64, size[-1] ** -0.5)[0]
    big = {n: abs(want[n]).max() for n in ("dq", "dk", "dv")}
    assert all(b < 60000 for b in big.values()), big
    run(lstm, "f16", size, dout)


def test_fp16_gradients_that_grow_and_shrink_along_the_sum(lstm):
    """Rows of dout over eight powers of ten, rising and falling along the rows and the keys' values alike."""
    size = (256, 512, 1, 2, 2, 64)
    x, x64 = inputs("f16", *size)
    for name, n, turn in (("rise", 1, False), ("fall", 1, True)):
        by = [10.0 ** (-4 + 8 * i / 255) for i in range(256)]
        at = torch.tensor(by[::-1] if turn else by)[:, None, None, None]
        vat = torch.logspace(-3, 0, 512)[:, None, None, None]
        g, v = (x[3].float() * at / 4).half(), (x[2].float() * (vat.flip(0) if turn else vat)).half()
        c = [t.cuda() for t in (x[0], x[1], v, g)]
        m = lstm.Attention(256, 512, 1, 2, 2, 64, lstm.F16)
        o, _ = m.forward(*c[:3])
        got = dict(zip(("o", "dq", "dk", "dv"), (host(t) for t in (o, *m.backward(c[3], *c[:3])))))
        print(name, flush=True)
        ab.check("f16", got, x64[0], x64[1], v.double().numpy(), g.double().numpy(), m.shape.scale)


@pytest.mark.parametrize("size", [s for s in SIZES if s[1] >= 5000] + [(300, 4096, 2, 2, 2, 128), (64, 4096, 1, 1, 1, 64)])
@pytest.mark.parametrize("dout", [0.01, 1.0, 100.0])
def test_fp16_gradients_over_thousands_of_keys(lstm, size, dout):
    run(lstm, "f16", size, dout)


def test_fp16_probabilities_of_millionths(lstm):
    """p of about 2^-17 each, below fp16's normal numbers, where dv is a normal number: its error is p's rounding and
    its own, one unit each, and less than a third for the sums."""
    Tq, Tk, D = 16, 131072, 16
    x, x64 = inputs("f16", Tq, Tk, 1, 1, 1, D, dout=64.0)
    q, k, v, g = (t.cuda() for t in x)
    m = lstm.Attention(Tq, Tk, 1, 1, 1, D, lstm.F16)
    m.forward(q, k, v)
    dv = host(m.backward(g, q, k, v)[2])
    want = ab.results("f16", *x64, m.shape.scale)[0]["dv"]
    assert np.linalg.norm(dv - want) <= 3 * UNIT["f16"] * np.linalg.norm(want)


@pytest.mark.parametrize("B,Tq", [(1, 1), (130, 33)])
def test_fp16_small_probabilities_beside_a_large_one(lstm, B, Tq):
    """One key of value 0 with nearly all of p, the others of value 1 with p of 2^-14 to 2^-20 each: o is their share,
    whose error is p's rounding and its own, half a unit each, and less than a quarter for the sums."""
    Tk, D = 1500, 16
    k, v = torch.zeros(Tk, B, 1, D), torch.ones(Tk, B, 1, D)
    k[0], v[0] = 1.0, 0.0
    q, k, v = (t.half().cuda() for t in (torch.ones(Tq, B, 1, D), k, v))
    for lower in (14.3, 15.6, 16.7, 17.6, 18.6, 19.7, 20.4):
        scale = float(np.float32(lower * np.log(2) / D))
        o, _ = lstm.Attention(Tq, Tk, B, 1, 1, D, lstm.F16, scale=scale).forward(q, k, v)
        rest = (Tk - 1) * np.exp(-scale * D)
        want = rest / (1 + rest)
        assert (abs(host(o) - want) <= 1.25 * UNIT["f16"] * want + 2.0**-25).all(), lower
