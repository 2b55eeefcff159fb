"""Cross attention's results against fp64 within what their own roundings
account for (attend_bounds.py)."""
import pytest

import attend_bounds as ab
from seq_util import code, host
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
