"""Linear attention's 16-bit results within the roundings that the kernels make
(linattn_bounds.py), and its states within those of fp32 sums."""
import numpy as np
import pytest

import linattn_bounds as lb
from oracle import model_oracle as mo
from seq_util import U32, host
from test_gpu_linattn import make, run

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lstm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from layer_lstm_amd import lstm as mod
    return mod


SIZES = [(1, 3, 6, 2, 17, 40), (8, 4, 10, 2, 80, 50), (9, 4, 2, 2, 8, 8), (31, 2, 2, 2, 32, 16), (33, 2, 4, 4, 128, 128),
         (65, 4, 6, 3, 80, 48), (97, 2, 8, 2, 200, 136), (100, 1, 5, 1, 37, 201), (130, 2, 2, 2, 256, 256), (300, 2, 3, 3, 129, 64),
         (600, 1, 2, 1, 64, 96), (2100, 2, 4, 2, 64, 64), (2100, 1, 2, 2, 64, 128),
         # as many heads as compute units, alone and shared, small rows and large ones
         (45, 70, 8, 8, 40, 64), (40, 64, 4, 4, 72, 80), (70, 64, 8, 4, 96, 128), (35, 40, 16, 8, 136, 200), (50, 140, 8, 4, 37, 51),
         (40, 32, 4, 2, 128, 128), (200, 64, 4, 4, 64, 64)]


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("T,B,Hq,Hk,D,Dv", SIZES)
def test_results(lstm, dt, T, B, Hq, Hk, D, Dv):
    print(f"case: linear attention's roundings {dt} T={T} B={B} heads {Hq}/{Hk} D={D} Dv={Dv}", flush=True)
    c, x = make(dt, T, B, Hq, Hk, D, Dv, seed=11)
    _, o, _, g = run(lstm, dt, c)
    lb.check(dt, dict(zip(("o", "dq", "dk", "dv"), (host(i) for i in (o, *g[:3])))), x, 0.37)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,B,Hq,Hk,D,Dv", [(96, 2, 4, 4, 64, 64), (96, 2, 4, 2, 128, 128), (96, 2, 2, 2, 50, 70), (96, 1, 4, 1, 256, 256),
                                            (96, 64, 8, 4, 64, 64), (96, 64, 8, 8, 128, 96), (1200, 1, 4, 2, 64, 64)])
def test_states(lstm, dt, T, B, Hq, Hk, D, Dv):
    """The last state and the first one's gradient are fp32 sums in every type: of the norm, u32 for each of a chunk's
    product and its matrix products (six at most), which add up in the square mean (sqrt(7 T / 32) < 17 for T = 1200), and
    a few for the powers and V's parts.  V in two bf16 numbers alone would be off by 2^-18: 64 u32."""
    c, x = make(dt, T, B, Hq, Hk, D, Dv, decays=[-0.05, -0.002, -0.3])
    _, _, S, g = run(lstm, dt, c)
    want = mo.linattn(x["q"], x["k"], x["v"], x["log_decay"], 0.37, x["state"], x["length"], x["do"], x["dstate"])
    for name, got, w in (("state", S, want[1]), ("dstate", g[3], want[5])):
        err = np.linalg.norm(host(got) - w) / np.linalg.norm(w)
        print(f"  {name}: {err / U32:.1f} u32", flush=True)
        assert err <= 24 * U32, name
