"""The encoder-decoder's step by the library's optimiser: every parameter moves
by its own gradient, as the formula has it."""
import numpy as np
import pytest

from oracle import model_oracle as mo
from seq_util import TINY, U32, UNIT, host, within

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def seq2seq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from layer_lstm_amd import seq2seq as mod
    return mod


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("kind,clip", [("adamw", None), ("adamw", 0.05), ("adamw8", None), ("adamw8", 0.05)])
def test_parameters_move_by_their_own_gradients(seq2seq, dt, kind, clip):
    """Three steps from states of zeros.  The first: m and v are the gradient's alone, so each weight moves by lr (decay w +
    g / (|g| + eps)), 3 u32 |w| and 16 u32 of the move (test_gpu_adamw.py); with 32-bit states the next two follow the
    formula from the fp64 m and v, whose errors add as many again each."""
    from layer_lstm_amd import lstm
    model = seq2seq.Seq2Seq(7, 5, 11, I=12, heads=2, head_dim=16, seed=3, memory=True, dtype=lstm.F32 if dt == "f32" else lstm.BF16)
    opt = seq2seq.make_optimizer(kind, model.p, clip)
    o = opt.opt
    lr, (b1, b2) = o.lr, o.betas
    states = {k: (np.zeros(p.numel()), np.zeros(p.numel())) for k, p in model.p.items()}

    def weights():
        if dt == "f32":
            return {k: host(p).reshape(-1) for k, p in model.p.items()}
        return {k: host(o.master[at : at + model.p[k].numel()]) for k, at in zip(opt.names, o.places)}

    for t in range(1, 4 if kind == "adamw" else 2):
        model.forward(*seq2seq.make_batch(7, 5, 11, torch.Generator(device="cuda").manual_seed(t)))
        grads = {k: v.clone() for k, v in model.backward().items()}
        g = {k: host(v).reshape(-1) for k, v in grads.items()}
        norm = np.sqrt(sum((x**2).sum() for x in g.values()))
        scale = 1.0 if clip is None else min(1.0, clip / norm)
        before = weights()
        opt.step(model.p, grads)
        after = weights()
        for k in model.p:
            assert np.abs(g[k]).max() > 0, k
            m, v = states[k]
            x = g[k] * scale
            w, m, v = mo.adamw(before[k], x, m, v, t, lr, b1, b2, 1e-8, 0.01)
            states[k] = m, v
            move = lr * (abs(b1 * m) + (1 - b1) * abs(x)) / (1 - b1**t) / (np.sqrt(v / (1 - b2**t)) + 1e-8)
            tol = 3 * U32 * abs(before[k]) + 16 * t * U32 * np.maximum(move, lr) + TINY["f32"]
            within(after[k], w, tol, f"{k}, step {t}")
            if dt != "f32":
                within(host(model.p[k]).reshape(-1), w, tol + UNIT[dt] * 1.01 * abs(w) + TINY[dt], f"{k}, step {t}, stored")
