"""The encoder-decoder example: its gradient against central differences of its
own loss, and that it learns and answers."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def seq2seq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from layer_lstm_amd import seq2seq as mod
    return mod


def test_gradient_by_differences(seq2seq):
    """Along each parameter's own gradient direction d = g / |g| the loss's
    slope is |g|.  fp32 losses of about 3 resolve 3e-7, so the slope 1e-5, and
    the step of 2e-2 has a truncation of about its square: within 2 % of |g|
    for |g| over 5e-4."""
    m = seq2seq.Seq2Seq(7, 5, 11, I=12, heads=2, head_dim=16, seed=3)
    g = torch.Generator(device="cuda").manual_seed(1)
    batch = seq2seq.make_batch(7, 5, 11, g)
    m.forward(*batch)
    grads = {k: v.clone() for k, v in m.backward().items()}
    m.enc.check(), m.dec.check()
    for k, d in grads.items():
        norm = float(d.double().norm())
        assert norm > 5e-4, k
        keep, step = m.p[k].clone(), 2e-2
        loss = []
        for sign in (1, -1):
            m.p[k].copy_(keep + sign * step * d / norm)
            loss.append(-float(m.forward(*batch)))
        m.p[k].copy_(keep)
        slope = (loss[0] - loss[1]) / (2 * step)
        assert abs(slope - norm) <= 0.02 * norm, (k, slope, norm)
    # the padding's row takes no gradient
    assert not grads["table"][seq2seq.PAD].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_learns_to_reverse(seq2seq, dtype):
    from layer_lstm_amd import lstm
    model, score = seq2seq.train(400, S=8, B=64, V=12, dtype=lstm.F32 if dtype == "f32" else lstm.BF16, log=50)
    right = seq2seq.accuracy(model)
    print("log probability", score, "right", right, flush=True)
    assert score > -0.3 and right > 0.9
