"""The encoder-decoder with linear attention over its own steps, the library's
optimiser and constrained answers: its gradients against differences, its single
steps against whole sequences, and that training and answering run."""
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
    """Along each parameter's own gradient direction d = g / |g| the loss's slope is |g|.  fp32 losses of about 3 resolve
    3e-7, so the slope 1e-5, and the step of 2e-2 has a truncation of about its square: within 2 % of |g| for |g| over
    5e-4."""
    m = seq2seq.Seq2Seq(7, 5, 11, I=12, heads=2, head_dim=16, seed=3, memory=True)
    batch = seq2seq.make_batch(7, 5, 11, torch.Generator(device="cuda").manual_seed(1))
    m.forward(*batch)
    grads = {k: v.clone() for k, v in m.backward().items()}
    m.enc.check(), m.dec.check()
    for k, d in grads.items():
        norm = float(d.double().norm())
        assert norm > 5e-4, k
        keep, step, loss = m.p[k].clone(), 2e-2, []
        for sign in (1, -1):
            m.p[k].copy_(keep + sign * step * d / norm)
            loss.append(-float(m.forward(*batch)))
        m.p[k].copy_(keep)
        slope = (loss[0] - loss[1]) / (2 * step)
        assert abs(slope - norm) <= 0.02 * norm, (k, slope, norm)


@pytest.mark.parametrize("memory", [False, True])
def test_single_steps_follow_the_whole_sequence(seq2seq, memory):
    """The tokens that the steps choose are the largest logits of the whole sequence fed with them.  The two sum the same
    fp32 products in different orders: logits of about 1 differ by less than 1e-4, so a chosen one is within that of the
    row's largest."""
    S, B, V = 12, 6, 40
    m = seq2seq.Seq2Seq(S, B, V, I=16, heads=2, head_dim=32, seed=5, memory=memory)
    source, _, targets, length = seq2seq.make_batch(S, B, V, torch.Generator(device="cuda").manual_seed(2))
    said = m.answer(source, length, S)
    start = torch.full((1, B), seq2seq.START, dtype=torch.int64, device="cuda")
    m.forward(source, torch.cat([start, said[:-1]]), targets, length)
    logits = m.logits.view(S, B, V)
    chosen = logits.gather(2, said[..., None])[..., 0]
    assert float((logits.amax(2) - chosen).max()) < 1e-4


def test_constrained_answers(seq2seq):
    """With a large penalty and a mask no token comes twice and none is forbidden."""
    S, B, V = 8, 6, 40
    m = seq2seq.Seq2Seq(S, B, V, I=16, heads=2, head_dim=32, seed=5, memory=True)
    source, _, _, length = seq2seq.make_batch(S, B, V, torch.Generator(device="cuda").manual_seed(2))
    said = m.answer(source, length, S, repetition=torch.full((B,), 1e9, device="cuda"), mask=seq2seq.allowed_words(m))
    assert int(said.min()) >= 2 and int(said.max()) < V
    assert all(len(set(column)) == S for column in said.t().tolist())


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("kind,clip", [("adamw", None), ("adamw", 1.0), ("adamw8", 1.0)])
def test_training_and_answering_run(seq2seq, dtype, kind, clip):
    from layer_lstm_amd import lstm
    model, score = seq2seq.train(20, S=8, B=16, V=12, dtype=lstm.F32 if dtype == "f32" else lstm.BF16, memory=True,
                                 optimizer=kind, clip=clip)
    assert all(bool(torch.isfinite(p).all()) for p in model.p.values()) and score < 0
    assert 0 <= seq2seq.accuracy(model, repetition=1.1) <= 1


def test_the_command(seq2seq, capsys):
    seq2seq.main(["--steps", "4", "--batch", "8", "--length", "6", "--words", "12", "--memory", "--optimizer", "adamw8",
                  "--clip", "1.0", "--repetition", "1.05"])
    assert "%" in capsys.readouterr().out
    with pytest.raises(ValueError, match="clip"):
        seq2seq.train(1, S=4, B=4, V=8, clip=1.0)
