"""Linear attention's outputs are no inputs of the same call: an operator that
several layers share has its o read by the next of them."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lstm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from layer_lstm_amd import lstm as mod
    return mod


@pytest.mark.parametrize("T", [1, 40])
def test_an_output_given_as_an_input_is_refused(lstm, T):
    B, H, D = 2, 3, 16
    x = torch.randn(T, B, H, D, device="cuda")
    ld, state = torch.full((H,), -0.1, device="cuda"), torch.zeros(B, H, D, D, device="cuda")
    m = lstm.LinearAttention(T, B, H, H, D, D)
    o = m.forward(x, x, x, ld)[0]
    first = o.clone()
    grads = m.backward(x, x, x, x, ld)[:3]
    for i in range(3):
        args = [o if j == i else x for j in range(3)]
        with pytest.raises(lstm.LstmError, match="DIMS"):
            m.forward(*args, ld)
        if T == 1:
            with pytest.raises(lstm.LstmError, match="DIMS"):
                m.step(*args, ld, state)
    for g in grads:
        for i in range(4):
            with pytest.raises(lstm.LstmError, match="DIMS"):
                m.backward(*(g if j == i else x for j in range(4)), ld)
    assert torch.equal(o, first) and not state.any()
    # a copy, and o as the gradient's inputs, are what they always were
    m.forward(first, first, first, ld)
    m.backward(m.o, m.o, m.o, m.o, ld)
    torch.cuda.synchronize()
