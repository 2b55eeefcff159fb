"""Where the penalties may write: the logits themselves, other columns of their
rows, other memory; nothing that is partly theirs."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lstm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from layer_lstm_amd import lstm as mod
    return mod


@pytest.mark.parametrize("N,V", [(1, 40), (5, 40), (5, 9)])
def test_places_of_out(lstm, N, V):
    m, bias = lstm.Penalty(N, V), torch.randn(V, device="cuda")
    wide = torch.empty(N, 3 * V + 2, device="cuda")
    values = torch.randn(N, V, device="cuda")

    def forward(x, y):
        x.copy_(values)
        m.forward(x, bias=bias, out=y)
        assert torch.equal(y, values + bias)

    x = wide[:, V : 2 * V]
    forward(x, x)
    for at in (0, 2 * V, 2 * V + 2):  # beside them, right up to them
        forward(x, wide[:, at : at + V])
        forward(wide[:, at : at + V], x)
    forward(x, torch.empty(N, V, device="cuda"))
    for at in (V - 1, V + 1, 1, 2 * V - 1):
        with pytest.raises(lstm.LstmError, match="DIMS"):
            m.forward(x, bias=bias, out=wide[:, at : at + V])
        with pytest.raises(lstm.LstmError, match="DIMS"):
            m.forward(wide[:, at : at + V], bias=bias, out=x)
    flat = torch.empty(2 * N * V, device="cuda")
    forward(flat[: N * V].view(N, V), flat[N * V :].view(N, V))
    if N > 1:  # rows further down: the same places of the rows, other rows, or rows of another length
        rows = torch.empty(2 * N, V, device="cuda")
        forward(rows[:N], rows[N:])
        for y in (rows[1 : N + 1], rows.view(N, 2 * V)[:, :V]):
            with pytest.raises(lstm.LstmError, match="DIMS"):
                m.forward(rows[:N], bias=bias, out=y)
    torch.cuda.synchronize()
