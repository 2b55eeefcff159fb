"""AdamW steps on a stream that the caller names."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
OPT = dict(lr=0.01, betas=(0.9, 0.98), eps=1e-6)


@pytest.fixture(scope="module")
def lstm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from layer_lstm_amd import lstm as mod
    return mod


@pytest.mark.parametrize("bits", [32, 8])
def test_a_step_on_another_stream_comes_after_the_states_filling(lstm, bits):
    """The current stream is still busy (some 50 ms of products) when the optimiser is made on it and its first step goes
    to another."""
    a = torch.randn(4096, 4096, device="cuda")
    b = torch.mm(a, a)
    g = torch.Generator(device="cuda").manual_seed(1)
    p, grad = torch.randn(5000, generator=g, device="cuda"), torch.randn(5000, generator=g, device="cuda")
    q, s = p.clone(), torch.cuda.Stream()
    want = lstm.AdamW([q], bits=bits, clip=1.0, **OPT)
    want.set_step(7)
    want.step([grad])
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        for _ in range(50):
            torch.mm(a, a, out=b)
        opt = lstm.AdamW([p], bits=bits, clip=1.0, **OPT)
    opt.set_step(7, stream=s)
    opt.step([grad], stream=s)
    torch.cuda.synchronize()
    assert torch.equal(p, q) and int(opt.control[0]) == 8
    for n in ("m", "v", "m_scale", "v_scale"):
        x, y = getattr(opt, n), getattr(want, n)
        assert (x is None and y is None) or torch.equal(x.view(torch.uint8), y.view(torch.uint8)), n


def test_a_step_into_another_streams_graph_needs_its_number_on_the_device(lstm):
    """The stream that is captured is the one the step goes to, not the current one."""
    p, grad = torch.randn(40, device="cuda"), torch.randn(40, device="cuda")
    plain = lstm.AdamW([p], **OPT)
    plain.step([grad])
    graph, s, other = torch.cuda.CUDAGraph(), torch.cuda.Stream(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=s):
        with torch.cuda.stream(other), pytest.raises(ValueError, match="graph"):
            plain.step([grad], stream=s)
    torch.cuda.synchronize()
    assert plain.shape.step == 1
