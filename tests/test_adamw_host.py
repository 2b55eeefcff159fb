"""What AdamW makes of its parameters, on the host (no GPU needed)."""
import pytest

torch = pytest.importorskip("torch")


@pytest.fixture
def settled():
    """The devices whose current stream was waited for."""
    return []


@pytest.fixture
def lstm(monkeypatch, settled):
    """The binding with buffers in host memory and cuda:0 the current device."""
    from layer_lstm_amd import lstm as mod
    zeros = torch.zeros
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(mod, "_on_device", lambda *a: None)
    monkeypatch.setattr(mod, "_settle", settled.append)
    monkeypatch.setattr(torch, "zeros", lambda *a, device=None, **k: zeros(*a, **k))
    return mod


def test_the_copy_is_no_part_of_a_graph(lstm):
    """16-bit leaves that take gradients: their fp32 copy takes none, and may be changed in place."""
    params = [torch.nn.Parameter(torch.randn(300).bfloat16()), torch.nn.Parameter(torch.randn(4, 5).bfloat16())]
    opt = lstm.AdamW(params)
    assert not opt.master.requires_grad and opt.master.grad_fn is None and opt.master.is_leaf
    for p, at in zip(params, opt.places):
        assert torch.equal(opt.master[at : at + p.numel()], p.detach().float().reshape(-1))
    opt.master.copy_(torch.ones_like(opt.master))
    opt.master.numpy()


def test_the_filling_that_is_waited_for_is_that_of_the_states_device(lstm, settled):
    lstm.AdamW([torch.zeros(4)], device="cuda:1")
    lstm.AdamW([torch.zeros(4)])
    assert settled == [1, 0]
