"""What the operators' classes refuse before any call into the library, with
the library and the device replaced by stand-ins (no GPU needed)."""
import ctypes

import pytest

torch = pytest.importorskip("torch")


class Library:
    """Answers the queries and records every launch."""

    def __init__(self):
        self.launches = []

    def __getattr__(self, name):
        def call(shape, *args):
            if name.endswith("_query"):
                for a in args:
                    ctypes.cast(a, ctypes.POINTER(ctypes.c_size_t))[0] = 64
            else:
                self.launches.append(name)
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    """(binding, recorded launches): buffers are made in host memory, the current device is cuda:0."""
    from layer_lstm_amd import lstm
    fake, empty = Library(), torch.empty
    monkeypatch.setattr(lstm, "_lib", fake)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(lstm, "_stream", lambda stream: 0)
    monkeypatch.setattr(lstm, "_raw_stream", None)
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **k: empty(*a, **k))
    return lstm, fake.launches


def test_host_tensors_are_refused(lib):
    lstm, launches = lib
    e = lstm.Embedding(4, 9, 8)
    ids, table = torch.zeros(4, dtype=torch.int64), torch.zeros(9, 8)
    a = lstm.Attention(2, 3, 2, 2, 1, 8)
    q, k = torch.zeros(2, 2, 2, 8), torch.zeros(3, 2, 1, 8)
    p = lstm.LogProb(4, 9)
    x = torch.zeros(4, 9)
    for call in (lambda: e.forward(ids, table), lambda: e.backward(ids, table[:4]), lambda: a.forward(q, k, k),
                 lambda: a.backward(q, q, k, k), lambda: p.forward(x, ids), lambda: p.backward(x, ids, x[:, 0].clone())):
        with pytest.raises(ValueError, match="cuda:0"):
            call()
    assert not launches


def test_buffers_are_on_a_gpu_and_it_is_the_current_one(lib, monkeypatch):
    lstm, launches = lib
    for make in (lambda: lstm.Embedding(4, 9, 8, device="cpu"), lambda: lstm.Attention(2, 3, 2, 2, 1, 8, device="cpu"),
                 lambda: lstm.LogProb(4, 9, device="cpu")):
        with pytest.raises(ValueError, match="a GPU"):
            make()
    m = lstm.Embedding(4, 9, 8, device="cuda:1")
    monkeypatch.setattr(lstm, "_on_device", lambda *a: None)
    ids, table = torch.zeros(4, dtype=torch.int64), torch.zeros(9, 8)
    with pytest.raises(ValueError, match="current device"):
        m.forward(ids, table)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)

    class Stream:
        device_index = 0
    with pytest.raises(ValueError, match="current device"):
        m.forward(ids, table, stream=Stream())
    assert not launches
    m.forward(ids, table)
    assert launches == ["lstm_embed_fwd"]


def test_rows_that_overlap_are_refused(lib, monkeypatch):
    """A row expanded over the tokens (the gradient of a sum over them), a
    table or logits of one row, rows closer than their width: the kernels
    would read past them.  One row alone may have any stride."""
    lstm, launches = lib
    monkeypatch.setattr(lstm, "_on_device", lambda *a: None)
    e, p = lstm.Embedding(6, 9, 8), lstm.LogProb(6, 8)
    ids, row = torch.zeros(6, dtype=torch.int64), torch.zeros(8)
    near = torch.zeros(100).as_strided((6, 8), (7, 1))
    for call in (lambda: e.forward(ids, row.expand(9, 8)), lambda: e.backward(ids, row.expand(6, 8)),
                 lambda: e.backward(ids.view(2, 3), row.expand(2, 3, 8)), lambda: e.backward(ids, near),
                 lambda: e.backward(ids.view(2, 3), torch.zeros(3, 2, 8).transpose(0, 1)),
                 lambda: p.forward(row.expand(6, 8), ids), lambda: p.forward(near, ids),
                 lambda: p.backward(row.expand(6, 8), ids), lambda: lstm.LogProb(6, 1).forward(row[:1].expand(6, 1), ids)):
        with pytest.raises(ValueError, match="rows"):
            call()
    assert not launches
    lstm.Embedding(1, 9, 8).backward(ids[:1], torch.zeros(100).as_strided((1, 8), (3, 1)))
    lstm.LogProb(1, 8).forward(row.expand(1, 8), ids[:1])
    assert len(launches) == 2
