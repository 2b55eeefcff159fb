"""Host-side checks of linear attention's, the penalties' and AdamW's entry
points and classes (no GPU needed): constants, argument errors that are found
before the device is asked, and what the classes refuse before any call."""
import ctypes
import math
import os
import re

import pytest

torch = pytest.importorskip("torch")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = open(os.path.join(ROOT, "include", "lstm.h")).read()


@pytest.fixture(scope="module")
def lstm():
    from layer_lstm_amd import lstm as mod
    return mod


def test_constants(lstm):
    for name, value in (("LSTM_LINATTN_STEP", lstm.LINATTN_STEP), ("LSTM_ADAMW_BLOCK", lstm.ADAMW_BLOCK)):
        assert int(re.search(rf"#define {name} (\d+)", HEADER).group(1)) == value
    assert "10 linear attention   11 logit penalties   12 AdamW" in HEADER
    assert lstm.KERNEL_KINDS[10:] == ("linear_attention", "penalty", "adamw")
    ms, n = ctypes.c_double(0), ctypes.c_int64(0)
    assert lstm.lib().lstm_timing_read(len(lstm.KERNEL_KINDS), ctypes.byref(ms), ctypes.byref(n)) == -2


def linattn_shape(lstm):
    q, k, v = lstm.Stride(2 * 4 * 16, 64, 16), lstm.Stride(2 * 2 * 16, 32, 16), lstm.Stride(2 * 2 * 8, 16, 8)
    o = lstm.Stride(2 * 4 * 8, 32, 8)
    return lstm.LinattnShape(5, 2, 4, 2, 16, 8, q, k, v, o, o, q, k, v, 0.25, 0)


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), -2), (dict(B=-1), -2), (dict(Hq=3), -2), (dict(Hk=3), -2), (dict(Hk=0), -2), (dict(Hq=0), -2),
    (dict(D=0), -2), (dict(Dv=0), -2), (dict(scale=math.nan), -2), (dict(scale=math.inf), -2), (dict(dtype=3), -3),
    (dict(D=257, T=1, B=1, Hq=1, Hk=1), -6), (dict(Dv=257, T=1, B=1, Hq=1, Hk=1), -6), (dict(T=1 << 26), -6),
    (dict(B=1 << 18, T=1, Hq=1, Hk=1), -6)])
def test_linattn_shapes(lstm, change, code):
    s = linattn_shape(lstm)
    for k, v in change.items():
        setattr(s, k, v)
    a, b = ctypes.c_size_t(77), ctypes.c_size_t(77)
    L = lstm.lib()
    assert L.lstm_linattn_query(ctypes.byref(s), ctypes.byref(a), ctypes.byref(b)) == code
    assert a.value == b.value == 77
    assert L.lstm_linattn_fwd(ctypes.byref(s), *([None] * 7), 0, None, None, None) == code
    assert L.lstm_linattn_bwd(ctypes.byref(s), *([None] * 9), 0, *([None] * 5)) == code
    assert L.lstm_linattn_query(None, ctypes.byref(a), ctypes.byref(b)) == -1
    assert L.lstm_linattn_query(ctypes.byref(s), None, ctypes.byref(b)) == -1


@pytest.mark.parametrize("name,field,value", [
    ("q", "t", -1), ("k", "b", -1), ("v", "h", 1 << 36), ("o", "h", 4), ("o", "t", 0)])
def test_linattn_strides(lstm, name, field, value):
    s = linattn_shape(lstm)
    setattr(getattr(s, name), field, value)
    a, b = ctypes.c_size_t(0), ctypes.c_size_t(0)
    assert lstm.lib().lstm_linattn_query(ctypes.byref(s), ctypes.byref(a), ctypes.byref(b)) == -2
    s = linattn_shape(lstm)
    s.k.b = s.v.t = 0  # inputs may overlap
    assert lstm.lib().lstm_linattn_query(ctypes.byref(s), ctypes.byref(a), ctypes.byref(b)) in (0, -10)  # -10: no GPU
    s.dv.b = 0
    assert lstm.lib().lstm_linattn_bwd(ctypes.byref(s), *([None] * 9), 0, *([None] * 5)) == -2


@pytest.mark.parametrize("change,code", [
    (dict(N=-1), -2), (dict(V=-1), -2), (dict(L=-1), -2), (dict(ld=8), -2), (dict(ld_out=8), -2), (dict(history_n=-1), -2),
    (dict(history_t=-1), -2), (dict(ld_bias=-1), -2), (dict(ld_mask=-1), -2), (dict(dtype=3), -3), (dict(id_type=2), -3),
    (dict(N=1 << 24), -6), (dict(V=1 << 30, ld=1 << 30, ld_out=1 << 30), -6), (dict(L=1 << 31), -6), (dict(ld=1 << 36), -6),
    (dict(N=1 << 20, V=1 << 20, ld=1 << 20, ld_out=1 << 20), -6)])
def test_penalty_shapes(lstm, change, code):
    s = lstm.PenaltyShape(4, 9, 9, 9, 3, 3, 1, 0, 1, 0, 1)
    for k, v in change.items():
        setattr(s, k, v)
    assert lstm.lib().lstm_penalty(ctypes.byref(s), *([None] * 10)) == code
    assert lstm.lib().lstm_penalty(None, *([None] * 10)) == -1


def adamw_case(lstm, **change):
    s = lstm.AdamwShape(0.01, 0.9, 0.99, 1e-8, 1, 0, 32)
    t = (lstm.AdamwTensor * 2)()
    for x in t:
        x.param = x.grad = x.m = x.v = x.m_scale = x.v_scale = 4096
        x.n, x.weight_decay = 10, 0.1
    for k, v in change.items():
        setattr(s if k in ("lr", "beta1", "beta2", "eps", "step", "dtype", "bits") else t[1], k, v)
    return s, t


@pytest.mark.parametrize("change,code", [
    (dict(lr=-1.0), -2), (dict(lr=math.nan), -2), (dict(lr=math.inf), -2), (dict(beta1=1.0), -2), (dict(beta1=-0.1), -2),
    (dict(beta2=1.0), -2), (dict(eps=-1.0), -2), (dict(step=0), -2), (dict(n=-1), -2), (dict(weight_decay=-0.1), -2),
    (dict(weight_decay=math.nan), -2), (dict(dtype=3), -3), (dict(bits=16), -3), (dict(n=1 << 40), -6), (dict(grad=None), -1),
    (dict(param=None), -1), (dict(m=None), -1), (dict(v=None), -1), (dict(bits=8, v_scale=None), -1), (dict(param=4098), -4),
    (dict(dtype=1, grad=4097), -4), (dict(dtype=1, master=4098), -4), (dict(m=4098), -4), (dict(bits=8, m_scale=4097), -4)])
def test_adamw_steps(lstm, change, code):
    s, t = adamw_case(lstm, **change)
    L, n = lstm.lib(), ctypes.c_size_t(0)
    assert L.lstm_adamw_step(ctypes.byref(s), t, 2, None, None) == code
    assert L.lstm_adamw_step(None, t, 2, None, None) == L.lstm_adamw_step(ctypes.byref(s), None, 2, None, None) == -1
    assert L.lstm_adamw_query(ctypes.byref(s), None, 2, ctypes.byref(n)) == L.lstm_adamw_query(ctypes.byref(s), t, 2, None) == -1


def test_adamw_norms(lstm):
    s, t = adamw_case(lstm)
    L, n = lstm.lib(), ctypes.c_size_t(0)
    t[0].n = 100000
    assert L.lstm_adamw_query(ctypes.byref(s), t, 2, ctypes.byref(n)) == 0 and n.value == 256
    assert L.lstm_adamw_query(ctypes.byref(s), t, -1, ctypes.byref(n)) == -2
    for most, un in ((0.0, 1.0), (-1.0, 1.0), (math.nan, 1.0), (1.0, 0.0), (1.0, math.inf), (1.0, math.nan)):
        assert L.lstm_adamw_norm(ctypes.byref(s), t, 2, most, un, 4096, 4096, 4096, None) == -2
    # (its size in the header, 8 + 4 x 4 + 2 x 4 bytes; -10: no GPU here to say how many compute units it has)
    assert ctypes.sizeof(lstm.AdamwControl) == 32
    assert L.lstm_adamw_norm(ctypes.byref(s), t, 2, 1.0, 1.0, 4096, 8, 4096, None) in (-5, -10)


class Library:
    """Answers the queries and records every launch."""

    def __init__(self):
        self.launches = []

    def __getattr__(self, name):
        def call(*args):
            if name.endswith("_query"):
                for a in args[1:]:
                    if not isinstance(a, (int, ctypes.Array)):
                        ctypes.cast(a, ctypes.POINTER(ctypes.c_size_t))[0] = 64
            else:
                self.launches.append(name)
            return 0
        return call


@pytest.fixture
def fake(monkeypatch):
    """(binding, recorded launches): buffers are made in host memory, the current device is cuda:0."""
    from layer_lstm_amd import lstm
    lib, empty, zeros = Library(), torch.empty, torch.zeros
    monkeypatch.setattr(lstm, "_lib", lib)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(lstm, "_stream", lambda stream: 0)
    monkeypatch.setattr(lstm, "_raw_stream", None)
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **k: empty(*a, **k))
    monkeypatch.setattr(torch, "zeros", lambda *a, device=None, **k: zeros(*a, **k))
    return lstm, lib.launches


def test_host_tensors_are_refused(fake):
    lstm, launches = fake
    m = lstm.LinearAttention(3, 2, 4, 2, 8, 16)
    q, k, v, g, ld = torch.zeros(3, 2, 4, 8), torch.zeros(3, 2, 2, 8), torch.zeros(3, 2, 2, 16), torch.zeros(3, 2, 4, 16), torch.zeros(2)
    p, x = lstm.Penalty(4, 9), torch.zeros(4, 9)
    for call in (lambda: m.forward(q, k, v, ld), lambda: m.step(q, k, v, ld, torch.zeros(2, 2, 8, 16)),
                 lambda: m.backward(g, q, k, v, ld), lambda: p.forward(x), lambda: lstm.AdamW([x])):
        with pytest.raises(ValueError, match="cuda:0"):
            call()
    for make in (lambda: lstm.LinearAttention(3, 2, 4, 2, 8, device="cpu"), lambda: lstm.Penalty(4, 9, device="cpu"),
                 lambda: lstm.AdamW([x], device="cpu")):
        with pytest.raises(ValueError, match="a GPU"):
            make()
    assert not launches


def test_shapes_types_and_rows_are_checked(fake, monkeypatch):
    lstm, launches = fake
    monkeypatch.setattr(lstm, "_on_device", lambda *a: None)
    m = lstm.LinearAttention(3, 2, 4, 2, 8, 16)
    q, k, v, ld = torch.zeros(3, 2, 4, 8), torch.zeros(3, 2, 2, 8), torch.zeros(3, 2, 2, 16), torch.zeros(2)
    s, n = torch.zeros(2, 2, 8, 16), torch.zeros(2, dtype=torch.int32)
    p, x, h = lstm.Penalty(4, 40), torch.zeros(4, 40), torch.zeros(4, 3, dtype=torch.int64)
    one = torch.ones(4)
    for call in (lambda: m.forward(q.half(), k, v, ld), lambda: m.forward(q, k[:2], v, ld), lambda: m.forward(q, v, v, ld),
                 lambda: m.forward(q, k, v.transpose(2, 3).contiguous().transpose(2, 3), ld), lambda: m.forward(q, k, v, ld[:1]),
                 lambda: m.forward(q, k, v, ld.double()), lambda: m.forward(q, k, v, ld, s.half()),
                 lambda: m.forward(q, k, v, ld, s.transpose(0, 1)), lambda: m.forward(q, k, v, ld, s, n.long()),
                 lambda: m.backward(q, q, k, v, ld), lambda: m.backward(torch.zeros(3, 2, 4, 16), q, k, v, ld, dstate=s[:1]),
                 lambda: p.forward(x.half()), lambda: p.forward(x[:, :9]), lambda: p.forward(x, out=x.half()),
                 lambda: p.forward(x[:1].expand(4, 40)), lambda: p.forward(x, repetition=one), lambda: p.forward(x, h.int()[:2]),
                 lambda: p.forward(x, h.float()), lambda: p.forward(x, h, n), lambda: p.forward(x, h, repetition=one[:2]),
                 lambda: p.forward(x, h, presence=one.double()), lambda: p.forward(x, bias=one), lambda: p.forward(x, bias=x.double()),
                 lambda: p.forward(x, mask=torch.zeros(4, 1, dtype=torch.int32)), lambda: p.forward(x, mask=torch.zeros(4, 2))):
        with pytest.raises(ValueError):
            call()
    assert not launches
    m.forward(q, k, v, ld, s, n), m.forward(q, k[:, :, :1].expand(3, 2, 2, 8), v, ld)
    p.forward(x, h, repetition=one, bias=x, mask=torch.zeros(4, 3, dtype=torch.int32))
    assert launches == ["lstm_linattn_fwd"] * 2 + ["lstm_penalty"] and p.shape.ld_bias == 40 and p.shape.ld_mask == 3
    p.forward(x, bias=x[:1].expand(4, 40))
    assert p.shape.ld_bias == 0
