"""Host-side checks of the sequence-to-sequence entry points (no GPU needed):
constants, and argument errors that are found before the device is asked."""
import ctypes
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = open(os.path.join(ROOT, "include", "lstm.h")).read()


@pytest.fixture(scope="module")
def lstm():
    from layer_lstm_amd import lstm as mod
    return mod


def test_constants(lstm):
    assert re.search(r"LSTM_I32 = 0, LSTM_I64 = 1", HEADER) and (lstm.I32, lstm.I64) == (0, 1)
    assert int(re.search(r"#define LSTM_MAX_TOP (\d+)", HEADER).group(1)) == lstm.MAX_TOP


@pytest.mark.parametrize("change,code", [
    (dict(N=-1), -2), (dict(V=-1), -2), (dict(D=-1), -2), (dict(ld_table=7), -2), (dict(ld_out=7), -2),
    (dict(padding=9), -2), (dict(padding=-2), -2), (dict(dtype=3), -3), (dict(id_type=2), -3), (dict(N=1 << 26), -6),
    (dict(V=1 << 26), -6), (dict(D=(1 << 20) + 1, ld_table=1 << 21, ld_out=1 << 21), -6), (dict(ld_out=1 << 36), -6)])
def test_embed_shapes(lstm, change, code):
    s = lstm.EmbedShape(4, 9, 8, 8, 8, -1, 1.0, 0, 1)
    for k, v in change.items():
        setattr(s, k, v)
    n = ctypes.c_size_t(77)
    L = lstm.lib()
    assert L.lstm_embed_query(ctypes.byref(s), ctypes.byref(n)) == code and n.value == 77
    assert L.lstm_embed_fwd(ctypes.byref(s), None, None, None, None) == code
    assert L.lstm_embed_bwd(ctypes.byref(s), None, None, None, 0, None, None) == code
    assert L.lstm_embed_query(None, ctypes.byref(n)) == L.lstm_embed_query(ctypes.byref(s), None) == -1


@pytest.mark.parametrize("change,code", [
    (dict(N=-1), -2), (dict(V=-1), -2), (dict(ld=8), -2), (dict(ld_grad=8), -2), (dict(top=-1), -2),
    (dict(top=33), -2), (dict(top=10), -2), (dict(scale=0.0), -2), (dict(scale=-1.0), -2),
    (dict(scale=float("nan")), -2), (dict(scale=float("inf")), -2), (dict(dtype=-1), -3), (dict(id_type=-1), -3),
    (dict(N=1 << 24), -6), (dict(V=1 << 30, ld=1 << 30, ld_grad=1 << 30), -6),
    (dict(N=1 << 20, V=1 << 20, ld=1 << 20, ld_grad=1 << 20), -6), (dict(ld=1 << 36), -6)])
def test_logprob_shapes(lstm, change, code):
    s = lstm.LogprobShape(4, 9, 9, 9, 1.0, 3, 0, 1)
    for k, v in change.items():
        setattr(s, k, v)
    n = ctypes.c_size_t(77)
    L = lstm.lib()
    assert L.lstm_logprob_query(ctypes.byref(s), ctypes.byref(n)) == code and n.value == 77
    assert L.lstm_logprob_fwd(ctypes.byref(s), None, None, None, 0, *([None] * 6), None) == code
    assert L.lstm_logprob_bwd(ctypes.byref(s), *([None] * 9), None) == code
    assert L.lstm_logprob_query(None, ctypes.byref(n)) == L.lstm_logprob_query(ctypes.byref(s), None) == -1


def attend_shape(lstm):
    q, k = lstm.Stride(2 * 4 * 16, 4 * 16, 16), lstm.Stride(2 * 2 * 16, 2 * 16, 16)
    return lstm.AttendShape(3, 5, 2, 4, 2, 16, q, k, k, q, q, q, k, k, 5, 0.25, 0)


@pytest.mark.parametrize("change,code", [
    (dict(Tq=-1), -2), (dict(Tk=-1), -2), (dict(B=-1), -2), (dict(Hq=3), -2), (dict(Hk=3), -2), (dict(Hk=0), -2),
    (dict(Hq=0), -2), (dict(D=0), -2), (dict(scale=0.0), -2), (dict(scale=float("nan")), -2), (dict(mask_b=-1), -2),
    (dict(dtype=3), -3), (dict(D=257, Tq=1, Tk=1, B=1, Hq=1, Hk=1), -6), (dict(Tk=1 << 26), -6), (dict(Tq=1 << 25), -6)])
def test_attend_shapes(lstm, change, code):
    s = attend_shape(lstm)
    for k, v in change.items():
        setattr(s, k, v)
    a, b = ctypes.c_size_t(77), ctypes.c_size_t(77)
    L = lstm.lib()
    assert L.lstm_attend_query(ctypes.byref(s), ctypes.byref(a), ctypes.byref(b)) == code
    assert a.value == b.value == 77
    assert L.lstm_attend_fwd(ctypes.byref(s), *([None] * 6), 0, None, None, None) == code
    assert L.lstm_attend_bwd(ctypes.byref(s), *([None] * 9), 0, None, None, None, None) == code
    assert L.lstm_attend_query(None, ctypes.byref(a), ctypes.byref(b)) == -1
    assert L.lstm_attend_query(ctypes.byref(s), None, ctypes.byref(b)) == -1


@pytest.mark.parametrize("name,field,value", [
    ("q", "t", -1), ("k", "b", -1), ("v", "h", 1 << 36), ("o", "h", 8), ("o", "t", 0)])
def test_attend_strides(lstm, name, field, value):
    """A stride out of range, or an output whose rows overlap; inputs may overlap."""
    s = attend_shape(lstm)
    setattr(getattr(s, name), field, value)
    a, b = ctypes.c_size_t(0), ctypes.c_size_t(0)
    assert lstm.lib().lstm_attend_query(ctypes.byref(s), ctypes.byref(a), ctypes.byref(b)) == -2
    s = attend_shape(lstm)
    s.k.b = s.v.t = 0
    assert lstm.lib().lstm_attend_query(ctypes.byref(s), ctypes.byref(a), ctypes.byref(b)) in (0, -10)  # -10: no GPU
    s.dk.b = 0
    assert lstm.lib().lstm_attend_bwd(ctypes.byref(s), *([None] * 9), 0, None, None, None, None) == -2


def test_scales_whose_exponents_overflow(lstm):
    """scale log2 e has to be a number (above 2.36e38 it is not, and 0 times it is NaN)."""
    L, n, k = lstm.lib(), ctypes.c_size_t(0), ctypes.c_size_t(0)
    for scale, ok in ((2.3e38, True), (2.5e38, False), (3.0e38, False)):
        s = attend_shape(lstm)
        s.scale = scale
        assert (L.lstm_attend_query(ctypes.byref(s), ctypes.byref(n), ctypes.byref(k)) == -2) != ok
        s = lstm.LogprobShape(4, 9, 9, 9, scale, 3, 0, 1)
        assert (L.lstm_logprob_query(ctypes.byref(s), ctypes.byref(n)) == -2) != ok


def test_embedding_scales_are_finite(lstm):
    """An infinite or NaN scale would make NaN of the rows that are zeros by definition."""
    L, n = lstm.lib(), ctypes.c_size_t(0)
    for scale, ok in ((0.0, True), (-1.5, True), (float("inf"), False), (float("-inf"), False), (float("nan"), False)):
        s = lstm.EmbedShape(4, 9, 8, 8, 8, -1, scale, 0, 1)
        assert (L.lstm_embed_query(ctypes.byref(s), ctypes.byref(n)) == -2) != ok
