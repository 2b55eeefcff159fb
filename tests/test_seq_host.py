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
