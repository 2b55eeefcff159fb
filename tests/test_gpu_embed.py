"""Embedding and its table's gradient on the GPU against fp64.

Bounds, element by element: the forward multiplies in fp32 and rounds once
(equal to the same two roundings on the CPU); a gradient element sums n terms
in fp32 in any order, scales and rounds to the storage type:
(n + 2) u32 scale sum|terms| + u |result| + half the smallest step."""
import numpy as np
import pytest

from oracle import seq_oracle as so
from seq_util import TINY, U32, UNIT, code, host, stored, tdtype, within

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lstm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from layer_lstm_amd import lstm as mod
    return mod


def make_ids(rng, N, V, kind):
    if kind == "one":  # a single id
        return np.full(N, V // 2, np.int64)
    if kind == "zipf":  # id r with a share of about 1/r, some outside the table
        ids = np.exp(rng.random(N) * np.log(V)).astype(np.int64) - 1
        ids[rng.random(N) < 0.05] = -1
        ids[rng.random(N) < 0.05] = V
        ids[rng.random(N) < 0.02] = 2**40 if N % 2 else -2**33
        return ids
    return rng.integers(0, V, N)


def check_grad(got, ids, dout, V, scale, padding, dt, what):
    want = so.embed_grad(ids, dout, V, scale, padding)
    mass = so.embed_grad(ids, np.abs(dout), V, scale, padding)
    n = so.embed_grad(ids, np.ones((ids.size, 1)), V, 1.0, padding)
    return within(got, want, (n + 2) * U32 * mass + UNIT[dt] * np.abs(want) * 1.01 + TINY[dt], what)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,V,D,kind", [
    (1, 1, 1, "flat"), (1, 5, 8, "flat"), (3, 100, 7, "flat"),
    (63, 10, 16, "flat"), (64, 3, 33, "one"), (65, 4, 512, "one"), (129, 1, 24, "one"),
    (1000, 50, 130, "zipf"), (4096, 300, 40, "zipf"), (4097, 300, 40, "zipf"),  # the two sorts
    (5000, 2047, 20, "zipf"), (5000, 2048, 17, "zipf"),  # one pass of 11 bits; two
    (20011, 70001, 8, "zipf"), (140001, 3, 4, "zipf"), (6000, 5, 1030, "flat"),
])
def test_embedding(lstm, dt, N, V, D, kind):
    print(f"case: embedding {dt} N={N} V={V} D={D} {kind}", flush=True)
    rng = np.random.default_rng(N + V)
    ids = make_ids(rng, N, V, kind)
    table, table64 = stored(torch, rng.normal(size=(V, D)), dt)
    dout, dout64 = stored(torch, rng.normal(size=(N, D)), dt)
    scale, padding = 1.3, (0 if V > 2 else None)
    m = lstm.Embedding(N, V, D, code(lstm, dt), scale=scale, padding=padding)
    gids = torch.from_numpy(ids).cuda()
    out = m.forward(gids, table.cuda())
    m.dtable = torch.full((V, D), float("nan"), dtype=table.dtype, device="cuda")
    grad = m.backward(gids, dout.cuda())
    again = m.backward(gids, dout.cuda()).clone()
    torch.cuda.synchronize()
    ok = torch.from_numpy((ids >= 0) & (ids < V))
    rows = table[torch.where(ok, torch.from_numpy(ids), 0)].float() * scale
    assert torch.equal(out.cpu(), torch.where(ok[:, None], rows, 0.0).to(table.dtype))
    check_grad(host(grad), ids, dout64, V, scale, padding, dt, "dtable")
    assert torch.equal(grad, again)


def test_strided_rows_int32_and_shapes(lstm):
    """Rows of wider tables, out of line with 16 bytes; int32 ids of shape [T, B]; another stream."""
    rng = np.random.default_rng(5)
    T, B, V, D = 9, 7, 40, 24
    ids = rng.integers(0, V, (T, B))
    wide, wide64 = stored(torch, rng.normal(size=(V, 31)), "bf16")
    dwide, dwide64 = stored(torch, rng.normal(size=(T * B, 37)), "bf16")
    m = lstm.Embedding(T * B, V, D, lstm.BF16, scale=2.0)
    s = torch.cuda.Stream()
    g32 = torch.from_numpy(ids.astype(np.int32)).cuda()
    gw, gd = wide.cuda(), dwide.cuda()
    torch.cuda.synchronize()
    out = m.forward(g32, gw[:, 3:27], stream=s)
    grad = m.backward(g32.reshape(-1), gd[:, 5:29], stream=s)
    s.synchronize()
    assert out.shape == (T, B, D)
    np.testing.assert_array_equal(host(out), so.embed(ids, wide64[:, 3:27], 2.0))
    check_grad(host(grad), ids.reshape(-1), dwide64[:, 5:29], V, 2.0, None, "bf16", "dtable")


def test_no_tokens_and_no_rows(lstm):
    m = lstm.Embedding(0, 6, 5, lstm.F32)
    m.dtable = torch.full((6, 5), float("nan"), device="cuda")
    e = torch.empty(0, dtype=torch.int64, device="cuda")
    assert m.forward(e, torch.ones(6, 5, device="cuda")).shape == (0, 5)
    assert not m.backward(e, torch.empty(0, 5, device="cuda")).any()
    m = lstm.Embedding(3, 0, 4, lstm.F32)
    ids = torch.tensor([0, 1, -1], device="cuda")
    assert not m.forward(ids, torch.empty(0, 4, device="cuda")).any()
    assert m.backward(ids, torch.ones(3, 4, device="cuda")).shape == (0, 4)


def test_values_a_table_may_hold(lstm):
    """Infinities and NaN of one token's row stay in that row, forward and backward."""
    table = torch.ones(5, 8, device="cuda")
    table[1], table[2] = float("inf"), float("nan")
    ids = torch.tensor([0, 1, 2, 3, 1], device="cuda")
    m = lstm.Embedding(5, 5, 8, lstm.F32)
    out = m.forward(ids, table)
    assert torch.isinf(out[[1, 4]]).all() and torch.isnan(out[2]).all() and (out[[0, 3]] == 1).all()
    grad = m.backward(ids, table[ids])
    assert torch.isinf(grad[1]).all() and torch.isnan(grad[2]).all() and (grad[[0, 3]] == 1).all()
    assert not grad[4].any()


def test_graph_replays(lstm):
    """Captured once, replayed on new inputs: each replay equals the eager call."""
    rng = np.random.default_rng(8)
    N, V, D = 5000, 700, 64
    m = lstm.Embedding(N, V, D, lstm.F32)
    ids = torch.zeros(N, dtype=torch.int64, device="cuda")
    dout = torch.zeros(N, D, device="cuda")
    table = torch.randn(V, D, device="cuda")
    m.forward(ids, table), m.backward(ids, dout)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.forward(ids, table)
        m.backward(ids, dout)
    ref = lstm.Embedding(N, V, D, lstm.F32)
    for _ in range(3):
        ids.copy_(torch.from_numpy(make_ids(rng, N, V, "zipf")))
        dout.normal_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(m.out, ref.forward(ids, table)) and torch.equal(m.dtable, ref.backward(ids, dout))


def test_refusals(lstm):
    e = lstm.LstmError
    for kw in (dict(N=-1), dict(V=-1), dict(D=-1), dict(padding=9), dict(padding=-2), dict(dtype=7)):
        with pytest.raises(e):
            lstm.Embedding(**{**dict(N=4, V=9, D=8, dtype=lstm.F32), **kw})
    with pytest.raises(e) as x:
        lstm.Embedding(1 << 26, 8, 8)
    assert x.value.code == -6
    m = lstm.Embedding(4, 9, 8, lstm.F32)
    ids, table = torch.zeros(4, dtype=torch.int64, device="cuda"), torch.zeros(9, 8, device="cuda")
    for bad in (ids[:3], ids.float(), torch.zeros(8, dtype=torch.int64, device="cuda")[::2]):
        with pytest.raises(ValueError):
            m.forward(bad, table)
    with pytest.raises(ValueError):
        m.forward(ids, table.half())
    with pytest.raises(ValueError):
        m.forward(ids, torch.zeros(8, 9, device="cuda").t())
    import ctypes
    L, s = lstm.lib(), m.shape
    s.ld_table = s.ld_out = 8
    out = torch.full((9, 8), 7.0, device="cuda")
    P = lambda t: t.data_ptr()  # noqa: E731
    assert L.lstm_embed_fwd(ctypes.byref(s), None, P(table), P(out), None) == -1
    assert L.lstm_embed_fwd(ctypes.byref(s), P(ids), P(table) + 2, P(out), None) == -4
    assert L.lstm_embed_fwd(ctypes.byref(s), P(ids) + 4, P(table), P(out), None) == -4
    many = lstm.Embedding(5000, 9, 8, lstm.F32)  # enough tokens to need a workspace
    ws, ids5, rows5 = many.workspace, torch.zeros(5000, dtype=torch.int64, device="cuda"), torch.zeros(5000, 8, device="cuda")
    bwd = lambda w, n: L.lstm_embed_bwd(ctypes.byref(many.shape), P(ids5), P(rows5), w, n, P(out), None)  # noqa: E731
    assert bwd(P(ws), ws.numel() - 1) == -5 and bwd(P(ws) + 8, ws.numel()) == -4 and bwd(None, ws.numel()) == -1
    s.ld_out = 7
    assert L.lstm_embed_fwd(ctypes.byref(s), P(ids), P(table), P(out), None) == -2
    s.ld_out, s.id_type = 8, 5
    assert L.lstm_embed_fwd(ctypes.byref(s), P(ids), P(table), P(out), None) == -3
    torch.cuda.synchronize()
    assert (out == 7.0).all()


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("N,V,D,kind", [
    (1, 65537, 3, "flat"), (50, 70001, 8, "one"), (300, 33001, 600, "zipf"), (4096, 66000, 20, "zipf"),
])
def test_few_tokens_of_a_large_table(lstm, dt, N, V, D, kind):
    """Few tokens, but a table too large for the one-launch gradient."""
    test_embedding(lstm, dt, N, V, D, kind)
    assert lstm.Embedding(N, V, D, code(lstm, dt)).workspace.numel() > 0


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_no_tokens_of_a_large_table(lstm, dt):
    m = lstm.Embedding(0, 70001, 8, code(lstm, dt))
    d = m.backward(torch.zeros(0, dtype=torch.int64, device="cuda"),
                   torch.zeros(0, 8, dtype=lstm.torch_dtype(code(lstm, dt)), device="cuda"))
    torch.cuda.synchronize()
    assert d.shape == (70001, 8) and not d.any()
