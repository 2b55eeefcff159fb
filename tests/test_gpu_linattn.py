"""Linear attention on the GPU against fp64: outputs, states, gradients.

Bounds, element by element.  Every output is a sum of products with positive
powers of the decay, so the same recurrence on absolute values gives the sum of
its terms' sizes, `mass`.  In 16 bits two operands of each term are rounded to
the storage type (q . k and the state, u relative each); sums are fp32.  The
powers: at most T / 32 products of chunks' powers and one of 32 at most, whose
exponents are rounded, (3 |log decay| T + T / 8 + 16) u32; the sums' own lengths,
T / 32 chunks of products of 32 and D, as many again:
  |error| <= mass (2 u + c u32) + u |result| + TINY,  c = 3 |ld| T + T + 2 D + 64
(u = 0 in fp32 but for its rounding in c).  States are summed from V weighted as
two or three numbers of 16 bits: 2^-21 relative, c u32."""
import numpy as np
import pytest

from oracle import model_oracle as mo
from seq_util import TINY, U32, UNIT, code, host, stored, tdtype, within

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lstm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from layer_lstm_amd import lstm as mod
    return mod


def make(dt, T, B, Hq, Hk, D, Dv, seed=0, state=True, ragged=True, decays=None, size=1.0):
    """(device tensors, their fp64 values)."""
    r = np.random.default_rng(seed + T + D)
    c, x = {}, {}
    for n, shape in (("q", (T, B, Hq, D)), ("k", (T, B, Hk, D)), ("v", (T, B, Hk, Dv)), ("do", (T, B, Hq, Dv))):
        t, x[n] = stored(torch, r.normal(size=shape) * size, dt)
        c[n] = t.cuda()
    for n in ("state", "dstate"):
        c[n] = x[n] = None
        if state:
            t, x[n] = stored(torch, r.normal(size=(B, Hk, D, Dv)), "f32")
            c[n] = t.cuda()
    ld = np.array([decays[h % len(decays)] for h in range(Hk)] if decays else -np.exp(r.uniform(-7, 0, Hk)))
    t, x["log_decay"] = stored(torch, ld, "f32")
    c["log_decay"] = t.cuda()
    c["length"] = x["length"] = None
    if ragged:
        n = r.integers(0, T + 1, B)
        n[: min(B, 3)] = [T + 5, 0, -2][: min(B, 3)]
        x["length"] = n
        c["length"] = torch.from_numpy(n.astype(np.int32)).cuda()
    return c, x


def check(dt, x, scale, o, S, grads=None):
    q, k, v, ld, n = (x[i] for i in ("q", "k", "v", "log_decay", "length"))
    T, D, Dv = q.shape[0], q.shape[3], v.shape[3]
    train = grads is not None
    args = (x["state"], n) + ((x["do"], x["dstate"]) if train else ())
    want = mo.linattn(q, k, v, ld, scale, *args)
    mass = mo.linattn(abs(q), abs(k), abs(v), ld, abs(scale), *(i if i is None else abs(i) if i is not n else i for i in args))
    low = np.where(np.isfinite(ld), np.minimum(ld, 0), 0)
    c = (3 * abs(low).max(initial=0) * T + T + 2 * max(D, Dv) + 64) * U32
    u = 0.0 if dt == "f32" else 2 * UNIT[dt]
    names = ("o", "state", "dq", "dk", "dv", "dstate")
    for name, got, w, s in zip(names, (o, S, *(grads or ())), want, mass):
        if name in ("state", "dstate"):
            within(host(got), w, s * (2.0**-21 + c) + TINY["f32"], name)
        else:
            within(host(got), w, s * (u + c) + UNIT[dt] * 1.01 * abs(w) + TINY[dt], name)


def run(lstm, dt, c, scale=0.37, grads=True):
    T, B, Hq, D = c["q"].shape
    m = lstm.LinearAttention(T, B, Hq, c["k"].shape[2], D, c["v"].shape[3], code(lstm, dt), scale=scale)
    m.o.fill_(float("nan"))
    o, S = m.forward(c["q"], c["k"], c["v"], c["log_decay"], c["state"], c["length"])
    if not grads:
        return m, o, S, None
    m.dq, m.dk, m.dv = (torch.full(c[n].shape, float("nan"), dtype=c[n].dtype, device="cuda") for n in ("q", "k", "v"))
    m.dstate = torch.full((B, c["k"].shape[2], D, c["v"].shape[3]), float("nan"), device="cuda")
    m.workspace = torch.full((max(m._fwd_bytes, m._bwd_bytes),), 255, dtype=torch.uint8, device="cuda")
    return m, o, S, m.backward(c["do"], c["q"], c["k"], c["v"], c["log_decay"], c["state"], c["length"], c["dstate"])


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,B,Hq,Hk,D,Dv", [
    (1, 1, 1, 1, 1, 1), (1, 3, 6, 2, 17, 40), (2, 2, 2, 1, 64, 64), (8, 4, 10, 2, 80, 50), (9, 4, 2, 2, 8, 8),
    (31, 2, 2, 2, 32, 16), (32, 3, 3, 1, 65, 33), (33, 2, 4, 4, 128, 128), (65, 4, 6, 3, 80, 48), (100, 1, 5, 1, 37, 201),
    (130, 2, 2, 2, 256, 256), (97, 2, 8, 2, 200, 136), (40, 3, 2, 1, 256, 8), (40, 3, 2, 2, 8, 256),
    (600, 1, 2, 1, 64, 96), (300, 2, 3, 3, 129, 64),       # segments of the time axis
    (40, 64, 4, 4, 72, 80), (70, 64, 8, 4, 96, 128),       # as many heads as compute units; shared ones together
    (45, 70, 8, 8, 40, 64), (35, 40, 16, 8, 136, 200),
])
def test_linear_attention(lstm, dt, T, B, Hq, Hk, D, Dv):
    print(f"case: linear attention {dt} T={T} B={B} heads {Hq}/{Hk} D={D} Dv={Dv}", flush=True)
    c, x = make(dt, T, B, Hq, Hk, D, Dv)
    _, o, S, g = run(lstm, dt, c)
    check(dt, x, 0.37, o, S, g)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T,B,Hq,Hk,D,Dv", [
    (40, 130, 8, 4, 64, 48), (50, 140, 8, 4, 37, 51),      # small rows, many heads, shared
    (40, 100, 6, 3, 33, 64), (40, 32, 4, 2, 128, 128),     # fewer than compute units hold; as many, cut by columns
    (33, 70, 8, 4, 67, 99), (40, 70, 4, 4, 100, 64),
    (400, 1, 3, 1, 33, 65), (2100, 4, 8, 4, 64, 64),       # segments; of heads that share a state
    (191, 8, 6, 3, 80, 48), (191, 8, 6, 3, 41, 127),
])
def test_every_way_of_cutting_a_call(lstm, dt, T, B, Hq, Hk, D, Dv):
    print(f"case: linear attention {dt} T={T} B={B} heads {Hq}/{Hk} D={D} Dv={Dv}", flush=True)
    c, x = make(dt, T, B, Hq, Hk, D, Dv, seed=3)
    _, o, S, g = run(lstm, dt, c)
    check(dt, x, 0.37, o, S, g)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_without_states_and_lengths(lstm, dt):
    for T in (1, 50, 260):
        c, x = make(dt, T, 2, 2, 2, 64, 64, state=False, ragged=False)
        _, o, S, g = run(lstm, dt, c, scale=-1.5)
        check(dt, x, -1.5, o, S, g)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_decays_at_their_ends(lstm, dt):
    """None (0, or a positive one, which counts as 0), all of it (-inf), strong ones, and one that fp32 barely tells from none."""
    for T in (5, 70, 400):
        c, x = make(dt, T, 2, 6, 6, 32, 32, decays=[0.0, 2.0, -np.inf, -40.0, -3.0, -2e-8])
        _, o, S, g = run(lstm, dt, c)
        assert all(bool(torch.isfinite(i).all()) for i in (o, S, *g))
        check(dt, x, 0.37, o, S, g)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("D", [64, 37])
def test_rows_past_the_end_are_not_read_as_numbers(lstm, dt, D):
    for T, B in ((8, 4), (75, 4), (300, 2)):
        c, x = make(dt, T, B, 4, 2, D, D)
        past = torch.arange(T, device="cuda")[:, None] >= c["length"][None]
        for i, n in enumerate(("q", "k", "v", "do")):
            c[n][past] = (float("nan"), float("inf"), float("-inf"), float("nan"))[i]
        _, o, S, g = run(lstm, dt, c)
        check(dt, x, 0.37, o, S, g)
        for t in (o, *g[:3]):
            assert not t[past].any()


def test_empty_sequences_hold_their_state(lstm):
    for T in (1, 60, 300):
        c, x = make("bf16", T, 3, 2, 2, 16, 24)
        c["length"].zero_()
        _, o, S, g = run(lstm, "bf16", c)
        assert torch.equal(S, c["state"]) and torch.equal(g[3], c["dstate"])
        assert not o.any() and not any(i.any() for i in g[:3])


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_strided_and_expanded_rows(lstm, dt):
    """q, k, v in one buffer; batch first; one key and value row for all heads."""
    T, B, H, D = 70, 3, 4, 40
    c, x = make(dt, T, B, H, H, D, D)
    buf = torch.empty(T, B, H, 3, D, dtype=tdtype(torch, dt), device="cuda")
    for i, n in enumerate(("q", "k", "v")):
        buf[:, :, :, i] = c[n]
        c[n] = buf[:, :, :, i]
    c["do"] = c["do"].transpose(0, 1).contiguous().transpose(0, 1)
    _, o, S, g = run(lstm, dt, c)
    check(dt, x, 0.37, o, S, g)
    c["k"], c["v"] = (c[n][:, :, :1].expand(T, B, H, D) for n in ("k", "v"))
    x["k"], x["v"] = (np.broadcast_to(x[n][:, :, :1], (T, B, H, D)) for n in ("k", "v"))
    _, o, S, g = run(lstm, dt, c)
    check(dt, x, 0.37, o, S, g)


def test_offsets_past_32_bits(lstm):
    T, B, H, D = 40, 2, 2, 64
    far = (1 << 31) + 64
    c, x = make("bf16", T, B, H, H, D, D)
    for n in ("q", "k", "v", "do"):
        big = torch.empty(far + T * H * D, dtype=torch.bfloat16, device="cuda")
        view = big.as_strided((T, B, H, D), (H * D, far, D, 1))
        view.copy_(c[n])
        c[n] = view
    _, o, S, g = run(lstm, "bf16", c)
    check("bf16", x, 0.37, o, S, g)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_token_by_token_equals_the_whole(lstm, dt):
    """Steps of 1, 3 and 8 in place, and a forward of the rest, against one recurrence over all."""
    B, Hq, Hk, D, Dv = 3, 6, 3, 48, 72
    c, x = make(dt, 52, B, Hq, Hk, D, Dv, ragged=False)
    state, outs, at = c["state"].clone(), [], 0
    for T in (1, 3, 8, 1, 39):
        m = lstm.LinearAttention(T, B, Hq, Hk, D, Dv, code(lstm, dt), scale=0.37)
        part = [c[n][at : at + T] for n in ("q", "k", "v")]
        if T <= lstm.LINATTN_STEP:
            outs.append(m.step(*part, c["log_decay"], state).clone())
        else:
            o, last = m.forward(*part, c["log_decay"], state)
            outs.append(o.clone())
        at += T
    check(dt, x, 0.37, torch.cat(outs), last)


def test_steps_of_a_ragged_batch_in_place(lstm):
    for G in (1, 7):
        c, x = make("f16", 5, 6, 2 * G, 2, 33, 65)
        m = lstm.LinearAttention(5, 6, 2 * G, 2, 33, 65, lstm.F16, scale=0.37)
        state = c["state"].clone()
        o = m.step(c["q"], c["k"], c["v"], c["log_decay"], state, c["length"])
        check("f16", x, 0.37, o, state)


def test_fp16_scores_past_its_range_and_among_its_denormals(lstm):
    """q . k of 1e6 on v of 1e-3, and cotangents of 1e-6: operands in fp16 are scaled so that neither is lost.  A term
    of a wave's tile is at least 2^-25 of its largest, rounded 2^-12 relative: the bound of check() holds for it."""
    for T in (33, 200):
        c, x = make("f16", T, 2, 2, 2, 64, 64, state=False, size=1.0)
        for n, by in (("q", 100.0), ("k", 100.0), ("v", 1e-3), ("do", 1e-6)):
            c[n] = (c[n].float() * by).half()
            x[n] = host(c[n])
        _, o, S, g = run(lstm, "f16", c, scale=0.1)
        assert float(S.abs().max()) < 1e4 and float(o.abs().max()) > 100
        check("f16", x, 0.1, o, S, g)


def test_gradients_by_differences(lstm):
    """The loss is linear in each of q, k, v and the state alone: its difference over a step of any size is the slope.
    The two losses are sums of a few thousand fp32 terms, each off by c u32 of its mass."""
    T, B, Hq, Hk, D, Dv = 70, 2, 4, 2, 16, 24
    c, x = make("f32", T, B, Hq, Hk, D, Dv)
    m, o, S, g = run(lstm, "f32", c)
    g = dict(zip(("q", "k", "v", "state"), (i.clone() for i in g)))
    r = torch.Generator(device="cuda").manual_seed(1)
    mass = mo.linattn(*(abs(x[n]) for n in ("q", "k", "v")), x["log_decay"], 0.37, abs(x["state"]), x["length"])
    size = (mass[0] * abs(x["do"])).sum() + (mass[1] * abs(x["dstate"])).sum()
    for n, grad in g.items():
        d = torch.randn(grad.shape, generator=r, device="cuda")
        loss = []
        for sign in (0.5, -0.5):
            y = dict(c, **{n: c[n] + sign * d})
            o, S = m.forward(y["q"], y["k"], y["v"], y["log_decay"], y["state"], y["length"])
            loss.append(float((o.double() * c["do"].double()).sum() + (S.double() * c["dstate"].double()).sum()))
        slope = float((grad.double() * d.double()).sum())
        assert abs(loss[0] - loss[1] - slope) <= 3 * (4 * T + 2 * D + 64) * U32 * 3 * size, (n, loss, slope)


def test_same_bits_other_streams_and_graphs(lstm):
    """Repeated, on another stream, and replayed from a graph with other work and new inputs between the replays."""
    for T, B, Hq, Hk, D in ((1, 4, 4, 2, 64), (300, 2, 4, 2, 64), (64, 64, 8, 4, 80)):
        c, _ = make("bf16", T, B, Hq, Hk, D, D)
        args = [c[n] for n in ("q", "k", "v", "log_decay", "state", "length")]
        m = lstm.LinearAttention(T, B, Hq, Hk, D, D, lstm.BF16)

        def both(stream=None):
            o, S = m.forward(*args, stream=stream)
            return [i.clone() for i in (o, S, *m.backward(c["do"], *args, c["dstate"], stream=stream))]

        want = both()
        assert all(torch.equal(a, b) for a, b in zip(want, both()))
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        m.forward(*args, stream=s), m.backward(c["do"], *args, c["dstate"], stream=s)
        s.synchronize()
        got = (m.o, m.state, m.dq, m.dk, m.dv, m.dstate)
        assert all(torch.equal(a, b) for a, b in zip(want, got))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            m.forward(*args), m.backward(c["do"], *args, c["dstate"])
        keep = [i.clone() for i in (c["q"], c["do"])]
        for k in range(3):
            c["q"].copy_(keep[0] * (1 + k)), c["do"].copy_(keep[1] * (1 - k))
            want = both()
            for t in got:
                t.fill_(7)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(want, got)), k


@pytest.mark.parametrize("D,Dv", [(64, 128), (128, 64)])
def test_segments_of_narrow_and_wide_rows(lstm, D, Dv):
    """A long backward whose runs have different instances, all of them in segments."""
    c, x = make("bf16", 2100, 4, 4, 4, D, Dv)
    m, o, S, g = run(lstm, "bf16", c)
    assert m._bwd_bytes > 0
    check("bf16", x, 0.37, o, S, g)


def test_a_captured_forward_keeps_its_workspace(lstm):
    """The first backward, after the capture, makes buffers: none of them the one that the replays write to."""
    T, B, H, D = 4000, 1, 1, 64
    c, _ = make("bf16", T, B, H, H, D, D, ragged=False)
    args = [c[n] for n in ("q", "k", "v", "log_decay", "state")]
    m = lstm.LinearAttention(T, B, H, H, D, D, lstm.BF16)
    assert 0 < m._fwd_bytes < m._bwd_bytes
    want = [i.clone() for i in m.forward(*args)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        m.forward(*args)
    space = m.workspace.data_ptr()
    m.backward(c["do"], *args, dstate=c["dstate"])
    torch.cuda.synchronize()
    assert m.workspace.data_ptr() == space and m.bwd_workspace.data_ptr() != space
    other = [torch.full((m._fwd_bytes,), 1, dtype=torch.uint8, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    for _ in range(2):
        m.o.fill_(7), m.state.fill_(7)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(m.o, want[0]) and torch.equal(m.state, want[1])
    assert all(int(i.min()) == 1 == int(i.max()) for i in other)


def test_empty_calls(lstm):
    for T, B, H in ((0, 2, 2), (3, 0, 2), (3, 2, 0), (40, 0, 2), (40, 2, 0)):
        c, _ = make("f32", T, B, H, H, 8, 8, ragged=False)
        _, o, S, g = run(lstm, "f32", c)
        torch.cuda.synchronize()
        assert o.shape == (T, B, H, 8)
        if T == 0:
            assert torch.equal(S, c["state"]) and torch.equal(g[3], c["dstate"])


def test_refusals(lstm):
    c, _ = make("f32", 9, 2, 2, 2, 8, 8)
    args = [c[n] for n in ("q", "k", "v", "log_decay", "state", "length")]
    m = lstm.LinearAttention(9, 2, 2, 2, 8, 8)
    m.forward(*args)
    for i in range(len(args)):
        with pytest.raises(ValueError, match="cuda:0"):
            m.forward(*(a.cpu() if j == i else a for j, a in enumerate(args)))
    with pytest.raises(ValueError, match="at most"):
        m.step(*args)
    with pytest.raises(ValueError, match="buffer"):
        m.forward(*args[:4], m.state)
    m.backward(c["do"], *args, c["dstate"])
    with pytest.raises(ValueError, match="buffer"):
        m.backward(c["do"], *args, m.dstate)
    # in place past the steps' kernel, through the C call
    import ctypes
    rc = lstm.lib().lstm_linattn_fwd(ctypes.byref(m.shape), *(a.data_ptr() for a in args[:4]), None, m.state.data_ptr(),
                                     None, 0, m.o.data_ptr(), m.state.data_ptr(), None)
    assert rc == -2
    for D, Dv in ((257, 8), (8, 257)):
        with pytest.raises(lstm.LstmError, match="UNSUPPORTED"):
            lstm.LinearAttention(9, 2, 2, 2, D, Dv)
    torch.cuda.synchronize()
