"""Linear attention with memories of thousands of steps: the decay of a step, or
of a chunk, is applied as often, so what its rounding takes from or adds to it
would add up, a fp32 number's 2^-25 a time.  States are held against the
definition in fp64.

Bounds, of the whole tensor's norm.  A step's (a chunk's) own roundings are
independent: r of them of at most u32 of the state, in the square mean u32 /
sqrt(3), over n steps or chunks sqrt(n r / 3) u32.  Tokens: r = 2, bound
2 sqrt(n) u32 (2.4 times that); chunks of fp32: a product and the matrix cores'
sums of 32 steps, r = 17, bound 6 sqrt(n) u32 (2.5 times), in segments (their
sums are of 8 chunks here) for all types.  The terms are positive, so that a
decay's error does not average out: with one of 2^-25 a time it is n u32 / 4 for
memories longer than the text."""
import math

import numpy as np
import pytest

from seq_util import U32, code, host, stored

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lstm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from layer_lstm_amd import lstm as mod
    return mod


def badly_rounded(steps, n, lo, hi):
    """n fp32 log decays of memories from lo to hi steps whose powers over `steps` steps fp32 holds worst."""
    out = []
    for a, b in zip(np.geomspace(lo, hi, n + 1)[:-1], np.geomspace(lo, hi, n + 1)[1:]):
        c = (-1 / np.linspace(a, b, 400)).astype(np.float32)
        p = np.exp(c.astype(np.float64) * steps)
        out.append(c[np.argmax(abs(p.astype(np.float32) - p))])
    return np.array(out, np.float32)


def final_state(k, v, ld):
    """Of one sequence: k [T, H, D], v [T, H, Dv], fp64."""
    T = k.shape[0]
    w = np.exp(ld[None] * np.arange(T - 1, -1, -1)[:, None])
    return np.einsum("thd,the->hde", k * w[:, :, None], v, optimize=True)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("T", [1, 8])
def test_tokens(lstm, dt, T):
    n, B, H, D = 4096, 1, 4, 32
    r = np.random.default_rng(5)
    ld = badly_rounded(1, H, 3000, 60000)
    k, kx = stored(torch, r.uniform(0.5, 1, (n, B, H, D)), dt)
    v, vx = stored(torch, r.uniform(0.5, 1, (n, B, H, D)), dt)
    k, v, ldt = k.cuda(), v.cuda(), torch.from_numpy(ld).cuda()
    m = lstm.LinearAttention(T, B, H, H, D, D, code(lstm, dt))
    state = torch.zeros(B, H, D, D, device="cuda")
    for t in range(0, n, T):
        m.step(k[t : t + T], k[t : t + T], v[t : t + T], ldt, state)
    want = final_state(kx[:, 0], vx[:, 0], ld.astype(np.float64))
    err = np.linalg.norm(host(state)[0] - want) / np.linalg.norm(want)
    print(f"  {dt}, steps of {T}: {err / U32:.1f} u32 of {2 * math.sqrt(n):.1f}", flush=True)
    assert err <= 2 * math.sqrt(n) * U32


@pytest.mark.parametrize("dt,B,H,D", [("f32", 16, 16, 16), ("f32", 16, 16, 128), ("f32", 1, 2, 64), ("bf16", 1, 2, 64),
                                      ("f16", 1, 2, 64)])
def test_chunks(lstm, dt, B, H, D):
    """Whole sequences by chunks of 32 steps (one row for all of the batch), and one cut into segments; the same backwards,
    where q and dout give the first state's gradient."""
    T = 65536 if D < 128 else 16384
    r = np.random.default_rng(6)
    ld = badly_rounded(32, H, 20000, 400000)
    k, kx = stored(torch, r.uniform(0.5, 1, (T, 1, H, D)), dt)
    v, vx = stored(torch, r.uniform(0.5, 1, (T, 1, H, 16)), dt)
    k, v, ldt = k.cuda().expand(T, B, H, D), v.cuda().expand(T, B, H, 16), torch.from_numpy(ld).cuda()
    m = lstm.LinearAttention(T, B, H, H, D, 16, code(lstm, dt), scale=1.0)
    state = m.forward(k, k, v, ldt)[1]
    ld = ld.astype(np.float64)
    bound = 6 * math.sqrt(T / 32) * U32
    want = final_state(kx[:, 0], vx[:, 0], ld)
    err = np.linalg.norm(host(state)[-1] - want) / np.linalg.norm(want)
    print(f"  {dt} {B} x {H} x {D}, state: {err / U32:.1f} u32 of {bound / U32:.1f}", flush=True)
    assert err <= bound and torch.equal(state, state[:1].expand_as(state))
    d = m.backward(v, k, k, v, ldt)[3]
    want = final_state(kx[::-1, 0], vx[::-1, 0], ld) * np.exp(ld)[:, None, None]
    err = np.linalg.norm(host(d)[-1] - want) / np.linalg.norm(want)
    print(f"  {dt} {B} x {H} x {D}, gradient: {err / U32:.1f} u32 of {bound / U32:.1f}", flush=True)
    assert err <= bound
