"""AdamW steps on the GPU against fp64.

Bounds, element by element.  One step's fp32 operations: m and v three each
(3 u32 of their terms' sizes); w: its decay and difference 2 u32 |w|, the update
lr |u| (the errors of m 3, v 3 / 2, root, quotient and rate: 12 u32 of the
update's size with |m| in place of m's sum).  8-bit states: half a step of e4m3
times the block's scale, 1 + 4 u32 of it; a sqrt(v) held up to the smallest
number: up to that number."""
import math

import numpy as np
import pytest

from oracle import model_oracle as mo
from seq_util import TINY, U32, UNIT, host, tdtype, within

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
OPT = dict(lr=0.01, betas=(0.9, 0.98), eps=1e-6)


@pytest.fixture(scope="module")
def lstm():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from layer_lstm_amd import lstm as mod
    return mod


def pieces(opt, x):
    """A state buffer's parts, one for each parameter, in fp64."""
    return [host(x.float() if x.dtype == torch.float8_e4m3fn else x)[at : at + p.numel()] for p, at in zip(opt.params, opt.places)]


def scales(opt, x):
    return [host(x)[at // 256 : at // 256 + -(-p.numel() // 256)] for p, at in zip(opt.params, opt.places)]


def states(opt):
    """fp64 w, m, and v (32 bits) or sqrt(v) (8 bits) of each parameter, as held."""
    w = [host(p).reshape(-1) for p in opt.params] if opt.master is None else pieces(opt, opt.master)
    m, v = pieces(opt, opt.m), pieces(opt, opt.v)
    if opt.bits == 8:
        spread = lambda s, n: np.repeat(s, 256)[:n]  # noqa: E731
        m = [a * spread(s, a.size) for a, s in zip(m, scales(opt, opt.m_scale))]
        v = [a * spread(s, a.size) for a, s in zip(v, scales(opt, opt.v_scale))]
    return w, m, v


def check_step(opt, before, grads, t, decay, scale=1.0):
    """The states after a step from those before it (fp64 of what was held)."""
    (lr, (b1, b2), eps), dt = (opt.lr, opt.betas, opt.eps), {torch.float32: "f32", torch.bfloat16: "bf16", torch.float16: "f16"}[opt.tdtype]
    after = states(opt)
    for i, (p, g) in enumerate(zip(opt.params, grads)):
        g = g.reshape(-1) * scale
        w0, m0, v0 = before[0][i], before[1][i], before[2][i]
        if opt.bits == 8:
            v0 = v0 * v0
        d = decay[i] if isinstance(decay, (list, tuple)) else decay
        w, m, v = mo.adamw(w0, g, m0, v0, t, lr, b1, b2, eps, d)
        em = 6 * U32 * (abs(b1 * m0) + (1 - b1) * abs(g)) + TINY["f32"]
        ev = 8 * U32 * v + TINY["f32"]
        up = lr * (abs(b1 * m0) + (1 - b1) * abs(g)) / (1 - b1**t) / (np.sqrt(v / (1 - b2**t)) + eps)
        ew = 3 * U32 * abs(w0) + 16 * U32 * up + TINY["f32"]
        if opt.master is None:
            within(after[0][i], w, ew + UNIT[dt] * 1.01 * abs(w) * (dt != "f32") + TINY[dt], f"w {i}")
        else:
            within(after[0][i], w, ew, f"master {i}")
            within(host(p).reshape(-1), w, ew + UNIT[dt] * 1.01 * abs(w) + TINY[dt], f"param {i}")
        if opt.bits == 32:
            within(after[1][i], m, em, f"m {i}")
            within(after[2][i], v, ev, f"v {i}")
            continue
        for name, x, e, sc, got in (("m", m, em, scales(opt, opt.m_scale)[i], after[1][i]),
                                    ("sqrt v", np.sqrt(v), ev / np.maximum(np.sqrt(v), 1e-30), scales(opt, opt.v_scale)[i], after[2][i])):
            b, eb = mo.blocks(x), mo.blocks(e)
            most = abs(b).max(1)
            held = most > 2.0**-100
            within(sc, np.where(held, most / 448, 0), 3 * U32 * most / 448 + eb.max(1) / 448 + TINY["f32"], f"scale of {name} {i}")
            s64 = np.where(held, most / 448, 0)[:, None]
            step = mo.e4m3_step(np.divide(b, s64, out=np.zeros_like(b), where=s64 > 0)) * s64 / 2
            if name == "sqrt v":
                step = np.where((b > 0) & (b < 2.0**-9 * s64), 2.0**-9 * s64, step)
            tol = step * (1 + 4 * U32) + 4 * eb + 8 * U32 * abs(b) + 2.0**-100
            within(mo.blocks(got), b, tol, f"{name} {i}")


def make(dt, sizes, seed=0, off=0):
    """(parameters, gradients): views `off` elements into buffers of their own."""
    r = torch.Generator(device="cuda").manual_seed(seed)

    def one(n, by):
        buf = torch.empty(n + off, dtype=tdtype(torch, dt), device="cuda")
        buf[off:] = torch.randn(n, generator=r, device="cuda") * torch.exp(torch.randn(n, generator=r, device="cuda")) * by
        return buf[off:]

    return [one(n, 1.0) for n in sizes], [one(n, 0.1) for n in sizes]


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("sizes,off", [([1], 0), ([255, 256, 257], 0), ([7, 2048, 2049, 100003], 0), ([5, 0, 4096, 513], 1),
                                       ([3000] * 5, 3), ([1 + 37 * i for i in range(110)], 0), ([2200000, 9], 0)])
def test_steps(lstm, dt, bits, sizes, off):
    print(f"case: adamw {dt} {bits} bits {len(sizes)} tensors of {sizes[:4]} off {off}", flush=True)
    params, grads = make(dt, sizes, off=off)
    opt = lstm.AdamW(params, weight_decay=0.1, bits=bits, **OPT)
    for t in range(1, 4):
        before = states(opt)
        for g in grads:
            g.mul_(-0.5 if t == 2 else 1.5)
        opt.step(grads)
        check_step(opt, before, [host(g) for g in grads], t, 0.1)


@pytest.mark.parametrize("bits", [32, 8])
def test_decay_of_each_and_without_a_copy(lstm, bits):
    params, grads = make("bf16", [300, 40, 700])
    decay = [0.0, 0.5, 0.01]
    opt = lstm.AdamW(params, weight_decay=decay, bits=bits, master=False, **OPT)
    assert opt.master is None
    before = states(opt)
    opt.step(grads)
    check_step(opt, before, [host(g) for g in grads], 1, decay)


@pytest.mark.parametrize("dt", ["f32", "f16"])
@pytest.mark.parametrize("bits", [32, 8])
def test_gradients_held_to_a_norm(lstm, dt, bits):
    params, grads = make(dt, [70001, 300, 1, 16384])
    opt = lstm.AdamW(params, weight_decay=0.0, bits=bits, clip=0.7, loss_scale=4.0, **OPT)
    for t in (1, 2):
        norm = math.sqrt(sum((host(g) ** 2).sum() for g in grads)) / 4
        before = states(opt)
        opt.step(grads)
        assert abs(float(opt.norm) - norm) <= 2 * U32 * norm
        check_step(opt, before, [host(g) for g in grads], t, 0.0, min(1.0, 0.7 / norm) / 4)
        for g in grads:  # below the norm the second time
            g.mul_(0.5 / norm)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_step_that_is_not_finite_is_left_out(lstm, bad):
    params, grads = make("f16", [5000, 300])
    opt = lstm.AdamW(params, bits=8, clip=math.inf, **OPT)
    opt.step(grads)
    names = ("m", "v", "m_scale", "v_scale", "master")
    keep = [getattr(opt, n).clone() for n in names] + [p.clone() for p in params]
    old = float(grads[1][77])
    grads[1][77] = bad
    opt.step(grads)
    now = [getattr(opt, n) for n in names] + params
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(keep, now))
    assert int(opt.control[0]) == 1
    grads[1][77] = old
    before = states(opt)
    opt.step(grads)
    check_step(opt, before, [host(g) for g in grads], 2, 0.01)


def test_states_of_rows_without_gradients(lstm):
    """Nothing but zeros stays zeros and weights decay alone; an m that has died away (below 2^-100) is held as zeros."""
    params, grads = make("f32", [600])
    grads[0].zero_()
    opt = lstm.AdamW(params, weight_decay=0.1, bits=8, **OPT)
    w = params[0].clone()
    opt.step(grads)
    assert torch.equal(params[0], w * np.float32(1 - 0.01 * 0.1)) and not opt.m.float().any() and not opt.v.float().any()
    opt.m[:600].fill_(1.0), opt.m_scale.fill_(2.0**-101)  # (past 600: nobody's)
    opt.step(grads)
    assert not opt.m_scale.any() and not opt.m.float().any() and torch.isfinite(params[0]).all()


def test_many_steps_follow_the_formula(lstm):
    """30 steps of 32-bit states: the errors of each, and of the states before, add up to 30 times the step's."""
    params, grads = make("f32", [4000])
    opt = lstm.AdamW(params, weight_decay=0.1, **OPT)
    w, m, v = host(params[0]), np.zeros(4000), np.zeros(4000)
    w0 = abs(w).max()
    for t in range(1, 31):
        grads[0].copy_(torch.randn(4000, device="cuda"))
        w, m, v = mo.adamw(w, host(grads[0]), m, v, t, 0.01, 0.9, 0.98, 1e-6, 0.1)
        opt.step(grads)
    # sqrt(v) is at least 0.1 of the gradients' here; each update at most lr 10
    within(host(params[0]), w, 30 * (3 * U32 * w0 + 60 * U32 * 0.1) * np.ones(4000), "w")


def test_values_past_2_to_the_32(lstm):
    """A tensor of 2^31 + 300 values: its last ones, and those around 2^31."""
    if torch.cuda.mem_get_info()[0] < 60e9:
        pytest.skip("needs 60 GB of free device memory")
    n = (1 << 31) + 300
    p, g = torch.ones(n, dtype=torch.bfloat16, device="cuda"), torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    at = torch.tensor([0, 5, (1 << 31) - 1, 1 << 31, (1 << 31) + 255, n - 1], device="cuda")
    g[at] = torch.tensor([1.0, -2.0, 3.0, -4.0, 5.0, -6.0], device="cuda").bfloat16()
    opt = lstm.AdamW([p], weight_decay=0.0, bits=8, master=False, clip=math.inf, **dict(OPT, lr=0.5))
    opt.step([g])
    assert abs(float(opt.norm) - math.sqrt(91)) < 1e-5
    assert torch.equal(p[at].float().cpu(), torch.tensor([0.5, 1.5] * 3)) and int((p != 1).sum()) == 6
    del p, g, opt
    torch.cuda.empty_cache()


def test_replayed_steps_count_on(lstm):
    """A captured step replayed with other work and gradients between: the bits of eager steps."""
    for bits in (32, 8):
        sizes = [513, 4000, 70000]
        pa, grads = make("f32", sizes)
        pb = [p.clone() for p in pa]
        kw = dict(weight_decay=0.1, bits=bits, clip=1.0, **OPT)
        a, b = lstm.AdamW(pa, **kw), lstm.AdamW(pb, **kw)
        for o in (a, b):
            o.step(grads)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            b.step(grads)
        for k in range(3):
            for g in grads:
                g.mul_(-1.25)
            a.step(grads)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(x, y) for x, y in zip(pa, pb)) and torch.equal(a.control, b.control)
        assert int(a.control[0]) == 4
    plain = lstm.AdamW(pa, **OPT)
    plain.step(grads)
    with pytest.raises(ValueError, match="graph"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            plain.step(grads)
    torch.cuda.synchronize()


def test_another_stream(lstm):
    pa, grads = make("f32", [5000, 9])
    pb = [p.clone() for p in pa]
    a, b = lstm.AdamW(pa, clip=1.0, **OPT), lstm.AdamW(pb, clip=1.0, **OPT)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    a.step(grads), b.step(grads, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(pa, pb))


def test_a_parameter_that_moved_is_refused(lstm):
    params, grads = make("f32", [40, 8])
    opt = lstm.AdamW(params, **OPT)
    opt.step(grads)
    held = params[1].clone()
    params[1].data = held
    with pytest.raises(ValueError, match="memory"):
        opt.step(grads)
    assert opt.shape.step == 1


def test_refusals(lstm):
    params, grads = make("f32", [40, 8])
    opt = lstm.AdamW(params, **OPT)
    for bad in ([grads[0]], [grads[0], grads[1].cpu()], [grads[0], grads[1].double()], [grads[0], grads[1][:7]],
                [grads[0], torch.zeros(16, device="cuda")[::2]]):
        with pytest.raises(ValueError, match="grads"):
            opt.step(bad)
    for make_it in (lambda: lstm.AdamW([params[0], params[0]]), lambda: lstm.AdamW([params[0], params[0][8:16]]),
                    lambda: lstm.AdamW([params[0], params[1].cpu()]), lambda: lstm.AdamW([params[0], params[1].half()]),
                    lambda: lstm.AdamW([params[0][::2]]), lambda: lstm.AdamW(params, bits=16),
                    lambda: lstm.AdamW(params, weight_decay=[0.1]), lambda: lstm.AdamW([])):
        with pytest.raises(ValueError):
            make_it()
    opt.lr = -1.0
    with pytest.raises(lstm.LstmError, match="DIMS"):
        opt.step(grads)
    assert opt.shape.step == 0
    opt.lr = 0.01
    opt.step(grads)
    assert opt.shape.step == 1
    with pytest.raises(lstm.LstmError, match="DIMS"):
        lstm.AdamW(params, clip=0.0).step(grads)
    torch.cuda.synchronize()
