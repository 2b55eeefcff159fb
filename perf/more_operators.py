"""The operators that train and run a sequence model beside its LSTM layers, as
cases to measure: linear attention with a decay for each head (prompts,
training, single tokens), the penalties, biases and masks on logits before a
token is chosen, and the AdamW step over all of a model's tensors.

`run` computes a case in plain 32-bit torch operations, or, with `own` set,
through layer_lstm_amd.lstm.  `exact` gives the same outputs in 64 bits from
the definitions.

Sequences are time-major as everywhere in the library: [T,B,heads,D], lengths
int32 [B]; states are fp32 [B,heads,D,Dv].
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
BLOCK = 256  # values of an 8-bit state that share a scale, and where each tensor begins in the state's buffers


def listed():
    return [
        # one token of each of 16 sequences through a layer of 16 heads of 128 (H = 2048)
        dict(name="linear step bf16", op="linear", dir="step", T=1, B=16, Hq=16, Hk=16, D=128, Dv=128, dtype="bf16", ragged=False, state=True),
        # one token of a busy server's 256 sequences, four query heads to a state, odd head sizes
        dict(name="linear step f16 odd", op="linear", dir="step", T=1, B=256, Hq=8, Hk=2, D=80, Dv=112, dtype="f16", ragged=False, state=True),
        # a long document read as a prompt, four query heads to a state
        dict(name="linear prompt long f16", op="linear", dir="fwd", T=32768, B=1, Hq=32, Hk=8, D=128, Dv=128, dtype="f16", ragged=False, state=False),
        # a small fp32 training step, ragged, odd length and head sizes, state carried over from the previous piece of text
        dict(name="linear train f32 odd", op="linear", dir="train", T=191, B=8, Hq=6, Hk=3, D=80, Dv=48, dtype="f32", ragged=True, state=True),
        # training at T=256 B=64 H=1024, 16 heads of 64
        dict(name="linear train bf16", op="linear", dir="train", T=256, B=64, Hq=16, Hk=16, D=64, Dv=64, dtype="bf16", ragged=True, state=False),
        # training on long documents
        dict(name="linear train long bf16", op="linear", dir="train", T=4096, B=8, Hq=16, Hk=16, D=128, Dv=128, dtype="bf16", ragged=False, state=False),
        # one sampling step of 16 sequences over a large vocabulary, fp32 logits, the answers so far time-major
        dict(name="penalty step f32", op="penalty", N=16, V=131072, L=512, time_major=True, bias=False, mask=False, dtype="f32"),
        # constrained answers, an odd vocabulary, a grammar's mask and a bias
        dict(name="penalty grammar f16 odd", op="penalty", N=37, V=10007, L=300, time_major=False, bias=True, mask=True, dtype="f16"),
        # a large batch with long answers
        dict(name="penalty batch bf16", op="penalty", N=512, V=50000, L=2048, time_major=False, bias=True, mask=True, dtype="bf16"),
        # the parameters of the small encoder-decoder (32 words, heads 4 x 32)
        dict(name="adamw small f32", op="adamw", I=64, H=128, layers=1, V=32, bits=32, clip=False, dtype="f32"),
        # four layers of I=512 H=1024 and an odd vocabulary's table, the gradient's norm held below 1
        dict(name="adamw layers f32", op="adamw", I=512, H=1024, layers=4, V=10007, bits=32, clip=True, dtype="f32"),
        # four layers of I=512 H=2048 and a large vocabulary's table, 8-bit states, bf16 with a 32-bit copy
        dict(name="adamw large bf16 8-bit", op="adamw", I=512, H=2048, layers=4, V=50000, bits=8, clip=False, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "penalty", "adamw"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op == "linear":
        way = rng.choice(["step", "fwd", "train"])
        Hk, G = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([1, 1, 2, 4])
        D = rng.choice([32, 64, 64, 128, 128, 256, rng.randint(8, 256)])
        Dv = D if rng.random() < 0.6 else rng.choice([64, 128, 256, rng.randint(8, 256)])
        B = _log(rng, 1, 256 if way == "step" else 64)
        T = 1 if way == "step" else _log(rng, 2, 32768 if way == "fwd" else 4096)
        # no more work than the longest training case, fp32 products running at a quarter of the rate at best, and no
        # states of more than 256 MB
        most = 8 * 16 * 4096 * 128 * 128 // (4 if dtype == "f32" else 1)
        while B * Hk * G * (T + 16) * D * Dv > most or B * Hk * D * Dv > 1 << 26:
            B, T = max(1, B // 2), T if B > 1 else max(2, T // 2)
        return dict(op=op, dir=way, T=T, B=B, Hq=Hk * G, Hk=Hk, D=D, Dv=Dv, dtype=dtype, ragged=way != "step" and rng.random() < 0.5,
                    state=way == "step" or rng.random() < 0.5)
    if op == "penalty":
        V = _log(rng, 100, 131072)
        N = _log(rng, 1, 512)
        while N * V > 512 * 50000:
            N = max(1, N // 2)
        return dict(op=op, N=N, V=V, L=_log(rng, 1, 4096), time_major=rng.random() < 0.5, bias=rng.random() < 0.5,
                    mask=rng.random() < 0.5, dtype=dtype)
    return dict(op=op, I=_log(rng, 16, 512), H=_log(rng, 16, 2048), layers=rng.randint(1, 4), V=_log(rng, 32, 50000),
                bits=rng.choice([8, 32]), clip=rng.random() < 0.5, dtype=dtype)


def _shapes(case):
    """The parameters of an embedding, LSTM layers and the linear layer to the logits."""
    I, H, V = case["I"], case["H"], case["V"]
    shapes = [(V, I)]
    for n in range(case["layers"]):
        shapes += [(4 * H, H + (H if n else I)), (4 * H,)]
    return shapes + [(V, H), (V,)]


def _places(shapes):
    """Where each tensor begins, at a multiple of a block, and the length of them all."""
    at, end = [], 0
    for s in shapes:
        at.append(end)
        end += -(-math.prod(s) // BLOCK) * BLOCK
    return at, end


def prepare(case, seed):
    dev = torch.device("cuda" if torch.cuda.is_available() else "cpu")
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev)

    s = dict(case=case)
    if case["op"] == "linear":
        T, B, Hq, Hk, D, Dv = (case[k] for k in ("T", "B", "Hq", "Hk", "D", "Dv"))
        s["scale"] = D ** -0.5
        s["q"], s["k"], s["v"] = normal(T, B, Hq, D).to(dt), normal(T, B, Hk, D).to(dt), normal(T, B, Hk, Dv).to(dt)
        # memories of 8 steps up to 2000, spread over the heads
        s["log_decay"] = -torch.exp(torch.linspace(math.log(1 / 8), math.log(1 / 2000), Hk, device=dev)) * (0.8 + 0.4 * torch.rand(Hk, generator=g, device=dev))
        s["state"] = normal(B, Hk, D, Dv) * 2 if case["state"] else None
        s["length"] = None
        if case["ragged"]:
            u = torch.rand(B, generator=g, device=dev)
            s["length"] = (T * (0.25 + 0.75 * u)).ceil().clamp(1, T).to(torch.int32)
        if case["dir"] == "train":
            s["do"] = normal(T, B, Hq, Dv).to(dt)
            s["dstate"] = normal(B, Hk, D, Dv) if case["state"] else None
    elif case["op"] == "penalty":
        N, V, L = case["N"], case["V"], case["L"]
        s["logits"] = (normal(N, V) * 2.5).to(dt)
        # the answers so far as text has them: id r with a share of about 1/r, -1 past each answer's end
        u = torch.rand((N, L), generator=g, device=dev)
        ids = (torch.exp(u * math.log(V)).long()).clamp(max=V - 1)
        s["length"] = (L * torch.rand(N, generator=g, device=dev)).ceil().clamp(1, L).to(torch.int32)
        ids = ids.masked_fill(torch.arange(L, device=dev)[None] >= s["length"][:, None], -1)
        s["history"] = ids.t().contiguous().t() if case["time_major"] else ids
        s["repetition"], s["presence"], s["frequency"] = (1 + 0.3 * torch.rand(N, generator=g, device=dev), 0.5 * torch.rand(N, generator=g, device=dev),
                                                          0.2 * torch.rand(N, generator=g, device=dev))
        s["bias"] = normal(V) if case["bias"] else None
        # a grammar allows a third of the tokens: bit v % 32 of word v / 32
        s["mask"] = None
        if case["mask"]:
            allowed = torch.rand((N, -(-V // 32) * 32), generator=g, device=dev) < 1 / 3
            bits = torch.arange(32, device=dev)
            s["mask"] = (allowed.view(N, -1, 32).long() << bits).sum(2).to(torch.int32)
    else:
        shapes = _shapes(case)
        at, n = _places(shapes)
        there = torch.zeros(n, dtype=torch.bool, device=dev)
        for o, shape in zip(at, shapes):
            there[o : o + math.prod(shape)] = True
        s["t"], s["lr"], s["betas"], s["eps"], s["decay"], s["clip"] = 100, 1e-4, (0.9, 0.98), 1e-8, 0.01, 1.0 if case["clip"] else None
        master = normal(n) * 0.03 * there
        s["params"] = master.to(dt)
        s["master"] = None if dt == torch.float32 else master
        # gradients of a few large and many small values
        s["grads"] = (normal(n) * torch.exp(normal(n)) * 0.01 * there).to(dt)
        m = normal(n) * torch.exp(normal(n)) * 0.003 * there
        v = (m * m + 1e-6 * torch.rand(n, generator=g, device=dev)) * 4 * there
        if case["bits"] == 8:
            s["m"], s["m_scale"] = _to8(m, False)
            s["v"], s["v_scale"] = _to8(torch.sqrt(v), True)
        else:
            s["m"], s["v"] = m, v
    if own:
        from layer_lstm_amd import lstm
        code = {"f32": lstm.F32, "bf16": lstm.BF16, "f16": lstm.F16}[case["dtype"]]
        if case["op"] == "linear":
            s["op"] = lstm.LinearAttention(T, B, Hq, Hk, D, Dv, code, scale=s["scale"])
        elif case["op"] == "penalty":
            s["op"] = lstm.Penalty(N, V, code)
        else:
            def tensors(x):
                return [x[o : o + math.prod(shape)].view(shape) for o, shape in zip(at, shapes)]
            s["op"] = lstm.AdamW(tensors(s["params"]), s["lr"], s["betas"], s["eps"], s["decay"], bits=case["bits"], clip=s["clip"])
            s["op"].set_step(s["t"])
            s["list"] = tensors(s["grads"])
            for name in ("master", "m", "v", "m_scale", "v_scale"):
                if s.get(name) is not None:
                    getattr(s["op"], name).copy_(s[name])
    return s


def run(s):
    case = s["case"]
    if case["op"] == "linear":
        if case["dir"] == "step":
            if own:
                return s["op"].step(s["q"], s["k"], s["v"], s["log_decay"], s["state"]), s["state"]
            return _linear_step(s["q"], s["k"], s["v"], s["log_decay"], s["scale"], s["state"]), s["state"]
        if not own:
            return _linear(s["q"], s["k"], s["v"], s["log_decay"], s["scale"], s["state"], s["length"], s.get("do"), s.get("dstate"))
        out = s["op"].forward(s["q"], s["k"], s["v"], s["log_decay"], s["state"], s["length"])
        if case["dir"] == "fwd":
            return out
        return (*out, *s["op"].backward(s["do"], s["q"], s["k"], s["v"], s["log_decay"], s["state"], s["length"], s["dstate"]))
    if case["op"] == "penalty":
        args = [s[k] for k in ("logits", "history", "length", "repetition", "presence", "frequency", "bias", "mask")]
        return s["op"].forward(*args) if own else _penalty(*args)
    if not own:
        return _adamw(s)
    op = s["op"]
    op.step(s["list"])
    out = [s["params"], op.m, op.v]
    return tuple(out + [x for x in (op.m_scale, op.v_scale, op.master) if x is not None])


# ---- the operators in plain 32-bit operations ----

def _linear_step(q, k, v, log_decay, scale, state):
    """o of one step, the state moved on in place."""
    B, Hk, D, Dv = state.shape
    state.mul_(torch.exp(log_decay.clamp(max=0.0))[None, :, None, None]).add_(k[0].float()[..., None] * v[0].float()[:, :, None])
    o = torch.matmul(q[0].float().view(B, Hk, -1, D), state) * scale
    return o.to(q.dtype).view(1, B, -1, Dv)


def _linear(q, k, v, log_decay, scale, state, length, do=None, dstate=None):
    """o, the state after the last step and, with do, dq, dk, dv and the gradient of the state before the first: products
    of chunks of C steps, and of chunks with the states of the chunks before them."""
    T, B, Hq, D = q.shape
    Hk, Dv = k.shape[2], v.shape[3]
    G = Hq // Hk
    C = 64 if T > 64 else T
    n = -(-T // C)
    dev = q.device
    t = torch.arange(n * C, device=dev)
    last = torch.full((B,), T, device=dev) if length is None else length.long().clamp(0, T)
    real = t[None] < last[:, None]  # [B, n C]

    def rows(x):  # [T, B, H, d] -> [B, Hk, G or 1, n, C, d], zeros past the end
        x = torch.nn.functional.pad(x.float(), (0, 0, 0, 0, 0, 0, 0, n * C - T)).permute(1, 2, 0, 3)
        x = torch.where(real[:, None, :, None], x, 0.0)
        return x.reshape(B, Hk, x.shape[1] // Hk, n, C, x.shape[3])

    def back(x, dtype):  # the reverse
        x = x.reshape(B, -1, n * C, x.shape[-1])[:, :, :T]
        return torch.where(real[:, None, :T, None], x, 0.0).permute(2, 0, 1, 3).to(dtype).contiguous()

    # powers of the decay, from differences of whole numbers in 64 bits
    ld = log_decay.double().clamp(max=0.0)
    i = torch.arange(C, device=dev)

    def power(e):  # decay^e of a [..] tensor of whole numbers, 0 for negative ones: [Hk, ..]
        p = torch.exp(ld.view(-1, *([1] * e.dim())) * e.clamp(min=0).double())
        return torch.where(e >= 0, p, 0.0).float()

    inner = power(i[:, None] - i[None])[None, :, None, None]  # [1, Hk, 1, 1, C, C]: row i, column j
    # steps of sequence b in chunk c, and their sum over chunks: chunk c's contributions reach the start of chunk d
    steps = (last[:, None] - C * torch.arange(n, device=dev)[None]).clamp(0, C)  # [B, n]
    before = torch.cumsum(steps, 1) - steps  # steps before chunk c

    def powers(e):  # decay^e of [B, ..], 0 for negative ones: [B, Hk, ..]
        p = torch.exp(ld.view(1, -1, *([1] * (e.dim() - 1))) * e.clamp(min=0)[:, None].double())
        return torch.where(e[:, None] >= 0, p, 0.0).float()

    tri = torch.arange(n, device=dev)
    qf, kf, vf = rows(q), rows(k), rows(v)
    S0 = torch.zeros((B, Hk, D, Dv), device=dev) if state is None else state

    def ahead(x, y):
        """Sum over a chunk's steps j of decay^(steps left after j) x_j y_j^T, over its heads: [B, Hk, n, d, e]."""
        w = powers(steps[:, :, None] - 1 - i[None, None])  # [B, Hk, n, C]
        return torch.matmul((x * w[:, :, None, :, :, None]).transpose(4, 5), y).sum(2)

    # the state before each chunk and after the last
    U = ahead(kf, vf)
    end = before + steps
    gap = before[:, None, :] - end[:, :, None]  # from the end of chunk c (row) to the start of chunk d (column)
    far = powers(torch.where(tri[:, None] < tri[None], gap, -1))  # [B, Hk, n, n]
    flat = U.reshape(B, Hk, n, D * Dv)
    S = torch.matmul(far.transpose(2, 3), flat) + powers(before)[..., None] * S0.reshape(B, Hk, 1, D * Dv)
    S = S.view(B, Hk, 1, n, D, Dv)
    final = (powers(end[:, -1:] - end)[..., None] * flat).sum(2) + powers(last[:, None])[..., None].view(B, Hk, 1) * S0.reshape(B, Hk, D * Dv)
    final = final.view(B, Hk, D, Dv)
    since = power(i + 1)[None, :, None, None, :, None]  # [1, Hk, 1, 1, C, 1]
    o = torch.matmul(qf, S) * since + torch.matmul(torch.matmul(qf, kf.transpose(4, 5)) * inner, vf)
    o = back(o * scale, q.dtype)
    if do is None:
        return o, final
    dof = rows(do)
    dq = torch.matmul(dof, S.transpose(4, 5)) * since + torch.matmul(torch.matmul(dof, vf.transpose(4, 5)) * inner, kf)
    # the gradient of the state after each chunk and before the first
    dT = torch.zeros((B, Hk, D, Dv), device=dev) if dstate is None else dstate
    w = power(i + 1)[None, :, None, None, :, None]
    X = torch.matmul((qf * w).transpose(4, 5), dof).sum(2) * scale  # as it reaches the state before the chunk
    gap = before[:, None, :] - end[:, :, None]
    far = powers(torch.where(tri[:, None] < tri[None], gap, -1))  # from the end of chunk c to the start of chunk d
    flat = X.reshape(B, Hk, n, D * Dv)
    R = torch.matmul(far, flat) + powers(end[:, -1:] - end)[..., None] * dT.reshape(B, Hk, 1, D * Dv)
    R = R.view(B, Hk, n, D, Dv)
    dS0 = (powers(before)[..., None] * flat).sum(2) + powers(last[:, None])[..., None].view(B, Hk, 1) * dT.reshape(B, Hk, D * Dv)
    left = powers(steps[:, :, None] - 1 - i[None, None])[..., None]  # [B, Hk, n, C, 1]
    kg, vg = kf[:, :, 0], vf[:, :, 0]  # [B, Hk, n, C, d]
    p = torch.matmul(qf, kf.transpose(4, 5)) * inner * scale
    dv = torch.matmul(kg, R) * left + torch.matmul(p.transpose(4, 5), dof).sum(2)
    dp = torch.matmul(dof, vf.transpose(4, 5)) * inner * scale
    dk = torch.matmul(vg, R.transpose(3, 4)) * left + torch.matmul(dp.transpose(4, 5), qf).sum(2)
    return o, final, back(dq * scale, q.dtype), back(dk, q.dtype), back(dv, q.dtype), dS0.view(B, Hk, D, Dv)


def _penalty(logits, history, length, repetition, presence, frequency, bias, mask):
    N, V = logits.shape
    L = history.shape[1]
    x = logits.float()
    real = (torch.arange(L, device=x.device)[None] < length[:, None]) & (history >= 0) & (history < V)
    count = torch.zeros((N, V + 1), device=x.device).scatter_add_(1, torch.where(real, history, V), torch.ones_like(history, dtype=torch.float32))[:, :V]
    seen = count > 0
    x = torch.where(seen, torch.where(x > 0, x / repetition[:, None], x * repetition[:, None]), x)
    x = torch.where(seen, x - (presence[:, None] + frequency[:, None] * count), x)
    if bias is not None:
        x = x + bias
    if mask is not None:
        allowed = (mask[:, :, None] >> torch.arange(32, dtype=torch.int32, device=x.device)) & 1
        x = torch.where(allowed.view(N, -1)[:, :V] != 0, x, -math.inf)
    return x.to(logits.dtype)


def _to8(x, up):
    """x in blocks as e4m3 numbers times a scale each; `up`: a value over zero is held as at least the smallest number.
    Blocks of nothing above 2^-100 are zeros."""
    b = x.view(-1, BLOCK)
    most = b.abs().amax(1, keepdim=True)
    most = torch.where(most > 2.0**-100, most, 0.0)
    scale = most / 448.0
    y = b * torch.where(most > 0, 448.0 / most, 0.0)
    if up:
        y = torch.where((b > 0) & (most > 0), y.clamp(min=2.0**-9), 0.0)
    return y.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(-1), scale[:, 0]


def _from8(x, scale):
    return (x.float().view(-1, BLOCK) * scale[:, None]).view(-1)


def _adamw(s):
    s["t"] += 1
    (b1, b2), t, bits = s["betas"], s["t"], s["case"]["bits"]
    g = s["grads"].float()
    if s["clip"] is not None:
        norm = torch.sqrt((g.double() * g.double()).sum())
        g = g * torch.where(norm > s["clip"], s["clip"] / norm, 1.0).float()
    p = s["params"] if s["master"] is None else s["master"]
    m = s["m"] if bits == 32 else _from8(s["m"], s["m_scale"])
    v = s["v"] if bits == 32 else _from8(s["v"], s["v_scale"]).square()
    m = m * b1 + g * (1 - b1)
    v = v * b2 + (g * g) * (1 - b2)
    root = torch.sqrt(v)
    step = m / (root * (1 / math.sqrt(1 - b2**t)) + s["eps"])
    p.copy_(p * (1 - s["lr"] * s["decay"]) - step * (s["lr"] / (1 - b1**t)))
    out = [s["params"], s["m"], s["v"]]
    if bits == 32:
        s["m"].copy_(m), s["v"].copy_(v)
    else:
        for name, new in (("m", _to8(m, False)), ("v", _to8(root, True))):
            s[name].copy_(new[0]), s[name + "_scale"].copy_(new[1])
        out += [s["m_scale"], s["v_scale"]]
    if s["master"] is not None:
        s["params"].copy_(p)
        out.append(s["master"])
    return tuple(out)


# ---- the definitions in 64 bits ----

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "linear":
        return _linear_exact(s)
    if case["op"] == "penalty":
        return _penalty_exact(s)
    return _adamw_exact(s)


def _linear_exact(s):
    """Every step's sum over all steps before it, one sequence and head at a time, a block of rows at a time; gradients
    by automatic differentiation."""
    case = s["case"]
    T, B, Hq, Hk = (case[k] for k in ("T", "B", "Hq", "Hk"))
    train, G = case["dir"] == "train", Hq // Hk
    # the sums over pairs of steps, and the launches
    if B * Hq * T * T * (case["D"] + case["Dv"]) * (3 if train else 1) > 2e13 or B * Hk * (1 + G * (T // 2048 + 1)) * (3 if train else 1) > 15000:
        return None
    q, k, v = (s[n].double() for n in ("q", "k", "v"))
    S0 = torch.zeros((B, Hk, case["D"], case["Dv"]), dtype=torch.float64, device=q.device) if s["state"] is None else s["state"].double()
    dq, dk, dv, dS0 = (torch.zeros_like(x) for x in (q, k, v, S0))
    o, final = torch.zeros((T, B, Hq, case["Dv"]), dtype=torch.float64, device=q.device), S0.clone()
    for b in range(B):
        n = T if s["length"] is None else int(s["length"][b])
        at = torch.arange(n, device=q.device)
        for h in range(Hk):
            ld = s["log_decay"][h].double()
            heads = slice(h * G, (h + 1) * G)
            leaves = [x.clone().requires_grad_(train) for x in (q[:n, b, heads], k[:n, b, h], v[:n, b, h], S0[b, h])]
            qh, kh, vh, Sh = leaves
            S = torch.exp(ld * n) * Sh + (kh * torch.exp(ld * (n - 1 - at))[:, None]).t() @ vh
            final[b, h] = S.detach()
            if train and s["dstate"] is not None:
                S.backward(s["dstate"][b, h].double(), retain_graph=True)
            for lo in range(0, n, 2048):
                r = at[lo : lo + 2048]
                keys = kh[: lo + r.numel()]
                w = r[:, None] - at[None, : keys.shape[0]]
                w = torch.where(w >= 0, torch.exp(ld * w.clamp(min=0)), 0.0)
                for g in range(G):
                    y = ((qh[r, g] @ keys.t()) * w) @ vh[: keys.shape[0]] + torch.exp(ld * (r + 1))[:, None] * (qh[r, g] @ Sh)
                    y = y * s["scale"]
                    o[r, b, h * G + g] = y.detach()
                    if train:
                        y.backward(s["do"][r, b, h * G + g].double(), retain_graph=True)
            if train:
                zero = [torch.zeros_like(x) if x.grad is None else x.grad for x in leaves]
                dq[:n, b, heads], dk[:n, b, h], dv[:n, b, h], dS0[b, h] = zero
    return (o, final, dq, dk, dv, dS0) if train else (o, final)


def _penalty_exact(s):
    x = s["logits"].double()
    N, V = x.shape
    for n in range(N):
        said = s["history"][n, : int(s["length"][n])]
        ids, count = torch.unique(said[(said >= 0) & (said < V)], return_counts=True)
        r, old = s["repetition"][n].double(), x[n, ids]
        x[n, ids] = torch.where(old > 0, old / r, old * r) - s["presence"][n].double() - s["frequency"][n].double() * count
    if s["bias"] is not None:
        x = x + s["bias"].double()
    if s["mask"] is not None:
        v = torch.arange(V, device=x.device)
        x[(torch.bitwise_right_shift(s["mask"].long()[:, v // 32], v % 32) & 1) == 0] = -math.inf
    return x


def _adamw_exact(s):
    (b1, b2), t, bits = s["betas"], s["t"] + 1, s["case"]["bits"]
    g = s["grads"].double()
    if s["clip"] is not None:
        g = g * min(1.0, s["clip"] / float(torch.linalg.vector_norm(g)))
    p = (s["params"] if s["master"] is None else s["master"]).double()
    if bits == 8:
        m = (s["m"].double().view(-1, BLOCK) * s["m_scale"].double()[:, None]).view(-1)
        v = (s["v"].double().view(-1, BLOCK) * s["v_scale"].double()[:, None]).view(-1) ** 2
    else:
        m, v = s["m"].double(), s["v"].double()
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    new = p - s["lr"] * (s["decay"] * p + (m / (1 - b1**t)) / (torch.sqrt(v / (1 - b2**t)) + s["eps"]))
    out = [new, m, v]
    if bits == 8:  # the 8-bit numbers themselves are roundings
        out = [new, None, None, m.view(-1, BLOCK).abs().amax(1) / 448, torch.sqrt(v).view(-1, BLOCK).amax(1) / 448]
    return tuple(out + ([new] if s["master"] is not None else []))


# ---- what a pass cannot do without ----

def work(case):
    e = SIZE[case["dtype"]]
    if case["op"] == "linear":
        T, B, Hq, Hk, D, Dv = (case[k] for k in ("T", "B", "Hq", "Hk", "D", "Dv"))
        rows = B * T * (0.625 if case["ragged"] else 1.0)  # of the mean length
        state = 4 * B * Hk * D * Dv
        q, o, k, v = e * rows * Hq * D, e * rows * Hq * Dv, e * rows * Hk * D, e * rows * Hk * Dv
        # the recurrence's own products: the state's update, and its product with each query
        flops = 2 * rows * D * Dv * (Hk + Hq)
        if case["dir"] != "train":
            return dict(bytes=q + o + k + v + state * (2 if case["state"] else 1), flops=flops)
        # q, do read, o, dq written, k, v read, dk, dv written; both states again, dk, dv and dq each a product with a state
        return dict(bytes=2 * (q + o + k + v) + state * (4 if case["state"] else 2), flops=flops + 2 * rows * D * Dv * (2 * Hq + 3 * Hk))
    if case["op"] == "penalty":
        N, V, L = case["N"], case["V"], case["L"]
        return dict(bytes=2 * e * N * V + 8 * N * L // 2 + (4 * V if case["bias"] else 0) + (N * V // 8 if case["mask"] else 0), flops=3 * N * V)
    n = sum(math.prod(s) for s in _shapes(case))
    state = 16 if case["bits"] == 32 else 4
    return dict(bytes=n * (state + (12 if e == 4 else 4 + 8)), flops=15 * n)
