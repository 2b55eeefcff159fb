"""The operators around an LSTM that turn it into a sequence-to-sequence model,
as cases to measure: the embedding of tokens and its gradient, the decoder's
cross attention to the encoder's states and its gradient, and the log
probabilities of given tokens with their entropy and best alternatives.

`run` computes a case in plain 32-bit torch operations, or, with `own` set,
through layer_lstm_amd.lstm.  `exact` gives the same outputs in 64 bits from
the definitions, by indexing and automatic differentiation.

Tensors are time-major as everywhere in the library: tokens [T,B], states
[T,B,heads,D], lengths int32 [B].
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


def listed():
    return [
        # the decoder's next input in serving: one token of each of 16 sequences, 2048 features
        dict(name="embed step bf16", op="embed", dir="fwd", T=1, B=16, V=32768, D=2048, dtype="bf16"),
        # all inputs of the largest training batch (T=256 B=256 I=1024)
        dict(name="embed batch bf16", op="embed", dir="fwd", T=256, B=256, V=50000, D=1024, dtype="bf16"),
        # the table's gradient in a small fp32 training step (T=64 B=32), an odd vocabulary, rows no multiple of 16 bytes
        dict(name="embed gradient f32 odd", op="embed", dir="bwd", T=64, B=32, V=10007, D=257, dtype="f32"),
        # the table's gradient of the largest training batch
        dict(name="embed gradient bf16", op="embed", dir="bwd", T=256, B=256, V=50000, D=1024, dtype="bf16"),
        # one decoder step of 16 sequences against a 512-step encoder, H = 2048 in 16 heads
        dict(name="attend step bf16", op="attend", dir="fwd", Tq=1, Tk=512, B=16, Hq=16, Hk=16, D=128, dtype="bf16", holes=False),
        # one decoder step against very long encoder states, four query heads to a key head
        dict(name="attend step long f16", op="attend", dir="fwd", Tq=1, Tk=32768, B=8, Hq=32, Hk=8, D=128, dtype="f16", holes=False),
        # a small fp32 training step, odd lengths and head size, key holes (dropped encoder states)
        dict(name="attend train f32 odd", op="attend", dir="train", Tq=37, Tk=191, B=8, Hq=6, Hk=3, D=80, dtype="f32", holes=True),
        # training at T=256 B=64 H=1024, 16 heads of 64
        dict(name="attend train bf16", op="attend", dir="train", Tq=256, Tk=256, B=64, Hq=16, Hk=16, D=64, dtype="bf16", holes=False),
        # training on long documents, shared key heads
        dict(name="attend train long bf16", op="attend", dir="train", Tq=1024, Tk=4096, B=8, Hq=32, Hk=8, D=128, dtype="bf16", holes=False),
        # one sampling step of 16 sequences: the chosen token's score and 8 alternatives of a large vocabulary, fp32 logits
        dict(name="logprob step f32", op="logprob", dir="fwd", N=16, V=131072, K=8, dtype="f32"),
        # scoring given sequences, an odd vocabulary, banned tokens, alternatives for inspection
        dict(name="logprob score f16 odd", op="logprob", dir="fwd", N=2049, V=10007, K=5, dtype="f16"),
        # the loss of a training step (T=256 B=64) with an entropy bonus, and the logits' gradient
        dict(name="logprob train bf16", op="logprob", dir="train", N=16384, V=32768, K=0, dtype="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["embed", "attend", "logprob"])
    dtype = rng.choice(["f32", "bf16", "f16"])
    if op == "embed":
        D = rng.choice([_log(rng, 16, 2048), 8 * _log(rng, 2, 256)])
        N = _log(rng, 1, 65536)
        B = min(N, _log(rng, 1, 256))
        return dict(op=op, dir=rng.choice(["fwd", "bwd"]), T=max(1, N // B), B=B, V=_log(rng, 100, 65536), D=D, dtype=dtype)
    if op == "attend":
        Hk, G = rng.choice([1, 2, 3, 4, 8, 16]), rng.choice([1, 1, 2, 4, 8])
        Hk = max(1, min(Hk, 32 // G))
        D = rng.choice([32, 64, 80, 128, 128, 256, rng.randint(8, 256)])
        B = _log(rng, 1, 64)
        step = rng.random() < 0.4
        Tq = 1 if step else _log(rng, 2, 1024)
        Tk = _log(rng, 1, 32768 if step else 4096)
        # no more work than the longest training case, fp32 products running at a sixteenth of the rate, and no more
        # keys and values than the longest step
        most = 8 * 32 * 1024 * 4096 * 128 // (16 if dtype == "f32" else 1)
        while B * Hk * G * Tq * Tk * D > most or B * Hk * Tk * D > 8 * 8 * 32768 * 128:
            B, Tk, Tq = max(1, B // 2), max(1, (Tk * 3 + 3) // 4), max(1, (Tq * 3 + 3) // 4)
        return dict(op=op, dir="fwd" if step else rng.choice(["fwd", "train"]), Tq=Tq, Tk=Tk, B=B, Hq=Hk * G, Hk=Hk, D=D,
                    dtype=dtype, holes=rng.random() < 0.3)
    V = _log(rng, 100, 131072)
    N = _log(rng, 1, 16384)
    while N * V > 16384 * 32768:
        N = max(1, N // 2)
    train = rng.random() < 0.5
    return dict(op=op, dir="train" if train else "fwd", N=N, V=V, K=rng.choice([0, 1, 5, 8, 20]), dtype=dtype)


def _lengths(n, longest, g, dev):
    """Ragged lengths from a quarter of the longest up to all of it."""
    u = torch.rand(n, generator=g, device=dev)
    return (longest * (0.25 + 0.75 * u)).ceil().clamp(1, longest).to(torch.int32)


def _tokens(T, B, V, g, dev):
    """Tokens as text has them: id r with a share of about 1/r, id 0 the padding past each sequence's end."""
    u = torch.rand((T, B), generator=g, device=dev)
    ids = (torch.exp(u * math.log(V)).long()).clamp(1, max(1, V - 1))
    past = torch.arange(T, device=dev)[:, None] >= _lengths(B, T, g, dev)[None, :]
    return ids.masked_fill(past, 0)


def prepare(case, seed):
    dev = torch.device("cuda" if torch.cuda.is_available() else "cpu")
    g = torch.Generator(device=dev).manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(shape, generator=g, device=dev).to(dt)

    s = dict(case=case)
    if case["op"] == "embed":
        T, B, V, D = case["T"], case["B"], case["V"], case["D"]
        s["scale"], s["padding"] = math.sqrt(D), 0
        s["ids"] = _tokens(T, B, V, g, dev)
        if case["dir"] == "fwd":
            s["table"] = normal(V, D) / math.sqrt(D)
        else:
            s["dout"] = normal(T, B, D)
    elif case["op"] == "attend":
        Tq, Tk, B, Hq, Hk, D = (case[k] for k in ("Tq", "Tk", "B", "Hq", "Hk", "D"))
        s["scale"] = 1 / math.sqrt(D)
        s["q"], s["k"], s["v"] = normal(Tq, B, Hq, D), normal(Tk, B, Hk, D), normal(Tk, B, Hk, D)
        s["length"] = _lengths(B, Tk, g, dev)
        s["mask"] = (torch.rand((B, Tk), generator=g, device=dev) < 0.8).to(torch.uint8) if case["holes"] else None
        if case["dir"] == "train":
            s["do"] = normal(Tq, B, Hq, D)
    else:
        N, V, K = case["N"], case["V"], case["K"]
        # a peaked distribution, as a model's answers have it
        s["logits"] = (torch.randn((N, V), generator=g, device=dev) * 2.5).to(dt)
        if case["dir"] == "fwd":  # banned tokens
            s["logits"][:, torch.randperm(V, generator=g, device=dev)[: V // 100]] = -math.inf
        best = s["logits"].argmax(1)
        ids = torch.randint(0, V, (N,), generator=g, device=dev)
        u = torch.rand(N, generator=g, device=dev)
        s["targets"] = torch.where(u < 0.5, best, ids).masked_fill(u > 0.9, -1)  # a tenth is padding
        if case["dir"] == "train":
            # the mean loss, scaled up in fp16 as its training does
            each = (4096.0 if case["dtype"] == "f16" else 1.0) / N
            s["dlogp"] = torch.full((N,), -each, device=dev)
            s["dentropy"] = torch.full((N,), -0.01 * each, device=dev)
            s["dtop"] = torch.randn((N, K), generator=g, device=dev) * each if K else None
    if own:
        from layer_lstm_amd import lstm
        code = {"f32": lstm.F32, "bf16": lstm.BF16, "f16": lstm.F16}[case["dtype"]]
        if case["op"] == "embed":
            s["op"] = lstm.Embedding(case["T"] * case["B"], V, D, code, scale=s["scale"], padding=s["padding"])
        elif case["op"] == "attend":
            s["op"] = lstm.Attention(Tq, Tk, B, Hq, Hk, D, code, scale=s["scale"])
        else:
            s["op"] = lstm.LogProb(N, V, code, top=K)
    return s


def run(s):
    op, way = s["case"]["op"], s["case"]["dir"]
    if op == "embed":
        if way == "fwd":
            return s["op"].forward(s["ids"], s["table"]) if own else _embed(s["ids"], s["table"], s["scale"])
        if own:
            return s["op"].backward(s["ids"], s["dout"])
        return _embed_gradient(s["ids"], s["dout"], s["case"]["V"], s["scale"], s["padding"])
    if op == "attend":
        if not own:
            return _attend(s["q"], s["k"], s["v"], s["length"], s["mask"], s["scale"], s.get("do"))
        o, lse = s["op"].forward(s["q"], s["k"], s["v"], s["length"], s["mask"])
        if way == "fwd":
            return o, lse
        dq, dk, dv = s["op"].backward(s["do"], s["q"], s["k"], s["v"], s["length"], s["mask"])
        return o, lse, dq, dk, dv
    if not own:
        return _logprob(s["logits"], s["targets"], s["case"]["K"], way == "train", s.get("dlogp"), s.get("dentropy"), s.get("dtop"))
    out = s["op"].forward(s["logits"], s["targets"])
    if way == "fwd":
        return out
    return (*out, s["op"].backward(s["logits"], s["targets"], s["dlogp"], s["dentropy"], s["dtop"]))


# ---- the operators in plain 32-bit operations ----

def _embed(ids, table, scale):
    return (table[ids].float() * scale).to(table.dtype)


def _embed_gradient(ids, dout, V, scale, padding):
    rows = dout.reshape(-1, dout.shape[-1]).float() * scale
    flat = ids.reshape(-1)
    rows = rows.masked_fill((flat == padding)[:, None], 0.0)
    out = torch.zeros((V, rows.shape[1]), dtype=torch.float32, device=rows.device)
    return out.index_add_(0, flat, rows).to(dout.dtype)


def _attend(q, k, v, length, mask, scale, do):
    """o, lse and, with do, dq, dk, dv.  Rows of one key head: the query steps of each of its query heads."""
    Tq, B, Hq, D = q.shape
    Tk, Hk = k.shape[0], k.shape[2]
    G = Hq // Hk
    there = torch.arange(Tk, device=q.device)[None, :] < length[:, None]
    if mask is not None:
        there = there & (mask != 0)

    def rows(x):  # [Tq,B,Hq,D] -> [B,Hk,G*Tq,D]
        return x.float().permute(1, 2, 0, 3).reshape(B, Hk, G * Tq, D)

    def back(x):
        return x.reshape(B, Hq, Tq, D).permute(2, 0, 1, 3).to(q.dtype).contiguous()

    zero = ~there[:, None, :, None]
    qf, kf, vf = rows(q), k.float().permute(1, 2, 0, 3).masked_fill(zero, 0.0), v.float().permute(1, 2, 0, 3).masked_fill(zero, 0.0)
    s = (torch.matmul(qf, kf.transpose(2, 3)) * scale).masked_fill(~there[:, None, None, :], -math.inf)
    m = s.amax(3, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(s - m)
    total = p.sum(3, keepdim=True)
    lse = (torch.log(total) + m).reshape(B, Hq, Tq)
    p = p / torch.where(total == 0, 1.0, total)
    of = torch.matmul(p, vf)
    if do is None:
        return back(of), lse
    dof = rows(do)
    dp = torch.matmul(dof, vf.transpose(2, 3))
    ds = p * (dp - (dof * of).sum(3, keepdim=True)) * scale
    dq = torch.matmul(ds, kf)
    dk = torch.matmul(ds.transpose(2, 3), qf)
    dv = torch.matmul(p.transpose(2, 3), dof)
    return back(of), lse, back(dq), dk.permute(2, 0, 1, 3).to(q.dtype).contiguous(), dv.permute(2, 0, 1, 3).to(q.dtype).contiguous()


def _logprob(logits, targets, K, train, dlogp, dentropy, dtop):
    """logp, entropy, the K best alternatives' log probabilities and ids (equal logits by the lower id), and the
    logits' gradient in training."""
    x = logits.float() + 0.0
    m = x.amax(1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    e = torch.exp(x - m)
    lse = torch.log(e.sum(1, keepdim=True)) + m
    lp = torch.where(lse == -math.inf, -math.inf, x - lse)
    p = torch.exp(lp)
    plp = torch.where(p == 0, 0.0, p * lp)
    entropy = -plp.sum(1)
    real = (targets >= 0) & (targets < x.shape[1])
    at = torch.where(real, targets, 0)[:, None]
    logp = torch.where(real, lp.gather(1, at)[:, 0], 0.0)
    out = [logp, entropy]
    top = None
    if K:
        bits = x.view(torch.int32)
        order = bits ^ ((bits >> 31) & 0x7FFFFFFF)
        low = 0xFFFFFFFF - torch.arange(x.shape[1], device=x.device)
        best = torch.topk((order.long() << 32) | low, K, dim=1).values
        top = 0xFFFFFFFF - (best & 0xFFFFFFFF)
        out += [lp.gather(1, top), top]
    if train:
        gl = torch.where(real, dlogp, 0.0)[:, None]
        sums = gl if dtop is None else gl + dtop.sum(1, keepdim=True)
        grad = -p * sums - dentropy[:, None] * (plp + p * entropy[:, None])
        grad = grad.scatter_add(1, at, gl)
        if dtop is not None:
            grad = grad.scatter_add(1, top, dtop)
        out.append(grad.to(logits.dtype))
    return tuple(out)


# ---- the definitions in 64 bits ----

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "embed":
        if case["dir"] == "fwd":
            return torch.nn.functional.embedding(s["ids"], s["table"].double()) * s["scale"]
        table = torch.zeros((case["V"], case["D"]), dtype=torch.float64, device=s["ids"].device, requires_grad=True)
        keep = (s["ids"] != s["padding"])[..., None]
        torch.autograd.backward([table[s["ids"]] * s["scale"]], [s["dout"].double() * keep])
        return table.grad
    if case["op"] == "attend":
        return _attend_exact(s)
    return _logprob_exact(s)


def _attend_exact(s):
    """One sequence at a time, over its own keys alone, one softmax for every query head."""
    train = "do" in s
    G = s["case"]["Hq"] // s["case"]["Hk"]
    q, k, v = (s[n].double().requires_grad_(train) for n in ("q", "k", "v"))
    outs, lses = [], []
    for b in range(q.shape[1]):
        keys = torch.arange(int(s["length"][b]), device=q.device)
        if s["mask"] is not None:
            keys = keys[s["mask"][b, : keys.numel()] != 0]
        kb = k[:, b][keys].repeat_interleave(G, 1).permute(1, 2, 0)
        vb = v[:, b][keys].repeat_interleave(G, 1).permute(1, 0, 2)
        score = torch.matmul(q[:, b].permute(1, 0, 2), kb.contiguous()) * s["scale"]
        lse = torch.logsumexp(score, 2)
        o = torch.matmul(torch.exp(score - torch.where(lse == -math.inf, 0.0, lse)[..., None]), vb.contiguous()).permute(1, 0, 2)
        if train:
            torch.autograd.backward([o], [s["do"][:, b].double()])
        outs.append(o.detach())
        lses.append(lse.detach())
    out = [torch.stack(outs, 1), torch.stack(lses)]
    return tuple(out + [q.grad, k.grad, v.grad] if train else out)


def _logprob_exact(s):
    """A block of rows at a time; the ids of the alternatives are whole numbers and have no 64-bit value."""
    K, train = s["case"]["K"], s["case"]["dir"] == "train"
    parts = []
    for lo in range(0, s["case"]["N"], 2048):
        rows = slice(lo, lo + 2048)
        x = s["logits"][rows].double().requires_grad_(train)
        lp = torch.log_softmax(x, 1)
        t = s["targets"][rows]
        pick = torch.nn.functional.one_hot(t.clamp(min=0), x.shape[1]).bool()
        logp = torch.where(t >= 0, torch.where(pick, lp, 0.0).sum(1), 0.0)
        entropy = -torch.where(lp == -math.inf, 0.0, torch.exp(lp) * lp).sum(1)
        part = [logp.detach(), entropy.detach()]
        if K:
            ordered = lp.sort(dim=1, descending=True, stable=True)
            part.append(ordered.values[:, :K].detach())
        if train:
            loss = (logp * s["dlogp"][rows]).sum() + (entropy * s["dentropy"][rows]).sum()
            if K:
                loss = loss + (ordered.values[:, :K] * s["dtop"][rows]).sum()
            loss.backward()
            part.append(x.grad)
        parts.append(part)
    out = [torch.cat(p) for p in zip(*parts)]
    if K:
        out.insert(3, None)
    return tuple(out)


# ---- what a pass cannot do without ----

def work(case):
    e = SIZE[case["dtype"]]
    if case["op"] == "embed":
        n = case["T"] * case["B"]
        V, D = case["V"], case["D"]
        if case["dir"] == "fwd":  # ids, the rows of the table that occur (at most all), the output
            return dict(bytes=8 * n + e * D * (min(n, V) + n), flops=n * D)
        return dict(bytes=8 * n + e * D * (n + V), flops=2 * n * D)
    if case["op"] == "attend":
        Tq, Tk, B, Hq, Hk, D = (case[k] for k in ("Tq", "Tk", "B", "Hq", "Hk", "D"))
        keys = 0.625 * Tk * (0.8 if case["holes"] else 1.0)  # of the mean length
        q, kv = e * B * Tq * Hq * D, e * B * keys * Hk * D
        product = 2 * B * Hq * Tq * keys * D
        if case["dir"] == "fwd":
            return dict(bytes=2 * q + 2 * kv + 4 * B * Hq * Tq, flops=2 * product)
        # q, do, o, dq; k, v read; dk, dv written whole
        return dict(bytes=4 * q + 2 * kv + 2 * e * B * Tk * Hk * D + 4 * B * Hq * Tq, flops=7 * product)
    N, V, K = case["N"], case["V"], case["K"]
    train = case["dir"] == "train"
    return dict(bytes=(2 if train else 1) * e * N * V + (16 + 12 * K) * N, flops=(10 if train else 6) * N * V)
