"""A small encoder-decoder on the library's operators.

    python -m layer_lstm_amd.seq2seq [--steps 1000] [--batch 64] [--length 16]

Learns to write a sequence backwards: tokens -> embedding -> bidirectional
LSTM encoder; the shifted answer -> embedding -> LSTM decoder -> cross
attention over the encoder's states -> one linear layer over [state, context]
-> log probabilities.  Everything but that layer's products and the
optimiser's elementwise update runs in liblstm.so, forward and backward; the
decoder then answers token by token from the same operators at one step.
Sequences are ragged: padded steps hold the encoder's state (seq_length), are
no keys (k_length) and no targets (-1).
"""
from __future__ import annotations

import argparse
import math

import torch

from layer_lstm_amd import lstm

PAD, START = 0, 1  # ids; the words are 2 .. V - 1


class Seq2Seq:
    """Parameters and the plans of one batch shape: sources of up to S steps,
    answers of up to S steps, B sequences, V tokens, embedding size I, heads x
    head_dim the decoder's state (and both directions of the encoder's)."""

    def __init__(self, S, B, V, I=64, heads=4, head_dim=32, dtype=lstm.F32, seed=0, device="cuda"):
        self.S, self.B, self.V, self.I, self.heads, self.D, self.dtype = S, B, V, I, heads, head_dim, dtype
        self.H = H = heads * head_dim
        td = lstm.torch_dtype(dtype)
        g = torch.Generator(device=device).manual_seed(seed)

        def uniform(*shape, k):
            return ((torch.rand(shape, generator=g, device=device) * 2 - 1) * k).to(td)

        self.p = dict(
            table=uniform(V, I, k=1.0),
            enc_W=uniform(2, 2 * H, H // 2 + I, k=1 / math.sqrt(H // 2)), enc_b=uniform(2, 2 * H, k=0.1),
            dec_W=uniform(4 * H, H + I, k=1 / math.sqrt(H)), dec_b=uniform(4 * H, k=0.1),
            out_W=uniform(V, 2 * H, k=1 / math.sqrt(2 * H)))
        # one embedding call for the sources and the answers: ids [2 S, B]
        self.embed = lstm.Embedding(2 * S * B, V, I, dtype, padding=PAD)
        self.enc = lstm.Lstm(S, B, I, H // 2, dtype, bidirectional=True)
        self.dec = lstm.Lstm(S, B, I, H, dtype)
        self.attend = lstm.Attention(S, S, B, heads, heads, head_dim, dtype)
        self.logprob = lstm.LogProb(S * B, V, dtype)
        self._step = None

    def heads_of(self, x):
        return x.view(x.shape[0], x.shape[1], self.heads, self.D)

    def forward(self, source, answer_in, targets, length):
        """Mean log probability of the targets [S, B] (-1: none)."""
        S, B, p = self.S, self.B, self.p
        self.ids = torch.cat([source, answer_in])
        x = self.embed.forward(self.ids, p["table"])
        self.x_enc, self.x_dec = x[:S], x[S:]
        states, _, _ = self.enc.forward(self.x_enc, p["enc_W"], p["enc_b"], seq_length=length)
        y, _, _ = self.dec.forward(self.x_dec, p["dec_W"], p["dec_b"])
        self.keys, self.length = self.heads_of(states), length
        context, _ = self.attend.forward(self.heads_of(y), self.keys, self.keys, length)
        self.features = torch.cat([y, context.view(S, B, self.H)], 2).view(S * B, 2 * self.H)
        self.logits = self.features @ p["out_W"].t()
        self.targets = targets.reshape(-1)
        logp, _ = self.logprob.forward(self.logits, self.targets)
        self.count = (self.targets >= 0).sum()
        return logp.sum() / self.count

    def backward(self):
        """Gradients of minus the mean log probability, by parameter name."""
        S, B, H, p = self.S, self.B, self.H, self.p
        dlogp = (-1.0 / self.count.float()).expand(S * B).contiguous()
        dlogits = self.logprob.backward(self.logits, self.targets, dlogp)
        df = (dlogits @ p["out_W"]).view(S, B, 2 * H)
        q, dcontext = self.heads_of(self.dec.y), self.heads_of(df[:, :, H:].contiguous())
        dq, dk, dv = self.attend.backward(dcontext, q, self.keys, self.keys, self.length)
        zero = torch.zeros((B, H), dtype=df.dtype, device=df.device)
        dx_dec, dec_W, dec_b, _, _ = self.dec.backward(df[:, :, :H] + dq.view(S, B, H), zero, zero, self.x_dec,
                                                       p["dec_W"])
        zero = zero.view(2, B, H // 2)
        # the states are keys and values both
        dx_enc, enc_W, enc_b, _, _ = self.enc.backward((dk + dv).view(S, B, H), zero, zero, self.x_enc, p["enc_W"],
                                                       seq_length=self.length)
        table = self.embed.backward(self.ids, torch.cat([dx_enc, dx_dec]))
        return dict(table=table, enc_W=enc_W, enc_b=enc_b, dec_W=dec_W, dec_b=dec_b,
                    out_W=dlogits.t().contiguous() @ self.features)

    def answer(self, source, length, steps):
        """The likeliest token at every step, fed back: [steps, B]."""
        S, B, H, p = self.S, self.B, self.H, self.p
        if self._step is None:
            self._step = (lstm.Embedding(B, self.V, self.I, self.dtype), lstm.Lstm(1, B, self.I, H, self.dtype),
                          lstm.Attention(1, S, B, self.heads, self.heads, self.D, self.dtype),
                          lstm.LogProb(B, self.V, self.dtype, top=1))
        embed, cell, attend, logprob = self._step
        x = lstm.Embedding(S * B, self.V, self.I, self.dtype).forward(source, p["table"])
        states, _, _ = self.enc.forward(x, p["enc_W"], p["enc_b"], seq_length=length)
        keys = self.heads_of(states)
        token = torch.full((1, B), START, dtype=torch.int64, device=source.device)
        none = torch.full((B,), -1, dtype=torch.int64, device=source.device)
        h = c = None
        said = []
        for _ in range(steps):
            y, h, c = cell.forward(embed.forward(token, p["table"]), p["dec_W"], p["dec_b"], h, c)
            h, c = h.clone(), c.clone()  # the next call writes hT and cT again
            context, _ = attend.forward(self.heads_of(y), keys, keys, length)
            logits = torch.cat([y, context.view(1, B, H)], 2).view(B, 2 * H) @ p["out_W"].t()
            token = logprob.forward(logits, none)[3].view(1, B).clone()
            said.append(token)
        return torch.cat(said)


def make_batch(S, B, V, g, device="cuda"):
    """Ragged sources, their reversals as targets, and the decoder's inputs (START, then the targets)."""
    length = torch.randint(max(1, S // 2), S + 1, (B,), generator=g, device=device)
    t = torch.arange(S, device=device)[:, None]
    source = torch.randint(2, V, (S, B), generator=g, device=device).masked_fill(t >= length, PAD)
    back = source.gather(0, (length[None] - 1 - t).clamp(min=0))
    targets = back.masked_fill(t >= length, -1)
    start = torch.full((1, B), START, dtype=torch.int64, device=device)
    answer_in = torch.cat([start, targets[:-1].clamp(min=PAD)])
    return source, answer_in, targets, length.to(torch.int32)


class Adam:
    def __init__(self, params, lr=3e-3, betas=(0.9, 0.98), eps=1e-8):
        self.lr, self.betas, self.eps, self.t = lr, betas, eps, 0
        self.m, self.v, self.master = ({k: f(x) for k, x in params.items()} for f in (
            lambda x: torch.zeros_like(x, dtype=torch.float32), lambda x: torch.zeros_like(x, dtype=torch.float32),
            lambda x: x.float()))

    def step(self, params, grads):
        self.t += 1
        b1, b2 = self.betas
        lr = self.lr * math.sqrt(1 - b2**self.t) / (1 - b1**self.t)
        for k, x in params.items():
            g = grads[k].float()
            self.m[k].mul_(b1).add_(g, alpha=1 - b1)
            self.v[k].mul_(b2).addcmul_(g, g, value=1 - b2)
            self.master[k].addcdiv_(self.m[k], self.v[k].sqrt() + self.eps, value=-lr)
            x.copy_(self.master[k])


def train(steps=1000, S=16, B=64, V=32, dtype=lstm.F32, seed=0, log=None):
    """(model, mean log probability of the last step)."""
    model = Seq2Seq(S, B, V, dtype=dtype, seed=seed)
    opt = Adam(model.p)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    score = None
    for i in range(steps):
        score = model.forward(*make_batch(S, B, V, g))
        opt.step(model.p, model.backward())
        if log and (i % log == 0 or i == steps - 1):
            print(f"step {i}: loss {-float(score):.4f}", flush=True)
    model.enc.check(), model.dec.check()
    return model, float(score)


def accuracy(model, seed=99):
    """Share of the tokens of a new batch that the decoder writes right, step by step."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    source, _, targets, length = make_batch(model.S, model.B, model.V, g)
    said = model.answer(source, length, model.S)
    real = targets >= 0
    return float((said == targets)[real].float().mean())


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=1000)
    ap.add_argument("--batch", type=int, default=64)
    ap.add_argument("--length", type=int, default=16)
    ap.add_argument("--words", type=int, default=32)
    ap.add_argument("--dtype", choices=("f32", "bf16"), default="f32")
    args = ap.parse_args(argv)
    model, _ = train(args.steps, args.length, args.batch, args.words, lstm.F32 if args.dtype == "f32" else lstm.BF16,
                     log=100)
    print(f"tokens written right, one step at a time: {100 * accuracy(model):.1f} %")


if __name__ == "__main__":
    main()
