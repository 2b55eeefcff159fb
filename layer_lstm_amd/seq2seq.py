"""A small encoder-decoder on the library's operators.

    python -m layer_lstm_amd.seq2seq [--steps 1000] [--batch 64] [--length 16]
        [--memory] [--optimizer adam|adamw|adamw8] [--clip 1.0] [--repetition 1.0]

Learns to write a sequence backwards: tokens -> embedding -> bidirectional
LSTM encoder; the shifted answer -> embedding -> LSTM decoder -> cross
attention over the encoder's states -> one linear layer over [state, context]
-> log probabilities.  Everything but that layer's products and the
optimiser's elementwise update runs in liblstm.so, forward and backward; the
decoder then answers token by token from the same operators at one step.
Sequences are ragged: padded steps hold the encoder's state (seq_length), are
no keys (k_length) and no targets (-1).

--memory gives the decoder linear attention over its own steps (a matrix state
per head, its decay fixed, beside the LSTM's vector); --optimizer adamw takes
the library's step over all parameters in one launch (adamw8: states in 8 bits),
--clip holds the gradient to a norm; answers may be constrained by a mask of
allowed tokens and a penalty for those said before.
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
    head_dim the decoder's state (and both directions of the encoder's);
    `memory`: linear attention over the decoder's steps, its queries and keys
    the decoder's states, its values their contexts."""

    def __init__(self, S, B, V, I=64, heads=4, head_dim=32, dtype=lstm.F32, seed=0, device="cuda", memory=False):
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
            out_W=uniform(V, (3 if memory else 2) * H, k=1 / math.sqrt(2 * H)))
        # one embedding call for the sources and the answers: ids [2 S, B]
        self.embed = lstm.Embedding(2 * S * B, V, I, dtype, padding=PAD)
        self.enc = lstm.Lstm(S, B, I, H // 2, dtype, bidirectional=True)
        self.dec = lstm.Lstm(S, B, I, H, dtype)
        self.attend = lstm.Attention(S, S, B, heads, heads, head_dim, dtype)
        self.logprob = lstm.LogProb(S * B, V, dtype)
        self.memory = self.log_decay = None
        if memory:
            self.memory = lstm.LinearAttention(S, B, heads, heads, head_dim, head_dim, dtype, scale=1 / head_dim)
            # heads that remember 4, 8, 16 .. steps
            self.log_decay = -(0.5 ** torch.arange(2, 2 + heads, device=device, dtype=torch.float32))
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
        parts = [y, context.view(S, B, self.H)]
        if self.memory is not None:
            recalled, _ = self.memory.forward(self.heads_of(y), self.heads_of(y), context, self.log_decay)
            parts.append(recalled.view(S, B, self.H))
        self.features = torch.cat(parts, 2).view(S * B, -1)
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
        df = (dlogits @ p["out_W"]).view(S, B, -1)
        q, dcontext = self.heads_of(self.dec.y), self.heads_of(df[:, :, H : 2 * H].contiguous())
        dy = df[:, :, :H]
        if self.memory is not None:
            mq, mk, mv, _ = self.memory.backward(self.heads_of(df[:, :, 2 * H :].contiguous()), q, q, self.attend.o, self.log_decay)
            dy, dcontext = dy + (mq + mk).view(S, B, H), dcontext + mv
        dq, dk, dv = self.attend.backward(dcontext, q, self.keys, self.keys, self.length)
        zero = torch.zeros((B, H), dtype=df.dtype, device=df.device)
        dx_dec, dec_W, dec_b, _, _ = self.dec.backward(dy + dq.view(S, B, H), zero, zero, self.x_dec,
                                                       p["dec_W"])
        zero = zero.view(2, B, H // 2)
        # the states are keys and values both
        dx_enc, enc_W, enc_b, _, _ = self.enc.backward((dk + dv).view(S, B, H), zero, zero, self.x_enc, p["enc_W"],
                                                       seq_length=self.length)
        table = self.embed.backward(self.ids, torch.cat([dx_enc, dx_dec]))
        return dict(table=table, enc_W=enc_W, enc_b=enc_b, dec_W=dec_W, dec_b=dec_b,
                    out_W=dlogits.t().contiguous() @ self.features)

    def answer(self, source, length, steps, repetition=None, mask=None):
        """The likeliest token at every step, fed back: [steps, B].  repetition: a
        penalty (fp32 [B]) for tokens said before; mask: int32 words [B, ceil(V / 32)]
        of the allowed tokens' bits."""
        S, B, H, p = self.S, self.B, self.H, self.p
        if self._step is None:
            self._step = (lstm.Embedding(B, self.V, self.I, self.dtype), lstm.Lstm(1, B, self.I, H, self.dtype),
                          lstm.Attention(1, S, B, self.heads, self.heads, self.D, self.dtype),
                          lstm.LogProb(B, self.V, self.dtype, top=1), lstm.Penalty(B, self.V, self.dtype),
                          self.memory and lstm.LinearAttention(1, B, self.heads, self.heads, self.D, self.D, self.dtype,
                                                               scale=1 / self.D))
        embed, cell, attend, logprob, penalty, memory = self._step
        x = lstm.Embedding(S * B, self.V, self.I, self.dtype).forward(source, p["table"])
        states, _, _ = self.enc.forward(x, p["enc_W"], p["enc_b"], seq_length=length)
        keys = self.heads_of(states)
        token = torch.full((1, B), START, dtype=torch.int64, device=source.device)
        none = torch.full((B,), -1, dtype=torch.int64, device=source.device)
        h = c = None
        said = torch.full((steps, B), -1, dtype=torch.int64, device=source.device)
        state = memory and torch.zeros((B, self.heads, self.D, self.D), device=source.device)
        for t in range(steps):
            y, h, c = cell.forward(embed.forward(token, p["table"]), p["dec_W"], p["dec_b"], h, c)
            h, c = h.clone(), c.clone()  # the next call writes hT and cT again
            context, _ = attend.forward(self.heads_of(y), keys, keys, length)
            parts = [y, context.view(1, B, H)]
            if memory:
                parts.append(memory.step(self.heads_of(y), self.heads_of(y), context, self.log_decay, state).view(1, B, H))
            logits = torch.cat(parts, 2).view(B, -1) @ p["out_W"].t()
            if repetition is not None or mask is not None:
                penalty.forward(logits, said[:t].t(), repetition=repetition, mask=mask, out=logits)
            token = logprob.forward(logits, none)[3].view(1, B).clone()
            said[t] = token[0]
        return said


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


class AdamW:
    """The library's step over all parameters, with the same rate."""

    def __init__(self, params, lr=3e-3, betas=(0.9, 0.98), bits=32, clip=None):
        self.names = list(params)
        self.opt = lstm.AdamW([params[k] for k in self.names], lr, betas, weight_decay=0.01, bits=bits, clip=clip)

    def step(self, params, grads):
        self.opt.step([grads[k] for k in self.names])


def make_optimizer(kind, params, clip=None):
    if kind == "adam":
        if clip is not None:
            raise ValueError("clip: with adamw")
        return Adam(params)
    return AdamW(params, bits=8 if kind == "adamw8" else 32, clip=clip)


def train(steps=1000, S=16, B=64, V=32, dtype=lstm.F32, seed=0, log=None, memory=False, optimizer="adam", clip=None):
    """(model, mean log probability of the last step)."""
    model = Seq2Seq(S, B, V, dtype=dtype, seed=seed, memory=memory)
    opt = make_optimizer(optimizer, model.p, clip)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    score = None
    for i in range(steps):
        score = model.forward(*make_batch(S, B, V, g))
        opt.step(model.p, model.backward())
        if log and (i % log == 0 or i == steps - 1):
            print(f"step {i}: loss {-float(score):.4f}", flush=True)
    model.enc.check(), model.dec.check()
    return model, float(score)


def allowed_words(model):
    """The mask that leaves the words: no padding, no start."""
    bits = torch.zeros((model.V + 31) // 32 * 32, dtype=torch.int64, device="cuda")
    bits[2 : model.V] = 1
    words = (bits.view(-1, 32) << torch.arange(32, device="cuda")).sum(1).to(torch.int32)
    return words.expand(model.B, -1).contiguous()


def accuracy(model, seed=99, repetition=1.0):
    """Share of the tokens of a new batch that the decoder writes right, step by step."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    source, _, targets, length = make_batch(model.S, model.B, model.V, g)
    how = {}
    if repetition != 1.0:
        how = dict(repetition=torch.full((model.B,), repetition, device="cuda"), mask=allowed_words(model))
    said = model.answer(source, length, model.S, **how)
    real = targets >= 0
    return float((said == targets)[real].float().mean())


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=1000)
    ap.add_argument("--batch", type=int, default=64)
    ap.add_argument("--length", type=int, default=16)
    ap.add_argument("--words", type=int, default=32)
    ap.add_argument("--dtype", choices=("f32", "bf16"), default="f32")
    ap.add_argument("--memory", action="store_true", help="linear attention over the decoder's steps")
    ap.add_argument("--optimizer", choices=("adam", "adamw", "adamw8"), default="adam")
    ap.add_argument("--clip", type=float, help="the norm that gradients are held to (with adamw)")
    ap.add_argument("--repetition", type=float, default=1.0, help="the answers' penalty for words said before")
    args = ap.parse_args(argv)
    model, _ = train(args.steps, args.length, args.batch, args.words, lstm.F32 if args.dtype == "f32" else lstm.BF16,
                     log=100, memory=args.memory, optimizer=args.optimizer, clip=args.clip)
    print(f"tokens written right, one step at a time: {100 * accuracy(model, repetition=args.repetition):.1f} %")


if __name__ == "__main__":
    main()
