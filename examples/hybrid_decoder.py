"""A small decoder of alternating layers, window attention with sinks and linear
attention with decay: reads a prompt, continues it token by token over a paged
cache and the layers' states, and trains for a few steps.

    python examples/hybrid_decoder.py [--layers 4] [--prompt 300] [--new 16] [--steps 5]

Weights and tokens are random. The continuation is checked against the same
tokens read as one prompt.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import memory_efficient_im2win_amd as m  # noqa: E402

VOCAB, HEADS, KV_HEADS, D, WINDOW, SINKS, PAGE = 512, 8, 2, 64, 96, 4, 16
WIDTH = HEADS * D


class WindowAttention(torch.autograd.Function):
    """Gradients are explicit calls of the package; this is all it takes to have
    autograd make them."""

    @staticmethod
    def forward(ctx, q, k, v):
        out, lse = m.window_attention(q, k, v, window=WINDOW, sinks=SINKS, return_lse=True)
        ctx.save_for_backward(q, k, v, out, lse)
        return out

    @staticmethod
    def backward(ctx, dout):
        return m.window_attention_backward(dout.contiguous(), *ctx.saved_tensors, window=WINDOW, sinks=SINKS)


class LinearAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, log_decay):
        ctx.save_for_backward(q, k, v, log_decay)
        return m.linear_attention(q, k, v, log_decay)[0]

    @staticmethod
    def backward(ctx, dout):
        return (*m.linear_attention_backward(dout.contiguous(), *ctx.saved_tensors)[:3], None)


class Decoder(torch.nn.Module):
    def __init__(self, layers):
        super().__init__()
        self.window = [i % 2 == 0 for i in range(layers)]
        kv = [KV_HEADS if w else HEADS for w in self.window]
        self.kv = kv
        self.embed = torch.nn.Embedding(VOCAB, WIDTH)
        torch.nn.init.normal_(self.embed.weight, std=WIDTH ** -0.5)
        self.qkv = torch.nn.ModuleList(torch.nn.Linear(WIDTH, (HEADS + 2 * n) * D, bias=False) for n in kv)
        self.out = torch.nn.ModuleList(torch.nn.Linear(WIDTH, WIDTH, bias=False) for _ in kv)
        self.register_buffer("log_decay", -torch.exp2(-8.0 * (torch.arange(HEADS) + 1) / HEADS), persistent=False)

    def heads(self, i, x):
        x = self.qkv[i](torch.nn.functional.layer_norm(x, (WIDTH,)))
        return (y.unflatten(-1, (-1, D)) for y in x.split([HEADS * D, self.kv[i] * D, self.kv[i] * D], -1))

    def logits(self, x):
        return torch.nn.functional.layer_norm(x, (WIDTH,)) @ self.embed.weight.T

    def forward(self, tokens):
        """Logits of whole sequences (B, L), for training."""
        x = self.embed(tokens)
        for i, window in enumerate(self.window):
            q, k, v = self.heads(i, x)
            y = WindowAttention.apply(q, k, v) if window else LinearAttention.apply(q, k, v, self.log_decay.float())
            x = x + self.out[i](y.flatten(2))
        return self.logits(x)

    def cache(self, B, tokens):
        """Pages for window layers, states for linear ones."""
        per = -(-tokens // PAGE)
        dev, dtype = self.embed.weight.device, self.embed.weight.dtype
        self.table = torch.randperm(B * per, device=dev).to(torch.int32).view(B, per)
        self.filled = torch.zeros(B, dtype=torch.int32, device=dev)
        pool = lambda: torch.empty(2, B * per, PAGE, KV_HEADS, D, dtype=dtype, device=dev)  # noqa: E731
        state = lambda: torch.zeros(B, HEADS, D, D, device=dev)  # noqa: E731
        return [pool() if w else state() for w in self.window]

    def read(self, tokens, cache, start):
        """Logits of (B, n) tokens that stand at start, start + 1, ...; the cache moves on by n."""
        B, n = tokens.shape
        x = self.embed(tokens)
        at = torch.arange(start, start + n, device=tokens.device)
        page, slot = self.table[:, at // PAGE].long(), (at % PAGE).expand(B, n)
        self.filled.fill_(start + n)
        for i, window in enumerate(self.window):
            q, k, v = self.heads(i, x)
            if window:
                cache[i][0][page, slot], cache[i][1][page, slot] = k, v
                y = m.window_attention(q, *cache[i], window=WINDOW, sinks=SINKS, kv_lens=self.filled,
                                       page_table=self.table)
            elif n == 1:
                y = m.linear_attention_step(q[:, 0], k[:, 0], v[:, 0], self.log_decay.float(), cache[i]).unsqueeze(1)
            else:
                y, _ = m.linear_attention(q, k, v, self.log_decay.float(), state=cache[i], state_out=cache[i])
            x = x + self.out[i](y.flatten(2))
        return self.logits(x)


def generate(model, prompt, new):
    """The prompt continued greedily by `new` tokens, and the logits of every step."""
    cache = model.cache(prompt.shape[0], prompt.shape[1] + new)
    tokens, logits = prompt, [model.read(prompt, cache, 0)[:, -1]]
    for i in range(new):
        tokens = torch.cat([tokens, logits[-1].argmax(-1, keepdim=True)], 1)
        if i + 1 < new:
            logits.append(model.read(tokens[:, -1:], cache, tokens.shape[1] - 1)[:, 0])
    return tokens, torch.stack(logits, 1)


def train(model, tokens, steps):
    """Losses of `steps` steps on one batch."""
    optimizer = torch.optim.SGD(model.parameters(), lr=0.05)
    losses = []
    for _ in range(steps):
        optimizer.zero_grad()
        logits = model(tokens[:, :-1]).float()
        loss = torch.nn.functional.cross_entropy(logits.flatten(0, 1), tokens[:, 1:].flatten())
        loss.backward()
        optimizer.step()
        losses.append(loss.item())
    return losses


def main(argv=None):
    args = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    for name, value in (("layers", 4), ("batch", 2), ("prompt", 300), ("new", 16), ("steps", 5)):
        args.add_argument("--" + name, type=int, default=value)
    a = args.parse_args(argv)
    torch.manual_seed(0)
    model = Decoder(a.layers).to("cuda", torch.bfloat16)
    prompt = torch.randint(VOCAB, (a.batch, a.prompt), device="cuda")
    with torch.no_grad():
        tokens, stepped = generate(model, prompt, a.new)
        whole = model(tokens[:, :-1])[:, a.prompt - 1:]
    off = ((stepped - whole).float().norm() / whole.float().norm()).item()
    print(f"{a.new} tokens after a prompt of {a.prompt}: logits off the whole sequence's by {off:.2g} (relative)")
    losses = train(model, tokens, a.steps)
    print("losses:", " ".join(f"{x:.4f}" for x in losses))
    return off, losses


if __name__ == "__main__":
    main()
