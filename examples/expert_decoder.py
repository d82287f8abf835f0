"""A decoder layer with experts, trained for a few steps and then run token by
token over a paged cache, on the library's moves of tokens:

  queries and keys turned by three axes of positions       rotary / its inverse
  new keys and values into the cache's pages                paged_append
  the router's choices sorted by expert                     expert_sort
  rows to their experts and back, weighted                  expert_dispatch, expert_combine
  and the gradients of both                                 expert_combine, expert_combine_backward

The products between them (projections, attention, the experts' two layers)
are plain torch.  Run it with

    python examples/expert_decoder.py

It prints the loss of each step and, at the end, how far the token-by-token
outputs are from those of the whole sequence at once.
"""

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bmmc_index_transforms_gb300 as bm  # noqa: E402


class Rotary(torch.autograd.Function):
    """Heads turned by their positions; the gradient is turned back."""

    @staticmethod
    def forward(ctx, x, positions, inv_freq, pair_axes):
        ctx.save_for_backward(positions, inv_freq, pair_axes)
        return bm.rotary(x, positions, inv_freq, pair_axes)

    @staticmethod
    def backward(ctx, grad):
        return bm.rotary(grad.contiguous(), *ctx.saved_tensors, inverse=True), None, None, None


class Dispatch(torch.autograd.Function):
    """Tokens' rows to the rows of their choices; the gradient adds them up."""

    @staticmethod
    def forward(ctx, x, slot):
        ctx.save_for_backward(slot)
        return bm.expert_dispatch(x, slot)

    @staticmethod
    def backward(ctx, grad):
        return bm.expert_combine(grad.contiguous(), *ctx.saved_tensors), None


class Combine(torch.autograd.Function):
    """The rows of a token's choices added up with the router's weights."""

    @staticmethod
    def forward(ctx, rows, slot, weights):
        ctx.save_for_backward(rows, slot, weights)
        return bm.expert_combine(rows, slot, weights)

    @staticmethod
    def backward(ctx, grad):
        grad_rows, grad_weights = bm.expert_combine_backward(grad.contiguous(), *ctx.saved_tensors)
        return grad_rows, None, grad_weights


class Layer(torch.nn.Module):
    def __init__(self, hidden=256, q_heads=8, kv_heads=2, head_dim=32, experts=8, choices=2, dtype=torch.float32):
        super().__init__()
        self.q_heads, self.kv_heads, self.head_dim, self.experts, self.choices = q_heads, kv_heads, head_dim, experts, choices
        new = lambda *shape: torch.nn.Parameter(torch.randn(*shape, device="cuda", dtype=dtype) / shape[-2] ** 0.5)  # noqa: E731
        self.qkv = new(hidden, (q_heads + 2 * kv_heads) * head_dim)
        self.out = new(q_heads * head_dim, hidden)
        self.router = new(hidden, experts)
        self.up, self.down = new(experts, hidden, 2 * hidden), new(experts, 2 * hidden, hidden)
        pairs = head_dim // 2
        self.register_buffer("inv_freq", 100.0 ** (-torch.arange(pairs, device="cuda") / pairs))
        self.register_buffer("pair_axes", (torch.arange(pairs, device="cuda") % 3).int())

    def split(self, x):
        """Queries, keys and values of tokens, as slices of one product."""
        heads = (x @ self.qkv).view(x.shape[0], -1, self.head_dim)
        return heads.split([self.q_heads, self.kv_heads, self.kv_heads], dim=1)

    def attend(self, q, k, v, seen):
        """q [tokens, q_heads, dim] over k, v [entries, kv_heads, dim]; seen
        [tokens, entries]: which entries a token sees."""
        k, v = (y.repeat_interleave(self.q_heads // self.kv_heads, dim=1) for y in (k, v))
        score = torch.einsum("thd,ehd->hte", q, k) / self.head_dim ** 0.5
        weight = torch.softmax(score.masked_fill(~seen, float("-inf")), dim=-1)
        return torch.einsum("hte,ehd->thd", weight, v).flatten(1) @ self.out

    def expert_layer(self, x):
        weights, ids = torch.softmax(x @ self.router, dim=1).topk(self.choices, dim=1)
        slot, _, offsets = bm.expert_sort(ids, self.experts)
        rows = Dispatch.apply(x, slot)
        sizes = (offsets[1:] - offsets[:-1]).tolist()
        done = [torch.relu(part @ self.up[e]) @ self.down[e] for e, part in enumerate(rows.split(sizes))]
        return Combine.apply(torch.cat(done), slot, weights.contiguous())

    def forward(self, x, positions):
        """A whole sequence at once, for training."""
        q, k, v = self.split(x)
        q, k = (Rotary.apply(y, positions, self.inv_freq, self.pair_axes) for y in (q, k))
        n = x.shape[0]
        seen = torch.ones(n, n, dtype=torch.bool, device="cuda").tril()
        x = x + self.attend(q, k, v, seen)
        return x + self.expert_layer(x)


class Cache:
    """Keys and values of some sequences in pages of 16 entries."""

    def __init__(self, layer, sequences, entries, page=16):
        each = -(-entries // page)
        shape = (sequences * each, page, layer.kv_heads, layer.head_dim)
        self.k, self.v = (torch.zeros(shape, device="cuda", dtype=layer.qkv.dtype) for _ in range(2))
        self.table = torch.randperm(sequences * each, device="cuda").int().view(sequences, each)  # any pages will do
        self.lengths = torch.zeros(sequences, dtype=torch.int32, device="cuda")

    def sequence(self, b, entries):
        """Keys and values of sequence b's first entries."""
        pages = self.table[b].long()
        return (m[pages].flatten(0, 1)[:entries] for m in (self.k, self.v))


@torch.no_grad()
def step(layer, cache, x, positions):
    """The next token x[b] of every sequence: appended, then attended."""
    q, k, v = layer.split(x)
    q = bm.paged_append(k, v, cache.k, cache.v, cache.table, cache.lengths, q=q, positions=positions,
                        inv_freq=layer.inv_freq, pair_axes=layer.pair_axes)
    cache.lengths += 1
    out = []
    for b, n in enumerate(cache.lengths.tolist()):
        keys, values = cache.sequence(b, n)
        out.append(layer.attend(q[b:b + 1], keys, values, torch.ones(1, n, dtype=torch.bool, device="cuda")))
    x = x + torch.cat(out)
    return x + layer.expert_layer(x)


def image_positions(n, width=7):
    """Positions on three axes: some text, then the rows and columns of an image."""
    i = torch.arange(n, device="cuda")
    j = (i - 8).clamp(min=0)
    return torch.where(i < 8, i, 8 + torch.stack([torch.zeros_like(j), j // width, j % width])).contiguous()


def train(layer, steps=10, tokens=96, seed=0):
    """A few steps towards a random target; the losses."""
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(tokens, layer.qkv.shape[0], generator=g, device="cuda")
    target = torch.randn(tokens, layer.qkv.shape[0], generator=g, device="cuda")
    optimizer = torch.optim.SGD(layer.parameters(), lr=0.05)
    losses = []
    for _ in range(steps):
        loss = (layer(x, image_positions(tokens)) - target).square().mean()
        optimizer.zero_grad()
        loss.backward()
        optimizer.step()
        losses.append(loss.item())
    return losses


@torch.no_grad()
def generate(layer, sequences=3, tokens=50, seed=1):
    """Sequences run token by token over the cache: the largest difference
    from running each at once, and the largest value."""
    g = torch.Generator("cuda").manual_seed(seed)
    x = torch.randn(sequences, tokens, layer.qkv.shape[0], generator=g, device="cuda")
    positions = image_positions(tokens)
    cache = Cache(layer, sequences, tokens)
    got = torch.stack([step(layer, cache, x[:, t].contiguous(), positions[:, t:t + 1].expand(3, sequences).contiguous())
                       for t in range(tokens)], dim=1)
    want = torch.stack([layer(x[b], positions) for b in range(sequences)])
    return float((got - want).abs().max()), float(want.abs().max())


def main():
    torch.manual_seed(0)
    layer = Layer()
    for i, loss in enumerate(train(layer)):
        print(f"step {i}: loss {loss:.5f}")
    off, size = generate(layer)
    print(f"token by token: off by at most {off:.2e} of values up to {size:.2f}")


if __name__ == "__main__":
    main()
