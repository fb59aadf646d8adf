"""A small decoder trained with the two transformer-layer operators, then run a
token at a time from its cache.

    python examples/transformer_layer.py [steps]

Each layer is attention with a learned relative-position bias and dropout on
its probabilities, then output bias + dropout + residual + layer norm, then a
feed-forward sublayer that ends in the same operator.  No mask is stored: the
backward pass draws it again from the layer's seed of this step.

The task is synthetic: a token is the one five places back, or one time in
eight a random one, which a layer has to find by relative position.
"""
import math
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dropout_lowbias32_hash32_gb300 as rng  # noqa: E402


class Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, table, options):
        o = torch.empty_like(q)
        lse = torch.empty(q.shape[0], q.shape[2], q.shape[1], device=q.device)
        rng.rng_attention_fwd(q, k, v, o, lse=lse, bias_table=table, **options)
        ctx.save_for_backward(q, k, v, table, o, lse)
        ctx.options = options
        return o

    @staticmethod
    def backward(ctx, do):
        q, k, v, table, o, lse = ctx.saved_tensors
        dq, dk, dv, dtable = (torch.empty_like(t) for t in (q, k, v, table))
        rng.rng_attention_bwd(do.contiguous(), q, k, v, o, lse, dq, dk, dv, bias_table=table, dbias_table=dtable,
                              **ctx.options)
        return dq, dk, dv, dtable, None


class DropoutLayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, bias, residual, gamma, beta, p, seed):
        y, h = torch.empty_like(x), torch.empty_like(x)
        mean, rstd = (torch.empty(x.shape[:-1], device=x.device) for _ in range(2))
        rng.rng_dropout_layer_norm_fwd(x, gamma, beta, y, mean, rstd, bias=bias, residual=residual, h=h, p=p, seed=seed)
        ctx.save_for_backward(h, mean, rstd, gamma)
        ctx.mask = dict(p=p, seed=seed)
        return y

    @staticmethod
    def backward(ctx, dy):
        h, mean, rstd, gamma = ctx.saved_tensors
        dx, dresidual = torch.empty_like(h), torch.empty_like(h)
        dgamma, dbeta, dbias = (torch.empty_like(gamma) for _ in range(3))
        rng.rng_dropout_layer_norm_bwd(dy.contiguous(), h, gamma, mean, rstd, dx, dgamma, dbeta, dresidual=dresidual,
                                       dbias=dbias, **ctx.mask)
        return dx, dbias, dresidual, dgamma, dbeta, None, None


class Layer(torch.nn.Module):
    def __init__(self, width, heads, heads_kv, buckets, max_distance, p):
        super().__init__()
        self.heads, self.heads_kv, self.dim, self.p = heads, heads_kv, width // heads, p
        self.place = dict(causal=True, max_distance=max_distance, bidirectional=False)
        new = torch.nn.Linear
        self.qkv = new(width, (heads + 2 * heads_kv) * self.dim, bias=False)
        self.out, self.up, self.down = new(width, width, bias=False), new(width, 4 * width), new(4 * width, width, bias=False)
        self.table = torch.nn.Parameter(torch.zeros(buckets, heads))
        for name in ("attention", "feed"):
            self.register_parameter(name + "_bias", torch.nn.Parameter(torch.zeros(width)))
            self.register_parameter(name + "_gamma", torch.nn.Parameter(torch.ones(width)))
            self.register_parameter(name + "_beta", torch.nn.Parameter(torch.zeros(width)))

    def heads_of(self, x):
        qkv = self.qkv(x).unflatten(-1, (-1, self.dim))
        return qkv.split((self.heads, self.heads_kv, self.heads_kv), 2)

    def end(self, name, x, residual, p, seed):
        return DropoutLayerNorm.apply(x, getattr(self, name + "_bias"), residual, getattr(self, name + "_gamma"),
                                      getattr(self, name + "_beta"), p, seed)

    def forward(self, x, seed=0):
        """seed: this step's for the layer; its three masks take counters of their own seeds."""
        p = self.p if self.training else 0.0
        q, k, v = self.heads_of(x)
        o = Attention.apply(q, k, v, self.table, dict(self.place, p=p, seed=3 * seed))
        x = self.end("attention", self.out(o.flatten(2)), x, p, 3 * seed + 1)
        return self.end("feed", self.down(F.gelu(self.up(x))), x, p, 3 * seed + 2)

    @torch.no_grad()
    def step(self, x, cache, lengths):
        """One new token an entry, x [batch, 1, width]; lengths counts it already."""
        q, k, v = self.heads_of(x)
        batch = torch.arange(len(lengths), device=x.device)
        cache[0][batch, lengths.long() - 1], cache[1][batch, lengths.long() - 1] = k[:, 0], v[:, 0]
        o = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        rng.rng_attention_fwd(q, cache[0], cache[1], o, key_lengths=lengths, queries_last=True, bias_table=self.table, **self.place)
        x = self.end("attention", self.out(o.flatten(2)), x, 0.0, 0)
        return self.end("feed", self.down(F.gelu(self.up(x))), x, 0.0, 0)


class Decoder(torch.nn.Module):
    def __init__(self, tokens=64, width=256, heads=4, heads_kv=2, layers=2, buckets=32, max_distance=128, p=0.1):
        super().__init__()
        self.embed = torch.nn.Embedding(tokens, width)
        self.layers = torch.nn.ModuleList(Layer(width, heads, heads_kv, buckets, max_distance, p) for _ in range(layers))
        self.head = torch.nn.Linear(width, tokens)

    def forward(self, tokens, step=0):
        x = self.embed(tokens)
        for n, layer in enumerate(self.layers):
            x = layer(x, step * len(self.layers) + n)
        return self.head(x)

    def caches(self, batch, length, like):
        return [[torch.zeros(batch, length, layer.heads_kv, layer.dim, dtype=like.dtype, device=like.device) for _ in range(2)]
                for layer in self.layers]

    @torch.no_grad()
    def step(self, tokens, caches, lengths):
        x = self.embed(tokens)[:, None]
        for layer, cache in zip(self.layers, caches):
            x = layer.step(x, cache, lengths)
        return self.head(x)[:, 0]


def sequences(batch, length, tokens, generator):
    s = torch.randint(tokens, (batch, length), generator=generator, device="cuda")
    new = torch.rand(batch, length, generator=generator, device="cuda") < 1 / 8
    for i in range(5, length):
        s[:, i] = torch.where(new[:, i], s[:, i], s[:, i - 5])
    return s


def train(model, steps, batch=32, length=96, tokens=64, lr=2e-3):
    """Losses of the steps; the weights train in f32 copies, the layers compute in bf16."""
    g = torch.Generator(device="cuda").manual_seed(1)
    masters = [p.detach().float().clone().requires_grad_() for p in model.parameters()]
    optimizer = torch.optim.Adam(masters, lr=lr)
    losses = []
    for step in range(steps):
        s = sequences(batch, length, tokens, g)
        loss = F.cross_entropy(model(s[:, :-1], step)[:, 5:].float().flatten(0, 1), s[:, 6:].flatten())
        loss.backward()
        for master, p in zip(masters, model.parameters()):
            master.grad, p.grad = p.grad.float(), None
        optimizer.step()
        with torch.no_grad():
            for master, p in zip(masters, model.parameters()):
                p.copy_(master)
        losses.append(loss.detach())
    return torch.stack(losses).tolist()


@torch.no_grad()
def cached_against_whole(model, batch=4, length=60, tokens=64):
    """Largest difference of the logits, a token at a time from the cache against whole sequences."""
    model.eval()
    s = sequences(batch, length, tokens, torch.Generator(device="cuda").manual_seed(2))
    whole = model(s).float()
    caches, worst = model.caches(batch, length, model.head.weight), 0.0
    for i in range(length):
        lengths = torch.full((batch,), i + 1, dtype=torch.int32, device="cuda")
        logits = model.step(s[:, i], caches, lengths).float()
        worst = max(worst, float((logits - whole[:, i]).abs().max()))
    return worst, float(whole.abs().max())


def main():
    steps = int(sys.argv[1]) if len(sys.argv) > 1 else 300
    torch.manual_seed(0)
    model = Decoder().cuda().bfloat16()
    losses = train(model, steps)
    print(f"loss {losses[0]:.3f} -> {sum(losses[-10:]) / len(losses[-10:]):.3f} in {steps} steps (uniform guess {math.log(64):.3f})")
    worst, most = cached_against_whole(model)
    print(f"a token at a time against whole sequences: logits differ by {worst:.3f} at most, of {most:.1f}")


if __name__ == "__main__":
    main()
