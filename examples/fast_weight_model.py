"""A small model around the fast-weight layer, from token ids to hidden states:

  X0 = embed(ids)                                  the layer's token embeddings
  R  = X0 + W_o . delta_rule(q, k, v, g, beta)     of layer_norm(X0), projected
  H  = layer_norm(R)                               the layer's hidden states
  Y  = R + forward(H, X0, ...)                     the In-Place TTT layer

Two fast weights work side by side: the delta rule's, written once a token, and
the layer's W_down, written once a chunk.  `prefill` runs whole prompts,
`decode` one token of each running sequence on pools of both states, and
`train` takes gradient steps on the mixer (lookup, norms, projections, delta
rule) with automatic differentiation around the operators' gradients: the calls
themselves are not recorded, Embed, LayerNorm and DeltaRule below record them, once
(a second derivative is an error).

    python examples/fast_weight_model.py
"""
import os
import sys
import time

import torch
import torch.nn.functional as F
from torch.autograd.function import once_differentiable

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from chunk_wise_weight_gb300 import build, ittt  # noqa: E402


class Embed(torch.autograd.Function):
    @staticmethod
    def forward(ctx, ids, table, scale):
        ctx.save_for_backward(ids)
        ctx.rows, ctx.scale, ctx.dtype = table.shape[0], scale, table.dtype
        return ittt.embed(ids, table, scale)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        (ids,) = ctx.saved_tensors
        return None, ittt.embed_grad(ids, dy.contiguous(), ctx.rows, ctx.scale, grad_dtype=ctx.dtype), None


class LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias):
        mean, rstd = (torch.empty(x.shape[:-1], device=x.device) for _ in range(2))
        y = ittt.layer_norm(x, weight, bias, mean=mean, rstd=rstd)
        ctx.save_for_backward(x, weight, mean, rstd)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        return ittt.layer_norm_grad(dy.contiguous(), *ctx.saved_tensors)


class DeltaRule(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, beta):
        ctx.save_for_backward(q, k, v, g, beta)
        return ittt.delta_rule(q, k, v, g, beta)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        return ittt.delta_rule_grad(*ctx.saved_tensors, dy.contiguous())


class Model:
    def __init__(self, vocab=1000, d=256, f=512, key_heads=2, heads=4, dk=64, dv=64, eta=0.01, chunk=64, seed=0):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)

        def normal(*shape, std):
            return (torch.randn(*shape, generator=gen, device="cuda") * std).bfloat16()

        self.sizes = [key_heads * dk, key_heads * dk, heads * dv, heads, heads]
        self.key_heads, self.heads, self.dk, self.dv = key_heads, heads, dk, dv
        self.d, self.f, self.eta, self.chunk, self.scale = d, f, eta, chunk, d ** 0.5
        self.table = normal(vocab, d, std=d ** -0.5)
        self.norms = [torch.ones(d, device="cuda") if i % 2 == 0 else torch.zeros(d, device="cuda") for i in range(4)]
        self.w_in = normal(sum(self.sizes), d, std=d ** -0.5)
        self.w_out = normal(d, heads * dv, std=(heads * dv) ** -0.5)
        self.layer = [normal(f, d, std=d ** -0.5), normal(f, d, std=d ** -0.5), normal(d, f, std=f ** -0.5),
                      normal(d, d, std=d ** -0.5), torch.full((d, 3), 1 / 3, device="cuda")]

    def project(self, x):
        """q, k (of length one), v and the two gates of rows x [..., d]."""
        q, k, v, g, beta = F.linear(x, self.w_in).split(self.sizes, -1)
        q, k = (F.normalize(y.unflatten(-1, (self.key_heads, self.dk)).float(), dim=-1).bfloat16() for y in (q, k))
        return q, k, v.unflatten(-1, (self.heads, self.dv)), -F.softplus(g.float()), beta.float().sigmoid()

    def prefill(self, ids, states, fast):
        """Y [B,T,d] of whole prompts; `states` [B,heads,dv,dk] and `fast`
        [B,d,f] (fp32) receive what the sequences have written."""
        x0 = ittt.embed(ids.contiguous(), self.table, self.scale)
        x = self.project(ittt.layer_norm(x0, *self.norms[:2]))
        o = ittt.delta_rule(*x, state_in=states, state_out=states)
        r = x0 + F.linear(o.flatten(-2), self.w_out)
        h = ittt.layer_norm(r, *self.norms[2:])
        return r + ittt.forward(h, x0, *self.layer, self.eta, self.chunk, state_in=fast, state_out=fast)

    def decode(self, ids, states, slots):
        """H [B,d] of one token a sequence; sequence i keeps its state in row
        slots[i] of the pool (outside the pool: an empty row of the batch)."""
        x0 = ittt.embed(ids.contiguous(), self.table, self.scale)
        x = self.project(ittt.layer_norm(x0, *self.norms[:2]))
        o = ittt.delta_step(*x, states, slots=slots)
        return ittt.layer_norm(x0 + F.linear(o.flatten(-2), self.w_out), *self.norms[2:])

    def mixer(self, ids):
        """H [B,T,d], differentiable."""
        x0 = Embed.apply(ids.contiguous(), self.table, self.scale)
        o = DeltaRule.apply(*self.project(LayerNorm.apply(x0, *self.norms[:2])))
        return LayerNorm.apply(x0 + F.linear(o.flatten(-2), self.w_out), *self.norms[2:])

    def train(self, ids, steps, rate=0.05):
        """Gradient steps on the next token's cross entropy over the rows of
        the table; the losses."""
        weights = [self.table, self.w_in, self.w_out, *self.norms]
        losses = []
        for w in weights:
            w.requires_grad_()
        for _ in range(steps):
            logits = F.linear(self.mixer(ids[:, :-1]), self.table).float()
            loss = F.cross_entropy(logits.flatten(0, 1), ids[:, 1:].flatten().long())
            grads = torch.autograd.grad(loss, weights)
            with torch.no_grad():
                for w, g in zip(weights, grads):
                    w -= rate * g / g.norm().clamp(min=1.0)
            losses.append(float(loss.detach()))
        for w in weights:
            w.requires_grad_(False)
        return losses


def main():
    build.build()
    m = Model(vocab=32000, d=1024, f=2816, key_heads=4, heads=8, dk=128, dv=128, chunk=512)
    B, T, steps = 4, 2048, 64
    ids = torch.randint(0, 32000, (B, T), device="cuda", dtype=torch.int32)
    states = torch.zeros(B, m.heads, m.dv, m.dk, device="cuda")
    fast = m.layer[2].float().expand(B, m.d, m.f).contiguous()

    def timed(what, rows, f):
        f()
        torch.cuda.synchronize()
        t = time.perf_counter()
        out = f()
        torch.cuda.synchronize()
        t = time.perf_counter() - t
        print(f"{what}: {t * 1e3:.3f} ms, {rows / t:,.0f} tokens/s")
        return out

    timed(f"prefill {B} x {T}", B * T, lambda: m.prefill(ids, states, fast))
    slots = torch.arange(B, device="cuda", dtype=torch.int32)
    side, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        m.decode(ids[:, 0], states, slots)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            m.decode(ids[:, 0], states, slots)
    timed(f"decode {B} sequences, a graph", B * steps, lambda: [graph.replay() for _ in range(steps)])
    losses = timed(f"4 gradient steps {B} x 512", 4 * B * 512, lambda: m.train(ids[:, :513], 4))
    print("losses", " ".join(f"{x:.4f}" for x in losses))


if __name__ == "__main__":
    main()
