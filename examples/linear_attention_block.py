"""A block of a language model around linear attention with one decay per head, from the package's
operators: trained a few steps on a toy task, then run as a server would, a chunked prefill followed
by one-token steps over a pool of states.

    residual norm -> one projection to q, k, v and gate -> norm of q and k per head, turned by position
                  -> linear attention, every head at its own constant rate
                  -> gated norm -> output projection (-> the next block's residual norm)

    python examples/linear_attention_block.py
"""
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

import chunked_linear_attention_kda_gb300 as kda  # noqa: E402
from examples.gated_delta_block import GatedNorm, ResidualNorm  # noqa: E402


class QueryKeyNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, positions, freqs):
        ctx.save_for_backward(q, k, q_weight, k_weight, positions, freqs)
        return kda.qk_norm_rope_fwd(q, k, q_weight, k_weight, positions, freqs)

    @staticmethod
    def backward(ctx, dq, dk):
        grads = kda.qk_norm_rope_bwd(dq.contiguous(), dk.contiguous(), *ctx.saved_tensors)
        return (*grads, None, None)


class LinearAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, cu):
        ctx.save_for_backward(q, k, v, g, cu)
        return kda.dla_chunk_fwd(q, k, v, g, None, cu, output_final_state=False)[0]

    @staticmethod
    def backward(ctx, dout):
        q, k, v, g, cu = ctx.saved_tensors
        grads = kda.dla_chunk_bwd(q, k, v, g, None, cu, dout.contiguous(), want_dg=ctx.needs_input_grad[3],
                                  want_dh0=False)
        return (*grads[:4], None)


class Block(torch.nn.Module):
    def __init__(self, d_model, heads, d, rotary):
        super().__init__()
        self.heads, self.d = heads, d
        self.proj = torch.nn.Linear(d_model, 4 * heads * d, bias=False, dtype=torch.bfloat16)
        self.out = torch.nn.Linear(heads * d, d_model, bias=False, dtype=torch.bfloat16)
        self.norm = torch.nn.Parameter(torch.ones(d_model))
        self.scale = torch.nn.Parameter(torch.full((d_model,), 0.5))
        self.q_norm = torch.nn.Parameter(torch.ones(d))
        self.k_norm = torch.nn.Parameter(torch.ones(d))
        self.out_norm = torch.nn.Parameter(torch.ones(d))
        # the logarithms of the rates: memories from one token to hundreds
        self.rate = torch.nn.Parameter(torch.linspace(0, -5.5, heads))
        self.register_buffer("freqs", kda.rotary_frequencies(rotary, device="cpu"))

    def decays(self):
        return -self.rate.exp()

    def project(self, y):
        return (x.unflatten(-1, (self.heads, self.d)) for x in self.proj(y).chunk(4, -1))

    def forward(self, x, residual, cu, positions):
        """``x`` the previous block's output, ``residual`` the stream: this block's output and the
        stream with x in it, for packed sequences [N, d_model]."""
        y, residual = ResidualNorm.apply(x, residual, self.norm, self.scale)
        q, k, v, gate = self.project(y)  # slices of the projection, and stay such
        q, k = QueryKeyNorm.apply(q, k, self.q_norm, self.k_norm, positions, self.freqs)
        o = LinearAttention.apply(q, k, v, self.decays(), cu)
        return self.out(GatedNorm.apply(o, gate, self.out_norm).flatten(1)), residual

    @torch.no_grad()
    def prefill(self, x, residual, cu, positions, pool, slots):
        y, residual = kda.residual_norm_fwd(x, self.norm, residual, self.scale)
        q, k, v, gate = self.project(y)
        q, k = kda.qk_norm_rope_fwd(q, k, self.q_norm, self.k_norm, positions, self.freqs)
        o, final = kda.dla_chunk_fwd(q, k, v, self.decays(), None, cu)
        pool[slots.long()] = final
        return self.out(kda.gated_norm_fwd(o, gate, self.out_norm, activation="silu").flatten(1)), residual

    @torch.no_grad()
    def step(self, x, residual, positions, pool, slots):
        y, residual = kda.residual_norm_fwd(x, self.norm, residual, self.scale)
        q, k, v, gate = self.project(y)
        q, k = kda.qk_norm_rope_fwd(q, k, self.q_norm, self.k_norm, positions, self.freqs)
        o = kda.dla_step(q, k, v, self.decays(), pool, slots)
        return self.out(kda.gated_norm_fwd(o, gate, self.out_norm, activation="silu").flatten(1)), residual


class Model(torch.nn.Module):
    def __init__(self, vocab=64, d_model=256, blocks=2, heads=4, d=64, rotary=32):
        super().__init__()
        self.embed = torch.nn.Embedding(vocab, d_model, dtype=torch.bfloat16)
        self.blocks = torch.nn.ModuleList(Block(d_model, heads, d, rotary) for _ in range(blocks))
        self.norm = torch.nn.Parameter(torch.ones(d_model))
        self.scale = torch.nn.Parameter(torch.ones(d_model))

    def run(self, tokens, each):
        x = self.embed(tokens)
        residual = torch.zeros_like(x)
        for i, b in enumerate(self.blocks):
            x, residual = each(i, b, x, residual)
        y, _ = ResidualNorm.apply(x, residual, self.norm, self.scale)
        return y @ self.embed.weight.T

    def forward(self, tokens, cu):
        positions = token_positions(cu, tokens.shape[0])
        return self.run(tokens, lambda i, b, x, r: b(x, r, cu, positions))

    def new_pools(self, slots):
        return [torch.zeros((slots, b.heads, b.d, b.d), device=self.norm.device) for b in self.blocks]


def token_positions(cu, n):
    """Each token's place in its sequence."""
    t = torch.arange(n, dtype=torch.int32, device=cu.device)
    return t - cu[torch.searchsorted(cu[1:], t, right=True)]


def train(model, steps=30, sequences=8, length=96, vocab=64, seed=0):
    """Repeat a pattern seen once: the second half of every sequence copies the first."""
    gen = torch.Generator().manual_seed(seed)
    opt = torch.optim.Adam(model.parameters(), lr=2e-3)
    cu = torch.arange(sequences + 1, dtype=torch.int32, device="cuda") * length
    losses = []
    for _ in range(steps):
        half = torch.randint(0, vocab, (sequences, length // 2), generator=gen)
        tokens = torch.cat([half, half], 1).flatten().to("cuda")
        logits = model(tokens, cu).float().view(sequences, length, -1)[:, length // 2:-1]
        target = tokens.view(sequences, length)[:, length // 2 + 1:]
        loss = F.cross_entropy(logits.flatten(0, 1), target.flatten())
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.item())
    return losses


@torch.no_grad()
def serve(model, prompts, tokens_to_go):
    """Greedy continuation of ragged prompts. Returns the tokens and the logits that chose them."""
    n, slots_total = len(prompts), len(prompts) + 2
    pools = model.new_pools(slots_total)
    slots = torch.arange(n, 0, -1, dtype=torch.int32, device="cuda")
    lens = [len(p) for p in prompts]
    cu = torch.tensor([sum(lens[:i]) for i in range(n + 1)], dtype=torch.int32, device="cuda")
    packed, at = torch.cat(prompts).to("cuda"), token_positions(cu, sum(lens))
    logits = model.run(packed, lambda i, b, x, r: b.prefill(x, r, cu, at, pools[i], slots))[cu[1:].long() - 1]
    at = torch.tensor(lens, dtype=torch.int32, device="cuda")
    out, seen = [], []
    for _ in range(tokens_to_go):
        nxt = logits.argmax(-1)
        out.append(nxt)
        seen.append(logits)
        logits = model.run(nxt, lambda i, b, x, r: b.step(x, r, at, pools[i], slots))
        at += 1
    return torch.stack(out, 1), torch.stack(seen, 1)


if __name__ == "__main__":
    torch.manual_seed(0)
    net = Model().cuda()
    curve = train(net)
    print("loss %.3f -> %.3f over %d steps" % (curve[0], curve[-1], len(curve)))
    gen = torch.Generator().manual_seed(1)
    asked = [torch.randint(0, 64, (n,), generator=gen) for n in (5, 70, 131)]
    answer, _ = serve(net, asked, 8)
    for p, a in zip(asked, answer.tolist()):
        print(len(p), "tokens ->", a)
