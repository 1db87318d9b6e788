"""A block of a language model around the gated delta rule with one decay per head, from the
package's operators: trained a few steps on a toy task, then run as a server would, a chunked
prefill followed by one-token steps over a pool of states.

    residual norm -> one projection to q, k, v, decay, beta and gate -> gated delta rule
                  -> gated norm -> output projection (-> the next block's residual norm)

    python examples/gated_delta_block.py
"""
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.join(os.path.dirname(os.path.abspath(__file__)), ".."))

import chunked_linear_attention_kda_gb300 as kda  # noqa: E402


class ResidualNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, weight, scale):
        y, r = kda.residual_norm_fwd(x, weight, residual, scale)
        ctx.save_for_backward(r, weight, x, scale)
        return y, r

    @staticmethod
    def backward(ctx, dy, dr):
        r, weight, x, scale = ctx.saved_tensors
        dx, dres, dw, dscale = kda.residual_norm_bwd(dy.contiguous(), r, weight, dr.contiguous(), x, scale)
        return dx, dres, dw, dscale


class GatedNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, gate, weight):
        ctx.save_for_backward(x, gate, weight)
        return kda.gated_norm_fwd(x, gate, weight, activation="silu")

    @staticmethod
    def backward(ctx, dy):
        return kda.gated_norm_bwd(dy.contiguous(), *ctx.saved_tensors, activation="silu")


class GatedDeltaRule(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, g, beta, cu):
        ctx.save_for_backward(q, k, v, g, beta, cu)
        return kda.gdr_chunk_fwd(q, k, v, g, beta, None, cu, output_final_state=False)[0]

    @staticmethod
    def backward(ctx, dout):
        q, k, v, g, beta, cu = ctx.saved_tensors
        grads = kda.gdr_chunk_bwd(q, k, v, g, beta, None, cu, dout.contiguous(), want_dh0=False)
        return (*grads[:5], None)


class Block(torch.nn.Module):
    def __init__(self, d_model, hk, hv, dk, dv):
        super().__init__()
        self.sizes = [hk * dk, hk * dk, hv * dv, hv * dv, hv, hv]
        self.hk, self.hv, self.dk, self.dv = hk, hv, dk, dv
        self.proj = torch.nn.Linear(d_model, sum(self.sizes), bias=False, dtype=torch.bfloat16)
        self.out = torch.nn.Linear(hv * dv, d_model, bias=False, dtype=torch.bfloat16)
        self.norm = torch.nn.Parameter(torch.ones(d_model))
        self.scale = torch.nn.Parameter(torch.full((d_model,), 0.5))
        self.out_norm = torch.nn.Parameter(torch.ones(dv))
        self.decay = torch.nn.Parameter(torch.linspace(-3, 1, hv))

    def project(self, y):
        q, k, v, gate, a, b = self.proj(y).split(self.sizes, -1)
        q, k = (F.normalize(x.unflatten(-1, (self.hk, self.dk)).float(), dim=-1).to(y.dtype) for x in (q, k))
        g = -self.decay.exp() * F.softplus(a.float())
        return (q, k, v.unflatten(-1, (self.hv, self.dv)), g, torch.sigmoid(b.float())), \
            gate.unflatten(-1, (self.hv, self.dv))

    def forward(self, x, residual, cu):
        """``x`` the previous block's output, ``residual`` the stream: this block's output and the
        stream with x in it, for packed sequences [N, d_model]."""
        y, residual = ResidualNorm.apply(x, residual, self.norm, self.scale)
        (q, k, v, g, beta), gate = self.project(y)
        o = GatedDeltaRule.apply(q, k, v, g, beta, cu)  # v and gate stay slices of the projection
        return self.out(GatedNorm.apply(o, gate, self.out_norm).flatten(1)), residual

    @torch.no_grad()
    def prefill(self, x, residual, cu, pool, slots):
        y, residual = kda.residual_norm_fwd(x, self.norm, residual, self.scale)
        (q, k, v, g, beta), gate = self.project(y)
        o, final = kda.gdr_chunk_fwd(q, k, v, g, beta, None, cu)
        pool[slots.long()] = final
        return self.out(kda.gated_norm_fwd(o, gate, self.out_norm, activation="silu").flatten(1)), residual

    @torch.no_grad()
    def step(self, x, residual, pool, slots):
        y, residual = kda.residual_norm_fwd(x, self.norm, residual, self.scale)
        (q, k, v, g, beta), gate = self.project(y)
        o = kda.gdr_step(q, k, v, g, beta, pool, slots)
        return self.out(kda.gated_norm_fwd(o, gate, self.out_norm, activation="silu").flatten(1)), residual


class Model(torch.nn.Module):
    def __init__(self, vocab=64, d_model=256, blocks=2, hk=2, hv=4, dk=64, dv=64):
        super().__init__()
        self.embed = torch.nn.Embedding(vocab, d_model, dtype=torch.bfloat16)
        self.blocks = torch.nn.ModuleList(Block(d_model, hk, hv, dk, dv) for _ in range(blocks))
        self.norm = torch.nn.Parameter(torch.ones(d_model))
        self.scale = torch.nn.Parameter(torch.ones(d_model))

    def logits(self, x, residual):
        y, _ = ResidualNorm.apply(x, residual, self.norm, self.scale)
        return y @ self.embed.weight.T

    def run(self, tokens, each):
        x = self.embed(tokens)
        residual = torch.zeros_like(x)
        for i, b in enumerate(self.blocks):
            x, residual = each(i, b, x, residual)
        return self.logits(x, residual)

    def forward(self, tokens, cu):
        return self.run(tokens, lambda i, b, x, r: b(x, r, cu))

    def new_pools(self, slots):
        return [torch.zeros((slots, b.hv, b.dk, b.dv), device=self.norm.device) for b in self.blocks]


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
    packed = torch.cat(prompts).to("cuda")
    logits = model.run(packed, lambda i, b, x, r: b.prefill(x, r, cu, pools[i], slots))[cu[1:].long() - 1]
    out, seen = [], []
    for _ in range(tokens_to_go):
        nxt = logits.argmax(-1)
        out.append(nxt)
        seen.append(logits)
        logits = model.run(nxt, lambda i, b, x, r: b.step(x, r, pools[i], slots))
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
