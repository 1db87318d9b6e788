"""fp64 definitions of the operators around the gated delta rule with one decay per head.

TEST INFRASTRUCTURE ONLY (see the package docstring).

Plain PyTorch fp64 CPU operations: the recurrence one token at a time (all heads at once),
the norms written out. Gradients come from reverse-mode differentiation of these forward
definitions; the tests hold them to central differences.
"""
from __future__ import annotations

import torch


def f64(t):
    return None if t is None else t.detach().to("cpu", torch.float64)


def gdr(q, k, v, g, beta, h0, cu):
    """``q, k`` [N, H_k, d_k], ``v`` [N, H, d_v], ``g, beta`` [N, H], ``h0`` [n, H, d_k, d_v] or
    None, ``cu`` the sequence offsets. Returns ``(out, h_final)``."""
    group = v.shape[1] // q.shape[1]
    scale = q.shape[2] ** -0.5
    outs, ends = [], []
    for n, (a, b) in enumerate(zip(cu[:-1], cu[1:])):
        S = torch.zeros(v.shape[1], q.shape[2], v.shape[2], dtype=torch.float64) if h0 is None else h0[n]
        for t in range(a, b):
            kt, qt = (x[t].repeat_interleave(group, 0) for x in (k, q))
            S = g[t].exp()[:, None, None] * S
            u = beta[t][:, None] * (v[t] - torch.einsum("hkv,hk->hv", S, kt))
            S = S + kt[:, :, None] * u[:, None, :]
            outs.append(scale * torch.einsum("hkv,hk->hv", S, qt))
        ends.append(S)
    out = torch.stack(outs) if outs else v.new_zeros(0, *v.shape[1:])
    return out, torch.stack(ends) if ends else v.new_zeros(0, v.shape[1], q.shape[2], v.shape[2])


def gdr_grads(q, k, v, g, beta, h0, cu, dout, dh_final):
    """Gradients of ``<dout, out> + <dh_final, h_final>``: ``(dq, dk, dv, dg, dbeta, dh0)``
    (``dh0`` with respect to a zero start state when ``h0`` is None)."""
    if h0 is None:
        h0 = torch.zeros(len(cu) - 1, v.shape[1], q.shape[2], v.shape[2], dtype=torch.float64)
    xs = [x.clone().requires_grad_(True) for x in (q, k, v, g, beta, h0)]
    out, end = gdr(*xs, cu)
    loss = (out * dout).sum()
    if dh_final is not None:
        loss = loss + (end * dh_final).sum()
    return torch.autograd.grad(loss, xs, allow_unused=True, materialize_grads=True)


def residual_norm(x, weight, residual, scale, eps):
    """``(y, r)``."""
    r = x if scale is None else scale * x
    r = r if residual is None else residual + r
    return weight * r / torch.sqrt((r * r).mean(-1, keepdim=True) + eps), r


def residual_norm_grads(dy, r, weight, dr, x, scale, eps):
    """From the r that the forward pass wrote: ``(dx, dresidual, dweight, dscale)``."""
    r, w = r.clone().requires_grad_(True), weight.clone().requires_grad_(True)
    y = w * r / torch.sqrt((r * r).mean(-1, keepdim=True) + eps)
    loss = (y * dy).sum() if dr is None else (y * dy).sum() + (r * dr).sum()
    dres, dw = torch.autograd.grad(loss, (r, w))
    if scale is None:
        return dres, dres, dw, None
    return scale * dres, dres, dw, (x * dres).sum(0)


def gated_norm(x, gate, weight, eps, activation):
    a = torch.sigmoid(gate)
    a = gate * a if activation == "silu" else a
    return weight * x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * a


def gated_norm_grads(dy, x, gate, weight, eps, activation):
    xs = [t.clone().requires_grad_(True) for t in (x, gate, weight)]
    return torch.autograd.grad((gated_norm(*xs, eps, activation) * dy).sum(), xs)
