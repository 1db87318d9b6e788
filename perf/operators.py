"""The operators of a gated delta rule block, as cases to be measured: the gated delta rule
with one decay per head (chunked forward, its backward pass, the one-token step over a
pool of states), the residual norm before a block and the gated norm after it.

    S_t = exp(g_t) S_{t-1} + beta_t k_t (v_t - exp(g_t) S_{t-1}^T k_t)^T
    o_t = d_k^-1/2 S_t^T q_t                      (value head h reads key head h / (H_v / H_k))
    r = residual + scale * x,   y = r / rms(r) * weight
    y = x / rms(x) * weight * act(gate)           (per token and head)

``run`` computes them in elementary torch operations in 32 bits where ``own`` is false, and
calls the package's entry points where it is true.
"""
import math

import torch
import torch.nn.functional as F

own = False

DEV = "cuda"
CHUNK = 64
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
EPS = 1e-6


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a short chat prompt: one sequence, latency counts
        dict(name="gdr_fwd_prompt40", op="gdr_fwd", total=40, n_seq=1, hk=16, hv=32, dk=128,
             dv=128, dtype="bf16", h0=False, resets=0),
        # prefill of the 64K-token context workload, two value heads per key head
        dict(name="gdr_fwd_context64k", op="gdr_fwd", total=65536, n_seq=1, hk=16, hv=32, dk=128,
             dv=128, dtype="bf16", h0=False, resets=0),
        # packed ragged sequences (an empty one, a one-token one), continued states, document
        # boundaries inside a sequence (log-decay -inf)
        dict(name="gdr_fwd_packed", op="gdr_fwd", total=20011, n_seq=12, hk=16, hv=16, dk=128,
             dv=128, dtype="bf16", h0=True, resets=9),
        # fp32 at head sizes that are no powers of two
        dict(name="gdr_fwd_fp32_odd", op="gdr_fwd", total=1531, n_seq=3, hk=2, hv=6, dk=72,
             dv=100, dtype="fp32", h0=True, resets=2),
        # a training step's backward pass over two 8K sequences
        dict(name="gdr_bwd_8k", op="gdr_bwd", total=16384, n_seq=2, hk=16, hv=32, dk=128, dv=128,
             dtype="bf16", h0=False, resets=0),
        # fp32 backward, ragged sequences, carried states and their gradients
        dict(name="gdr_bwd_fp32_ragged", op="gdr_bwd", total=777, n_seq=5, hk=2, hv=4, dk=64,
             dv=40, dtype="fp32", h0=True, resets=1),
        # one token of one sequence: generation at batch 1
        dict(name="gdr_step_b1", op="gdr_step", batch=1, slots=4, hk=16, hv=32, dk=128, dv=128,
             dtype="bf16"),
        # one token of 253 running sequences of a pool of 300 states, a few rows padded
        dict(name="gdr_step_b253", op="gdr_step", batch=253, slots=300, hk=16, hv=32, dk=128,
             dv=128, dtype="bf16"),
        # the norm of one token in generation
        dict(name="res_norm_fwd_1", op="res_norm_fwd", rows=1, d=4096, dtype="bf16", scale=True),
        # its backward over a training batch, residual scale trained
        dict(name="res_norm_bwd_32k", op="res_norm_bwd", rows=32768, d=4096, dtype="bf16",
             scale=True),
        # the output norm of a 64K-token prefill, gate a slice of a wider projection
        dict(name="gated_norm_fwd_64k", op="gated_norm_fwd", rows=65536, heads=32, d=128,
             dtype="bf16", act="silu", wide=True),
        # its backward over an odd number of tokens
        dict(name="gated_norm_bwd_8191", op="gated_norm_bwd", rows=8191, heads=32, d=128,
             dtype="bf16", act="sigmoid", wide=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gdr_fwd", "gdr_fwd", "gdr_bwd", "gdr_bwd", "gdr_step", "res_norm_fwd",
                     "res_norm_bwd", "gated_norm_fwd", "gated_norm_bwd"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    if op in ("gdr_fwd", "gdr_bwd"):
        hk = rng.choice([1, 2, 3, 4, 8, 16])
        hv = hk * rng.choice([1, 2, 3, 4] if hk <= 4 else [1, 2])
        most = (65536 if op == "gdr_fwd" else 16384) // (1 if dtype == "bf16" else 8)
        total = _log(rng, 1, most)
        return dict(op=op, total=total, n_seq=min(rng.choice([1, 1, 2, 3, 7, 16]), total), hk=hk,
                    hv=hv, dk=rng.choice([128, 128, 64, 96, 40, 33]),
                    dv=rng.choice([128, 128, 64, 112, 72, 31]), dtype=dtype,
                    h0=rng.random() < 0.5, resets=rng.choice([0, 0, 1, 5]))
    if op == "gdr_step":
        batch = _log(rng, 1, 250)
        hk = rng.choice([2, 4, 8, 16])
        return dict(op=op, batch=batch, slots=batch + rng.randrange(0, 50), hk=hk,
                    hv=hk * rng.choice([1, 2]), dk=rng.choice([128, 128, 64, 40]),
                    dv=rng.choice([128, 128, 64, 72]), dtype=dtype)
    if op.startswith("res_norm"):
        d = rng.choice([rng.randrange(1, 2000), 1024, 2048, 4096, 7168])
        top = 32768 * 4096 // d // (1 if dtype == "bf16" else 2)
        return dict(op=op, rows=_log(rng, 1, min(65536, top)), d=d, dtype=dtype,
                    scale=rng.random() < 0.5)
    heads = rng.choice([1, 4, 16, 31, 32])
    top = 65536 if op == "gated_norm_fwd" else 32768
    return dict(op=op, rows=_log(rng, 1, top // (1 if dtype == "bf16" else 2)), heads=heads,
                d=rng.choice([128, 128, 64, 100, 256]), dtype=dtype,
                act=rng.choice(["sigmoid", "silu"]), wide=rng.random() < 0.5)


# ---------------------------------------------------------------- inputs

def _lengths(case, gen):
    """Ragged lengths that sum to ``total``: an empty and a one-token sequence among three or
    more, the rest cut at random."""
    total, n = case["total"], case["n_seq"]
    if n == 1:
        return [total]
    if n == 2:
        return [total // 2, total - total // 2]
    fixed = [0, 1] if total > 1 else [0]
    m = n - len(fixed)
    left = total - sum(fixed)
    w = torch.rand(m, generator=gen, dtype=torch.float64) + 0.05
    cut = [0] + [int(x) for x in (w.cumsum(0) / w.sum() * left).round().tolist()]
    cut[-1] = left
    rest = [b - a for a, b in zip(cut[:-1], cut[1:])]
    return rest[:1] + fixed + rest[1:]


def _unit(x):
    return x / x.norm(dim=-1, keepdim=True).clamp_min(1e-6)


def prepare(case, seed):
    cpu = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=DEV)

    def rand(*shape):
        return torch.rand(shape, generator=gen, device=DEV)

    op, dt = case["op"], DT[case["dtype"]]
    s = {"case": case}
    if op.startswith("gdr"):
        hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
        n = case["batch"] if op == "gdr_step" else case["total"]
        # keys and queries of unit length; neighbouring keys alike, as text gives them
        k = randn(n, hk, dk)
        k = _unit(k + 0.5 * k.roll(1, 0))
        s["q"], s["k"] = _unit(randn(n, hk, dk)).to(dt), k.to(dt)
        s["v"] = randn(n, hv, dv).to(dt)
        # g = -A softplus(x + b): A per head in (0, 16), time steps of 0.001 to 0.1
        a = 16 * rand(hv)
        step = torch.exp(rand(hv) * math.log(100.0) + math.log(0.001))
        s["g"] = -a * F.softplus(0.5 * randn(n, hv) + step + torch.log(-torch.expm1(-step)))
        s["beta"] = torch.sigmoid(randn(n, hv))
    if op in ("gdr_fwd", "gdr_bwd"):
        lens = _lengths(case, cpu)
        s["lengths"] = lens
        s["cu"] = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32,
                               device=DEV)
        if case["resets"]:  # a new document starts: nothing of the state is kept
            at = torch.randint(0, n, (case["resets"],), generator=cpu)
            s["g"][at.to(DEV)] = -math.inf
        s["h0"] = 0.3 * randn(len(lens), hv, dk, dv) if case["h0"] else None
    if op == "gdr_bwd":
        s["dout"] = randn(n, hv, dv).to(dt)
        s["dhf"] = 0.3 * randn(len(lens), hv, dk, dv) if case["h0"] else None
    if op == "gdr_step":
        s["state"] = 0.3 * randn(case["slots"], hv, dk, dv)
        slots = torch.randperm(case["slots"], generator=cpu)[:n].to(torch.int32)
        if n >= 8:  # rows of a padded batch that hold no sequence
            slots[torch.randperm(n, generator=cpu)[:n // 32 + 1]] = -1
        s["slots"] = slots.to(DEV)
    if op.startswith("res_norm"):
        n, d = case["rows"], case["d"]
        s["x"], s["res"] = randn(n, d).to(dt), (2 * randn(n, d)).to(dt)
        s["w"] = 1 + 0.2 * randn(d)
        s["scale"] = 0.3 + 0.1 * randn(d) if case["scale"] else None
        if op == "res_norm_bwd":
            s["dy"], s["dr"] = randn(n, d).to(dt), randn(n, d).to(dt)
    if op.startswith("gated_norm"):
        n, h, d = case["rows"], case["heads"], case["d"]
        s["x"] = (randn(n, h, d) * torch.exp(0.5 * randn(n, h, 1))).to(dt)
        gate = randn(n, 2 * h if case["wide"] else h, d).to(dt)
        s["gate"] = gate[:, -h:]
        s["w"] = 1 + 0.2 * randn(d)
        if op == "gated_norm_bwd":
            s["dy"] = randn(n, h, d).to(dt)
    return s


# ---------------------------------------------------------------- plain forms

def _index(lengths):
    """Token index [B, chunks, CHUNK] of every chunk position and whether it holds a token."""
    lens = torch.tensor(lengths, device=DEV)
    start = lens.cumsum(0) - lens
    nc = max(1, -(-max(lengths) // CHUNK))
    t = torch.arange(nc * CHUNK, device=DEV).view(1, nc, CHUNK)
    ok = t < lens.view(-1, 1, 1)
    return torch.where(ok, start.view(-1, 1, 1) + t, 0), ok


def _invert(m):
    """Inverse of unit lower triangular matrices [..., n, n], n a power of two, by halves:
    [[a, 0], [c, b]]^-1 = [[a', 0], [-b' c a', b']], doubling the blocks that are done."""
    n = m.shape[-1]
    x = torch.eye(n, device=m.device).expand_as(m).clone()
    size = 1
    while size < n:
        blocks = m.unflatten(-2, (-1, 2, size)).unflatten(-1, (-1, 2, size))
        done = x.unflatten(-2, (-1, 2, size)).unflatten(-1, (-1, 2, size))
        i = torch.arange(n // (2 * size), device=m.device)
        c = blocks[..., i, 1, :, i, 0, :].movedim(0, -3)
        a = done[..., i, 0, :, i, 0, :].movedim(0, -3)
        b = done[..., i, 1, :, i, 1, :].movedim(0, -3)
        done[..., i, 1, :, i, 0, :] = -(b @ c @ a).movedim(-3, 0)
        size *= 2
    return x


def _chunk_terms(s):
    """What of each chunk does not depend on the state, [B, H, chunks, ...] in 32 bits."""
    hv, hk = s["v"].shape[1], s["q"].shape[1]
    idx, ok = _index(s["lengths"])

    def take(x):
        x = x.float()[idx] * ok.view(*ok.shape, *([1] * (x.dim() - 1)))
        return x.movedim(3, 1)

    q, k = (take(x.repeat_interleave(hv // hk, 1)) for x in (s["q"], s["k"]))
    v, beta = take(s["v"]), take(s["beta"]).unsqueeze(-1)
    g = torch.where(ok.unsqueeze(1), s["g"].float()[idx].movedim(3, 1), 0.0)
    # d[r, j] = sum of g over (j, r]: summed from j + 1 on, so that -inf gives no inf - inf
    low = torch.ones(CHUNK, CHUNK, device=DEV).tril(-1).bool()
    d = torch.where(low, g.unsqueeze(-1), 0.0).cumsum(-2)
    e = torch.where(low | torch.eye(CHUNK, device=DEV).bool(), torch.exp(d), 0.0)
    head = torch.exp(g.cumsum(-1)).unsqueeze(-1)
    tail = e[..., -1, :].unsqueeze(-1)
    kk, qk = k @ k.mT, q @ k.mT
    x = _invert(torch.eye(CHUNK, device=DEV) + torch.where(low, beta * e * kk, 0.0))
    return dict(idx=idx, ok=ok, q=q, k=k, v=v, beta=beta, e=e, low=low, head=head, tail=tail,
                kk=kk, qk=qk, x=x, p=e * qk, whole=head[..., -1:, :])


def _gdr_states(s, t):
    """The state at each chunk's start, the corrected values, and the final states."""
    n, hv, dk, dv = len(s["lengths"]), s["v"].shape[1], s["q"].shape[2], s["v"].shape[2]
    st = torch.zeros(n, hv, dk, dv, device=DEV) if s["h0"] is None else s["h0"]
    wk = t["x"] @ (t["beta"] * t["head"] * t["k"])
    u0 = t["x"] @ (t["beta"] * t["v"])
    kt = (t["tail"] * t["k"]).mT
    starts, us = [], []
    for c in range(t["k"].shape[2]):  # the chunks of a sequence follow one another
        starts.append(st)
        us.append(u0[:, :, c] - wk[:, :, c] @ st)
        st = t["whole"][:, :, c] * st + kt[:, :, c] @ us[-1]
    return torch.stack(starts, 2), torch.stack(us, 2), st


def _scatter(x, t, like):
    out = torch.empty(like.shape, dtype=like.dtype, device=DEV)
    out[t["idx"][t["ok"]]] = x.movedim(1, 3)[t["ok"]].to(like.dtype)
    return out


def _plain_gdr_fwd(s):
    t = _chunk_terms(s)
    starts, u, final = _gdr_states(s, t)
    o = (t["head"] * t["q"]) @ starts + t["p"] @ u
    return {"out": _scatter(o * s["q"].shape[2] ** -0.5, t, s["v"]), "h_final": final}


def _plain_gdr_bwd(s):
    t = _chunk_terms(s)
    starts, u, _ = _gdr_states(s, t)
    q, k, e, low, beta, head, tail, x = (t[n] for n in
                                         ("q", "k", "e", "low", "beta", "head", "tail", "x"))
    do = s["dout"].float()[t["idx"]] * t["ok"].view(*t["ok"].shape, 1, 1)
    do = do.movedim(3, 1) * s["q"].shape[2] ** -0.5
    n, hv, dk, dv = starts.shape[0], starts.shape[1], starts.shape[3], starts.shape[4]
    ds = torch.zeros(n, hv, dk, dv, device=DEV) if s["dhf"] is None else s["dhf"]
    pdo, kt, xt = t["p"].mT @ do, tail * k, x.mT
    qdo = (head * q).mT @ do
    kh = (head * beta * k).mT
    ends, errs = [], []
    for c in reversed(range(k.shape[2])):
        ends.append(ds)
        errs.append(xt[:, :, c] @ (pdo[:, :, c] + kt[:, :, c] @ ds))
        ds = t["whole"][:, :, c] * ds + qdo[:, :, c] - kh[:, :, c] @ errs[-1]
    ends, err = torch.stack(ends[::-1], 2), torch.stack(errs[::-1], 2)
    z = t["v"] - head * (k @ starts)
    eu = torch.where(low, err @ u.mT, 0.0) * e
    dqk = (do @ u.mT) * e
    dkk = -beta * eu
    dos, dzs, uds = do @ starts.mT, (beta * err) @ starts.mT, u @ ends.mT
    dq = head * dos + dqk @ k
    dk_ = -head * dzs + tail * uds + dqk.mT @ q + (dkk + dkk.mT) @ k
    db = (err * z).sum(-1) - (eu * t["kk"]).sum(-1)
    m = torch.where(low, dkk * t["kk"] + dqk * t["qk"], 0.0)
    a = (head * (q * dos - k * dzs)).sum(-1)
    b = (tail * k * uds).sum(-1)
    whole = (t["whole"] * starts * ends).sum((-1, -2)).unsqueeze(-1)
    # g_i reaches a_r for r >= i, b_r for r < i and m[r, j] for j < i <= r
    inner = (m.cumsum(-1) - m).flip(-2).cumsum(-2).flip(-2).diagonal(dim1=-2, dim2=-1)
    dg = whole + a.flip(-1).cumsum(-1).flip(-1) + b.cumsum(-1) - b + inner
    group = s["v"].shape[1] // s["q"].shape[1]

    def shared(x):
        return x.unflatten(1, (-1, group)).sum(2)

    return {"dq": _scatter(shared(dq), t, s["q"]), "dk": _scatter(shared(dk_), t, s["k"]),
            "dv": _scatter(beta * err, t, s["v"]), "dg": _scatter(dg, t, s["g"]),
            "dbeta": _scatter(db, t, s["beta"]), "dh0": ds}


def _plain_gdr_step(s):
    live = s["slots"] >= 0
    at = s["slots"][live].long()
    rep = s["v"].shape[1] // s["q"].shape[1]
    q, k = (x.float()[live].repeat_interleave(rep, 1).unsqueeze(-1) for x in (s["q"], s["k"]))
    st = s["state"][at] * torch.exp(s["g"][live])[..., None, None]
    u = s["beta"][live][..., None, None] * (s["v"].float()[live].unsqueeze(-2) - k.mT @ st)
    st = st + k * u
    s["state"][at] = st
    out = torch.zeros_like(s["v"])
    out[live] = ((q.mT @ st).squeeze(-2) * s["q"].shape[2] ** -0.5).to(out.dtype)
    return {"out": out, "state": s["state"]}


def _plain_res_norm_fwd(s):
    x, res = s["x"].float(), s["res"].float()
    r = res + (x if s["scale"] is None else s["scale"] * x)
    y = r * torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS) * s["w"]
    return {"y": y.to(s["x"].dtype), "r": r.to(s["x"].dtype)}


def _plain_res_norm_bwd(s):
    # the residual stream as the forward pass left it stands in "res"
    r, dy = s["res"].float(), s["dy"].float()
    rstd = torch.rsqrt(r.square().mean(-1, keepdim=True) + EPS)
    n, dn = r * rstd, dy * s["w"]
    dr = rstd * (dn - n * (dn * n).mean(-1, keepdim=True)) + s["dr"].float()
    out = {"dres": dr.to(s["x"].dtype), "dw": (dy * n).sum(0)}
    if s["scale"] is not None:
        out["dx"] = (s["scale"] * dr).to(s["x"].dtype)
        out["dscale"] = (dr * s["x"].float()).sum(0)
    return out


def _act(gate, act):
    sig = 1 / (1 + torch.exp(-gate))
    if act == "sigmoid":
        return sig, sig * (1 - sig)
    return gate * sig, sig * (1 + gate * (1 - sig))


def _plain_gated_norm_fwd(s):
    x = s["x"].float()
    n = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return (n * s["w"] * _act(s["gate"].float(), s["case"]["act"])[0]).to(s["x"].dtype)


def _plain_gated_norm_bwd(s):
    x, dy = s["x"].float(), s["dy"].float()
    a, da = _act(s["gate"].float(), s["case"]["act"])
    rstd = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    n = x * rstd
    dn = dy * s["w"] * a
    dx = rstd * (dn - n * (dn * n).mean(-1, keepdim=True))
    return {"dx": dx.to(s["x"].dtype), "dgate": (dy * n * s["w"] * da).to(s["x"].dtype),
            "dw": (dy * n * a).sum((0, 1))}


PLAIN = {"gdr_fwd": _plain_gdr_fwd, "gdr_bwd": _plain_gdr_bwd, "gdr_step": _plain_gdr_step,
         "res_norm_fwd": _plain_res_norm_fwd, "res_norm_bwd": _plain_res_norm_bwd,
         "gated_norm_fwd": _plain_gated_norm_fwd, "gated_norm_bwd": _plain_gated_norm_bwd}


# ---------------------------------------------------------------- the package's operators

def _own(s):
    import chunked_linear_attention_kda_gb300 as kda
    op = s["case"]["op"]
    if op == "gdr_fwd":
        out, final = kda.gdr_chunk_fwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["h0"], s["cu"])
        return {"out": out, "h_final": final}
    if op == "gdr_bwd":
        grads = kda.gdr_chunk_bwd(s["q"], s["k"], s["v"], s["g"], s["beta"], s["h0"], s["cu"],
                                  s["dout"], s["dhf"])
        return dict(zip(("dq", "dk", "dv", "dg", "dbeta", "dh0"), grads))
    if op == "gdr_step":
        out = kda.gdr_step(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], s["slots"])
        return {"out": out, "state": s["state"]}
    if op == "res_norm_fwd":
        y, r = kda.residual_norm_fwd(s["x"], s["w"], s["res"], s["scale"], eps=EPS)
        return {"y": y, "r": r}
    if op == "res_norm_bwd":
        dx, dres, dw, dscale = kda.residual_norm_bwd(
            s["dy"], s["res"], s["w"], s["dr"], None if s["scale"] is None else s["x"],
            s["scale"], eps=EPS)
        out = {"dres": dres, "dw": dw}
        return out if s["scale"] is None else {**out, "dx": dx, "dscale": dscale}
    if op == "gated_norm_fwd":
        return kda.gated_norm_fwd(s["x"], s["gate"], s["w"], eps=EPS, activation=s["case"]["act"])
    dx, dgate, dw = kda.gated_norm_bwd(s["dy"], s["x"], s["gate"], s["w"], eps=EPS,
                                       activation=s["case"]["act"])
    return {"dx": dx, "dgate": dgate, "dw": dw}


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op, es = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op.startswith("gdr"):
        hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
        n = case["batch"] if op == "gdr_step" else case["total"]
        tok = n * ((2 * hk * dk + hv * dv) * es + 8 * hv)   # q, k, v, g, beta
        st = 4 * hv * dk * dv
        outer = 2 * dk * dv * n * hv                        # one product with, or update of, the state
        if op == "gdr_step":
            live = n - (n // 32 + 1 if n >= 8 else 0)
            return {"bytes": tok + n * hv * dv * es + 4 * n + 2 * live * st, "flops": 3.5 * outer}
        seqs = case["n_seq"] * st * (2 if case["h0"] else 1)
        if op == "gdr_fwd":  # S^T k, the write, S^T q
            return {"bytes": tok + n * hv * dv * es + seqs, "flops": 3 * outer}
        # the forward's state again, then dS: two products read dS, two write it, three read S
        return {"bytes": 2 * tok + n * hv * dv * es + seqs * 2, "flops": 8 * outer}
    if op.startswith("res_norm"):
        n = case["rows"] * case["d"]
        params = 4 * case["d"] * (2 if case["scale"] else 1)
        if op == "res_norm_fwd":
            return {"bytes": 4 * n * es + params, "flops": 6 * n}
        return {"bytes": (6 if case["scale"] else 4) * n * es + 2 * params, "flops": 14 * n}
    n = case["rows"] * case["heads"] * case["d"]
    if op == "gated_norm_fwd":
        return {"bytes": 3 * n * es + 4 * case["d"], "flops": 10 * n}
    return {"bytes": 5 * n * es + 8 * case["d"], "flops": 24 * n}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "gdr_step":
        return _exact_step(s)
    if op.startswith("gdr"):
        # about 60 us a token forward, 400 us with the backward pass
        if max(s["lengths"]) > (70000 if op == "gdr_fwd" else 20000):
            return None
        return _exact_scan(s, op == "gdr_bwd")
    if op.startswith("res_norm"):
        return _exact_res_norm(s, op.endswith("bwd"))
    return _exact_gated_norm(s, op.endswith("bwd"))


def _exact_step(s):
    state, out = s["state"].double(), torch.zeros(s["v"].shape, dtype=torch.float64, device=DEV)
    rep = s["v"].shape[1] // s["q"].shape[1]
    for b, slot in enumerate(s["slots"].tolist()):
        if slot < 0:
            continue
        k = s["k"][b].double().repeat_interleave(rep, 0)
        q = s["q"][b].double().repeat_interleave(rep, 0)
        old = state[slot] * s["g"][b].double().exp().view(-1, 1, 1)
        err = s["v"][b].double() - torch.einsum("hkv,hk->hv", old, k)
        state[slot] = old + torch.einsum("h,hk,hv->hkv", s["beta"][b].double(), k, err)
        out[b] = torch.einsum("hkv,hk->hv", state[slot], q) / math.sqrt(s["q"].shape[2])
    return {"out": out, "state": state}


def _exact_scan(s, backward):
    """Token after token, all sequences side by side; a token past its sequence's end has
    g = 0 and beta = 0 and leaves the state alone."""
    lens, rep = s["lengths"], s["v"].shape[1] // s["q"].shape[1]
    cu = [sum(lens[:i]) for i in range(len(lens) + 1)]
    T, nb, hv, dk, dv = max(lens), len(lens), s["v"].shape[1], s["q"].shape[2], s["v"].shape[2]

    def lay(x):  # [T, B, ...]
        o = torch.zeros(T, nb, *x.shape[1:], dtype=torch.float64, device=DEV)
        for b in range(nb):
            o[:lens[b], b] = x[cu[b]:cu[b + 1]].double()
        return o

    def back(o, like):
        x = torch.zeros(like.shape, dtype=torch.float64, device=DEV)
        for b in range(nb):
            x[cu[b]:cu[b + 1]] = o[:lens[b], b]
        return x

    q, k, v, g, beta = (lay(s[n]) for n in ("q", "k", "v", "g", "beta"))
    alpha = g.exp()
    c = 1 / math.sqrt(dk)

    def heads(x):  # [B, Hk, dk] -> [B * Hv, 1, dk]
        return x.repeat_interleave(rep, 1).reshape(nb * hv, 1, dk)

    def forward(S, t):
        kt = heads(k[t])
        S = S * alpha[t].reshape(-1, 1, 1)
        u = beta[t].reshape(-1, 1, 1) * (v[t].reshape(-1, 1, dv) - torch.bmm(kt, S))
        return torch.baddbmm(S, kt.transpose(1, 2), u), u

    S = torch.zeros(nb * hv, dk, dv, dtype=torch.float64, device=DEV) if s["h0"] is None \
        else s["h0"].double().reshape(nb * hv, dk, dv)
    if not backward:
        out = torch.zeros(T, nb, hv, dv, dtype=torch.float64, device=DEV)
        for t in range(T):
            S, _ = forward(S, t)
            out[t] = (c * torch.bmm(heads(q[t]), S)).view(nb, hv, dv)
        return {"out": back(out, s["v"]), "h_final": S.view(nb, hv, dk, dv)}

    block = 64
    marks = []
    for t in range(T):
        if t % block == 0:
            marks.append(S)
        S, _ = forward(S, t)
    do = lay(s["dout"])
    dq, dk_, dv_ = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg, db = torch.zeros_like(g), torch.zeros_like(beta)
    dS = torch.zeros_like(S) if s["dhf"] is None else s["dhf"].double().reshape(nb * hv, dk, dv)
    for m in reversed(range(len(marks))):
        t0, t1 = m * block, min(T, (m + 1) * block)
        chain = [marks[m]]
        for t in range(t0, t1):
            chain.append(forward(chain[-1], t)[0])
        for t in reversed(range(t0, t1)):
            kt, qt = heads(k[t]).transpose(1, 2), heads(q[t]).transpose(1, 2)
            al, be = alpha[t].reshape(-1, 1, 1), beta[t].reshape(-1, 1, 1)
            d = c * do[t].reshape(-1, 1, dv)
            old = chain[t - t0] * al
            err = v[t].reshape(-1, 1, dv) - torch.bmm(kt.transpose(1, 2), old)
            dqt = torch.bmm(chain[t - t0 + 1], d.transpose(1, 2))
            dS = torch.baddbmm(dS, qt, d)
            kd = torch.bmm(kt.transpose(1, 2), dS)          # [*, 1, dv]
            derr = be * kd
            dkt = be * torch.bmm(dS, err.transpose(1, 2)) - torch.bmm(old, derr.transpose(1, 2))
            db[t] = (kd * err).sum((1, 2)).view(nb, hv)
            dv_[t] = derr.view(nb, hv, dv)
            dold = torch.baddbmm(dS, kt, -derr)
            dg[t] = (dold * old).sum((1, 2)).view(nb, hv)
            dS = dold * al
            dq[t] = dqt.view(nb, -1, rep, dk).sum(2)
            dk_[t] = dkt.view(nb, -1, rep, dk).sum(2)
    return {"dq": back(dq, s["q"]), "dk": back(dk_, s["k"]), "dv": back(dv_, s["v"]),
            "dg": back(dg, s["g"]), "dbeta": back(db, s["beta"]),
            "dh0": dS.view(nb, hv, dk, dv)}


def _exact_res_norm(s, backward):
    w = s["w"].double()
    if not backward:
        r = s["x"].double() * (1.0 if s["scale"] is None else s["scale"].double()) + s["res"].double()
        y = w * r / ((r * r).sum(1, keepdim=True) / r.shape[1] + EPS).sqrt()
        return {"y": y, "r": r}
    r, dy = s["res"].double(), s["dy"].double()
    ms = (r * r).sum(1, keepdim=True) / r.shape[1] + EPS
    # y_i = w_i r_i ms^-1/2: dL/dr_j = w_j dy_j ms^-1/2 - r_j ms^-3/2 (sum_i w_i dy_i r_i) / d
    wd = w * dy
    dr = wd * ms ** -0.5 - r * ms ** -1.5 * (wd * r).sum(1, keepdim=True) / r.shape[1]
    dr = dr + s["dr"].double()
    out = {"dres": dr, "dw": (dy * r * ms ** -0.5).sum(0)}
    if s["scale"] is not None:
        out["dx"] = dr * s["scale"].double()
        out["dscale"] = (dr * s["x"].double()).sum(0)
    return out


def _exact_gated_norm(s, backward):
    w, x, z = s["w"].double(), s["x"].double(), s["gate"].double()
    ms = (x * x).sum(2, keepdim=True) / x.shape[2] + EPS
    sig = torch.sigmoid(z)
    a = sig if s["case"]["act"] == "sigmoid" else z * sig
    if not backward:
        return w * a * x / ms.sqrt()
    da = sig * (1 - sig) if s["case"]["act"] == "sigmoid" else sig + z * sig * (1 - sig)
    dy = s["dy"].double()
    wd = w * a * dy
    dx = wd * ms ** -0.5 - x * ms ** -1.5 * (wd * x).sum(2, keepdim=True) / x.shape[2]
    nx = x * ms ** -0.5
    return {"dx": dx, "dgate": dy * nx * w * da, "dw": (dy * a * nx).sum((0, 1))}
