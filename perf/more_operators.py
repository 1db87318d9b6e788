"""Linear attention with one decay per head (chunked forward, its backward pass, the one-token
step over a pool of states) and the norm of queries and keys per head with the position rotation
that comes before it, as cases to be measured.

    S_t = exp(g_t) S_{t-1} + k_t v_t^T,   o_t = d_k^-1/2 S_t^T q_t
                                          (value head h reads key head h / (H_v / H_k))
    y = rotate(x / rms(x) * weight, position * frequencies)      (per token and head of q and k)

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
BASE = 10000.0


# ---------------------------------------------------------------- cases

def listed():
    return [
        # a short chat prompt: one sequence, latency counts; every head forgets at its own
        # constant rate
        dict(name="dla_fwd_prompt40", op="dla_fwd", total=40, n_seq=1, hk=32, hv=32, dk=128,
             dv=128, dtype="bf16", decay="head", h0=False, resets=0),
        # prefill of the 64K-token context workload of 32 heads
        dict(name="dla_fwd_context64k", op="dla_fwd", total=65536, n_seq=1, hk=32, hv=32, dk=128,
             dv=128, dtype="bf16", decay="token", h0=False, resets=0),
        # packed ragged sequences (an empty one, a one-token one), continued states, document
        # boundaries inside a sequence (log-decay -inf), many value heads to a key head
        dict(name="dla_fwd_packed", op="dla_fwd", total=20011, n_seq=12, hk=4, hv=32, dk=128,
             dv=64, dtype="bf16", decay="token", h0=True, resets=9),
        # fp32 at head sizes that are no powers of two
        dict(name="dla_fwd_fp32_odd", op="dla_fwd", total=1531, n_seq=3, hk=2, hv=6, dk=72,
             dv=100, dtype="fp32", decay="token", h0=True, resets=2),
        # a training step's backward pass over two 8K sequences
        dict(name="dla_bwd_8k", op="dla_bwd", total=16384, n_seq=2, hk=32, hv=32, dk=128, dv=128,
             dtype="bf16", decay="token", h0=False, resets=0),
        # ragged sequences, value heads that share keys, carried states and their gradients
        dict(name="dla_bwd_packed", op="dla_bwd", total=5003, n_seq=7, hk=4, hv=16, dk=128, dv=64,
             dtype="bf16", decay="token", h0=True, resets=3),
        # fp32 backward of a short ragged batch, the rates themselves trained
        dict(name="dla_bwd_fp32_ragged", op="dla_bwd", total=777, n_seq=5, hk=2, hv=4, dk=64,
             dv=40, dtype="fp32", decay="head", h0=True, resets=0),
        # one token of one sequence: generation at batch 1
        dict(name="dla_step_b1", op="dla_step", batch=1, slots=4, hk=32, hv=32, dk=128, dv=128,
             dtype="bf16", decay="head"),
        # one token of 253 running sequences of a pool of 300 states, a few rows padded
        dict(name="dla_step_b253", op="dla_step", batch=253, slots=300, hk=32, hv=32, dk=128,
             dv=128, dtype="bf16", decay="token"),
        # one token in generation, far into its sequence
        dict(name="qk_norm_rope_fwd_1", op="qkn_fwd", total=1, hq=32, hk=32, d=128, rot=64,
             dtype="bf16", interleaved=False, wide=True),
        # a 64K-token prefill: grouped heads, slices of one projection, all channels rotated
        dict(name="qk_norm_rope_fwd_64k", op="qkn_fwd", total=65536, hq=32, hk=8, d=128, rot=128,
             dtype="bf16", interleaved=False, wide=True),
        # the backward pass over an odd number of tokens, half the channels rotated in pairs
        dict(name="qk_norm_rope_bwd_8191", op="qkn_bwd", total=8191, hq=32, hk=32, d=128, rot=64,
             dtype="bf16", interleaved=True, wide=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["dla_fwd", "dla_fwd", "dla_bwd", "dla_bwd", "dla_step", "qkn_fwd",
                     "qkn_bwd"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "fp32"])
    decay = rng.choice(["head", "token", "token"])
    if op in ("dla_fwd", "dla_bwd"):
        hk = rng.choice([1, 2, 3, 4, 8, 16, 32])
        hv = hk * rng.choice([1, 2, 3, 4, 8] if hk <= 4 else [1, 1, 2] if hk <= 16 else [1])
        most = (65536 if op == "dla_fwd" else 16384) // (1 if dtype == "bf16" else 8)
        total = _log(rng, 1, most)
        return dict(op=op, total=total, n_seq=min(rng.choice([1, 1, 2, 3, 7, 16]), total), hk=hk,
                    hv=hv, dk=rng.choice([128, 128, 64, 96, 40, 33]),
                    dv=rng.choice([128, 128, 64, 112, 72, 31]), dtype=dtype, decay=decay,
                    h0=rng.random() < 0.5,
                    resets=rng.choice([0, 0, 1, 5]) if decay == "token" else 0)
    if op == "dla_step":
        batch = _log(rng, 1, 250)
        hk = rng.choice([2, 4, 8, 16, 32])
        return dict(op=op, batch=batch, slots=batch + rng.randrange(0, 50), hk=hk,
                    hv=hk * rng.choice([1, 2]) if hk < 32 else hk,
                    dk=rng.choice([128, 128, 64, 40]), dv=rng.choice([128, 128, 64, 72]),
                    dtype=dtype, decay=decay)
    hk = rng.choice([1, 2, 4, 8, 16])
    hq = min(32, hk * rng.choice([1, 1, 2, 4, 7]))
    d = rng.choice([128, 128, 64, 80, 100, 256])
    top = (65536 if op == "qkn_fwd" else 8192) * 40 * 128 // ((hq + hk) * d)
    return dict(op=op, total=_log(rng, 1, min(65536, top // (1 if dtype == "bf16" else 2))),
                hq=hq, hk=hk, d=d, rot=rng.choice([d, d, d // 2, d // 4 * 2, 0]), dtype=dtype,
                interleaved=rng.random() < 0.5, wide=rng.random() < 0.5)


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


def prepare(case, seed):
    cpu = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device=DEV).manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=DEV)

    def rand(*shape):
        return torch.rand(shape, generator=gen, device=DEV)

    op, dt = case["op"], DT[case["dtype"]]
    s = {"case": case}
    if op.startswith("dla"):
        hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
        n = case["batch"] if op == "dla_step" else case["total"]
        # queries and keys as a norm over the head's channels leaves them; neighbouring keys
        # alike, as text gives them
        k = randn(n, hk, dk)
        k = k + 0.5 * k.roll(1, 0)
        s["q"] = randn(n, hk, dk).to(dt)
        s["k"] = (k * torch.rsqrt(k.square().mean(-1, keepdim=True) + EPS)).to(dt)
        s["v"] = randn(n, hv, dv).to(dt)
        if case["decay"] == "head":
            # rates spread over the heads, from a memory of one token to one of hundreds
            s["g"] = -torch.exp2(-8 * (torch.arange(hv, device=DEV) + rand(hv)) / hv)
        else:
            # g = -A softplus(x + b): A per head in (0, 16), time steps of 0.001 to 0.1
            a = 16 * rand(hv)
            step = torch.exp(rand(hv) * math.log(100.0) + math.log(0.001))
            s["g"] = -a * F.softplus(0.5 * randn(n, hv) + step + torch.log(-torch.expm1(-step)))
    if op in ("dla_fwd", "dla_bwd"):
        lens = _lengths(case, cpu)
        s["lengths"] = lens
        s["cu"] = torch.tensor([sum(lens[:i]) for i in range(len(lens) + 1)], dtype=torch.int32,
                               device=DEV)
        if case["resets"]:  # a new document starts: nothing of the state is kept
            at = torch.randint(0, n, (case["resets"],), generator=cpu)
            s["g"][at.to(DEV)] = -math.inf
        s["h0"] = randn(len(lens), hv, dk, dv) if case["h0"] else None
    if op == "dla_bwd":
        s["dout"] = randn(n, hv, dv).to(dt)
        s["dhf"] = randn(len(lens), hv, dk, dv) if case["h0"] else None
    if op == "dla_step":
        s["state"] = randn(case["slots"], hv, dk, dv)
        slots = torch.randperm(case["slots"], generator=cpu)[:n].to(torch.int32)
        if n >= 8:  # rows of a padded batch that hold no sequence
            slots[torch.randperm(n, generator=cpu)[:n // 32 + 1]] = -1
        s["slots"] = slots.to(DEV)
    if op.startswith("qkn"):
        n, hq, hk, d, rot = case["total"], case["hq"], case["hk"], case["d"], case["rot"]
        # channels of unequal size, heads of unequal norm; with `wide` q and k are slices of a
        # projection that holds v as well
        qkv = randn(n, hq + hk + (hk if case["wide"] else 0), d)
        qkv = (qkv * torch.exp(0.5 * randn(1, 1, d)) * torch.exp(0.5 * randn(n, 1, 1))).to(dt)
        s["q"], s["k"] = qkv[:, :hq], qkv[:, hq:hq + hk]
        if not case["wide"]:
            s["q"], s["k"] = s["q"].contiguous(), s["k"].contiguous()
        s["wq"], s["wk"] = 1 + 0.2 * randn(d), 1 + 0.2 * randn(d)
        # sequences packed one after the other, the first one continued far into its context
        cut = int(torch.randint(0, n + 1, (1,), generator=cpu))
        far = int(torch.randint(0, 1 << 20, (1,), generator=cpu))
        pos = torch.arange(n) + torch.where(torch.arange(n) < cut, far, -cut)
        s["pos"] = pos.to(DEV, torch.int32)
        i = torch.arange(rot // 2, dtype=torch.float64)
        s["freqs"] = (BASE ** (-2 * i / max(rot, 1))).to(DEV)
        if op == "qkn_bwd":
            s["dyq"], s["dyk"] = randn(n, hq, d).to(dt), randn(n, hk, d).to(dt)
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


def _chunks(s):
    """The inputs by chunks, [B, H, chunks, ...] in 32 bits, and their decays."""
    n, hv, hk = s["v"].shape[0], s["v"].shape[1], s["q"].shape[1]
    idx, ok = _index(s["lengths"])

    def take(x):
        x = x.float()[idx] * ok.view(*ok.shape, 1, 1)
        return x.movedim(3, 1)

    q, k = (take(x.repeat_interleave(hv // hk, 1)) for x in (s["q"], s["k"]))
    v = take(s["v"])
    g = s["g"].expand(n, hv)
    g = torch.where(ok.unsqueeze(1), g[idx].movedim(3, 1), 0.0)
    # d[r, j] = sum of g over (j, r]: summed from j + 1 on, so that -inf gives no inf - inf
    low = torch.ones(CHUNK, CHUNK, device=DEV).tril(-1).bool()
    d = torch.where(low, g.unsqueeze(-1), 0.0).cumsum(-2)
    e = torch.where(low | torch.eye(CHUNK, device=DEV).bool(), torch.exp(d), 0.0)
    head = torch.exp(g.cumsum(-1)).unsqueeze(-1)
    tail = e[..., -1, :].unsqueeze(-1)
    return dict(idx=idx, ok=ok, q=q, k=k, v=v, e=e, low=low, head=head, tail=tail,
                whole=head[..., -1:, :])


def _states(s, t):
    """The state at each chunk's start and the final states."""
    n, hv, dk, dv = len(s["lengths"]), s["v"].shape[1], s["q"].shape[2], s["v"].shape[2]
    st = torch.zeros(n, hv, dk, dv, device=DEV) if s["h0"] is None else s["h0"]
    add = (t["tail"] * t["k"]).mT @ t["v"]
    starts = []
    for c in range(add.shape[2]):  # the chunks of a sequence follow one another
        starts.append(st)
        st = t["whole"][:, :, c] * st + add[:, :, c]
    return torch.stack(starts, 2), st


def _scatter(x, t, like):
    out = torch.empty(like.shape, dtype=like.dtype, device=DEV)
    out[t["idx"][t["ok"]]] = x.movedim(1, 3)[t["ok"]].to(like.dtype)
    return out


def _plain_dla_fwd(s):
    t = _chunks(s)
    starts, final = _states(s, t)
    o = (t["head"] * t["q"]) @ starts + (t["e"] * (t["q"] @ t["k"].mT)) @ t["v"]
    return {"out": _scatter(o * s["q"].shape[2] ** -0.5, t, s["v"]), "h_final": final}


def _plain_dla_bwd(s):
    t = _chunks(s)
    starts, _ = _states(s, t)
    q, k, v, e, low, head, tail = (t[n] for n in ("q", "k", "v", "e", "low", "head", "tail"))
    do = s["dout"].float()[t["idx"]] * t["ok"].view(*t["ok"].shape, 1, 1)
    do = do.movedim(3, 1) * s["q"].shape[2] ** -0.5
    n, hv, dk, dv = starts.shape[0], starts.shape[1], starts.shape[3], starts.shape[4]
    ds = torch.zeros(n, hv, dk, dv, device=DEV) if s["dhf"] is None else s["dhf"]
    add = (head * q).mT @ do
    ends = []
    for c in reversed(range(k.shape[2])):
        ends.append(ds)
        ds = t["whole"][:, :, c] * ds + add[:, :, c]
    ends = torch.stack(ends[::-1], 2)
    qk = q @ k.mT
    w = (do @ v.mT) * e
    dos, vds = head * (do @ starts.mT), tail * (v @ ends.mT)
    dq = dos + w @ k
    dk_ = vds + w.mT @ q
    dv_ = (e * qk).mT @ do + tail * (k @ ends)
    # g_i reaches the first part of dq_r for r >= i, that of dk_r for r < i, and w[r, j] for
    # j < i <= r
    m = torch.where(low, w * qk, 0.0)
    a, b = (q * dos).sum(-1), (k * vds).sum(-1)
    inner = (m.cumsum(-1) - m).flip(-2).cumsum(-2).flip(-2).diagonal(dim1=-2, dim2=-1)
    whole = (t["whole"] * starts * ends).sum((-1, -2)).unsqueeze(-1)
    dg = whole + a.flip(-1).cumsum(-1).flip(-1) + b.cumsum(-1) - b + inner
    group = s["v"].shape[1] // s["q"].shape[1]

    def shared(x):
        return x.unflatten(1, (-1, group)).sum(2)

    every = torch.empty(s["v"].shape[:2], device=DEV)
    dg = _scatter(dg, t, every)
    return {"dq": _scatter(shared(dq), t, s["q"]), "dk": _scatter(shared(dk_), t, s["k"]),
            "dv": _scatter(dv_, t, s["v"]), "dg": dg if s["g"].dim() == 2 else dg.sum(0),
            "dh0": ds}


def _plain_dla_step(s):
    live = s["slots"] >= 0
    at = s["slots"][live].long()
    rep = s["v"].shape[1] // s["q"].shape[1]
    q, k = (x.float()[live].repeat_interleave(rep, 1).unsqueeze(-1) for x in (s["q"], s["k"]))
    g = s["g"].expand(s["v"].shape[:2])[live]
    st = s["state"][at] * torch.exp(g)[..., None, None] + k * s["v"].float()[live].unsqueeze(-2)
    s["state"][at] = st
    out = torch.zeros_like(s["v"])
    out[live] = ((q.mT @ st).squeeze(-2) * s["q"].shape[2] ** -0.5).to(out.dtype)
    return {"out": out, "state": s["state"]}


def _turn(x, cos, sin, interleaved):
    """The first 2 R channels of x [N, H, d] turned pair by pair; cos, sin [N, R]."""
    r = cos.shape[1]
    cos, sin = cos.unsqueeze(1), sin.unsqueeze(1)
    y = x.clone()
    a, b = (slice(0, 2 * r, 2), slice(1, 2 * r, 2)) if interleaved else \
        (slice(0, r), slice(r, 2 * r))
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def _angles(s):
    a = s["pos"].double().unsqueeze(1) * s["freqs"]
    return torch.cos(a).float(), torch.sin(a).float()


def _plain_qkn_fwd(s):
    cos, sin = _angles(s)
    out = {}
    for name in "qk":
        x = s[name].float()
        y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * s["w" + name]
        out[name] = _turn(y, cos, sin, s["case"]["interleaved"]).to(s[name].dtype)
    return out


def _plain_qkn_bwd(s):
    cos, sin = _angles(s)
    out = {}
    for name in "qk":
        x, w = s[name].float(), s["w" + name]
        dn = _turn(s["dy" + name].float(), cos, -sin, s["case"]["interleaved"])
        rstd = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
        n = x * rstd
        t = dn * w
        out["d" + name] = (rstd * (t - n * (t * n).mean(-1, keepdim=True))).to(s[name].dtype)
        out["dw" + name] = (dn * n).sum((0, 1))
    return out


PLAIN = {"dla_fwd": _plain_dla_fwd, "dla_bwd": _plain_dla_bwd, "dla_step": _plain_dla_step,
         "qkn_fwd": _plain_qkn_fwd, "qkn_bwd": _plain_qkn_bwd}


# ---------------------------------------------------------------- the package's operators

def _own(s):
    import chunked_linear_attention_kda_gb300 as kda
    case = s["case"]
    if case["op"] == "dla_fwd":
        out, final = kda.dla_chunk_fwd(s["q"], s["k"], s["v"], s["g"], s["h0"], s["cu"])
        return {"out": out, "h_final": final}
    if case["op"] == "dla_bwd":
        grads = kda.dla_chunk_bwd(s["q"], s["k"], s["v"], s["g"], s["h0"], s["cu"], s["dout"],
                                  s["dhf"])
        return dict(zip(("dq", "dk", "dv", "dg", "dh0"), grads))
    if case["op"] == "dla_step":
        out = kda.dla_step(s["q"], s["k"], s["v"], s["g"], s["state"], s["slots"])
        return {"out": out, "state": s["state"]}
    if case["op"] == "qkn_fwd":
        q, k = kda.qk_norm_rope_fwd(s["q"], s["k"], s["wq"], s["wk"], s["pos"], s["freqs"],
                                    eps=EPS, interleaved=case["interleaved"])
        return {"q": q, "k": k}
    grads = kda.qk_norm_rope_bwd(s["dyq"], s["dyk"], s["q"], s["k"], s["wq"], s["wk"], s["pos"],
                                 s["freqs"], eps=EPS, interleaved=case["interleaved"])
    return dict(zip(("dq", "dk", "dwq", "dwk"), grads))


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ---------------------------------------------------------------- what a pass cannot do without

def work(case):
    op, es = case["op"], 2 if case["dtype"] == "bf16" else 4
    if op.startswith("dla"):
        hk, hv, dk, dv = case["hk"], case["hv"], case["dk"], case["dv"]
        n = case["batch"] if op == "dla_step" else case["total"]
        decay = 4 * hv * (n if case["decay"] == "token" else 1)
        tok = n * (2 * hk * dk + hv * dv) * es                # q, k, v
        st = 4 * hv * dk * dv
        outer = 2 * dk * dv * n * hv                          # one product with, or update of, the state
        if op == "dla_step":
            live = n - (n // 32 + 1 if n >= 8 else 0)
            return {"bytes": tok + decay + n * hv * dv * es + 4 * n + 2 * live * st,
                    "flops": 2.5 * outer}
        seqs = case["n_seq"] * st * (2 if case["h0"] else 1)
        if op == "dla_fwd":  # the write, S^T q
            return {"bytes": tok + decay + n * hv * dv * es + seqs, "flops": 2 * outer}
        # the forward's state again, then dS: one product reads S, two read dS, both for dg
        return {"bytes": 2 * (tok + decay) + n * hv * dv * es + seqs * 2, "flops": 6 * outer}
    n = case["total"] * (case["hq"] + case["hk"]) * case["d"]
    small = 4 * case["total"] + 4 * case["rot"] + 8 * case["d"]
    if op == "qkn_fwd":
        return {"bytes": 2 * n * es + small, "flops": 8 * n}
    return {"bytes": 3 * n * es + small + 8 * case["d"], "flops": 16 * n}


# ---------------------------------------------------------------- the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "dla_step":
        return _exact_step(s)
    if case["op"].startswith("dla"):
        # about 60 us a token forward, 400 us with the backward pass
        if max(s["lengths"]) > (70000 if case["op"] == "dla_fwd" else 20000):
            return None
        return _exact_scan(s, case["op"] == "dla_bwd")
    return _exact_qkn(s, case["op"] == "qkn_bwd")


def _exact_step(s):
    state, out = s["state"].double(), torch.zeros(s["v"].shape, dtype=torch.float64, device=DEV)
    rep = s["v"].shape[1] // s["q"].shape[1]
    for b, slot in enumerate(s["slots"].tolist()):
        if slot < 0:
            continue
        k = s["k"][b].double().repeat_interleave(rep, 0)
        q = s["q"][b].double().repeat_interleave(rep, 0)
        g = (s["g"][b] if s["g"].dim() == 2 else s["g"]).double()
        state[slot] = state[slot] * g.exp().view(-1, 1, 1) + \
            torch.einsum("hk,hv->hkv", k, s["v"][b].double())
        out[b] = torch.einsum("hkv,hk->hv", state[slot], q) / math.sqrt(s["q"].shape[2])
    return {"out": out, "state": state}


def _exact_scan(s, backward):
    """Token after token, all sequences side by side; a token past its sequence's end has
    g = 0 and k = 0 and leaves the state alone."""
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

    rates = s["g"].expand(s["v"].shape[:2])
    q, k, v, g = (lay(x) for x in (s["q"], s["k"], s["v"], rates))
    alpha = g.exp()
    c = 1 / math.sqrt(dk)

    def heads(x):  # [B, Hk, dk] -> [B * Hv, 1, dk]
        return x.repeat_interleave(rep, 1).reshape(nb * hv, 1, dk)

    def forward(S, t):
        return torch.baddbmm(S * alpha[t].reshape(-1, 1, 1), heads(k[t]).transpose(1, 2),
                             v[t].reshape(-1, 1, dv))

    S = torch.zeros(nb * hv, dk, dv, dtype=torch.float64, device=DEV) if s["h0"] is None \
        else s["h0"].double().reshape(nb * hv, dk, dv)
    if not backward:
        out = torch.zeros(T, nb, hv, dv, dtype=torch.float64, device=DEV)
        for t in range(T):
            S = forward(S, t)
            out[t] = (c * torch.bmm(heads(q[t]), S)).view(nb, hv, dv)
        return {"out": back(out, s["v"]), "h_final": S.view(nb, hv, dk, dv)}

    block = 64
    marks = []
    for t in range(T):
        if t % block == 0:
            marks.append(S)
        S = forward(S, t)
    do = lay(s["dout"])
    dq, dk_, dv_, dg = (torch.zeros_like(x) for x in (q, k, v, g))
    dS = torch.zeros_like(S) if s["dhf"] is None else s["dhf"].double().reshape(nb * hv, dk, dv)
    for m in reversed(range(len(marks))):
        t0, t1 = m * block, min(T, (m + 1) * block)
        chain = [marks[m]]
        for t in range(t0, t1):
            chain.append(forward(chain[-1], t))
        for t in reversed(range(t0, t1)):
            d, vt = c * do[t].reshape(-1, 1, dv), v[t].reshape(-1, 1, dv)
            al = alpha[t].reshape(-1, 1, 1)
            dq[t] = torch.bmm(chain[t - t0 + 1], d.transpose(1, 2)).view(nb, -1, rep, dk).sum(2)
            dS = torch.baddbmm(dS, heads(q[t]).transpose(1, 2), d)
            dk_[t] = torch.bmm(dS, vt.transpose(1, 2)).view(nb, -1, rep, dk).sum(2)
            dv_[t] = torch.bmm(heads(k[t]), dS).view(nb, hv, dv)
            dS = dS * al
            dg[t] = (dS * chain[t - t0]).sum((1, 2)).view(nb, hv)
    dg = back(dg, rates)
    return {"dq": back(dq, s["q"]), "dk": back(dk_, s["k"]), "dv": back(dv_, s["v"]),
            "dg": dg if s["g"].dim() == 2 else dg.sum(0), "dh0": dS.view(nb, hv, dk, dv)}


def _exact_qkn(s, backward):
    # each pair of channels as a complex number times e^{i angle}
    angle = s["pos"].double().unsqueeze(1) * s["freqs"]
    e = torch.complex(torch.cos(angle), torch.sin(angle)).unsqueeze(1)
    r = s["freqs"].numel()

    def turned(x, by):
        head, rest = x[..., :2 * r], x[..., 2 * r:]
        if s["case"]["interleaved"]:
            z = torch.complex(head[..., 0::2].contiguous(), head[..., 1::2].contiguous()) * by
            head = torch.stack((z.real, z.imag), -1).flatten(-2)
        else:
            z = torch.complex(head[..., :r].contiguous(), head[..., r:].contiguous()) * by
            head = torch.cat((z.real, z.imag), -1)
        return torch.cat((head, rest), -1)

    out = {}
    for name in "qk":
        x, w = s[name].double(), s["w" + name].double()
        ms = (x * x).sum(2, keepdim=True) / x.shape[2] + EPS
        if not backward:
            out[name] = turned(w * x / ms.sqrt(), e)
            continue
        dn = turned(s["dy" + name].double(), e.conj())
        wd = w * dn
        out["d" + name] = wd * ms ** -0.5 - \
            x * ms ** -1.5 * (wd * x).sum(2, keepdim=True) / x.shape[2]
        out["dw" + name] = (dn * x * ms ** -0.5).sum((0, 1))
    return out
