"""Refusals of linear attention with one decay per head and of the norm of queries and keys without a
GPU: every bad argument is turned into an error on the host, through the C ABI (fake addresses that no
refused call dereferences) and through the Python binding (CPU tensors, shapes, strides)."""
import pytest
import torch

import chunked_linear_attention_kda_gb300 as kda
from chunked_linear_attention_kda_gb300 import block
from chunked_linear_attention_kda_gb300 import build as kbuild

STEP = 0x1000000


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kda.load_library()


def addresses(names):
    return {n: STEP * (i + 1) for i, n in enumerate(names)}


DLA = addresses("q k v g h0 cu out hf dout dhf dq dk dv dg dh0 state slots".split())
WS = 1 << 40
USUAL = {**DLA, "ws": WS, "ws_bytes": 1 << 30, "qs": 128, "ks": 128, "vs": 256, "gs": 2, "scale": 0.5, "n_tok": 64,
         "n_seq": 1, "hk": 1, "hv": 2, "d_k": 128, "d_v": 128, "dtype": 1}


def fwd(lib, **kw):
    a = {**USUAL, **kw}
    return lib.kda_dla_chunk_fwd(a["q"], a["k"], a["v"], a["qs"], a["ks"], a["vs"], a["g"], a["gs"], a["h0"],
                                 a["cu"], a["scale"], a["out"], a["hf"], a["ws"], a["ws_bytes"], a["n_tok"],
                                 a["n_seq"], a["hk"], a["hv"], a["d_k"], a["d_v"], a["dtype"], None)


def bwd(lib, **kw):
    a = {**USUAL, **kw}
    return lib.kda_dla_chunk_bwd(a["q"], a["k"], a["v"], a["qs"], a["ks"], a["vs"], a["g"], a["gs"], a["h0"],
                                 a["cu"], a["scale"], a["dout"], a["dhf"], a["dq"], a["dk"], a["dv"], a["dg"],
                                 a["dh0"], a["ws"], a["ws_bytes"], a["n_tok"], a["n_seq"], a["hk"], a["hv"],
                                 a["d_k"], a["d_v"], a["dtype"], None)


INF, NAN = float("inf"), float("nan")
SHARED = [(dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(g=None), 1), (dict(cu=None), 1),
          (dict(n_tok=-1), 1), (dict(n_seq=-1), 1), (dict(n_seq=0), 1), (dict(hk=0), 1), (dict(hv=0), 1),
          (dict(hk=2, hv=3), 1), (dict(d_k=0), 1), (dict(d_v=-1), 1), (dict(d_k=129), 2), (dict(d_v=256), 2),
          (dict(dtype=5), 2), (dict(qs=127), 1), (dict(ks=0), 1), (dict(vs=255), 1), (dict(gs=1), 1),
          (dict(gs=-2), 1), (dict(gs=4), 1), (dict(scale=INF), 1), (dict(scale=NAN), 1),
          (dict(q=DLA["q"] + 1), 1), (dict(g=DLA["g"] + 2), 1), (dict(h0=DLA["h0"] + 1), 1), (dict(ws=None), 1),
          (dict(ws_bytes=100), 1), (dict(ws=WS + 8), 1), (dict(n_tok=1 << 31), 2),
          (dict(hv=65536, vs=65536 * 128, gs=65536), 2), (dict(hv=65535, vs=65535 * 128, gs=0, n_tok=1 << 22), 2)]


@pytest.mark.parametrize("kw,status", SHARED + [(dict(out=None), 1), (dict(hf=DLA["hf"] + 2), 1),
                                                (dict(out=DLA["v"]), 1), (dict(hf=DLA["h0"]), 1),
                                                (dict(out=DLA["g"]), 1), (dict(ws=DLA["k"] - 16), 1)])
def test_forward_refuses(lib, kw, status):
    assert fwd(lib, **kw) == status, lib.kda_last_error()
    assert lib.kda_last_error() != b""


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(dout=None), 1), (dict(dq=None), 1), (dict(dk=None), 1), (dict(dv=None), 1), (dict(dq=DLA["dk"]), 1),
    (dict(dv=DLA["dout"]), 1), (dict(dh0=DLA["dhf"]), 1), (dict(dg=DLA["dg"] + 1), 1), (dict(dg=DLA["g"], gs=0), 1)])
def test_backward_refuses(lib, kw, status):
    assert bwd(lib, **kw) == status, lib.kda_last_error()
    assert lib.kda_last_error() != b""


def test_no_sequence_is_nothing_to_do(lib):
    assert fwd(lib, n_tok=0, n_seq=0) == 0 and bwd(lib, n_tok=0, n_seq=0) == 0
    assert lib.kda_last_error() == b""


def test_workspace_sizes(lib):
    f, b = lib.kda_dla_chunk_fwd_workspace_bytes, lib.kda_dla_chunk_bwd_workspace_bytes
    for dtype in (0, 1):
        assert 0 < f(100, 2, 2, 4, 128, 128, dtype) <= f(100000, 2, 2, 4, 128, 128, dtype)
        assert f(100, 2, 2, 4, 128, 128, dtype) < b(100, 2, 2, 4, 128, 128, dtype) < b(10000, 2, 2, 4, 128, 128, dtype)
    for fn in (f, b):
        assert fn(-1, 2, 2, 4, 128, 128, 1) == 0 and fn(10, 1, 1, 1, 129, 64, 1) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(state=None), 1), (dict(out=None), 1), (dict(g=None), 1), (dict(hk=2, hv=3), 1),
    (dict(d_k=200), 2), (dict(dtype=3), 2), (dict(n_rows=-1), 1), (dict(n_rows=9, slots=None), 1), (dict(qs=100), 1),
    (dict(state=DLA["v"]), 1), (dict(out=DLA["k"]), 1), (dict(slots=DLA["slots"] + 1), 1), (dict(gs=3), 1),
    (dict(scale=-INF), 1), (dict(n_rows=1 << 29), 1)])
def test_step_refuses(lib, kw, status):
    a = {**USUAL, "n_rows": 4, "n_slots": 8, **kw}
    got = lib.kda_dla_step(a["q"], a["k"], a["v"], a["qs"], a["ks"], a["vs"], a["g"], a["gs"], a["state"], a["slots"],
                           a["scale"], a["out"], a["n_rows"], a["n_slots"], a["hk"], a["hv"], a["d_k"], a["d_v"],
                           a["dtype"], None)
    assert got == status, lib.kda_last_error()


QK = addresses("q k wq wk pos freqs qo ko dqo dko dq dk dwq dwk".split())


def qk_fwd(lib, **kw):
    a = {**QK, "qs": 512, "ks": 256, "pb": 4, "nf": 32, "n": 8, "hq": 4, "hk": 2, "d": 128, "eps": 1e-6, "dtype": 1, **kw}
    return lib.kda_qk_norm_rope_fwd(a["q"], a["qs"], a["k"], a["ks"], a["wq"], a["wk"], a["pos"], a["pb"], a["freqs"],
                                    a["nf"], a["qo"], a["ko"], a["n"], a["hq"], a["hk"], a["d"], a["eps"], 0,
                                    a["dtype"], None)


def qk_bwd(lib, **kw):
    a = {**QK, "qs": 512, "ks": 256, "dqs": 512, "dks": 256, "pb": 8, "nf": 32, "ws": WS, "ws_bytes": 1 << 24, "n": 8,
         "hq": 4, "hk": 2, "d": 128, "eps": 1e-6, "dtype": 1, **kw}
    return lib.kda_qk_norm_rope_bwd(a["dqo"], a["dqs"], a["dko"], a["dks"], a["q"], a["qs"], a["k"], a["ks"], a["wq"],
                                    a["wk"], a["pos"], a["pb"], a["freqs"], a["nf"], a["dq"], a["dk"], a["dwq"],
                                    a["dwk"], a["ws"], a["ws_bytes"], a["n"], a["hq"], a["hk"], a["d"], a["eps"], 1,
                                    a["dtype"], None)


QK_SHARED = [(dict(q=None), 1), (dict(k=None), 1), (dict(wq=None), 1), (dict(wk=None), 1), (dict(pos=None), 1),
             (dict(freqs=None), 1), (dict(pb=2), 1), (dict(nf=-1), 1), (dict(nf=65), 1), (dict(n=-1), 1),
             (dict(n=1 << 31), 2), (dict(hq=0), 1), (dict(hk=-1), 1), (dict(hq=40000, qs=40000 * 128), 2),
             (dict(d=0), 1), (dict(d=257, qs=4096, ks=4096), 2), (dict(eps=0.0), 1), (dict(eps=NAN), 1),
             (dict(dtype=7), 2), (dict(qs=511), 1), (dict(ks=255), 1), (dict(q=QK["q"] + 1), 1),
             (dict(freqs=QK["freqs"] + 4), 1), (dict(pos=QK["pos"] + 2), 1), (dict(wk=QK["wk"] + 1), 1)]


@pytest.mark.parametrize("kw,status", QK_SHARED + [(dict(qo=None), 1), (dict(ko=None), 1), (dict(qo=QK["q"]), 1),
                                                   (dict(ko=QK["qo"]), 1), (dict(ko=QK["ko"] + 1), 1)])
def test_norm_refuses(lib, kw, status):
    assert qk_fwd(lib, **kw) == status, lib.kda_last_error()


@pytest.mark.parametrize("kw,status", QK_SHARED + [
    (dict(dqo=None), 1), (dict(dko=None), 1), (dict(dq=None), 1), (dict(dwq=None), 1), (dict(dwk=QK["dwk"] + 2), 1),
    (dict(dq=QK["dqo"]), 1), (dict(dks=10), 1), (dict(ws=None), 1), (dict(ws_bytes=64), 1), (dict(ws=WS + 4), 1),
    (dict(pos=QK["pos"] + 4), 1)])
def test_norm_backward_refuses(lib, kw, status):
    assert qk_bwd(lib, **kw) == status, lib.kda_last_error()


def test_no_token_to_norm_is_nothing_to_do(lib):
    assert qk_fwd(lib, n=0) == 0 and qk_fwd(lib, n=0, q=None, qo=None, pos=None) == 0


# ---------------------------------------------------------------- the Python binding

def test_cpu_tensors_are_refused():
    x, w = torch.zeros(4, 2, 8), torch.ones(8)
    for call in (lambda: kda.dla_chunk_fwd(x, x, x, torch.zeros(2)),
                 lambda: kda.dla_chunk_bwd(x, x, x, torch.zeros(2), None, None, x),
                 lambda: kda.dla_step(x, x, x, torch.zeros(2), torch.zeros(4, 2, 8, 8)),
                 lambda: kda.qk_norm_rope_fwd(x, x, w, w), lambda: kda.qk_norm_rope_bwd(x, x, x, x, w, w)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


@pytest.fixture
def on_host(monkeypatch):
    """The checks run on CPU tensors (device index -1) and without a library: a call that passes
    them fails on it."""
    monkeypatch.setattr(block, "_start", lambda t, what: (None, 0, -1))
    monkeypatch.setattr(block, "_empty", lambda shape, dtype, dev: torch.empty(shape, dtype=dtype))


def dla_inputs(n=8, hk=1, hv=2, dk=8, dv=8):
    return dict(q=torch.zeros(n, hk, dk), k=torch.zeros(n, hk, dk), v=torch.zeros(n, hv, dv), g=torch.zeros(n, hv))


BAD_DLA = [dict(v=torch.zeros(7, 2, 8)), dict(k=torch.zeros(8, 1, 7)), dict(v=torch.zeros(8, 2, 8).bfloat16()),
           dict(q=torch.zeros(8, 8)), dict(v=torch.zeros(8, 3, 8), q=torch.zeros(8, 2, 8)), dict(g=torch.zeros(8, 1)),
           dict(g=torch.zeros(1)), dict(g=torch.zeros(())), dict(g=torch.zeros(8, 2).double()),
           dict(g=torch.zeros(2, 8).T), dict(g=torch.zeros(1, 2).expand(8, 2)),
           dict(q=torch.zeros(8, 2, 8)[:, :, ::2].expand(8, 2, 4)), dict(v=torch.zeros(2, 8, 8).transpose(0, 1))]


@pytest.mark.parametrize("bad", BAD_DLA)
def test_linear_attention_checks_its_inputs(on_host, bad):
    a = {**dla_inputs(), **bad}
    cu = torch.tensor([0, 8], dtype=torch.int32)
    for call in (lambda: kda.dla_chunk_fwd(**a, cu_seqlens=cu),
                 lambda: kda.dla_chunk_bwd(**a, h0=None, cu_seqlens=cu, dout=torch.zeros_like(a["v"])),
                 lambda: kda.dla_step(**a, state=torch.zeros(8, 2, 8, 8))):
        with pytest.raises(ValueError):
            call()


@pytest.mark.parametrize("kw", [dict(h0=torch.zeros(1, 2, 8, 7)), dict(cu_seqlens=torch.tensor([0, 8])),
                                dict(out=torch.zeros(8, 2, 7)), dict(h_final=torch.zeros(2, 2, 8, 8)),
                                dict(cu_seqlens=torch.zeros(0, dtype=torch.int32)), dict(workspace=torch.zeros(64)[::2])])
def test_forward_checks_its_tensors(on_host, kw):
    kw = {"cu_seqlens": torch.tensor([0, 8], dtype=torch.int32), "workspace": torch.zeros(16), **kw}
    with pytest.raises(ValueError):
        kda.dla_chunk_fwd(**dla_inputs(), **kw)


@pytest.mark.parametrize("kw", [dict(dout=torch.zeros(8, 2, 7)), dict(dout=torch.zeros(16, 2, 8)[::2]),
                                dict(dh_final=torch.zeros(1, 2, 8)), dict(workspace=torch.zeros(1).expand(99))])
def test_backward_checks_its_tensors(on_host, kw):
    kw = {"h0": None, "cu_seqlens": torch.tensor([0, 8], dtype=torch.int32), "dout": torch.zeros(8, 2, 8),
          "workspace": torch.zeros(16), **kw}
    with pytest.raises(ValueError):
        kda.dla_chunk_bwd(**dla_inputs(), **kw)


@pytest.mark.parametrize("kw", [dict(state=torch.zeros(8, 2, 8, 4)), dict(state=torch.zeros(8, 2, 8, 8).double()),
                                dict(slots=torch.zeros(8)), dict(slots=torch.zeros(7, dtype=torch.int32)),
                                dict(out=torch.zeros(8, 2, 9))])
def test_step_checks_its_tensors(on_host, kw):
    with pytest.raises(ValueError):
        kda.dla_step(**dla_inputs(), **{"state": torch.zeros(8, 2, 8, 8), **kw})


@pytest.mark.parametrize("kw", [
    dict(q=torch.zeros(8, 4)), dict(k=torch.zeros(7, 1, 16)), dict(k=torch.zeros(8, 1, 15)),
    dict(k=torch.zeros(8, 1, 16).bfloat16()), dict(q=torch.zeros(8, 4, 32)[..., ::2]), dict(q_weight=torch.ones(15)),
    dict(k_weight=torch.ones(16).double()), dict(positions=None), dict(freqs=None),
    dict(positions=torch.zeros(7, dtype=torch.int32)), dict(positions=torch.zeros(8)),
    dict(positions=torch.zeros(16, dtype=torch.int64)[::2]), dict(freqs=torch.ones(4)),
    dict(freqs=torch.ones(9, dtype=torch.float64)), dict(freqs=torch.ones(2, 2, dtype=torch.float64)),
    dict(dq_out=torch.zeros(8, 3, 16)), dict(dk_out=torch.zeros(8, 1, 16).bfloat16()),
    dict(workspace=torch.zeros(64)[::2])])
def test_norm_checks_its_tensors(on_host, kw):
    a = {"q": torch.zeros(8, 4, 16), "k": torch.zeros(8, 1, 16), "q_weight": torch.ones(16), "k_weight": torch.ones(16),
         "positions": torch.arange(8), "freqs": torch.ones(4, dtype=torch.float64), **kw}
    grads = {"dq_out": a.pop("dq_out", torch.zeros(8, 4, 16)), "dk_out": a.pop("dk_out", torch.zeros(8, 1, 16)),
             "workspace": a.pop("workspace", torch.zeros(64))}
    if not any(n in kw for n in grads):
        with pytest.raises(ValueError):
            kda.qk_norm_rope_fwd(**a)
    with pytest.raises(ValueError):
        kda.qk_norm_rope_bwd(**grads, **a)


def test_rotary_frequencies():
    f = kda.rotary_frequencies(8, base=100.0, device="cpu")
    assert f.dtype is torch.float64 and torch.allclose(f, torch.tensor([1, 0.1 ** 0.5, 0.1, 0.1 ** 1.5], dtype=torch.float64))
    assert kda.rotary_frequencies(0, device="cpu").shape == (0,)
    with pytest.raises(ValueError):
        kda.rotary_frequencies(7, device="cpu")
