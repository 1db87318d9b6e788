"""Refusals of the block operators without a GPU: every bad argument is turned into an error on
the host, through the C ABI (fake addresses that no refused call dereferences) and through the
Python binding (CPU tensors, shapes, strides)."""
import ctypes

import pytest
import torch

import chunked_linear_attention_kda_gb300 as kda
from chunked_linear_attention_kda_gb300 import build as kbuild

STEP = 0x1000000
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kda.load_library()


def addresses(names):
    return {n: STEP * (i + 1) for i, n in enumerate(names)}


GDR = addresses("q k v g beta h0 cu out hf dout dhf dq dk dv dg db dh0 state slots".split())
WS = 1 << 40


def fwd(lib, **kw):
    a = {**GDR, "ws": WS, "ws_bytes": 1 << 30, "qs": 128, "ks": 128, "vs": 256, "n_tok": 64, "n_seq": 1,
         "hk": 1, "hv": 2, "d_k": 128, "d_v": 128, "dtype": 1, **kw}
    return lib.kda_gdr_chunk_fwd(a["q"], a["k"], a["v"], a["qs"], a["ks"], a["vs"], a["g"], a["beta"], a["h0"],
                                 a["cu"], a["out"], a["hf"], a["ws"], a["ws_bytes"], a["n_tok"], a["n_seq"],
                                 a["hk"], a["hv"], a["d_k"], a["d_v"], a["dtype"], None)


def bwd(lib, **kw):
    a = {**GDR, "ws": WS, "ws_bytes": 1 << 30, "qs": 128, "ks": 128, "vs": 256, "n_tok": 64, "n_seq": 1,
         "hk": 1, "hv": 2, "d_k": 128, "d_v": 128, "dtype": 1, **kw}
    return lib.kda_gdr_chunk_bwd(a["q"], a["k"], a["v"], a["qs"], a["ks"], a["vs"], a["g"], a["beta"], a["h0"],
                                 a["cu"], a["dout"], a["dhf"], a["dq"], a["dk"], a["dv"], a["dg"], a["db"],
                                 a["dh0"], a["ws"], a["ws_bytes"], a["n_tok"], a["n_seq"], a["hk"], a["hv"],
                                 a["d_k"], a["d_v"], a["dtype"], None)


SHARED = [(dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(g=None), 1), (dict(beta=None), 1),
          (dict(cu=None), 1), (dict(n_tok=-1), 1), (dict(n_seq=-1), 1), (dict(n_seq=0), 1), (dict(hk=0), 1),
          (dict(hv=0), 1), (dict(hk=2, hv=3), 1), (dict(d_k=0), 1), (dict(d_v=-1), 1), (dict(d_k=129), 2),
          (dict(d_v=256), 2), (dict(dtype=5), 2), (dict(qs=127), 1), (dict(ks=0), 1), (dict(vs=255), 1),
          (dict(q=GDR["q"] + 1), 1), (dict(g=GDR["g"] + 2), 1), (dict(h0=GDR["h0"] + 1), 1),
          (dict(ws=None), 1), (dict(ws_bytes=100), 1), (dict(ws=WS + 8), 1), (dict(n_tok=1 << 31), 2)]


@pytest.mark.parametrize("kw,status", SHARED + [(dict(out=None), 1), (dict(hf=GDR["hf"] + 2), 1),
                                                (dict(out=GDR["v"]), 1), (dict(hf=GDR["h0"]), 1),
                                                (dict(ws=GDR["k"] - 16), 1)])
def test_forward_refuses(lib, kw, status):
    assert fwd(lib, **kw) == status, lib.kda_last_error()
    assert lib.kda_last_error() != b""


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(dout=None), 1), (dict(dq=None), 1), (dict(dk=None), 1), (dict(dv=None), 1), (dict(dg=None), 1),
    (dict(db=None), 1), (dict(dq=GDR["dk"]), 1), (dict(dv=GDR["dout"]), 1), (dict(dh0=GDR["dhf"]), 1),
    (dict(dg=GDR["dg"] + 1), 1)])
def test_backward_refuses(lib, kw, status):
    assert bwd(lib, **kw) == status, lib.kda_last_error()
    assert lib.kda_last_error() != b""


def test_no_sequence_is_nothing_to_do(lib):
    assert fwd(lib, n_tok=0, n_seq=0) == 0 and bwd(lib, n_tok=0, n_seq=0) == 0
    assert lib.kda_last_error() == b""


def test_workspace_sizes(lib):
    f, b = lib.kda_gdr_chunk_fwd_workspace_bytes, lib.kda_gdr_chunk_bwd_workspace_bytes
    assert 0 < f(100, 2, 2, 4, 128, 128, 1) < f(10000, 2, 2, 4, 128, 128, 1)
    assert f(100, 2, 2, 4, 128, 128, 1) < b(100, 2, 2, 4, 128, 128, 1)
    for bad in ((-1, 1, 1, 1, 8, 8), (1, -1, 1, 1, 8, 8), (1, 1, 0, 1, 8, 8), (1, 1, 1, 0, 8, 8),
                (1, 1, 1, 1, 129, 8), (1, 1, 1, 1, 8, 0)):
        assert f(*bad, 1) == 0 and b(*bad, 1) == 0


def step(lib, **kw):
    a = {**GDR, "qs": 128, "ks": 128, "vs": 256, "rows": 3, "n_slots": 4, "hk": 1, "hv": 2, "d_k": 128,
         "d_v": 128, "dtype": 1, **kw}
    return lib.kda_gdr_step(a["q"], a["k"], a["v"], a["qs"], a["ks"], a["vs"], a["g"], a["beta"], a["state"],
                            a["slots"], a["out"], a["rows"], a["n_slots"], a["hk"], a["hv"], a["d_k"], a["d_v"],
                            a["dtype"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=None), 1), (dict(k=None), 1), (dict(v=None), 1), (dict(g=None), 1), (dict(beta=None), 1),
    (dict(out=None), 1), (dict(state=None), 1), (dict(rows=-1), 1), (dict(n_slots=-1), 1),
    (dict(slots=None, rows=5), 1), (dict(hk=0), 1), (dict(hk=2, hv=3), 1), (dict(d_k=0), 1), (dict(d_v=129), 2),
    (dict(dtype=9), 2), (dict(vs=100), 1), (dict(v=GDR["v"] + 1), 1), (dict(state=GDR["state"] + 2), 1),
    (dict(slots=GDR["slots"] + 1), 1), (dict(out=GDR["q"]), 1), (dict(out=GDR["state"] + 4096), 1),
    (dict(state=GDR["k"] - 4096), 1)])
def test_step_refuses(lib, kw, status):
    assert step(lib, **kw) == status, lib.kda_last_error()


def test_step_of_no_row_is_nothing_to_do(lib):
    assert step(lib, rows=0) == 0


NORM = addresses("x res scale w r y dy dr dx dres ds dw gate dgate".split())


def rn_fwd(lib, **kw):
    a = {**NORM, "xs": 64, "rs": 64, "n": 4, "d": 64, "eps": 1e-6, "dtype": 1, **kw}
    return lib.kda_residual_norm_fwd(a["x"], a["xs"], a["res"], a["rs"], a["scale"], a["w"], a["r"], a["y"], a["n"],
                                     a["d"], a["eps"], a["dtype"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), 1), (dict(w=None), 1), (dict(y=None), 1), (dict(xs=63), 1), (dict(rs=1), 1), (dict(n=-1), 1),
    (dict(d=0), 1), (dict(d=32769, xs=40000, rs=40000), 2), (dict(eps=0.0), 1), (dict(eps=float("nan")), 1),
    (dict(dtype=3), 2), (dict(x=NORM["x"] + 1), 1), (dict(scale=NORM["scale"] + 2), 1), (dict(y=NORM["x"]), 1),
    (dict(r=NORM["y"]), 1)])
def test_residual_norm_refuses(lib, kw, status):
    assert rn_fwd(lib, **kw) == status, lib.kda_last_error()


def rn_bwd(lib, **kw):
    a = {**NORM, "st": 64, "ws": WS, "bytes": 1 << 30, "n": 4, "d": 64, "eps": 1e-6, "dtype": 1, **kw}
    return lib.kda_residual_norm_bwd(a["dy"], a["st"], a["dr"], a["st"], a["r"], a["st"], a["x"], a["st"], a["scale"],
                                     a["w"], a["dx"], a["dres"], a["ds"], a["dw"], a["ws"], a["bytes"], a["n"],
                                     a["d"], a["eps"], a["dtype"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), 1), (dict(r=None), 1), (dict(w=None), 1), (dict(dres=None), 1), (dict(dw=None), 1),
    (dict(x=None), 1), (dict(dx=None), 1), (dict(ds=None), 1), (dict(scale=None), 1),   # ds without a scale
    (dict(st=60), 1), (dict(eps=-1.0), 1), (dict(d=40000, st=40000), 2), (dict(ws=None), 1), (dict(bytes=8), 1),
    (dict(ws=WS + 4), 1), (dict(dres=NORM["dr"]), 1), (dict(dx=NORM["dres"]), 1), (dict(dw=NORM["w"]), 1)])
def test_residual_norm_backward_refuses(lib, kw, status):
    assert rn_bwd(lib, **kw) == status, lib.kda_last_error()


def gn_fwd(lib, **kw):
    a = {**NORM, "xs": 128, "gs": 128, "n": 4, "h": 2, "d": 64, "eps": 1e-6, "act": 0, "dtype": 1, **kw}
    return lib.kda_gated_norm_fwd(a["x"], a["xs"], a["gate"], a["gs"], a["w"], a["y"], a["n"], a["h"], a["d"],
                                  a["eps"], a["act"], a["dtype"], None)


def gn_bwd(lib, **kw):
    a = {**NORM, "st": 128, "ws": WS, "bytes": 1 << 30, "n": 4, "h": 2, "d": 64, "eps": 1e-6, "act": 1, "dtype": 1,
         **kw}
    return lib.kda_gated_norm_bwd(a["dy"], a["st"], a["x"], a["st"], a["gate"], a["st"], a["w"], a["dx"],
                                  a["dgate"], a["dw"], a["ws"], a["bytes"], a["n"], a["h"], a["d"], a["eps"],
                                  a["act"], a["dtype"], None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), 1), (dict(gate=None), 1), (dict(w=None), 1), (dict(y=None), 1), (dict(xs=127), 1),
    (dict(gs=64), 1), (dict(h=0), 1), (dict(d=257, xs=600, gs=600), 2), (dict(act=2), 1), (dict(eps=0.0), 1),
    (dict(dtype=4), 2), (dict(gate=NORM["gate"] + 1), 1), (dict(y=NORM["gate"]), 1),
    (dict(n=1 << 31), 2)])
def test_gated_norm_refuses(lib, kw, status):
    assert gn_fwd(lib, **kw) == status, lib.kda_last_error()


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), 1), (dict(dx=None), 1), (dict(dgate=None), 1), (dict(dw=None), 1), (dict(st=100), 1),
    (dict(act=-1), 1), (dict(ws=None), 1), (dict(bytes=0), 1), (dict(dx=NORM["dy"]), 1),
    (dict(dgate=NORM["dx"]), 1)])
def test_gated_norm_backward_refuses(lib, kw, status):
    assert gn_bwd(lib, **kw) == status, lib.kda_last_error()


def test_norms_of_no_row_are_nothing_to_do(lib):
    assert rn_fwd(lib, n=0) == 0 and gn_fwd(lib, n=0) == 0


def test_binding_refuses_cpu_tensors():
    x, w = torch.zeros(4, 2, 8), torch.ones(8)
    g = torch.zeros(4, 2)
    for call in (lambda: kda.gdr_chunk_fwd(x, x, x, g, g), lambda: kda.gdr_chunk_bwd(x, x, x, g, g, None, None, x),
                 lambda: kda.gdr_step(x, x, x, g, g, torch.zeros(4, 2, 8, 8)),
                 lambda: kda.residual_norm_fwd(x[:, 0], w), lambda: kda.residual_norm_bwd(x[:, 0], x[:, 0], w),
                 lambda: kda.gated_norm_fwd(x, x, w), lambda: kda.gated_norm_bwd(x, x, x, w)):
        with pytest.raises(ValueError, match="CUDA tensors only"):
            call()
