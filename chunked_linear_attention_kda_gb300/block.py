"""The operators of a block around the gated delta rule with one decay per head: the
recurrence itself (chunked forward, one-token step over a pool of states), the residual
norm before a block and the gated norm after the recurrence, with their backward passes.

Like the rest of the package a thin binding of the C ABI in ``include/kda.h``: metadata
checks, output and workspace allocation through torch, raw pointers and the current
stream. Inputs are torch CUDA tensors; q, k, v and the norms' activations may be slices of
a wider tensor (any stride between tokens, a token's row contiguous), everything else is
contiguous. The tensors' device has to be the current one. There is no CPU path. The calls
record nothing for autograd, whatever their inputs require: a gradient is a call of its own, and
``examples/gated_delta_block.py`` has the autograd functions that join the two.
"""
from __future__ import annotations

import functools

import torch

import chunked_linear_attention_kda_gb300 as _kda

_CODE = {torch.float32: 0, torch.bfloat16: 1}
_F32, _I32 = torch.float32, torch.int32
ACTIVATIONS = {"sigmoid": 0, "silu": 1}

# The checks below run on every call, in front of kernels of a few microseconds: they read a
# tensor's attributes once, compare device indexes, and take the raw stream handle.
_stream = torch._C._cuda_getCurrentRawStream
_current = torch._C._cuda_getDevice


def _start(t, what):
    """The library and the stream of ``t``'s device for a call on ``t``."""
    if not t.is_cuda:
        raise ValueError(f"{what} runs on CUDA tensors only (there is no CPU path)")
    if t.dtype not in _CODE:
        raise ValueError(f"{what}: activations must be bfloat16 or float32, got {t.dtype}")
    dev = t.get_device()
    if _current() != dev:  # kernels go to the current device, whatever stream they are given
        raise ValueError(f"{what}: the tensors are on cuda:{dev}, the current device is cuda:{_current()} "
                         f"(call it under torch.cuda.device)")
    return _kda._lib or _kda.load_library(), _stream(dev), dev


def _refuse(name, t, shape, dtype, dev):
    raise ValueError(f"{name} must be {dtype} with shape {tuple(shape)} on cuda:{dev}, got {t.dtype} "
                     f"{tuple(t.shape)} on {t.device}")


def _rows(name, t, shape, dtype, dev):
    """The distance between tokens of ``t`` ([tokens, ...], a token's row contiguous)."""
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev:
        _refuse(name, t, shape, dtype, dev)
    width = shape[1] if len(shape) == 2 else shape[1] * shape[2]
    if t.is_contiguous():
        return width
    want = 1
    for size, stride in zip(reversed(shape[1:]), reversed(t.stride()[1:])):
        if size != 1 and stride != want:
            raise ValueError(f"{name}: a token's row must be contiguous")
        want *= size
    step = t.stride(0)
    if shape[0] > 1 and step < width:
        raise ValueError(f"{name}: tokens may not overlap or run backwards")
    return step if step > width else width


def _flat(name, t, shape, dtype, dev):
    if t.shape != shape or t.dtype is not dtype or t.get_device() != dev:
        _refuse(name, t, shape, dtype, dev)
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _p(t):
    return None if t is None else t.data_ptr()  # an empty tensor's is 0


def _done(lib, status):
    if status != 0:
        _kda._check(lib, status)


# torch.empty parses its arguments for 1.5 us more than the allocation takes; the entry that
# compiled graphs allocate by takes sizes and strides, on the current device
_strided = getattr(getattr(torch._C._dynamo, "guards", None), "_empty_strided_cuda", None) \
    if hasattr(torch._C, "_dynamo") else None


def _empty(shape, dtype, dev):
    """A contiguous tensor of one to four dimensions on ``dev``, the current device's index."""
    if _strided is None:
        return torch.empty(shape, dtype=dtype, device=torch.device("cuda", dev))
    n = len(shape)  # a plain tuple is asked for, torch.Size is none
    if n == 3:
        a, b, c = shape
        return _strided((a, b, c), (b * c, c, 1), dtype)
    if n == 2:
        a, b = shape
        return _strided((a, b), (b, 1), dtype)
    if n == 1:
        return _strided((shape[0],), (1,), dtype)
    a, b, c, d = shape
    return _strided((a, b, c, d), (b * c * d, c * d, d, 1), dtype)


@functools.lru_cache(maxsize=1024)
def _need(what, *sizes):
    """What a workspace size function says of these sizes."""
    return getattr(_kda._lib or _kda.load_library(), what)(*sizes)


def _workspace(given, dev, what, *sizes):
    """The caller's workspace, or a new one of the bytes that the size function ``what`` says of
    ``sizes``. Whether the caller's is large enough and aligned the library checks."""
    if given is None:
        return _empty((_need(what, *sizes),), torch.uint8, dev)
    if given.get_device() != dev or not given.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{dev}")
    return given


def _gdr_inputs(q, k, v, g, beta, dev):
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q and k must be [N, H_k, d_k], v [N, H, d_v] (packed, token-major)")
    shape = q.shape
    n, hk, dk = shape
    _, h, dv = v.shape
    if hk == 0 or h % hk != 0:
        raise ValueError(f"v's {h} heads must be a multiple of q's {hk}")
    dtype = q.dtype
    # the usual call: everything as it should be, without a function call for each tensor
    if (k.shape == shape and v.shape[0] == n and k.dtype is dtype and v.dtype is dtype and
            g.dtype is _F32 and beta.dtype is _F32 and g.shape == (n, h) and beta.shape == (n, h) and
            k.get_device() == dev and v.get_device() == dev and g.get_device() == dev and
            beta.get_device() == dev and q.is_contiguous() and k.is_contiguous() and
            v.is_contiguous() and g.is_contiguous() and beta.is_contiguous()):
        return n, hk, h, dk, dv, (hk * dk, hk * dk, h * dv)
    strides = (_rows("q", q, shape, dtype, dev), _rows("k", k, shape, dtype, dev),
               _rows("v", v, (n, h, dv), dtype, dev))
    _flat("g", g, (n, h), _F32, dev)
    _flat("beta", beta, (n, h), _F32, dev)
    return n, hk, h, dk, dv, strides


def _sequences(q, dev, n, h, dk, dv, h0, cu_seqlens):
    if cu_seqlens is None:
        # formed on the device: a list would be copied from pageable memory, which a graph cannot capture
        cu_seqlens = torch.arange(2, dtype=torch.int32, device=q.device).mul_(n)
    n_seq = cu_seqlens.numel() - 1
    if n_seq < 0:
        raise ValueError("cu_seqlens needs at least one entry")
    _flat("cu_seqlens", cu_seqlens, (n_seq + 1,), _I32, dev)
    if h0 is not None:
        _flat("h0", h0, (n_seq, h, dk, dv), _F32, dev)
    return n_seq, cu_seqlens


def gdr_chunk_fwd(q, k, v, g, beta, h0=None, cu_seqlens=None, *, out=None, h_final=None,
                  output_final_state=True, workspace=None):
    """Chunked forward of the gated delta rule with one log-decay ``g`` per token and head
    through ``kda_gdr_chunk_fwd``. ``q, k`` [N, H_k, d_k], ``v`` [N, H, d_v] (H a multiple of
    H_k; bf16 or fp32), ``g, beta`` [N, H] fp32, ``h0`` [n_seq, H, d_k, d_v] fp32 or None,
    ``cu_seqlens`` int32 [n_seq + 1] (None: one sequence). Returns ``(out, h_final)``, the
    latter None when ``output_final_state`` is False."""
    lib, stream, dev = _start(q, "gdr_chunk_fwd")
    n, hk, h, dk, dv, strides = _gdr_inputs(q, k, v, g, beta, dev)
    n_seq, cu_seqlens = _sequences(q, dev, n, h, dk, dv, h0, cu_seqlens)
    if out is None:
        out = _empty((n, h, dv), q.dtype, dev)
    else:
        _flat("out", out, (n, h, dv), q.dtype, dev)
    if h_final is not None:
        _flat("h_final", h_final, (n_seq, h, dk, dv), _F32, dev)
    elif output_final_state:
        h_final = _empty((n_seq, h, dk, dv), torch.float32, dev)
    code = _CODE[q.dtype]
    workspace = _workspace(workspace, dev, "kda_gdr_chunk_fwd_workspace_bytes", n, n_seq, hk, h, dk, dv, code)
    _done(lib, lib.kda_gdr_chunk_fwd(
        _p(q), _p(k), _p(v), *strides, _p(g), _p(beta), _p(h0), _p(cu_seqlens), _p(out),
        _p(h_final), _p(workspace), workspace.numel() * workspace.element_size(), n, n_seq, hk,
        h, dk, dv, code, stream))
    return out, h_final


def gdr_chunk_bwd(q, k, v, g, beta, h0, cu_seqlens, dout, dh_final=None, *, want_dh0=True,
                  workspace=None):
    """Backward of ``gdr_chunk_fwd`` through ``kda_gdr_chunk_bwd``: the gradients of ``<dout,
    out> + <dh_final, h_final>``. Returns ``(dq, dk, dv, dg, dbeta, dh0)`` (``dh0`` None unless
    ``want_dh0``); ``dq`` and ``dk`` are summed over the value heads of a key head. What a sequence
    is packed with changes its gradients within their accuracy: bf16 calls below 8192 (token, head)
    pairs carry more bits than larger ones, and the order of some sums follows the call's sizes."""
    lib, stream, dev = _start(q, "gdr_chunk_bwd")
    n, hk, h, dk, dv, strides = _gdr_inputs(q, k, v, g, beta, dev)
    n_seq, cu_seqlens = _sequences(q, dev, n, h, dk, dv, h0, cu_seqlens)
    _flat("dout", dout, (n, h, dv), q.dtype, dev)
    if dh_final is not None:
        _flat("dh_final", dh_final, (n_seq, h, dk, dv), _F32, dev)
    grads = (_empty((n, hk, dk), q.dtype, dev),
             _empty((n, hk, dk), q.dtype, dev),
             _empty((n, h, dv), q.dtype, dev),
             _empty((n, h), torch.float32, dev),
             _empty((n, h), torch.float32, dev),
             _empty((n_seq, h, dk, dv), torch.float32, dev)
             if want_dh0 else None)
    code = _CODE[q.dtype]
    workspace = _workspace(workspace, dev, "kda_gdr_chunk_bwd_workspace_bytes", n, n_seq, hk, h, dk, dv, code)
    _done(lib, lib.kda_gdr_chunk_bwd(
        _p(q), _p(k), _p(v), *strides, _p(g), _p(beta), _p(h0), _p(cu_seqlens), _p(dout),
        _p(dh_final), *[_p(t) for t in grads], _p(workspace),
        workspace.numel() * workspace.element_size(), n, n_seq, hk, h, dk, dv, code, stream))
    return grads


def gdr_step(q, k, v, g, beta, state, slots=None, *, out=None):
    """One token per row through ``kda_gdr_step``: row b updates ``state[slots[b]]`` in place
    (``state`` [n_slots, H, d_k, d_v] fp32; ``slots`` int32 [B], None: row b has state b). A
    slot outside the pool marks a padded row: its output is 0. The other tensors as for
    ``gdr_chunk_fwd`` with B tokens. Returns ``out`` [B, H, d_v]."""
    lib, stream, dev = _start(q, "gdr_step")
    n, hk, h, dk, dv, strides = _gdr_inputs(q, k, v, g, beta, dev)
    _flat("state", state, (state.shape[0], h, dk, dv), _F32, dev)
    if slots is not None:
        _flat("slots", slots, (n,), _I32, dev)
    if out is None:
        out = _empty((n, h, dv), q.dtype, dev)
    else:
        _flat("out", out, (n, h, dv), q.dtype, dev)
    status = lib.kda_gdr_step(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), *strides, g.data_ptr(), beta.data_ptr(),
        state.data_ptr(), None if slots is None else slots.data_ptr(), out.data_ptr(), n,
        state.shape[0], hk, h, dk, dv, _CODE[q.dtype], stream)
    if status:
        _kda._check(lib, status)
    return out


def residual_norm_fwd(x, weight, residual=None, scale=None, *, eps=1e-6, out=None,
                      residual_out=None):
    """``r = residual + scale * x`` and ``y = weight * r / sqrt(mean(r^2) + eps)`` through
    ``kda_residual_norm_fwd``: ``x, residual`` [N, d] bf16 or fp32, ``weight, scale`` [d] fp32.
    Returns ``(y, r)``; with neither residual nor scale ``r`` is ``x`` itself."""
    lib, stream, dev = _start(x, "residual_norm_fwd")
    if x.dim() != 2:
        raise ValueError("x must be [N, d]")
    shape, dtype = x.shape, x.dtype
    n, d = shape
    xs = _rows("x", x, shape, dtype, dev)
    _flat("weight", weight, (d,), _F32, dev)
    if scale is not None:
        _flat("scale", scale, (d,), _F32, dev)
    rs = 0 if residual is None else _rows("residual", residual, shape, dtype, dev)
    same = residual is None and scale is None and residual_out is None
    if residual_out is not None:
        _flat("residual_out", residual_out, shape, dtype, dev)
    elif not same:
        residual_out = _empty(shape, dtype, dev)
    if out is None:
        out = _empty(shape, dtype, dev)
    else:
        _flat("out", out, shape, dtype, dev)
    status = lib.kda_residual_norm_fwd(
        x.data_ptr(), xs, None if residual is None else residual.data_ptr(), rs,
        None if scale is None else scale.data_ptr(), weight.data_ptr(),
        None if residual_out is None else residual_out.data_ptr(), out.data_ptr(), n, d, eps,
        _CODE[dtype], stream)
    if status:
        _kda._check(lib, status)
    return out, (x if same else residual_out)


def residual_norm_bwd(dy, r, weight, dr=None, x=None, scale=None, *, eps=1e-6, workspace=None):
    """Gradients of ``residual_norm_fwd`` through ``kda_residual_norm_bwd`` from its ``r``:
    ``dy`` the gradient of y, ``dr`` the one that reaches r from elsewhere (None: zero), ``x``
    needed with a ``scale`` only. Returns ``(dx, dresidual, dweight, dscale)``; without a scale
    ``dx`` is ``dresidual`` and ``dscale`` None."""
    lib, stream, dev = _start(r, "residual_norm_bwd")
    if r.dim() != 2:
        raise ValueError("r must be [N, d]")
    n, d = r.shape
    ss = [_rows("dy", dy, (n, d), r.dtype, dev), 0 if dr is None else _rows("dr", dr, (n, d), r.dtype, dev),
          _rows("r", r, (n, d), r.dtype, dev), 0]
    _flat("weight", weight, (d,), _F32, dev)
    if scale is not None:
        _flat("scale", scale, (d,), _F32, dev)
        if x is None:
            raise ValueError("a scale's gradient needs x")
        ss[3] = _rows("x", x, (n, d), r.dtype, dev)
    dres = _empty((n, d), r.dtype, dev)
    dw = _empty((d,), _F32, dev)
    dx = None if scale is None else _empty((n, d), r.dtype, dev)
    ds = None if scale is None else _empty((d,), _F32, dev)
    workspace = _workspace(workspace, dev, "kda_residual_norm_bwd_workspace_bytes", n, d, scale is not None)
    _done(lib, lib.kda_residual_norm_bwd(
        _p(dy), ss[0], _p(dr), ss[1], _p(r), ss[2], None if scale is None else _p(x), ss[3],
        _p(scale), _p(weight), _p(dx), _p(dres), _p(ds), _p(dw), _p(workspace),
        workspace.numel() * workspace.element_size(), n, d, eps, _CODE[r.dtype], stream))
    return (dres if scale is None else dx), dres, dw, ds


def _gated_inputs(x, gate, weight, activation, dev):
    if x.dim() != 3:
        raise ValueError("x must be [N, H, d]")
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}")
    _flat("weight", weight, (x.shape[2],), _F32, dev)
    return _rows("x", x, x.shape, x.dtype, dev), _rows("gate", gate, x.shape, x.dtype, dev)


def gated_norm_fwd(x, gate, weight, *, eps=1e-6, activation="sigmoid", out=None):
    """``y = weight * x / sqrt(mean(x^2) + eps) * act(gate)`` per token and head through
    ``kda_gated_norm_fwd``: ``x, gate`` [N, H, d] bf16 or fp32, ``weight`` [d] fp32,
    ``activation`` "sigmoid" or "silu". Returns ``y`` [N, H, d]."""
    lib, stream, dev = _start(x, "gated_norm_fwd")
    xs, gs = _gated_inputs(x, gate, weight, activation, dev)
    n, h, d = x.shape
    if out is None:
        out = _empty((n, h, d), x.dtype, dev)
    else:
        _flat("out", out, (n, h, d), x.dtype, dev)
    _done(lib, lib.kda_gated_norm_fwd(_p(x), xs, _p(gate), gs, _p(weight), _p(out), n, h, d, eps,
                                      ACTIVATIONS[activation], _CODE[x.dtype], stream))
    return out


def gated_norm_bwd(dy, x, gate, weight, *, eps=1e-6, activation="sigmoid", workspace=None):
    """Gradients of ``gated_norm_fwd`` through ``kda_gated_norm_bwd``: ``(dx, dgate, dweight)``."""
    lib, stream, dev = _start(x, "gated_norm_bwd")
    xs, gs = _gated_inputs(x, gate, weight, activation, dev)
    ys = _rows("dy", dy, x.shape, x.dtype, dev)
    n, h, d = x.shape
    dx = _empty((n, h, d), x.dtype, dev)
    dgate = _empty((n, h, d), x.dtype, dev)
    dw = _empty((d,), _F32, dev)
    workspace = _workspace(workspace, dev, "kda_gated_norm_bwd_workspace_bytes", n, h, d)
    _done(lib, lib.kda_gated_norm_bwd(
        _p(dy), ys, _p(x), xs, _p(gate), gs, _p(weight), _p(dx), _p(dgate), _p(dw),
        _p(workspace), workspace.numel() * workspace.element_size(), n, h, d, eps,
        ACTIVATIONS[activation], _CODE[x.dtype], stream))
    return dx, dgate, dw
