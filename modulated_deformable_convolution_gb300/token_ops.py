"""Operators on tokens: rotary positions over several axes with the norms of
queries and keys in the same pass, and attention over packed sequences, each
with its gradient.

The functions named ``mdcn_*`` mirror the C entry points of include/mdcn.h one
to one and only marshal arguments; ``rotary``, ``rotary_backward``,
``attention`` and ``attention_backward`` allocate their outputs (and workspace)
with torch and run on the current stream. A tensor is [tokens, heads, head_dim]
with the last index contiguous; the other two may have any positive strides, so
slices of one projection's output serve as they are.
"""
from __future__ import annotations

import ctypes

import torch

from . import _abi

LAYOUTS = {"half": _abi.MDCN_ROTARY_HALF, "interleaved": _abi.MDCN_ROTARY_INTERLEAVED,
           "blocks": _abi.MDCN_ROTARY_BLOCKS}


def _base():
    from . import _check, _dtype, _lib, _ptr, _stream

    return _check, _dtype, _lib, _ptr, _stream


def _heads(name, t, like=None):
    if t.dim() != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim]")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device")
    if t.shape[2] > 1 and t.stride(2) != 1:
        raise ValueError(f"the last index of {name} must be contiguous")
    if like is not None:
        if t.dtype != like.dtype:
            raise TypeError(f"{name} must have the dtype of the other tensors ({like.dtype})")
        if t.device != like.device:
            raise ValueError(f"{name} must be on the device of the other tensors ({like.device})")


def _same_shape(name, t, like):
    if t.shape != like.shape:
        raise ValueError(f"{name} must have the shape {tuple(like.shape)}, not {tuple(t.shape)}")


def _flat(name, t, dtype, shape, device):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have the shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous and on {device}")


def _strides(s, t):
    if t is not None:
        s.token, s.head = t.stride(0), t.stride(1)


def _bytes(ws):
    return 0 if ws is None else ws.numel() * ws.element_size()


# ---------------------------------------------------------------- rotary
def rotary_frequencies(sections, base: float = 10000.0, shared: bool = False, device="cuda") -> torch.Tensor:
    """float32 frequencies of the pairs: base ** (-i / n), i counting the n
    pairs of each section anew, or (``shared``) the pairs of all sections."""
    if shared:
        n = sum(sections)
        i, n = torch.arange(n, dtype=torch.float64), max(n, 1)
        f = base ** (-i / n)
    else:
        f = torch.cat([base ** (-torch.arange(n, dtype=torch.float64) / max(n, 1)) for n in sections])
    return f.to(torch.float32).to(device)


def _rotary_problem(q, k, positions, inv_freq, sections, layout, norm, q_weight, k_weight, eps):
    """Checks what the C side cannot see and returns (attrs, dims); q and k
    are the tensors that give shapes and strides."""
    _heads("q", q)
    if k is not None:
        _heads("k", k, q)
        if k.shape[0] != q.shape[0] or k.shape[2] != q.shape[2]:
            raise ValueError("k must have the tokens and head_dim of q")
    if layout not in LAYOUTS:
        raise ValueError(f"unknown layout {layout!r}")
    sections = [int(n) for n in sections]
    if not 1 <= len(sections) <= 4:
        raise ValueError("1 to 4 sections")
    _flat("positions", positions, torch.int32, (q.shape[0], len(sections)), q.device)
    _flat("inv_freq", inv_freq, torch.float32, (sum(sections),), q.device)
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            _flat(name, w, q.dtype, (q.shape[2],), q.device)
    if k is None and k_weight is not None:
        raise ValueError("k_weight without k")
    a = _abi.mdcn_rotary_attrs(LAYOUTS[layout], int(bool(norm)), float(eps))
    d = _abi.mdcn_rotary_dims()
    d.tokens, d.q_heads, d.head_dim = q.shape
    d.k_heads = 0 if k is None else k.shape[1]
    d.axes = len(sections)
    d.sections[: len(sections)] = sections
    return a, d


def mdcn_rotary_forward(q, k, positions, inv_freq, sections, q_out, k_out, layout="half", norm=False, q_weight=None,
                        k_weight=None, eps=1e-6, stream=None) -> None:
    """mdcn_rotary_forward on torch tensors; k and k_out may be None."""
    check, dtype, lib, ptr, stream_of = _base()
    a, d = _rotary_problem(q, k, positions, inv_freq, sections, layout, norm, q_weight, k_weight, eps)
    for name, o, t in (("q_out", q_out, q), ("k_out", k_out, k)):
        if (o is None) != (t is None):
            raise ValueError(f"{name} is given exactly when its input is")
        if o is not None:
            _heads(name, o, q)
            _same_shape(name, o, t)
    _strides(d.q, q)
    _strides(d.k, k)
    _strides(d.q_out, q_out)
    _strides(d.k_out, k_out)
    with torch.cuda.device(q.device):
        check(lib().mdcn_rotary_forward(ctypes.byref(a), ctypes.byref(d), dtype(q), ptr(q), ptr(k), ptr(positions),
                                        ptr(inv_freq), ptr(q_weight), ptr(k_weight), ptr(q_out), ptr(k_out),
                                        stream_of(q.device, stream)), "mdcn_rotary_forward")


def rotary(q, k, positions, inv_freq, sections, layout="half", norm=False, q_weight=None, k_weight=None, eps=1e-6,
           q_out=None, k_out=None):
    """Queries q and keys k (or None) of one layer, [tokens, heads, head_dim],
    normed per head (``norm``) and rotated by the int32 positions [tokens,
    axes]: axis a turns sections[a] pairs of elements, with the float32
    frequencies inv_freq. Returns (q_out, k_out), which may be q and k."""
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    if k_out is None and k is not None:
        k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
    mdcn_rotary_forward(q, k, positions, inv_freq, sections, q_out, k_out, layout, norm, q_weight, k_weight, eps)
    return q_out, k_out


def mdcn_rotary_backward(grad_q_out, grad_k_out, q, k, positions, inv_freq, sections, grad_q, grad_k, grad_q_weight,
                         grad_k_weight, workspace, layout="half", norm=False, q_weight=None, k_weight=None, eps=1e-6,
                         stream=None) -> None:
    """mdcn_rotary_backward on torch tensors. q and k may be None without
    ``norm``; the k tensors may all be None; the weights' gradients are given
    exactly when the weights are."""
    check, dtype, lib, ptr, stream_of = _base()
    a, d = _rotary_problem(grad_q_out, grad_k_out, positions, inv_freq, sections, layout, norm, q_weight, k_weight,
                           eps)
    if norm and (q is None or (k is None) != (grad_k_out is None)):
        raise ValueError("with norm, q and k are needed")
    if (grad_k is None) != (grad_k_out is None):
        raise ValueError("grad_k is given exactly when grad_k_out is")
    for name, t, like in (("q", q if norm else None, grad_q_out), ("k", k if norm else None, grad_k_out),
                          ("grad_q", grad_q, grad_q_out), ("grad_k", grad_k, grad_k_out)):
        if t is not None:
            _heads(name, t, grad_q_out)
            _same_shape(name, t, like)
    for name, t, w in (("grad_q_weight", grad_q_weight, q_weight), ("grad_k_weight", grad_k_weight, k_weight)):
        if (t is None) != (w is None):
            raise ValueError(f"{name} is given exactly when the weight is")
        if t is not None:
            _flat(name, t, grad_q_out.dtype, w.shape, grad_q_out.device)
    if norm:
        _strides(d.q, q)
        _strides(d.k, k)
    _strides(d.q_out, grad_q_out)
    _strides(d.k_out, grad_k_out)
    _strides(d.q_grad, grad_q)
    _strides(d.k_grad, grad_k)
    with torch.cuda.device(grad_q_out.device):
        check(lib().mdcn_rotary_backward(ctypes.byref(a), ctypes.byref(d), dtype(grad_q_out), ptr(grad_q_out),
                                         ptr(grad_k_out), ptr(q if norm else None), ptr(k if norm else None),
                                         ptr(positions), ptr(inv_freq), ptr(q_weight), ptr(k_weight), ptr(grad_q),
                                         ptr(grad_k), ptr(grad_q_weight), ptr(grad_k_weight), ptr(workspace),
                                         _bytes(workspace), stream_of(grad_q_out.device, stream)),
              "mdcn_rotary_backward")


def mdcn_rotary_backward_workspace_size(grad_q_out, grad_k_out, positions, inv_freq, sections, layout="half",
                                        norm=False, eps=1e-6) -> int:
    check, dtype, lib, _, _ = _base()
    a, d = _rotary_problem(grad_q_out, grad_k_out, positions, inv_freq, sections, layout, norm, None, None, eps)
    for s in (d.q, d.k, d.q_out, d.k_out, d.q_grad, d.k_grad):  # sizes do not depend on the strides
        s.token = s.head = 1
    n = ctypes.c_size_t()
    check(lib().mdcn_rotary_backward_workspace_size(ctypes.byref(a), ctypes.byref(d), dtype(grad_q_out),
                                                    ctypes.byref(n)), "mdcn_rotary_backward_workspace_size")
    return int(n.value)


def rotary_backward(grad_q_out, grad_k_out, q, k, positions, inv_freq, sections, layout="half", norm=False,
                    q_weight=None, k_weight=None, eps=1e-6, workspace=None):
    """Gradients of sum(grad_q_out * q_out) + sum(grad_k_out * k_out) for
    (q_out, k_out) = rotary(q, k, ...). Returns a dict with q, k, q_weight and
    k_weight (None for what was not given)."""
    new = lambda t: None if t is None else torch.empty(t.shape, dtype=t.dtype, device=t.device)
    g = {"q": new(grad_q_out), "k": new(grad_k_out), "q_weight": new(q_weight), "k_weight": new(k_weight)}
    if q_weight is not None or k_weight is not None:
        need = mdcn_rotary_backward_workspace_size(grad_q_out, grad_k_out, positions, inv_freq, sections, layout, norm,
                                                   eps)
        if workspace is None or _bytes(workspace) < need:
            workspace = torch.empty(need, dtype=torch.uint8, device=grad_q_out.device)
    mdcn_rotary_backward(grad_q_out, grad_k_out, q, k, positions, inv_freq, sections, g["q"], g["k"], g["q_weight"],
                         g["k_weight"], workspace, layout, norm, q_weight, k_weight, eps)
    return g


# ---------------------------------------------------------------- attention
def sequence_starts(lengths, device="cuda") -> torch.Tensor:
    """int32 [sequences + 1]: where each of the packed sequences starts."""
    starts = [0]
    for n in lengths:
        starts.append(starts[-1] + int(n))
    return torch.tensor(starts, dtype=torch.int32, device=device)


def _attention_problem(q, k, v, q_starts, k_starts, k_lengths, causal, scale):
    _heads("q", q)
    _heads("k", k, q)
    _heads("v", v, q)
    _same_shape("v", v, k)
    if k.shape[2] != q.shape[2]:
        raise ValueError("k must have the head_dim of q")
    if q_starts.dim() != 1 or q_starts.shape[0] < 1:
        raise ValueError("q_starts must be [sequences + 1]")
    _flat("q_starts", q_starts, torch.int32, q_starts.shape, q.device)
    _flat("k_starts", k_starts, torch.int32, q_starts.shape, q.device)
    if k_lengths is not None:
        _flat("k_lengths", k_lengths, torch.int32, (q_starts.shape[0] - 1,), q.device)
    if scale is None:
        scale = q.shape[2] ** -0.5
    a = _abi.mdcn_attention_attrs(int(bool(causal)), float(scale))
    d = _abi.mdcn_attention_dims()
    d.batch = q_starts.shape[0] - 1
    d.q_tokens, d.q_heads, d.head_dim = q.shape
    d.k_tokens, d.k_heads = k.shape[0], k.shape[1]
    _strides(d.q, q)
    _strides(d.k, k)
    _strides(d.v, v)
    return a, d


def _lse(name, lse, q):
    _flat(name, lse, torch.float32, (q.shape[1], q.shape[0]), q.device)


def _attention_size(fn, what, a, d, q):
    check, dtype, lib, _, _ = _base()
    n = ctypes.c_size_t()
    check(getattr(lib(), fn)(ctypes.byref(a), ctypes.byref(d), dtype(q), ctypes.byref(n)), what)
    return int(n.value)


def mdcn_attention_workspace_size(q, k, v, out, q_starts, k_starts, k_lengths=None, causal=False, scale=None) -> int:
    a, d = _attention_problem(q, k, v, q_starts, k_starts, k_lengths, causal, scale)
    _strides(d.out, out)
    return _attention_size("mdcn_attention_workspace_size", "mdcn_attention_workspace_size", a, d, q)


def mdcn_attention_forward(q, k, v, q_starts, k_starts, out, lse, workspace, k_lengths=None, causal=False, scale=None,
                           stream=None) -> None:
    """mdcn_attention_forward on torch tensors (scale None: head_dim ** -0.5)."""
    check, dtype, lib, ptr, stream_of = _base()
    a, d = _attention_problem(q, k, v, q_starts, k_starts, k_lengths, causal, scale)
    _heads("out", out, q)
    _same_shape("out", out, q)
    _lse("lse", lse, q)
    _strides(d.out, out)
    with torch.cuda.device(q.device):
        check(lib().mdcn_attention_forward(ctypes.byref(a), ctypes.byref(d), dtype(q), ptr(q), ptr(k), ptr(v),
                                           ptr(q_starts), ptr(k_starts), ptr(k_lengths), ptr(out), ptr(lse),
                                           ptr(workspace), _bytes(workspace), stream_of(q.device, stream)),
              "mdcn_attention_forward")


def attention(q, k, v, q_starts, k_starts, k_lengths=None, causal=False, scale=None, out=None, lse=None,
              workspace=None):
    """Attention over packed sequences: q [q_tokens, q_heads, head_dim], k and
    v [k_tokens, k_heads, head_dim] with k_heads dividing q_heads; sequence b
    holds the queries q_starts[b] .. q_starts[b + 1] and the keys k_starts[b] ..
    k_starts[b + 1], or the first k_lengths[b] of them. ``causal``: the last
    query sees every key, each one before it one key less. Returns (out, lse):
    the attended values, like q, and float32 [q_heads, q_tokens], the log of
    the sum of exp(scale * q . k)."""
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    if lse is None:
        lse = torch.empty((q.shape[1], q.shape[0]), dtype=torch.float32, device=q.device)
    need = mdcn_attention_workspace_size(q, k, v, out, q_starts, k_starts, k_lengths, causal, scale)
    if workspace is None or _bytes(workspace) < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    mdcn_attention_forward(q, k, v, q_starts, k_starts, out, lse, workspace, k_lengths, causal, scale)
    return out, lse


def _backward_problem(grad_out, q, k, v, out, lse, q_starts, k_starts, k_lengths, causal, scale, grads):
    a, d = _attention_problem(q, k, v, q_starts, k_starts, k_lengths, causal, scale)
    for name, t, like in (("out", out, q), ("grad_out", grad_out, q), ("grad_q", grads["q"], q),
                          ("grad_k", grads["k"], k), ("grad_v", grads["v"], k)):
        _heads(name, t, q)
        _same_shape(name, t, like)
    _lse("lse", lse, q)
    _strides(d.out, out)
    _strides(d.grad_out, grad_out)
    _strides(d.grad_q, grads["q"])
    _strides(d.grad_k, grads["k"])
    _strides(d.grad_v, grads["v"])
    return a, d


def mdcn_attention_backward_workspace_size(grad_out, q, k, v, out, lse, q_starts, k_starts, grad_q, grad_k, grad_v,
                                           k_lengths=None, causal=False, scale=None) -> int:
    a, d = _backward_problem(grad_out, q, k, v, out, lse, q_starts, k_starts, k_lengths, causal, scale,
                             {"q": grad_q, "k": grad_k, "v": grad_v})
    return _attention_size("mdcn_attention_backward_workspace_size", "mdcn_attention_backward_workspace_size", a, d, q)


def mdcn_attention_backward(grad_out, q, k, v, out, lse, q_starts, k_starts, grad_q, grad_k, grad_v, workspace,
                            k_lengths=None, causal=False, scale=None, stream=None) -> None:
    """mdcn_attention_backward on torch tensors."""
    check, dtype, lib, ptr, stream_of = _base()
    a, d = _backward_problem(grad_out, q, k, v, out, lse, q_starts, k_starts, k_lengths, causal, scale,
                             {"q": grad_q, "k": grad_k, "v": grad_v})
    with torch.cuda.device(q.device):
        check(lib().mdcn_attention_backward(ctypes.byref(a), ctypes.byref(d), dtype(q), ptr(grad_out), ptr(q), ptr(k),
                                            ptr(v), ptr(out), ptr(lse), ptr(q_starts), ptr(k_starts), ptr(k_lengths),
                                            ptr(grad_q), ptr(grad_k), ptr(grad_v), ptr(workspace), _bytes(workspace),
                                            stream_of(q.device, stream)), "mdcn_attention_backward")


def attention_backward(grad_out, q, k, v, out, lse, q_starts, k_starts, k_lengths=None, causal=False, scale=None,
                       workspace=None):
    """Gradients of sum(grad_out * out) for (out, lse) = attention(q, k, v,
    ...), as a dict with q, k and v."""
    g = {n: torch.empty(t.shape, dtype=t.dtype, device=t.device) for n, t in (("q", q), ("k", k), ("v", v))}
    need = mdcn_attention_backward_workspace_size(grad_out, q, k, v, out, lse, q_starts, k_starts, g["q"], g["k"],
                                                  g["v"], k_lengths, causal, scale)
    if workspace is None or _bytes(workspace) < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    mdcn_attention_backward(grad_out, q, k, v, out, lse, q_starts, k_starts, g["q"], g["k"], g["v"], workspace,
                            k_lengths, causal, scale)
    return g
