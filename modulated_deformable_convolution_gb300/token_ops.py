"""Operators on tokens: rotary positions over several axes with the norms of
queries and keys in the same pass, and attention over packed sequences, each
with its gradient.

The functions named ``mdcn_*`` mirror the C entry points of include/mdcn.h one
to one and only marshal arguments; ``rotary``, ``rotary_backward``,
``attention`` and ``attention_backward`` allocate their outputs (and workspace)
with torch and run on the current stream. A tensor is [tokens, heads, head_dim]
with the last index contiguous; the other two may have any positive strides, so
slices of one projection's output serve as they are.

A call on few tokens costs little more on the GPU than its launch, so the
marshalling is kept short: each tensor is looked at once, and the C structs are
packed in one go (``struct``; the layouts are those of ``_abi``'s ctypes
structures, which the tests hold against each other).
"""
from __future__ import annotations

import ctypes
import functools
import struct

import torch

from . import _abi

LAYOUTS = {"half": _abi.MDCN_ROTARY_HALF, "interleaved": _abi.MDCN_ROTARY_INTERLEAVED,
           "blocks": _abi.MDCN_ROTARY_BLOCKS}
_DTYPES = {torch.float32: _abi.MDCN_F32, torch.float16: _abi.MDCN_F16, torch.bfloat16: _abi.MDCN_BF16}
_NONE = (None, 0, 0)

_rotary_attrs = struct.Struct("=iif").pack
_rotary_dims = struct.Struct("=21q").pack
_attention_attrs = struct.Struct("=if").pack
_attention_dims = struct.Struct("=22q").pack


def _new(t):
    """A new contiguous tensor like t (None: none)."""
    return None if t is None else torch.empty_like(t, memory_format=torch.contiguous_format)


def _made(t, shape):
    """What _view answers for a tensor that _new made."""
    return t.data_ptr(), shape[1] * shape[2], shape[2]


def _dtype_of(t):
    try:
        return _DTYPES[t.dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {t.dtype}") from None


def _first(name, t):
    """Shape and device of the tensor that the others have to match."""
    shape = t.shape
    if len(shape) != 3:
        raise ValueError(f"{name} must be [tokens, heads, head_dim]")
    dev = t.get_device()
    if dev < 0:
        raise ValueError(f"{name} must be on a CUDA device")
    return shape, dev


def _view(name, t, dtype, dev, shape):
    """Address, token stride and head stride of one tensor, after its checks."""
    if t.dtype != dtype:
        raise TypeError(f"{name} must have the dtype of the other tensors ({dtype}), not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} must be on the device of the other tensors")
    st, sh, se = t.stride()
    if se != 1 and shape[2] > 1:
        raise ValueError(f"the last index of {name} must be contiguous")
    return t.data_ptr(), st, sh


def _flat(name, t, dtype, shape, dev):
    if t is None:
        return None
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name} must have the shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous and on the device of the other tensors")
    return t.data_ptr()


def _workspace(ws, dev):
    if ws is None:
        return None, 0
    if ws.get_device() != dev or not ws.is_contiguous():
        raise ValueError("workspace must be contiguous and on the device of the other tensors")
    return ws.data_ptr(), ws.numel() * ws.element_size()


@functools.lru_cache(maxsize=None)
def _function(name):
    from . import _check  # the package is loaded by now

    return getattr(_abi.load(), name), _check


def _call(name, dev, stream, *args):
    """The C function on device dev, with the stream (default: the current
    one) as its last argument."""
    fn, check = _function(name)
    if stream is None:
        stream = torch._C._cuda_getCurrentRawStream(dev)
    elif hasattr(stream, "cuda_stream"):
        stream = stream.cuda_stream
    if torch.cuda.current_device() == dev:
        status = fn(*args, stream)
    else:
        with torch.cuda.device(dev):
            status = fn(*args, stream)
    if status:
        check(status, name)


@functools.lru_cache(maxsize=4096)
def _size(name, attrs, dims, dtype):
    """A workspace size: the C function's answer for these attributes and
    sizes, asked once."""
    fn, check = _function(name)
    n = ctypes.c_size_t()
    check(fn(attrs, dims, dtype, ctypes.byref(n)), name)
    return n.value


# ---------------------------------------------------------------- rotary
def rotary_frequencies(sections, base: float = 10000.0, shared: bool = False, device="cuda") -> torch.Tensor:
    """float32 frequencies of the pairs: base ** (-i / n), i counting the n
    pairs of each section anew, or (``shared``) the pairs of all sections."""
    if shared:
        n = sum(sections)
        f = base ** (-torch.arange(n, dtype=torch.float64) / max(n, 1))
    else:
        f = torch.cat([base ** (-torch.arange(n, dtype=torch.float64) / max(n, 1)) for n in sections])
    return f.to(torch.float32).to(device)


def _rotary_problem(q, k, positions, inv_freq, sections, layout, norm, q_weight, k_weight, eps):
    """What both directions check of the tensors that give the shapes (q and
    k, or their outputs' gradients): (dtype, device, attrs, sizes, positions,
    inv_freq, q_weight, k_weight)."""
    shape, dev = _first("q", q)
    dt = q.dtype
    if layout not in LAYOUTS:
        raise ValueError(f"unknown layout {layout!r}")
    axes = len(sections)
    if not 1 <= axes <= 4:
        raise ValueError("1 to 4 sections")
    tokens, _, d = shape
    k_heads = 0
    if k is not None:
        ks = k.shape
        if len(ks) != 3 or ks[0] != tokens or ks[2] != d:
            raise ValueError("k must be [tokens, heads, head_dim] with the tokens and head_dim of q")
        k_heads = ks[1]
    elif k_weight is not None:
        raise ValueError("k_weight without k")
    sizes = (tokens, shape[1], k_heads, d, axes, *sections, *((0,) * (4 - axes)))
    return (dt, dev, _rotary_attrs(LAYOUTS[layout], 1 if norm else 0, eps), sizes,
            _flat("positions", positions, torch.int32, (tokens, axes), dev),
            _flat("inv_freq", inv_freq, torch.float32, (sum(sections),), dev),
            _flat("q_weight", q_weight, dt, (d,), dev), _flat("k_weight", k_weight, dt, (d,), dev))


def _rotary_forward(q, k, positions, inv_freq, sections, q_out, k_out, layout, norm, q_weight, k_weight, eps, stream,
                    made):
    dt, dev, attrs, sizes, pos, freq, qw, kw = _rotary_problem(q, k, positions, inv_freq, sections, layout, norm,
                                                               q_weight, k_weight, eps)
    if (k is None) != (k_out is None):
        raise ValueError("k_out is given exactly when k is")
    shape = q.shape
    qp, q0, q1 = _view("q", q, dt, dev, shape)
    yp, y0, y1 = _made(q_out, shape) if made else _view("q_out", q_out, dt, dev, shape)
    kp, k0, k1, zp, z0, z1 = None, 0, 0, None, 0, 0
    if k is not None:
        shape = k.shape
        kp, k0, k1 = _view("k", k, dt, dev, shape)
        zp, z0, z1 = _made(k_out, shape) if made else _view("k_out", k_out, dt, dev, shape)
    _call("mdcn_rotary_forward", dev, stream, attrs,
          _rotary_dims(*sizes, q0, q1, k0, k1, y0, y1, z0, z1, 0, 0, 0, 0), _dtype_of(q), qp, kp, pos, freq, qw, kw,
          yp, zp)


def mdcn_rotary_forward(q, k, positions, inv_freq, sections, q_out, k_out, layout="half", norm=False, q_weight=None,
                        k_weight=None, eps=1e-6, stream=None) -> None:
    """mdcn_rotary_forward on torch tensors; k and k_out may be None."""
    _rotary_forward(q, k, positions, inv_freq, sections, q_out, k_out, layout, norm, q_weight, k_weight, eps, stream,
                    False)


def rotary(q, k, positions, inv_freq, sections, layout="half", norm=False, q_weight=None, k_weight=None, eps=1e-6,
           q_out=None, k_out=None):
    """Queries q and keys k (or None) of one layer, [tokens, heads, head_dim],
    normed per head (``norm``) and rotated by the int32 positions [tokens,
    axes]: axis a turns sections[a] pairs of elements, with the float32
    frequencies inv_freq. Returns (q_out, k_out), which may be q and k."""
    made = q_out is None and k_out is None
    if q_out is None:
        q_out = _new(q)
    if k_out is None:
        k_out = _new(k)
    _rotary_forward(q, k, positions, inv_freq, sections, q_out, k_out, layout, norm, q_weight, k_weight, eps, None,
                    made)
    return q_out, k_out


def mdcn_rotary_backward(grad_q_out, grad_k_out, q, k, positions, inv_freq, sections, grad_q, grad_k, grad_q_weight,
                         grad_k_weight, workspace, layout="half", norm=False, q_weight=None, k_weight=None, eps=1e-6,
                         stream=None) -> None:
    """mdcn_rotary_backward on torch tensors. q and k may be None without
    ``norm``; the k tensors may all be None; the weights' gradients are given
    exactly when the weights are."""
    dt, dev, attrs, sizes, pos, freq, qw, kw = _rotary_problem(grad_q_out, grad_k_out, positions, inv_freq, sections,
                                                               layout, norm, q_weight, k_weight, eps)
    if norm and (q is None or (k is None) != (grad_k_out is None)):
        raise ValueError("with norm, q and k are needed")
    if (grad_k is None) != (grad_k_out is None):
        raise ValueError("grad_k is given exactly when grad_k_out is")
    if (grad_q_weight is None) != (q_weight is None) or (grad_k_weight is None) != (k_weight is None):
        raise ValueError("a weight's gradient is given exactly when the weight is")
    shape = grad_q_out.shape
    yp, y0, y1 = _view("grad_q_out", grad_q_out, dt, dev, shape)
    gp, g0, g1 = _view("grad_q", grad_q, dt, dev, shape)
    qp, q0, q1 = _view("q", q, dt, dev, shape) if norm else _NONE
    kp, k0, k1 = zp, z0, z1 = hp, h0, h1 = _NONE
    if grad_k_out is not None:
        shape = grad_k_out.shape
        zp, z0, z1 = _view("grad_k_out", grad_k_out, dt, dev, shape)
        hp, h0, h1 = _view("grad_k", grad_k, dt, dev, shape)
        if norm:
            kp, k0, k1 = _view("k", k, dt, dev, shape)
    d = (sizes[3],)
    gqw, gkw = _flat("grad_q_weight", grad_q_weight, dt, d, dev), _flat("grad_k_weight", grad_k_weight, dt, d, dev)
    ws, nbytes = _workspace(workspace, dev)
    _call("mdcn_rotary_backward", dev, stream, attrs,
          _rotary_dims(*sizes, q0, q1, k0, k1, y0, y1, z0, z1, g0, g1, h0, h1), _dtype_of(grad_q_out), yp, zp, qp, kp,
          pos, freq, qw, kw, gp, hp, gqw, gkw, ws, nbytes)


def mdcn_rotary_backward_workspace_size(grad_q_out, grad_k_out, positions, inv_freq, sections, layout="half",
                                        norm=False, eps=1e-6) -> int:
    _, _, attrs, sizes, *_ = _rotary_problem(grad_q_out, grad_k_out, positions, inv_freq, sections, layout, norm, None,
                                             None, eps)
    # sizes do not depend on the strides
    return _size("mdcn_rotary_backward_workspace_size", attrs, _rotary_dims(*sizes, *((1,) * 12)),
                 _dtype_of(grad_q_out))


def rotary_backward(grad_q_out, grad_k_out, q, k, positions, inv_freq, sections, layout="half", norm=False,
                    q_weight=None, k_weight=None, eps=1e-6, workspace=None):
    """Gradients of sum(grad_q_out * q_out) + sum(grad_k_out * k_out) for
    (q_out, k_out) = rotary(q, k, ...). Returns a dict with q, k, q_weight and
    k_weight (None for what was not given)."""
    g = {"q": _new(grad_q_out), "k": _new(grad_k_out), "q_weight": _new(q_weight), "k_weight": _new(k_weight)}
    if q_weight is not None or k_weight is not None:
        need = mdcn_rotary_backward_workspace_size(grad_q_out, grad_k_out, positions, inv_freq, sections, layout, norm,
                                                   eps)
        if workspace is None or workspace.numel() * workspace.element_size() < need:
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


class _Attention:
    """What both directions check and pack of a call's inputs."""

    __slots__ = ("dtype", "dev", "q_shape", "k_shape", "attrs", "sizes", "q", "k", "v", "starts", "code")

    def __init__(self, q, k, v, q_starts, k_starts, k_lengths, causal, scale):
        self.q_shape, self.dev = shape, dev = _first("q", q)
        self.dtype = dt = q.dtype
        self.code = _dtype_of(q)
        self.k_shape = ks = k.shape
        if len(ks) != 3 or ks[2] != shape[2]:
            raise ValueError("k must be [tokens, heads, head_dim] with the head_dim of q")
        self.q = _view("q", q, dt, dev, shape)
        self.k = _view("k", k, dt, dev, ks)
        self.v = _view("v", v, dt, dev, ks)
        n = q_starts.shape
        if len(n) != 1 or n[0] < 1:
            raise ValueError("q_starts must be [sequences + 1]")
        batch = n[0] - 1
        self.starts = (_flat("q_starts", q_starts, torch.int32, n, dev),
                       _flat("k_starts", k_starts, torch.int32, n, dev),
                       _flat("k_lengths", k_lengths, torch.int32, (batch,), dev))
        self.attrs = _attention_attrs(1 if causal else 0, shape[2] ** -0.5 if scale is None else scale)
        self.sizes = (batch, shape[0], ks[0], shape[1], ks[1], shape[2])

    def like_q(self, name, t):
        return _view(name, t, self.dtype, self.dev, self.q_shape)

    def like_k(self, name, t):
        return _view(name, t, self.dtype, self.dev, self.k_shape)

    def lse(self, t):
        return _flat("lse", t, torch.float32, (self.q_shape[1], self.q_shape[0]), self.dev)

    def dims(self, out, g=_NONE, gq=_NONE, gk=_NONE, gv=_NONE):
        q, k, v = self.q, self.k, self.v
        return _attention_dims(*self.sizes, q[1], q[2], k[1], k[2], v[1], v[2], out[1], out[2], g[1], g[2], gq[1],
                               gq[2], gk[1], gk[2], gv[1], gv[2])


def mdcn_attention_workspace_size(q, k, v, out, q_starts, k_starts, k_lengths=None, causal=False, scale=None) -> int:
    p = _Attention(q, k, v, q_starts, k_starts, k_lengths, causal, scale)
    return _size("mdcn_attention_workspace_size", p.attrs, p.dims(p.like_q("out", out)), p.code)


def _forward(p, dims, out, lse, workspace, stream):
    ws, nbytes = _workspace(workspace, p.dev)
    _call("mdcn_attention_forward", p.dev, stream, p.attrs, dims, p.code, p.q[0], p.k[0], p.v[0], *p.starts, out[0],
          p.lse(lse), ws, nbytes)


def mdcn_attention_forward(q, k, v, q_starts, k_starts, out, lse, workspace, k_lengths=None, causal=False, scale=None,
                           stream=None) -> None:
    """mdcn_attention_forward on torch tensors (scale None: head_dim ** -0.5)."""
    p = _Attention(q, k, v, q_starts, k_starts, k_lengths, causal, scale)
    o = p.like_q("out", out)
    _forward(p, p.dims(o), o, lse, workspace, stream)


def attention(q, k, v, q_starts, k_starts, k_lengths=None, causal=False, scale=None, out=None, lse=None,
              workspace=None):
    """Attention over packed sequences: q [q_tokens, q_heads, head_dim], k and
    v [k_tokens, k_heads, head_dim] with k_heads dividing q_heads; sequence b
    holds the queries q_starts[b] .. q_starts[b + 1] and the keys k_starts[b] ..
    k_starts[b + 1], or the first k_lengths[b] of them. ``causal``: the last
    query sees every key, each one before it one key less. Returns (out, lse):
    the attended values, like q, and float32 [q_heads, q_tokens], the log of
    the sum of exp(scale * q . k)."""
    p = _Attention(q, k, v, q_starts, k_starts, k_lengths, causal, scale)
    shape = p.q_shape
    if out is None:
        out = _new(q)
        o = _made(out, shape)
    else:
        o = p.like_q("out", out)
    if lse is None:
        lse = torch.empty((shape[1], shape[0]), dtype=torch.float32, device=q.device)
    dims = p.dims(o)
    need = _size("mdcn_attention_workspace_size", p.attrs, dims, p.code)
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    _forward(p, dims, o, lse, workspace, None)
    return out, lse


def _backward_dims(p, grad_out, out, grad_q, grad_k, grad_v):
    o, g = p.like_q("out", out), p.like_q("grad_out", grad_out)
    gq, gk, gv = p.like_q("grad_q", grad_q), p.like_k("grad_k", grad_k), p.like_k("grad_v", grad_v)
    return p.dims(o, g, gq, gk, gv), (g[0], p.q[0], p.k[0], p.v[0], o[0]), (gq[0], gk[0], gv[0])


def mdcn_attention_backward_workspace_size(grad_out, q, k, v, out, lse, q_starts, k_starts, grad_q, grad_k, grad_v,
                                           k_lengths=None, causal=False, scale=None) -> int:
    p = _Attention(q, k, v, q_starts, k_starts, k_lengths, causal, scale)
    dims, _, _ = _backward_dims(p, grad_out, out, grad_q, grad_k, grad_v)
    return _size("mdcn_attention_backward_workspace_size", p.attrs, dims, p.code)


def _backward(p, dims, inputs, lse, outputs, workspace, stream):
    ws, nbytes = _workspace(workspace, p.dev)
    _call("mdcn_attention_backward", p.dev, stream, p.attrs, dims, p.code, *inputs, p.lse(lse), *p.starts, *outputs,
          ws, nbytes)


def mdcn_attention_backward(grad_out, q, k, v, out, lse, q_starts, k_starts, grad_q, grad_k, grad_v, workspace,
                            k_lengths=None, causal=False, scale=None, stream=None) -> None:
    """mdcn_attention_backward on torch tensors."""
    p = _Attention(q, k, v, q_starts, k_starts, k_lengths, causal, scale)
    dims, inputs, outputs = _backward_dims(p, grad_out, out, grad_q, grad_k, grad_v)
    _backward(p, dims, inputs, lse, outputs, workspace, stream)


def attention_backward(grad_out, q, k, v, out, lse, q_starts, k_starts, k_lengths=None, causal=False, scale=None,
                       workspace=None):
    """Gradients of sum(grad_out * out) for (out, lse) = attention(q, k, v,
    ...), as a dict with q, k and v."""
    p = _Attention(q, k, v, q_starts, k_starts, k_lengths, causal, scale)
    g = {"q": _new(q), "k": _new(k), "v": _new(v)}
    dims, inputs, outputs = _backward_dims(p, grad_out, out, g["q"], g["k"], g["v"])
    need = _size("mdcn_attention_backward_workspace_size", p.attrs, dims, p.code)
    if workspace is None or workspace.numel() * workspace.element_size() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    _backward(p, dims, inputs, lse, outputs, workspace, None)
    return g
