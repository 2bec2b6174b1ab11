"""Operators on tokens: rotary positions over several axes with the norms of
queries and keys in the same pass, and attention over packed sequences, each
with its gradient.

The functions named ``mdcn_*`` mirror the C entry points of include/mdcn.h one
to one; ``rotary``, ``rotary_backward``, ``attention`` and
``attention_backward`` allocate their outputs (and workspace) with torch and run
on the current stream. A tensor is [tokens, heads, head_dim] with the last index
contiguous; the other two may have any positive strides, so slices of one
projection's output serve as they are. The marshalling itself is in C++
(csrc/mdcn_token_binding.cpp): a call on few tokens costs little more on the GPU
than its launch.
"""
from __future__ import annotations

import ctypes
import functools
import importlib.util
import os

import torch

from . import _abi

LAYOUTS = {"half": _abi.MDCN_ROTARY_HALF, "interleaved": _abi.MDCN_ROTARY_INTERLEAVED,
           "blocks": _abi.MDCN_ROTARY_BLOCKS}
BINDING_PATH = os.path.join(_abi.HERE, "_token_binding.so")


@functools.lru_cache(maxsize=None)
def _native():
    """The binding, with the library's entry points. Raises if it is not
    built: there is no fallback."""
    lib = _abi.load()
    if not os.path.exists(BINDING_PATH):
        raise RuntimeError(f"_token_binding.so not built ({BINDING_PATH}); run modulated_deformable_convolution_gb300.build")
    spec = importlib.util.spec_from_file_location("_token_binding", BINDING_PATH)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    mod.bind(*(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value
               for name in ("mdcn_rotary_forward", "mdcn_rotary_backward", "mdcn_rotary_backward_workspace_size",
                            "mdcn_attention_forward", "mdcn_attention_workspace_size", "mdcn_attention_backward",
                            "mdcn_attention_backward_workspace_size")))
    return mod


def _done(result, name):
    """The outputs, or an MdcnError for the status that came in their place."""
    if type(result) is int:
        from . import MdcnError

        raise MdcnError(result, name)
    return result


def _call(function, args, small, name):
    """function(*args). The C entry points take addresses on 16 bytes; where
    one of the small inputs (the places ``small`` of args), a slice of a longer
    tensor, is not, the call is made with copies of those that are not."""
    result = function(*args)
    if type(result) is int and result == _abi.MDCN_ERR_ALIGN:
        off = [i for i in small if args[i] is not None and args[i].data_ptr() % 16]
        if off:
            args = list(args)
            for i in off:
                args[i] = args[i].clone()
            result = function(*args)
    return _done(result, name)


def _bytes(result, name):
    status, n = result
    if status:
        _done(status, name)
    return n


def _layout(name):
    try:
        return LAYOUTS[name]
    except KeyError:
        raise ValueError(f"unknown layout {name!r}") from None


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


def mdcn_rotary_forward(q, k, positions, inv_freq, sections, q_out, k_out, layout="half", norm=False, q_weight=None,
                        k_weight=None, eps=1e-6, stream=None) -> None:
    """mdcn_rotary_forward on torch tensors; k and k_out may be None."""
    if q_out is None or (k is None) != (k_out is None):
        raise ValueError("an output is given exactly when its input is")
    _done(_native().rotary_forward(q, k, positions, inv_freq, sections, q_out, k_out, _layout(layout), norm, q_weight,
                                   k_weight, eps, stream), "mdcn_rotary_forward")


def rotary(q, k, positions, inv_freq, sections, layout="half", norm=False, q_weight=None, k_weight=None, eps=1e-6,
           q_out=None, k_out=None):
    """Queries q and keys k (or None) of one layer, [tokens, heads, head_dim],
    normed per head (``norm``) and rotated by the int32 positions [tokens,
    axes]: axis a turns sections[a] pairs of elements, with the float32
    frequencies inv_freq. Returns (q_out, k_out), which may be q and k.
    positions and the other small inputs may be slices that start anywhere."""
    return _call(_native().rotary_forward, (q, k, positions, inv_freq, sections, q_out, k_out, _layout(layout), norm,
                                            q_weight, k_weight, eps, None), (2, 3, 9, 10), "mdcn_rotary_forward")


def mdcn_rotary_backward(grad_q_out, grad_k_out, q, k, positions, inv_freq, sections, grad_q, grad_k, grad_q_weight,
                         grad_k_weight, workspace, layout="half", norm=False, q_weight=None, k_weight=None, eps=1e-6,
                         stream=None) -> None:
    """mdcn_rotary_backward on torch tensors. q and k may be None without
    ``norm``; the k tensors may all be None; the weights' gradients are given
    exactly when the weights are."""
    if grad_q is None:
        raise ValueError("grad_q is needed")
    _done(_native().rotary_backward(grad_q_out, grad_k_out, q, k, positions, inv_freq, sections, grad_q, grad_k,
                                    grad_q_weight, grad_k_weight, workspace, False, _layout(layout), norm, q_weight,
                                    k_weight, eps, stream), "mdcn_rotary_backward")


def mdcn_rotary_backward_workspace_size(grad_q_out, grad_k_out, positions, inv_freq, sections, layout="half",
                                        norm=False, eps=1e-6) -> int:
    return _bytes(_native().rotary_backward_size(grad_q_out, grad_k_out, positions, inv_freq, sections,
                                                 _layout(layout), norm, eps), "mdcn_rotary_backward_workspace_size")


def rotary_backward(grad_q_out, grad_k_out, q, k, positions, inv_freq, sections, layout="half", norm=False,
                    q_weight=None, k_weight=None, eps=1e-6, workspace=None):
    """Gradients of sum(grad_q_out * q_out) + sum(grad_k_out * k_out) for
    (q_out, k_out) = rotary(q, k, ...). Returns a dict with q, k, q_weight and
    k_weight (None for what was not given)."""
    g = _call(_native().rotary_backward, (grad_q_out, grad_k_out, q, k, positions, inv_freq, sections, None, None, None,
                                          None, workspace, True, _layout(layout), norm, q_weight, k_weight, eps, None),
              (4, 5, 15, 16), "mdcn_rotary_backward")
    return {"q": g[0], "k": g[1], "q_weight": g[2], "k_weight": g[3]}


# ---------------------------------------------------------------- attention
def sequence_starts(lengths, device="cuda") -> torch.Tensor:
    """int32 [sequences + 1]: where each of the packed sequences starts."""
    starts = [0]
    for n in lengths:
        starts.append(starts[-1] + int(n))
    return torch.tensor(starts, dtype=torch.int32, device=device)


def mdcn_attention_workspace_size(q, k, v, out, q_starts, k_starts, k_lengths=None, causal=False, scale=None) -> int:
    return _bytes(_native().attention_size(q, k, v, q_starts, k_starts, k_lengths, causal, scale, out),
                  "mdcn_attention_workspace_size")


def mdcn_attention_forward(q, k, v, q_starts, k_starts, out, lse, workspace, k_lengths=None, causal=False, scale=None,
                           stream=None) -> None:
    """mdcn_attention_forward on torch tensors (scale None: head_dim ** -0.5)."""
    if out is None or lse is None:
        raise ValueError("out and lse are needed")
    _done(_native().attention_forward(q, k, v, q_starts, k_starts, k_lengths, causal, scale, out, lse, workspace, False,
                                      stream), "mdcn_attention_forward")


def attention(q, k, v, q_starts, k_starts, k_lengths=None, causal=False, scale=None, out=None, lse=None,
              workspace=None):
    """Attention over packed sequences: q [q_tokens, q_heads, head_dim], k and
    v [k_tokens, k_heads, head_dim] with k_heads dividing q_heads; sequence b
    holds the queries q_starts[b] .. q_starts[b + 1] and the keys k_starts[b] ..
    k_starts[b + 1], or the first k_lengths[b] of them. ``causal``: the last
    query sees every key, each one before it one key less. Returns (out, lse):
    the attended values, like q, and float32 [q_heads, q_tokens], the log of
    the sum of exp(scale * q . k). Rows of no sequence are not written: where
    ``out`` or ``lse`` is None they hold anything. A kernel's wait that gave up
    is seen with mdcn_query_status on a ``workspace`` of one's own (of
    mdcn_attention_workspace_size bytes or more); a workspace that is None or
    too small is replaced by one that the call drops. Starts and lengths may be
    slices that start anywhere."""
    return _call(_native().attention_forward, (q, k, v, q_starts, k_starts, k_lengths, causal, scale, out, lse, workspace,
                                               True, None), (3, 4, 5), "mdcn_attention_forward")


def mdcn_attention_backward_workspace_size(grad_out, q, k, v, out, lse, q_starts, k_starts, grad_q, grad_k, grad_v,
                                           k_lengths=None, causal=False, scale=None) -> int:
    return _bytes(_native().attention_backward_size(q, k, v, q_starts, k_starts, k_lengths, causal, scale, grad_out,
                                                    out, grad_q, grad_k, grad_v),
                  "mdcn_attention_backward_workspace_size")


def mdcn_attention_backward(grad_out, q, k, v, out, lse, q_starts, k_starts, grad_q, grad_k, grad_v, workspace,
                            k_lengths=None, causal=False, scale=None, stream=None) -> None:
    """mdcn_attention_backward on torch tensors."""
    if grad_q is None or grad_k is None or grad_v is None:
        raise ValueError("grad_q, grad_k and grad_v are needed")
    _done(_native().attention_backward(q, k, v, q_starts, k_starts, k_lengths, causal, scale, grad_out, out, grad_q,
                                       grad_k, grad_v, lse, workspace, False, stream), "mdcn_attention_backward")


def attention_backward(grad_out, q, k, v, out, lse, q_starts, k_starts, k_lengths=None, causal=False, scale=None,
                       workspace=None):
    """Gradients of sum(grad_out * out) for (out, lse) = attention(q, k, v,
    ...), as a dict with q, k and v. Rows of no sequence hold anything; starts,
    lengths and ``workspace`` as for attention, lse may start anywhere."""
    g = _call(_native().attention_backward, (q, k, v, q_starts, k_starts, k_lengths, causal, scale, grad_out, out, None,
                                             None, None, lse, workspace, True, None), (3, 4, 5, 13),
              "mdcn_attention_backward")
    return {"q": g[0], "k": g[1], "v": g[2]}
