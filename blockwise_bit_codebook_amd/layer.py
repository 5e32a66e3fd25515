"""The operators around a quantized layer: int8 linear layers, rotary
positions, norms of query and key heads with the rotation in the same pass
and its gradient, and the append to a paged cache.

Their signatures and documentation; the checks, output allocation and calls of
the C entry points (``include/kbit_layer.h``) are in ``_layer``
(``csrc/layer_bind.cpp``), whose host time is a fraction of what they cost
here.  Calls run on torch's current stream of the inputs' device.  Tensors
may be strided; the last axis has to be contiguous where it is a row of codes,
of a matrix or of a head.  A given output may be the input where that is said;
one that overlaps itself or another operand's heads or rows is refused (the
caches of ``append_kv_paged`` apart, whose slots are the caller's).  Nothing is recorded for autograd: gradients are
calls of their own (``rope(..., inverse=True)``, ``qk_norm_rope_backward``), to
be put into a ``torch.autograd.Function`` where a model is trained that way.
An argument that requires a gradient while gradients are recorded gives a
UserWarning, and given outputs count as modified in place.
If ``_layer`` was not built the import raises: there is no other path.
"""

import ctypes as ct

import numpy as np
import torch

from . import _check, lib

_lib = lib()  # before _layer, which links to the same library

from . import _layer  # noqa: E402

__all__ = [
    "quantize_rows_int8", "linear_int8", "linear_int8_dynamic", "rope_frequencies", "rope_table", "rope",
    "qk_norm_rope", "qk_norm_rope_backward", "append_kv_paged",
]

_SCALINGS = {None: 0, "linear": 1, "ntk": 2, "yarn": 3}


# --------------------------------------------------------------------------
# int8 linear
# --------------------------------------------------------------------------
def quantize_rows_int8(X, codes=None, scale=None):
    """Codes of the rows of X [rows, d] (fp32/fp16/bf16) -> (codes int8
    [rows, d], scale fp32 [rows]); codes * scale[:, None] stands for X.

    A row is a token of an activation or an output channel of a weight.  The
    rows of ``codes`` start at multiples of 16 bytes (its row stride is d
    rounded up to 16), which the product's fast path needs.  Where d is no
    multiple of 128, given ``codes`` whose rows start at multiples of 128 bytes
    make products of many rows 10 to 25% faster (a step of 128 codes is one
    cache line then, not parts of two) and those of a few rows up to 10% slower
    (more bytes)."""
    return _layer.quantize_rows_int8(X, codes, scale)


def linear_int8(codes, scale, w_codes, w_scale, bias=None, dtype=torch.bfloat16, out=None, workspace=None):
    """out[M, N] = (codes[M, K] @ w_codes[N, K]^T) * scale[:, None] * w_scale + bias.

    codes, w_codes: int8, exact sums; scale: fp32, one a row (it may be longer,
    like the one ``quantize_rows_int8`` was given); w_scale: N fp32 values;
    bias: N values of ``dtype`` (fp32/fp16/bf16), the output's type.  The workspace
    (uint8, ``lib().linear_int8_workspace_bytes(M, N, K)`` bytes, which serve any
    fewer rows as well) is allocated here unless given."""
    return _layer.linear_int8(codes, scale, w_codes, w_scale, bias, dtype, out, workspace)


def linear_int8_dynamic(X, w_codes, w_scale, bias=None, out=None, workspace=None):
    """linear_int8 of X [M, K] (fp32/fp16/bf16) quantized on the way, the
    output in X's type: the values of ``quantize_rows_int8`` followed by
    ``linear_int8``.  workspace: as there, of
    ``lib().linear_int8_dynamic_workspace_bytes(M, N, K)`` bytes."""
    return _layer.linear_int8_dynamic(X, w_codes, w_scale, bias, out, workspace)


# --------------------------------------------------------------------------
# rotary positions
# --------------------------------------------------------------------------
def rope_frequencies(rot, base=10000.0, scaling=None, factor=1.0, original_length=0, slow_turns=1.0,
                     fast_turns=32.0):
    """(frequencies fp64 [rot / 2] as a numpy array, amplitude) of ``rot``
    rotated elements.  ``scaling`` for contexts ``factor`` times longer than
    trained: None, "linear" (positions interpolated), "ntk" (a larger base) or
    "yarn" (by the pairs' turns over ``original_length``)."""
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be one of {list(_SCALINGS)}, got {scaling!r}")
    freq = np.zeros(max(int(rot) // 2, 1), dtype=np.float64)
    amplitude = ct.c_double()
    _check("rope_frequencies", _lib.rope_frequencies(
        rot, base, _SCALINGS[scaling], factor, original_length, slow_turns, fast_turns,
        freq.ctypes.data_as(ct.c_void_p), ct.byref(amplitude)))
    return freq, amplitude.value


def rope_table(freq, max_pos, amplitude=1.0, device="cuda", out=None):
    """Cosines and sines of positions 0 .. max_pos - 1 for ``rope`` and the
    operators that rotate: fp32 [max_pos, rot], cosines then sines.  freq: the
    rot / 2 frequencies (array or tensor); made once and kept."""
    f = torch.as_tensor(freq, dtype=torch.float64).to(device).contiguous()
    if f.dim() != 1 or f.numel() < 1:
        raise ValueError("freq must hold the rot / 2 frequencies")
    if not f.is_cuda:
        raise ValueError("device must be a GPU")
    rot = 2 * f.numel()
    if out is None:
        out = torch.empty((max_pos, rot), dtype=torch.float32, device=f.device)
    if out.dtype != torch.float32 or out.shape != (max_pos, rot) or not out.is_contiguous() or out.device != f.device:
        raise ValueError(f"out must be a contiguous float32 tensor of shape {(max_pos, rot)} on {f.device}")
    with torch.cuda.device(f.device):
        _check("rope_table", _lib.rope_table(f.data_ptr(), rot, max_pos, amplitude, out.data_ptr(),
                                             torch.cuda.current_stream(f.device).cuda_stream))
    if not out.is_inference():
        torch.autograd.graph.increment_version(out)
    return out


def rope(x, positions, table, layout="half", inverse=False, out=None):
    """Rotates the first ``table.shape[1]`` elements of every head of x
    ([tokens, heads, dim] or [batch, tokens, heads, dim], fp32/fp16/bf16) by
    its token's position (int32/int64 [tokens] or [batch, tokens]).

    layout: pairs (i, i + rot/2) ("half") or (2i, 2i + 1) ("interleaved").
    ``inverse=True`` is the transposed rotation: the gradient of x from that of
    the output (with an amplitude a, R^T R = a^2).  ``out`` may be x.  A position
    outside the table gives NaN.  More than 65535 batches only where they follow
    one another in memory like the tokens."""
    return _layer.rope(x, positions, table, layout, inverse, out)


# --------------------------------------------------------------------------
# norms of queries and keys
# --------------------------------------------------------------------------
def qk_norm_rope(q, k, q_weight, k_weight, positions, table, eps=1e-6, layout="half", q_out=None, k_out=None):
    """RMS norm of every head of q and k ([.., tokens, heads, dim], the same
    tokens) with its weight ([dim], in q's type or fp32), and the rotation of
    ``rope`` in the same pass -> (q_out, k_out), which may be q and k."""
    return _layer.qk_norm_rope(q, k, q_weight, k_weight, positions, table, eps, layout, q_out, k_out)


def qk_norm_rope_backward(dq_out, dk_out, q, k, q_weight, k_weight, positions, table, eps=1e-6, layout="half",
                          dq=None, dk=None, workspace=None):
    """Gradients of ``qk_norm_rope`` from those of its outputs and its inputs
    -> (dq, dk, dq_weight, dk_weight): the weights' in fp32, summed over
    tokens and heads in a fixed order.  dq may be dq_out, dk may be dk_out."""
    return _layer.qk_norm_rope_backward(dq_out, dk_out, q, k, q_weight, k_weight, positions, table, eps, layout, dq,
                                        dk, workspace)


# --------------------------------------------------------------------------
# paged cache
# --------------------------------------------------------------------------
def append_kv_paged(k, v, slots, k_cache, v_cache, positions=None, table=None, layout="half"):
    """Writes the tokens' keys (rotated by ``positions`` and ``table`` if
    given, else as they are) and values to the slots of a paged cache.

    k [tokens, heads, dim], v [tokens, heads, v_dim]; k_cache [pages,
    page_size, heads, dim], v_cache likewise (a transposed view of [pages,
    heads, page_size, dim] is as good); slots int32/int64 [tokens], slot =
    page * page_size + place, distinct; a slot below 0 or beyond the cache
    writes nothing.  Returns (k_cache, v_cache)."""
    return _layer.append_kv_paged(k, v, slots, k_cache, v_cache, positions, table, layout)
