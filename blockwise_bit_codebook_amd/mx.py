"""Microscaled 4-bit (MXFP4) linear layers, forward and backward, and the layer
norm in front of them.

Their signatures and documentation; the checks, output allocation and calls of
the C entry points (``include/kbit_mx.h``) are in ``_layer``
(``csrc/mx_bind.cpp``).  What ``layer.py`` says of its operators holds here:
calls run on torch's current stream of the inputs' device; rows may be
strided, their elements have to be contiguous; outputs that overlap themselves
or an operand are refused where not said otherwise, and so is a workspace that
shares what a call uses of it with the call's tensors; nothing is recorded for
autograd, gradients are calls of their own, an argument that requires one
gives a UserWarning, and given outputs count as modified in place.

MXFP4: blocks of 32 neighbouring values of a row share a power of two, 2^e with
e = max(floor(log2(max |x|)) - 2, -127), kept as the byte e + 127; a code is x /
2^e rounded to the nearest of 0, 1/2, 1, 3/2, 2, 3, 4, 6 (ties to the even
code, at most 6) with a sign.  A block with a NaN or an infinity has the byte
255 (NaN) and codes 0.  ``codes`` are uint8 [rows, 16 ceil(d / 32)], two codes a
byte, the first in the low half, whole blocks with codes 0 past d; its rows
start at multiples of 16 bytes.  ``scales`` are uint8 [rows, ceil(d / 32)].

A layer is trained like this (x, weight, dout: values; a transposed view is
quantized without a copy)::

    w = quantize_mxfp4(weight)
    out = linear_mxfp4_dynamic(x, *w, bias=bias)
    dx, dweight, dbias = linear_mxfp4_backward(dout, x, weight)
"""

import torch

from . import _check, lib  # noqa: F401

_lib = lib()  # before _layer, which links to the same library

from . import _layer  # noqa: E402

__all__ = ["quantize_mxfp4", "dequantize_mxfp4", "linear_mxfp4", "linear_mxfp4_dynamic", "linear_mxfp4_backward",
           "layer_norm", "layer_norm_backward"]


def quantize_mxfp4(X, codes=None, scales=None):
    """Codes and scales of the rows of X [rows, d] (fp32/fp16/bf16) -> (codes,
    scales).  The rows or the columns of X are contiguous: ``quantize_mxfp4(W.t())``
    quantizes the columns of W without a copy."""
    return _layer.quantize_mxfp4(X, codes, scales)


def dequantize_mxfp4(codes, scales, d, dtype=torch.bfloat16, out=None):
    """The values [rows, d] of codes and scales; exact in the type that was
    quantized (and wherever ``dtype`` holds them)."""
    return _layer.dequantize_mxfp4(codes, scales, d, dtype, out)


def linear_mxfp4(codes, scales, w_codes, w_scales, bias=None, dtype=torch.bfloat16, out=None, workspace=None):
    """out[M, N] = x @ w^T + bias of operands in MXFP4, fp32 sums in a fixed
    order, one rounding to ``dtype`` (fp32/fp16/bf16); bias: N values of ``dtype``.

    Rows of codes and scales are less than 4 MiB apart.  The workspace (uint8,
    ``lib().linear_mxfp4_workspace_bytes(M, N, K)`` bytes, which serve any
    fewer rows as well) is allocated here unless given."""
    return _layer.linear_mxfp4(codes, scales, w_codes, w_scales, bias, dtype, out, workspace)


def linear_mxfp4_dynamic(X, w_codes, w_scales, bias=None, out=None, workspace=None):
    """linear_mxfp4 of X [M, K] (fp32/fp16/bf16) quantized on the way, the output
    in X's type; a few tokens in one launch.  K is at most 2^23 - 256 for more than
    one row.  workspace: as there, of
    ``lib().linear_mxfp4_dynamic_workspace_bytes(M, N, K)`` bytes."""
    return _layer.linear_mxfp4_dynamic(X, w_codes, w_scales, bias, out, workspace)


def linear_mxfp4_backward(dout, X, weight, input_grad=True, weight_grad=True, bias_grad=True, dX=None, dweight=None,
                          workspace=None):
    """Gradients of out = X @ weight^T + bias from dout [M, N], X [M, K] and weight
    [N, K] (values of one type) -> (dX in that type, dweight fp32, dbias fp32),
    None for those that are not asked for.

    dX = dout @ weight and dweight = dout^T @ X with both operands quantized to
    MXFP4 along the axis that is summed over (N, then M, at most 2^23 - 256 of
    either); dbias sums dout itself.  workspace:
    ``lib().linear_mxfp4_backward_workspace_bytes(M, N, K)`` bytes."""
    return _layer.linear_mxfp4_backward(dout, X, weight, input_grad, weight_grad, bias_grad, dX, dweight, workspace)


def layer_norm(x, weight, bias=None, eps=1e-5, out=None):
    """(x - mean) / sqrt(var + eps) * weight + bias of the rows of x [rows, d]
    (fp32/fp16/bf16), fp32 inside; weight and bias: d values in x's type or fp32.
    ``out`` may be x."""
    return _layer.layer_norm(x, weight, bias, eps, out)


def layer_norm_backward(dout, x, weight, eps=1e-5, dx=None, workspace=None):
    """Gradients of ``layer_norm`` from that of its output and its input -> (dx in
    x's type, dweight fp32, dbias fp32), the latter summed over rows in a fixed
    order.  dx may be dout.  workspace:
    ``lib().layer_norm_backward_workspace_bytes(rows, d)`` bytes."""
    return _layer.layer_norm_backward(dout, x, weight, eps, dx, workspace)
