"""The operators around a quantized layer: int8 linear layers, rotary
positions, norms of query and key heads with the rotation in the same pass
and its gradient, and the append to a paged cache.

Binding over the C entry points of ``include/kbit_layer.h``, in the manner of
the package's other functions: checks, output allocation, and forwarding of
addresses, strides and torch's current stream of the inputs' device.  Tensors
may be strided; the last axis has to be contiguous where it is a row of codes,
of a matrix or of a head.
"""

import ctypes as ct

import numpy as np
import torch

from . import KbitError, _buf, _check, _dtype_name, _same_device, lib

__all__ = [
    "quantize_rows_int8", "linear_int8", "linear_int8_dynamic", "rope_frequencies", "rope_table", "rope",
    "qk_norm_rope", "qk_norm_rope_backward", "append_kv_paged",
]

_LAYOUTS = {"half": 0, "interleaved": 1}
_SCALINGS = {None: 0, "linear": 1, "ntk": 2, "yarn": 3}
_INDEX = (torch.int32, torch.int64)


def _call(name, device, *args):
    """One C call on torch's current stream of the device, with it current
    (the library launches on the current device)."""
    fn = getattr(lib(), name)
    stream = torch.cuda.current_stream(device).cuda_stream
    if device.index != torch.cuda.current_device():
        with torch.cuda.device(device):
            status = fn(*args, stream)
    else:
        status = fn(*args, stream)
    if status:
        _check(name, status)


def _rows(t, what, dtypes):
    """A 2-D tensor of contiguous, non-overlapping rows on the GPU."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what}: expected a tensor, got {type(t).__name__}")
    if t.dtype not in dtypes or t.dim() != 2:
        raise TypeError(f"{what} must be a 2-D tensor of {' or '.join(str(d) for d in dtypes)}, "
                        f"got {t.dim()}-D {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{what} must live on the GPU")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError(f"{what}: the rows must be contiguous")
    if t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        raise ValueError(f"{what}: the rows overlap")
    return t


def _row_stride(t):
    # a single row may carry any stride
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1)


def _vector(t, what, dtype, count, ref):
    _buf(t, what, dtype, count)
    if not t.is_contiguous():
        raise ValueError(f"{what}: tensor must be contiguous")
    if t.device != ref.device:
        raise ValueError(f"{what} is on {t.device}, the input on {ref.device}")
    return t.data_ptr()


_FLOATS = (torch.float32, torch.float16, torch.bfloat16)


# --------------------------------------------------------------------------
# int8 linear
# --------------------------------------------------------------------------
def _codes_rows(rows, d, device):
    return torch.empty((rows, -(-d // 16) * 16), dtype=torch.int8, device=device)[:, :d]


def quantize_rows_int8(X, codes=None, scale=None):
    """Codes of the rows of X [rows, d] (fp32/fp16/bf16) -> (codes int8
    [rows, d], scale fp32 [rows]); codes * scale[:, None] stands for X.

    A row is a token of an activation or an output channel of a weight.  The
    rows of ``codes`` start at multiples of 16 bytes (its row stride is d
    rounded up to 16), which the product's fast path needs."""
    _rows(X, "X", _FLOATS)
    rows, d = X.shape
    if d < 1:
        raise ValueError("X must have at least one column")
    if codes is None:
        codes = _codes_rows(rows, d, X.device)
    else:
        _rows(codes, "codes", (torch.int8,))
        if codes.shape != X.shape:
            raise ValueError(f"codes: shape {tuple(codes.shape)}, expected {tuple(X.shape)}")
        if rows and (codes.untyped_storage().nbytes() - codes.storage_offset()
                     < (rows - 1) * codes.stride(0) + -(-d // 16) * 16):
            raise ValueError("codes: every row needs room up to the next multiple of 16 bytes")
    if scale is None:
        scale = torch.empty(rows, dtype=torch.float32, device=X.device)
    _same_device(X, codes=codes)
    ldc = codes.stride(0) if rows > 1 else -(-d // 16) * 16
    _call(f"quantize_rows_int8_{_dtype_name(X.dtype)}", X.device, X.data_ptr(), rows, d, _row_stride(X),
          codes.data_ptr(), ldc, _vector(scale, "scale", torch.float32, rows, X))
    return codes, scale


def _product_args(x, w_codes, w_scale, bias, dtype, out, what):
    M, K = x.shape
    _rows(w_codes, "w_codes", (torch.int8,))
    N = w_codes.shape[0]
    if w_codes.shape[1] != K:
        raise ValueError(f"w_codes: rows of {w_codes.shape[1]} codes, {what} has {K}")
    if N < 1 or K < 1:
        raise ValueError("the weight must have at least one row and one column")
    if w_codes.device != x.device:
        raise ValueError(f"w_codes is on {w_codes.device}, the input on {x.device}")
    ws = _vector(w_scale, "w_scale", torch.float32, N, x)
    b = None if bias is None else _vector(bias, "bias", dtype, N, x)
    if out is None:
        out = torch.empty((M, N), dtype=dtype, device=x.device)
    else:
        _rows(out, "out", (dtype,))
        if out.shape != (M, N):
            raise ValueError(f"out: shape {tuple(out.shape)}, expected {(M, N)}")
        _same_device(x, out=out)
    return M, K, N, ws, b, out


def _workspace(need, workspace, name, ref):
    if need < 0:
        raise KbitError(name, -1, "size out of range")
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=ref.device) if need else None
    _vector(workspace, "workspace", torch.uint8, need, ref)
    return workspace


def _space(workspace):
    return (None, 0) if workspace is None else (workspace.data_ptr(), workspace.numel())


def linear_int8(codes, scale, w_codes, w_scale, bias=None, dtype=torch.bfloat16, out=None, workspace=None):
    """out[M, N] = (codes[M, K] @ w_codes[N, K]^T) * scale[:, None] * w_scale + bias.

    codes, w_codes: int8, exact sums; scale, w_scale: fp32, one a row; bias: N
    values of ``dtype`` (fp32/fp16/bf16), the output's type.  The workspace
    (uint8, ``linear_int8_workspace_bytes``) is allocated here unless given."""
    _rows(codes, "codes", (torch.int8,))
    t = _dtype_name(dtype)
    M, K, N, ws, b, out = _product_args(codes, w_codes, w_scale, bias, dtype, out, "codes")
    workspace = _workspace(lib().linear_int8_workspace_bytes(M, N, K), workspace, "linear_int8", codes)
    _call(f"linear_int8_{t}", codes.device, codes.data_ptr(), _vector(scale, "scale", torch.float32, M, codes), M, K,
          _row_stride(codes), w_codes.data_ptr(), ws, N, _row_stride(w_codes), b, out.data_ptr(), _row_stride(out),
          *_space(workspace))
    return out


def linear_int8_dynamic(X, w_codes, w_scale, bias=None, out=None, workspace=None):
    """linear_int8 of X [M, K] (fp32/fp16/bf16) quantized on the way, the
    output in X's type: the values of ``quantize_rows_int8`` followed by
    ``linear_int8``."""
    _rows(X, "X", _FLOATS)
    M, K, N, ws, b, out = _product_args(X, w_codes, w_scale, bias, X.dtype, out, "X")
    workspace = _workspace(lib().linear_int8_dynamic_workspace_bytes(M, N, K), workspace, "linear_int8_dynamic", X)
    if M == 0:
        return out
    _call(f"linear_int8_dynamic_{_dtype_name(X.dtype)}", X.device, X.data_ptr(), M, K, _row_stride(X),
          w_codes.data_ptr(), ws, N, _row_stride(w_codes), b, out.data_ptr(), _row_stride(out), *_space(workspace))
    return out


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
    _check("rope_frequencies", lib().rope_frequencies(
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
    rot = 2 * f.numel()
    if out is None:
        out = torch.empty((max_pos, rot), dtype=torch.float32, device=f.device)
    _call("rope_table", f.device, f.data_ptr(), rot, max_pos, amplitude,
          _vector(out, "out", torch.float32, max_pos * rot, f))
    return out


def _heads(t, what, dtypes=_FLOATS, dim=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what}: expected a tensor, got {type(t).__name__}")
    if t.dtype not in dtypes:
        raise TypeError(f"{what}: element type {t.dtype}, expected {' or '.join(str(d) for d in dtypes)}")
    if t.dim() != 3 and (dim is not None or t.dim() != 4):
        raise ValueError(f"{what} must be [tokens, heads, dim]" + ("" if dim else " or [batch, tokens, heads, dim]"))
    if not t.is_cuda:
        raise ValueError(f"{what} must live on the GPU")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{what}: the elements of a head must be contiguous")
    return t


def _view(t):
    """(address, batch, token and head strides) of [.., tokens, heads, dim]."""
    st = t.stride()
    return (t.data_ptr(), 0, st[0], st[1]) if len(st) == 3 else (t.data_ptr(), st[0], st[1], st[2])


def _out_like(x, out, what):
    if out is None:
        return torch.empty(x.shape, dtype=x.dtype, device=x.device)
    _heads(out, what, (x.dtype,))
    if out.shape != x.shape:
        raise ValueError(f"{what}: shape {tuple(out.shape)}, expected {tuple(x.shape)}")
    if out.device != x.device:
        raise ValueError(f"{what} is on {out.device}, the input on {x.device}")
    return out


def _index(t, what, shape, ref):
    if not isinstance(t, torch.Tensor) or t.dtype not in _INDEX:
        raise TypeError(f"{what} must be an int32 or int64 tensor")
    if t.shape != shape:
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.device != ref.device:
        raise ValueError(f"{what} is on {t.device}, the input on {ref.device}")
    if not t.is_contiguous():
        raise ValueError(f"{what}: tensor must be contiguous")
    return t.data_ptr(), t.element_size()


def _turn(positions, table, layout, x, dim):
    """The arguments of a rotation: positions, table, rot, max_pos, layout."""
    if layout not in _LAYOUTS:
        raise ValueError(f"layout must be 'half' or 'interleaved', got {layout!r}")
    if not isinstance(table, torch.Tensor) or table.dtype != torch.float32 or table.dim() != 2:
        raise TypeError("table must be the 2-D float32 tensor of rope_table")
    max_pos, rot = table.shape
    if rot > dim:
        raise ValueError(f"table rotates {rot} elements, a head has {dim}")
    address = _vector(table, "table", torch.float32, max_pos * rot, x)
    p, nbytes = _index(positions, "positions", x.shape[:-2], x)
    return p, nbytes, address, rot, max_pos, _LAYOUTS[layout]


def rope(x, positions, table, layout="half", inverse=False, out=None):
    """Rotates the first ``table.shape[1]`` elements of every head of x
    ([tokens, heads, dim] or [batch, tokens, heads, dim], fp32/fp16/bf16) by
    its token's position (int32/int64 [tokens] or [batch, tokens]).

    layout: pairs (i, i + rot/2) ("half") or (2i, 2i + 1) ("interleaved").
    ``inverse=True`` is the transposed rotation: the gradient of x from that of
    the output.  ``out`` may be x.  A position outside the table gives NaN."""
    _heads(x, "x")
    turn = _turn(positions, table, layout, x, x.shape[-1])
    out = _out_like(x, out, "out")
    shape = x.shape if x.dim() == 4 else (1, *x.shape)
    _call(f"rope_{_dtype_name(x.dtype)}", x.device, *_view(x), *_view(out), *shape, *turn, int(bool(inverse)))
    return out


def _norm_args(q, k, q_weight, k_weight, eps):
    _heads(q, "q")
    _heads(k, "k", (q.dtype,))
    if k.dim() != q.dim() or k.shape[:-2] != q.shape[:-2] or k.shape[-1] != q.shape[-1]:
        raise ValueError(f"q {tuple(q.shape)} and k {tuple(k.shape)} may differ in their heads only")
    if k.device != q.device:
        raise ValueError(f"k is on {k.device}, the input on {q.device}")
    dim = q.shape[-1]
    wt = q_weight.dtype if isinstance(q_weight, torch.Tensor) else None
    if wt not in (q.dtype, torch.float32):
        raise TypeError(f"q_weight must be a {q.dtype} or float32 tensor")
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if isinstance(w, torch.Tensor) and w.shape != (dim,):
            raise ValueError(f"{name}: shape {tuple(w.shape)}, expected {(dim,)}")
    qw, kw = _vector(q_weight, "q_weight", wt, dim, q), _vector(k_weight, "k_weight", wt, dim, q)
    batch, tokens = (1, q.shape[0]) if q.dim() == 3 else q.shape[:2]
    return (batch, tokens, q.shape[-2], k.shape[-2], dim, qw, kw, int(wt == torch.float32))


def qk_norm_rope(q, k, q_weight, k_weight, positions, table, eps=1e-6, layout="half", q_out=None, k_out=None):
    """RMS norm of every head of q and k ([.., tokens, heads, dim], the same
    tokens) with its weight ([dim], in q's type or fp32), and the rotation of
    ``rope`` in the same pass -> (q_out, k_out), which may be q and k."""
    sizes = _norm_args(q, k, q_weight, k_weight, eps)
    turn = _turn(positions, table, layout, q, q.shape[-1])
    q_out, k_out = _out_like(q, q_out, "q_out"), _out_like(k, k_out, "k_out")
    _call(f"qk_norm_rope_{_dtype_name(q.dtype)}", q.device, *_view(q), *_view(k), *_view(q_out), *_view(k_out),
          *sizes, eps, *turn)
    return q_out, k_out


def qk_norm_rope_backward(dq_out, dk_out, q, k, q_weight, k_weight, positions, table, eps=1e-6, layout="half",
                          dq=None, dk=None, workspace=None):
    """Gradients of ``qk_norm_rope`` from those of its outputs and its inputs
    -> (dq, dk, dq_weight, dk_weight): the weights' in fp32, summed over
    tokens and heads in a fixed order.  dq may be dq_out, dk may be dk_out."""
    sizes = _norm_args(q, k, q_weight, k_weight, eps)
    turn = _turn(positions, table, layout, q, q.shape[-1])
    for name, g, x in (("dq_out", dq_out, q), ("dk_out", dk_out, k)):
        _heads(g, name, (q.dtype,))
        if g.shape != x.shape or g.device != x.device:
            raise ValueError(f"{name}: {tuple(g.shape)} on {g.device}, expected {tuple(x.shape)} on {x.device}")
    dq, dk = _out_like(q, dq, "dq"), _out_like(k, dk, "dk")
    dim = q.shape[-1]
    dw = torch.empty((2, dim), dtype=torch.float32, device=q.device)
    workspace = _workspace(lib().qk_norm_rope_backward_workspace_bytes(dim), workspace, "qk_norm_rope_backward", q)
    _call(f"qk_norm_rope_backward_{_dtype_name(q.dtype)}", q.device, *_view(dq_out), *_view(dk_out), *_view(q),
          *_view(k), *_view(dq), *_view(dk), *sizes, dw.data_ptr(), dw.data_ptr() + 4 * dim, eps, *turn,
          *_space(workspace))
    return dq, dk, dw[0], dw[1]


def append_kv_paged(k, v, slots, k_cache, v_cache, positions=None, table=None, layout="half"):
    """Writes the tokens' keys (rotated by ``positions`` and ``table`` if
    given, else as they are) and values to the slots of a paged cache.

    k [tokens, heads, dim], v [tokens, heads, v_dim]; k_cache [pages,
    page_size, heads, dim], v_cache likewise (a transposed view of [pages,
    heads, page_size, dim] is as good); slots int32/int64 [tokens], slot =
    page * page_size + place, distinct; a slot below 0 or beyond the cache
    writes nothing.  Returns (k_cache, v_cache)."""
    _heads(k, "k", dim=3)
    _heads(v, "v", (k.dtype,), dim=3)
    if v.shape[:2] != k.shape[:2]:
        raise ValueError(f"k {tuple(k.shape)} and v {tuple(v.shape)} differ in tokens or heads")
    tokens, heads, dim = k.shape
    v_dim = v.shape[2]
    for name, c, d in (("k_cache", k_cache, dim), ("v_cache", v_cache, v_dim)):
        _heads(c, name, (k.dtype,))
        if c.dim() != 4 or c.shape[2:] != (heads, d) or c.shape[:2] != k_cache.shape[:2]:
            raise ValueError(f"{name}: shape {tuple(c.shape)}, expected [pages, page_size, {heads}, {d}]")
    _same_device(k, v=v, k_cache=k_cache, v_cache=v_cache)
    pages, page_size = k_cache.shape[:2]
    slot = _index(slots, "slots", (tokens,), k)
    if (positions is None) != (table is None):
        raise TypeError("give both positions and table, or neither")
    turn = (None, 0, None, 0, 0, 0) if table is None else _turn(positions, table, layout, k, dim)
    sk, sv, ck, cv = k.stride(), v.stride(), k_cache.stride(), v_cache.stride()
    _call(f"append_kv_paged_{_dtype_name(k.dtype)}", k.device, k.data_ptr(), sk[0], sk[1], v.data_ptr(), sv[0], sv[1],
          tokens, heads, dim, v_dim, *slot, k_cache.data_ptr(), *ck[:3], v_cache.data_ptr(), *cv[:3], pages,
          page_size, *turn)
    return k_cache, v_cache
