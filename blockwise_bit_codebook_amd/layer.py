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

from . import KbitError, _check, lib

__all__ = [
    "quantize_rows_int8", "linear_int8", "linear_int8_dynamic", "rope_frequencies", "rope_table", "rope",
    "qk_norm_rope", "qk_norm_rope_backward", "append_kv_paged",
]

_LAYOUTS = {"half": 0, "interleaved": 1}
_SCALINGS = {None: 0, "linear": 1, "ntk": 2, "yarn": 3}
_INDEX_BYTES = {torch.int32: 4, torch.int64: 8}
_NAMES = {torch.float32: "fp32", torch.float16: "fp16", torch.bfloat16: "bf16"}
_FLOATS = tuple(_NAMES)
_INT8 = (torch.int8,)
_Tensor = torch.Tensor
_lib = lib()

# The smallest calls last a few microseconds on the GPU, so the host's share
# counts: functions are looked up once per type, and the current stream's
# handle is taken without building a Stream object where torch offers that
# (0.1 against 1.9 us).
_FUNCTIONS = {op: {dt: (getattr(_lib, f"{op}_{n}"), f"{op}_{n}") for dt, n in _NAMES.items()}
              for op in ("quantize_rows_int8", "linear_int8", "linear_int8_dynamic", "rope", "qk_norm_rope",
                         "qk_norm_rope_backward", "append_kv_paged")}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(index):
    return _raw_stream(index) if _raw_stream else torch.cuda.current_stream(index).cuda_stream


def _call(fn, name, device, *args):
    """One C call on torch's current stream of the device, with it current
    (the library launches on the current device)."""
    index = device.index
    if index == torch.cuda.current_device():
        status = fn(*args, _stream(index))
    else:
        with torch.cuda.device(device):
            status = fn(*args, _stream(index))
    if status:
        _check(name, status)


def _rows(t, what, dtypes):
    """(rows, columns, row stride) of a 2-D tensor of contiguous rows that do
    not overlap, on the GPU."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{what}: expected a tensor, got {type(t).__name__}")
    if t.dtype not in dtypes or t.dim() != 2:
        raise TypeError(f"{what} must be a 2-D tensor of {' or '.join(str(d) for d in dtypes)}, "
                        f"got {t.dim()}-D {t.dtype}")
    if not t.is_cuda:
        raise ValueError(f"{what} must live on the GPU")
    n, d = t.shape
    stride, one = t.stride()
    if one != 1 and d > 1:
        raise ValueError(f"{what}: the rows must be contiguous")
    if n <= 1:
        return n, d, max(d, 1)  # a single row may carry any stride
    if stride < d:
        raise ValueError(f"{what}: the rows overlap")
    return n, d, stride


def _vector(t, what, dtype, count, ref):
    """Address of a contiguous tensor of at least count elements on ref's device."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{what}: expected a tensor, got {type(t).__name__}")
    if t.dtype != dtype:
        raise TypeError(f"{what}: element type {t.dtype}, expected {dtype}")
    if t.numel() < count:
        raise ValueError(f"{what}: {t.numel()} elements, at least {count} needed")
    if not t.is_contiguous():
        raise ValueError(f"{what}: tensor must be contiguous")
    _on(t, what, ref)
    return t.data_ptr()


def _on(t, what, ref):
    if t.device != ref.device:
        raise ValueError(f"{what} is on {t.device}, the input on {ref.device}")


# --------------------------------------------------------------------------
# int8 linear
# --------------------------------------------------------------------------
def quantize_rows_int8(X, codes=None, scale=None):
    """Codes of the rows of X [rows, d] (fp32/fp16/bf16) -> (codes int8
    [rows, d], scale fp32 [rows]); codes * scale[:, None] stands for X.

    A row is a token of an activation or an output channel of a weight.  The
    rows of ``codes`` start at multiples of 16 bytes (its row stride is d
    rounded up to 16), which the product's fast path needs."""
    rows, d, ldx = _rows(X, "X", _FLOATS)
    if d < 1:
        raise ValueError("X must have at least one column")
    whole = -(-d // 16) * 16
    if codes is None:
        codes, ldc = torch.empty((rows, whole), dtype=torch.int8, device=X.device)[:, :d], whole
    else:
        _, _, ldc = _rows(codes, "codes", _INT8)
        if codes.shape != X.shape:
            raise ValueError(f"codes: shape {tuple(codes.shape)}, expected {tuple(X.shape)}")
        _on(codes, "codes", X)
        ldc = max(ldc, whole) if rows <= 1 else ldc
        if rows and codes.untyped_storage().nbytes() - codes.storage_offset() < (rows - 1) * ldc + whole:
            raise ValueError("codes: every row needs room up to the next multiple of 16 bytes")
    if scale is None:
        scale = torch.empty(rows, dtype=torch.float32, device=X.device)
    fn, name = _FUNCTIONS["quantize_rows_int8"][X.dtype]
    _call(fn, name, X.device, X.data_ptr(), rows, d, ldx, codes.data_ptr(), ldc,
          _vector(scale, "scale", torch.float32, rows, X))
    return codes, scale


def _weight(x, K, w_codes, w_scale, bias, dtype, out, M, what):
    """(address, row stride, N, scales, bias, out, its row stride)."""
    N, k, ldw = _rows(w_codes, "w_codes", _INT8)
    if k != K:
        raise ValueError(f"w_codes: rows of {k} codes, {what} has {K}")
    if N < 1 or K < 1:
        raise ValueError("the weight must have at least one row and one column")
    _on(w_codes, "w_codes", x)
    ws = _vector(w_scale, "w_scale", torch.float32, N, x)
    b = None if bias is None else _vector(bias, "bias", dtype, N, x)
    if out is None:
        out, ldo = x.new_empty((M, N), dtype=dtype), N
    else:
        _, _, ldo = _rows(out, "out", (dtype,))
        if out.shape != (M, N):
            raise ValueError(f"out: shape {tuple(out.shape)}, expected {(M, N)}")
        _on(out, "out", x)
    return w_codes.data_ptr(), ldw, N, ws, b, out, ldo


def _workspace(need, workspace, name, ref):
    """(tensor, address, bytes)."""
    if need < 0:
        raise KbitError(name, -1, "size out of range")
    if workspace is None:
        if need == 0:
            return None, None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=ref.device)
        return workspace, workspace.data_ptr(), need
    return workspace, _vector(workspace, "workspace", torch.uint8, need, ref), workspace.numel()


def linear_int8(codes, scale, w_codes, w_scale, bias=None, dtype=torch.bfloat16, out=None, workspace=None):
    """out[M, N] = (codes[M, K] @ w_codes[N, K]^T) * scale[:, None] * w_scale + bias.

    codes, w_codes: int8, exact sums; scale, w_scale: fp32, one a row; bias: N
    values of ``dtype`` (fp32/fp16/bf16), the output's type.  The workspace
    (uint8, ``linear_int8_workspace_bytes``) is allocated here unless given."""
    M, K, ldx = _rows(codes, "codes", _INT8)
    if dtype not in _NAMES:
        raise TypeError(f"unsupported element dtype {dtype}")
    w, ldw, N, ws, b, out, ldo = _weight(codes, K, w_codes, w_scale, bias, dtype, out, M, "codes")
    s = _vector(scale, "scale", torch.float32, M, codes)
    keep, space, nbytes = _workspace(_lib.linear_int8_workspace_bytes(M, N, K), workspace, "linear_int8", codes)
    fn, name = _FUNCTIONS["linear_int8"][dtype]
    _call(fn, name, codes.device, codes.data_ptr(), s, M, K, ldx, w, ws, N, ldw, b, out.data_ptr(), ldo, space, nbytes)
    return out


def linear_int8_dynamic(X, w_codes, w_scale, bias=None, out=None, workspace=None):
    """linear_int8 of X [M, K] (fp32/fp16/bf16) quantized on the way, the
    output in X's type: the values of ``quantize_rows_int8`` followed by
    ``linear_int8``."""
    M, K, ldx = _rows(X, "X", _FLOATS)
    w, ldw, N, ws, b, out, ldo = _weight(X, K, w_codes, w_scale, bias, X.dtype, out, M, "X")
    if M == 0:
        return out
    if M <= 8 and w % 16 == 0 and _lib.linear_int8_dynamic_fused(M, N, K, ldw):
        keep, space, nbytes = None, None, 0
    else:
        keep, space, nbytes = _workspace(_lib.linear_int8_dynamic_workspace_bytes(M, N, K), workspace,
                                         "linear_int8_dynamic", X)
    fn, name = _FUNCTIONS["linear_int8_dynamic"][X.dtype]
    _call(fn, name, X.device, X.data_ptr(), M, K, ldx, w, ws, N, ldw, b, out.data_ptr(), ldo, space, nbytes)
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
    _call(_lib.rope_table, "rope_table", f.device, f.data_ptr(), rot, max_pos, amplitude,
          _vector(out, "out", torch.float32, max_pos * rot, f))
    return out


def _heads(t, what, dtypes=_FLOATS):
    """Checks [.., tokens, heads, dim] with contiguous heads on the GPU."""
    if not isinstance(t, _Tensor):
        raise TypeError(f"{what}: expected a tensor, got {type(t).__name__}")
    if t.dtype not in dtypes:
        raise TypeError(f"{what}: element type {t.dtype}, expected {' or '.join(str(d) for d in dtypes)}")
    if not 3 <= t.dim() <= 4:
        raise ValueError(f"{what} must be [tokens, heads, dim] or [batch, tokens, heads, dim]")
    if not t.is_cuda:
        raise ValueError(f"{what} must live on the GPU")
    st = t.stride()
    if st[-1] != 1 and t.shape[-1] > 1:
        raise ValueError(f"{what}: the elements of a head must be contiguous")
    return (t.data_ptr(), 0, st[0], st[1]) if len(st) == 3 else (t.data_ptr(), st[0], st[1], st[2])


def _out_like(x, out, what):
    """(tensor, view) of an output shaped like x, in x's layout if new."""
    if out is None:
        out = torch.empty_like(x)
        if out.stride(-1) != 1 and out.shape[-1] > 1:
            out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        st = out.stride()
        return out, ((out.data_ptr(), 0, st[0], st[1]) if len(st) == 3 else (out.data_ptr(), st[0], st[1], st[2]))
    view = _heads(out, what, (x.dtype,))
    if out.shape != x.shape:
        raise ValueError(f"{what}: shape {tuple(out.shape)}, expected {tuple(x.shape)}")
    _on(out, what, x)
    for n, st in zip(out.shape, out.stride()):
        if st == 0 and n > 1:
            raise ValueError(f"{what}: elements overlap")
    return out, view


def _index(t, what, shape, ref):
    """(address, bytes of an element) of a contiguous index tensor."""
    nbytes = _INDEX_BYTES.get(t.dtype) if isinstance(t, _Tensor) else None
    if nbytes is None:
        raise TypeError(f"{what} must be an int32 or int64 tensor")
    if t.shape != shape:
        raise ValueError(f"{what}: shape {tuple(t.shape)}, expected {tuple(shape)}")
    _on(t, what, ref)
    if not t.is_contiguous():
        raise ValueError(f"{what}: tensor must be contiguous")
    return t.data_ptr(), nbytes


def _turn(positions, table, layout, x, dim):
    """The arguments of a rotation: positions, their bytes, table, rot,
    max_pos, layout."""
    if layout not in _LAYOUTS:
        raise ValueError(f"layout must be 'half' or 'interleaved', got {layout!r}")
    if not isinstance(table, _Tensor) or table.dtype != torch.float32 or table.dim() != 2:
        raise TypeError("table must be the 2-D float32 tensor of rope_table")
    max_pos, rot = table.shape
    if rot > dim:
        raise ValueError(f"table rotates {rot} elements, a head has {dim}")
    if not table.is_contiguous():
        raise ValueError("table: tensor must be contiguous")
    _on(table, "table", x)
    p, nbytes = _index(positions, "positions", x.shape[:-2], x)
    return p, nbytes, table.data_ptr(), rot, max_pos, _LAYOUTS[layout]


def rope(x, positions, table, layout="half", inverse=False, out=None):
    """Rotates the first ``table.shape[1]`` elements of every head of x
    ([tokens, heads, dim] or [batch, tokens, heads, dim], fp32/fp16/bf16) by
    its token's position (int32/int64 [tokens] or [batch, tokens]).

    layout: pairs (i, i + rot/2) ("half") or (2i, 2i + 1) ("interleaved").
    ``inverse=True`` is the transposed rotation: the gradient of x from that of
    the output.  ``out`` may be x.  A position outside the table gives NaN."""
    view = _heads(x, "x")
    shape = x.shape
    turn = _turn(positions, table, layout, x, shape[-1])
    out, out_view = _out_like(x, out, "out")
    fn, name = _FUNCTIONS["rope"][x.dtype]
    if len(shape) == 3:
        shape = (1, *shape)
    _call(fn, name, x.device, *view, *out_view, *shape, *turn, 1 if inverse else 0)
    return out


def _norm_args(q, k, q_weight, k_weight):
    """Views of q and k, and the sizes and weights of the norm."""
    vq, vk = _heads(q, "q"), _heads(k, "k", (q.dtype,))
    sq, sk = q.shape, k.shape
    dim = sq[-1]
    if len(sk) != len(sq) or sk[:-2] != sq[:-2] or sk[-1] != dim:
        raise ValueError(f"q {tuple(sq)} and k {tuple(sk)} may differ in their heads only")
    _on(k, "k", q)
    wt = q_weight.dtype if isinstance(q_weight, _Tensor) else None
    if wt != q.dtype and wt != torch.float32:
        raise TypeError(f"q_weight must be a {q.dtype} or float32 tensor")
    qw, kw = _vector(q_weight, "q_weight", wt, dim, q), _vector(k_weight, "k_weight", wt, dim, q)
    if q_weight.numel() != dim or k_weight.numel() != dim:
        raise ValueError(f"q_weight and k_weight must have {dim} elements")
    batch, tokens = (1, sq[0]) if len(sq) == 3 else sq[:2]
    return vq, vk, (batch, tokens, sq[-2], sk[-2], dim, qw, kw, 1 if wt == torch.float32 else 0)


def qk_norm_rope(q, k, q_weight, k_weight, positions, table, eps=1e-6, layout="half", q_out=None, k_out=None):
    """RMS norm of every head of q and k ([.., tokens, heads, dim], the same
    tokens) with its weight ([dim], in q's type or fp32), and the rotation of
    ``rope`` in the same pass -> (q_out, k_out), which may be q and k."""
    vq, vk, sizes = _norm_args(q, k, q_weight, k_weight)
    turn = _turn(positions, table, layout, q, sizes[4])
    q_out, vqo = _out_like(q, q_out, "q_out")
    k_out, vko = _out_like(k, k_out, "k_out")
    fn, name = _FUNCTIONS["qk_norm_rope"][q.dtype]
    _call(fn, name, q.device, *vq, *vk, *vqo, *vko, *sizes, eps, *turn)
    return q_out, k_out


def qk_norm_rope_backward(dq_out, dk_out, q, k, q_weight, k_weight, positions, table, eps=1e-6, layout="half",
                          dq=None, dk=None, workspace=None):
    """Gradients of ``qk_norm_rope`` from those of its outputs and its inputs
    -> (dq, dk, dq_weight, dk_weight): the weights' in fp32, summed over
    tokens and heads in a fixed order.  dq may be dq_out, dk may be dk_out."""
    vq, vk, sizes = _norm_args(q, k, q_weight, k_weight)
    dim = sizes[4]
    turn = _turn(positions, table, layout, q, dim)
    vgq, vgk = _heads(dq_out, "dq_out", (q.dtype,)), _heads(dk_out, "dk_out", (q.dtype,))
    for name, g, x in (("dq_out", dq_out, q), ("dk_out", dk_out, k)):
        if g.shape != x.shape:
            raise ValueError(f"{name}: shape {tuple(g.shape)}, expected {tuple(x.shape)}")
        _on(g, name, q)
    dq, vdq = _out_like(q, dq, "dq")
    dk, vdk = _out_like(k, dk, "dk")
    dw = torch.empty((2, dim), dtype=torch.float32, device=q.device)
    keep, space, nbytes = _workspace(_lib.qk_norm_rope_backward_workspace_bytes(dim), workspace,
                                     "qk_norm_rope_backward", q)
    fn, name = _FUNCTIONS["qk_norm_rope_backward"][q.dtype]
    at = dw.data_ptr()
    _call(fn, name, q.device, *vgq, *vgk, *vq, *vk, *vdq, *vdk, *sizes, at, at + 4 * dim, eps, *turn, space, nbytes)
    return dq, dk, dw[0], dw[1]


def append_kv_paged(k, v, slots, k_cache, v_cache, positions=None, table=None, layout="half"):
    """Writes the tokens' keys (rotated by ``positions`` and ``table`` if
    given, else as they are) and values to the slots of a paged cache.

    k [tokens, heads, dim], v [tokens, heads, v_dim]; k_cache [pages,
    page_size, heads, dim], v_cache likewise (a transposed view of [pages,
    heads, page_size, dim] is as good); slots int32/int64 [tokens], slot =
    page * page_size + place, distinct; a slot below 0 or beyond the cache
    writes nothing.  Returns (k_cache, v_cache)."""
    dt = (k.dtype,) if isinstance(k, _Tensor) else _FLOATS
    vk, vv = _heads(k, "k"), _heads(v, "v", dt)
    ck, cv = _heads(k_cache, "k_cache", dt), _heads(v_cache, "v_cache", dt)
    if k.dim() != 3 or v.dim() != 3 or v.shape[:2] != k.shape[:2]:
        raise ValueError(f"k {tuple(k.shape)} and v {tuple(v.shape)} must be [tokens, heads, dim], and may differ in "
                         "dim only")
    tokens, heads, dim = k.shape
    v_dim = v.shape[2]
    kc, vc = k_cache.shape, v_cache.shape
    if len(kc) != 4 or kc[2] != heads or kc[3] != dim:
        raise ValueError(f"k_cache: shape {tuple(kc)}, expected [pages, page_size, {heads}, {dim}]")
    if len(vc) != 4 or vc[2] != heads or vc[3] != v_dim or vc[0] != kc[0] or vc[1] != kc[1]:
        raise ValueError(f"v_cache: shape {tuple(vc)}, expected [{kc[0]}, {kc[1]}, {heads}, {v_dim}]")
    _on(v, "v", k), _on(k_cache, "k_cache", k), _on(v_cache, "v_cache", k)
    slot, slot_bytes = _index(slots, "slots", (tokens,), k)
    if (positions is None) != (table is None):
        raise TypeError("give both positions and table, or neither")
    turn = (None, 0, None, 0, 0, 0) if table is None else _turn(positions, table, layout, k, dim)
    fn, name = _FUNCTIONS["append_kv_paged"][k.dtype]
    _call(fn, name, k.device, vk[0], vk[2], vk[3], vv[0], vv[2], vv[3], tokens, heads, dim, v_dim, slot, slot_bytes,
          *ck, *cv, kc[0], kc[1], *turn)
    return k_cache, v_cache
