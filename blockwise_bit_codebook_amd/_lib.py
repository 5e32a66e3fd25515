"""ctypes loader for libkbit.so and signatures of every exported symbol.

Argument marshalling only.  If the library is missing the import of this
module raises, so no caller can silently fall back to another path.
"""

import ctypes as ct
import importlib.util
import os
import sys

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkbit.so")

DTYPES = ("fp32", "fp16", "bf16")
KS = (2, 3, 4, 5)

_p = ct.c_void_p
_i64 = ct.c_int64
_i32 = ct.c_int32
_f32 = ct.c_float


def _signatures():
    """(name, argtypes) for every C entry point declared in include/kbit.h."""
    sig = [
        ("kbit_strerror", [ct.c_int]),
        ("kbit_abi_version", []),
        ("kbit_codebook_nf", [ct.c_int, _p]),
        ("kbit_codebook_fp4", [_p]),
        ("kbit_codebook_lloyd_max_normal", [ct.c_int, _p]),
        ("kbit_dynamic_map8", [_p]),
        ("quantize_act_fwht_k4_bf16", [_p, _i64, _i32, _p, _p, _p, _p, _p]),
        ("quantize_act_rpbh_k4_bf16", [_p, _i64, _i32, _p, _p, _p, _p, _p, _p]),
        ("kbit_act_tables_bytes", []),
        ("act_tables_k4", [_p, _p, _p]),
        ("quantize_act_fwht_k4_bf16_tables", [_p, _i64, _i32, _p, _p, _p, _p, _p]),
        ("quantize_act_rpbh_k4_bf16_tables", [_p, _i64, _i32, _p, _p, _p, _p, _p, _p]),
        ("kbit_nested_workspace_bytes", [_i64]),
        ("linear_kbit_bf16_k4", [_p, _i64, _i32, _p, _p, _p, _i32, _i32, _p, _p]),
        ("linear_4bit_nested_bf16", [_p, _i64, _i32, _p, _p, _p, _p, _p, _f32, _i32, _i32, _p, _p]),
        ("linear_4bit_nested_bf16_offptr", [_p, _i64, _i32, _p, _p, _p, _p, _p, _p, _i32, _i32, _p, _p]),
        ("quantize_nested_absmax", [_p, _i64, _p, _p, _p, _p, _p, _i64, _p]),
        ("kbit_nested_noalloc_scratch_bytes", []),
        ("quantize_nested_absmax_noalloc", [_p, _i64, _p, _p, _p, _p, _p]),
        ("kbit_quantize_nested_workspace_bytes", []),
    ]
    for t in DTYPES:
        for k in KS:
            sig.append((f"quantize_kbit_{t}_k{k}", [_p, _p, _p, _p, _i64, _i32, _p]))
            sig.append((f"dequantize_kbit_{t}_k{k}", [_p, _p, _p, _p, _i64, _i32, _p]))
            sig.append((f"quantize_kbit_e4m4_{t}_k{k}", [_p, _p, _p, _p, _i64, _i32, _p]))
            sig.append((f"dequantize_kbit_e4m4_{t}_k{k}", [_p, _p, _p, _p, _i64, _i32, _p]))
        sig.append((f"dequantize_4bit_nested_{t}", [_p, _p, _p, _p, _p, _f32, _p, _i64, _i32, _p]))
        sig.append((f"dequantize_4bit_nested_{t}_offptr", [_p, _p, _p, _p, _p, _p, _p, _i64, _i32, _p]))
        sig.append((f"quantize_4bit_nested_{t}", [_p, _p, _p, _p, _p, _p, _p, _p, _i64, _i32, _p, _i64, _p]))
    return sig


SIGNATURES = _signatures()


def _layer_signatures():
    """(name, argtypes) for every C entry point declared in include/kbit_layer.h."""
    f64 = ct.c_double
    view = [_p, _i64, _i64, _i64]
    turn = [_p, _i32, _p, _i32, _i64, _i32]  # positions, their bytes, table, rot, max_pos, layout
    sig = [
        ("linear_int8_workspace_bytes", [_i64, _i32, _i32]),
        ("linear_int8_dynamic_workspace_bytes", [_i64, _i32, _i32]),
        ("linear_int8_dynamic_fused", [_i64, _i32, _i32, _i64]),
        ("qk_norm_rope_backward_workspace_bytes", [_i32]),
        ("rope_frequencies", [_i32, f64, _i32, f64, f64, f64, f64, _p, _p]),
        ("rope_table", [_p, _i32, _i64, f64, _p, _p]),
    ]
    for t in DTYPES:
        sig += [
            (f"quantize_rows_int8_{t}", [_p, _i64, _i32, _i64, _p, _i64, _p, _p]),
            (f"linear_int8_{t}", [_p, _p, _i64, _i32, _i64, _p, _p, _i32, _i64, _p, _p, _i64, _p, _i64, _p]),
            (f"linear_int8_dynamic_{t}", [_p, _i64, _i32, _i64, _p, _p, _i32, _i64, _p, _p, _i64, _p, _i64, _p]),
            (f"rope_{t}", view * 2 + [_i64, _i64, _i32, _i32] + turn + [_i32, _p]),
            (f"qk_norm_rope_{t}", view * 4 + [_i64, _i64, _i32, _i32, _i32, _p, _p, _i32, _f32] + turn + [_p]),
            (f"qk_norm_rope_backward_{t}",
             view * 6 + [_i64, _i64, _i32, _i32, _i32, _p, _p, _i32, _p, _p, _f32] + turn + [_p, _i64, _p]),
            (f"append_kv_paged_{t}",
             [_p, _i64, _i64] * 2 + [_i64, _i32, _i32, _i32, _p, _i32] + view * 2 + [_i64, _i32] + turn + [_p]),
        ]
    return sig


LAYER_SIGNATURES = _layer_signatures()


def _mx_signatures():
    """(name, argtypes) for every C entry point declared in include/kbit_mx.h."""
    sig = [
        ("linear_mxfp4_workspace_bytes", [_i64, _i32, _i32]),
        ("linear_mxfp4_dynamic_workspace_bytes", [_i64, _i32, _i32]),
        ("linear_mxfp4_dynamic_fused", [_i64, _i32, _i32, _i64, _i64]),
        ("linear_mxfp4_backward_workspace_bytes", [_i64, _i32, _i32]),
        ("layer_norm_backward_workspace_bytes", [_i64, _i32]),
    ]
    weight = [_p, _p, _i32, _i64, _i64]  # codes, scales, N, their rows' distances
    end = [_p, _p, _i64, _p, _i64, _p]   # bias, out, ldo, workspace, its bytes, stream
    for t in DTYPES:
        sig += [
            (f"quantize_mxfp4_{t}", [_p, _i64, _i32, _i64, _p, _i64, _p, _i64, _p]),
            (f"quantize_mxfp4_columns_{t}", [_p, _i64, _i32, _i64, _p, _i64, _p, _i64, _p]),
            (f"dequantize_mxfp4_{t}", [_p, _i64, _p, _i64, _i64, _i32, _p, _i64, _p]),
            (f"linear_mxfp4_{t}", [_p, _p, _i64, _i32, _i64, _i64] + weight + end),
            (f"linear_mxfp4_dynamic_{t}", [_p, _i64, _i32, _i64] + weight + end),
            (f"linear_mxfp4_backward_{t}",
             [_p, _i64] * 3 + [_i64, _i32, _i32] + [_p, _i64] * 2 + [_p, _p, _i64, _p]),
            (f"layer_norm_{t}", [_p, _i64, _i32, _i64, _p, _p, _i32, _f32, _p, _i64, _p]),
            (f"layer_norm_backward_{t}",
             [_p, _i64, _p, _i64, _i64, _i32, _p, _i32, _f32, _p, _i64, _p, _p, _p, _i64, _p]),
        ]
    return sig


MX_SIGNATURES = _mx_signatures()


def _share_torch_runtime():
    """torch ships a HIP runtime of its own.  Loaded first it serves libkbit.so
    too, which asks for the same soname; the other way round the process would
    hold two runtimes, and the second to touch the GPU fails.  So where torch is
    installed and not imported yet, its runtime (not torch) is loaded here."""
    if "torch" in sys.modules:
        return
    spec = importlib.util.find_spec("torch")
    if spec is None or spec.origin is None:
        return
    path = os.path.join(os.path.dirname(spec.origin), "lib", "libamdhip64.so")
    if os.path.exists(path):
        try:
            ct.CDLL(path)
        except OSError:
            pass  # a torch that cannot be imported here either


def load(path=LIB_PATH):
    if not os.path.exists(path):
        raise ImportError(
            f"libkbit.so not found at {path}; build it with "
            "`python -m blockwise_bit_codebook_amd.build` (hipcc, gfx950)")
    _share_torch_runtime()
    lib = ct.CDLL(path)
    for name, args in SIGNATURES + LAYER_SIGNATURES + MX_SIGNATURES:
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = {"kbit_strerror": ct.c_char_p, "kbit_nested_workspace_bytes": ct.c_int64,
                      "kbit_nested_noalloc_scratch_bytes": ct.c_int64,
                      "kbit_quantize_nested_workspace_bytes": ct.c_int64,
                      "kbit_act_tables_bytes": ct.c_int64,
                      "linear_int8_workspace_bytes": ct.c_int64,
                      "linear_int8_dynamic_workspace_bytes": ct.c_int64,
                      "qk_norm_rope_backward_workspace_bytes": ct.c_int64,
                      "linear_mxfp4_workspace_bytes": ct.c_int64,
                      "linear_mxfp4_dynamic_workspace_bytes": ct.c_int64,
                      "linear_mxfp4_backward_workspace_bytes": ct.c_int64,
                      "layer_norm_backward_workspace_bytes": ct.c_int64}.get(name, ct.c_int)
    return lib


lib = load()
