"""ctypes declarations of the ltx3drope C ABI (include/ltx3drope.h).

Loading fails loudly when the HIP library has not been built: there is no CPU
fallback anywhere in this package.
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libltx3drope.so")

OK = 0
E_INVALID = -1
E_UNSUPPORTED = -2
E_TABLE_MISMATCH = -3
E_HIP = -4
E_NOMEM = -5

DTYPE_F32 = 0
DTYPE_BF16 = 1

REASONS = {
    0: "OK", 1: "NULLPTR", 2: "DTYPE", 3: "NONPOSITIVE_DIM", 4: "SPLIT_ODD", 5: "SPLIT_SUM",
    6: "TABLE_GRID", 7: "TABLE_DEVICE", 8: "ALIGN", 9: "OVERLAP", 10: "TOO_LARGE",
    11: "NOT_DEVICE_PTR", 12: "HOST_MODE", 13: "EXTENT",
}
REASON_CODES = {v: k for k, v in REASONS.items()}

OPT_PATH = 1
OPT_GATE = 2
OPT_FORCE_GATE_MISMATCH = 3
OPT_HOST_TABLES = 4
OPT_LOG = 5

GATE_STATES = {0: "UNSEEN", 1: "TRUSTED", 2: "DISABLED"}

# every symbol the header declares (checked by the CPU test suite)
EXPORTS = (
    "ltx3drope_tables_build", "ltx3drope_tables_release", "ltx3drope_tables_describe", "ltx3drope_tables_read",
    "ltx3drope_cache_clear", "ltx3drope_can_use", "ltx3drope_apply_qk", "ltx3drope_apply_qk_noalloc",
    "ltx3drope_can_use_shard",
    "ltx3drope_apply_qk_shard", "ltx3drope_neox_can_use", "ltx3drope_neox_apply_qk",
    "ltx3drope_neox_position_errors", "ltx3drope_patchify", "ltx3drope_unpatchify", "ltx3drope_dit_freq_grid",
    "ltx3drope_gate_state",
    "ltx3drope_gate_reset", "ltx3drope_set_option", "ltx3drope_get_option", "ltx3drope_stats",
    "ltx3drope_stats_reset", "ltx3drope_kernel_choice", "ltx3drope_copy", "ltx3drope_status_string",
    "ltx3drope_reason_string", "ltx3drope_version",
    "ltx3drope_norm", "ltx3drope_norm_backward", "ltx3drope_norm_backward_workspace",
    "ltx3drope_gated_ffn", "ltx3drope_gated_ffn_workspace", "ltx3drope_gated_ffn_backward",
    "ltx3drope_gated_ffn_backward_workspace", "ltx3drope_q8_quantize", "ltx3drope_q8_matmul",
    "ltx3drope_q8_matmul_workspace",
    "ltx3drope_layer_norm", "ltx3drope_layer_norm_backward", "ltx3drope_layer_norm_backward_workspace",
    "ltx3drope_axes_apply", "ltx3drope_axes_frequencies",
    "ltx3drope_f8_quantize", "ltx3drope_f8_matmul", "ltx3drope_f8_matmul_workspace",
)

POSITION_I64, POSITION_I32, POSITION_F32 = 0, 1, 2
FREQUENCY_F64, FREQUENCY_F32 = 0, 1
PAIRINGS = {"adjacent": 0, "halves": 1}
ACTIVATIONS = {"silu": 0, "gelu": 1, "gelu_tanh": 2}

i64 = ctypes.c_int64
vp = ctypes.c_void_p
fp = ctypes.POINTER(ctypes.c_float)


class TablesDesc(ctypes.Structure):
    _fields_ = [("device", ctypes.c_int), ("T", i64), ("H", i64), ("W", i64), ("dim_t", i64), ("dim_h", i64),
                ("dim_w", i64), ("base", ctypes.c_double), ("packed", vp), ("packed_pairs", i64)]


class Shard(ctypes.Structure):
    _fields_ = [("t_offset", i64), ("h_offset", i64), ("w_offset", i64), ("inplace", ctypes.c_int32),
                ("reserved", ctypes.c_int32)]


class Stats(ctypes.Structure):
    _fields_ = [(n, i64) for n in (
        "cache_hits", "cache_misses", "cache_evictions", "cache_live", "tables_alive", "gate_verifications",
        "gate_trusted", "gate_disabled", "fast_launches", "plain_launches", "rejected")]

    def as_dict(self):
        return {n: int(getattr(self, n)) for n, _ in self._fields_}


_NORM_SCALARS = [(n, ctypes.c_int32) for n in ("dtype", "param_dtype", "after", "post_norm", "next_norm", "reserved")] + [
    (n, i64) for n in ("batch", "rows", "dim")] + [
    (n, ctypes.c_float) for n in ("eps", "weight_offset", "residual_scale")]


class Norm(ctypes.Structure):
    _fields_ = _NORM_SCALARS + [(n, vp) for n in (
        "y", "residual", "weight", "gate", "next_weight", "next_scale", "next_shift", "r", "n")]


class NormBackward(ctypes.Structure):
    _fields_ = _NORM_SCALARS + [(n, vp) for n in (
        "dr", "dn", "y", "r", "weight", "gate", "next_weight", "next_scale",
        "dresidual", "dy", "dweight", "dgate", "dnext_weight", "dnext_scale", "dnext_shift", "workspace")] + [
        ("workspace_bytes", i64)]


_LAYER_NORM_SCALARS = [(n, ctypes.c_int32) for n in ("dtype", "param_dtype", "after", "reserved")] + [
    (n, i64) for n in ("batch", "rows", "dim")] + [("eps", ctypes.c_float)]


class LayerNorm(ctypes.Structure):
    _fields_ = _LAYER_NORM_SCALARS + [(n, vp) for n in (
        "y", "residual", "gate", "weight", "bias", "scale", "shift", "r", "n")]


class LayerNormBackward(ctypes.Structure):
    _fields_ = _LAYER_NORM_SCALARS + [(n, vp) for n in (
        "dr", "dn", "y", "r", "gate", "weight", "bias", "scale",
        "dresidual", "dy", "dgate", "dweight", "dbias", "dscale", "dshift", "workspace")] + [("workspace_bytes", i64)]


_FFN_SIZES = [("dtype", ctypes.c_int32), ("activation", ctypes.c_int32)] + [(n, i64) for n in (
    "tokens", "dim", "hidden")]


class GatedFfn(ctypes.Structure):
    _fields_ = _FFN_SIZES + [(n, vp) for n in ("x", "w_gate", "w_up", "h", "g", "u", "workspace")] + [
        ("workspace_bytes", i64)]


class GatedFfnBackward(ctypes.Structure):
    _fields_ = _FFN_SIZES + [(n, vp) for n in (
        "dh", "x", "w_gate", "w_up", "g", "u", "dx", "dw_gate", "dw_up", "workspace")] + [("workspace_bytes", i64)]


class Q8Matmul(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32)] + [(n, i64) for n in (
        "tokens", "dim", "out")] + [(n, vp) for n in ("a", "b", "a_scale", "b_scale", "bias", "y", "workspace")] + [
        ("workspace_bytes", i64)]


class F8Quantize(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("blocks", ctypes.c_int32)] + [(n, i64) for n in (
        "rows", "dim", "turned_pitch")] + [(n, i64 * 2) for n in ("scale_strides", "scale_turned_strides")] + [
        (n, vp) for n in ("x", "q", "scale", "q_turned", "scale_turned")]


class F8Matmul(ctypes.Structure):
    _fields_ = [("dtype", ctypes.c_int32), ("b_rows", ctypes.c_int32)] + [(n, i64) for n in (
        "tokens", "dim", "out", "a_pitch", "b_pitch")] + [
        (n, i64 * 2) for n in ("a_scale_strides", "b_scale_strides")] + [(n, vp) for n in (
            "a", "b", "a_scale", "b_scale", "bias", "y", "workspace")] + [("workspace_bytes", i64)]


class Axes(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("dtype", "pairing", "inverse", "position_type", "frequency_type", "axes")] + [
        (n, i64) for n in ("batch", "tokens", "q_heads", "k_heads", "head_dim", "pairs")] + [
        (n, i64 * 3) for n in ("q_strides", "k_strides", "q_out_strides", "k_out_strides", "position_strides")] + [
        (n, vp) for n in ("q", "k", "q_out", "k_out", "positions", "frequencies", "axis")]


# The same descriptors as bytes, for the calls that single tokens wait for: a struct.pack takes a
# tenth of the time of filling a ctypes.Structure by name.
NORM_BYTES = struct.Struct("@6i3q3f9P")
NORM_BACKWARD_BYTES = struct.Struct("@6i3q3f16Pq")
LAYER_NORM_BYTES = struct.Struct("@4i3qf9P")
LAYER_NORM_BACKWARD_BYTES = struct.Struct("@4i3qf16Pq")
FFN_BYTES = struct.Struct("@2i3q7Pq")
FFN_BACKWARD_BYTES = struct.Struct("@2i3q10Pq")
Q8_BYTES = struct.Struct("@2i3q7Pq")
F8_QUANTIZE_BYTES = struct.Struct("@2i7q5P")
F8_BYTES = struct.Struct("@2i9q7Pq")
AXES_BYTES = struct.Struct("@6i21q7P")

# entry points that take a descriptor as bytes (bound in lib())
norm = norm_backward = layer_norm = layer_norm_backward = gated_ffn = gated_ffn_backward = q8_matmul = None
axes_apply = f8_quantize = f8_matmul = f8_matmul_workspace = None
norm_backward_workspace = layer_norm_backward_workspace = gated_ffn_workspace = gated_ffn_backward_workspace = None
q8_matmul_workspace = None


def _bind_bytes(L) -> None:
    call = ctypes.CFUNCTYPE(ctypes.c_int, ctypes.c_char_p, vp, vp)
    size = ctypes.CFUNCTYPE(i64, ctypes.c_char_p)
    for name in ("norm", "norm_backward", "layer_norm", "layer_norm_backward", "gated_ffn", "gated_ffn_backward",
                 "q8_matmul", "axes_apply", "f8_quantize", "f8_matmul"):
        globals()[name] = call(("ltx3drope_" + name, L))
        if name not in ("norm", "layer_norm", "axes_apply", "f8_quantize"):
            globals()[name + "_workspace"] = size((f"ltx3drope_{name}_workspace", L))


_lock = threading.Lock()
_lib = None


def lib() -> ctypes.CDLL:
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"ltx3drope HIP library not found at {LIB_PATH}; build it with "
                "`python -m rope_ltx3drope_amd.build` (there is no CPU fallback)")
        # torch first: its HIP runtime must be the process's one.  torch links the runtime under
        # another name than this library does, so loading this library first would bring in a
        # second runtime, to which torch's streams and allocations are unknown.
        try:
            import torch  # noqa: F401
        except ImportError:
            pass
        L = ctypes.CDLL(LIB_PATH)
        sig = {
            "ltx3drope_tables_build": (ctypes.c_int, [ctypes.c_int, i64, i64, i64, i64, i64, i64, ctypes.c_double, vp,
                                                      ctypes.POINTER(vp)]),
            "ltx3drope_tables_release": (ctypes.c_int, [vp]),
            "ltx3drope_tables_describe": (ctypes.c_int, [vp, ctypes.POINTER(TablesDesc)]),
            "ltx3drope_tables_read": (ctypes.c_int, [vp, fp, fp, fp, fp, fp, fp]),
            "ltx3drope_cache_clear": (ctypes.c_int, []),
            "ltx3drope_can_use": (ctypes.c_int, [vp, vp, vp, vp, ctypes.c_int, i64, i64, i64, i64, i64, i64, vp,
                                                 ctypes.POINTER(ctypes.c_int)]),
            "ltx3drope_apply_qk": (ctypes.c_int, [vp, vp, vp, vp, ctypes.c_int, i64, i64, i64, i64, i64, i64, vp, vp]),
            "ltx3drope_apply_qk_noalloc": (ctypes.c_int, [vp, vp, vp, vp, ctypes.c_int, i64, i64, i64, i64, i64, i64,
                                                          vp, vp]),
            "ltx3drope_can_use_shard": (ctypes.c_int, [vp, vp, vp, vp, ctypes.c_int, i64, i64, i64, i64, i64, i64,
                                                       ctypes.POINTER(Shard), vp, ctypes.POINTER(ctypes.c_int)]),
            "ltx3drope_apply_qk_shard": (ctypes.c_int, [vp, vp, vp, vp, ctypes.c_int, i64, i64, i64, i64, i64, i64,
                                                        ctypes.POINTER(Shard), vp, vp]),
            "ltx3drope_neox_can_use": (ctypes.c_int, [vp, vp, vp, vp, ctypes.c_int, i64, i64, i64, i64, vp, vp,
                                                      ctypes.c_int, i64, ctypes.POINTER(ctypes.c_int)]),
            "ltx3drope_neox_apply_qk": (ctypes.c_int, [vp, vp, vp, vp, ctypes.c_int, i64, i64, i64, i64, vp, vp,
                                                       ctypes.c_int, i64, vp]),
            "ltx3drope_neox_position_errors": (ctypes.c_int, [ctypes.c_int, ctypes.c_int, ctypes.POINTER(i64)]),
            "ltx3drope_patchify": (ctypes.c_int, [vp, vp, ctypes.c_int] + [i64] * 6 + [vp]),
            "ltx3drope_unpatchify": (ctypes.c_int, [vp, vp, ctypes.c_int] + [i64] * 6 + [vp]),
            "ltx3drope_dit_freq_grid": (ctypes.c_int, [ctypes.c_double, i64, i64, ctypes.c_int, vp, vp,
                                                       ctypes.POINTER(i64)]),
            "ltx3drope_gate_state": (ctypes.c_int, [ctypes.c_int, ctypes.c_int] + [i64] * 9),
            "ltx3drope_gate_reset": (ctypes.c_int, []),
            "ltx3drope_set_option": (ctypes.c_int, [ctypes.c_int, i64]),
            "ltx3drope_get_option": (i64, [ctypes.c_int]),
            "ltx3drope_stats": (ctypes.c_int, [ctypes.POINTER(Stats)]),
            "ltx3drope_stats_reset": (ctypes.c_int, []),
            "ltx3drope_kernel_choice": (ctypes.c_int, [vp, vp, vp, vp, ctypes.c_int, i64, i64, i64, i64, i64, i64,
                                                       vp]),
            "ltx3drope_copy": (ctypes.c_int, [vp, vp, i64, vp]),
            "ltx3drope_status_string": (ctypes.c_char_p, [ctypes.c_int]),
            "ltx3drope_reason_string": (ctypes.c_char_p, [ctypes.c_int]),
            "ltx3drope_version": (ctypes.c_int, []),
            "ltx3drope_norm": (ctypes.c_int, [ctypes.POINTER(Norm), vp, ctypes.POINTER(ctypes.c_int)]),
            "ltx3drope_norm_backward": (ctypes.c_int, [ctypes.POINTER(NormBackward), vp,
                                                       ctypes.POINTER(ctypes.c_int)]),
            "ltx3drope_norm_backward_workspace": (i64, [ctypes.POINTER(NormBackward)]),
            "ltx3drope_layer_norm": (ctypes.c_int, [ctypes.POINTER(LayerNorm), vp, ctypes.POINTER(ctypes.c_int)]),
            "ltx3drope_layer_norm_backward": (ctypes.c_int, [ctypes.POINTER(LayerNormBackward), vp,
                                                             ctypes.POINTER(ctypes.c_int)]),
            "ltx3drope_layer_norm_backward_workspace": (i64, [ctypes.POINTER(LayerNormBackward)]),
            "ltx3drope_f8_quantize": (ctypes.c_int, [ctypes.POINTER(F8Quantize), vp, ctypes.POINTER(ctypes.c_int)]),
            "ltx3drope_f8_matmul": (ctypes.c_int, [ctypes.POINTER(F8Matmul), vp, ctypes.POINTER(ctypes.c_int)]),
            "ltx3drope_f8_matmul_workspace": (i64, [ctypes.POINTER(F8Matmul)]),
            "ltx3drope_axes_apply": (ctypes.c_int, [ctypes.POINTER(Axes), vp, ctypes.POINTER(ctypes.c_int)]),
            "ltx3drope_axes_frequencies": (ctypes.c_int, [ctypes.c_int, ctypes.POINTER(i64), ctypes.c_double,
                                                          ctypes.c_int, ctypes.POINTER(ctypes.c_double),
                                                          ctypes.POINTER(ctypes.c_uint8)]),
            "ltx3drope_gated_ffn": (ctypes.c_int, [ctypes.POINTER(GatedFfn), vp, ctypes.POINTER(ctypes.c_int)]),
            "ltx3drope_gated_ffn_workspace": (i64, [ctypes.POINTER(GatedFfn)]),
            "ltx3drope_gated_ffn_backward": (ctypes.c_int, [ctypes.POINTER(GatedFfnBackward), vp,
                                                            ctypes.POINTER(ctypes.c_int)]),
            "ltx3drope_gated_ffn_backward_workspace": (i64, [ctypes.POINTER(GatedFfnBackward)]),
            "ltx3drope_q8_quantize": (ctypes.c_int, [ctypes.c_int, i64, i64, vp, vp, vp, vp,
                                                     ctypes.POINTER(ctypes.c_int)]),
            "ltx3drope_q8_matmul": (ctypes.c_int, [ctypes.POINTER(Q8Matmul), vp, ctypes.POINTER(ctypes.c_int)]),
            "ltx3drope_q8_matmul_workspace": (i64, [ctypes.POINTER(Q8Matmul)]),
        }
        assert set(sig) == set(EXPORTS)
        for name, (res, args) in sig.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _bind_bytes(L)
        _lib = L
        return L


def status_string(code: int) -> str:
    return lib().ltx3drope_status_string(code).decode()


def reason_string(code: int) -> str:
    return lib().ltx3drope_reason_string(code).decode()
