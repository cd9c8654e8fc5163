"""ctypes view of the C ABI declared in include/gemm_w4a4.h.

Only argument marshalling lives here: every step of the operator runs in the
HIP kernels of libgemm_w4a4.so. There is no fallback; if the library is
missing, loading fails loudly.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import threading

from .build import BINDING_PATH, LIB_PATH

OK = 0
EINVAL = -1
EALIGN = -2
ELAUNCH = -3
EOVERLAP = -4
EDEVICE = -5
ENOMEM = -6
ESCRATCH = -7
MAX_R = 1024

_PLAN_FIELDS = ("variant", "block_m", "block_n", "block_k", "stages", "waves_m", "waves_n",
                "threads", "lds_bytes", "lds_stage_bytes", "lds_limit", "tiles_m", "tiles_n",
                "grid", "k_stages", "lora_steps", "occupancy", "policy", "lora_place",
                "lds_ring_bytes", "lds_side_bytes", "flavour", "vgprs", "agprs", "sgprs",
                "regs_limit", "k_groups", "tail_variant", "tail_rows", "tail_block_m", "tail_block_n",
                "tail_grid", "tail_splits")


_QPLAN_FIELDS = ("variant", "wide", "rank_tiles", "rows", "threads", "lds_bytes", "row_blocks", "k_slices",
                 "spans_per_slice", "grid", "launches")


class QuantizePlan(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int) for f in _QPLAN_FIELDS] + [("scratch_bytes", ctypes.c_longlong)]

    def as_dict(self) -> dict:
        return {f: getattr(self, f) for f in _QPLAN_FIELDS + ("scratch_bytes",)}


class RotaryArgs(ctypes.Structure):
    """rotary_axes_t."""
    _fields_ = [("x", ctypes.c_void_p), ("out", ctypes.c_void_p), ("positions", ctypes.c_void_p),
                ("inv_freq", ctypes.c_void_p)] + \
               [(f, ctypes.c_int) for f in ("batch", "tokens", "heads", "head_dim", "axes")] + \
               [("sections", ctypes.c_int * 4), ("x_stride", ctypes.c_int64 * 3),
                ("out_stride", ctypes.c_int64 * 3), ("pos_stride", ctypes.c_int64 * 2),
                ("interleaved", ctypes.c_int), ("inverse", ctypes.c_int), ("f16", ctypes.c_int)]


class AttentionArgs(ctypes.Structure):
    """cross_attention_t."""
    _fields_ = [(f, ctypes.c_void_p) for f in ("q", "k", "v", "out", "lse", "kv_lens")] + \
               [(f, ctypes.c_int) for f in ("batch", "q_len", "kv_len", "q_heads", "kv_heads", "head_dim")] + \
               [(f, ctypes.c_int64 * 3) for f in ("q_stride", "k_stride", "v_stride", "out_stride")] + \
               [("scale", ctypes.c_float), ("f16", ctypes.c_int), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_int64)]


class BlockNormArgs(ctypes.Structure):
    """block_norm_t."""
    _fields_ = [(f, ctypes.c_void_p) for f in ("x", "y", "gate", "scale", "shift", "weight", "bias", "post_weight",
                                               "out", "residual")] + \
               [(f, ctypes.c_int) for f in ("batch", "tokens", "width")] + \
               [(f, ctypes.c_int64 * 2) for f in ("x_stride", "y_stride", "gate_stride", "scale_stride", "shift_stride",
                                                  "out_stride", "residual_stride")] + \
               [("residual_scale", ctypes.c_float), ("eps", ctypes.c_float)] + \
               [(f, ctypes.c_int) for f in ("layer", "post_norm", "f16")]


class CacheAppendArgs(ctypes.Structure):
    """cache_append_t."""
    _fields_ = [(f, ctypes.c_void_p) for f in ("k", "v", "k_cache", "v_cache", "slots")] + \
               [(f, ctypes.c_int) for f in ("tokens", "heads", "head_dim", "pages", "page_size")] + \
               [(f, ctypes.c_int64 * 2) for f in ("k_stride", "v_stride")] + \
               [(f, ctypes.c_int64 * 3) for f in ("k_cache_stride", "v_cache_stride")]


class LoraAdaptersArgs(ctypes.Structure):
    """lora_adapters_t."""
    _fields_ = [(f, ctypes.c_void_p) for f in ("x", "y", "down", "up", "out", "adapter", "scaling", "ranks")] + \
               [(f, ctypes.c_int) for f in ("rows", "K", "N", "adapters", "rank")] + \
               [(f, ctypes.c_int64) for f in ("x_stride", "y_stride", "out_stride")] + \
               [("f16", ctypes.c_int), ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_int64)]


class PackedAttentionArgs(ctypes.Structure):
    """packed_attention_t."""
    _fields_ = [(f, ctypes.c_void_p) for f in ("q", "k", "v", "out", "lse", "starts")] + \
               [(f, ctypes.c_int) for f in ("tokens", "seqs", "q_heads", "kv_heads", "head_dim")] + \
               [(f, ctypes.c_int64 * 2) for f in ("q_stride", "k_stride", "v_stride", "out_stride")] + \
               [("scale", ctypes.c_float), ("causal", ctypes.c_int), ("f16", ctypes.c_int)]


class PagedAttentionArgs(ctypes.Structure):
    """paged_attention_t."""
    _fields_ = [(f, ctypes.c_void_p) for f in ("q", "k_cache", "v_cache", "out", "lse", "table", "lens")] + \
               [(f, ctypes.c_int) for f in ("batch", "q_len", "q_heads", "kv_heads", "head_dim", "pages", "page_size", "table_width")] + \
               [(f, ctypes.c_int64 * 3) for f in ("q_stride", "k_stride", "v_stride", "out_stride")] + \
               [("table_stride", ctypes.c_int64), ("scale", ctypes.c_float), ("f16", ctypes.c_int),
                ("workspace", ctypes.c_void_p), ("workspace_bytes", ctypes.c_int64)]


class Plan(ctypes.Structure):
    _fields_ = [(f, ctypes.c_int) for f in _PLAN_FIELDS]

    def as_dict(self) -> dict:
        return {f: getattr(self, f) for f in _PLAN_FIELDS}


_lock = threading.Lock()
_lib = None
_binding = None


def library_path() -> str:
    return LIB_PATH


def load() -> ctypes.CDLL:
    """Load libgemm_w4a4.so (once). Raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it first (python -m bit_quantized_gemm_amd.build "
                "or __graft_entry__.build()); there is no non-HIP fallback")
        lib = ctypes.CDLL(LIB_PATH)
        vp, i = ctypes.c_void_p, ctypes.c_int
        lib.gemm_w4a4.argtypes = [vp] * 9 + [i, i, i, i, vp]
        lib.gemm_w4a4.restype = i
        lib.gemm_w4a4_f16.argtypes = [vp] * 9 + [i, i, i, i, vp]
        lib.gemm_w4a4_f16.restype = i
        lib.gemm_w4a4_plan.argtypes = [i, i, i, i, ctypes.POINTER(Plan)]
        lib.gemm_w4a4_plan.restype = i
        lib.gemm_w4a4_num_variants.argtypes = []
        lib.gemm_w4a4_num_variants.restype = i
        lib.gemm_w4a4_variant_info.argtypes = [i, ctypes.POINTER(Plan)]
        lib.gemm_w4a4_variant_info.restype = i
        for name in ("gemm_mxfp4", "gemm_mxfp4_f16"):
            getattr(lib, name).argtypes = [vp] * 9 + [i, i, i, i, vp]
            getattr(lib, name).restype = i
        lib.gemm_mxfp4_plan.argtypes = [i, i, i, i, ctypes.POINTER(Plan)]
        lib.gemm_mxfp4_plan.restype = i
        lib.gemm_mxfp4_num_variants.argtypes = []
        lib.gemm_mxfp4_num_variants.restype = i
        lib.gemm_mxfp4_variant_info.argtypes = [i, ctypes.POINTER(Plan)]
        lib.gemm_mxfp4_variant_info.restype = i
        lib.quantize_w4a4_act.argtypes = [vp] * 5 + [i, i, i, vp]
        lib.quantize_w4a4_act.restype = i
        lib.quantize_w4a4_act_noalloc.argtypes = [vp] * 5 + [i, i, i, vp]
        lib.quantize_w4a4_act_noalloc.restype = i
        lib.quantize_w4a4_act_plan.argtypes = [i, i, i, ctypes.POINTER(QuantizePlan)]
        lib.quantize_w4a4_act_plan.restype = i
        lib.gemm_w4a4_run.argtypes = [i, i, i] + [vp] * 9 + [i, i, i, i, vp]
        lib.gemm_w4a4_run.restype = i
        lib.gemm_w4a4_plan_variant.argtypes = [i, i, i, i, i, i, ctypes.POINTER(Plan)]
        lib.gemm_w4a4_plan_variant.restype = i
        i64 = ctypes.c_int64
        for name in ("quantize_mxfp4_act", "quantize_mxfp4_act_f16"):
            getattr(lib, name).argtypes = [vp] * 5 + [i, i, i, vp, i64, vp]
            getattr(lib, name).restype = i
        lib.quantize_mxfp4_workspace.argtypes = [i, i, i]
        lib.quantize_mxfp4_workspace.restype = i64
        for name in ("gemm_mxfp4_few", "gemm_mxfp4_few_f16"):
            getattr(lib, name).argtypes = [vp] * 9 + [i, i, i, i, vp]
            getattr(lib, name).restype = i
        lib.rotary_axes.argtypes = [vp, vp]
        lib.rotary_axes.restype = i
        lib.cross_attention.argtypes = [vp, vp]
        lib.cross_attention.restype = i
        lib.cross_attention_workspace.argtypes = [vp]
        lib.cross_attention_workspace.restype = i64
        for name in ("block_norm", "cache_append", "lora_adapters", "packed_attention", "paged_attention"):
            getattr(lib, name).argtypes = [vp, vp]
            getattr(lib, name).restype = i
        for name in ("lora_adapters_workspace", "paged_attention_workspace"):
            getattr(lib, name).argtypes = [vp]
            getattr(lib, name).restype = i64
        lib.gemm_w4a4_strerror.argtypes = [i]
        lib.gemm_w4a4_strerror.restype = ctypes.c_char_p
        _lib = lib
        return lib


def binding():
    """The native part of the binding, _torch_binding.so (loaded once, after torch and
    the library). Raises if it has not been built."""
    global _binding
    if _binding is None:
        import torch  # noqa: F401
        load()
        if not os.path.exists(BINDING_PATH):
            raise RuntimeError(
                f"{BINDING_PATH} is missing: build it first (python -m bit_quantized_gemm_amd.build "
                "or __graft_entry__.build()); there is no other path to these operators")
        loader = importlib.machinery.ExtensionFileLoader("_torch_binding", BINDING_PATH)
        spec = importlib.util.spec_from_file_location("_torch_binding", BINDING_PATH, loader=loader)
        _binding = importlib.util.module_from_spec(spec)
        loader.exec_module(_binding)
    return _binding


def strerror(code: int) -> str:
    return load().gemm_w4a4_strerror(code).decode()


def gemm_w4a4_raw(act, ascales, wgt, wscales, wcscale, bias, lora_act_in, lora_up, out,
                  M, N, K, R, stream) -> int:
    """Direct call of the C entry point with integer addresses; returns its code."""
    return load().gemm_w4a4(act, ascales, wgt, wscales, wcscale, bias, lora_act_in, lora_up,
                            out, M, N, K, R, stream)


def gemm_w4a4_f16_raw(act, ascales, wgt, wscales, wcscale, bias, lora_act_in, lora_up, out,
                      M, N, K, R, stream) -> int:
    """Direct call of the fp16 C entry point (LoRA and out in binary16); returns its code."""
    return load().gemm_w4a4_f16(act, ascales, wgt, wscales, wcscale, bias, lora_act_in, lora_up,
                                out, M, N, K, R, stream)


def gemm_mxfp4_raw(act, ascales, wgt, wscales, wcscale, bias, lora_act_in, lora_up, out,
                   M, N, K, R, stream) -> int:
    """Direct call of the MXFP4 C entry point (UE8M0 scales per 32 k); returns its code."""
    return load().gemm_mxfp4(act, ascales, wgt, wscales, wcscale, bias, lora_act_in, lora_up,
                             out, M, N, K, R, stream)


def gemm_mxfp4_f16_raw(act, ascales, wgt, wscales, wcscale, bias, lora_act_in, lora_up, out,
                       M, N, K, R, stream) -> int:
    """Direct call of the MXFP4 fp16 C entry point; returns its code."""
    return load().gemm_mxfp4_f16(act, ascales, wgt, wscales, wcscale, bias, lora_act_in, lora_up,
                                 out, M, N, K, R, stream)


QUANTIZE_MAX_R = 128


def quantize_raw(x, lora_down, act, ascales, lora_act_in, M, K, R, stream) -> int:
    """Direct call of quantize_w4a4_act with integer addresses; returns its code."""
    return load().quantize_w4a4_act(x, lora_down, act, ascales, lora_act_in, M, K, R, stream)


def quantize_noalloc_raw(x, lora_down, act, ascales, lora_act_in, M, K, R, stream) -> int:
    """Direct call of quantize_w4a4_act_noalloc (no device allocation; its
    scratch is a fixed array per GPU) with integer addresses; returns its code."""
    return load().quantize_w4a4_act_noalloc(x, lora_down, act, ascales, lora_act_in, M, K, R, stream)


FEW_MAX_M = 64
ROTARY_MAX_AXES = 4
ROTARY_MAX_HEAD_DIM = 256
ATTENTION_MAX_HEAD_DIM = 128
BLOCK_NORM_MAX_WIDTH = 16384
LORA_ADAPTERS_MAX_RANK = 128
LORA_ADAPTERS_MAX_ROWS = 3145728
PACKED_ATTENTION_MAX_SEQS = 4096
PAGED_ATTENTION_PAGE_MULTIPLE = 16


def quantize_mxfp4_raw(f16, x, lora_down, act, ascales, lora_act_in, M, K, R, workspace, workspace_bytes,
                       stream) -> int:
    """Direct call of quantize_mxfp4_act (f16: its _f16 twin) with integer addresses; returns its code."""
    fn = load().quantize_mxfp4_act_f16 if f16 else load().quantize_mxfp4_act
    return fn(x, lora_down, act, ascales, lora_act_in, M, K, R, workspace, workspace_bytes, stream)


def quantize_mxfp4_workspace(M: int, K: int, R: int) -> int:
    """Workspace bytes quantize_mxfp4_act needs for (M, K, R) (host only)."""
    n = load().quantize_mxfp4_workspace(M, K, R)
    if n < 0:
        raise ValueError(f"quantize_mxfp4_workspace: {strerror(n)} ({n})")
    return n


def gemm_mxfp4_few_raw(f16, act, ascales, wgt, wscales, wcscale, bias, lora_act_in, lora_up, out,
                       M, N, K, R, stream) -> int:
    """Direct call of gemm_mxfp4_few (f16: its _f16 twin) with integer addresses; returns its code."""
    fn = load().gemm_mxfp4_few_f16 if f16 else load().gemm_mxfp4_few
    return fn(act, ascales, wgt, wscales, wcscale, bias, lora_act_in, lora_up, out, M, N, K, R, stream)


def rotary_axes_raw(args: "RotaryArgs", stream) -> int:
    """Direct call of rotary_axes; returns its code."""
    return load().rotary_axes(ctypes.byref(args), stream)


def cross_attention_raw(args: "AttentionArgs", stream) -> int:
    """Direct call of cross_attention; returns its code."""
    return load().cross_attention(ctypes.byref(args), stream)


def cross_attention_workspace(args: "AttentionArgs") -> int:
    """Workspace bytes of a cross_attention call, or a negative code (host only)."""
    return load().cross_attention_workspace(ctypes.byref(args))


def block_norm_raw(args: "BlockNormArgs", stream) -> int:
    """Direct call of block_norm; returns its code."""
    return load().block_norm(ctypes.byref(args), stream)


def cache_append_raw(args: "CacheAppendArgs", stream) -> int:
    """Direct call of cache_append; returns its code."""
    return load().cache_append(ctypes.byref(args), stream)


def lora_adapters_raw(args: "LoraAdaptersArgs", stream) -> int:
    """Direct call of lora_adapters; returns its code."""
    return load().lora_adapters(ctypes.byref(args), stream)


def lora_adapters_workspace(args: "LoraAdaptersArgs") -> int:
    """Workspace bytes of a lora_adapters call, or a negative code (host only)."""
    return load().lora_adapters_workspace(ctypes.byref(args))


def packed_attention_raw(args: "PackedAttentionArgs", stream) -> int:
    """Direct call of packed_attention; returns its code."""
    return load().packed_attention(ctypes.byref(args), stream)


def paged_attention_raw(args: "PagedAttentionArgs", stream) -> int:
    """Direct call of paged_attention; returns its code."""
    return load().paged_attention(ctypes.byref(args), stream)


def paged_attention_workspace(args: "PagedAttentionArgs") -> int:
    """Workspace bytes of a paged_attention call, or a negative code (host only)."""
    return load().paged_attention_workspace(ctypes.byref(args))


def quantize_plan(M: int, K: int, R: int) -> dict:
    """The launch quantize_w4a4_act would make for (M, K, R) (host only)."""
    p = QuantizePlan()
    rc = load().quantize_w4a4_act_plan(M, K, R, ctypes.byref(p))
    if rc != OK:
        raise ValueError(f"quantize_w4a4_act_plan: {strerror(rc)} ({rc})")
    return p.as_dict()


def run_raw(fmt: str, out_f16: bool, variant: int, act, ascales, wgt, wscales, wcscale, bias,
            lora_act_in, lora_up, out, M, N, K, R, stream) -> int:
    """gemm_w4a4_run: the operator with the format, output type and compiled
    instance (-1: the solver's choice) named explicitly; returns its code."""
    return load().gemm_w4a4_run(_FMT_CODE[fmt], int(out_f16), variant, act, ascales, wgt,
                                wscales, wcscale, bias, lora_act_in, lora_up, out, M, N, K, R,
                                stream)


def plan_variant(M: int, N: int, K: int, R: int, variant: int, fmt: str = "nvfp4") -> dict:
    """The plan of compiled instance `variant` (-1: the solver's) for a shape."""
    p = Plan()
    rc = load().gemm_w4a4_plan_variant(_FMT_CODE[fmt], variant, M, N, K, R, ctypes.byref(p))
    if rc != OK:
        raise ValueError(f"gemm_w4a4_plan_variant: {strerror(rc)} ({rc})")
    return p.as_dict()


_FMT_CODE = {"nvfp4": 0, "mxfp4": 1}
FORMATS = ("nvfp4", "mxfp4")
_PREFIX = {"nvfp4": "gemm_w4a4", "mxfp4": "gemm_mxfp4"}


def _fn(fmt: str, suffix: str):
    if fmt not in _PREFIX:
        raise ValueError(f"fmt must be one of {FORMATS}, got {fmt!r}")
    return getattr(load(), _PREFIX[fmt] + suffix)


def plan(M: int, N: int, K: int, R: int, fmt: str = "nvfp4") -> dict:
    p = Plan()
    rc = _fn(fmt, "_plan")(M, N, K, R, ctypes.byref(p))
    if rc != OK:
        raise ValueError(f"{_PREFIX[fmt]}_plan: {strerror(rc)} ({rc})")
    return p.as_dict()


def variants(fmt: str = "nvfp4") -> list:
    out = []
    info = _fn(fmt, "_variant_info")
    for v in range(_fn(fmt, "_num_variants")()):
        p = Plan()
        if info(v, ctypes.byref(p)) != OK:
            raise RuntimeError("variant_info failed")
        out.append(p.as_dict())
    return out
