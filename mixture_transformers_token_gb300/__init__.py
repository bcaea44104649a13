"""MoT token-routed dense projection for GB300 (sm_103a): Python binding of libmot.so.

Argument marshalling only. Every step of the path -- routing pre-pass, fused add-RMSNorm,
routed GEMMs and their epilogues -- runs in the CUDA kernels of libmot.so, whose C ABI is
declared in include/mot.h. PyTorch provides device memory and streams. There is no CPU
fallback: a missing or stale library raises, and every nonzero status raises MotError.

Functions keep the C names. Tensors are contiguous CUDA tensors: bf16 for activations and
weights, uint8 for the modality index (0 = und, 1 = gen), int32 for positions, uint8 for
the workspace. `stream` (a torch.cuda.Stream or its handle) is the stream that a call is
launched on, None the current one; buffers that are not given are made on it, and may be used
on the current stream once that waits for it. The order of given tensors is the caller's.
"""

from __future__ import annotations

import ctypes
import math
import os

import torch

__all__ = [
    "MotError", "load_library", "library_path", "ABI_VERSION", "EPI_CAST", "EPI_SWIGLU",
    "DEV_BAD_MODALITY", "DEV_TIMEOUT", "DEV_PLAN_MISMATCH", "DEV_BAD_POSITION",
    "mot_abi_version", "mot_status_string", "mot_workspace_bytes", "mot_route_plan",
    "mot_fused_add_rmsnorm", "mot_routed_qkv_norm_rope", "mot_routed_gemm",
    "mot_swiglu_interleave", "mot_rope_table_fill_host", "mot_device_status", "mot_routed_gemm_noalloc",
    "mot_routed_qkv_norm_rope_fp32", "mot_rope_table_fill_host_fp32", "mot_add_rmsnorm_backward",
    "mot_rmsnorm_dweight", "mot_routed_gemm_dx", "mot_routed_gemm_dw", "mot_joint_attention", "DEV_BAD_SEQUENCE",
    "NOALLOC_MAX_TOKENS", "A_PLAN_ORDER", "OUT_PLAN_ORDER", "SET_UND", "SET_GEN", "SET_BOTH", "mot_gather_rows",
    "mot_selftest_wait_timeout",
    "DEV_BAD_TIME", "mot_flow_workspace_bytes", "mot_flow_schedule_host", "mot_cfg_combine_renorm",
    "mot_flow_sde_step", "mot_flow_cfg_sde_step", "mot_flow_noise",
    "DEV_BAD_PAGE", "KV_BF16", "KV_E4M3", "mot_kv_cache_write", "mot_kv_cache_read",
    "mot_paged_decode_workspace_bytes", "mot_paged_decode_attention",
    "mot_joint_attention_lse", "mot_joint_attention_backward_workspace_bytes", "mot_joint_attention_backward",
    "mot_qk_norm_rope_backward_workspace_bytes", "mot_qk_norm_rope_backward", "mot_qk_norm_rope_backward_fp32",
    "DEV_BAD_HYPER", "ADAMW_BLOCK", "AdamWTensors", "mot_adamw_hyper_host", "mot_adamw_step",
]

ABI_VERSION = 6
EPI_CAST = 0
EPI_SWIGLU = 1
A_PLAN_ORDER = 0x100
OUT_PLAN_ORDER = 0x200
SET_UND, SET_GEN, SET_BOTH = 1, 2, 3  # weight-set masks of the norm backward's partials and fold
DEV_BAD_MODALITY = 0x1
DEV_TIMEOUT = 0x2
DEV_PLAN_MISMATCH = 0x4
DEV_BAD_POSITION = 0x8
DEV_BAD_SEQUENCE = 0x10
DEV_BAD_TIME = 0x20
DEV_BAD_PAGE = 0x40
DEV_BAD_HYPER = 0x80
KV_BF16, KV_E4M3 = 0, 1  # element types of a paged key-value cache
NOALLOC_MAX_TOKENS = 65536
ADAMW_BLOCK = 256  # elements of an 8-bit optimizer state that share a scale
_ADAMW_GRAD_BF16, _ADAMW_STATE_E4M3, _ADAMW_HYPER_WORDS = 1, 2, 16

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB = None

_c_p = ctypes.c_void_p
_c_i64 = ctypes.c_int64
_c_i = ctypes.c_int
_c_f = ctypes.c_float
_c_sz = ctypes.c_size_t

_SIGNATURES = {
    "mot_abi_version": (_c_i, []),
    "mot_status_string": (ctypes.c_char_p, [_c_i]),
    "mot_workspace_bytes": (_c_sz, [_c_i64]),
    "mot_route_plan": (_c_i, [_c_p, _c_i64, _c_p, _c_sz, _c_p]),
    "mot_fused_add_rmsnorm": (_c_i, [_c_p, _c_p, _c_p, _c_p, _c_i64, _c_i, _c_f, _c_p, _c_p, _c_p, _c_sz, _c_p]),
    "mot_routed_qkv_norm_rope": (_c_i, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_i, _c_i64, _c_i, _c_i, _c_i,
                                        _c_i, _c_f, _c_p, _c_sz, _c_p, _c_p]),
    "mot_routed_qkv_norm_rope_fp32": (_c_i, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_i, _c_i64, _c_i, _c_i,
                                             _c_i, _c_i, _c_f, _c_p, _c_sz, _c_p, _c_p]),
    "mot_routed_gemm": (_c_i, [_c_p, _c_p, _c_i64, _c_i, _c_i, _c_i, _c_p, _c_sz, _c_p, _c_p]),
    "mot_routed_gemm_noalloc": (_c_i, [_c_p, _c_p, _c_p, _c_i64, _c_i, _c_i, _c_i, _c_p, _c_p, _c_p]),
    "mot_swiglu_interleave": (_c_i, [_c_p, _c_p, _c_i, _c_i, _c_p, _c_p]),
    "mot_gather_rows": (_c_i, [_c_p, _c_i64, _c_i, _c_p, _c_sz, _c_p, _c_p]),
    "mot_selftest_wait_timeout": (_c_i, [_c_p, _c_sz, _c_p]),
    "mot_rope_table_fill_host": (_c_i, [ctypes.c_double, _c_i, _c_i, _c_p]),
    "mot_rope_table_fill_host_fp32": (_c_i, [ctypes.c_double, _c_i, _c_i, _c_p]),
    "mot_add_rmsnorm_backward": (_c_i, [_c_p, _c_p, _c_p, _c_p, _c_i64, _c_i, _c_f, _c_p, _c_sz, _c_p, _c_p, _c_p,
                                        _c_i, _c_p]),
    "mot_rmsnorm_dweight": (_c_i, [_c_p, _c_i64, _c_i, _c_i, _c_p, _c_sz, _c_p, _c_p]),
    "mot_routed_gemm_dx": (_c_i, [_c_p, _c_p, _c_i64, _c_i, _c_i, _c_i, _c_p, _c_sz, _c_p, _c_p]),
    "mot_routed_gemm_dw": (_c_i, [_c_p, _c_p, _c_i64, _c_i, _c_i, _c_i, _c_i, _c_p, _c_sz, _c_p, _c_p]),
    "mot_joint_attention": (_c_i, [_c_p, _c_i64, _c_i, _c_i, _c_i, _c_p, _c_i, _c_f, _c_p, _c_sz, _c_p, _c_p]),
    "mot_flow_workspace_bytes": (_c_sz, [_c_i, _c_i64]),
    "mot_flow_schedule_host": (_c_i, [_c_i, ctypes.c_double, _c_p]),
    "mot_cfg_combine_renorm": (_c_i, [_c_p, _c_p, _c_p, _c_i, _c_i64, _c_p, _c_p, _c_sz, _c_p, _c_p]),
    "mot_flow_sde_step": (_c_i, [_c_p, _c_p, _c_p, _c_p, _c_i, _c_i64, _c_p, _c_p, _c_sz, _c_p, _c_p]),
    "mot_flow_cfg_sde_step": (_c_i, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_i, _c_i64, _c_p, _c_p, _c_sz,
                                     _c_p, _c_p, _c_p]),
    "mot_flow_noise": (_c_i, [_c_p, ctypes.c_uint64, _c_i, _c_i64, _c_p, _c_p]),
    "mot_kv_cache_write": (_c_i, [_c_p, _c_i64, _c_i, _c_i, _c_i, _c_p, _c_i, _c_i64, _c_i, _c_p, _c_p, _c_p, _c_p,
                                  _c_sz, _c_p]),
    "mot_kv_cache_read": (_c_i, [_c_p, _c_p, _c_p, _c_i, _c_i64, _c_i, _c_p, _c_i64, _c_i, _c_i, _c_i, _c_p, _c_p,
                                 _c_sz, _c_p]),
    "mot_paged_decode_workspace_bytes": (_c_sz, [_c_i64, _c_i, _c_i, _c_i, _c_i, _c_i]),
    "mot_paged_decode_attention": (_c_i, [_c_p, _c_i64, _c_i, _c_i, _c_i, _c_p, _c_p, _c_i, _c_i, _c_i64, _c_i, _c_p,
                                          _c_p, _c_p, _c_f, _c_p, _c_sz, _c_p, _c_p]),
    "mot_joint_attention_lse": (_c_i, [_c_p, _c_i64, _c_i, _c_i, _c_i, _c_p, _c_i, _c_f, _c_p, _c_sz, _c_p, _c_p, _c_p]),
    "mot_joint_attention_backward_workspace_bytes": (_c_sz, [_c_i64, _c_i, _c_i, _c_i, _c_i]),
    "mot_joint_attention_backward": (_c_i, [_c_p, _c_p, _c_p, _c_p, _c_i64, _c_i, _c_i, _c_i, _c_p, _c_i, _c_f, _c_p, _c_sz,
                                            _c_p, _c_p]),
    "mot_qk_norm_rope_backward_workspace_bytes": (_c_sz, [_c_i64, _c_i]),
    "mot_qk_norm_rope_backward": (_c_i, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_i, _c_i64, _c_i, _c_i, _c_i, _c_f, _c_p,
                                         _c_sz, _c_p, _c_p, _c_i, _c_p, _c_sz, _c_p]),
    "mot_qk_norm_rope_backward_fp32": (_c_i, [_c_p, _c_p, _c_p, _c_p, _c_p, _c_p, _c_i, _c_i64, _c_i, _c_i, _c_i, _c_f,
                                              _c_p, _c_sz, _c_p, _c_p, _c_i, _c_p, _c_sz, _c_p]),
    "mot_adamw_hyper_host": (_c_i, [ctypes.c_double, ctypes.c_double, ctypes.c_double, ctypes.c_double, ctypes.c_double,
                                    _c_i64, _c_p]),
    "mot_adamw_step": (_c_i, [_c_p, _c_i, _c_p, ctypes.c_uint64, _c_p, _c_sz, _c_p]),
    "mot_device_status": (_c_i, [_c_p, ctypes.POINTER(ctypes.c_uint32), _c_p]),
}


class MotError(RuntimeError):
    """A nonzero status returned by libmot.so."""

    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed with status {status}: {_lib().mot_status_string(status).decode()}")


def library_path() -> str:
    return os.environ.get("MOT_LIBRARY", os.path.join(_PKG, "libmot.so"))


def load_library(path: str | None = None) -> ctypes.CDLL:
    """Loads libmot.so and declares its C signatures; raises if it is missing or stale."""
    path = path or library_path()
    if not os.path.exists(path):
        raise ImportError(f"{path} is not built; run `python -m mixture_transformers_token_gb300.build`")
    lib = ctypes.CDLL(path)
    for name, (res, args) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if lib.mot_abi_version() != ABI_VERSION:
        raise ImportError(f"{path} has ABI {lib.mot_abi_version()}, the binding expects {ABI_VERSION}")
    return lib


def _lib() -> ctypes.CDLL:
    global _LIB
    if _LIB is None:
        _LIB = load_library()
    return _LIB


def _check(fn: str, status: int) -> None:
    if status != 0:
        raise MotError(fn, status)


def _dev(t: torch.Tensor, name: str, dtype: torch.dtype, ndim: int | None = None) -> int:
    # the common case first: a call checks up to eight tensors
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.is_cuda and t.is_contiguous() and ndim == t.dim():
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dimensions, got {t.dim()}")
    return t.data_ptr()


# The current stream's handle without a Stream object around it (2 us less a call), where torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(t: torch.Tensor, stream) -> int:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(t.get_device())
        stream = torch.cuda.current_stream(t.device)
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _new(make, shape, dtype: torch.dtype, t: torch.Tensor, stream, kept: bool = True) -> torch.Tensor:
    """A buffer that the caller did not give, made by torch.empty or torch.zeros on t's device. Its memory belongs to the
    stream that the call is launched on, where it is filled too: made on the current one, its fill and what that stream
    still does with the memory would not be ordered before the call's kernels, nor the memory's next use after them.
    What the caller receives (`kept`; else the call's own, let go at its return) may be used on the current stream."""
    if stream is None or not t.is_cuda:
        return make(shape, dtype=dtype, device=t.device)
    current, handle = torch.cuda.current_stream(t.device), _stream(t, stream)
    if handle == current.cuda_stream:
        return make(shape, dtype=dtype, device=t.device)
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(handle, device=t.device) if handle else torch.cuda.default_stream(t.device)
    with torch.cuda.stream(stream):
        b = make(shape, dtype=dtype, device=t.device)
    if kept:
        b.record_stream(current)
    return b


# ---------------------------------------------------------------------------
# entry points
# ---------------------------------------------------------------------------

def mot_abi_version() -> int:
    return _lib().mot_abi_version()


def mot_status_string(status: int) -> str:
    return _lib().mot_status_string(status).decode()


def mot_workspace_bytes(T: int) -> int:
    return int(_lib().mot_workspace_bytes(T))


def mot_route_plan(mod: torch.Tensor, ws: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Builds the routing plan of `mod` in `ws` (allocated if None) and returns ws."""
    T = mod.numel()
    _dev(mod, "mod", torch.uint8, 1)
    if ws is None:
        ws = _new(torch.empty, (max(mot_workspace_bytes(T), 16),), torch.uint8, mod, stream)
    _dev(ws, "ws", torch.uint8, 1)
    _check("mot_route_plan", _lib().mot_route_plan(mod.data_ptr(), T, ws.data_ptr(), ws.numel(), _stream(mod, stream)))
    return ws


def mot_fused_add_rmsnorm(x, res, w, mod, eps: float, y=None, res_out=None, ws=None, stream=None):
    """Residual add and routed RMSNorm; returns (y, res_out). res_out may be res (in place).
    If `ws` is given, the same launch also writes the routing plan of `mod` into it."""
    T, H = x.shape
    if y is None:
        y = _new(torch.empty, (T, H), torch.bfloat16, x, stream)
    if res_out is None:
        res_out = _new(torch.empty, (T, H), torch.bfloat16, x, stream)
    for t, n in ((x, "x"), (res, "res"), (y, "y"), (res_out, "res_out")):
        _dev(t, n, torch.bfloat16, 2)
        if tuple(t.shape) != (T, H):
            raise ValueError(f"{n} must be [{T}, {H}]")
    _dev(w, "w", torch.bfloat16, 2)
    _dev(mod, "mod", torch.uint8, 1)
    if tuple(w.shape) != (2, H) or mod.numel() != T:
        raise ValueError("w must be [2, H] and mod [T]")
    wsp = _dev(ws, "ws", torch.uint8, 1) if ws is not None else None
    wsb = ws.numel() if ws is not None else 0
    _check("mot_fused_add_rmsnorm", _lib().mot_fused_add_rmsnorm(
        x.data_ptr(), res.data_ptr(), w.data_ptr(), mod.data_ptr(), T, H, eps, y.data_ptr(), res_out.data_ptr(),
        wsp, wsb, _stream(x, stream)))
    return y, res_out


def mot_routed_qkv_norm_rope(x, w_qkv, q_norm_w, k_norm_w, pos, rope_cs, Hq: int, Hkv: int, D: int, eps: float,
                             ws, b_qkv=None, out=None, stream=None):
    """Routed QKV GEMM + per-head QK RMSNorm + RoPE; `ws` must hold the plan for T rows.
    A bf16 `rope_cs` selects the BF16 RoPE profile (mot_routed_qkv_norm_rope), an fp32 one
    the FP32 profile (mot_routed_qkv_norm_rope_fp32)."""
    T, H = x.shape
    N = (Hq + 2 * Hkv) * D
    _dev(x, "x", torch.bfloat16, 2)
    _dev(w_qkv, "w_qkv", torch.bfloat16, 3)
    _dev(q_norm_w, "q_norm_w", torch.bfloat16, 2)
    _dev(k_norm_w, "k_norm_w", torch.bfloat16, 2)
    _dev(pos, "pos", torch.int32, 1)
    fp32 = rope_cs.dtype == torch.float32
    _dev(rope_cs, "rope_cs", torch.float32 if fp32 else torch.bfloat16, 3)
    _dev(ws, "ws", torch.uint8, 1)
    if tuple(w_qkv.shape) != (2, N, H):
        raise ValueError(f"w_qkv must be [2, {N}, {H}]")
    if tuple(q_norm_w.shape) != (2, D) or tuple(k_norm_w.shape) != (2, D) or pos.numel() != T:
        raise ValueError("q_norm_w/k_norm_w must be [2, D] and pos [T]")
    if rope_cs.shape[1:] != (D // 2, 2):
        raise ValueError("rope_cs must be [P, D/2, 2]")
    bp = None
    if b_qkv is not None:
        bp = _dev(b_qkv, "b_qkv", torch.bfloat16, 2)
        if tuple(b_qkv.shape) != (2, N):
            raise ValueError(f"b_qkv must be [2, {N}]")
    if out is None:
        out = _new(torch.empty, (T, N), torch.bfloat16, x, stream)
    _dev(out, "out", torch.bfloat16, 2)
    name = "mot_routed_qkv_norm_rope_fp32" if fp32 else "mot_routed_qkv_norm_rope"
    _check(name, getattr(_lib(), name)(
        x.data_ptr(), w_qkv.data_ptr(), bp, q_norm_w.data_ptr(), k_norm_w.data_ptr(), pos.data_ptr(),
        rope_cs.data_ptr(), rope_cs.shape[0], T, H, Hq, Hkv, D, eps, ws.data_ptr(), ws.numel(), out.data_ptr(),
        _stream(x, stream)))
    return out


def mot_routed_qkv_norm_rope_fp32(x, w_qkv, q_norm_w, k_norm_w, pos, rope_cs_f32, Hq: int, Hkv: int, D: int,
                                  eps: float, ws, b_qkv=None, out=None, stream=None):
    """The FP32 RoPE profile of mot_routed_qkv_norm_rope; `rope_cs_f32` is the fp32 table."""
    if rope_cs_f32.dtype != torch.float32:
        raise TypeError("rope_cs_f32 must be float32 (mot_rope_table_fill_host_fp32)")
    return mot_routed_qkv_norm_rope(x, w_qkv, q_norm_w, k_norm_w, pos, rope_cs_f32, Hq, Hkv, D, eps, ws,
                                    b_qkv=b_qkv, out=out, stream=stream)


def mot_routed_gemm(a, w, ws, epilogue: int = EPI_CAST, out=None, stream=None):
    """Routed GEMM: out[T][N] = bf16(a W^T) (cast) or out[T][N/2] = SwiGLU (interleaved gate/up w).
    `epilogue` may carry A_PLAN_ORDER / OUT_PLAN_ORDER (rows of a / out in the plan's order)."""
    T, K = a.shape
    _dev(a, "a", torch.bfloat16, 2)
    _dev(w, "w", torch.bfloat16, 3)
    _dev(ws, "ws", torch.uint8, 1)
    if w.shape[0] != 2 or w.shape[2] != K:
        raise ValueError("w must be [2, N, K]")
    N = w.shape[1]
    ncols = N // 2 if (epilogue & 0xFF) == EPI_SWIGLU else N
    if out is None:
        out = _new(torch.empty, (T, ncols), torch.bfloat16, a, stream)
    _dev(out, "out", torch.bfloat16, 2)
    if tuple(out.shape) != (T, ncols):
        raise ValueError(f"out must be [{T}, {ncols}]")
    _check("mot_routed_gemm", _lib().mot_routed_gemm(
        a.data_ptr(), w.data_ptr(), T, N, K, epilogue, ws.data_ptr(), ws.numel(), out.data_ptr(), _stream(a, stream)))
    return out


def mot_routed_gemm_noalloc(a, w, mod, epilogue: int = EPI_CAST, out=None, device_flags=None, stream=None):
    """mot_routed_gemm for callers that cannot allocate device memory: the routing plan is kept
    in the library's own fixed device array (T <= NOALLOC_MAX_TOKENS), so no workspace is
    passed. Calls whose work may overlap on the GPU share that array and must be ordered by
    the caller. `device_flags`, an optional int32 CUDA tensor of one element, receives the
    call's device error bits."""
    T, K = a.shape
    _dev(a, "a", torch.bfloat16, 2)
    _dev(w, "w", torch.bfloat16, 3)
    _dev(mod, "mod", torch.uint8, 1)
    if w.shape[0] != 2 or w.shape[2] != K or mod.numel() != T:
        raise ValueError("w must be [2, N, K] and mod [T]")
    N = w.shape[1]
    ncols = N // 2 if epilogue == EPI_SWIGLU else N
    if out is None:
        out = _new(torch.empty, (T, ncols), torch.bfloat16, a, stream)
    _dev(out, "out", torch.bfloat16, 2)
    fp = _dev(device_flags, "device_flags", torch.int32, 1) if device_flags is not None else None
    _check("mot_routed_gemm_noalloc", _lib().mot_routed_gemm_noalloc(
        a.data_ptr(), w.data_ptr(), mod.data_ptr(), T, N, K, epilogue, out.data_ptr(), fp, _stream(a, stream)))
    return out


def mot_gather_rows(src, ws, out=None, stream=None):
    """Rows of src [T][K] in the plan's order (und rows ascending, then gen rows)."""
    T, K = src.shape
    _dev(src, "src", torch.bfloat16, 2)
    _dev(ws, "ws", torch.uint8, 1)
    if out is None:
        out = _new(torch.empty, (T, K), torch.bfloat16, src, stream)
    _dev(out, "out", torch.bfloat16, 2)
    _check("mot_gather_rows", _lib().mot_gather_rows(src.data_ptr(), T, K, ws.data_ptr(), ws.numel(), out.data_ptr(),
                                                     _stream(src, stream)))
    return out


def mot_swiglu_interleave(w_gate, w_up, out=None, stream=None):
    """[2][I][K] gate and up weights -> [2][2I][K] interleaved in 128-row blocks."""
    _dev(w_gate, "w_gate", torch.bfloat16, 3)
    _dev(w_up, "w_up", torch.bfloat16, 3)
    _, I, K = w_gate.shape
    if tuple(w_up.shape) != (2, I, K):
        raise ValueError("w_up must match w_gate")
    if out is None:
        out = _new(torch.empty, (2, 2 * I, K), torch.bfloat16, w_gate, stream)
    _dev(out, "out", torch.bfloat16, 3)
    _check("mot_swiglu_interleave", _lib().mot_swiglu_interleave(
        w_gate.data_ptr(), w_up.data_ptr(), I, K, out.data_ptr(), _stream(w_gate, stream)))
    return out


def mot_routed_gemm_dx(dout, w, ws, flags: int = 0, out=None, stream=None):
    """Input gradient of the routed GEMM through both weight sets: dx[T][K] = bf16(dout W[mod]).
    `w` is the forward's [2][N][K] weight; `flags` may carry A_PLAN_ORDER / OUT_PLAN_ORDER."""
    T, N = dout.shape
    _dev(dout, "dout", torch.bfloat16, 2)
    _dev(w, "w", torch.bfloat16, 3)
    _dev(ws, "ws", torch.uint8, 1)
    if w.shape[0] != 2 or w.shape[1] != N:
        raise ValueError(f"w must be [2, {N}, K]")
    K = w.shape[2]
    if out is None:
        out = _new(torch.empty, (T, K), torch.bfloat16, dout, stream)
    _dev(out, "out", torch.bfloat16, 2)
    if tuple(out.shape) != (T, K):
        raise ValueError(f"out must be [{T}, {K}]")
    _check("mot_routed_gemm_dx", _lib().mot_routed_gemm_dx(
        dout.data_ptr(), w.data_ptr(), T, N, K, flags, ws.data_ptr(), ws.numel(), out.data_ptr(),
        _stream(dout, stream)))
    return out


def mot_routed_gemm_dw(dout, a, ws, expert: int = 1, flags: int = 0, out=None, stream=None):
    """Gradient [N][K] fp32 of weight set `expert` from dout [T][N] and a [T][K]: rows in token
    order, or in the plan's order with flags = A_PLAN_ORDER (the same bits either way)."""
    T, N = dout.shape
    _dev(dout, "dout", torch.bfloat16, 2)
    _dev(a, "a", torch.bfloat16, 2)
    _dev(ws, "ws", torch.uint8, 1)
    if a.shape[0] != T:
        raise ValueError("dout and a must have the same rows")
    K = a.shape[1]
    if out is None:
        out = _new(torch.empty, (N, K), torch.float32, dout, stream)
    _dev(out, "out", torch.float32, 2)
    if tuple(out.shape) != (N, K):
        raise ValueError(f"out must be [{N}, {K}]")
    _check("mot_routed_gemm_dw", _lib().mot_routed_gemm_dw(
        dout.data_ptr(), a.data_ptr(), T, N, K, expert, flags, ws.data_ptr(), ws.numel(), out.data_ptr(),
        _stream(dout, stream)))
    return out


def mot_joint_attention(qkv, seqs, Hq: int, Hkv: int, D: int, ws, scale: float | None = None, out=None,
                        stream=None):
    """Attention of packed sequences over the fused QKV output [T][(Hq + 2 Hkv) D].
    `seqs` is a device int32 [n_seq][5] of (q_start, k_start, nq, nk, n_causal); `ws` (>= 64
    bytes) receives device errors. Returns out [T][Hq D] (rows that are no query untouched)."""
    T = qkv.shape[0]
    _dev(qkv, "qkv", torch.bfloat16, 2)
    _dev(seqs, "seqs", torch.int32, 2)
    _dev(ws, "ws", torch.uint8, 1)
    if qkv.shape[1] != (Hq + 2 * Hkv) * D:
        raise ValueError(f"qkv must be [T, {(Hq + 2 * Hkv) * D}]")
    if seqs.shape[1] != 5:
        raise ValueError("seqs must be [n_seq, 5]")
    if out is None:
        out = _new(torch.zeros, (T, Hq * D), torch.bfloat16, qkv, stream)
    _dev(out, "out", torch.bfloat16, 2)
    sc = 1.0 / math.sqrt(D) if scale is None else float(scale)
    _check("mot_joint_attention", _lib().mot_joint_attention(
        qkv.data_ptr(), T, Hq, Hkv, D, seqs.data_ptr(), seqs.shape[0], sc, ws.data_ptr(), ws.numel(),
        out.data_ptr(), _stream(qkv, stream)))
    return out


def mot_joint_attention_lse(qkv, seqs, Hq: int, Hkv: int, D: int, ws, scale: float | None = None, out=None, lse=None,
                            stream=None):
    """mot_joint_attention that also returns lse [Hq][T] fp32, the natural log of each query row's softmax sum, for
    mot_joint_attention_backward: (out, lse)."""
    qp = _dev(qkv, "qkv", torch.bfloat16, 2)
    sp = _dev(seqs, "seqs", torch.int32, 2)
    wp = _dev(ws, "ws", torch.uint8, 1)
    T, N = qkv.shape
    if N != (Hq + 2 * Hkv) * D:
        raise ValueError(f"qkv must be [T, {(Hq + 2 * Hkv) * D}]")
    if seqs.shape[1] != 5:
        raise ValueError("seqs must be [n_seq, 5]")
    if out is None:
        out = _new(torch.zeros, (T, Hq * D), torch.bfloat16, qkv, stream)
    if lse is None:
        lse = _new(torch.zeros, (Hq, T), torch.float32, qkv, stream)
    op = _dev(out, "out", torch.bfloat16, 2)
    lp = _dev(lse, "lse", torch.float32, 2)
    if out.shape != (T, Hq * D) or lse.shape != (Hq, T):
        raise ValueError(f"out must be [{T}, {Hq * D}] and lse [{Hq}, {T}]")
    sc = 1.0 / math.sqrt(D) if scale is None else float(scale)
    _check("mot_joint_attention_lse", _lib().mot_joint_attention_lse(
        qp, T, Hq, Hkv, D, sp, seqs.shape[0], sc, wp, ws.numel(), op, lp, _stream(qkv, stream)))
    return out, lse


def mot_joint_attention_backward_workspace_bytes(T: int, Hq: int, Hkv: int, D: int, n_seq: int) -> int:
    return int(_lib().mot_joint_attention_backward_workspace_bytes(T, Hq, Hkv, D, n_seq))


def mot_joint_attention_backward(dout, qkv, out, lse, seqs, Hq: int, Hkv: int, D: int, ws, scale: float | None = None,
                                 dqkv=None, stream=None):
    """Gradient of mot_joint_attention with respect to qkv, from dout and out [T][Hq D], qkv and the lse of
    mot_joint_attention_lse, over the same seqs. `ws` (>= mot_joint_attention_backward_workspace_bytes) is scratch after
    its 64-byte header. Returns dqkv [T][(Hq + 2 Hkv) D] bf16 (what is no sequence's query or key: left as it is, zeros
    if dqkv is None)."""
    dp = _dev(dout, "dout", torch.bfloat16, 2)
    qp = _dev(qkv, "qkv", torch.bfloat16, 2)
    op = _dev(out, "out", torch.bfloat16, 2)
    lp = _dev(lse, "lse", torch.float32, 2)
    sp = _dev(seqs, "seqs", torch.int32, 2)
    wp = _dev(ws, "ws", torch.uint8, 1)
    T, N = qkv.shape
    if N != (Hq + 2 * Hkv) * D:
        raise ValueError(f"qkv must be [T, {(Hq + 2 * Hkv) * D}]")
    if dout.shape != (T, Hq * D) or out.shape != (T, Hq * D) or lse.shape != (Hq, T):
        raise ValueError(f"dout and out must be [{T}, {Hq * D}] and lse [{Hq}, {T}]")
    if seqs.shape[1] != 5:
        raise ValueError("seqs must be [n_seq, 5]")
    if dqkv is None:
        dqkv = _new(torch.zeros, (T, N), torch.bfloat16, qkv, stream)
    gp = _dev(dqkv, "dqkv", torch.bfloat16, 2)
    if dqkv.shape != (T, N):
        raise ValueError(f"dqkv must be [{T}, {N}]")
    sc = 1.0 / math.sqrt(D) if scale is None else float(scale)
    _check("mot_joint_attention_backward", _lib().mot_joint_attention_backward(
        dp, qp, op, lp, T, Hq, Hkv, D, sp, seqs.shape[0], sc, wp, ws.numel(), gp, _stream(qkv, stream)))
    return dqkv


def mot_qk_norm_rope_backward_workspace_bytes(T: int, D: int) -> int:
    return int(_lib().mot_qk_norm_rope_backward_workspace_bytes(T, D))


def mot_qk_norm_rope_backward(d_out, x, q_norm_w, k_norm_w, pos, rope_cs, Hq: int, Hkv: int, D: int, eps: float, ws,
                              dx=None, dw=None, sets: int = SET_BOTH, scratch=None, stream=None):
    """Gradient through the epilogue of mot_routed_qkv_norm_rope: from d_out [T][(Hq + 2 Hkv) D] (gradient of its
    output) and x, the projection's rows before the norm, the gradient dx of x (may be d_out: in place) and the norm
    weights' gradients dw [2 (q, k)][2 (und, gen)][D] fp32 of the weight sets in `sets` (0: none, dw is None).
    `ws` holds the plan, `scratch` (>= mot_qk_norm_rope_backward_workspace_bytes, allocated if None) is overwritten.
    A bf16 `rope_cs` is the BF16 RoPE profile's, an fp32 one the FP32 profile's. Returns (dx, dw)."""
    dp = _dev(d_out, "d_out", torch.bfloat16, 2)
    xp = _dev(x, "x", torch.bfloat16, 2)
    qp = _dev(q_norm_w, "q_norm_w", torch.bfloat16, 2)
    kp = _dev(k_norm_w, "k_norm_w", torch.bfloat16, 2)
    pp = _dev(pos, "pos", torch.int32, 1)
    fp32 = getattr(rope_cs, "dtype", None) is torch.float32  # _dev refuses what is no tensor
    cp = _dev(rope_cs, "rope_cs", torch.float32 if fp32 else torch.bfloat16, 3)
    wp = _dev(ws, "ws", torch.uint8, 1)
    T, N = d_out.shape
    if N != (Hq + 2 * Hkv) * D or x.shape != (T, N):
        raise ValueError(f"d_out and x must be [T, {(Hq + 2 * Hkv) * D}]")
    if q_norm_w.shape != (2, D) or k_norm_w.shape != (2, D) or pos.shape[0] != T:
        raise ValueError("q_norm_w/k_norm_w must be [2, D] and pos [T]")
    if rope_cs.shape[1:] != (D // 2, 2):
        raise ValueError("rope_cs must be [P, D/2, 2]")
    if dx is None:
        dx = _new(torch.empty, (T, N), torch.bfloat16, d_out, stream)
    gp = _dev(dx, "dx", torch.bfloat16, 2)
    if dx.shape != (T, N):
        raise ValueError(f"dx must be [{T}, {N}]")
    wgp = sp = None
    sb = 0
    if sets != 0:
        if dw is None:
            dw = _new(torch.zeros, (2, 2, D), torch.float32, d_out, stream)
        wgp = _dev(dw, "dw", torch.float32, 3)
        if dw.shape != (2, 2, D):
            raise ValueError(f"dw must be [2, 2, {D}]")
        if scratch is None:
            scratch = _new(torch.empty, (max(mot_qk_norm_rope_backward_workspace_bytes(T, D), 16),), torch.uint8, d_out,
                           stream, kept=False)
        sp = _dev(scratch, "scratch", torch.uint8, 1)
        sb = scratch.numel()
    elif dw is not None:
        raise ValueError("dw is given but sets is 0")
    name = "mot_qk_norm_rope_backward_fp32" if fp32 else "mot_qk_norm_rope_backward"
    _check(name, getattr(_lib(), name)(
        dp, xp, qp, kp, pp, cp, rope_cs.shape[0], T, Hq, Hkv, D, eps, wp, ws.numel(), gp, wgp, sets, sp, sb,
        _stream(d_out, stream)))
    return dx, dw


def mot_qk_norm_rope_backward_fp32(d_out, x, q_norm_w, k_norm_w, pos, rope_cs_f32, Hq: int, Hkv: int, D: int, eps: float,
                                   ws, dx=None, dw=None, sets: int = SET_BOTH, scratch=None, stream=None):
    """The FP32 RoPE profile of mot_qk_norm_rope_backward; `rope_cs_f32` is the fp32 table."""
    if getattr(rope_cs_f32, "dtype", None) is not torch.float32:
        raise TypeError("rope_cs_f32 must be float32 (mot_rope_table_fill_host_fp32)")
    return mot_qk_norm_rope_backward(d_out, x, q_norm_w, k_norm_w, pos, rope_cs_f32, Hq, Hkv, D, eps, ws, dx=dx, dw=dw,
                                     sets=sets, scratch=scratch, stream=stream)


class _AdamWTensor(ctypes.Structure):
    _fields_ = [("p", _c_p), ("p16", _c_p), ("g", _c_p), ("m", _c_p), ("v", _c_p), ("scales", _c_p), ("n", _c_i64),
                ("weight_decay", _c_f), ("flags", ctypes.c_int32)]


class AdamWTensors:
    """The tensors of mot_adamw_step, checked once; keeps them alive. Lists of equal length, one entry a tensor (any
    shape; only the number of elements counts):
      params  fp32 weights, updated.            grads   fp32 or bf16.
      m, v    states, updated: fp32, or float8_e4m3fn codes of m and sqrt(v) with `scales`.
      p16     bf16 copies of the weights that the step writes, or None (also as an entry).
      scales  fp32 [ceil(n / ADAMW_BLOCK)][2] for 8-bit states (zeros to begin with, as m and v).
      weight_decay  a number, or one a tensor.
    The entries are slices like w[1] of a [2][N][K] weight as well as whole tensors."""

    def __init__(self, params, grads, m, v, p16=None, scales=None, weight_decay=0.0):
        n = len(params)
        p16 = [None] * n if p16 is None else p16
        scales = [None] * n if scales is None else scales
        decay = [float(weight_decay)] * n if isinstance(weight_decay, (int, float)) else [float(x) for x in weight_decay]
        if not n or any(len(x) != n for x in (grads, m, v, p16, scales, decay)):
            raise ValueError("the lists must have one entry for each parameter, at least one")
        self.table = (_AdamWTensor * n)()
        for i in range(n):
            e = self.table[i]
            e.p = _dev_any(params[i], f"params[{i}]", torch.float32)
            e.n = params[i].numel()
            bf16 = getattr(grads[i], "dtype", None) is torch.bfloat16
            e.g = _dev_any(grads[i], f"grads[{i}]", torch.bfloat16 if bf16 else torch.float32)
            e4m3 = getattr(m[i], "dtype", None) is torch.float8_e4m3fn
            state = torch.float8_e4m3fn if e4m3 else torch.float32
            e.m = _dev_any(m[i], f"m[{i}]", state)
            e.v = _dev_any(v[i], f"v[{i}]", state)
            sizes = [grads[i].numel(), m[i].numel(), v[i].numel()]
            if p16[i] is not None:
                e.p16 = _dev_any(p16[i], f"p16[{i}]", torch.bfloat16)
                sizes.append(p16[i].numel())
            if any(x != e.n for x in sizes):
                raise ValueError(f"grads, m, v and p16 of tensor {i} must have its {e.n} elements")
            if e4m3:
                e.scales = _dev_any(scales[i], f"scales[{i}]", torch.float32)
                if scales[i].numel() != 2 * -(-e.n // ADAMW_BLOCK):
                    raise ValueError(f"scales[{i}] must be [{-(-e.n // ADAMW_BLOCK)}, 2]")
            e.weight_decay = decay[i]
            e.flags = (_ADAMW_GRAD_BF16 if bf16 else 0) | (_ADAMW_STATE_E4M3 if e4m3 else 0)
        self.tensors = (list(params), list(grads), list(m), list(v), list(p16), list(scales))
        self.address = ctypes.addressof(self.table)

    def __len__(self):
        return len(self.table)


def _dev_any(t, name: str, dtype: torch.dtype) -> int:
    """_dev for a tensor of any rank."""
    return _dev(t, name, dtype, t.dim() if isinstance(t, torch.Tensor) else None)


def mot_adamw_hyper_host(lr: float, beta1: float, beta2: float, eps: float, step: int, grad_scale: float = 1.0) -> torch.Tensor:
    """The numbers of AdamW step `step` (from 1) as a CPU fp32 tensor [16]: copy it to the device, or a table of them."""
    t = torch.empty((_ADAMW_HYPER_WORDS,), dtype=torch.float32)
    _check("mot_adamw_hyper_host", _lib().mot_adamw_hyper_host(lr, beta1, beta2, eps, grad_scale, step, t.data_ptr()))
    return t


def mot_adamw_step(tensors: AdamWTensors, hyper, ws, seed: int = 0, stream=None) -> None:
    """One AdamW step of all `tensors`, in place. `hyper` is a device fp32 row [16] of mot_adamw_hyper_host, `ws` (>= 64
    bytes) receives DEV_BAD_HYPER (then nothing is updated), `seed` is that of the 8-bit states' rounding."""
    if not isinstance(tensors, AdamWTensors):
        raise TypeError("tensors must be AdamWTensors")
    hp = _dev(hyper, "hyper", torch.float32, 1)
    if hyper.shape[0] != _ADAMW_HYPER_WORDS:
        raise ValueError(f"hyper must be [{_ADAMW_HYPER_WORDS}]")
    wp = _dev(ws, "ws", torch.uint8, 1)
    _check("mot_adamw_step", _lib().mot_adamw_step(tensors.address, len(tensors.table), hp, int(seed) & (2 ** 64 - 1), wp,
                                                   ws.numel(), _stream(hyper, stream)))


def _kv_cache(k_cache, v_cache, scales):
    """Checks a cache's tensors: (kv_type, n_pages, Hkv, page, D, the three pointers; no scales: None)."""
    e4m3 = getattr(k_cache, "dtype", None) is torch.float8_e4m3fn  # _dev refuses what is no tensor
    dtype = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    kp = _dev(k_cache, "k_cache", dtype, 4)
    vp = _dev(v_cache, "v_cache", dtype, 4)
    shape = k_cache.shape
    if v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must have the same shape")
    n_pages, Hkv, page, D = shape
    if not e4m3:
        return KV_BF16, n_pages, Hkv, page, D, kp, vp, None
    if scales is None:
        raise ValueError("an e4m3 cache needs its scales")
    sp = _dev(scales, "scales", torch.float32, 4)
    if scales.shape != (n_pages, Hkv, page, 2):
        raise ValueError(f"scales must be [{n_pages}, {Hkv}, {page}, 2]")
    return KV_E4M3, n_pages, Hkv, page, D, kp, vp, sp


def _kv_rows(qkv, slots, Hq: int, Hkv: int, D: int):
    qp = _dev(qkv, "qkv", torch.bfloat16, 2)
    lp = _dev(slots, "slots", torch.int32, 1)
    T, N = qkv.shape
    if N != (Hq + 2 * Hkv) * D or slots.shape[0] != T:
        raise ValueError(f"qkv must be [T, {(Hq + 2 * Hkv) * D}] and slots [T]")
    return T, qp, lp


def mot_kv_cache_write(qkv, slots, k_cache, v_cache, Hq: int, ws, scales=None, stream=None) -> None:
    """Writes the K and V columns of the fused QKV rows [T][(Hq + 2 Hkv) D] into the cache's slots
    (int32 [T], -1: skip the row). The cache [n_pages][Hkv][page][D] is bf16, or float8_e4m3fn with
    fp32 `scales` [n_pages][Hkv][page][2]. `ws` (>= 64 bytes) receives device errors."""
    kt, n_pages, Hkv, page, D, kp, vp, sp = _kv_cache(k_cache, v_cache, scales)
    T, qp, lp = _kv_rows(qkv, slots, Hq, Hkv, D)
    wp = _dev(ws, "ws", torch.uint8, 1)
    _check("mot_kv_cache_write", _lib().mot_kv_cache_write(
        qp, T, Hq, Hkv, D, lp, kt, n_pages, page, kp, vp, sp, wp, ws.numel(), _stream(qkv, stream)))


def mot_kv_cache_read(k_cache, v_cache, slots, qkv, Hq: int, ws, scales=None, stream=None):
    """Reads cached vectors back into the K and V columns of the fused QKV rows `qkv` (the q columns
    and rows with slot -1 are kept). Arguments as mot_kv_cache_write; returns qkv."""
    kt, n_pages, Hkv, page, D, kp, vp, sp = _kv_cache(k_cache, v_cache, scales)
    T, qp, lp = _kv_rows(qkv, slots, Hq, Hkv, D)
    wp = _dev(ws, "ws", torch.uint8, 1)
    _check("mot_kv_cache_read", _lib().mot_kv_cache_read(
        kp, vp, sp, kt, n_pages, page, lp, T, Hq, Hkv, D, qp, wp, ws.numel(), _stream(qkv, stream)))
    return qkv


def mot_paged_decode_workspace_bytes(R: int, Hq: int, Hkv: int, D: int, max_pages: int, page: int) -> int:
    return int(_lib().mot_paged_decode_workspace_bytes(R, Hq, Hkv, D, max_pages, page))


def mot_paged_decode_attention(qkv, table, lens, k_cache, v_cache, Hq: int, ws, scales=None, scale: float | None = None,
                               out=None, stream=None):
    """Attention of one new token a row over its pages: the q heads of the fused QKV rows [R][(Hq + 2
    Hkv) D], page table int32 [R][max_pages], lens int32 [R] (0: a row of zeros), the cache as for
    mot_kv_cache_write. `ws` (>= mot_paged_decode_workspace_bytes) is scratch after its 64-byte header.
    Returns out [R][Hq D] bf16."""
    kt, n_pages, Hkv, page, D, kp, vp, sp = _kv_cache(k_cache, v_cache, scales)
    qp = _dev(qkv, "qkv", torch.bfloat16, 2)
    tp = _dev(table, "table", torch.int32, 2)
    lp = _dev(lens, "lens", torch.int32, 1)
    wp = _dev(ws, "ws", torch.uint8, 1)
    R, N = qkv.shape
    if N != (Hq + 2 * Hkv) * D:
        raise ValueError(f"qkv must be [R, {(Hq + 2 * Hkv) * D}]")
    max_pages = table.shape[1]
    if table.shape[0] != R or lens.shape[0] != R:
        raise ValueError("table must be [R, max_pages] and lens [R]")
    if out is None:
        out = _new(torch.empty, (R, Hq * D), torch.bfloat16, qkv, stream)
    op = _dev(out, "out", torch.bfloat16, 2)
    if out.shape != (R, Hq * D):
        raise ValueError(f"out must be [{R}, {Hq * D}]")
    sc = 1.0 / math.sqrt(D) if scale is None else float(scale)
    _check("mot_paged_decode_attention", _lib().mot_paged_decode_attention(
        qp, R, Hq, Hkv, D, tp, lp, max_pages, kt, n_pages, page, kp, vp, sp, sc, wp, ws.numel(), op,
        _stream(qkv, stream)))
    return out


def mot_add_rmsnorm_backward(dy, s, w, eps: float, ws, d_res_out=None, dx=None, rstd=None, dw_partials=None,
                             partial_sets: int = SET_BOTH, stream=None):
    """Input gradient of the fused add-RMSNorm: returns (dx [T][H] bf16, rstd [T] fp32).
    `s` is the forward's res_out and `ws` holds the routing plan of the forward's mod. If
    `dw_partials` (fp32 [H/64][T][64]) is given, the per-row weight-gradient partials of the
    rows of the weight sets in `partial_sets` are written there in the plan's row order."""
    T, H = dy.shape
    _dev(dy, "dy", torch.bfloat16, 2)
    _dev(s, "s", torch.bfloat16, 2)
    _dev(w, "w", torch.bfloat16, 2)
    _dev(ws, "ws", torch.uint8, 1)
    if tuple(s.shape) != (T, H) or tuple(w.shape) != (2, H):
        raise ValueError("s must be [T, H] and w [2, H]")
    rp = None
    if d_res_out is not None:
        _dev(d_res_out, "d_res_out", torch.bfloat16, 2)
        if tuple(d_res_out.shape) != (T, H):
            raise ValueError("d_res_out must be [T, H]")
        rp = d_res_out.data_ptr()
    pp = None
    if dw_partials is not None:
        _dev(dw_partials, "dw_partials", torch.float32, 3)
        if tuple(dw_partials.shape) != (H // 64, T, 64):
            raise ValueError(f"dw_partials must be [{H // 64}, {T}, 64]")
        pp = dw_partials.data_ptr()
    if dx is None:
        dx = _new(torch.empty, (T, H), torch.bfloat16, dy, stream)
    if rstd is None:
        rstd = _new(torch.empty, (T,), torch.float32, dy, stream)
    _dev(dx, "dx", torch.bfloat16, 2)
    _dev(rstd, "rstd", torch.float32, 1)
    _check("mot_add_rmsnorm_backward", _lib().mot_add_rmsnorm_backward(
        dy.data_ptr(), rp, s.data_ptr(), w.data_ptr(), T, H, eps, ws.data_ptr(), ws.numel(), dx.data_ptr(),
        rstd.data_ptr(), pp, partial_sets, _stream(dy, stream)))
    return dx, rstd


def mot_rmsnorm_dweight(dw_partials, ws, dw=None, sets: int = SET_BOTH, stream=None):
    """Gradient of the norm weight sets in `sets`, rows of dw [2][H] fp32: the ascending-row fp32
    left fold of the partials of mot_add_rmsnorm_backward over each set's rows (the other set's
    row of dw is left as it is)."""
    nb, T, c64 = dw_partials.shape
    _dev(dw_partials, "dw_partials", torch.float32, 3)
    _dev(ws, "ws", torch.uint8, 1)
    if c64 != 64:
        raise ValueError("dw_partials must be [H/64, T, 64]")
    H = nb * 64
    if dw is None:
        dw = _new(torch.empty, (2, H), torch.float32, dw_partials, stream)
    _dev(dw, "dw", torch.float32, 2)
    _check("mot_rmsnorm_dweight", _lib().mot_rmsnorm_dweight(
        dw_partials.data_ptr(), T, H, sets, ws.data_ptr(), ws.numel(), dw.data_ptr(), _stream(dw_partials, stream)))
    return dw


def mot_rope_table_fill_host(theta: float, D: int, P: int) -> torch.Tensor:
    """Host (cos, sin) table [P][D/2][2] as a CPU bf16 tensor (copy it to the device once)."""
    t = torch.empty((P, D // 2, 2), dtype=torch.bfloat16)
    _check("mot_rope_table_fill_host", _lib().mot_rope_table_fill_host(theta, D, P, t.data_ptr()))
    return t


def mot_rope_table_fill_host_fp32(theta: float, D: int, P: int) -> torch.Tensor:
    """Host fp32 (cos, sin) table [P][D/2][2] of the FP32 RoPE profile, as a CPU tensor."""
    t = torch.empty((P, D // 2, 2), dtype=torch.float32)
    _check("mot_rope_table_fill_host_fp32", _lib().mot_rope_table_fill_host_fp32(theta, D, P, t.data_ptr()))
    return t


def mot_flow_workspace_bytes(n_req: int, N: int) -> int:
    return int(_lib().mot_flow_workspace_bytes(n_req, N))


def mot_flow_schedule_host(n: int, shift: float) -> torch.Tensor:
    """The sampler's n step times from 1 down to 0 (built in double, stored fp32), a CPU tensor."""
    t = torch.empty((n,), dtype=torch.float32)
    _check("mot_flow_schedule_host", _lib().mot_flow_schedule_host(n, shift, t.data_ptr()))
    return t


def _flow_ws(ws, n_req: int, N: int, t: torch.Tensor, stream) -> torch.Tensor:
    if ws is None:
        ws = _new(torch.zeros, (max(mot_flow_workspace_bytes(n_req, N), 64),), torch.uint8, t, stream, kept=False)
    _dev(ws, "ws", torch.uint8, 1)
    return ws


def mot_cfg_combine_renorm(v_c, v_tu, v_iu, policy, ws=None, out=None, stream=None):
    """Three-branch renormalised CFG per request: v_c, v_tu, v_iu (or None) [n_req][N] bf16,
    policy a device fp32 [n_req][6] of (t, s_text, s_img, t_lo, t_hi, renorm_min). `ws` (>=
    mot_flow_workspace_bytes) is scratch after its 64-byte header. Returns out [n_req][N] fp32."""
    n_req, N = v_c.shape
    _dev(v_c, "v_c", torch.bfloat16, 2)
    _dev(v_tu, "v_tu", torch.bfloat16, 2)
    ip = None
    if v_iu is not None:
        _dev(v_iu, "v_iu", torch.bfloat16, 2)
        ip = v_iu.data_ptr()
    _dev(policy, "policy", torch.float32, 2)
    if tuple(v_tu.shape) != (n_req, N) or (v_iu is not None and tuple(v_iu.shape) != (n_req, N)):
        raise ValueError("the branches must all be [n_req, N]")
    if tuple(policy.shape) != (n_req, 6):
        raise ValueError("policy must be [n_req, 6]")
    ws = _flow_ws(ws, n_req, N, v_c, stream)
    if out is None:
        out = _new(torch.empty, (n_req, N), torch.float32, v_c, stream)
    _dev(out, "out", torch.float32, 2)
    _check("mot_cfg_combine_renorm", _lib().mot_cfg_combine_renorm(
        v_c.data_ptr(), v_tu.data_ptr(), ip, n_req, N, policy.data_ptr(), ws.data_ptr(), ws.numel(),
        out.data_ptr(), _stream(v_c, stream)))
    return out


def mot_flow_sde_step(x, v, z, times, ws=None, x_next=None, logp=None, stream=None):
    """One reverse-SDE step per request and its log-probability: x, v, z [n_req][N] fp32, times
    a device fp32 [n_req][2] of (t_i, t_next). With z None, x_next must be given and is scored
    instead of sampled. `ws`'s error word receives DEV_BAD_TIME. Returns (x_next, logp [n_req])."""
    n_req, N = x.shape
    _dev(x, "x", torch.float32, 2)
    _dev(v, "v", torch.float32, 2)
    _dev(times, "times", torch.float32, 2)
    if tuple(v.shape) != (n_req, N) or tuple(times.shape) != (n_req, 2):
        raise ValueError("v must be [n_req, N] and times [n_req, 2]")
    zp = None
    if z is not None:
        _dev(z, "z", torch.float32, 2)
        if tuple(z.shape) != (n_req, N):
            raise ValueError("z must be [n_req, N]")
        zp = z.data_ptr()
    elif x_next is None:
        raise ValueError("either z or x_next must be given")
    ws = _flow_ws(ws, n_req, N, x, stream)
    if x_next is None:
        x_next = _new(torch.empty, (n_req, N), torch.float32, x, stream)
    _dev(x_next, "x_next", torch.float32, 2)
    if tuple(x_next.shape) != (n_req, N):
        raise ValueError("x_next must be [n_req, N]")
    if logp is None:
        logp = _new(torch.empty, (n_req,), torch.float32, x, stream)
    _dev(logp, "logp", torch.float32, 1)
    _check("mot_flow_sde_step", _lib().mot_flow_sde_step(
        x.data_ptr(), v.data_ptr(), zp, x_next.data_ptr(), n_req, N, times.data_ptr(), ws.data_ptr(), ws.numel(),
        logp.data_ptr(), _stream(x, stream)))
    return x_next, logp


def mot_flow_cfg_sde_step(v_c, v_tu, v_iu, policy, x, z, times, ws=None, x_next=None, v_out=None, logp=None,
                          stream=None):
    """CFG combine + renorm and the SDE step in one call, without writing the guided velocity:
    the branches and policy as for mot_cfg_combine_renorm, x, z, times as for mot_flow_sde_step
    (z None: x_next is given and scored). v_out, if given ([n_req][N] fp32), receives the guided
    velocity. Returns (x_next, logp), bit for bit those of the two calls in sequence."""
    n_req, N = v_c.shape
    _dev(v_c, "v_c", torch.bfloat16, 2)
    _dev(v_tu, "v_tu", torch.bfloat16, 2)
    ip = None
    if v_iu is not None:
        _dev(v_iu, "v_iu", torch.bfloat16, 2)
        ip = v_iu.data_ptr()
    _dev(policy, "policy", torch.float32, 2)
    _dev(x, "x", torch.float32, 2)
    _dev(times, "times", torch.float32, 2)
    if tuple(v_tu.shape) != (n_req, N) or (v_iu is not None and tuple(v_iu.shape) != (n_req, N)) \
            or tuple(x.shape) != (n_req, N):
        raise ValueError("the branches and x must all be [n_req, N]")
    if tuple(policy.shape) != (n_req, 6) or tuple(times.shape) != (n_req, 2):
        raise ValueError("policy must be [n_req, 6] and times [n_req, 2]")
    zp = None
    if z is not None:
        _dev(z, "z", torch.float32, 2)
        if tuple(z.shape) != (n_req, N):
            raise ValueError("z must be [n_req, N]")
        zp = z.data_ptr()
    elif x_next is None:
        raise ValueError("either z or x_next must be given")
    ws = _flow_ws(ws, n_req, N, x, stream)
    if x_next is None:
        x_next = _new(torch.empty, (n_req, N), torch.float32, x, stream)
    _dev(x_next, "x_next", torch.float32, 2)
    if tuple(x_next.shape) != (n_req, N):
        raise ValueError("x_next must be [n_req, N]")
    vp = None
    if v_out is not None:
        _dev(v_out, "v_out", torch.float32, 2)
        if tuple(v_out.shape) != (n_req, N):
            raise ValueError("v_out must be [n_req, N]")
        vp = v_out.data_ptr()
    if logp is None:
        logp = _new(torch.empty, (n_req,), torch.float32, x, stream)
    _dev(logp, "logp", torch.float32, 1)
    _check("mot_flow_cfg_sde_step", _lib().mot_flow_cfg_sde_step(
        v_c.data_ptr(), v_tu.data_ptr(), ip, policy.data_ptr(), x.data_ptr(), zp, x_next.data_ptr(), n_req, N,
        times.data_ptr(), ws.data_ptr(), ws.numel(), vp, logp.data_ptr(), _stream(x, stream)))
    return x_next, logp


def mot_flow_noise(seeds, step: int, N: int, z=None, stream=None):
    """Per-sample standard normal noise [n_req][N] fp32 of sampler step `step`: `seeds` is a
    device int64 tensor [n_req] (reinterpreted as uint64), one seed per request."""
    _dev(seeds, "seeds", torch.int64, 1)
    n_req = seeds.shape[0]
    if z is None:
        z = _new(torch.empty, (n_req, N), torch.float32, seeds, stream)
    _dev(z, "z", torch.float32, 2)
    if tuple(z.shape) != (n_req, N):
        raise ValueError(f"z must be [{n_req}, {N}]")
    _check("mot_flow_noise", _lib().mot_flow_noise(seeds.data_ptr(), int(step) & (2 ** 64 - 1), n_req, N,
                                                   z.data_ptr(), _stream(seeds, stream)))
    return z


def mot_selftest_wait_timeout(ws, stream=None) -> None:
    """Runs a bounded wait that nothing satisfies; afterwards ws's error word has DEV_TIMEOUT."""
    _dev(ws, "ws", torch.uint8, 1)
    _check("mot_selftest_wait_timeout", _lib().mot_selftest_wait_timeout(ws.data_ptr(), ws.numel(), _stream(ws, stream)))


def mot_device_status(ws, stream=None) -> int:
    """Synchronizes the stream and returns the workspace's device error bits (0 = clean)."""
    _dev(ws, "ws", torch.uint8, 1)
    flags = ctypes.c_uint32(0)
    _check("mot_device_status", _lib().mot_device_status(ws.data_ptr(), ctypes.byref(flags), _stream(ws, stream)))
    return int(flags.value)
