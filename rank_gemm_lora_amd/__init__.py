"""Python binding of liblora_mi355x.so, the fused LoRA linear for MI355X (gfx950).

Argument marshalling only: every step of the computation runs in the HIP
kernels behind the C-ABI declared in ``include/lora_mi355x.h``. PyTorch is used
for device memory and streams (tensor ``data_ptr()`` and the current HIP
stream), nothing else. There is no CPU fallback: importing this package
without the built library raises.

Low-level functions carry the C names and take plain integers for pointers:
``lora_linear_fwd``, ``lora_linear_stacked_fwd``, ``lora_linear_nf4_fwd`` (and
``lora_linear_nf4_fwd_ex``, which names where the 4-bit weight is dequantized),
``lora_linear_routed_fwd``, ``lora_linear_routed_bwd``, ``lora_adamw_plan``,
``lora_adamw_step``, ``dense_patch_apply``, ``lora_linear_workspace_size``, ``lora_status_string``,
``lora_device_check``. Tensor-level helpers (``lora_linear``,
``lora_linear_stacked``, ``lora_linear_nf4``, ``lora_linear_routed``,
``lora_linear_routed_backward``, ``dense_patch``) check that the tensors sit on
one device, allocate the output and workspace with torch when not given, and
call the C functions on the current stream. ``LoraAdamW`` holds the moments and
the plan of ``lora_adamw_step``.
"""
from __future__ import annotations

import contextlib
import ctypes
import os

import torch  # loads the HIP runtime this library binds to (one runtime per process)

__all__ = [
    "LIB_PATH", "LoraError", "LORA_F32", "LORA_BF16", "LORA_LOSSLESS", "LORA_EXACT",
    "LORA_PATCH_ADD", "LORA_PATCH_REPLACE", "lora_linear_fwd", "lora_linear_stacked_fwd",
    "lora_linear_nf4_fwd", "lora_linear_nf4_fwd_ex", "LORA_NF4_AUTO", "LORA_NF4_PANEL", "LORA_NF4_IN_GEMM",
    "dense_patch_apply", "lora_linear_fwd_phase", "lora_linear_workspace_size",
    "lora_linear_nf4_workspace_size", "lora_linear_multi_fwd", "lora_linear_multi_workspace_size",
    "lora_linear_multi", "LoraAdapter", "lora_merge_apply", "lora_merge", "lora_linear_bwd",
    "lora_linear_bwd_workspace_size", "lora_linear_backward",
    "lora_status_string",
    "lora_device_check", "lora_mfma_probe", "lora_linear_fwd_noalloc", "LORA_NOALLOC_SCRATCH_BYTES", "lora_linear", "lora_linear_stacked", "lora_linear_nf4", "dense_patch",
    "LoraGroup", "hip_runtimes_mapped",
    "LoraPool", "lora_linear_routed_fwd", "lora_linear_routed_workspace_size", "lora_linear_routed_bwd",
    "lora_linear_routed_bwd_workspace_size", "lora_linear_routed", "lora_linear_routed_backward",
    "LoraAdamWTensor", "LoraAdamWPlan", "lora_adamw_table_size", "lora_adamw_plan", "lora_adamw_step", "LoraAdamW",
]

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "liblora_mi355x.so")

LORA_F32, LORA_BF16 = 0, 1
LORA_LOSSLESS, LORA_EXACT = 0, 1
LORA_PATCH_ADD, LORA_PATCH_REPLACE = 0, 1
LORA_NF4_AUTO, LORA_NF4_PANEL, LORA_NF4_IN_GEMM = 0, 1, 2
_DEQUANT = {"auto": LORA_NF4_AUTO, "panel": LORA_NF4_PANEL, "in_gemm": LORA_NF4_IN_GEMM}
_QUALITY = {"lossless": LORA_LOSSLESS, "exact": LORA_EXACT}
_MODE = {"add": LORA_PATCH_ADD, "replace": LORA_PATCH_REPLACE}

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is missing: build it with `python rank_gemm_lora_amd/_build.py` "
                      "(or __graft_entry__.build()); there is no fallback path")
_lib = ctypes.CDLL(LIB_PATH)

_p, _i64, _i32, _f64, _sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_double, ctypes.c_size_t


class LoraGroup(ctypes.Structure):
    """C ``lora_group``: one adapter of a stacked layer."""
    _fields_ = [("A", _p), ("B", _p), ("rank", _i32), ("reserved", _i32), ("alpha", _f64),
                ("col_offset", _i64), ("n_cols", _i64)]


class LoraAdapter(ctypes.Structure):
    """C ``lora_adapter``: one of several adapters on one layer."""
    _fields_ = [("A", _p), ("B", _p), ("B_bias", _p), ("rank", _i32), ("reserved", _i32), ("alpha", _f64),
                ("strength", _f64), ("col_offset", _i64), ("n_cols", _i64)]


class LoraPool(ctypes.Structure):
    """C ``lora_pool``: the adapters from which the tokens of a routed call take theirs."""
    _fields_ = [("A", _p), ("B", _p), ("scales", _p), ("ranks", _p), ("n_adapters", _i32), ("rank", _i32),
                ("reserved", _i64)]


class LoraAdamWTensor(ctypes.Structure):
    """C ``lora_adamw_tensor``: one tensor of an AdamW step."""
    _fields_ = [("param", _p), ("master", _p), ("grad", _p), ("m", _p), ("v", _p), ("m_scale", _p), ("v_scale", _p),
                ("n", _i64)]


class LoraAdamWPlan(ctypes.Structure):
    """C ``lora_adamw_plan_t``, filled by ``lora_adamw_plan``."""
    _fields_ = [("table", _p), ("n_blocks", _i64), ("n_tensors", _i32), ("chunk", _i32), ("param_dtype", _i32),
                ("grad_dtype", _i32), ("state_bits", _i32), ("reserved", _i32)]


_lib.lora_linear_fwd.argtypes = [_p, _i64, _i64, _i64, _p, _i64, _p, _p, _p, _i32, _i32, _f64, _f64, _f64,
                                 _p, _i64, _i32, _i32, _p, _sz, _p]
_lib.lora_linear_fwd.restype = ctypes.c_int
_lib.lora_linear_fwd_noalloc.argtypes = [_p, _i64, _i64, _i64, _p, _i64, _p, _p, _p, _i32, _i32, _f64, _f64, _f64,
                                         _p, _i64, _i32, _i32, _p]
_lib.lora_linear_fwd_noalloc.restype = ctypes.c_int
LORA_NOALLOC_SCRATCH_BYTES = 64 * 1024 * 1024
_lib.lora_mfma_probe.argtypes = [_i64, _i32, _p, _p, _p]
_lib.lora_mfma_probe.restype = ctypes.c_int
_lib.lora_linear_fwd_phase.argtypes = [_i32, _i32, _p, _i64, _i64, _i64, _p, _i64, _p, _p, _p, _i32, _i32, _f64,
                                       _f64, _f64, _p, _i64, _i32, _i32, _p, _sz, _p]
_lib.lora_linear_fwd_phase.restype = ctypes.c_int
_lib.lora_linear_stacked_fwd.argtypes = [_p, _i64, _i64, _i64, _p, _i64, _p, ctypes.POINTER(LoraGroup), _i32,
                                         _i32, _f64, _f64, _p, _i64, _i32, _i32, _p, _sz, _p]
_lib.lora_linear_stacked_fwd.restype = ctypes.c_int
_lib.lora_linear_nf4_fwd.argtypes = [_p, _i64, _i64, _i64, _p, _p, _p, _i32, _i64, _p, _p, _p, _i32, _i32,
                                     _f64, _f64, _f64, _p, _i64, _i32, _p, _sz, _p]
_lib.lora_linear_nf4_fwd.restype = ctypes.c_int
_lib.lora_linear_nf4_fwd_ex.argtypes = [_p, _i64, _i64, _i64, _p, _p, _p, _i32, _i64, _p, _p, _p, _i32, _i32,
                                        _f64, _f64, _f64, _p, _i64, _i32, _i32, _p, _sz, _p]
_lib.lora_linear_nf4_fwd_ex.restype = ctypes.c_int
_lib.dense_patch_apply.argtypes = [_p, _i32, ctypes.POINTER(_i64), _i32, _p, _i32, ctypes.POINTER(_i64), _i32,
                                   _f64, _i32, _p]
_lib.dense_patch_apply.restype = ctypes.c_int
_lib.lora_linear_workspace_size.argtypes = [_i64, _i64, _i64, ctypes.POINTER(_i32), _i32, _i32, _i32]
_lib.lora_linear_workspace_size.restype = _sz
_lib.lora_linear_multi_fwd.argtypes = [_p, _i64, _i64, _i64, _p, _i64, _p, ctypes.POINTER(LoraAdapter), _i32, _i32,
                                       _f64, _p, _i64, _i32, _i32, _p, _sz, _p]
_lib.lora_linear_multi_fwd.restype = ctypes.c_int
_lib.lora_linear_multi_workspace_size.argtypes = [_i64, _i64, _i64, ctypes.POINTER(LoraAdapter), _i32, _i32, _i32]
_lib.lora_linear_multi_workspace_size.restype = _sz
_lib.lora_linear_bwd.argtypes = [_p, _i64, _i64, _i64, _p, _i64, _p, _p, _i32, _f64, _f64, _f64, _p, _i64, _p, _i64,
                                 _p, _p, _p, _p, _i64, _p, _sz, _p]
_lib.lora_linear_bwd.restype = ctypes.c_int
_lib.lora_linear_bwd_workspace_size.argtypes = [_i64, _i64, _i64, _i32, _i32]
_lib.lora_linear_bwd_workspace_size.restype = _sz
_lib.lora_linear_routed_fwd.argtypes = [_p, _i64, _i64, _i64, _p, _i64, _p, ctypes.POINTER(LoraPool), _p, _p, _p,
                                        _i64, _p, _sz, _p]
_lib.lora_linear_routed_fwd.restype = ctypes.c_int
_lib.lora_linear_routed_workspace_size.argtypes = [_i64, _i64, _i64, _i32, _i32]
_lib.lora_linear_routed_workspace_size.restype = _sz
_lib.lora_linear_routed_bwd.argtypes = [_p, _i64, _i64, _i64, _p, _i64, ctypes.POINTER(LoraPool), _p, _p, _p, _i64,
                                        _p, _i64, _p, _p, _p, _sz, _p]
_lib.lora_linear_routed_bwd.restype = ctypes.c_int
_lib.lora_linear_routed_bwd_workspace_size.argtypes = [_i64, _i64, _i64, _i32, _i32, _i32]
_lib.lora_linear_routed_bwd_workspace_size.restype = _sz
_lib.lora_adamw_table_size.argtypes = [ctypes.POINTER(LoraAdamWTensor), _i32]
_lib.lora_adamw_table_size.restype = _sz
_lib.lora_adamw_plan.argtypes = [ctypes.POINTER(LoraAdamWTensor), _i32, _i32, _i32, _i32, _p, _sz,
                                 ctypes.POINTER(LoraAdamWPlan), _p]
_lib.lora_adamw_plan.restype = ctypes.c_int
_lib.lora_adamw_step.argtypes = [ctypes.POINTER(LoraAdamWPlan), _f64, _f64, _f64, _f64, _f64, _i64, _p, _f64, _p]
_lib.lora_adamw_step.restype = ctypes.c_int
_lib.lora_merge_apply.argtypes = [_p, _i32, _i64, _i64, _p, _p, _i32, _i32, _f64, _f64, _i32, _p]
_lib.lora_merge_apply.restype = ctypes.c_int
_lib.lora_linear_nf4_workspace_size.argtypes = [_i64, _i64, _i64, _i32, _i32, _i32]
_lib.lora_linear_nf4_workspace_size.restype = _sz
_lib.lora_status_string.argtypes = [ctypes.c_int]
_lib.lora_status_string.restype = ctypes.c_char_p
_lib.lora_device_check.argtypes = []
_lib.lora_device_check.restype = ctypes.c_int


class LoraError(RuntimeError):
    def __init__(self, status: int, fn: str):
        self.status = status
        super().__init__(f"{fn}: status {status} ({lora_status_string(status)})")


def _check(status: int, fn: str) -> int:
    if status != 0:
        raise LoraError(status, fn)
    return status


# ----------------------------------------------------------------- C names, plain integers

def lora_linear_fwd(x, T, K, ldx, W, N, bias, A, B, rank, adapter_dtype, alpha, strength, request_scale,
                    y, ldy, act_dtype, quality, workspace, workspace_bytes, stream):
    return _check(_lib.lora_linear_fwd(x, T, K, ldx, W, N, bias, A, B, rank, adapter_dtype, alpha, strength,
                                       request_scale, y, ldy, act_dtype, quality, workspace, workspace_bytes,
                                       stream), "lora_linear_fwd")


def lora_linear_fwd_noalloc(x, T, K, ldx, W, N, bias, A, B, rank, adapter_dtype, alpha, strength, request_scale,
                            y, ldy, act_dtype, quality, stream):
    return _check(_lib.lora_linear_fwd_noalloc(x, T, K, ldx, W, N, bias, A, B, rank, adapter_dtype, alpha, strength,
                                               request_scale, y, ldy, act_dtype, quality, stream),
                  "lora_linear_fwd_noalloc")


def lora_linear_fwd_phase(phase, gemm_tile, x, T, K, ldx, W, N, bias, A, B, rank, adapter_dtype, alpha, strength,
                          request_scale, y, ldy, act_dtype, quality, workspace, workspace_bytes, stream):
    return _check(_lib.lora_linear_fwd_phase(phase, gemm_tile, x, T, K, ldx, W, N, bias, A, B, rank, adapter_dtype,
                                             alpha, strength, request_scale, y, ldy, act_dtype, quality, workspace,
                                             workspace_bytes, stream), "lora_linear_fwd_phase")


def lora_linear_stacked_fwd(x, T, K, ldx, W, N_total, bias, groups, n_groups, adapter_dtype, strength,
                            request_scale, y, ldy, act_dtype, quality, workspace, workspace_bytes, stream):
    arr = (LoraGroup * max(1, n_groups))(*groups)
    return _check(_lib.lora_linear_stacked_fwd(x, T, K, ldx, W, N_total, bias, arr, n_groups, adapter_dtype,
                                               strength, request_scale, y, ldy, act_dtype, quality, workspace,
                                               workspace_bytes, stream), "lora_linear_stacked_fwd")


def lora_linear_multi_fwd(x, T, K, ldx, W, N, bias, adapters, n_adapters, adapter_dtype, request_scale, y, ldy,
                          act_dtype, quality, workspace, workspace_bytes, stream):
    arr = (LoraAdapter * max(1, n_adapters))(*adapters)
    return _check(_lib.lora_linear_multi_fwd(x, T, K, ldx, W, N, bias, arr, n_adapters, adapter_dtype, request_scale,
                                             y, ldy, act_dtype, quality, workspace, workspace_bytes, stream),
                  "lora_linear_multi_fwd")


def lora_linear_bwd(x, T, K, ldx, W, N, A, B, rank, alpha, strength, request_scale, dy, lddy, dx, lddx, dA, dB, db,
                    t_tilde, ldt, workspace, workspace_bytes, stream):
    return _check(_lib.lora_linear_bwd(x, T, K, ldx, W, N, A, B, rank, alpha, strength, request_scale, dy, lddy, dx,
                                       lddx, dA, dB, db, t_tilde, ldt, workspace, workspace_bytes, stream),
                  "lora_linear_bwd")


def lora_linear_bwd_workspace_size(T, K, N, rank, want_dx=True) -> int:
    return int(_lib.lora_linear_bwd_workspace_size(T, K, N, rank, 1 if want_dx else 0))


def lora_linear_routed_fwd(x, T, K, ldx, W, N, bias, pool, token_adapter, token_scale, y, ldy, workspace,
                           workspace_bytes, stream):
    return _check(_lib.lora_linear_routed_fwd(x, T, K, ldx, W, N, bias, ctypes.byref(pool), token_adapter, token_scale,
                                              y, ldy, workspace, workspace_bytes, stream), "lora_linear_routed_fwd")


def lora_linear_routed_workspace_size(T, K, N, n_adapters, rank) -> int:
    return int(_lib.lora_linear_routed_workspace_size(T, K, N, n_adapters, rank))


def lora_linear_routed_bwd(x, T, K, ldx, W, N, pool, token_adapter, token_scale, dy, lddy, dx, lddx, dA, dB,
                           workspace, workspace_bytes, stream):
    return _check(_lib.lora_linear_routed_bwd(x, T, K, ldx, W, N, ctypes.byref(pool), token_adapter, token_scale, dy,
                                              lddy, dx, lddx, dA, dB, workspace, workspace_bytes, stream),
                  "lora_linear_routed_bwd")


def lora_linear_routed_bwd_workspace_size(T, K, N, n_adapters, rank, want_dx=True) -> int:
    return int(_lib.lora_linear_routed_bwd_workspace_size(T, K, N, n_adapters, rank, 1 if want_dx else 0))


def lora_adamw_table_size(tensors) -> int:
    arr = (LoraAdamWTensor * max(1, len(tensors)))(*tensors)
    return int(_lib.lora_adamw_table_size(arr, len(tensors)))


def lora_adamw_plan(tensors, param_dtype, grad_dtype, state_bits, table, table_bytes, stream) -> LoraAdamWPlan:
    arr, plan = (LoraAdamWTensor * max(1, len(tensors)))(*tensors), LoraAdamWPlan()
    _check(_lib.lora_adamw_plan(arr, len(tensors), param_dtype, grad_dtype, state_bits, table, table_bytes,
                                ctypes.byref(plan), stream), "lora_adamw_plan")
    return plan


def lora_adamw_step(plan, lr, beta1, beta2, eps, weight_decay, step, lr_step, grad_scale, stream):
    return _check(_lib.lora_adamw_step(ctypes.byref(plan), lr, beta1, beta2, eps, weight_decay, step, lr_step,
                                       grad_scale, stream), "lora_adamw_step")


def lora_merge_apply(W, w_dtype, N, K, A, B, rank, adapter_dtype, alpha, strength, quality, stream):
    return _check(_lib.lora_merge_apply(W, w_dtype, N, K, A, B, rank, adapter_dtype, alpha, strength, quality, stream),
                  "lora_merge_apply")


def lora_linear_multi_workspace_size(T, K, N, adapters, adapter_dtype, quality=LORA_LOSSLESS) -> int:
    arr = (LoraAdapter * max(1, len(adapters)))(*adapters)
    return int(_lib.lora_linear_multi_workspace_size(T, K, N, arr, len(adapters), adapter_dtype, quality))


def lora_linear_nf4_fwd(x, T, K, ldx, codes, absmax, codebook, blocksize, N, bias, A, B, rank, adapter_dtype,
                        alpha, strength, request_scale, y, ldy, quality, workspace, workspace_bytes, stream):
    return _check(_lib.lora_linear_nf4_fwd(x, T, K, ldx, codes, absmax, codebook, blocksize, N, bias, A, B, rank,
                                           adapter_dtype, alpha, strength, request_scale, y, ldy, quality,
                                           workspace, workspace_bytes, stream), "lora_linear_nf4_fwd")


def lora_linear_nf4_fwd_ex(x, T, K, ldx, codes, absmax, codebook, blocksize, N, bias, A, B, rank, adapter_dtype,
                           alpha, strength, request_scale, y, ldy, quality, dequant, workspace, workspace_bytes,
                           stream):
    return _check(_lib.lora_linear_nf4_fwd_ex(x, T, K, ldx, codes, absmax, codebook, blocksize, N, bias, A, B, rank,
                                              adapter_dtype, alpha, strength, request_scale, y, ldy, quality,
                                              dequant, workspace, workspace_bytes, stream), "lora_linear_nf4_fwd_ex")


def dense_patch_apply(dst, dst_dtype, dst_shape, src, src_dtype, src_shape, strength, mode, stream):
    ds = (_i64 * max(1, len(dst_shape)))(*dst_shape)
    ss = (_i64 * max(1, len(src_shape)))(*src_shape)
    return _check(_lib.dense_patch_apply(dst, dst_dtype, ds, len(dst_shape), src, src_dtype, ss, len(src_shape),
                                         strength, mode, stream), "dense_patch_apply")


def lora_linear_workspace_size(T, K, N, ranks, adapter_dtype, quality=LORA_LOSSLESS) -> int:
    arr = (_i32 * max(1, len(ranks)))(*ranks)
    return int(_lib.lora_linear_workspace_size(T, K, N, arr, len(ranks), adapter_dtype, quality))


def lora_linear_nf4_workspace_size(T, K, N, rank, adapter_dtype, quality=LORA_LOSSLESS) -> int:
    return int(_lib.lora_linear_nf4_workspace_size(T, K, N, rank, adapter_dtype, quality))


def lora_status_string(status: int) -> str:
    return _lib.lora_status_string(status).decode()


def lora_device_check() -> int:
    return int(_lib.lora_device_check())


def lora_mfma_probe(iters, blocks, sink, clocks, stream):
    return _check(_lib.lora_mfma_probe(iters, blocks, sink, clocks, stream), "lora_mfma_probe")


def hip_runtimes_mapped() -> list:
    """Distinct libamdhip64 files mapped into this process (exactly one is expected)."""
    paths = set()
    with open("/proc/self/maps") as f:
        for line in f:
            if "libamdhip64" in line:
                paths.add(os.path.realpath(line.split()[-1]))
    return sorted(paths)


# ----------------------------------------------------------------- tensor-level helpers

def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return LORA_BF16
    if t.dtype == torch.float32:
        return LORA_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream):
    s = torch.cuda.current_stream() if stream is None else stream
    return s.cuda_stream


def _row_major(t: torch.Tensor, name: str):
    if t.dim() != 2 or t.stride(1) != 1:
        raise ValueError(f"{name} must be a 2-D tensor with unit column stride")
    return t.stride(0)


def _workspace(T, K, N, ranks, adapter_dtype, quality, workspace, device):
    need = lora_linear_workspace_size(T, K, N, list(ranks), adapter_dtype, quality)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=device)
    return workspace, need


def lora_linear(x, W, b, A, B, alpha, strength=1.0, request_scale=1.0, out=None, quality="lossless",
                workspace=None, stream=None, gemm_tile=None):
    """y = x.W^T + b + s.(x.A^T).B^T on the GPU; returns ``out`` (allocated when None).

    ``gemm_tile`` (lossless only): None or 0 lets the library pick the hot GEMM's output
    tile, 1 fixes 256 x 256, 2 fixes 128 x 128 (same bits, different speed)."""
    T, K = x.shape
    N = W.shape[0]
    ldx = _row_major(x, "x")
    if out is None:
        out = torch.empty((T, N), dtype=x.dtype, device=x.device)
    ldy = _row_major(out, "out")
    rank = 0 if A is None else A.shape[0]
    adt = _dt(A) if A is not None else _dt(x)
    q = _QUALITY[quality]
    ws, need = _workspace(T, K, N, [rank] if rank else [], adt, q, workspace, x.device)
    args = (x.data_ptr(), T, K, ldx, W.data_ptr(), N, _ptr(b), _ptr(A), _ptr(B), rank, adt, float(alpha),
            float(strength), float(request_scale), out.data_ptr(), ldy, _dt(x), q, ws.data_ptr(), ws.numel(),
            _stream(stream))
    if gemm_tile:
        lora_linear_fwd_phase(0, int(gemm_tile), *args)
    else:
        lora_linear_fwd(*args)
    return out


def lora_linear_stacked(x, W, b, groups, strength=1.0, request_scale=1.0, out=None, quality="lossless",
                        workspace=None, stream=None):
    """Stacked groups: ``groups`` is a list of dicts with A, B, alpha, col_offset, n_cols."""
    T, K = x.shape
    N = W.shape[0]
    ldx = _row_major(x, "x")
    if out is None:
        out = torch.empty((T, N), dtype=x.dtype, device=x.device)
    ldy = _row_major(out, "out")
    adt = _dt(groups[0]["A"]) if groups else _dt(x)
    cg = [LoraGroup(_ptr(g["A"]), _ptr(g["B"]), 0 if g["A"] is None else g["A"].shape[0], 0, float(g["alpha"]),
                    int(g["col_offset"]), int(g["n_cols"])) for g in groups]
    q = _QUALITY[quality]
    ws, need = _workspace(T, K, N, [g.rank for g in cg if g.rank > 0], adt, q, workspace, x.device)
    lora_linear_stacked_fwd(x.data_ptr(), T, K, ldx, W.data_ptr(), N, _ptr(b), cg, len(cg), adt, float(strength),
                            float(request_scale), out.data_ptr(), ldy, _dt(x), q, ws.data_ptr(), ws.numel(),
                            _stream(stream))
    return out


def lora_linear_multi(x, W, b, adapters, request_scale=1.0, out=None, quality="lossless", workspace=None,
                      stream=None):
    """Several adapters on one layer: ``adapters`` is a list of dicts with A, B, c (legacy
    lora_B bias or None), alpha, strength, col_offset, n_cols; column ranges may overlap."""
    T, K = x.shape
    N = W.shape[0]
    ldx = _row_major(x, "x")
    if out is None:
        out = torch.empty((T, N), dtype=x.dtype, device=x.device)
    ldy = _row_major(out, "out")
    adt = _dt(adapters[0]["A"]) if adapters else _dt(x)
    ca = [LoraAdapter(_ptr(a["A"]), _ptr(a["B"]), _ptr(a.get("c")), 0 if a["A"] is None else a["A"].shape[0], 0,
                      float(a["alpha"]), float(a["strength"]), int(a["col_offset"]), int(a["n_cols"]))
          for a in adapters]
    q = _QUALITY[quality]
    need = lora_linear_multi_workspace_size(T, K, N, ca, adt, q)
    ws = workspace if workspace is not None else torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    lora_linear_multi_fwd(x.data_ptr(), T, K, ldx, W.data_ptr(), N, _ptr(b), ca, len(ca), adt, float(request_scale),
                          out.data_ptr(), ldy, _dt(x), q, ws.data_ptr(), ws.numel(), _stream(stream))
    return out


def lora_linear_nf4(x, codes, absmax, codebook, N, b, A, B, alpha, strength=1.0, request_scale=1.0,
                    blocksize=64, out=None, quality="lossless", workspace=None, stream=None, dequant="auto"):
    """``dequant``: "auto", "panel" or "in_gemm" (where a lossless call with more than 64 tokens
    dequantizes the 4-bit weight; the same output bits either way)."""
    T, K = x.shape
    ldx = _row_major(x, "x")
    if out is None:
        out = torch.empty((T, N), dtype=x.dtype, device=x.device)
    ldy = _row_major(out, "out")
    rank = 0 if A is None else A.shape[0]
    adt = _dt(A) if A is not None else LORA_BF16
    q = _QUALITY[quality]
    need = lora_linear_nf4_workspace_size(T, K, N, rank, adt, q)
    ws = workspace if workspace is not None else torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    lora_linear_nf4_fwd_ex(x.data_ptr(), T, K, ldx, codes.data_ptr(), absmax.data_ptr(), codebook.data_ptr(),
                           blocksize, N, _ptr(b), _ptr(A), _ptr(B), rank, adt, float(alpha), float(strength),
                           float(request_scale), out.data_ptr(), ldy, q, _DEQUANT[dequant], ws.data_ptr(),
                           ws.numel(), _stream(stream))
    return out


def lora_merge(W, A, B, alpha, strength=1.0, quality="lossless", stream=None):
    """W <- RN(W + (alpha / rank) . strength . B.A) in place on the GPU; returns ``W``."""
    N, K = W.shape
    if not (W.is_contiguous() and A.is_contiguous() and B.is_contiguous()):
        raise ValueError("lora_merge needs contiguous tensors")
    lora_merge_apply(W.data_ptr(), _dt(W), N, K, A.data_ptr(), B.data_ptr(), A.shape[0], _dt(A), float(alpha),
                     float(strength), _QUALITY[quality], _stream(stream))
    return W


def lora_linear_backward(x, W, A, B, dy, alpha, strength=1.0, request_scale=1.0, want=("dx", "dA", "dB", "db"),
                         workspace=None, stream=None, t_tilde=None):
    """Gradients of the LoRA linear for the output gradient ``dy``: returns (dx, dA, dB, db),
    each None unless named in ``want`` (dx bf16; dA, dB, db fp32). ``t_tilde``: optional bf16
    [T, ldt] tensor holding the forward's t~ (for instance a view of the forward call's
    workspace), so that x is not read again to recompute it."""
    T, K = x.shape
    N = W.shape[0]
    r = A.shape[0]
    ldx, lddy = _row_major(x, "x"), _row_major(dy, "dy")
    dev = x.device
    dx = torch.empty((T, K), dtype=torch.bfloat16, device=dev) if "dx" in want else None
    dA = torch.empty((r, K), dtype=torch.float32, device=dev) if "dA" in want else None
    dB = torch.empty((N, r), dtype=torch.float32, device=dev) if "dB" in want else None
    db = torch.empty((N,), dtype=torch.float32, device=dev) if "db" in want else None
    need = lora_linear_bwd_workspace_size(T, K, N, r, dx is not None)
    ws = workspace if workspace is not None else torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
    ldt = _row_major(t_tilde, "t_tilde") if t_tilde is not None else 0
    lora_linear_bwd(x.data_ptr(), T, K, ldx, W.data_ptr(), N, A.data_ptr(), B.data_ptr(), r, float(alpha),
                    float(strength), float(request_scale), dy.data_ptr(), lddy, _ptr(dx), K, _ptr(dA), _ptr(dB),
                    _ptr(db), _ptr(t_tilde), ldt, ws.data_ptr(), ws.numel(), _stream(stream))
    return dx, dA, dB, db


def _of(t, name, shape, dtype, device):
    """The tensor checked: contiguous, of this shape and type, on the call's device (None passes)."""
    if t is None or (t.dtype == dtype and t.shape == shape and t.device == device and t.is_contiguous()):
        return t
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    raise ValueError(f"{name} must be a contiguous tensor of shape {tuple(shape)}, got {tuple(t.shape)}")


def _rows(t, name, shape, device):
    """Row stride of a bf16 matrix of this shape with unit column stride on the call's device."""
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.shape != shape or t.device != device:
        raise ValueError(f"{name} must have shape {tuple(shape)} on {device}, got {tuple(t.shape)} on {t.device}")
    rows, cols = shape
    ld, unit = t.stride()
    if unit != 1 and cols != 1 and rows * cols != 0:  # (one column may carry any stride)
        raise ValueError(f"{name} must have unit column stride")
    return ld if rows > 1 else -(-cols // 8) * 8  # (and so may one row)


def _routed_args(x, W, A, B, scales, token_adapter, token_scale, ranks):
    """Checks shared by the routed calls; returns T, K, N and the C pool."""
    dev = x.device
    if x.dim() != 2 or A.dim() != 3 or B.dim() != 3:
        raise ValueError("x must be [T, K], A [n, rank, K] and B [n, N, rank]")
    T, K = x.shape
    n, R, _ = A.shape
    N = B.shape[1]
    at, bf = x.get_device(), torch.bfloat16
    if not (A.dtype is bf and B.dtype is bf and scales.dtype is torch.float32 and token_adapter.dtype is torch.int32
            and A.get_device() == B.get_device() == scales.get_device() == token_adapter.get_device() == at
            and A.is_contiguous() and B.is_contiguous() and scales.is_contiguous() and token_adapter.is_contiguous()
            and A.shape[2] == K and B.shape == (n, N, R) and scales.shape == (n,) and token_adapter.shape == (T,)
            and (W is None or (W.dtype is bf and W.get_device() == at and W.is_contiguous() and W.shape == (N, K)))):
        _of(A, "A", (n, R, K), bf, dev)  # (these say what is wrong; a call that is right passes in 1-2 us less)
        _of(B, "B", (n, N, R), bf, dev)
        _of(scales, "scales", (n,), torch.float32, dev)
        _of(token_adapter, "token_adapter", (T,), torch.int32, dev)
        if W is not None:
            _of(W, "W", (N, K), bf, dev)
    if token_scale is not None:
        _of(token_scale, "token_scale", (T,), torch.float32, dev)
    if ranks is not None:
        _of(ranks, "ranks", (n,), torch.int32, dev)
    return T, K, N, LoraPool(A.data_ptr(), B.data_ptr(), scales.data_ptr(), _ptr(ranks), n, R, 0)


def _bytes_on(workspace, size, args, device):
    """The workspace given, checked, or one of size(*args) bytes. (Its length is checked by the call.)"""
    if workspace is None:
        return torch.empty(max(size(*args), 1), dtype=torch.uint8, device=device)
    if workspace.device != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be contiguous on {device}")
    return workspace


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_on(device, stream):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None and device.index is not None:  # (the handle alone, without a Stream object)
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


_HERE = contextlib.nullcontext()


def _on(device, stream=None):
    """The device, and a stream that is named, made current for a call: what the call allocates then belongs to
    the stream that uses it. (A context only where one is needed.)"""
    if stream is not None:
        if stream.device != device:
            raise ValueError(f"stream of {stream.device} for tensors on {device}")
        return torch.cuda.stream(stream)
    return _HERE if device.type != "cuda" or device.index == torch.cuda.current_device() else torch.cuda.device(device)


def lora_linear_routed(x, W, b, A, B, scales, token_adapter, token_scale=None, ranks=None, out=None, workspace=None,
                       stream=None):
    """A linear layer whose tokens take their adapters from a pool (bf16; returns ``out``):
    y[t] = x[t].W^T + b + s_t (x[t].A_a^T).B_a^T with a = token_adapter[t], s_t = scales[a] token_scale[t].

    A [n, rank, K] and B [n, N, rank] are the pool, ``scales`` fp32 [n], ``token_adapter`` int32 [T]
    (-1: no adapter), ``token_scale`` fp32 [T] or None, ``ranks`` int32 [n] or None (see lora_linear_routed_fwd)."""
    T, K, N, pool = _routed_args(x, W, A, B, scales, token_adapter, token_scale, ranks)
    dev = x.device
    ldx = _rows(x, "x", (T, K), dev)
    if b is not None:
        _of(b, "b", (N,), torch.bfloat16, dev)
    with _on(dev, stream):
        if out is None:
            out, ldy = torch.empty((T, N), dtype=torch.bfloat16, device=dev), N
        else:
            ldy = _rows(out, "out", (T, N), dev)
        ws = _bytes_on(workspace, _lib.lora_linear_routed_workspace_size, (T, K, N, pool.n_adapters, pool.rank), dev)
        lora_linear_routed_fwd(x.data_ptr(), T, K, ldx, W.data_ptr(), N, _ptr(b), pool, token_adapter.data_ptr(),
                               _ptr(token_scale), out.data_ptr(), ldy, ws.data_ptr(),
                               ws.numel() * ws.element_size(), _stream_on(dev, stream))
    return out


def lora_linear_routed_backward(x, W, A, B, dy, scales, token_adapter, token_scale=None, ranks=None,
                                want=("dx", "dA", "dB"), dx=None, dA=None, dB=None, workspace=None, stream=None):
    """Gradients of ``lora_linear_routed`` for the output gradient ``dy``: returns (dx, dA, dB), each
    None unless named in ``want`` (dx bf16 [T, K]; dA [n, rank, K] and dB [n, N, rank] fp32, written
    whole into the given tensors when there are any)."""
    T, K, N, pool = _routed_args(x, W, A, B, scales, token_adapter, token_scale, ranks)
    n, R, _ = A.shape
    dev = x.device
    ldx, lddy = _rows(x, "x", (T, K), dev), _rows(dy, "dy", (T, N), dev)
    with _on(dev, stream):
        if "dx" not in want:
            dx = None
        elif dx is None:
            dx = torch.empty((T, K), dtype=torch.bfloat16, device=dev)
        lddx = _rows(dx, "dx", (T, K), dev) if dx is not None else K
        grads = []
        for name, t, shape in (("dA", dA, (n, R, K)), ("dB", dB, (n, N, R))):
            if name not in want:
                t = None
            elif t is None:
                t = torch.empty(shape, dtype=torch.float32, device=dev)
            grads.append(_of(t, name, shape, torch.float32, dev))
        dA, dB = grads
        ws = _bytes_on(workspace, _lib.lora_linear_routed_bwd_workspace_size, (T, K, N, n, R, dx is not None), dev)
        lora_linear_routed_bwd(x.data_ptr(), T, K, ldx, _ptr(W), N, pool, token_adapter.data_ptr(),
                               _ptr(token_scale), dy.data_ptr(), lddy, _ptr(dx), lddx, _ptr(dA), _ptr(dB),
                               ws.data_ptr(), ws.numel() * ws.element_size(), _stream_on(dev, stream))
    return dx, dA, dB


class LoraAdamW:
    """AdamW over many tensors, one launch per step (see lora_adamw_step).

    ``params``: list of tensors of one dtype (bf16 or fp32), stepped in place; ``grads``: their gradient
    buffers (fp32 or bf16, the same shapes), read at every step: the backward calls write into them
    (``lora_linear_routed_backward(..., dA=, dB=)``). ``master``: True for fp32 masters of bf16 parameters
    (made from them), a list of tensors, or None. ``state_bits``: 32, or 8 for e4m3 moments with an fp32
    scale per 256 elements. ``state``: a dict as ``state()`` returns it, taken over (not copied); None
    starts at zero. ``lr_step``: optional fp64 device tensor {lr, step} that the kernel reads in place of
    ``lr`` and the step count, for captured steps (``state()["step"]`` counts the calls of ``step``, not
    replays). lr, betas, eps and weight_decay may be changed between
    steps. The optimizer keeps the tensors; their buffers must stay where they are. It is made outside of captures."""

    def __init__(self, params, grads, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, master=None,
                 state_bits=32, state=None, lr_step=None, stream=None):
        params, grads = list(params), list(grads)
        if not params or len(grads) != len(params):
            raise ValueError("LoraAdamW needs parameters and one gradient buffer for each")
        if state_bits not in (32, 8):
            raise ValueError("state_bits must be 32 or 8")
        dev = params[0].device
        if dev.type == "cuda" and torch.cuda.is_current_stream_capturing():
            raise RuntimeError("LoraAdamW cannot be made during a capture: every replay would start it anew")
        self.lr, self.betas, self.eps, self.weight_decay = lr, betas, eps, weight_decay
        self.state_bits, self.device = state_bits, dev
        self.lr_step = _of(lr_step, "lr_step", (2,), torch.float64, dev)
        if master is True:
            master = [p.float() for p in params]
        state = {} if state is None else state
        mdt = torch.float32 if state_bits == 32 else torch.float8_e4m3fn
        flat = lambda p: (p.numel(),)  # noqa: E731
        blocks = lambda p: (-(-p.numel() // 256),)  # noqa: E731

        def lists(name, dtype, shape):
            ts = state.get(name)
            if ts is None:
                ts = [torch.zeros(shape(p), dtype=dtype, device=dev) for p in params]
            if len(ts) != len(params):
                raise ValueError(f"{name} must hold one tensor per parameter")
            return [_of(t.view(-1), f"{name}[{i}]", shape(p), dtype, dev) for i, (t, p) in enumerate(zip(ts, params))]

        self.m, self.v = lists("m", mdt, flat), lists("v", mdt, flat)
        self.m_scale = self.v_scale = None
        if state_bits == 8:
            self.m_scale, self.v_scale = lists("m_scale", torch.float32, blocks), lists("v_scale", torch.float32, blocks)
        self.step_count = int(state.get("step", 0))
        for i, (p, g) in enumerate(zip(params, grads)):
            _of(p, f"params[{i}]", p.shape, params[0].dtype, dev)
            _of(g, f"grads[{i}]", p.shape, grads[0].dtype, dev)
        if master is not None:
            if len(master) != len(params):
                raise ValueError("master must hold one tensor per parameter")
            for i, (p, t) in enumerate(zip(params, master)):
                _of(t, f"master[{i}]", p.shape, torch.float32, dev)
        self.params, self.grads, self.master = params, grads, master
        none = [None] * len(params)
        ts = [LoraAdamWTensor(_ptr(p), _ptr(w), _ptr(g), _ptr(m), _ptr(v), _ptr(ms), _ptr(vs), p.numel())
              for p, w, g, m, v, ms, vs in zip(params, master or none, grads, self.m, self.v, self.m_scale or none,
                                               self.v_scale or none)]
        need = lora_adamw_table_size(ts)
        with _on(dev, stream):
            self._table = torch.empty(max(need, 1), dtype=torch.uint8, device=dev)
            self._plan = lora_adamw_plan(ts, _dt(params[0]), _dt(grads[0]), state_bits, self._table.data_ptr(),
                                         self._table.numel(), _stream_on(dev, stream))
        if dev.type == "cuda":
            # (the table, new masters and new moments are there for a step on any stream)
            torch.cuda.current_stream(dev).synchronize()
            if stream is not None:
                stream.synchronize()

    def step(self, grad_scale=1.0, stream=None):
        """One step on the gradients that the buffers hold (on the stream that runs it)."""
        count = self.step_count + 1
        with _on(self.device, stream):
            lora_adamw_step(self._plan, float(self.lr), float(self.betas[0]), float(self.betas[1]), float(self.eps),
                            float(self.weight_decay), count, _ptr(self.lr_step), float(grad_scale),
                            _stream_on(self.device, stream))
        self.step_count = count

    def state(self):
        """The moments (the tensors themselves) and the step count, as ``state=`` takes them."""
        return dict(m=self.m, v=self.v, m_scale=self.m_scale, v_scale=self.v_scale, step=self.step_count)


def dense_patch(dst, src, strength, mode="add", stream=None):
    """Apply a dense payload to ``dst`` in place; returns ``dst``."""
    if not (dst.is_contiguous() and src.is_contiguous()):
        raise ValueError("dense_patch needs contiguous tensors")
    dense_patch_apply(dst.data_ptr(), _dt(dst), list(dst.shape), src.data_ptr(), _dt(src), list(src.shape),
                      float(strength), _MODE[mode], _stream(stream))
    return dst
