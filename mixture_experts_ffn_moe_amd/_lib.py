"""ctypes binding of libmoe_mi355x.so: argument marshalling only.

Each function has the name of the C entry point it calls and takes torch
tensors, which supply device memory; the current torch stream is passed as
the HIP stream.  Every step of the layer runs in the library's HIP kernels:
if the library is missing this module raises on import instead of falling
back to anything else.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe_mi355x.so")

MOE_OK, MOE_ERR_INVALID_ARG, MOE_ERR_UNSUPPORTED, MOE_ERR_WORKSPACE, MOE_ERR_HIP = range(5)
MOE_F32, MOE_BF16 = 0, 1
MOE_Q4_INT4, MOE_Q4_E2M1 = 0, 1

EXPORTED = (
    "moe_status_string", "moe_workspace_size", "moe_get_workspace_layout", "moe_route",
    "moe_permute", "moe_grouped_gemm_w13_swiglu", "moe_grouped_gemm_down", "moe_finalize",
    "moe_forward", "moe_forward_noalloc",
    # shared expert (moe_shared.h)
    "moe_shared_workspace_size", "moe_get_shared_workspace_layout", "moe_shared_ffn",
    "moe_finalize_shared", "moe_forward_shared",
    # 4-bit expert weights (moe_q4.h)
    "moe_q4_get_sizes", "moe_q4_quantize_w13", "moe_q4_quantize_down", "moe_q4_w13_swiglu",
    "moe_q4_down", "moe_forward_q4",
    # router gradients (moe_router_grad.h)
    "moe_balance_workspace_size", "moe_balance_loss", "moe_route_backward",
    "moe_router_grad_workspace_size", "moe_router_weight_grad", "moe_finalize_backward",
    # shared expert's training and dropout (moe_shared_train.h)
    "moe_dropout_add", "moe_dropout_backward", "moe_shared_ffn_train", "moe_shared_backward_workspace_size",
    "moe_shared_ffn_backward",
    # request adapters (moe_lora.h)
    "moe_lora_workspace_size", "moe_lora_w13_swiglu", "moe_lora_down", "moe_shared_ffn_lora",
    # measurement probes (moe_probe.h)
    "moe_probe_mfma_bf16", "moe_probe_mfma_flops", "moe_probe_read",
)


class MoeError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {status_string(code)}")


class MoeShape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("E", ctypes.c_int32),
                ("k", ctypes.c_int32), ("Im", ctypes.c_int32), ("micro_count", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("renormalize", ctypes.c_int32)]


class MoeWorkspaceLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in
                ("logits", "topk_ids", "topk_w", "counts", "offsets", "perm", "inv", "h", "y",
                 "scratch", "total")]


class MoeSharedLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in ("hs", "ys", "total")]


class MoeQ4Spec(ctypes.Structure):
    _fields_ = [("format", ctypes.c_int32), ("group", ctypes.c_int32)]


class MoeQ4Sizes(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in ("w1_codes", "w1_scales", "w2_codes", "w2_scales")]


class MoeLoraSpec(ctypes.Structure):
    _fields_ = [("adapters", ctypes.c_int32), ("rank", ctypes.c_int32)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built; run python __graft_entry__.py build")
    lib = ctypes.CDLL(LIB_PATH)
    P = ctypes.c_void_p
    S = ctypes.POINTER(MoeShape)
    i32 = ctypes.c_int32
    lib.moe_status_string.argtypes = [i32]
    lib.moe_status_string.restype = ctypes.c_char_p
    lib.moe_workspace_size.argtypes = [S]
    lib.moe_workspace_size.restype = ctypes.c_size_t
    lib.moe_get_workspace_layout.argtypes = [S, ctypes.POINTER(MoeWorkspaceLayout)]
    lib.moe_get_workspace_layout.restype = i32
    lib.moe_route.argtypes = [S, P, P, P, P, P, P, P]
    lib.moe_route.restype = i32
    lib.moe_permute.argtypes = [S, P, P, P, P, P, P, P, P]
    lib.moe_permute.restype = i32
    lib.moe_grouped_gemm_w13_swiglu.argtypes = [S, P, P, P, P, P, P]
    lib.moe_grouped_gemm_w13_swiglu.restype = i32
    lib.moe_grouped_gemm_down.argtypes = [S, P, P, P, P, P]
    lib.moe_grouped_gemm_down.restype = i32
    lib.moe_finalize.argtypes = [S, P, P, P, P, P]
    lib.moe_finalize.restype = i32
    lib.moe_forward.argtypes = [S, P, P, P, P, P, P, P, ctypes.c_size_t, P]
    lib.moe_forward.restype = i32
    lib.moe_forward_noalloc.argtypes = [S, P, P, P, P, P, P, P]
    lib.moe_forward_noalloc.restype = i32
    lib.moe_shared_workspace_size.argtypes = [S, i32]
    lib.moe_shared_workspace_size.restype = ctypes.c_size_t
    lib.moe_get_shared_workspace_layout.argtypes = [S, i32, ctypes.POINTER(MoeSharedLayout)]
    lib.moe_get_shared_workspace_layout.restype = i32
    lib.moe_shared_ffn.argtypes = [S, i32, P, P, P, P, P, P]
    lib.moe_shared_ffn.restype = i32
    lib.moe_finalize_shared.argtypes = [S, P, P, P, P, P, P]
    lib.moe_finalize_shared.restype = i32
    lib.moe_forward_shared.argtypes = [S, i32, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
    lib.moe_forward_shared.restype = i32
    Q = ctypes.POINTER(MoeQ4Spec)
    lib.moe_q4_get_sizes.argtypes = [S, Q, ctypes.POINTER(MoeQ4Sizes)]
    lib.moe_q4_quantize_w13.argtypes = [S, Q, P, P, P, P]
    lib.moe_q4_quantize_down.argtypes = [S, Q, P, P, P, P]
    lib.moe_q4_w13_swiglu.argtypes = [S, Q, P, P, P, P, P, P, P]
    lib.moe_q4_down.argtypes = [S, Q, P, P, P, P, P, P]
    lib.moe_forward_q4.argtypes = [S, Q, P, P, P, P, P, P, P, P, P, ctypes.c_size_t, P]
    for f in (lib.moe_q4_get_sizes, lib.moe_q4_quantize_w13, lib.moe_q4_quantize_down, lib.moe_q4_w13_swiglu,
              lib.moe_q4_down, lib.moe_forward_q4):
        f.restype = i32
    lib.moe_balance_workspace_size.argtypes = [S]
    lib.moe_balance_workspace_size.restype = ctypes.c_size_t
    lib.moe_balance_loss.argtypes = [S, P, P, P, P, P, P, P, ctypes.c_size_t, P]
    lib.moe_balance_loss.restype = i32
    lib.moe_route_backward.argtypes = [S, P, P, P, P, P, P, P, P, P]
    lib.moe_route_backward.restype = i32
    lib.moe_router_grad_workspace_size.argtypes = [S]
    lib.moe_router_grad_workspace_size.restype = ctypes.c_size_t
    lib.moe_router_weight_grad.argtypes = [S, P, P, P, P, P, P, ctypes.c_size_t, P]
    lib.moe_router_weight_grad.restype = i32
    lib.moe_finalize_backward.argtypes = [S, P, P, P, P, P]
    lib.moe_finalize_backward.restype = i32
    f64, size = ctypes.c_double, ctypes.c_size_t
    A = ctypes.POINTER(MoeLoraSpec)
    lib.moe_dropout_add.argtypes = [S, f64, P, P, P, P, P]
    lib.moe_dropout_backward.argtypes = [S, f64, P, P, P, P]
    lib.moe_shared_ffn_train.argtypes = [S, i32, f64] + [P] * 9
    lib.moe_shared_backward_workspace_size.argtypes = [S, i32]
    lib.moe_shared_ffn_backward.argtypes = [S, i32, f64] + [P] * 11 + [size, P]
    lib.moe_lora_workspace_size.argtypes = [S, i32, A]
    lib.moe_lora_w13_swiglu.argtypes = [S, i32, A] + [P] * 8 + [size, P]
    lib.moe_lora_down.argtypes = [S, i32, A] + [P] * 9 + [size, P]
    lib.moe_shared_ffn_lora.argtypes = [S, i32, A] + [P] * 13 + [size, P]
    for f in (lib.moe_dropout_add, lib.moe_dropout_backward, lib.moe_shared_ffn_train, lib.moe_shared_ffn_backward,
              lib.moe_lora_w13_swiglu, lib.moe_lora_down, lib.moe_shared_ffn_lora):
        f.restype = i32
    lib.moe_shared_backward_workspace_size.restype = size
    lib.moe_lora_workspace_size.restype = size
    lib.moe_probe_mfma_bf16.argtypes = [i32, P, P]
    lib.moe_probe_mfma_bf16.restype = i32
    lib.moe_probe_mfma_flops.argtypes = [i32]
    lib.moe_probe_mfma_flops.restype = ctypes.c_double
    lib.moe_probe_read.argtypes = [P, ctypes.c_size_t, P, P]
    lib.moe_probe_read.restype = i32
    return lib


lib = _load()


def status_string(code: int) -> str:
    return lib.moe_status_string(code).decode()


def make_shape(T, H, E, k, Im, micro_count=1, dtype="bf16", renormalize=True) -> MoeShape:
    d = {"bf16": MOE_BF16, "f32": MOE_F32, MOE_BF16: MOE_BF16, MOE_F32: MOE_F32}[dtype]
    return MoeShape(T, H, E, k, Im, micro_count, d, int(bool(renormalize)))


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return ctypes.c_void_p(t.data_ptr())


def _layer_dtype(shape) -> torch.dtype:
    return torch.bfloat16 if shape.dtype == MOE_BF16 else torch.float32


def _arg(name: str, t, dtype: torch.dtype, numel: int, nullable: bool = False):
    """Check one tensor argument against the element type and element count
    the C entry point will read or write through its raw pointer (the library
    cannot check sizes itself), then return the pointer."""
    if isinstance(t, torch.Tensor) and t.is_cuda and t.dtype == dtype and t.numel() == numel and t.is_contiguous():
        return t.data_ptr()
    if t is None:
        if nullable:
            return None
        raise ValueError(f"{name}: a tensor is required")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.device.type != "cuda":
        raise ValueError(f"{name}: must be a GPU tensor (got {t.device})")
    if t.dtype != dtype:
        raise ValueError(f"{name}: dtype {t.dtype}, expected {dtype}")
    if t.numel() != numel:
        raise ValueError(f"{name}: {t.numel()} elements, expected {numel} for this shape")
    return _ptr(t)


Y_BLOCK = 256  # columns per exponent of a block-scaled half y (moe_mi355x.h)


def y_nbytes(shape, rows: int) -> int:
    """Bytes of a y buffer of `rows` rows: block-scaled half (fp16 values,
    then one int8 exponent per Y_BLOCK columns) in the bf16 layers, fp32 in
    the fp32 layer."""
    H = shape.H
    if shape.dtype == MOE_BF16:
        return rows * H * 2 + rows * (-(-H // Y_BLOCK))
    return rows * H * 4


def _arg_bytes(name: str, t, nbytes: int):
    """A contiguous GPU tensor of exactly nbytes bytes (any element type)."""
    if isinstance(t, torch.Tensor) and t.is_cuda and t.numel() * t.element_size() == nbytes and t.is_contiguous():
        return t.data_ptr()
    if t is None:
        raise ValueError(f"{name}: a tensor is required")
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor, got {type(t).__name__}")
    if t.device.type != "cuda":
        raise ValueError(f"{name}: must be a GPU tensor (got {t.device})")
    if t.numel() * t.element_size() != nbytes:
        raise ValueError(f"{name}: {t.numel() * t.element_size()} bytes, expected {nbytes} for this shape")
    return _ptr(t)


# the current stream's handle without a Stream object (which costs as much as a small launch)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device())
    return torch.cuda.current_stream().cuda_stream


def _check(code: int, where: str):
    if code != MOE_OK:
        raise MoeError(code, where)


def moe_workspace_size(shape: MoeShape) -> int:
    return int(lib.moe_workspace_size(ctypes.byref(shape)))


def moe_get_workspace_layout(shape: MoeShape) -> dict:
    L = MoeWorkspaceLayout()
    _check(lib.moe_get_workspace_layout(ctypes.byref(shape), ctypes.byref(L)), "moe_get_workspace_layout")
    return {n: int(getattr(L, n)) for n, _ in MoeWorkspaceLayout._fields_}


def moe_route(shape, x, wg, bias, logits, topk_ids, topk_w, stream=None):
    T, H, E, k = shape.T, shape.H, shape.E, shape.k
    dt = _layer_dtype(shape)
    _check(lib.moe_route(ctypes.byref(shape), _arg("x", x, dt, T * H), _arg("wg", wg, torch.float32, E * H),
                         _arg("gate_bias", bias, torch.float32, E, nullable=True),
                         _arg("logits", logits, torch.float32, T * E),
                         _arg("topk_ids", topk_ids, torch.int32, T * k),
                         _arg("topk_w", topk_w, torch.float32, T * k), _stream(stream)), "moe_route")


def moe_permute(shape, topk_ids, counts, offsets, perm, inv, x=None, permuted_x=None, stream=None):
    T, H, E, k = shape.T, shape.H, shape.E, shape.k
    R = T * k
    dt = _layer_dtype(shape)
    _check(lib.moe_permute(ctypes.byref(shape), _arg("topk_ids", topk_ids, torch.int32, R),
                           _arg("counts", counts, torch.int32, E), _arg("offsets", offsets, torch.int32, E + 1),
                           _arg("perm", perm, torch.int32, R), _arg("inv", inv, torch.int32, R),
                           _arg("x", x, dt, T * H, nullable=True),
                           _arg("permuted_x", permuted_x, dt, R * H, nullable=True), _stream(stream)),
           "moe_permute")


def moe_grouped_gemm_w13_swiglu(shape, x, perm, offsets, w1, h, stream=None):
    T, H, E, k, Im, mu = shape.T, shape.H, shape.E, shape.k, shape.Im, shape.micro_count
    R = T * k
    dt = _layer_dtype(shape)
    _check(lib.moe_grouped_gemm_w13_swiglu(ctypes.byref(shape), _arg("x", x, dt, T * H),
                                           _arg("perm", perm, torch.int32, R),
                                           _arg("offsets", offsets, torch.int32, E + 1),
                                           _arg("w1", w1, dt, mu * E * 2 * Im * H),
                                           _arg("h", h, dt, R * mu * Im), _stream(stream)),
           "moe_grouped_gemm_w13_swiglu")


def moe_grouped_gemm_down(shape, h, offsets, w2, y, stream=None):
    T, H, E, k, Im, mu = shape.T, shape.H, shape.E, shape.k, shape.Im, shape.micro_count
    R = T * k
    dt = _layer_dtype(shape)
    _check(lib.moe_grouped_gemm_down(ctypes.byref(shape), _arg("h", h, dt, R * mu * Im),
                                     _arg("offsets", offsets, torch.int32, E + 1),
                                     _arg("w2", w2, dt, mu * E * H * Im), _arg_bytes("y", y, y_nbytes(shape, R)),
                                     _stream(stream)), "moe_grouped_gemm_down")


def moe_finalize(shape, y, inv, topk_w, out, stream=None):
    T, H, k = shape.T, shape.H, shape.k
    R = T * k
    dt = _layer_dtype(shape)
    _check(lib.moe_finalize(ctypes.byref(shape), _arg_bytes("y", y, y_nbytes(shape, R)),
                            _arg("inv", inv, torch.int32, R),
                            _arg("topk_w", topk_w, torch.float32, R), _arg("out", out, dt, T * H),
                            _stream(stream)), "moe_finalize")


def _workspace(workspace):
    if workspace is None:
        raise ValueError("workspace: a tensor is required")
    if not isinstance(workspace, torch.Tensor) or workspace.device.type != "cuda" or not workspace.is_contiguous():
        raise ValueError("workspace: must be a contiguous GPU tensor")
    return _ptr(workspace), ctypes.c_size_t(workspace.numel() * workspace.element_size())


def moe_forward(shape, x, wg, bias, w1, w2, out, workspace, stream=None):
    T, H, E, Im, mu = shape.T, shape.H, shape.E, shape.Im, shape.micro_count
    dt = _layer_dtype(shape)
    ws, nbytes = _workspace(workspace)
    _check(lib.moe_forward(ctypes.byref(shape), _arg("x", x, dt, T * H), _arg("wg", wg, torch.float32, E * H),
                           _arg("gate_bias", bias, torch.float32, E, nullable=True),
                           _arg("w1", w1, dt, mu * E * 2 * Im * H), _arg("w2", w2, dt, mu * E * H * Im),
                           _arg("out", out, dt, T * H), ws, nbytes, _stream(stream)),
           "moe_forward")


NOALLOC_SCRATCH_BYTES = 16 << 20  # MOE_NOALLOC_SCRATCH_BYTES of moe_mi355x.h


def moe_forward_noalloc(shape, x, wg, bias, w1, w2, out, stream=None):
    """moe_forward on the library's static per-GPU scratch (no workspace)."""
    T, H, E, Im, mu = shape.T, shape.H, shape.E, shape.Im, shape.micro_count
    dt = _layer_dtype(shape)
    _check(lib.moe_forward_noalloc(ctypes.byref(shape), _arg("x", x, dt, T * H),
                                   _arg("wg", wg, torch.float32, E * H),
                                   _arg("gate_bias", bias, torch.float32, E, nullable=True),
                                   _arg("w1", w1, dt, mu * E * 2 * Im * H),
                                   _arg("w2", w2, dt, mu * E * H * Im),
                                   _arg("out", out, dt, T * H), _stream(stream)),
           "moe_forward_noalloc")


def moe_shared_workspace_size(shape: MoeShape, Is: int) -> int:
    return int(lib.moe_shared_workspace_size(ctypes.byref(shape), int(Is)))


def moe_get_shared_workspace_layout(shape: MoeShape, Is: int) -> dict:
    L = MoeSharedLayout()
    _check(lib.moe_get_shared_workspace_layout(ctypes.byref(shape), int(Is), ctypes.byref(L)),
           "moe_get_shared_workspace_layout")
    return {n: int(getattr(L, n)) for n, _ in MoeSharedLayout._fields_}


def moe_shared_ffn(shape, Is, x, w1s, w2s, hs, ys, stream=None):
    T, H = shape.T, shape.H
    dt = _layer_dtype(shape)
    _check(lib.moe_shared_ffn(ctypes.byref(shape), int(Is), _arg("x", x, dt, T * H),
                              _arg("w1s", w1s, dt, 2 * Is * H), _arg("w2s", w2s, dt, H * Is),
                              _arg("hs", hs, dt, T * Is), _arg_bytes("ys", ys, y_nbytes(shape, T)),
                              _stream(stream)),
           "moe_shared_ffn")


def moe_finalize_shared(shape, y, inv, topk_w, ys, out, stream=None):
    T, H, k = shape.T, shape.H, shape.k
    R = T * k
    dt = _layer_dtype(shape)
    _check(lib.moe_finalize_shared(ctypes.byref(shape), _arg_bytes("y", y, y_nbytes(shape, R)),
                                   _arg("inv", inv, torch.int32, R),
                                   _arg("topk_w", topk_w, torch.float32, R), _arg_bytes("ys", ys, y_nbytes(shape, T)),
                                   _arg("out", out, dt, T * H), _stream(stream)), "moe_finalize_shared")


def moe_forward_shared(shape, Is, x, wg, bias, w1, w2, w1s, w2s, out, workspace, stream=None):
    T, H, E, Im, mu = shape.T, shape.H, shape.E, shape.Im, shape.micro_count
    dt = _layer_dtype(shape)
    ws, nbytes = _workspace(workspace)
    _check(lib.moe_forward_shared(ctypes.byref(shape), int(Is), _arg("x", x, dt, T * H),
                                  _arg("wg", wg, torch.float32, E * H),
                                  _arg("gate_bias", bias, torch.float32, E, nullable=True),
                                  _arg("w1", w1, dt, mu * E * 2 * Im * H), _arg("w2", w2, dt, mu * E * H * Im),
                                  _arg("w1s", w1s, dt, 2 * Is * H), _arg("w2s", w2s, dt, H * Is),
                                  _arg("out", out, dt, T * H), ws, nbytes, _stream(stream)),
           "moe_forward_shared")


def _on_current(*tensors, stream=None):
    """The library launches on the current device: every (GPU) tensor and the stream have to be on it."""
    here = torch.cuda.current_device()
    if stream is not None and getattr(stream, "device_index", here) != here:
        raise ValueError(f"the stream is on cuda:{stream.device_index}, the current device is cuda:{here}")
    for t in tensors:
        if t is not None and t.get_device() != here:
            raise ValueError(f"a tensor is on {t.device}, the current device is cuda:{here}")


# ---- 4-bit expert weights (moe_q4.h)


def make_q4(format="int4", group=128) -> MoeQ4Spec:
    """A 4-bit weight format: "int4" or "e2m1", `group` columns per scale (32, 64 or 128)."""
    return MoeQ4Spec({"int4": MOE_Q4_INT4, "e2m1": MOE_Q4_E2M1, MOE_Q4_INT4: MOE_Q4_INT4, MOE_Q4_E2M1: MOE_Q4_E2M1}[format], group)


def moe_q4_get_sizes(shape, q4) -> dict:
    """Bytes of the stored 4-bit weights of a layer."""
    z = MoeQ4Sizes()
    _check(lib.moe_q4_get_sizes(ctypes.byref(shape), ctypes.byref(q4), ctypes.byref(z)), "moe_q4_get_sizes")
    return {n: int(getattr(z, n)) for n, _ in MoeQ4Sizes._fields_}


def moe_q4_quantize_w13(shape, q4, w1, codes, scales, stream=None):
    """Quantise w1 [mu, E, 2*Im, H] (layer dtype) into 4-bit storage."""
    z = moe_q4_get_sizes(shape, q4)
    args = (_arg("w1", w1, _layer_dtype(shape), shape.micro_count * shape.E * 2 * shape.Im * shape.H),
            _arg_bytes("codes", codes, z["w1_codes"]), _arg_bytes("scales", scales, z["w1_scales"]))
    _on_current(w1, codes, scales, stream=stream)
    _check(lib.moe_q4_quantize_w13(ctypes.byref(shape), ctypes.byref(q4), *args, _stream(stream)),
           "moe_q4_quantize_w13")


def moe_q4_quantize_down(shape, q4, w2, codes, scales, stream=None):
    """Quantise w2 [mu, E, H, Im] (layer dtype) into 4-bit storage."""
    z = moe_q4_get_sizes(shape, q4)
    args = (_arg("w2", w2, _layer_dtype(shape), shape.micro_count * shape.E * shape.H * shape.Im),
            _arg_bytes("codes", codes, z["w2_codes"]), _arg_bytes("scales", scales, z["w2_scales"]))
    _on_current(w2, codes, scales, stream=stream)
    _check(lib.moe_q4_quantize_down(ctypes.byref(shape), ctypes.byref(q4), *args, _stream(stream)),
           "moe_q4_quantize_down")


def moe_q4_w13_swiglu(shape, q4, x, perm, offsets, w1_codes, w1_scales, h, stream=None):
    T, H, E, R = shape.T, shape.H, shape.E, shape.T * shape.k
    dt, z = _layer_dtype(shape), moe_q4_get_sizes(shape, q4)
    args = (_arg("x", x, dt, T * H), _arg("perm", perm, torch.int32, R), _arg("offsets", offsets, torch.int32, E + 1),
            _arg_bytes("w1_codes", w1_codes, z["w1_codes"]), _arg_bytes("w1_scales", w1_scales, z["w1_scales"]),
            _arg("h", h, dt, R * shape.micro_count * shape.Im))
    _on_current(x, perm, offsets, w1_codes, w1_scales, h, stream=stream)
    _check(lib.moe_q4_w13_swiglu(ctypes.byref(shape), ctypes.byref(q4), *args, _stream(stream)), "moe_q4_w13_swiglu")


def moe_q4_down(shape, q4, h, offsets, w2_codes, w2_scales, y, stream=None):
    E, R = shape.E, shape.T * shape.k
    z = moe_q4_get_sizes(shape, q4)
    args = (_arg("h", h, _layer_dtype(shape), R * shape.micro_count * shape.Im),
            _arg("offsets", offsets, torch.int32, E + 1), _arg_bytes("w2_codes", w2_codes, z["w2_codes"]),
            _arg_bytes("w2_scales", w2_scales, z["w2_scales"]), _arg_bytes("y", y, y_nbytes(shape, R)))
    _on_current(h, offsets, w2_codes, w2_scales, y, stream=stream)
    _check(lib.moe_q4_down(ctypes.byref(shape), ctypes.byref(q4), *args, _stream(stream)), "moe_q4_down")


def moe_forward_q4(shape, q4, x, wg, bias, w1_codes, w1_scales, w2_codes, w2_scales, out, workspace, stream=None):
    """moe_forward over 4-bit expert weights."""
    T, H, E = shape.T, shape.H, shape.E
    dt, z = _layer_dtype(shape), moe_q4_get_sizes(shape, q4)
    args = (_arg("x", x, dt, T * H), _arg("wg", wg, torch.float32, E * H),
            _arg("gate_bias", bias, torch.float32, E, nullable=True),
            _arg_bytes("w1_codes", w1_codes, z["w1_codes"]), _arg_bytes("w1_scales", w1_scales, z["w1_scales"]),
            _arg_bytes("w2_codes", w2_codes, z["w2_codes"]), _arg_bytes("w2_scales", w2_scales, z["w2_scales"]),
            _arg("out", out, dt, T * H))
    ws, nbytes = _workspace(workspace)
    _on_current(x, wg, bias, w1_codes, w1_scales, w2_codes, w2_scales, out, workspace, stream=stream)
    _check(lib.moe_forward_q4(ctypes.byref(shape), ctypes.byref(q4), *args, ws, nbytes, _stream(stream)),
           "moe_forward_q4")


# ---- router gradients (moe_router_grad.h)


def moe_balance_workspace_size(shape: MoeShape) -> int:
    return int(lib.moe_balance_workspace_size(ctypes.byref(shape)))


def moe_balance_loss(shape, logits, topk_ids, token_mask, counts, mean_prob, loss, workspace, stream=None):
    """Per-expert counts, mean router probabilities and the balance loss of the valid tokens."""
    T, E, k = shape.T, shape.E, shape.k
    args = (_arg("logits", logits, torch.float32, T * E), _arg("topk_ids", topk_ids, torch.int32, T * k),
            _arg("token_mask", token_mask, torch.uint8, T, nullable=True), _arg("counts", counts, torch.int32, E),
            _arg("mean_prob", mean_prob, torch.float32, E), _arg("loss", loss, torch.float32, 1))
    ws, nbytes = _workspace(workspace)
    _on_current(logits, topk_ids, token_mask, counts, mean_prob, loss, workspace, stream=stream)
    _check(lib.moe_balance_loss(ctypes.byref(shape), *args, ws, nbytes, _stream(stream)), "moe_balance_loss")


def moe_route_backward(shape, logits, topk_ids, topk_w, token_mask, counts, d_topk_w, d_loss, d_logits, stream=None):
    """Gradient of the router logits from those of the routing weights and of the balance loss (either may be None)."""
    T, E, k = shape.T, shape.E, shape.k
    unread = d_topk_w is None
    args = (_arg("logits", logits, torch.float32, T * E),
            _arg("topk_ids", topk_ids, torch.int32, T * k, nullable=unread),
            _arg("topk_w", topk_w, torch.float32, T * k, nullable=unread),
            _arg("token_mask", token_mask, torch.uint8, T, nullable=True),
            _arg("counts", counts, torch.int32, E, nullable=True),
            _arg("d_topk_w", d_topk_w, torch.float32, T * k, nullable=True),
            _arg("d_loss", d_loss, torch.float32, 1, nullable=True),
            _arg("d_logits", d_logits, torch.float32, T * E))
    _on_current(logits, topk_ids, topk_w, token_mask, counts, d_topk_w, d_loss, d_logits, stream=stream)
    _check(lib.moe_route_backward(ctypes.byref(shape), *args, _stream(stream)), "moe_route_backward")


def moe_router_grad_workspace_size(shape: MoeShape) -> int:
    return int(lib.moe_router_grad_workspace_size(ctypes.byref(shape)))


def moe_router_weight_grad(shape, x, d_logits, token_mask, d_wg, d_bias, workspace, stream=None):
    """Gradients of the router's weight and (unless d_bias is None) bias."""
    T, H, E = shape.T, shape.H, shape.E
    args = (_arg("x", x, _layer_dtype(shape), T * H), _arg("d_logits", d_logits, torch.float32, T * E),
            _arg("token_mask", token_mask, torch.uint8, T, nullable=True),
            _arg("d_wg", d_wg, torch.float32, E * H), _arg("d_bias", d_bias, torch.float32, E, nullable=True))
    ws, nbytes = _workspace(workspace)
    _on_current(x, d_logits, token_mask, d_wg, d_bias, workspace, stream=stream)
    _check(lib.moe_router_weight_grad(ctypes.byref(shape), *args, ws, nbytes, _stream(stream)),
           "moe_router_weight_grad")


def moe_finalize_backward(shape, y, inv, d_out, d_topk_w, stream=None):
    """Gradient of the routing weights from the output's (y as the down projection wrote it)."""
    T, H, k = shape.T, shape.H, shape.k
    R = T * k
    args = (_arg_bytes("y", y, y_nbytes(shape, R)), _arg("inv", inv, torch.int32, R),
            _arg("d_out", d_out, _layer_dtype(shape), T * H), _arg("d_topk_w", d_topk_w, torch.float32, R))
    _on_current(y, inv, d_out, d_topk_w, stream=stream)
    _check(lib.moe_finalize_backward(ctypes.byref(shape), *args, _stream(stream)), "moe_finalize_backward")


# ---- shared expert's training and dropout (moe_shared_train.h)

_get_device = getattr(torch._C, "_cuda_getDevice", None)


def _here() -> int:
    """The current device (without torch.cuda's initialisation check: a GPU tensor exists, or no argument passes)."""
    try:
        return _get_device() if _get_device is not None else torch.cuda.current_device()
    except RuntimeError:
        return -2


def _on(here: int, name: str, t, dtype: torch.dtype, numel: int, nullable: bool = False):
    """_arg for a tensor that has to be on the current device."""
    try:
        if t.dtype is dtype and t.numel() == numel and t.get_device() == here and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:  # no tensor: _arg says so
        pass
    p = _arg(name, t, dtype, numel, nullable)
    if t is not None:
        _on_current(t)
    return p


def _workspace_on(here: int, workspace):
    ws, nbytes = _workspace(workspace)
    if workspace.get_device() != here:
        _on_current(workspace)
    return ws, nbytes


def _stream_on(here: int, stream):
    if stream is None and _raw_stream is not None:
        return _raw_stream(here)
    _on_current(stream=stream)
    return _stream(stream)


def _rng_on(here: int, p, rng):
    """The random stream's seed and offset (an int64 tensor of two on the GPU); unread where nothing is dropped."""
    return _on(here, "rng", rng, torch.int64, 2, nullable=not p >= 1 / 131072)


def moe_dropout_add(shape, p, rng, y, residual, out, stream=None):
    """out = residual (or None) + dropout(y); rng: int64 [2] on the GPU, seed and offset."""
    n, dt, here = shape.T * shape.H, _layer_dtype(shape), _here()
    _check(lib.moe_dropout_add(ctypes.byref(shape), float(p), _rng_on(here, p, rng), _on(here, "y", y, dt, n),
                               _on(here, "residual", residual, dt, n, True), _on(here, "out", out, dt, n),
                               _stream_on(here, stream)), "moe_dropout_add")


def moe_dropout_backward(shape, p, rng, d_out, d_y, stream=None):
    """Gradient of moe_dropout_add's y, with the forward call's p and rng."""
    n, dt, here = shape.T * shape.H, _layer_dtype(shape), _here()
    _check(lib.moe_dropout_backward(ctypes.byref(shape), float(p), _rng_on(here, p, rng), _on(here, "d_out", d_out, dt, n),
                                    _on(here, "d_y", d_y, dt, n), _stream_on(here, stream)), "moe_dropout_backward")


def moe_shared_ffn_train(shape, Is, p, rng, x, w1s, w2s, residual, gu, hs, out, stream=None):
    """The shared expert's forward pass with dropout of its hidden values; keeps gu (fp32) and hs for the backward pass."""
    T, H, dt, here = shape.T, shape.H, _layer_dtype(shape), _here()
    _check(lib.moe_shared_ffn_train(ctypes.byref(shape), int(Is), float(p), _rng_on(here, p, rng), _on(here, "x", x, dt, T * H),
                                    _on(here, "w1s", w1s, dt, 2 * Is * H), _on(here, "w2s", w2s, dt, H * Is),
                                    _on(here, "residual", residual, dt, T * H, True),
                                    _on(here, "gu", gu, torch.float32, T * 2 * Is), _on(here, "hs", hs, dt, T * Is),
                                    _on(here, "out", out, dt, T * H), _stream_on(here, stream)), "moe_shared_ffn_train")


def moe_shared_backward_workspace_size(shape: MoeShape, Is: int) -> int:
    return int(lib.moe_shared_backward_workspace_size(ctypes.byref(shape), int(Is)))


def moe_shared_ffn_backward(shape, Is, p, rng, x, w1s, w2s, gu, hs, d_out, d_x, d_w1s, d_w2s, workspace, stream=None):
    """Gradients of x (unless d_x is None) and of both weights (unless d_w1s and d_w2s are None)."""
    T, H, dt, here = shape.T, shape.H, _layer_dtype(shape), _here()
    no_x, no_w = d_x is None, d_w1s is None and d_w2s is None
    _check(lib.moe_shared_ffn_backward(
        ctypes.byref(shape), int(Is), float(p), _rng_on(here, p, rng), _on(here, "x", x, dt, T * H, no_w),
        _on(here, "w1s", w1s, dt, 2 * Is * H, no_x), _on(here, "w2s", w2s, dt, H * Is),
        _on(here, "gu", gu, torch.float32, T * 2 * Is), _on(here, "hs", hs, dt, T * Is, no_w),
        _on(here, "d_out", d_out, dt, T * H), _on(here, "d_x", d_x, dt, T * H, True),
        _on(here, "d_w1s", d_w1s, dt, 2 * Is * H, True), _on(here, "d_w2s", d_w2s, dt, H * Is, True), *_workspace_on(here, workspace),
        _stream_on(here, stream)), "moe_shared_ffn_backward")


# ---- request adapters (moe_lora.h)


def make_lora(adapters, rank) -> MoeLoraSpec:
    """A set of `adapters` low-rank adapters of one rank (a multiple of 8)."""
    return MoeLoraSpec(adapters, rank)


def moe_lora_workspace_size(shape: MoeShape, Is: int, lora: MoeLoraSpec) -> int:
    return int(lib.moe_lora_workspace_size(ctypes.byref(shape), int(Is), ctypes.byref(lora)))


def moe_lora_w13_swiglu(shape, Is, lora, x, w1s, a1, b1, scale, adapter_ids, hs, workspace, stream=None):
    """SwiGLU of the shared expert's gate and up projection, every token with its own adapter."""
    T, H, dt, here = shape.T, shape.H, _layer_dtype(shape), _here()
    L, n = lora.adapters, lora.adapters * lora.rank
    _check(lib.moe_lora_w13_swiglu(
        ctypes.byref(shape), int(Is), ctypes.byref(lora), _on(here, "x", x, dt, T * H), _on(here, "w1s", w1s, dt, 2 * Is * H),
        _on(here, "a1", a1, dt, n * H), _on(here, "b1", b1, dt, n * 2 * Is), _on(here, "scale", scale, torch.float32, L),
        _on(here, "adapter_ids", adapter_ids, torch.int32, T), _on(here, "hs", hs, dt, T * Is), *_workspace_on(here, workspace),
        _stream_on(here, stream)), "moe_lora_w13_swiglu")


def moe_lora_down(shape, Is, lora, hs, w2s, a2, b2, scale, adapter_ids, residual, out, workspace, stream=None):
    """The shared expert's down projection, every token with its own adapter, plus the residual (or None)."""
    T, H, dt, here = shape.T, shape.H, _layer_dtype(shape), _here()
    L, n = lora.adapters, lora.adapters * lora.rank
    _check(lib.moe_lora_down(
        ctypes.byref(shape), int(Is), ctypes.byref(lora), _on(here, "hs", hs, dt, T * Is), _on(here, "w2s", w2s, dt, H * Is),
        _on(here, "a2", a2, dt, n * Is), _on(here, "b2", b2, dt, n * H), _on(here, "scale", scale, torch.float32, L),
        _on(here, "adapter_ids", adapter_ids, torch.int32, T), _on(here, "residual", residual, dt, T * H, True),
        _on(here, "out", out, dt, T * H), *_workspace_on(here, workspace), _stream_on(here, stream)), "moe_lora_down")


def moe_shared_ffn_lora(shape, Is, lora, x, w1s, w2s, a1, b1, a2, b2, scale, adapter_ids, residual, hs, out, workspace,
                        stream=None):
    """The shared expert with adapters on both projections, plus the residual (or None)."""
    T, H, dt, here = shape.T, shape.H, _layer_dtype(shape), _here()
    L, n = lora.adapters, lora.adapters * lora.rank
    _check(lib.moe_shared_ffn_lora(
        ctypes.byref(shape), int(Is), ctypes.byref(lora), _on(here, "x", x, dt, T * H), _on(here, "w1s", w1s, dt, 2 * Is * H),
        _on(here, "w2s", w2s, dt, H * Is), _on(here, "a1", a1, dt, n * H), _on(here, "b1", b1, dt, n * 2 * Is),
        _on(here, "a2", a2, dt, n * Is), _on(here, "b2", b2, dt, n * H), _on(here, "scale", scale, torch.float32, L),
        _on(here, "adapter_ids", adapter_ids, torch.int32, T), _on(here, "residual", residual, dt, T * H, True),
        _on(here, "hs", hs, dt, T * Is), _on(here, "out", out, dt, T * H), *_workspace_on(here, workspace),
        _stream_on(here, stream)), "moe_shared_ffn_lora")


def moe_probe_mfma_bf16(iterations: int, sink, stream=None) -> float:
    """Enqueue the bf16 matrix-rate probe; returns the FLOPs it performs."""
    _check(lib.moe_probe_mfma_bf16(int(iterations), _arg("sink", sink, torch.float32, 1), _stream(stream)),
           "moe_probe_mfma_bf16")
    return float(lib.moe_probe_mfma_flops(int(iterations)))


def moe_probe_read(buf, sink, stream=None) -> int:
    """Enqueue the streaming-read probe over all of `buf`; returns its bytes."""
    if not isinstance(buf, torch.Tensor) or buf.device.type != "cuda":
        raise ValueError("buf: must be a GPU tensor")
    nbytes = buf.numel() * buf.element_size()
    _check(lib.moe_probe_read(_ptr(buf), ctypes.c_size_t(nbytes), _arg("sink", sink, torch.int32, 1),
                              _stream(stream)), "moe_probe_read")
    return nbytes
