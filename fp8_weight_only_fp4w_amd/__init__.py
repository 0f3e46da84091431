"""Python binding of libfp4w: block-scaled weight-only FP4 / FP8 matmul on
AMD MI355X (gfx950).

Argument marshalling only.  Every step of the computation runs in the HIP
kernels of libfp4w.so; torch supplies device memory and the current stream.
There is no fallback: if the library is missing, every call raises.

The functions carry the C ABI's names (include/fp4w.h):

* ``fp4w_matmul(A, B, weight_scale, weight_scale_2, bias=None, block_size=16)``
  Y = A * dequant(B)^T (+ bias), B packed E2M1 [N, K/2] (low nibble = even k),
  weight_scale E4M3 bytes [N, cols], weight_scale_2 a 1-element FP32 device
  tensor ("MatMulBlockQuantizedFp4Weight - CUDA Operator Documentation" §2).
* ``fp8w_matmul(A, B, b_scale, bias=None, block_size=128)``: B E4M3 [N, K],
  b_scale FP32 [N, cols] ("MatMulBlockQuantizedFp8Weight - CUDA Operator
  Documentation" §2).
* ``fp4w_dequant(B, weight_scale, weight_scale_2, block_size=16, dtype=...)``:
  the [N, K] FP16/BF16 expansion of B.
* ``fp8w_dequant(B, b_scale, block_size=128, dtype=...)``: the [N, K]
  FP16/BF16 expansion of FP8 weights (FP8 document §5, step 1).
* ``fp8w_qdq_activation(A, a_scale)``: fp8_e4m3(A / a_scale) * a_scale in A's
  dtype, the activation step of the FP8 operator's optional W8A8 mode (FP8
  document §6).
* ``fp8w_matmul_w8a8(A, B, b_scale, a_scale, bias=None, block_size=128)``:
  that step into a workspace, then ``fp8w_matmul`` on it.
* ``fp4w_quantize_activation(A)``: (codes [M, K/2], scales [M, K/16]), the
  NVFP4 activation of the FP4 operator's native FP4 x FP4 path (FP4 document
  §6, Native SM120 FP4 x FP4 Path); ``fp4w_qdq_activation(A)``: the same,
  decoded back to A's dtype.
* ``fp4w_matmul_w4a4(A, B, weight_scale, weight_scale_2, bias=None,
  block_size=16)``: that activation times the FP4 weights (W4A4);
  ``fp4w_matmul_w4a4_noalloc(...)``: the same with the activation staged in
  the library's own device scratch, for callers that cannot allocate.
* ``fp4w_moe(A, ids, weights, w13, w13_scale, w13_scale_2, w2, w2_scale,
  w2_scale_2)`` and ``fp8w_moe(A, ids, weights, w13, w13_scale, w2, w2_scale)``:
  a whole mixture-of-experts layer for a few tokens on such weights;
  ``fp4w_moe_route(logits, topk)``: its ids and weights from router logits;
  ``fp4w_block_norm(x, residual, pre_weight, ...)``: the norms after one block
  and before the next, with gate and residual scale.
* ``fp4w_qk_norm_rope(q, k, ...)``: norms of query and key heads with the
  rotation by position; ``fp8w_kv_append(k, v, cache, ...)``: new keys and
  values (normed and rotated on the way) into a paged cache of E4M3 codes with
  a power of two for each page and head (``fp8w_kv_cache`` makes one);
  ``fp8w_attention(q, cache, ...)``: attention over it, for decoded tokens and
  prompts.

A keeps any leading dimensions; Y has A's leading dimensions, last dimension
N and A's dtype.
"""

import ctypes
import functools
import os
from typing import NamedTuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libfp4w.so")

# status codes (fp4w_status)
OK, ERR_NULL, ERR_SHAPE, ERR_DTYPE, ERR_BLOCK, ERR_PATH, ERR_LAUNCH, ERR_ALIAS = 0, -1, -2, -3, -4, -5, -6, -7
# kernel paths (fp4w_path)
PATH_AUTO, PATH_NONE = 0, 1
PATH_FP4_GEMV, PATH_FP4_GEMM, PATH_FP4_GENERIC = 2, 3, 4
PATH_FP8_GEMV, PATH_FP8_GEMM, PATH_FP8_GENERIC = 5, 6, 7
PATH_DEQUANT_VEC, PATH_DEQUANT_GENERIC = 8, 9
PATH_QDQ_VEC, PATH_QDQ_GENERIC = 10, 11
PATH_FP4_SKINNY, PATH_FP8_SKINNY = 12, 13
PATH_FP8_DEQUANT_VEC, PATH_FP8_DEQUANT_GENERIC = 14, 15
PATH_NVFP4_VEC, PATH_NVFP4_GENERIC = 16, 17
PATH_MOE_FP4_STREAM, PATH_MOE_FP4_GENERIC, PATH_MOE_FP8_STREAM, PATH_MOE_FP8_GENERIC = 18, 19, 20, 21
PATH_ATTN_DECODE, PATH_ATTN_PROMPT, PATH_ATTN_GENERIC = 22, 23, 24
# operations (fp4w_op)
OP_FP4_MATMUL, OP_FP8_MATMUL, OP_FP4_DEQUANT, OP_FP8_QDQ, OP_FP8_DEQUANT, OP_NVFP4_ACT = 0, 1, 2, 3, 4, 5
# dtypes (fp4w_dtype)
F16, BF16, F32 = 0, 1, 2
# scores (fp4w_score) and activations (fp4w_activation) by name
SCORES = {"softmax": 0, "sigmoid": 1}
ACTIVATIONS = {"silu": 0, "gelu": 1}
MOE_MAX_EXPERTS, MOE_MAX_TOPK = 1024, 64
MAX_HEAD_SIZE = 1024  # FP8W_MAX_HEAD_SIZE

EXPORTED = (
    "fp4w_matmul", "fp4w_matmul_ex", "fp8w_matmul", "fp8w_matmul_ex", "fp4w_dequant",
    "fp4w_dequant_ex", "fp8w_dequant", "fp8w_dequant_ex", "fp8w_qdq_activation", "fp8w_qdq_activation_ex", "fp8w_matmul_w8a8",
    "fp4w_quantize_activation", "fp4w_quantize_activation_ex", "fp4w_qdq_activation", "fp4w_qdq_activation_ex",
    "fp4w_matmul_w4a4", "fp4w_matmul_w4a4_noalloc",
    "fp4w_block_norm", "fp4w_moe_route", "fp4w_moe_workspace", "fp4w_moe", "fp4w_moe_ex", "fp8w_moe", "fp8w_moe_ex",
    "fp4w_qk_norm_rope", "fp8w_kv_append", "fp8w_attention", "fp8w_attention_ex", "fp8w_attention_workspace",
    "fp4w_select_path", "fp4w_status_string", "fp4w_path_name",
)


class FP4WError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {fp4w_status_string(status)} (status {status})")
        self.status = status


_lib = None


def load_library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libfp4w.so once (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m fp8_weight_only_fp4w_amd.build`")
    lib = ctypes.CDLL(path)
    i64, vp, i32 = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int
    lib.fp4w_matmul_ex.argtypes = [vp, i64, i64, vp, i64, vp, i64, i64, vp, vp, vp, i32, vp, i32]
    lib.fp4w_matmul_ex.restype = i32
    lib.fp4w_matmul.argtypes = [vp, i64, i64, vp, i64, vp, i64, i64, vp, vp, vp, i32, vp]
    lib.fp4w_matmul.restype = i32
    lib.fp8w_matmul_ex.argtypes = [vp, i64, i64, vp, i64, vp, i64, i64, vp, vp, i32, vp, i32]
    lib.fp8w_matmul_ex.restype = i32
    lib.fp8w_matmul.argtypes = [vp, i64, i64, vp, i64, vp, i64, i64, vp, vp, i32, vp]
    lib.fp8w_matmul.restype = i32
    lib.fp4w_dequant_ex.argtypes = [vp, i64, i64, vp, i64, i64, vp, vp, i32, vp, i32]
    lib.fp4w_dequant_ex.restype = i32
    lib.fp4w_dequant.argtypes = [vp, i64, i64, vp, i64, i64, vp, vp, i32, vp]
    lib.fp4w_dequant.restype = i32
    lib.fp8w_dequant_ex.argtypes = [vp, i64, i64, vp, i64, i64, vp, i32, vp, i32]
    lib.fp8w_dequant_ex.restype = i32
    lib.fp8w_dequant.argtypes = [vp, i64, i64, vp, i64, i64, vp, i32, vp]
    lib.fp8w_dequant.restype = i32
    lib.fp8w_qdq_activation_ex.argtypes = [vp, i64, i64, vp, vp, i32, vp, i32]
    lib.fp8w_qdq_activation_ex.restype = i32
    lib.fp8w_qdq_activation.argtypes = [vp, i64, i64, vp, vp, i32, vp]
    lib.fp8w_qdq_activation.restype = i32
    lib.fp8w_matmul_w8a8.argtypes = [vp, i64, i64, vp, i64, vp, i64, i64, vp, vp, vp, vp, i32, vp]
    lib.fp8w_matmul_w8a8.restype = i32
    lib.fp4w_quantize_activation_ex.argtypes = [vp, i64, i64, vp, vp, i32, vp, i32]
    lib.fp4w_quantize_activation_ex.restype = i32
    lib.fp4w_quantize_activation.argtypes = [vp, i64, i64, vp, vp, i32, vp]
    lib.fp4w_quantize_activation.restype = i32
    lib.fp4w_qdq_activation_ex.argtypes = [vp, i64, i64, vp, i32, vp, i32]
    lib.fp4w_qdq_activation_ex.restype = i32
    lib.fp4w_qdq_activation.argtypes = [vp, i64, i64, vp, i32, vp]
    lib.fp4w_qdq_activation.restype = i32
    lib.fp4w_matmul_w4a4.argtypes = [vp, i64, i64, vp, i64, vp, i64, i64, vp, vp, vp, vp, i32, vp]
    lib.fp4w_matmul_w4a4.restype = i32
    lib.fp4w_matmul_w4a4_noalloc.argtypes = [vp, i64, i64, vp, i64, vp, i64, i64, vp, vp, vp, i32, vp]
    lib.fp4w_matmul_w4a4_noalloc.restype = i32
    f32 = ctypes.c_float
    lib.fp4w_block_norm.argtypes = [vp, i64, i64, vp, vp, i64, f32, vp, vp, f32, f32, vp, vp, i32, vp]
    lib.fp4w_block_norm.restype = i32
    lib.fp4w_moe_route.argtypes = [vp, i64, i64, i64, i32, vp, i32, f32, vp, vp, i32, vp]
    lib.fp4w_moe_route.restype = i32
    lib.fp4w_moe_workspace.argtypes = [i64, i64, i64, i64]
    lib.fp4w_moe_workspace.restype = i64
    moe = [vp, i64, i64, vp, vp, i64, vp, vp, vp, vp, vp, vp, i64, i64, i64, i32, vp, i64, vp, i32, vp]
    lib.fp4w_moe.argtypes, lib.fp4w_moe.restype = moe, i32
    lib.fp4w_moe_ex.argtypes, lib.fp4w_moe_ex.restype = moe + [i32], i32
    moe = [vp, i64, i64, vp, vp, i64, vp, vp, vp, vp, i64, i64, i64, i32, vp, i64, vp, i32, vp]
    lib.fp8w_moe.argtypes, lib.fp8w_moe.restype = moe, i32
    lib.fp8w_moe_ex.argtypes, lib.fp8w_moe_ex.restype = moe + [i32], i32
    rope = [vp, vp, f32, f32, vp, vp, i64, i64, i32, vp]
    cache = [vp, vp, vp, vp, i64, i64]
    lib.fp4w_qk_norm_rope.argtypes = [vp, i64, i64, vp, i64, i64, i64, i64, *rope, vp, i64, vp, i64, i32, vp]
    lib.fp4w_qk_norm_rope.restype = i32
    lib.fp8w_kv_append.argtypes = [vp, i64, vp, i64, i64, i64, i64, vp, i64, i64, *rope, vp, i64, vp, i64, vp, vp, i64,
                                   *cache, i32, vp]
    lib.fp8w_kv_append.restype = i32
    lib.fp8w_attention_workspace.argtypes = [i64] * 6
    lib.fp8w_attention_workspace.restype = i64
    attn = [vp, i64, i64, i64, i64, i64, vp, i64, vp, vp, i64, i64, *cache, f32, i32, i64, vp, i64, vp, vp, i32, vp]
    lib.fp8w_attention.argtypes, lib.fp8w_attention.restype = attn, i32
    lib.fp8w_attention_ex.argtypes, lib.fp8w_attention_ex.restype = attn + [i32], i32
    lib.fp4w_select_path.argtypes = [i32, i64, i64, i64, i64, i64]
    lib.fp4w_select_path.restype = i32
    lib.fp4w_status_string.argtypes = [i32]
    lib.fp4w_status_string.restype = ctypes.c_char_p
    lib.fp4w_path_name.argtypes = [i32]
    lib.fp4w_path_name.restype = ctypes.c_char_p
    _lib = lib
    return lib


def fp4w_status_string(status: int) -> str:
    return load_library().fp4w_status_string(int(status)).decode()


def fp4w_path_name(path: int) -> str:
    return load_library().fp4w_path_name(int(path)).decode()


def fp4w_select_path(op: int, M: int, N: int, K: int, block_size: int, scale_cols: int) -> int:
    return int(load_library().fp4w_select_path(op, M, N, K, block_size, scale_cols))


# ---------------------------------------------------------------- marshalling

def _dtype_code(t: torch.dtype) -> int:
    if t is torch.bfloat16:
        return BF16
    if t is torch.float16:
        return F16
    raise TypeError(f"activation dtype must be float16 or bfloat16, got {t}")


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _bytes(t: torch.Tensor) -> torch.Tensor:
    """uint8 view of a uint8 / float8_e4m3fn tensor."""
    if t.dtype == torch.uint8:
        return t
    if t.dtype == torch.float8_e4m3fn:
        return t.view(torch.uint8)
    raise TypeError(f"expected uint8 or float8_e4m3fn bytes, got {t.dtype}")


def _need(t: torch.Tensor, name: str, device: torch.device):
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")


def _stream(device: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _check(status: int, what: str):
    if status != OK:
        raise FP4WError(status, what)


def fp4w_matmul(A: torch.Tensor, B: torch.Tensor, weight_scale: torch.Tensor,
                weight_scale_2: torch.Tensor, bias: torch.Tensor = None, block_size: int = 16,
                out: torch.Tensor = None, path: int = PATH_AUTO) -> torch.Tensor:
    lib = load_library()
    dev = A.device
    B, weight_scale = _bytes(B), _bytes(weight_scale)
    K = A.shape[-1]
    M = A.numel() // K if K else int(torch.tensor(A.shape[:-1]).prod().item())
    N = B.shape[0]
    if B.dim() != 2 or B.shape[1] * 2 != K:
        raise ValueError(f"B must be [N, K/2] = [N, {K // 2}], got {tuple(B.shape)}")
    if weight_scale.dim() != 2 or weight_scale.shape[0] != N:
        raise ValueError("weight_scale must be [N, scale_cols]")
    if weight_scale_2.dtype != torch.float32 or weight_scale_2.numel() != 1:
        raise ValueError("weight_scale_2 must be a 1-element float32 tensor")
    for t, name in ((A, "A"), (B, "B"), (weight_scale, "weight_scale"), (weight_scale_2, "weight_scale_2")):
        _need(t, name, dev)
    if bias is not None:
        _need(bias, "bias", dev)
        if bias.dtype != A.dtype or bias.numel() != N:
            raise ValueError("bias must be [N] with A's dtype")
    if out is None:
        out = torch.empty(*A.shape[:-1], N, dtype=A.dtype, device=dev)
    _need(out, "out", dev)
    st = lib.fp4w_matmul_ex(_ptr(A), M, K, _ptr(B), N, _ptr(weight_scale), weight_scale.shape[1],
                            block_size, _ptr(weight_scale_2), _ptr(bias), _ptr(out),
                            _dtype_code(A.dtype), _stream(dev), path)
    _check(st, "fp4w_matmul")
    return out


def fp8w_matmul(A: torch.Tensor, B: torch.Tensor, b_scale: torch.Tensor, bias: torch.Tensor = None,
                block_size: int = 128, out: torch.Tensor = None, path: int = PATH_AUTO) -> torch.Tensor:
    lib = load_library()
    dev = A.device
    B = _bytes(B)
    K = A.shape[-1]
    M = A.numel() // K if K else int(torch.tensor(A.shape[:-1]).prod().item())
    N = B.shape[0]
    if B.dim() != 2 or B.shape[1] != K:
        raise ValueError(f"B must be [N, K] = [N, {K}], got {tuple(B.shape)}")
    if b_scale.dtype != torch.float32 or b_scale.dim() != 2 or b_scale.shape[0] != N:
        raise ValueError("b_scale must be float32 [N, scale_cols]")
    for t, name in ((A, "A"), (B, "B"), (b_scale, "b_scale")):
        _need(t, name, dev)
    if bias is not None:
        _need(bias, "bias", dev)
        if bias.dtype != A.dtype or bias.numel() != N:
            raise ValueError("bias must be [N] with A's dtype")
    if out is None:
        out = torch.empty(*A.shape[:-1], N, dtype=A.dtype, device=dev)
    _need(out, "out", dev)
    st = lib.fp8w_matmul_ex(_ptr(A), M, K, _ptr(B), N, _ptr(b_scale), b_scale.shape[1], block_size,
                            _ptr(bias), _ptr(out), _dtype_code(A.dtype), _stream(dev), path)
    _check(st, "fp8w_matmul")
    return out


def fp4w_dequant(B: torch.Tensor, weight_scale: torch.Tensor, weight_scale_2: torch.Tensor,
                 block_size: int = 16, dtype: torch.dtype = torch.bfloat16, out: torch.Tensor = None,
                 path: int = PATH_AUTO) -> torch.Tensor:
    lib = load_library()
    dev = B.device
    B, weight_scale = _bytes(B), _bytes(weight_scale)
    N, K = B.shape[0], 2 * B.shape[1]
    for t, name in ((B, "B"), (weight_scale, "weight_scale"), (weight_scale_2, "weight_scale_2")):
        _need(t, name, dev)
    if weight_scale_2.dtype != torch.float32 or weight_scale_2.numel() != 1:
        raise ValueError("weight_scale_2 must be a 1-element float32 tensor")
    if out is None:
        out = torch.empty(N, K, dtype=dtype, device=dev)
    _need(out, "out", dev)
    st = lib.fp4w_dequant_ex(_ptr(B), N, K, _ptr(weight_scale), weight_scale.shape[1], block_size,
                             _ptr(weight_scale_2), _ptr(out), _dtype_code(out.dtype), _stream(dev), path)
    _check(st, "fp4w_dequant")
    return out


def _scalar_f32(t: torch.Tensor, name: str):
    if t.dtype != torch.float32 or t.numel() != 1:
        raise ValueError(f"{name} must be a 1-element float32 tensor")


def fp8w_qdq_activation(A: torch.Tensor, a_scale: torch.Tensor, out: torch.Tensor = None,
                        path: int = PATH_AUTO) -> torch.Tensor:
    """fp8_e4m3(A / a_scale) * a_scale in A's dtype; ``out`` may be ``A``."""
    lib = load_library()
    dev = A.device
    K = A.shape[-1] if A.dim() else 1
    M = A.numel() // K if K else 0
    _need(A, "A", dev)
    _need(a_scale, "a_scale", dev)
    _scalar_f32(a_scale, "a_scale")
    if out is None:
        out = torch.empty_like(A)
    _need(out, "out", dev)
    if out.shape != A.shape or out.dtype != A.dtype:
        raise ValueError("out must have A's shape and dtype")
    st = lib.fp8w_qdq_activation_ex(_ptr(A), M, K, _ptr(a_scale), _ptr(out),
                                    _dtype_code(A.dtype), _stream(dev), path)
    _check(st, "fp8w_qdq_activation")
    return out


def fp8w_matmul_w8a8(A: torch.Tensor, B: torch.Tensor, b_scale: torch.Tensor, a_scale: torch.Tensor,
                     bias: torch.Tensor = None, block_size: int = 128, out: torch.Tensor = None,
                     workspace: torch.Tensor = None) -> torch.Tensor:
    """fp8w_matmul on fp8_e4m3(A / a_scale) * a_scale.  ``workspace`` (A's shape
    and dtype, or ``A`` itself to quantize in place) receives the quantized
    activation; it is allocated here when not given."""
    lib = load_library()
    dev = A.device
    B = _bytes(B)
    K = A.shape[-1]
    M = A.numel() // K if K else int(torch.tensor(A.shape[:-1]).prod().item())
    N = B.shape[0]
    if B.dim() != 2 or B.shape[1] != K:
        raise ValueError(f"B must be [N, K] = [N, {K}], got {tuple(B.shape)}")
    if b_scale.dtype != torch.float32 or b_scale.dim() != 2 or b_scale.shape[0] != N:
        raise ValueError("b_scale must be float32 [N, scale_cols]")
    _scalar_f32(a_scale, "a_scale")
    for t, name in ((A, "A"), (B, "B"), (b_scale, "b_scale"), (a_scale, "a_scale")):
        _need(t, name, dev)
    if bias is not None:
        _need(bias, "bias", dev)
        if bias.dtype != A.dtype or bias.numel() != N:
            raise ValueError("bias must be [N] with A's dtype")
    if workspace is None:
        workspace = torch.empty_like(A)
    _need(workspace, "workspace", dev)
    if workspace.shape != A.shape or workspace.dtype != A.dtype:
        raise ValueError("workspace must have A's shape and dtype")
    if out is None:
        out = torch.empty(*A.shape[:-1], N, dtype=A.dtype, device=dev)
    _need(out, "out", dev)
    st = lib.fp8w_matmul_w8a8(_ptr(A), M, K, _ptr(B), N, _ptr(b_scale), b_scale.shape[1], block_size,
                              _ptr(a_scale), _ptr(bias), _ptr(workspace), _ptr(out),
                              _dtype_code(A.dtype), _stream(dev))
    _check(st, "fp8w_matmul_w8a8")
    return out


def fp8w_dequant(B: torch.Tensor, b_scale: torch.Tensor, block_size: int = 128,
                 dtype: torch.dtype = torch.bfloat16, out: torch.Tensor = None,
                 path: int = PATH_AUTO) -> torch.Tensor:
    lib = load_library()
    dev = B.device
    B = _bytes(B)
    N, K = B.shape
    for t, name in ((B, "B"), (b_scale, "b_scale")):
        _need(t, name, dev)
    if b_scale.dtype != torch.float32 or b_scale.dim() != 2 or b_scale.shape[0] != N:
        raise ValueError("b_scale must be float32 [N, scale_cols]")
    if out is None:
        out = torch.empty(N, K, dtype=dtype, device=dev)
    _need(out, "out", dev)
    st = lib.fp8w_dequant_ex(_ptr(B), N, K, _ptr(b_scale), b_scale.shape[1], block_size, _ptr(out),
                             _dtype_code(out.dtype), _stream(dev), path)
    _check(st, "fp8w_dequant")
    return out


def _rows_k(A: torch.Tensor):
    K = A.shape[-1] if A.dim() else 1
    return (A.numel() // K if K else 0), K


def fp4w_quantize_activation(A: torch.Tensor, codes: torch.Tensor = None, scales: torch.Tensor = None,
                             path: int = PATH_AUTO):
    """NVFP4 activation: (codes uint8 [..., K/2], scales uint8 [..., K/16])."""
    lib = load_library()
    dev = A.device
    M, K = _rows_k(A)
    _need(A, "A", dev)
    if codes is None:
        codes = torch.empty(*A.shape[:-1], K // 2, dtype=torch.uint8, device=dev)
    if scales is None:
        scales = torch.empty(*A.shape[:-1], K // 16, dtype=torch.uint8, device=dev)
    for t, name, n in ((codes, "codes", K // 2), (scales, "scales", K // 16)):
        _need(t, name, dev)
        if t.dtype != torch.uint8 or t.numel() != M * n:
            raise ValueError(f"{name} must be uint8 with {M * n} elements")
    st = lib.fp4w_quantize_activation_ex(_ptr(A), M, K, _ptr(codes), _ptr(scales), _dtype_code(A.dtype),
                                         _stream(dev), path)
    _check(st, "fp4w_quantize_activation")
    return codes, scales


def fp4w_qdq_activation(A: torch.Tensor, out: torch.Tensor = None, path: int = PATH_AUTO) -> torch.Tensor:
    """The NVFP4 activation decoded back to A's dtype; ``out`` may be ``A``."""
    lib = load_library()
    dev = A.device
    M, K = _rows_k(A)
    _need(A, "A", dev)
    if out is None:
        out = torch.empty_like(A)
    _need(out, "out", dev)
    if out.shape != A.shape or out.dtype != A.dtype:
        raise ValueError("out must have A's shape and dtype")
    st = lib.fp4w_qdq_activation_ex(_ptr(A), M, K, _ptr(out), _dtype_code(A.dtype), _stream(dev), path)
    _check(st, "fp4w_qdq_activation")
    return out


def fp4w_matmul_w4a4(A: torch.Tensor, B: torch.Tensor, weight_scale: torch.Tensor,
                     weight_scale_2: torch.Tensor, bias: torch.Tensor = None, block_size: int = 16,
                     out: torch.Tensor = None, workspace: torch.Tensor = None) -> torch.Tensor:
    """W4A4: fp4w_matmul on the NVFP4 activation of A.  ``workspace`` (A's
    shape and dtype, or ``A`` itself) receives that activation; it is
    allocated here when not given."""
    lib = load_library()
    dev = A.device
    B, weight_scale = _bytes(B), _bytes(weight_scale)
    K = A.shape[-1]
    M = A.numel() // K if K else int(torch.tensor(A.shape[:-1]).prod().item())
    N = B.shape[0]
    if B.dim() != 2 or B.shape[1] * 2 != K:
        raise ValueError(f"B must be [N, K/2] = [N, {K // 2}], got {tuple(B.shape)}")
    if weight_scale.dim() != 2 or weight_scale.shape[0] != N:
        raise ValueError("weight_scale must be [N, scale_cols]")
    _scalar_f32(weight_scale_2, "weight_scale_2")
    for t, name in ((A, "A"), (B, "B"), (weight_scale, "weight_scale"), (weight_scale_2, "weight_scale_2")):
        _need(t, name, dev)
    if bias is not None:
        _need(bias, "bias", dev)
        if bias.dtype != A.dtype or bias.numel() != N:
            raise ValueError("bias must be [N] with A's dtype")
    if workspace is None:
        workspace = torch.empty_like(A)
    _need(workspace, "workspace", dev)
    if workspace.shape != A.shape or workspace.dtype != A.dtype:
        raise ValueError("workspace must have A's shape and dtype")
    if out is None:
        out = torch.empty(*A.shape[:-1], N, dtype=A.dtype, device=dev)
    _need(out, "out", dev)
    st = lib.fp4w_matmul_w4a4(_ptr(A), M, K, _ptr(B), N, _ptr(weight_scale), weight_scale.shape[1], block_size,
                              _ptr(weight_scale_2), _ptr(bias), _ptr(workspace), _ptr(out),
                              _dtype_code(A.dtype), _stream(dev))
    _check(st, "fp4w_matmul_w4a4")
    return out


STATIC_SCRATCH_BYTES = 32 * 1024 * 1024  # FP4W_STATIC_SCRATCH_BYTES


def fp4w_matmul_w4a4_noalloc(A: torch.Tensor, B: torch.Tensor, weight_scale: torch.Tensor,
                             weight_scale_2: torch.Tensor, bias: torch.Tensor = None, block_size: int = 16,
                             out: torch.Tensor = None) -> torch.Tensor:
    """fp4w_matmul_w4a4 with the activation staged in the library's own
    device scratch (STATIC_SCRATCH_BYTES per device) instead of a workspace:
    the C call allocates nothing.  Calls that overlap on one device race on
    that scratch.  ``out`` is allocated here when not given."""
    lib = load_library()
    dev = A.device
    B, weight_scale = _bytes(B), _bytes(weight_scale)
    K = A.shape[-1]
    M = A.numel() // K if K else int(torch.tensor(A.shape[:-1]).prod().item())
    N = B.shape[0]
    if B.dim() != 2 or B.shape[1] * 2 != K:
        raise ValueError(f"B must be [N, K/2] = [N, {K // 2}], got {tuple(B.shape)}")
    if weight_scale.dim() != 2 or weight_scale.shape[0] != N:
        raise ValueError("weight_scale must be [N, scale_cols]")
    _scalar_f32(weight_scale_2, "weight_scale_2")
    for t, name in ((A, "A"), (B, "B"), (weight_scale, "weight_scale"), (weight_scale_2, "weight_scale_2")):
        _need(t, name, dev)
    if bias is not None:
        _need(bias, "bias", dev)
        if bias.dtype != A.dtype or bias.numel() != N:
            raise ValueError("bias must be [N] with A's dtype")
    if out is None:
        out = torch.empty(*A.shape[:-1], N, dtype=A.dtype, device=dev)
    _need(out, "out", dev)
    st = lib.fp4w_matmul_w4a4_noalloc(_ptr(A), M, K, _ptr(B), N, _ptr(weight_scale), weight_scale.shape[1],
                                      block_size, _ptr(weight_scale_2), _ptr(bias), _ptr(out),
                                      _dtype_code(A.dtype), _stream(dev))
    _check(st, "fp4w_matmul_w4a4_noalloc")
    return out


# ---------------------------------------------------------------- around a mixture-of-experts block

# A call of these takes the GPU a few microseconds, so its marshalling is kept
# short: the stream's handle comes straight from torch (a torch.cuda.Stream
# object costs 1.8 us, the launch itself about 3), and each tensor is checked by
# one expression; what does not fit is looked at again for the message.

def _call(device: torch.device, f, what: str, *args):
    """Call f(*args, stream) on the device's current stream, with that device current."""
    index = device.index
    if device.type != "cuda":
        raise ValueError(f"{what} runs on the GPU, got tensors on {device}")
    if index == torch._C._cuda_getDevice():
        status = f(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            status = f(*args, torch._C._cuda_getCurrentRawStream(index))
    if status:
        raise FP4WError(status, what)


def _data(t):
    return None if t is None else t.data_ptr()


def _typed(t: torch.Tensor, name: str, dtype: torch.dtype, shape, device: torch.device):
    """t has this type and shape, is contiguous and on the device."""
    if t.dtype is dtype and t.shape == shape and t.is_contiguous() and t.device == device:
        return
    if t.dtype is not dtype or t.shape != shape:
        raise ValueError(f"{name} must be {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    _need(t, name, device)


def fp4w_block_norm(x: torch.Tensor, residual: torch.Tensor = None, pre_weight: torch.Tensor = None,
                    post_weight: torch.Tensor = None, gate: torch.Tensor = None, scale: float = 1.0,
                    eps: float = 1e-6, weight_offset: float = 0.0, residual_out: torch.Tensor = None,
                    out: torch.Tensor = None, write_residual: bool = True):
    """The norms after one block and before the next: (residual_out, out) with

        b = x, or rms_norm(x) * (weight_offset + post_weight)
        residual_out = residual + scale * gate * b
        out = rms_norm(residual_out, unrounded) * (weight_offset + pre_weight)

    ``gate`` is [K] (or [1, K]), or x's shape.  ``out`` is None without
    ``pre_weight``; with ``write_residual=False`` residual_out is neither
    written nor returned.  ``residual_out`` and ``out`` may be x or residual."""
    lib = load_library()
    shape, dtype, dev = x.shape, x.dtype, x.device
    K = shape[-1] if shape else 1
    M = x.numel() // K if K else 0
    code = _dtype_code(dtype)
    _need(x, "x", dev)
    if residual is not None:
        _typed(residual, "residual", dtype, shape, dev)
    if pre_weight is not None:
        _typed(pre_weight, "pre_weight", dtype, (K,), dev)
    if post_weight is not None:
        _typed(post_weight, "post_weight", dtype, (K,), dev)
    gate_rows = 1
    if gate is not None:
        if gate.shape == shape:
            gate_rows = M
        elif gate.shape != (K,) and gate.shape != (1, K):
            raise ValueError(f"gate must be [{K}] or {tuple(shape)}, got {tuple(gate.shape)}")
        _typed(gate, "gate", dtype, gate.shape, dev)
    if not write_residual:
        if residual_out is not None or pre_weight is None:
            raise ValueError("write_residual=False goes with a pre_weight and without a residual_out")
    elif residual_out is None:
        residual_out = torch.empty_like(x)
    else:
        _typed(residual_out, "residual_out", dtype, shape, dev)
    if pre_weight is None:
        if out is not None:
            raise ValueError("out needs a pre_weight")
    elif out is None:
        out = torch.empty_like(x)
    else:
        _typed(out, "out", dtype, shape, dev)
    _call(dev, lib.fp4w_block_norm, "fp4w_block_norm", x.data_ptr(), M, K, _data(post_weight), _data(gate),
          gate_rows, scale, _data(residual), _data(pre_weight), weight_offset, eps, _data(residual_out), _data(out),
          code)
    return residual_out, out


def fp4w_moe_route(logits: torch.Tensor, topk: int, score: str = "softmax", select_bias: torch.Tensor = None,
                   renormalize: bool = True, scale: float = 1.0, ids: torch.Tensor = None,
                   weights: torch.Tensor = None):
    """(ids int32, weights float32), each [..., topk], of router logits
    [..., E] in float16, bfloat16 or float32: the topk experts of each token,
    best first, ties to the lowest index, and scale * their scores
    (renormalised to a sum of scale by default).  ``select_bias`` (float32
    [E]) takes part in the choice only.  Experts with a logit or a logit's score
    plus bias of -inf or NaN are never chosen (those with such a bias alone keep
    their share of a softmax); places left over get id -1 and weight 0."""
    lib = load_library()
    dev = logits.device
    code = F32 if logits.dtype == torch.float32 else _dtype_code(logits.dtype)
    if score not in SCORES:
        raise ValueError(f"score must be one of {sorted(SCORES)}, got {score!r}")
    _need(logits, "logits", dev)
    if logits.dim() < 1:
        raise ValueError("logits must be [..., E]")
    E, lead = logits.shape[-1], logits.shape[:-1]
    M = lead.numel()
    if select_bias is not None:
        _typed(select_bias, "select_bias", torch.float32, (E,), dev)
    if topk < 0:
        raise ValueError("topk must not be negative")
    shape = (*lead, topk)
    if ids is None:
        ids = torch.empty(shape, dtype=torch.int32, device=dev)
    else:
        _typed(ids, "ids", torch.int32, shape, dev)
    if weights is None:
        weights = torch.empty(shape, dtype=torch.float32, device=dev)
    else:
        _typed(weights, "weights", torch.float32, shape, dev)
    _call(dev, lib.fp4w_moe_route, "fp4w_moe_route", logits.data_ptr(), M, E, topk, SCORES[score],
          _data(select_bias), int(renormalize), scale, ids.data_ptr(), weights.data_ptr(), code)
    return ids, weights


def fp4w_moe_workspace(M: int, topk: int, K: int, I: int) -> int:  # noqa: E741
    """Bytes of workspace that fp4w_moe and fp8w_moe need; enough for every smaller call too."""
    n = int(load_library().fp4w_moe_workspace(M, topk, K, I))
    if n < 0:
        raise FP4WError(n, "fp4w_moe_workspace")
    return n


def _moe(fp8, A, ids, weights, w13, s13, g13, w2, s2, g2, block_size, activation, out, workspace, path):
    lib = load_library()
    dev = A.device
    what = "fp8w_moe" if fp8 else "fp4w_moe"
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}, got {activation!r}")
    code = _dtype_code(A.dtype)
    if block_size < 1:
        raise FP4WError(ERR_BLOCK, what)
    u8, f32 = torch.uint8, torch.float32
    if w13.dtype is not u8 or w2.dtype is not u8:
        w13, w2 = _bytes(w13), _bytes(w2)
    shape, chosen, size2 = A.shape, ids.shape, w2.shape
    if not shape or chosen[:-1] != shape[:-1] or not chosen:
        raise ValueError(f"A must be [..., K] and ids [..., topk] with the same leading dimensions, got {tuple(shape)} "
                         f"and {tuple(chosen)}")
    K, topk = shape[-1], chosen[-1]
    M = A.numel() // K if K else shape[:-1].numel()
    if w13.dim() != 3 or len(size2) != 3:
        raise ValueError("w13 must be [E, 2 I, K] and w2 [E, K, I] (FP4: two codes per byte)")
    E, half = size2[0], 1 if fp8 else 2
    I = size2[2] * half  # noqa: E741
    if K % half or w13.shape != (E, 2 * I, K // half) or size2[1] != K:
        raise ValueError(f"w13 {tuple(w13.shape)} and w2 {tuple(size2)} do not fit A's K = {K}")
    _need(A, "A", dev)
    _typed(ids, "ids", torch.int32, chosen, dev)
    _typed(weights, "weights", f32, chosen, dev)
    _need(w13, "w13", dev)
    _need(w2, "w2", dev)
    scale_type = f32 if fp8 else u8
    if not fp8:
        if s13.dtype is not u8 or s2.dtype is not u8:
            s13, s2 = _bytes(s13), _bytes(s2)
        _typed(g13, "w13_scale_2", f32, (E,), dev)
        _typed(g2, "w2_scale_2", f32, (E,), dev)
    _typed(s13, "w13_scale", scale_type, (E, 2 * I, -(-K // block_size)), dev)
    _typed(s2, "w2_scale", scale_type, (E, K, -(-I // block_size)), dev)
    if workspace is None:
        held = lib.fp4w_moe_workspace(M, topk, K, I)
        if held < 0:
            raise FP4WError(held, what)
        workspace = torch.empty(held, dtype=u8, device=dev)
    else:
        _need(workspace, "workspace", dev)
        held = workspace.numel() * workspace.element_size()
    if out is None:
        out = torch.empty_like(A)
    else:
        _typed(out, "out", A.dtype, A.shape, dev)
    tail = (E, I, block_size, ACTIVATIONS[activation], workspace.data_ptr(), held, out.data_ptr(), code)
    if fp8:
        args = (A.data_ptr(), M, K, ids.data_ptr(), weights.data_ptr(), topk, w13.data_ptr(), s13.data_ptr(),
                w2.data_ptr(), s2.data_ptr(), *tail)
    else:
        args = (A.data_ptr(), M, K, ids.data_ptr(), weights.data_ptr(), topk, w13.data_ptr(), s13.data_ptr(),
                g13.data_ptr(), w2.data_ptr(), s2.data_ptr(), g2.data_ptr(), *tail)
    if path == PATH_AUTO:
        _call(dev, lib.fp8w_moe if fp8 else lib.fp4w_moe, what, *args)
    else:
        f = lib.fp8w_moe_ex if fp8 else lib.fp4w_moe_ex
        _call(dev, lambda *a: f(*a, path), what, *args)
    return out


def fp4w_moe(A: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, w13: torch.Tensor, w13_scale: torch.Tensor,
             w13_scale_2: torch.Tensor, w2: torch.Tensor, w2_scale: torch.Tensor, w2_scale_2: torch.Tensor,
             block_size: int = 16, activation: str = "silu", out: torch.Tensor = None,
             workspace: torch.Tensor = None, path: int = PATH_AUTO) -> torch.Tensor:
    """A whole mixture-of-experts layer on FP4 weights, made for a few tokens and
    taking any number: for each token the sum over its choices j, e = ids[..., j], of

        weights[..., j] * ((act(A w13[e, :I]^T) * (A w13[e, I:]^T)) w2[e]^T)

    ``ids`` int32 and ``weights`` float32 are [..., topk] with A's leading
    dimensions (fp4w_moe_route's outputs); an id outside [0, E) contributes
    nothing.  ``w13`` [E, 2 I, K/2], ``w2`` [E, K, I/2] packed E2M1 with E4M3
    scales per block and one float32 scale per expert.  ``workspace`` holds
    ``fp4w_moe_workspace(M, topk, K, I)`` bytes; it is allocated here when not
    given.  Calls that may run at once need one each."""
    return _moe(False, A, ids, weights, w13, w13_scale, w13_scale_2, w2, w2_scale, w2_scale_2, block_size, activation,
                out, workspace, path)


def fp8w_moe(A: torch.Tensor, ids: torch.Tensor, weights: torch.Tensor, w13: torch.Tensor, w13_scale: torch.Tensor,
             w2: torch.Tensor, w2_scale: torch.Tensor, block_size: int = 128, activation: str = "silu",
             out: torch.Tensor = None, workspace: torch.Tensor = None, path: int = PATH_AUTO) -> torch.Tensor:
    """fp4w_moe on FP8 weights: ``w13`` E4M3 [E, 2 I, K], ``w2`` [E, K, I],
    float32 scales per ``block_size`` values of a row."""
    return _moe(True, A, ids, weights, w13, w13_scale, None, w2, w2_scale, None, block_size, activation, out,
                workspace, path)


# ---------------------------------------------------------------- between the projections of an attention block

class KVCache(NamedTuple):
    """A paged cache of keys and values: E4M3 codes ``k`` [pages, heads,
    page_size, D] and ``v`` [pages, heads, D, page_size] (uint8 or
    float8_e4m3fn), and a power of two for each page and head, ``k_scale`` and
    ``v_scale`` [pages, heads] (uint8 or float8_e8m0fnu: 2^(byte - 127))."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor


def fp8w_kv_cache(num_pages: int, heads: int, page_size: int, head_size: int, device="cuda") -> KVCache:
    """An empty cache (0.5 KB a token for 2 heads of 128): pages are filled by fp8w_kv_append."""
    codes = torch.zeros(2, num_pages * heads * page_size * head_size, dtype=torch.uint8, device=device)
    scale = torch.full((2, num_pages, heads), 127, dtype=torch.uint8, device=device)
    return KVCache(codes[0].view(num_pages, heads, page_size, head_size),
                   codes[1].view(num_pages, heads, head_size, page_size), scale[0], scale[1])


_CODES = (torch.uint8, torch.float8_e4m3fn)
_POWERS = (torch.uint8, torch.float8_e8m0fnu)


def _cache(cache: KVCache, heads: int, D: int, device: torch.device):
    """(pages, page_size) of a cache that fits; raises otherwise."""
    k, v, ks, vs = cache
    shape = k.shape
    if len(shape) != 4 or shape[1] != heads or shape[3] != D or v.shape != (shape[0], heads, D, shape[2]):
        raise ValueError(f"the cache must hold k [pages, {heads}, page_size, {D}] and v [pages, {heads}, {D}, page_size], "
                         f"got {tuple(shape)} and {tuple(v.shape)}")
    if ks.shape != shape[:2] or vs.shape != shape[:2]:
        raise ValueError(f"the cache's scales must be [{shape[0]}, {heads}], got {tuple(ks.shape)} and {tuple(vs.shape)}")
    if k.dtype not in _CODES or v.dtype not in _CODES:
        raise TypeError(f"the cache's k and v must be one of {_CODES}, got {k.dtype} and {v.dtype}")
    if ks.dtype not in _POWERS or vs.dtype not in _POWERS:
        raise TypeError(f"the cache's scales must be one of {_POWERS}, got {ks.dtype} and {vs.dtype}")
    if not (k.is_contiguous() and v.is_contiguous() and ks.is_contiguous() and vs.is_contiguous() and k.device == device
            and v.device == device and ks.device == device and vs.device == device):
        for t, name in ((k, "k"), (v, "v"), (ks, "k_scale"), (vs, "v_scale")):
            _need(t, f"the cache's {name}", device)
    return shape[0], shape[2]


def _heads(t: torch.Tensor, name: str, M: int, D: int, dtype: torch.dtype, device: torch.device):
    """(heads, token stride) of t [M, heads, D], whose tokens may be apart."""
    shape = t.shape
    if len(shape) != 3 or shape[0] != M or shape[2] != D or t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype} [{M}, heads, {D}], got {t.dtype} {tuple(shape)}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    H = shape[1]
    if t.is_contiguous():
        return H, H * D
    stride = t.stride()
    if (stride[2] != 1 and D > 1) or (stride[1] != D and H > 1):
        raise ValueError(f"{name}'s heads must lie side by side, got strides {stride}")
    return H, (stride[0] if M > 1 else H * D)


def _heads_out(out, name: str, like: torch.Tensor, M: int, H: int, D: int, dtype: torch.dtype, device: torch.device):
    """(out, token stride): what is given, or a new tensor of like's shape (whose heads lie side by side)."""
    if out is None:
        return torch.empty_like(like, memory_format=torch.contiguous_format), H * D
    n, stride = _heads(out, name, M, D, dtype, device)
    if n != H:
        raise ValueError(f"{name} must have {H} heads, got {n}")
    return out, stride


def _rope_args(dtype, device, M, D, q_weight, k_weight, weight_offset, eps, cos, sin, interleaved, positions):
    if q_weight is not None:
        _typed(q_weight, "q_weight", dtype, (D,), device)
    if k_weight is not None:
        _typed(k_weight, "k_weight", dtype, (D,), device)
    rows = dims = 0
    if cos is not None or sin is not None:
        shape = None if cos is None else cos.shape
        if shape is None or sin is None or len(shape) != 2 or not shape[0] or not shape[1]:  # (no pointer to an empty table)
            raise ValueError("cos and sin go together, each [positions, rotated values / 2] and not empty")
        rows, dims = shape[0], 2 * shape[1]
        if dims > D:
            raise ValueError(f"cos has {dims // 2} angles, heads of {D} have at most {D // 2}")
        _typed(cos, "cos", torch.float32, shape, device)
        _typed(sin, "sin", torch.float32, shape, device)
    if positions is not None:
        _typed(positions, "positions", torch.int32, (M,), device)
    return (_data(q_weight), _data(k_weight), weight_offset, eps, _data(cos), _data(sin), rows, dims, int(interleaved),
            _data(positions))


def fp4w_qk_norm_rope(q: torch.Tensor, k: torch.Tensor = None, q_weight: torch.Tensor = None,
                      k_weight: torch.Tensor = None, cos: torch.Tensor = None, sin: torch.Tensor = None,
                      positions: torch.Tensor = None, interleaved: bool = False, weight_offset: float = 0.0,
                      eps: float = 1e-6, q_out: torch.Tensor = None, k_out: torch.Tensor = None):
    """(q_out, k_out): the heads of q [M, Hq, D] and k [M, Hk, D] (or None)
    normed, x * rsqrt(mean(x^2) + eps) * (weight_offset + weight), where their
    weight is given, and rotated by the angles of ``cos`` and ``sin`` (float32
    [positions, R / 2]) at ``positions`` (int32 [M]; None: 0, 1, ...): pairs
    (i, i + R / 2) of the first R values, or (2 i, 2 i + 1) if ``interleaved``.
    Tokens may be apart (views into a projection's output), and ``q_out`` and
    ``k_out`` may be q and k."""
    lib = load_library()
    if q.dim() != 3:
        raise ValueError(f"q must be [M, heads, D], got {tuple(q.shape)}")
    dtype, dev, (M, _, D) = q.dtype, q.device, q.shape
    code = _dtype_code(dtype)
    Hq, q_stride = _heads(q, "q", M, D, dtype, dev)
    q_out, qo_stride = _heads_out(q_out, "q_out", q, M, Hq, D, dtype, dev)
    Hk = k_stride = ko_stride = 0
    if k is not None:
        Hk, k_stride = _heads(k, "k", M, D, dtype, dev)
        k_out, ko_stride = _heads_out(k_out, "k_out", k, M, Hk, D, dtype, dev)
    elif k_out is not None or k_weight is not None:
        raise ValueError("k_out and k_weight need a k")
    rope = _rope_args(dtype, dev, M, D, q_weight, k_weight, weight_offset, eps, cos, sin, interleaved, positions)
    _call(dev, lib.fp4w_qk_norm_rope, "fp4w_qk_norm_rope", q.data_ptr(), q_stride, Hq, _data(k), k_stride, Hk, M, D, *rope,
          q_out.data_ptr(), qo_stride, _data(k_out), ko_stride, code)
    return q_out, k_out


def _sequences(page_table, seq_lens, starts, M, device):
    """(B, max_pages) of a batch that fits; raises otherwise."""
    if page_table.dim() != 2:
        raise ValueError(f"page_table must be int32 [B, pages of a sequence], got {tuple(page_table.shape)}")
    B, pages = page_table.shape
    _typed(page_table, "page_table", torch.int32, (B, pages), device)
    _typed(seq_lens, "seq_lens", torch.int32, (B,), device)
    if starts is not None:
        _typed(starts, "starts", torch.int32, (B + 1,), device)
    elif B != M:
        raise ValueError(f"without starts there is one new token for each sequence, got {M} for {B}")
    return B, pages


def fp8w_kv_append(k: torch.Tensor, v: torch.Tensor, cache: KVCache, page_table: torch.Tensor, seq_lens: torch.Tensor,
                   starts: torch.Tensor = None, q: torch.Tensor = None, q_weight: torch.Tensor = None,
                   k_weight: torch.Tensor = None, cos: torch.Tensor = None, sin: torch.Tensor = None,
                   positions: torch.Tensor = None, interleaved: bool = False, weight_offset: float = 0.0,
                   eps: float = 1e-6, q_out: torch.Tensor = None):
    """Writes new keys and values [M, Hk, D] into the pages of their sequences,
    the keys normed and rotated on the way as by fp4w_qk_norm_rope; returns
    ``q`` [M, Hq, D] normed and rotated (``q_out``), or None without a q.

    Sequence b's new tokens are rows starts[b] .. starts[b + 1] - 1 (int32
    [B + 1]; None: one row each); ``seq_lens`` (int32 [B]) counts its tokens with
    them, and ``page_table`` (int32 [B, pages]) names its pages.  The rotation
    takes ``positions`` (int32 [M]), or a token's place in its sequence.  No page
    may be named twice in one call (full pages that are only read later may)."""
    lib = load_library()
    if k.dim() != 3:
        raise ValueError(f"k must be [M, heads, D], got {tuple(k.shape)}")
    dtype, dev, (M, _, D) = k.dtype, k.device, k.shape
    code = _dtype_code(dtype)
    Hk, k_stride = _heads(k, "k", M, D, dtype, dev)
    nv, v_stride = _heads(v, "v", M, D, dtype, dev)
    if nv != Hk:
        raise ValueError(f"v must have k's {Hk} heads, got {nv}")
    pages, page = _cache(cache, Hk, D, dev)
    B, max_pages = _sequences(page_table, seq_lens, starts, M, dev)
    Hq = q_stride = qo_stride = 0
    if q is not None:
        Hq, q_stride = _heads(q, "q", M, D, dtype, dev)
        q_out, qo_stride = _heads_out(q_out, "q_out", q, M, Hq, D, dtype, dev)
    elif q_out is not None or q_weight is not None:
        raise ValueError("q_out and q_weight need a q")
    rope = _rope_args(dtype, dev, M, D, q_weight, k_weight, weight_offset, eps, cos, sin, interleaved, positions)
    _call(dev, lib.fp8w_kv_append, "fp8w_kv_append", k.data_ptr(), k_stride, v.data_ptr(), v_stride, M, Hk, D, _data(q),
          q_stride, Hq, *rope, _data(q_out), qo_stride, _data(starts), B, seq_lens.data_ptr(), page_table.data_ptr(),
          max_pages, cache.k.data_ptr(), cache.k_scale.data_ptr(), cache.v.data_ptr(), cache.v_scale.data_ptr(), pages,
          page, code)
    return q_out


@functools.lru_cache(maxsize=256)
def _attention_workspace(*sizes):
    return int(load_library().fp8w_attention_workspace(*sizes))


def fp8w_attention_workspace(M: int, Hq: int, Hk: int, D: int, B: int, max_new: int) -> int:
    """Bytes of workspace that fp8w_attention needs, however long the sequences are; enough for every smaller call too."""
    n = _attention_workspace(M, Hq, Hk, D, B, max_new)
    if n < 0:
        raise FP4WError(n, "fp8w_attention_workspace")
    return n


def fp8w_attention(q: torch.Tensor, cache: KVCache, page_table: torch.Tensor, seq_lens: torch.Tensor,
                   starts: torch.Tensor = None, max_new: int = None, scale: float = None, causal: bool = True,
                   window: int = 0, out: torch.Tensor = None, lse: torch.Tensor = None, workspace: torch.Tensor = None,
                   path: int = PATH_AUTO) -> torch.Tensor:
    """Attention of the new tokens' q [M, Hq, D] over the cache, which holds
    them already (fp8w_kv_append); [M, Hq, D].

    Rows and sequences as in fp8w_kv_append.  A token attends the tokens of its
    sequence up to its own position (all that are held if not ``causal``), of
    those the last ``window`` if it is not 0; one that attends none gets zeros.
    ``scale`` is D^-0.5 if None.  ``max_new`` (None: M, or 1 without ``starts``)
    is at least every sequence's number of new tokens, and chooses the kernel:
    rows behind it are left as they were.  ``lse`` (float32 [M, Hq]), where given,
    gets the logarithm of each row's sum of exponentials.  ``workspace`` holds
    ``fp8w_attention_workspace(M, Hq, Hk, D, B, max_new)`` bytes; it is allocated
    here when not given.  Calls that may run at once need one each."""
    lib = load_library()
    if q.dim() != 3:
        raise ValueError(f"q must be [M, heads, D], got {tuple(q.shape)}")
    dtype, dev, (M, _, D) = q.dtype, q.device, q.shape
    code = _dtype_code(dtype)
    Hq, q_stride = _heads(q, "q", M, D, dtype, dev)
    Hk = cache.k.shape[1] if cache.k.dim() == 4 else 0
    pages, page = _cache(cache, Hk, D, dev)
    B, max_pages = _sequences(page_table, seq_lens, starts, M, dev)
    if max_new is None or max_new > M:
        max_new = M
    if starts is None:
        max_new = 1
    if window < 0 or max_new < 0:
        raise ValueError("window and max_new must not be negative")
    if out is None:
        out = torch.empty_like(q, memory_format=torch.contiguous_format)
    else:
        _typed(out, "out", dtype, (M, Hq, D), dev)
    if lse is not None:
        _typed(lse, "lse", torch.float32, (M, Hq), dev)
    if workspace is None:
        held = _attention_workspace(M, Hq, Hk, D, B, max_new)
        if held < 0:
            raise FP4WError(held, "fp8w_attention")
        if held:
            workspace = torch.empty(held, dtype=torch.uint8, device=dev)
    else:
        _need(workspace, "workspace", dev)
        held = workspace.numel() * workspace.element_size()
    args = (q.data_ptr(), q_stride, M, Hq, Hk, D, _data(starts), B, seq_lens.data_ptr(), page_table.data_ptr(), max_pages,
            max_new, cache.k.data_ptr(), cache.k_scale.data_ptr(), cache.v.data_ptr(), cache.v_scale.data_ptr(), pages, page,
            D ** -0.5 if scale is None and D else scale or 0.0, int(causal), window, _data(workspace), held, out.data_ptr(),
            _data(lse), code)
    if path == PATH_AUTO:
        _call(dev, lib.fp8w_attention, "fp8w_attention", *args)
    else:
        _call(dev, lambda *a: lib.fp8w_attention_ex(*a, path), "fp8w_attention", *args)
    return out
