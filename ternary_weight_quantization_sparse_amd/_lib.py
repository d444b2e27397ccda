"""ctypes loader for libsherry.so (the C ABI declared in include/sherry.h).

There is no fallback: if the library is missing this raises, so nothing can
silently run a different implementation.
"""

from __future__ import annotations

import ctypes
import os

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG_DIR, "libsherry.so")

# status codes (sherry_status)
OK = 0
ERR_NULL, ERR_SHAPE, ERR_GROUP, ERR_GRANULARITY, ERR_DTYPE, ERR_UNSUPPORTED = 1, 2, 3, 4, 5, 6
ERR_ALIGN, ERR_WORKSPACE, ERR_BATCH, ERR_HIP = 7, 8, 9, 10

# enums
PER_TENSOR, PER_CHANNEL, PER_GROUP = 0, 1, 2
GRANULARITY = {"per_tensor": PER_TENSOR, "per_channel": PER_CHANNEL, "per_group": PER_GROUP}
CMP_2BIT, CMP_TL2 = 0, 1
F32, BF16, I8 = 0, 1, 2
OP_QUANTIZE_PACK, OP_UNPACK, OP_GEMV, OP_GEMM, OP_FAKE_QUANT, OP_ARENAS_GEMM = 0, 1, 2, 3, 4, 5
ERR_ARG = 11
ACTIVATIONS = {"none": 0, "relu": 1, "relu2": 2, "silu": 3, "gelu": 4, "gelu_tanh": 5}
SCORING = {"softmax": 0, "sigmoid": 1}
GATE_NONE, GATE_TOKEN, GATE_CHANNEL, GATE_ROWS = 0, 1, 2, 3
QUANTIZE_SCRATCH_BYTES = 8 << 20   # SHERRY_QUANTIZE_SCRATCH_BYTES

# every symbol include/sherry.h declares
SYMBOLS = (
    "sherry_abi_version", "sherry_status_string", "sherry_packed_bytes", "sherry_num_scales",
    "sherry_workspace_bytes", "sherry_quantize_pack", "sherry_unpack", "sherry_gemv", "sherry_gemm",
    "sherry_fake_quant", "sherry_arenas_gemm", "sherry_compare_bytes", "sherry_compare_repack",
    "sherry_compare_gemv", "sherry_arenas_lambda", "sherry_quantize_pack_noalloc",
)

# every symbol include/sherry_ops.h declares
OPS_SYMBOLS = (
    "sherry_block_norm", "sherry_block_norm_backward_bytes", "sherry_block_norm_backward",
    "sherry_adapter_workspace_bytes", "sherry_adapter_gemv", "sherry_adapter_gemm",
    "sherry_muon_workspace_bytes", "sherry_orthogonalize", "sherry_muon_step",
    "sherry_distill_workspace_bytes", "sherry_distill_loss", "sherry_distill_loss_backward",
    "sherry_linear_gemv", "sherry_linear_gemm", "sherry_moe_workspace_bytes", "sherry_moe_decode",
)

_i32, _i64, _sz, _vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_void_p

_f32 = ctypes.c_float

_SIGNATURES = {
    "sherry_abi_version": ([], _i32),
    "sherry_status_string": ([_i32], ctypes.c_char_p),
    "sherry_packed_bytes": ([_i64, _i64], _sz),
    "sherry_num_scales": ([_i64, _i64, _i32, _i32], _i64),
    "sherry_workspace_bytes": ([_i32, _i64, _i64, _i32, _i32, _i64, _i32], _sz),
    "sherry_quantize_pack": ([_i64, _i64, _i32, _i32, _vp, _i32, _vp, _vp, _vp, _sz, _vp], _i32),
    "sherry_quantize_pack_noalloc": ([_i64, _i64, _i32, _i32, _vp, _i32, _vp, _vp, _vp], _i32),
    "sherry_unpack": ([_i64, _i64, _i32, _i32, _vp, _vp, _vp, _i32, _vp], _i32),
    "sherry_gemv": ([_i64, _i64, _i32, _i32, _vp, _vp, _vp, _i32, _vp, _i32, _i32, _i64, _i64, _i64,
                     _vp, _sz, _vp], _i32),
    "sherry_gemm": ([_i64, _i64, _i32, _i32, _vp, _vp, _vp, _i64, _vp, _vp, _sz, _vp], _i32),
    "sherry_fake_quant": ([_i64, _i64, _i32, _i32, _vp, _i32, _vp, _i32, _vp, _vp, _sz, _vp], _i32),
    "sherry_arenas_gemm": ([_i64, _i64, _i32, _i32, _vp, _vp, _vp, ctypes.c_float, _vp, _i64, _vp, _vp, _sz, _vp],
                           _i32),
    "sherry_arenas_lambda": ([_i64, _i64, ctypes.c_double], ctypes.c_double),
    "sherry_compare_bytes": ([_i32, _i64, _i64], _sz),
    "sherry_compare_repack": ([_i32, _i64, _i64, _vp, _vp, _vp], _i32),
    "sherry_compare_gemv": ([_i32, _i64, _i64, _vp, _vp, _vp, _vp, _i32, _i64, _i64, _i64, _vp], _i32),
    "sherry_block_norm": ([_i64, _i64, _vp, _vp, _i32, _vp, _vp, _i32, _vp, _i32, _i64, _f32, _f32, _vp, _vp, _vp],
                          _i32),
    "sherry_block_norm_backward_bytes": ([_i64, _i64, _i32, _i64], _sz),
    "sherry_block_norm_backward": ([_i64, _i64, _vp, _vp, _vp, _vp, _i32, _vp, _vp, _i32, _vp, _i32, _i64, _f32, _f32,
                                    _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp], _i32),
    "sherry_adapter_workspace_bytes": ([_i64, _i64, _i32, _i32, _i64, _i32, _i32], _sz),
    "sherry_adapter_gemv": ([_i64, _i64, _i32, _i32, _vp, _vp, _vp, _i32, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _i32,
                             _i32, _vp, _sz, _vp], _i32),
    "sherry_adapter_gemm": ([_i64, _i64, _i32, _i32, _vp, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32,
                             _vp, _sz, _vp], _i32),
    "sherry_muon_workspace_bytes": ([_i32, _i64, _i64], _sz),
    "sherry_orthogonalize": ([_i32, _i64, _i64, _vp, _i32, _vp, _i32, _f32, _f32, _f32, _f32, _vp, _sz, _vp], _i32),
    "sherry_muon_step": ([_i32, _i64, _i64, _vp, _vp, _vp, _i32, _vp, _vp, _f32, _f32, _i32, _f32, _f32, _i32, _f32,
                          _f32, _f32, _f32, _vp, _sz, _vp], _i32),
    "sherry_distill_workspace_bytes": ([_i64, _i64, _i32], _sz),
    "sherry_distill_loss": ([_i64, _i64, _vp, _i64, _i32, _vp, _i32, _vp, _i32, _i32, _f32, _vp, _vp, _i32, _f32, _vp,
                             _vp, _vp, _sz, _vp], _i32),
    "sherry_distill_loss_backward": ([_i64, _i64, _vp, _vp, _i64, _i32, _vp, _i32, _i32, _f32, _vp, _i32, _f32, _vp,
                                      _vp, _i64, _vp], _i32),
    "sherry_linear_gemv": ([_i64, _i64, _i32, _i32, _vp, _vp, _vp, _i32, _vp, _i32, _vp, _i32, _i32, _i32, _vp, _f32,
                            _vp], _i32),
    "sherry_linear_gemm": ([_i64, _i64, _i32, _i32, _vp, _vp, _vp, _i64, _vp, _vp, _i32, _i32, _i32, _vp, _f32, _vp,
                            _sz, _vp], _i32),
    "sherry_moe_workspace_bytes": ([_i32, _i64, _i64, _i32, _i32, _i32], _sz),
    "sherry_moe_decode": ([_i32, _i64, _i64, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _i32, _vp, _f32, _i32, _i32, _vp,
                           _vp, _i32, _i32, _vp, _vp, _i32, _i32, _vp, _vp, _i32, _vp, _sz, _vp], _i32),
}

_lib = None


class SherryError(RuntimeError):
    """A non-argument failure reported by libsherry (the HIP runtime)."""


def load() -> ctypes.CDLL:
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with "
            "`python -m ternary_weight_quantization_sparse_amd.build` (needs hipcc)")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (args, res) in _SIGNATURES.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _lib = lib
    return lib


def status_string(code: int) -> str:
    return load().sherry_status_string(int(code)).decode()


def check(code: int) -> None:
    """Raise for a non-zero status: ValueError for argument errors (the
    conditions the pages' quantizer rejects and this build's limits),
    SherryError for runtime failures."""
    if code == OK:
        return
    msg = status_string(code)
    if code == ERR_HIP:
        raise SherryError(msg)
    if code == ERR_UNSUPPORTED:
        raise NotImplementedError(msg)
    raise ValueError(msg)
