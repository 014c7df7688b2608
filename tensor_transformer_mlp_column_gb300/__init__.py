"""tensor_transformer_mlp_column_gb300 — Python binding of libtpmlp (include/tpmlp.h).

The tensor-parallel MLP  Y = GeLU(X A) B  with A split by columns and B by
rows into n shards, each shard's partial computed on its own and the partials
summed (scratchllm.com "Tensor-Parallel MLP (Megatron)"), on one GB300.

This module only marshals arguments: torch tensors supply device memory and
the current CUDA stream, and every step runs in the library's CUDA kernels.
There is no CPU fallback; if libtpmlp.so is missing the first call raises.
Function names are those of the C ABI.
"""

from __future__ import annotations

import ctypes
import functools
import os
from array import array
from typing import Optional, Sequence

import torch

# TPMLP_DEBUG=1 loads the debug build (device-side index checks; build it with
# build_lib.build(debug=True)) instead of the normal one.
DEBUG = os.environ.get("TPMLP_DEBUG", "") not in ("", "0")
LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libtpmlp_debug.so" if DEBUG else "libtpmlp.so")

TPMLP_F32, TPMLP_BF16 = 0, 1
TPMLP_FAITHFUL, TPMLP_FUSED = 0, 1
TPMLP_MAX_SHARDS = 16

STATUS_NAMES = {
    0: "TPMLP_OK",
    -1: "TPMLP_ERR_ARG",
    -2: "TPMLP_ERR_DIVISIBILITY",
    -3: "TPMLP_ERR_ALIGN",
    -4: "TPMLP_ERR_SHAPE",
    -5: "TPMLP_ERR_CUDA",
    -6: "TPMLP_ERR_TIMEOUT",
    -7: "TPMLP_ERR_WORKSPACE",
    -8: "TPMLP_ERR_UNSUPPORTED",
    -9: "TPMLP_ERR_DEVICE",
    -10: "TPMLP_ERR_BOUNDS",
}
globals().update({v: k for k, v in STATUS_NAMES.items()})

# Every entry point of include/tpmlp.h with its ctypes signature.
_P, _I, _I64, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
SIGNATURES = {
    "tpmlp_version": (_I, []),
    "tpmlp_last_error": (ctypes.c_char_p, []),
    "tpmlp_check_status": (_I, [_P]),
    "tpmlp_gelu": (_I, [_P, _P, _I64, _I, _P]),
    "tpmlp_shard": (_I, [_P, _P, _I64, _I64, _I, _I, _P, ctypes.POINTER(_P)]),
    "tpmlp_shard_info": (_I, [_P, ctypes.POINTER(_I64), ctypes.POINTER(_I64), ctypes.POINTER(_I), ctypes.POINTER(_I)]),
    "tpmlp_shard_get": (_I, [_P, _I, ctypes.POINTER(_P), ctypes.POINTER(_P)]),
    "tpmlp_shard_get_transposed": (_I, [_P, _I, ctypes.POINTER(_P), ctypes.POINTER(_P)]),
    "tpmlp_shards_free": (None, [_P]),
    "tpmlp_workspace_bytes": (_SZ, [_I64, _P, _I, _I]),
    "tpmlp_forward": (_I, [_P, _I64, _P, _P, _I, _P, _SZ, _P]),
    "tpmlp_hidden": (_I, [_P, _I64, _P, _P, _P]),
    "tpmlp_partials": (_I, [_P, _I64, _P, _P, _P]),
    "tpmlp_allreduce": (_I, [_P, _I, _I64, _P, _P]),
    "tpmlp_fused_sum": (_I, [_P, _I64, _P, _P, _P]),
    "tpmlp_backward": (_I, [_P, _P, _I64, _P, _P, ctypes.POINTER(_P), ctypes.POINTER(_P), _I, _P, _SZ, _P]),
    "tpmlp_selftest_wait_timeout": (_I, [_I, _P]),
    "tpmlp_forward_noalloc": (_I, [_P, _I64, _P, _P, _I, _P]),
    "tpmlp_selftest_gemm_withheld_fill": (_I, [_P, _I64, _P, _P, _I, _I, _P]),
    "tpmlp_forward_save": (_I, [_P, _I64, _P, _P, _P, _I, _P, _SZ, _P]),
    "tpmlp_backward_saved": (_I, [_P, _P, _P, _I64, _P, _P, ctypes.POINTER(_P), ctypes.POINTER(_P), _I, _P, _SZ, _P]),
    "tpmlp_layer_norm": (_I, [_P, _I64, _I64, _I, ctypes.c_float, _P, _P]),
    "tpmlp_block_workspace_bytes": (_SZ, [_I64, _P, _I, _I]),
    "tpmlp_block_forward": (_I, [_P, _I64, _P, ctypes.c_float, _P, _P, _I, _P, _SZ, _P]),
    "tpmlp_block_backward": (_I, [_P, _P, _I64, _P, ctypes.c_float, _P, ctypes.POINTER(_P), ctypes.POINTER(_P), _I, _P,
                                  _SZ, _P]),
    "tpmlp_all_gather": (_I, [ctypes.POINTER(_P), _I, _I64, _P, _P]),
    "tpmlp_attn_shard": (_I, [_P, _P, _P, _P, _I64, _I, _I, _I, _P, ctypes.POINTER(_P)]),
    "tpmlp_attn_shard_get": (_I, [_P, _I, ctypes.POINTER(_P), ctypes.POINTER(_P)]),
    "tpmlp_attn_shards_free": (None, [_P]),
    "tpmlp_attn_workspace_bytes": (_SZ, [_I64, _I64, _P, _I]),
    "tpmlp_attn_heads": (_I, [_P, _I64, _I64, _P, _P, _P, _SZ, _P]),
    "tpmlp_attn_forward": (_I, [_P, _I64, _I64, _P, _P, _I, _P, _SZ, _P]),
    "tpmlp_reduce_scatter": (_I, [_P, _I, _I64, ctypes.POINTER(_P), _P]),
    "tpmlp_sp_workspace_bytes": (_SZ, [_I64, _P, _I, _I]),
    "tpmlp_forward_sp": (_I, [ctypes.POINTER(_P), _I64, _P, ctypes.POINTER(_P), _I, _P, _SZ, _P]),
    "tpmlp_backward_sp": (_I, [ctypes.POINTER(_P), ctypes.POINTER(_P), _I64, _P, ctypes.POINTER(_P),
                               ctypes.POINTER(_P), ctypes.POINTER(_P), _I, _P, _SZ, _P]),
    "tpmlp_xent_workspace_bytes": (_SZ, [_I64, _I64, _I64, _I, _I]),
    "tpmlp_xent_forward": (_I, [_P, _P, _P, _I64, _I64, _I64, _I, _P, _P, _P, _SZ, _P]),
    "tpmlp_xent_backward": (_I, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _I, _P, _P, _P, _SZ, _P]),
    "tpmlp_xent_backward_saved": (_I, [_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I, _P, _P, _P, _SZ, _P]),
    "tpmlp_selftest_xent_stage_timeout": (_I, [_P, _P, _P, _I64, _I64, _I64, _I, _P, _P, _I, _I, _P, _SZ, _P]),
    "tpmlp_embed_forward": (_I, [_P, _P, _I64, _I64, _I64, _I, ctypes.c_float, _P, _P]),
    "tpmlp_embed_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "tpmlp_embed_backward": (_I, [_P, _I, _P, _I64, _I64, _I64, ctypes.c_float, _P, _I, _I, _P, _SZ, _P]),
    "tpmlp_grad_workspace_bytes": (_SZ, [_I]),
    "tpmlp_grad_norm": (_I, [_P, _P, _P, _I, _P, _P, _SZ, _P]),
    "tpmlp_grad_clip": (_I, [_P, _P, _P, _I, ctypes.c_float, _P, _P, _P, _SZ, _P]),
    "tpmlp_attn_core_forward": (_I, [_P] * 5 + [_I64] * 3 + [_I] * 3 + [ctypes.c_float, _I, _I, _P, _P, _P]),
    "tpmlp_attn_core_workspace_bytes": (_SZ, [_I64] * 3 + [_I] * 4),
    "tpmlp_attn_core_backward": (_I, [_P] * 8 + [_I64] * 3 + [_I] * 3 + [ctypes.c_float, _I, _I] + [_P] * 4 + [_SZ, _P]),
    "tpmlp_selftest_attn_core_timeout": (_I, [_P] * 6 + [_I64, _I, _I] + [_P] * 4 + [_SZ, _I, _I, _I, _P]),
    "tpmlp_qk_rope_forward": (_I, [_P] * 5 + [ctypes.c_float] + [_P] * 3 + [_I64] + [_I] * 7 + [_P] * 3),
    "tpmlp_qk_rope_workspace_bytes": (_SZ, [_I64, _I, _I, _I]),
    "tpmlp_qk_rope_backward": (_I, [_P] * 7 + [ctypes.c_float] + [_P] * 3 + [_I64] + [_I] * 7 + [_P] * 5 + [_SZ, _P]),
    "tpmlp_trace_read": (_I, [ctypes.c_char_p, _SZ, ctypes.POINTER(_I)]),
    "tpmlp_trace_enabled": (_I, []),
    "tpmlp_build_flags": (_I, []),
    "tpmlp_selftest_forward_band_timeout": (_I, [_P, _I64, _P, _P, _I, _P, _SZ, _I, _P]),
    "tpmlp_selftest_backward_withheld_fill": (_I, [_P, _P, _I64, _P, _I, _I, _P, _SZ, _P]),
    "tpmlp_selftest_bounds": (_I, [_I, _P]),
}

_lib: Optional[ctypes.CDLL] = None


class TpmlpError(RuntimeError):
    def __init__(self, code: int, where: str, msg: str):
        super().__init__(f"{where} -> {STATUS_NAMES.get(code, code)}: {msg}")
        self.code = code


def lib() -> ctypes.CDLL:
    """The loaded C library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            how = ("`python -m tensor_transformer_mlp_column_gb300.build_lib --debug`" if DEBUG
                   else "`python -c 'import __graft_entry__ as g; g.build()'`")
            raise RuntimeError(f"{LIB_PATH} is missing: build it with {how}")
        l = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(l, name)
            f.restype = res
            f.argtypes = args
        _lib = l
    return _lib


def _check(code: int, where: str) -> None:
    if code != 0:
        raise TpmlpError(code, where, lib().tpmlp_last_error().decode())


def _stream(stream=None) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return TPMLP_BF16
    if t.dtype == torch.float32:
        return TPMLP_F32
    raise TypeError(f"unsupported dtype {t.dtype}; use torch.float32 or torch.bfloat16")


def _dev(t: torch.Tensor, name: str) -> int:
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    return t.data_ptr()


def _mode(mode) -> int:
    if mode in (TPMLP_FAITHFUL, "faithful"):
        return TPMLP_FAITHFUL
    if mode in (TPMLP_FUSED, "fused"):
        return TPMLP_FUSED
    raise ValueError(f"unknown mode {mode!r}")


class _DeviceArray:
    """Exposes library-owned device memory to torch without copying."""

    def __init__(self, ptr: int, shape, typestr: str):
        self.__cuda_array_interface__ = {"shape": tuple(shape), "typestr": typestr, "data": (ptr, False),
                                         "version": 3, "strides": None}


def _alias(ptr: int, shape, dtype: torch.dtype) -> torch.Tensor:
    if dtype == torch.bfloat16:
        return torch.as_tensor(_DeviceArray(ptr, shape, "<i2"), device="cuda").view(torch.bfloat16)
    return torch.as_tensor(_DeviceArray(ptr, shape, "<f4"), device="cuda")


# ----------------------------------------------------------------- API

def tpmlp_version() -> int:
    return lib().tpmlp_version()


def tpmlp_last_error() -> str:
    return lib().tpmlp_last_error().decode()


def tpmlp_check_status(stream=None) -> None:
    """Waits for the stream and raises TpmlpError if a kernel timed out on a wait."""
    _check(lib().tpmlp_check_status(_stream(stream)), "tpmlp_check_status")


def tpmlp_gelu(x: torch.Tensor, out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """GeLU(x) elementwise (GPT-2 tanh form), same dtype as x."""
    y = torch.empty_like(x) if out is None else out
    _check(lib().tpmlp_gelu(_dev(x, "x"), _dev(y, "y"), x.numel(), _dt(x), _stream(stream)), "tpmlp_gelu")
    return y


class Shards:
    """The n shard pairs (A_i, B_i) owned by the library (tpmlp_shards handle)."""

    def __init__(self, handle: int, D: int, F: int, n: int, dtype: torch.dtype):
        self.handle, self.D, self.F, self.n, self.dtype = handle, D, F, n, dtype
        self.Fs = F // n

    def get(self, i: int):
        """(A_i [D, F/n], B_i [F/n, D]) as tensors aliasing the library's copies."""
        a, b = ctypes.c_void_p(), ctypes.c_void_p()
        _check(lib().tpmlp_shard_get(self.handle, i, ctypes.byref(a), ctypes.byref(b)), "tpmlp_shard_get")
        return _alias(a.value, (self.D, self.Fs), self.dtype), _alias(b.value, (self.Fs, self.D), self.dtype)

    def get_transposed(self, i: int):
        """(A_i^T [F/n, D], B_i^T [D, F/n]) for bf16 shards."""
        a, b = ctypes.c_void_p(), ctypes.c_void_p()
        _check(lib().tpmlp_shard_get_transposed(self.handle, i, ctypes.byref(a), ctypes.byref(b)),
               "tpmlp_shard_get_transposed")
        return _alias(a.value, (self.Fs, self.D), self.dtype), _alias(b.value, (self.D, self.Fs), self.dtype)

    def free(self) -> None:
        if self.handle:
            lib().tpmlp_shards_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def tpmlp_shard(A: torch.Tensor, B: torch.Tensor, n: int, stream=None) -> Shards:
    """shard_mlp(A, B, n): the library's own copies of every (A_i, B_i)."""
    D, F = A.shape
    h = ctypes.c_void_p()
    _check(lib().tpmlp_shard(_dev(A, "A"), _dev(B, "B"), D, F, n, _dt(A), _stream(stream), ctypes.byref(h)),
           "tpmlp_shard")
    return Shards(h.value, D, F, n, A.dtype)


def tpmlp_workspace_bytes(T: int, shards: Shards, mode="faithful", backward: int = 0) -> int:
    """backward: 0 = forward, 1 = tpmlp_backward, 2 = tpmlp_backward_saved."""
    return int(lib().tpmlp_workspace_bytes(T, shards.handle, _mode(mode), int(backward)))


def _workspace(nbytes: int, workspace: Optional[torch.Tensor]) -> torch.Tensor:
    if workspace is not None:
        if workspace.numel() * workspace.element_size() < nbytes:
            raise ValueError(f"workspace too small: need {nbytes} bytes")
        return workspace
    return torch.empty(max(nbytes, 16), dtype=torch.uint8, device="cuda")


def tpmlp_forward(X: torch.Tensor, shards: Shards, mode="faithful", Y: Optional[torch.Tensor] = None,
                  workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """tp_mlp(X, shards): Y = sum_i GeLU(X A_i) B_i, fp32 [T, D]."""
    T = X.shape[0]
    Y = torch.empty((T, shards.D), dtype=torch.float32, device=X.device) if Y is None else Y
    nb = tpmlp_workspace_bytes(T, shards, mode, False)
    ws = _workspace(nb, workspace)
    _check(lib().tpmlp_forward(_dev(X, "X"), T, shards.handle, _dev(Y, "Y"), _mode(mode), ws.data_ptr(),
                               ws.numel() * ws.element_size(), _stream(stream)), "tpmlp_forward")
    return Y


def tpmlp_hidden(X: torch.Tensor, shards: Shards, H: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """H_i = GeLU(X A_i) for all shards: [n, T, F/n] in the shards' dtype."""
    T = X.shape[0]
    H = torch.empty((shards.n, T, shards.Fs), dtype=shards.dtype, device=X.device) if H is None else H
    _check(lib().tpmlp_hidden(_dev(X, "X"), T, shards.handle, _dev(H, "H"), _stream(stream)), "tpmlp_hidden")
    return H


def tpmlp_partials(H: torch.Tensor, shards: Shards, Yp: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Y_i = H_i B_i for all shards: [n, T, D] fp32."""
    T = H.shape[1]
    Yp = torch.empty((shards.n, T, shards.D), dtype=torch.float32, device=H.device) if Yp is None else Yp
    _check(lib().tpmlp_partials(_dev(H, "H"), T, shards.handle, _dev(Yp, "Yp"), _stream(stream)), "tpmlp_partials")
    return Yp


def tpmlp_allreduce(Yp: torch.Tensor, Y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Simulated all-reduce: Y = ((Yp[0] + Yp[1]) + ...) + Yp[n-1], fp32."""
    n = Yp.shape[0]
    Y = torch.empty(Yp.shape[1:], dtype=torch.float32, device=Yp.device) if Y is None else Y
    _check(lib().tpmlp_allreduce(_dev(Yp, "Yp"), n, Y.numel(), _dev(Y, "Y"), _stream(stream)), "tpmlp_allreduce")
    return Y


def tpmlp_fused_sum(H: torch.Tensor, shards: Shards, Y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Y = sum_i H_i B_i accumulated on chip in shard order: [T, D] fp32."""
    T = H.shape[1]
    Y = torch.empty((T, shards.D), dtype=torch.float32, device=H.device) if Y is None else Y
    _check(lib().tpmlp_fused_sum(_dev(H, "H"), T, shards.handle, _dev(Y, "Y"), _stream(stream)), "tpmlp_fused_sum")
    return Y


def tpmlp_backward(X: torch.Tensor, dY: torch.Tensor, shards: Shards, mode="faithful",
                   dX: Optional[torch.Tensor] = None, dA: Optional[Sequence[torch.Tensor]] = None,
                   dB: Optional[Sequence[torch.Tensor]] = None, workspace: Optional[torch.Tensor] = None,
                   stream=None, P: Optional[torch.Tensor] = None):
    """Gradients of sum(Y * dY): (dX [T, D], [dA_i [D, F/n]], [dB_i [F/n, D]]), all fp32.

    With P (from tpmlp_forward_save) this is tpmlp_backward_saved, which skips
    recomputing the pre-activations."""
    T, D, Fs, n = X.shape[0], shards.D, shards.Fs, shards.n
    dev = X.device
    dX = torch.empty((T, D), dtype=torch.float32, device=dev) if dX is None else dX
    dA = [torch.empty((D, Fs), dtype=torch.float32, device=dev) for _ in range(n)] if dA is None else list(dA)
    dB = [torch.empty((Fs, D), dtype=torch.float32, device=dev) for _ in range(n)] if dB is None else list(dB)
    pa = (ctypes.c_void_p * n)(*[_dev(t, "dA_i") for t in dA])
    pb = (ctypes.c_void_p * n)(*[_dev(t, "dB_i") for t in dB])
    nb = tpmlp_workspace_bytes(T, shards, mode, 2 if P is not None else 1)
    ws = _workspace(nb, workspace)
    if P is None:
        _check(lib().tpmlp_backward(_dev(X, "X"), _dev(dY, "dY"), T, shards.handle, _dev(dX, "dX"), pa, pb,
                                    _mode(mode), ws.data_ptr(), ws.numel() * ws.element_size(), _stream(stream)),
               "tpmlp_backward")
    else:
        _check(lib().tpmlp_backward_saved(_dev(X, "X"), _dev(dY, "dY"), _dev(P, "P"), T, shards.handle,
                                          _dev(dX, "dX"), pa, pb, _mode(mode), ws.data_ptr(),
                                          ws.numel() * ws.element_size(), _stream(stream)),
               "tpmlp_backward_saved")
    return dX, dA, dB


def tpmlp_backward_saved(X: torch.Tensor, dY: torch.Tensor, P: torch.Tensor, shards: Shards, mode="faithful", **kw):
    """tpmlp_backward with the pre-activations P saved by tpmlp_forward_save."""
    return tpmlp_backward(X, dY, shards, mode, P=P, **kw)


def tpmlp_forward_save(X: torch.Tensor, shards: Shards, mode="faithful", Y: Optional[torch.Tensor] = None,
                       P: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """Training-mode forward: (Y [T, D] fp32, P [n, T, F/n] fp32 pre-activations)."""
    T = X.shape[0]
    Y = torch.empty((T, shards.D), dtype=torch.float32, device=X.device) if Y is None else Y
    P = torch.empty((shards.n, T, shards.Fs), dtype=torch.float32, device=X.device) if P is None else P
    nb = tpmlp_workspace_bytes(T, shards, mode, 0)
    ws = _workspace(nb, workspace)
    _check(lib().tpmlp_forward_save(_dev(X, "X"), T, shards.handle, _dev(Y, "Y"), _dev(P, "P"), _mode(mode),
                                    ws.data_ptr(), ws.numel() * ws.element_size(), _stream(stream)),
           "tpmlp_forward_save")
    return Y, P


def tpmlp_forward_noalloc(X: torch.Tensor, shards: Shards, Y: torch.Tensor, mode="faithful", stream=None) -> torch.Tensor:
    """tp_mlp(X, shards) for callers that cannot allocate device memory: the
    library's fixed 64 MiB scratch replaces the workspace, and the caller
    passes the output Y [T, D] fp32 (nothing is allocated here either)."""
    _check(lib().tpmlp_forward_noalloc(_dev(X, "X"), X.shape[0], shards.handle, _dev(Y, "Y"), _mode(mode),
                                       _stream(stream)), "tpmlp_forward_noalloc")
    return Y


def tpmlp_layer_norm(x: torch.Tensor, eps: float = 1e-5, y: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y = (x - mean) / sqrt(var + eps) per row of x [T, D] (no scale or shift), same dtype as x."""
    y = torch.empty_like(x) if y is None else y
    T, D = x.shape
    _check(lib().tpmlp_layer_norm(_dev(x, "x") if T else 0, T, D, _dt(x), float(eps), _dev(y, "y") if T else 0,
                                  _stream(stream)), "tpmlp_layer_norm")
    return y


def tpmlp_block_workspace_bytes(T: int, shards: Shards, mode="faithful", backward: int = 0) -> int:
    return int(lib().tpmlp_block_workspace_bytes(T, shards.handle, _mode(mode), int(backward)))


def tpmlp_block_forward(x: torch.Tensor, shards: Shards, mode="faithful", eps: float = 1e-5,
                        out: Optional[torch.Tensor] = None, xn: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """out = x + sum_i GeLU(LN(x) A_i) B_i, fp32 [T, D]. With xn, LN(x) is also written there."""
    T = x.shape[0]
    out = torch.empty((T, shards.D), dtype=torch.float32, device=x.device) if out is None else out
    ws = _workspace(tpmlp_block_workspace_bytes(T, shards, mode, 0), workspace)
    _check(lib().tpmlp_block_forward(_dev(x, "x"), T, shards.handle, float(eps), _dev(out, "out"),
                                     _dev(xn, "xn") if xn is not None else None, _mode(mode), ws.data_ptr(),
                                     ws.numel() * ws.element_size(), _stream(stream)), "tpmlp_block_forward")
    return out


def tpmlp_block_backward(x: torch.Tensor, dout: torch.Tensor, shards: Shards, mode="faithful", eps: float = 1e-5,
                         dx: Optional[torch.Tensor] = None, dA: Optional[Sequence[torch.Tensor]] = None,
                         dB: Optional[Sequence[torch.Tensor]] = None, workspace: Optional[torch.Tensor] = None,
                         stream=None):
    """Gradients of sum(out * dout) for tpmlp_block_forward: (dx [T, D], [dA_i], [dB_i]), all fp32."""
    T, D, Fs, n = x.shape[0], shards.D, shards.Fs, shards.n
    dev = x.device
    dx = torch.empty((T, D), dtype=torch.float32, device=dev) if dx is None else dx
    dA = [torch.empty((D, Fs), dtype=torch.float32, device=dev) for _ in range(n)] if dA is None else list(dA)
    dB = [torch.empty((Fs, D), dtype=torch.float32, device=dev) for _ in range(n)] if dB is None else list(dB)
    pa = (ctypes.c_void_p * n)(*[_dev(t, "dA_i") for t in dA])
    pb = (ctypes.c_void_p * n)(*[_dev(t, "dB_i") for t in dB])
    ws = _workspace(tpmlp_block_workspace_bytes(T, shards, mode, 1), workspace)
    _check(lib().tpmlp_block_backward(_dev(x, "x"), _dev(dout, "dout"), T, shards.handle, float(eps), _dev(dx, "dx"),
                                      pa, pb, _mode(mode), ws.data_ptr(), ws.numel() * ws.element_size(),
                                      _stream(stream)), "tpmlp_block_backward")
    return dx, dA, dB


def _ptrs(ts, name):
    return (ctypes.c_void_p * len(ts))(*[_dev(t, name) for t in ts])


def tpmlp_all_gather(slices: Sequence[torch.Tensor], out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The rank slices [T/n, ...] back to back: out [T, ...] (the simulated all-gather)."""
    n = len(slices)
    out = torch.empty((n * slices[0].shape[0],) + tuple(slices[0].shape[1:]), dtype=slices[0].dtype,
                      device=slices[0].device) if out is None else out
    nbytes = slices[0].numel() * slices[0].element_size()
    _check(lib().tpmlp_all_gather(_ptrs(slices, "slice"), n, nbytes, _dev(out, "out"), _stream(stream)),
           "tpmlp_all_gather")
    return out


def tpmlp_reduce_scatter(Yp: torch.Tensor, Y_slices: Optional[Sequence[torch.Tensor]] = None,
                         stream=None) -> list:
    """Rank j's rows of the shard-ordered sum of Yp [n, T, D] fp32: n tensors [T/n, D]."""
    n, T = Yp.shape[0], Yp.shape[1]
    rest = tuple(Yp.shape[2:])
    if Y_slices is None:
        Y_slices = [torch.empty((T // n,) + rest, dtype=torch.float32, device=Yp.device) for _ in range(n)]
    count = Yp[0].numel()
    _check(lib().tpmlp_reduce_scatter(_dev(Yp, "Yp"), n, count, _ptrs(Y_slices, "Y_slice"), _stream(stream)),
           "tpmlp_reduce_scatter")
    return list(Y_slices)


def tpmlp_sp_workspace_bytes(T: int, shards: Shards, mode="faithful", backward: int = 0) -> int:
    return int(lib().tpmlp_sp_workspace_bytes(T, shards.handle, _mode(mode), int(backward)))


def tpmlp_forward_sp(X_slices: Sequence[torch.Tensor], shards: Shards, mode="faithful",
                     Y_slices: Optional[Sequence[torch.Tensor]] = None, workspace: Optional[torch.Tensor] = None,
                     stream=None) -> list:
    """Sequence-parallel forward: rank j's rows of sum_i GeLU(X A_i) B_i, X the all-gather of X_slices."""
    n = shards.n
    Ts = X_slices[0].shape[0]
    dev = X_slices[0].device
    if Y_slices is None:
        Y_slices = [torch.empty((Ts, shards.D), dtype=torch.float32, device=dev) for _ in range(n)]
    T = Ts * len(X_slices)
    ws = _workspace(tpmlp_sp_workspace_bytes(T, shards, mode, 0), workspace)
    _check(lib().tpmlp_forward_sp(_ptrs(X_slices, "X_slice"), T, shards.handle, _ptrs(Y_slices, "Y_slice"),
                                  _mode(mode), ws.data_ptr(), ws.numel() * ws.element_size(), _stream(stream)),
           "tpmlp_forward_sp")
    return list(Y_slices)


def tpmlp_backward_sp(X_slices: Sequence[torch.Tensor], dY_slices: Sequence[torch.Tensor], shards: Shards,
                      mode="faithful", dX_slices: Optional[Sequence[torch.Tensor]] = None,
                      dA: Optional[Sequence[torch.Tensor]] = None, dB: Optional[Sequence[torch.Tensor]] = None,
                      workspace: Optional[torch.Tensor] = None, stream=None):
    """Sequence-parallel backward: ([dX_j [T/n, D]], [dA_i], [dB_i]), all fp32."""
    n, D, Fs = shards.n, shards.D, shards.Fs
    Ts = X_slices[0].shape[0]
    dev = X_slices[0].device
    T = Ts * len(X_slices)
    if dX_slices is None:
        dX_slices = [torch.empty((Ts, D), dtype=torch.float32, device=dev) for _ in range(n)]
    dA = [torch.empty((D, Fs), dtype=torch.float32, device=dev) for _ in range(n)] if dA is None else list(dA)
    dB = [torch.empty((Fs, D), dtype=torch.float32, device=dev) for _ in range(n)] if dB is None else list(dB)
    ws = _workspace(tpmlp_sp_workspace_bytes(T, shards, mode, 1), workspace)
    _check(lib().tpmlp_backward_sp(_ptrs(X_slices, "X_slice"), _ptrs(dY_slices, "dY_slice"), T, shards.handle,
                                   _ptrs(dX_slices, "dX_slice"), _ptrs(dA, "dA_i"), _ptrs(dB, "dB_i"), _mode(mode),
                                   ws.data_ptr(), ws.numel() * ws.element_size(), _stream(stream)),
           "tpmlp_backward_sp")
    return list(dX_slices), dA, dB


class AttnShards:
    """Handle of head-split attention weights (tpmlp_attn_shard)."""

    def __init__(self, handle, D: int, heads: int, n: int, dtype: torch.dtype, device):
        self.handle = handle
        self.D, self.heads, self.n, self.dtype, self.device = D, heads, n, dtype, device
        self.Dn = D // n
        self.dh = D // heads

    def get(self, i: int):
        """Rank i's (Wqkv_i, Wo_i) as tensors aliasing the handle's memory (layouts in tpmlp.h)."""
        a, b = ctypes.c_void_p(), ctypes.c_void_p()
        _check(lib().tpmlp_attn_shard_get(self.handle, i, ctypes.byref(a), ctypes.byref(b)), "tpmlp_attn_shard_get")
        if self.dtype == torch.bfloat16:
            return _alias(a.value, (3 * self.Dn, self.D), self.dtype), _alias(b.value, (self.D, self.Dn), self.dtype)
        return _alias(a.value, (self.D, 3 * self.Dn), self.dtype), _alias(b.value, (self.Dn, self.D), self.dtype)

    def free(self):
        if self.handle:
            lib().tpmlp_attn_shards_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.free()
        except Exception:
            pass


def tpmlp_attn_shard(Wq, Wk, Wv, Wo, heads: int, n: int, stream=None) -> AttnShards:
    """Split Wq, Wk, Wv by columns and Wo by rows into n ranks of heads/n heads each."""
    D = Wq.shape[0]
    h = ctypes.c_void_p()
    _check(lib().tpmlp_attn_shard(_dev(Wq, "Wq"), _dev(Wk, "Wk"), _dev(Wv, "Wv"), _dev(Wo, "Wo"), D, heads, n,
                                  _dt(Wq), _stream(stream), ctypes.byref(h)), "tpmlp_attn_shard")
    return AttnShards(h.value, D, heads, n, Wq.dtype, Wq.device)


def tpmlp_attn_workspace_bytes(batch: int, seq: int, shards: AttnShards, mode="faithful") -> int:
    m = -1 if mode is None else _mode(mode)
    return int(lib().tpmlp_attn_workspace_bytes(batch, seq, shards.handle, m))


def tpmlp_attn_heads(X: torch.Tensor, batch: int, shards: AttnShards, O: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Every rank's local attention heads: O [n, T, D/n] of X's dtype."""
    T = X.shape[0]
    seq = T // batch
    O = torch.empty((shards.n, T, shards.Dn), dtype=X.dtype, device=X.device) if O is None else O
    ws = _workspace(tpmlp_attn_workspace_bytes(batch, seq, shards, None), workspace)
    _check(lib().tpmlp_attn_heads(_dev(X, "X"), batch, seq, shards.handle, _dev(O, "O"), ws.data_ptr(),
                                  ws.numel() * ws.element_size(), _stream(stream)), "tpmlp_attn_heads")
    return O


def tpmlp_attn_forward(X: torch.Tensor, batch: int, shards: AttnShards, mode="faithful",
                       Y: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                       stream=None) -> torch.Tensor:
    """Y = sum_i O_i Wo_i, fp32 [T, D]."""
    T = X.shape[0]
    seq = T // batch
    Y = torch.empty((T, shards.D), dtype=torch.float32, device=X.device) if Y is None else Y
    ws = _workspace(tpmlp_attn_workspace_bytes(batch, seq, shards, mode), workspace)
    _check(lib().tpmlp_attn_forward(_dev(X, "X"), batch, seq, shards.handle, _dev(Y, "Y"), _mode(mode),
                                    ws.data_ptr(), ws.numel() * ws.element_size(), _stream(stream)),
           "tpmlp_attn_forward")
    return Y


# ------------------------------------------------- the two ends of a training step

# These calls may be a few microseconds of GPU work (one token's lookup, one
# small layer's clipping), so the binding keeps its own part short: one pass
# over the tensors, the raw stream, no array objects built element by element.

_DTYPES = {torch.float32: TPMLP_F32, torch.bfloat16: TPMLP_BF16}


def _ptr(t: torch.Tensor, dev: int, name: str) -> int:
    """Address of a contiguous tensor on device `dev`, the current one."""
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, but CUDA device {dev} is current")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _type(t: torch.Tensor) -> int:
    dt = _DTYPES.get(t.dtype)
    if dt is None:
        raise TypeError(f"unsupported dtype {t.dtype}; use torch.float32 or torch.bfloat16")
    return dt


def _ids(t: torch.Tensor, T: int, dev: int, name: str) -> int:
    if t.dtype != torch.int64 or t.dim() != 1 or t.shape[0] != T:
        raise ValueError(f"{name} must be an int64 tensor of {T} ids")
    return _ptr(t, dev, name)


def _like(t: torch.Tensor, shape, dtype: torch.dtype, dev: int, name: str) -> int:
    if t.dtype != dtype or t.shape != shape:
        raise ValueError(f"{name} must be {dtype} of shape {tuple(shape)}")
    return _ptr(t, dev, name)


def _output(t: Optional[torch.Tensor], shape, dtype: torch.dtype, dev: int, name: str):
    """(tensor, address) of an output, the caller's or a new one."""
    if t is None:
        t = torch.empty(shape, dtype=dtype, device="cuda")
        return t, t.data_ptr()
    return t, _like(t, shape, dtype, dev, name)


def _space(nbytes: int, workspace: Optional[torch.Tensor], dev: int):
    """(tensor, address, bytes) of a call's workspace."""
    if workspace is None:
        workspace = torch.empty(max(nbytes, 16), dtype=torch.uint8, device="cuda")
        return workspace, workspace.data_ptr(), workspace.numel()
    have = workspace.numel() * workspace.element_size()
    if have < nbytes:
        raise ValueError(f"workspace too small: need {nbytes} bytes")
    return workspace, _ptr(workspace, dev, "workspace"), have


class _On:
    """A call's device and stream. Outputs and workspace are allocated with the
    call's stream current, so that the caching allocator does not hand their
    memory to another stream's work while the call may still use it."""

    __slots__ = ("dev", "raw", "ctx")

    def __init__(self, stream):
        self.ctx = None
        if not torch.cuda.is_initialized():
            torch.cuda.init()
        self.dev = torch._C._cuda_getDevice()
        self.raw = torch._C._cuda_getCurrentRawStream(self.dev)
        if stream is not None:
            raw = _stream(stream)
            if raw != self.raw:
                self.raw = raw
                s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(raw)
                self.ctx = torch.cuda.stream(s)

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()
        return self

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)


def tpmlp_xent_workspace_bytes(T: int, D: int, V: int, dtype: torch.dtype, backward: int = 0) -> int:
    return int(lib().tpmlp_xent_workspace_bytes(T, D, V, TPMLP_BF16 if dtype == torch.bfloat16 else TPMLP_F32,
                                                int(backward)))


def _xent_shapes(X: torch.Tensor, W: torch.Tensor):
    xs, vs = X.shape, W.shape
    if len(xs) != 2 or len(vs) != 2 or xs[1] != vs[1] or X.dtype != W.dtype:
        raise ValueError("X must be [T, D] and W [V, D], of one dtype")
    return xs[0], xs[1], vs[0]


@functools.lru_cache(maxsize=1024)
def _xent_workspace(dev: int, T: int, D: int, V: int, dt: int, backward: int) -> int:
    return int(lib().tpmlp_xent_workspace_bytes(T, D, V, dt, backward))


def tpmlp_xent_forward(X: torch.Tensor, W: torch.Tensor, targets: torch.Tensor, loss: Optional[torch.Tensor] = None,
                       lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """Cross entropy of softmax(X W^T) at the targets without keeping the logits:
    (loss [T], lse [T]) fp32. A negative target's row has no loss."""
    T, D, V = _xent_shapes(X, W)
    dt, l = _type(X), lib()
    with _On(stream) as on:
        dev = on.dev
        x, w, t = _ptr(X, dev, "X"), _ptr(W, dev, "W"), _ids(targets, T, dev, "targets")
        loss, lp = _output(loss, (T,), torch.float32, dev, "loss")
        lse, ep = _output(lse, (T,), torch.float32, dev, "lse")
        ws, wp, wn = _space(_xent_workspace(dev, T, D, V, dt, 0), workspace, dev)
        _check(l.tpmlp_xent_forward(x, w, t, T, D, V, dt, lp, ep, wp, wn, on.raw), "tpmlp_xent_forward")
    return loss, lse


def tpmlp_xent_backward(X: torch.Tensor, W: torch.Tensor, targets: torch.Tensor, lse: torch.Tensor,
                        dloss: torch.Tensor, dX: Optional[torch.Tensor] = None, dW: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, stream=None, loss: Optional[torch.Tensor] = None):
    """Gradients of sum(dloss * loss) of tpmlp_xent_forward: (dX [T, D], dW [V, D]) of X's dtype.
    With the forward's loss (tpmlp_xent_backward_saved) nearly certain rows keep their target's part."""
    T, D, V = _xent_shapes(X, W)
    dt, l = _type(X), lib()
    with _On(stream) as on:
        dev = on.dev
        x, w, t = _ptr(X, dev, "X"), _ptr(W, dev, "W"), _ids(targets, T, dev, "targets")
        dX, xp = _output(dX, (T, D), X.dtype, dev, "dX")
        dW, vp = _output(dW, (V, D), X.dtype, dev, "dW")
        ws, wp, wn = _space(_xent_workspace(dev, T, D, V, dt, 1), workspace, dev)
        rest = (_like(lse, (T,), torch.float32, dev, "lse"), _like(dloss, (T,), torch.float32, dev, "dloss"), T, D, V, dt,
                xp, vp, wp, wn, on.raw)
        if loss is None:
            _check(l.tpmlp_xent_backward(x, w, t, *rest), "tpmlp_xent_backward")
        else:
            _check(l.tpmlp_xent_backward_saved(x, w, t, _like(loss, (T,), torch.float32, dev, "loss"), *rest),
                   "tpmlp_xent_backward_saved")
    return dX, dW


def tpmlp_embed_forward(E: torch.Tensor, ids: torch.Tensor, scale: float = 1.0, out: Optional[torch.Tensor] = None,
                        stream=None) -> torch.Tensor:
    """out[t] = scale * E[ids[t]], of E's dtype; zero rows for negative ids."""
    V, D = E.shape
    T, dt = ids.shape[0], _type(E)
    with _On(stream) as on:
        dev = on.dev
        e, i = _ptr(E, dev, "E"), _ids(ids, T, dev, "ids")
        out, o = _output(out, (T, D), E.dtype, dev, "out")
        _check(lib().tpmlp_embed_forward(e, i, T, D, V, dt, float(scale), o, on.raw), "tpmlp_embed_forward")
    return out


def tpmlp_embed_workspace_bytes(T: int, D: int, V: int) -> int:
    return int(lib().tpmlp_embed_workspace_bytes(T, D, V))


def tpmlp_embed_backward(dout: torch.Tensor, ids: torch.Tensor, V: int, scale: float = 1.0,
                         dE: Optional[torch.Tensor] = None, accumulate: bool = False,
                         dtype: Optional[torch.dtype] = None, workspace: Optional[torch.Tensor] = None,
                         stream=None) -> torch.Tensor:
    """dE[v] = scale * sum of dout[t] over ids[t] = v, [V, D] of `dtype` (default
    dout's); with accumulate, added to the given dE."""
    T, D = dout.shape
    if accumulate and dE is None:
        raise ValueError("accumulate needs dE")
    if dE is None:
        dtype = dout.dtype if dtype is None else dtype
    elif dtype is not None and dtype != dE.dtype:
        raise ValueError("dtype and dE disagree")
    l = lib()
    with _On(stream) as on:
        dev = on.dev
        g, i = _ptr(dout, dev, "dout"), _ids(ids, T, dev, "ids")
        dE, e = _output(dE, (V, D), dtype if dE is None else dE.dtype, dev, "dE")
        ws, wp, wn = _space(l.tpmlp_embed_workspace_bytes(T, D, V), workspace, dev)
        _check(l.tpmlp_embed_backward(g, _type(dout), i, T, D, V, float(scale), e, _type(dE), 1 if accumulate else 0,
                                      wp, wn, on.raw), "tpmlp_embed_backward")
    return dE


def tpmlp_grad_workspace_bytes(n: int) -> int:
    return int(lib().tpmlp_grad_workspace_bytes(n))


_DATA_PTR, _NUMEL = torch.Tensor.data_ptr, torch.Tensor.numel
_DEVICE, _CONTIGUOUS = torch.Tensor.get_device, torch.Tensor.is_contiguous


def _addresses(ts: Sequence[torch.Tensor], dev: int, name: str) -> array:
    devices = list(map(_DEVICE, ts))
    if devices.count(dev) != len(devices) or not all(map(_CONTIGUOUS, ts)):
        for t in ts:
            _ptr(t, dev, name)  # says what is wrong
    return array("Q", list(map(_DATA_PTR, ts)))


def _grads(grads: Sequence[torch.Tensor], dev: int):
    """Addresses, element counts and types of the gradients, as arrays."""
    try:
        types = array("i", [_DTYPES[g.dtype] for g in grads])
    except KeyError as e:
        raise TypeError(f"unsupported dtype {e}; use torch.float32 or torch.bfloat16") from None
    return _addresses(grads, dev, "a gradient"), array("q", list(map(_NUMEL, grads))), types


def tpmlp_grad_norm(grads: Sequence[torch.Tensor], norm: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The global norm of all gradients (fp32 and bf16 tensors mixed): [1] fp32."""
    n, l = len(grads), lib()
    with _On(stream) as on:
        p, c, d = _grads(grads, on.dev)
        norm, np_ = _output(norm, (1,), torch.float32, on.dev, "norm")
        ws, wp, wn = _space(l.tpmlp_grad_workspace_bytes(n), workspace, on.dev)
        _check(l.tpmlp_grad_norm(p.buffer_info()[0], c.buffer_info()[0], d.buffer_info()[0], n, np_, wp, wn, on.raw),
               "tpmlp_grad_norm")
    return norm


def tpmlp_grad_clip(grads: Sequence[torch.Tensor], max_norm: float, out: Optional[Sequence[torch.Tensor]] = None,
                    norm: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """Scales all gradients by min(1, max_norm / (norm + 1e-6)), in place or into
    `out`, and returns their global norm before that: [1] fp32."""
    n, l = len(grads), lib()
    with _On(stream) as on:
        p, c, d = _grads(grads, on.dev)
        o = None
        if out is not None:
            if len(out) != n or list(map(_NUMEL, out)) != c.tolist() or [t.dtype for t in out] != [g.dtype for g in grads]:
                raise ValueError("out must have a tensor of each gradient's size and dtype")
            o = _addresses(out, on.dev, "an output")
        norm, np_ = _output(norm, (1,), torch.float32, on.dev, "norm")
        ws, wp, wn = _space(l.tpmlp_grad_workspace_bytes(n), workspace, on.dev)
        _check(l.tpmlp_grad_clip(p.buffer_info()[0], c.buffer_info()[0], d.buffer_info()[0], n, float(max_norm),
                                 None if o is None else o.buffer_info()[0], np_, wp, wn, on.raw), "tpmlp_grad_clip")
    return norm


# ------------------------------------------------- the attention of a training step


def _heads(t: torch.Tensor, T: int, heads: int, dim: int, dtype: torch.dtype, dev: int, strides: list, name: str) -> int:
    """Address of a tensor [T, heads, dim] on device `dev`; its two strides go to `strides`."""
    if t.dtype != dtype or t.shape != (T, heads, dim):
        raise ValueError(f"{name} must be {dtype} of shape {(T, heads, dim)}")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, but CUDA device {dev} is current")
    token, head, one = t.stride()
    if one != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    strides += (token, head)
    return t.data_ptr()


def _heads_output(t: Optional[torch.Tensor], T: int, heads: int, dim: int, dtype: torch.dtype, dev: int, strides: list,
                  name: str):
    """(tensor, address) of an output [T, heads, dim], the caller's or a new one."""
    if t is None:
        t = torch.empty((T, heads, dim), dtype=dtype, device="cuda")
        strides += (heads * dim, dim)
        return t, t.data_ptr()
    return t, _heads(t, T, heads, dim, dtype, dev, strides, name)


def _qkv_shape(q: torch.Tensor, k: torch.Tensor):
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q must be [T, heads, head_dim] and k [T, kv_heads, head_dim]")
    T, heads, dim = q.shape
    return T, heads, k.shape[1], dim


def _sequences(starts: Optional[torch.Tensor], max_seq: Optional[int], batch: Optional[int], T: int, dev: int):
    """(address of starts or 0, batch, max_seq)."""
    if starts is None:
        batch = 1 if batch is None else int(batch)
        if batch < 1 or T % batch != 0 or max_seq not in (None, T // batch):
            raise ValueError(f"without starts the {T} tokens must be {batch} equal sequences")
        return 0, batch, T // batch
    shape = starts.shape
    if starts.dtype != torch.int32 or len(shape) != 1 or shape[0] < 1:
        raise ValueError("starts must be an int32 tensor of one more element than there are sequences")
    if batch not in (None, shape[0] - 1):
        raise ValueError("batch and starts disagree")
    return _ptr(starts, dev, "starts"), shape[0] - 1, T if max_seq is None else min(int(max_seq), T)


def tpmlp_attn_core_forward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, starts: Optional[torch.Tensor] = None,
                            max_seq: Optional[int] = None, batch: Optional[int] = None, scale: Optional[float] = None,
                            causal: bool = True, o: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                            stream=None):
    """Softmax attention of q [T, heads, head_dim] over k, v [T, kv_heads, head_dim]: (o as q, lse [heads, T] fp32).

    The T tokens are `batch` equal sequences (default 1), or those from starts[b] to starts[b + 1] - 1 (int32 on the
    GPU), none longer than max_seq (default T; the longest length is the better value: see tpmlp_attn_core_backward).
    Rows of no sequence are left as they were: undefined in an o or lse that the call allocates. scale is 1 / sqrt(head_dim) by default."""
    T, heads, kv, dim = _qkv_shape(q, k)
    dt, strides = _type(q), []
    with _On(stream) as on:
        dev = on.dev
        qp = _heads(q, T, heads, dim, q.dtype, dev, strides, "q")
        kp = _heads(k, T, kv, dim, q.dtype, dev, strides, "k")
        vp = _heads(v, T, kv, dim, q.dtype, dev, strides, "v")
        sp, n, most = _sequences(starts, max_seq, batch, T, dev)
        o, op = _heads_output(o, T, heads, dim, q.dtype, dev, strides, "o")
        lse, lp = _output(lse, (heads, T), torch.float32, dev, "lse")
        strides = array("q", strides)
        _check(lib().tpmlp_attn_core_forward(qp, kp, vp, strides.buffer_info()[0], sp, T, n, most, heads, kv, dim,
                                             dim ** -0.5 if scale is None else float(scale), 1 if causal else 0, dt, op,
                                             lp, on.raw), "tpmlp_attn_core_forward")
    return o, lse


@functools.lru_cache(maxsize=1024)
def _core_workspace(dev: int, T: int, batch: int, max_seq: int, heads: int, kv_heads: int, head_dim: int, dt: int) -> int:
    return int(lib().tpmlp_attn_core_workspace_bytes(T, batch, max_seq, heads, kv_heads, head_dim, dt))


def tpmlp_attn_core_workspace_bytes(T: int, heads: int, kv_heads: int, head_dim: int, dtype: torch.dtype, batch: int = 1,
                                    max_seq: Optional[int] = None) -> int:
    """Of tpmlp_attn_core_backward on `batch` sequences of at most max_seq tokens (default T / batch)."""
    return int(lib().tpmlp_attn_core_workspace_bytes(T, batch, T // max(batch, 1) if max_seq is None else max_seq, heads, kv_heads,
                                                     head_dim, TPMLP_BF16 if dtype == torch.bfloat16 else TPMLP_F32))


def tpmlp_attn_core_backward(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, o: torch.Tensor, lse: torch.Tensor,
                             do: torch.Tensor, starts: Optional[torch.Tensor] = None, max_seq: Optional[int] = None,
                             batch: Optional[int] = None, scale: Optional[float] = None, causal: bool = True,
                             dq: Optional[torch.Tensor] = None, dk: Optional[torch.Tensor] = None,
                             dv: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradients of sum(o * do) of tpmlp_attn_core_forward with the same arguments: (dq, dk, dv), as q, k, v. The
    probabilities are made again from lse. Rows of no sequence are left as they were: undefined in gradients that the
    call allocates. With max_seq far above the lengths, dk and dv of few sequences on few kv heads take longer (bf16, 8 of
    512 tokens, 32 heads on one: 211 us in the place of 64), and dq and dk of sequences within 64 tokens (heads above 64:
    128) are off by 0.0024 in the place of 0.0017."""
    T, heads, kv, dim = _qkv_shape(q, k)
    dt, l, strides = _type(q), lib(), []
    with _On(stream) as on:
        dev = on.dev
        qp = _heads(q, T, heads, dim, q.dtype, dev, strides, "q")
        kp = _heads(k, T, kv, dim, q.dtype, dev, strides, "k")
        vp = _heads(v, T, kv, dim, q.dtype, dev, strides, "v")
        op = _heads(o, T, heads, dim, q.dtype, dev, strides, "o")
        gp = _heads(do, T, heads, dim, q.dtype, dev, strides, "do")
        sp, n, most = _sequences(starts, max_seq, batch, T, dev)
        dq, dqp = _heads_output(dq, T, heads, dim, q.dtype, dev, strides, "dq")
        dk, dkp = _heads_output(dk, T, kv, dim, q.dtype, dev, strides, "dk")
        dv, dvp = _heads_output(dv, T, kv, dim, q.dtype, dev, strides, "dv")
        ws, wp, wn = _space(_core_workspace(dev, T, n, most, heads, kv, dim, dt), workspace, dev)
        strides = array("q", strides)
        _check(l.tpmlp_attn_core_backward(qp, kp, vp, op, _like(lse, (heads, T), torch.float32, dev, "lse"), gp,
                                          strides.buffer_info()[0], sp, T, n, most, heads, kv, dim,
                                          dim ** -0.5 if scale is None else float(scale), 1 if causal else 0, dt, dqp, dkp,
                                          dvp, wp, wn, on.raw), "tpmlp_attn_core_backward")
    return dq, dk, dv


@functools.lru_cache(maxsize=64)
def _turns(freqs: tuple, axis: Optional[tuple], axes: int):
    """The frequencies and their axes as host arrays, and the arrays' addresses."""
    if axis is not None and (len(axis) != len(freqs) or any(a < 0 or a >= min(axes, 256) for a in axis)):
        raise ValueError(f"axis must give one of {axes} axes for each of the {len(freqs)} frequencies")
    f, a = array("d", freqs), None if axis is None else array("B", axis)
    return f, a, f.buffer_info()[0], None if a is None else a.buffer_info()[0]


_last_turns = (None, None, 0, None)
_NUMBERS = {int, float}


def _axis_values(axis):
    """The axes by value: their bytes, () for none, None where they are no list of small integers."""
    if axis is None:
        return ()
    try:
        return bytes(axis) if type(axis) in (list, tuple) else None
    except (TypeError, ValueError, OverflowError):
        return None


def _rope_args(q, k, pos, freqs, axis, interleaved, wq, wk, eps, dev):
    """What both calls take: the shape and the arguments between the strides and the outputs."""
    T, heads, kv, dim = _qkv_shape(q, k)
    at = pos.shape
    if pos.dtype != torch.int64 or len(at) not in (1, 2) or at[-1] != T:
        raise ValueError(f"pos must be an int64 tensor of {T} positions, or [axes, {T}]")
    axes = at[0] if len(at) == 2 else 1
    # A program's frequencies are the same in every call: the last call's arrays serve while its values are equal. Only
    # Python's own numbers are compared so: 0-dim tensors and arrays may be views whose values change, in the kept copy of
    # the list too, and compare in their own precision.
    global _last_turns
    last = _last_turns
    turned_by = _axis_values(axis)
    plain = turned_by is not None and isinstance(freqs, (list, tuple)) and set(map(type, freqs)) <= _NUMBERS
    if plain and last[0] == freqs and last[1] == turned_by and last[2] == axes:
        keep = last[3]
    else:
        keep = _turns(tuple(map(float, freqs)), None if axis is None else tuple(map(int, axis)), axes)
        if plain:
            _last_turns = (freqs[:], turned_by, axes, keep)
    wqp = 0 if wq is None else _like(wq, (dim,), q.dtype, dev, "wq")
    wkp = 0 if wk is None else _like(wk, (dim,), q.dtype, dev, "wk")
    return (T, heads, kv, dim), (wqp, wkp, eps, _ptr(pos, dev, "pos"), keep[2], keep[3], T, heads, kv, dim,
                                 2 * len(keep[0]), axes, 1 if interleaved else 0, _type(q)), keep


def tpmlp_qk_rope_forward(q: torch.Tensor, k: torch.Tensor, pos: torch.Tensor, freqs: Sequence[float],
                          axis: Optional[Sequence[int]] = None, interleaved: bool = False,
                          wq: Optional[torch.Tensor] = None, wk: Optional[torch.Tensor] = None, eps: float = 1e-6,
                          yq: Optional[torch.Tensor] = None, yk: Optional[torch.Tensor] = None, stream=None):
    """Every head of q [T, heads, head_dim] and k [T, kv_heads, head_dim] normed (root mean square) and scaled by wq or
    wk (both None: not), then its pairs turned by pos * freqs: (yq, yk). Pair i is (i, i + len(freqs)), or
    (2 i, 2 i + 1) when interleaved. pos is int64 [T], or [axes, T] with axis[i] naming the axis that turns pair i.
    yq may be q and yk may be k."""
    strides = []
    with _On(stream) as on:
        dev = on.dev
        (T, heads, kv, dim), args, keep = _rope_args(q, k, pos, freqs, axis, interleaved, wq, wk, eps, dev)
        qp = _heads(q, T, heads, dim, q.dtype, dev, strides, "q")
        kp = _heads(k, T, kv, dim, q.dtype, dev, strides, "k")
        yq, yqp = _heads_output(yq, T, heads, dim, q.dtype, dev, strides, "yq")
        yk, ykp = _heads_output(yk, T, kv, dim, q.dtype, dev, strides, "yk")
        strides = array("q", strides)
        _check(lib().tpmlp_qk_rope_forward(qp, kp, strides.buffer_info()[0], *args, yqp, ykp, on.raw),
               "tpmlp_qk_rope_forward")
    return yq, yk


def tpmlp_qk_rope_workspace_bytes(T: int, heads: int, kv_heads: int, head_dim: int) -> int:
    return int(lib().tpmlp_qk_rope_workspace_bytes(T, heads, kv_heads, head_dim))


@functools.lru_cache(maxsize=1024)
def _rope_workspace(T: int, heads: int, kv_heads: int, head_dim: int) -> int:
    return int(lib().tpmlp_qk_rope_workspace_bytes(T, heads, kv_heads, head_dim))


def tpmlp_qk_rope_backward(dyq: torch.Tensor, dyk: torch.Tensor, q: torch.Tensor, k: torch.Tensor, pos: torch.Tensor,
                           freqs: Sequence[float], axis: Optional[Sequence[int]] = None, interleaved: bool = False,
                           wq: Optional[torch.Tensor] = None, wk: Optional[torch.Tensor] = None, eps: float = 1e-6,
                           dq: Optional[torch.Tensor] = None, dk: Optional[torch.Tensor] = None,
                           dwq: Optional[torch.Tensor] = None, dwk: Optional[torch.Tensor] = None,
                           workspace: Optional[torch.Tensor] = None, stream=None):
    """Gradients of sum(yq * dyq) + sum(yk * dyk) of tpmlp_qk_rope_forward: (dq, dk, dwq, dwk), the weights' in fp32 and
    None without weights. dq may be dyq and dk may be dyk."""
    l, strides = lib(), []
    with _On(stream) as on:
        dev = on.dev
        (T, heads, kv, dim), args, keep = _rope_args(q, k, pos, freqs, axis, interleaved, wq, wk, eps, dev)
        qp = _heads(q, T, heads, dim, q.dtype, dev, strides, "q")
        kp = _heads(k, T, kv, dim, q.dtype, dev, strides, "k")
        gq = _heads(dyq, T, heads, dim, q.dtype, dev, strides, "dyq")
        gk = _heads(dyk, T, kv, dim, q.dtype, dev, strides, "dyk")
        dq, dqp = _heads_output(dq, T, heads, dim, q.dtype, dev, strides, "dq")
        dk, dkp = _heads_output(dk, T, kv, dim, q.dtype, dev, strides, "dk")
        wqp = wkp = wp = wn = 0
        if wq is not None:
            dwq, wqp = _output(dwq, (dim,), torch.float32, dev, "dwq")
            dwk, wkp = _output(dwk, (dim,), torch.float32, dev, "dwk")
            ws, wp, wn = _space(_rope_workspace(T, heads, kv, dim), workspace, dev)
        elif dwq is not None or dwk is not None:
            raise ValueError("dwq and dwk need wq and wk")
        strides = array("q", strides)
        _check(l.tpmlp_qk_rope_backward(gq, gk, qp, kp, strides.buffer_info()[0], *args, dqp, dkp, wqp, wkp, wp, wn, on.raw),
               "tpmlp_qk_rope_backward")
    return dq, dk, dwq, dwk


def tpmlp_selftest_gemm_withheld_fill(X: torch.Tensor, shards: Shards, H: torch.Tensor, fill: int, limit_ms: int,
                                      stream=None) -> None:
    """Runs the GeLU(X A_i) product with stage fill `fill` withheld (test hook)."""
    _check(lib().tpmlp_selftest_gemm_withheld_fill(_dev(X, "X"), X.shape[0], shards.handle, _dev(H, "H"), fill,
                                                   limit_ms, _stream(stream)), "tpmlp_selftest_gemm_withheld_fill")


def tpmlp_selftest_wait_timeout(limit_ms: int, stream=None) -> None:
    _check(lib().tpmlp_selftest_wait_timeout(limit_ms, _stream(stream)), "tpmlp_selftest_wait_timeout")


def tpmlp_trace_enabled() -> bool:
    """True when the library records per-step times (TPMLP_TRACE=1 when it was loaded)."""
    return bool(lib().tpmlp_trace_enabled())


def tpmlp_trace_read(max_bytes: int = 1 << 20):
    """Waits for the steps recorded since the last read and returns them as
    [(step name, device milliseconds)] in the order they were enqueued; [] when
    tracing is off."""
    buf = ctypes.create_string_buffer(max_bytes)
    count = ctypes.c_int(0)
    _check(lib().tpmlp_trace_read(buf, max_bytes, ctypes.byref(count)), "tpmlp_trace_read")
    out = []
    for line in buf.value.decode().splitlines():
        name, ms = line.rsplit(" ", 1)
        out.append((name, float(ms)))
    return out


def tpmlp_build_flags() -> int:
    """Bit 0: the loaded library is the debug build (device-side index checks)."""
    return lib().tpmlp_build_flags()


def tpmlp_selftest_bounds(index: int, stream=None) -> None:
    """Debug build: a device-side check of `index` against a 32-element array
    (test hook; a failed check shows in the next tpmlp_check_status)."""
    _check(lib().tpmlp_selftest_bounds(index, _stream(stream)), "tpmlp_selftest_bounds")


def tpmlp_selftest_forward_band_timeout(X: torch.Tensor, shards: Shards, Y: torch.Tensor, mode, limit_ms: int,
                                        workspace: Optional[torch.Tensor] = None, stream=None) -> None:
    """Runs the one-launch forward with bands of H that never complete (test hook)."""
    ws = _workspace(tpmlp_workspace_bytes(X.shape[0], shards, mode, 0), workspace)
    _check(lib().tpmlp_selftest_forward_band_timeout(_dev(X, "X"), X.shape[0], shards.handle, _dev(Y, "Y"),
                                                     _mode(mode), ws.data_ptr(), ws.numel() * ws.element_size(),
                                                     limit_ms, _stream(stream)), "tpmlp_selftest_forward_band_timeout")


def tpmlp_selftest_backward_withheld_fill(X: torch.Tensor, dY: torch.Tensor, shards: Shards, fill: int,
                                          limit_ms: int, workspace: Optional[torch.Tensor] = None,
                                          stream=None) -> None:
    """Runs the backward's dual-accumulator kernel with stage fill `fill` withheld (test hook)."""
    ws = _workspace(tpmlp_workspace_bytes(X.shape[0], shards, "fused", 1), workspace)
    _check(lib().tpmlp_selftest_backward_withheld_fill(_dev(X, "X"), _dev(dY, "dY"), X.shape[0], shards.handle,
                                                       fill, limit_ms, ws.data_ptr(), ws.numel() * ws.element_size(),
                                                       _stream(stream)), "tpmlp_selftest_backward_withheld_fill")


def tpmlp_selftest_xent_stage_timeout(X: torch.Tensor, W: torch.Tensor, targets: torch.Tensor, stage: int, limit_ms: int,
                                      stream=None) -> None:
    """Runs the cross entropy's logits with stage `stage` of the operands' ring never complete (test hook)."""
    T, D, V = _xent_shapes(X, W)
    dt, l = _type(X), lib()
    with _On(stream) as on:
        dev = on.dev
        x, w, t = _ptr(X, dev, "X"), _ptr(W, dev, "W"), _ids(targets, T, dev, "targets")
        loss, lp = _output(None, (T,), torch.float32, dev, "loss")
        lse, ep = _output(None, (T,), torch.float32, dev, "lse")
        ws, wp, wn = _space(_xent_workspace(dev, T, D, V, dt, 0), None, dev)
        _check(l.tpmlp_selftest_xent_stage_timeout(x, w, t, T, D, V, dt, lp, ep, stage, limit_ms, wp, wn, on.raw),
               "tpmlp_selftest_xent_stage_timeout")


def tpmlp_selftest_attn_core_timeout(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, backward: bool, load: int,
                                     limit_ms: int, stream=None) -> None:
    """Runs the bf16 attention's forward or backward on one sequence with load `load` of every CTA withheld (test hook)."""
    if q.dim() != 3 or k.shape != q.shape or v.shape != q.shape or {q.dtype, k.dtype, v.dtype} != {torch.bfloat16}:
        raise ValueError("q, k and v must be torch.bfloat16 of one shape [T, heads, head_dim]")
    T, heads, dim = q.shape
    with _On(stream) as on:
        q, k, v = (t.contiguous() for t in (q, k, v))
        o, do, dq, dk, dv = (torch.zeros_like(q) for _ in range(5))
        lse = torch.zeros((heads, T), dtype=torch.float32, device="cuda")
        ws, wp, wn = _space(_core_workspace(on.dev, T, 1, T, heads, heads, dim, TPMLP_BF16), None, on.dev)
        p = [_ptr(t, on.dev, "q, k or v") for t in (q, k, v)]
        _check(lib().tpmlp_selftest_attn_core_timeout(*p, o.data_ptr(), lse.data_ptr(), do.data_ptr(), T, heads, dim,
                                                      dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), wp, wn,
                                                      1 if backward else 0, load, limit_ms, on.raw),
               "tpmlp_selftest_attn_core_timeout")
