"""Python binding of libq2 (the Q2_0 ternary linear for gfx950).

Argument marshalling only: every function hands torch tensors' device
pointers, sizes and torch's current HIP stream to the C ABI declared in
include/q2.h; all arithmetic runs in the library's HIP kernels.  Output
tensors are allocated with torch when the caller does not pass them.  The
library is loaded lazily; a missing or unloadable library raises at the first
call, never falls back to anything else.

Tensor conventions: activations torch.bfloat16 [M, K]; Q2_0 codes torch.uint8
[N, K/4]; scales, low-rank factors and 4-bit scales / zeros torch.float16;
outputs torch.float32, or torch.bfloat16 where a function takes out_dtype.  All
tensors must be contiguous and on the current device.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import NamedTuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# Q2_LIB names another build of the same library (for A/B measurements).
LIB_PATH = os.environ.get("Q2_LIB") or os.path.join(_HERE, "libq2.so")

Q2_OK, Q2_ERR_ARG, Q2_ERR_SHAPE, Q2_ERR_ALIGN, Q2_ERR_CODE, Q2_ERR_SCALE, Q2_ERR_DEVICE, Q2_ERR_HIP, \
    Q2_ERR_WORKSPACE, Q2_ERR_FORMAT = 0, -1, -2, -3, -4, -5, -6, -7, -8, -9

Q2_ACCUMULATE = 0x1      # q2_linear_ex flag: y += result

EXPORTS = ("q2_pack", "q2_import_gemlite", "q2_linear", "q2_lowrank_workspace_bytes", "q2_linear_lowrank", "q2_linear_lowrank_noalloc",
           "q2_linear_ex", "q2_slice",
           "q2_a8_workspace_bytes", "q2_linear_a8",
           "q2_linear_fused", "q2_linear_fused_workspace_bytes", "q4_linear_fused",
           "q2_linear_grouped", "q2_linear_grouped_workspace_bytes", "q4_linear_grouped",
           "q2_route", "q2_route_workspace_bytes", "q2_combine",
           "q4_linear", "q2_dequant", "q2_set_dispatch", "q2_strerror", "q2_last_error")

# q2_epilogue: activations by name, and flags
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
Q2_EPI_GATED, Q2_EPI_OUT_BF16, Q2_EPI_RESIDUAL_BF16 = 0x1, 0x2, 0x4
Q2_ROUTE_LOGITS_BF16, Q2_ROUTE_RENORM = 0x1, 0x2
Q2_COMBINE_Z_BF16, Q2_COMBINE_OUT_BF16, Q2_COMBINE_RESIDUAL_BF16 = 0x1, 0x2, 0x4


class Epilogue(ctypes.Structure):
    """The C ABI's q2_epilogue."""
    _fields_ = [("activation", ctypes.c_uint32), ("flags", ctypes.c_uint32), ("bias", ctypes.c_void_p),
                ("gate", ctypes.c_void_p), ("residual", ctypes.c_void_p)]


_lib = None


class Q2Error(RuntimeError):
    def __init__(self, status: int, message: str, bad_index: int = -1):
        super().__init__(message)
        self.status = status
        self.bad_index = bad_index


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load libq2.so (once) and declare the C signatures."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"libq2 is not built ({path} missing): run "
                           "`python -m ternary_weight_quantized_q2_amd.build_lib`")
    lib = ctypes.CDLL(path)
    p, i64, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
    sigs = {
        "q2_pack": ([p, p, i64, i64, p, p, ctypes.POINTER(ctypes.c_int64), p], ctypes.c_int),
        "q2_import_gemlite": ([p, p, p, i64, i64, i64, p, p, ctypes.POINTER(ctypes.c_int64), p], ctypes.c_int),
        "q2_linear": ([p, p, p, p, i64, i64, i64, p], ctypes.c_int),
        "q2_lowrank_workspace_bytes": ([i64, i64], sz),
        "q2_linear_lowrank": ([p, p, p, p, p, i64, p, i64, i64, i64, p, sz, p], ctypes.c_int),
        "q2_linear_lowrank_noalloc": ([p, p, p, p, p, i64, p, i64, i64, i64, p], ctypes.c_int),
        "q2_linear_ex": ([p, p, p, p, p, i64, p, i64, i64, i64, p, sz, ctypes.c_uint32, p], ctypes.c_int),
        "q2_slice": ([p, p, i64, i64, i64, i64, i64, i64, p, p, p], ctypes.c_int),
        "q2_a8_workspace_bytes": ([i64, i64], sz),
        "q2_linear_a8": ([p, p, p, p, i64, i64, i64, p, sz, p], ctypes.c_int),
        "q2_linear_fused": ([p, p, p, p, p, i64, p, p, i64, i64, i64, p, sz, p], ctypes.c_int),
        "q2_linear_fused_workspace_bytes": ([i64, i64, i64, i64], sz),
        "q4_linear_fused": ([p, p, p, p, p, p, i64, i64, i64, p], ctypes.c_int),
        "q2_linear_grouped": ([p, i64, p, p, p, p, p, p, i64, i64, i64, i64, p, sz, p], ctypes.c_int),
        "q2_linear_grouped_workspace_bytes": ([i64, i64, i64, i64], sz),
        "q4_linear_grouped": ([p, i64, p, p, p, p, p, p, p, i64, i64, i64, i64, p], ctypes.c_int),
        "q2_route": ([p, i64, i64, i64, ctypes.c_uint32, p, p, p, p, p, p, sz, p], ctypes.c_int),
        "q2_route_workspace_bytes": ([i64, i64, i64], sz),
        "q2_combine": ([p, i64, p, p, p, p, i64, i64, i64, ctypes.c_uint32, p], ctypes.c_int),
        "q4_linear": ([p, p, p, p, p, i64, i64, i64, p], ctypes.c_int),
        "q2_dequant": ([p, p, p, i64, i64, p], ctypes.c_int),
        "q2_set_dispatch": ([ctypes.c_char_p, ctypes.c_char_p, ctypes.c_int], ctypes.c_int),
        "q2_strerror": ([ctypes.c_int], ctypes.c_char_p),
        "q2_last_error": ([], ctypes.c_char_p),
    }
    for name, (args, res) in sigs.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = res
    _lib = lib
    return lib


def _check(status: int, bad_index: int = -1) -> None:
    if status != Q2_OK:
        lib = load()
        msg = f"{lib.q2_strerror(status).decode()}: {lib.q2_last_error().decode()}"
        raise Q2Error(status, msg, bad_index)


def _ptr(t) -> int | None:
    return None if t is None else (t.data_ptr() or None)


def _stream() -> int:
    # the current stream's handle, without building torch.cuda.current_stream()'s object (2.8 us of host time)
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _want(t: torch.Tensor, dtype: torch.dtype, shape: tuple, name: str) -> None:
    if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous():
        raise ValueError(f"{name}: expected contiguous {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
    if t.numel() and not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")


def q2_pack(codes: torch.Tensor, scales: torch.Tensor, packed=None, scales_f16=None):
    """codes u8 [N, K] in {0,1,2}, scales f32 [N, K/128] -> (packed u8 [N, K/4], scales f16 [N, K/128])."""
    lib = load()
    n, k = codes.shape
    _want(codes, torch.uint8, (n, k), "codes")
    _want(scales, torch.float32, (n, k // 128), "scales")
    dev = codes.device
    if packed is None:
        packed = torch.empty((n, k // 4), dtype=torch.uint8, device=dev)
    if scales_f16 is None:
        scales_f16 = torch.empty((n, k // 128), dtype=torch.float16, device=dev)
    bad = ctypes.c_int64(-1)
    st = lib.q2_pack(_ptr(codes), _ptr(scales), n, k, _ptr(packed), _ptr(scales_f16), ctypes.byref(bad), _stream())
    _check(st, bad.value)
    return packed, scales_f16


def q2_import_gemlite(codes_t, scales_t, zeros_t, group: int, packed=None, scales_f16=None):
    """Transposed group-quantised ternary weight -> Q2_0: codes_t u8 [K/4, N] (input-major),
    scales_t / zeros_t f32 [K/G, N] -> (packed u8 [N, K/4], scales f16 [N, K/128])."""
    lib = load()
    kq, n = codes_t.shape
    k = kq * 4
    _want(codes_t, torch.uint8, (kq, n), "codes_t")
    g = max(int(group), 1)
    _want(scales_t, torch.float32, (k // g, n), "scales_t")
    _want(zeros_t, torch.float32, (k // g, n), "zeros_t")
    dev = codes_t.device
    if packed is None:
        packed = torch.empty((n, kq), dtype=torch.uint8, device=dev)
    if scales_f16 is None:
        scales_f16 = torch.empty((n, k // 128), dtype=torch.float16, device=dev)
    bad = ctypes.c_int64(-1)
    st = lib.q2_import_gemlite(_ptr(codes_t), _ptr(scales_t), _ptr(zeros_t), n, k, int(group), _ptr(packed),
                               _ptr(scales_f16), ctypes.byref(bad), _stream())
    _check(st, bad.value)
    return packed, scales_f16


def q2_linear(x: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, y=None) -> torch.Tensor:
    """y [M, N] f32 = x W^T for Q2_0 weights (packed u8 [N, K/4], scales f16 [N, K/128])."""
    lib = load()
    m, k = x.shape
    n = packed.shape[0]
    _want(x, torch.bfloat16, (m, k), "x")
    _want(packed, torch.uint8, (n, k // 4), "packed")
    _want(scales, torch.float16, (n, k // 128), "scales")
    if y is None:
        y = torch.empty((m, n), dtype=torch.float32, device=x.device)
    _want(y, torch.float32, (m, n), "y")
    _check(lib.q2_linear(_ptr(x), _ptr(packed), _ptr(scales), _ptr(y), m, n, k, _stream()))
    return y


def lowrank_workspace_bytes(m: int, r: int) -> int:
    return int(load().q2_lowrank_workspace_bytes(m, r))


def q2_linear_lowrank(x, packed, scales, A, B, y=None, workspace=None) -> torch.Tensor:
    """y = x W^T + (x A^T) B^T; A f16 [r, K], B f16 [N, r]."""
    lib = load()
    m, k = x.shape
    n = packed.shape[0]
    r = A.shape[0]
    _want(x, torch.bfloat16, (m, k), "x")
    _want(packed, torch.uint8, (n, k // 4), "packed")
    _want(scales, torch.float16, (n, k // 128), "scales")
    _want(A, torch.float16, (r, k), "A")
    _want(B, torch.float16, (n, r), "B")
    if y is None:
        y = torch.empty((m, n), dtype=torch.float32, device=x.device)
    _want(y, torch.float32, (m, n), "y")
    need = lowrank_workspace_bytes(m, r)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    st = lib.q2_linear_lowrank(_ptr(x), _ptr(packed), _ptr(scales), _ptr(A), _ptr(B), r, _ptr(y), m, n, k,
                               _ptr(workspace), workspace.numel() * workspace.element_size(), _stream())
    _check(st)
    return y


NOALLOC_SCRATCH_BYTES = 8388608      # Q2_NOALLOC_SCRATCH_BYTES


def q2_linear_lowrank_noalloc(x, packed, scales, A, B, y=None) -> torch.Tensor:
    """q2_linear_lowrank with the library's per-device scratch instead of a workspace (no allocation in the
    library; y is allocated here only when not given)."""
    lib = load()
    m, k = x.shape
    n = packed.shape[0]
    r = A.shape[0]
    _want(x, torch.bfloat16, (m, k), "x")
    _want(packed, torch.uint8, (n, k // 4), "packed")
    _want(scales, torch.float16, (n, k // 128), "scales")
    _want(A, torch.float16, (r, k), "A")
    _want(B, torch.float16, (n, r), "B")
    if y is None:
        y = torch.empty((m, n), dtype=torch.float32, device=x.device)
    _want(y, torch.float32, (m, n), "y")
    _check(lib.q2_linear_lowrank_noalloc(_ptr(x), _ptr(packed), _ptr(scales), _ptr(A), _ptr(B), r, _ptr(y), m, n, k,
                                         _stream()))
    return y


def q2_linear_ex(x, packed, scales, y=None, A=None, B=None, accumulate=False, workspace=None) -> torch.Tensor:
    """q2_linear (A, B None) or q2_linear_lowrank with flags; accumulate=True adds the result into y,
    which must then be given."""
    lib = load()
    m, k = x.shape
    n = packed.shape[0]
    _want(x, torch.bfloat16, (m, k), "x")
    _want(packed, torch.uint8, (n, k // 4), "packed")
    _want(scales, torch.float16, (n, k // 128), "scales")
    if (A is None) != (B is None):
        raise ValueError("A and B come together")
    r = 0 if A is None else A.shape[0]
    if r:
        _want(A, torch.float16, (r, k), "A")
        _want(B, torch.float16, (n, r), "B")
    if y is None:
        if accumulate:
            raise ValueError("accumulate=True needs y")
        y = torch.empty((m, n), dtype=torch.float32, device=x.device)
    _want(y, torch.float32, (m, n), "y")
    ws_bytes = 0
    if r:
        need = lowrank_workspace_bytes(m, r)
        if workspace is None:
            workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
        ws_bytes = workspace.numel() * workspace.element_size()
    st = lib.q2_linear_ex(_ptr(x), _ptr(packed), _ptr(scales), _ptr(A), _ptr(B), r, _ptr(y), m, n, k,
                          _ptr(workspace), ws_bytes, Q2_ACCUMULATE if accumulate else 0, _stream())
    _check(st)
    return y


def q2_slice(packed, scales, n0: int, n1: int, k0: int, k1: int, out=None, out_scales=None):
    """Rows [n0, n1) and inputs [k0, k1) (multiples of 128) of a packed Q2_0 weight, as a new dense
    packed weight: (packed u8 [n1-n0, (k1-k0)/4], scales f16 [n1-n0, (k1-k0)/128])."""
    lib = load()
    n, kq = packed.shape
    k = kq * 4
    _want(packed, torch.uint8, (n, kq), "packed")
    _want(scales, torch.float16, (n, k // 128), "scales")
    rows, ks = max(n1 - n0, 0), max(k1 - k0, 0)
    dev = packed.device
    if out is None:
        out = torch.empty((rows, ks // 4), dtype=torch.uint8, device=dev)
    if out_scales is None:
        out_scales = torch.empty((rows, ks // 128), dtype=torch.float16, device=dev)
    _want(out, torch.uint8, (rows, ks // 4), "out")
    _want(out_scales, torch.float16, (rows, ks // 128), "out_scales")
    _check(lib.q2_slice(_ptr(packed), _ptr(scales), n, k, n0, n1, k0, k1, _ptr(out), _ptr(out_scales), _stream()))
    return out, out_scales


def a8_workspace_bytes(m: int, k: int) -> int:
    return int(load().q2_a8_workspace_bytes(m, k))


def q2_linear_a8(x, packed, scales, y=None, workspace=None) -> torch.Tensor:
    """y = s * (c W^T) with x quantised per row to 8-bit codes c and scales s (the codes and scales are left
    in the workspace: bf16 [M, K] at offset 0, f32 [M] after it, 256-byte aligned)."""
    lib = load()
    m, k = x.shape
    n = packed.shape[0]
    _want(x, torch.bfloat16, (m, k), "x")
    _want(packed, torch.uint8, (n, k // 4), "packed")
    _want(scales, torch.float16, (n, k // 128), "scales")
    if y is None:
        y = torch.empty((m, n), dtype=torch.float32, device=x.device)
    _want(y, torch.float32, (m, n), "y")
    need = a8_workspace_bytes(m, k)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=x.device)
    _check(lib.q2_linear_a8(_ptr(x), _ptr(packed), _ptr(scales), _ptr(y), m, n, k, _ptr(workspace),
                            workspace.numel() * workspace.element_size(), _stream()))
    return y


def q4_linear(x, packed4, scale, zero, y=None) -> torch.Tensor:
    """4-bit variant: packed4 u8 [N, K/2] (low nibble = even k), scale / zero f16 [N, K/128]."""
    lib = load()
    m, k = x.shape
    n = packed4.shape[0]
    _want(x, torch.bfloat16, (m, k), "x")
    _want(packed4, torch.uint8, (n, k // 2), "packed4")
    _want(scale, torch.float16, (n, k // 128), "scale")
    _want(zero, torch.float16, (n, k // 128), "zero")
    if y is None:
        y = torch.empty((m, n), dtype=torch.float32, device=x.device)
    _want(y, torch.float32, (m, n), "y")
    _check(lib.q4_linear(_ptr(x), _ptr(packed4), _ptr(scale), _ptr(zero), _ptr(y), m, n, k, _stream()))
    return y


def _here() -> int:
    """The current device, whose current stream the call goes to."""
    return torch.cuda.current_device()


def _have(t: torch.Tensor, dtype: torch.dtype, shape: tuple, name: str, dev: int) -> None:
    """_want, on device `dev`.  (These checks are most of a small call's host time: the common case is one test.)"""
    if t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous():
        return
    _want(t, dtype, shape, name)
    if t.is_cuda and t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, not on the current device cuda:{dev}")


def _maker(like: torch.Tensor, dev: int):
    """What allocates a call's outputs, on the device: an input without elements may be a host tensor.  (new_empty
    costs less host time.)"""
    return like.new_empty if like.is_cuda else functools.partial(torch.empty, device=f"cuda:{dev}")


def _epilogue(n, rows, bias_shape, bias, activation, gated, gate, residual, out_dtype, y, x, dev):
    """(q2_epilogue, y) of a fused or grouped linear over a weight of n rows; y is allocated when None."""
    if activation not in ACTIVATIONS:
        raise ValueError(f"unknown activation {activation!r}: one of {', '.join(ACTIVATIONS)}")
    if gated and n % 2:
        raise ValueError(f"a gated weight has two equal halves of rows, got {n} rows")
    if y is not None:
        out_dtype = y.dtype
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"the output is float32 or bfloat16, not {out_dtype}")
    shape = (rows, n // 2 if gated else n)
    flags = Q2_EPI_GATED if gated else 0
    if out_dtype == torch.bfloat16:
        flags |= Q2_EPI_OUT_BF16
    if bias is not None:
        _have(bias, torch.float32, bias_shape, "bias", dev)
    if gate is not None:
        _have(gate, torch.float32, shape[1:], "gate", dev)
    if residual is not None:
        if residual.dtype == torch.bfloat16:
            flags |= Q2_EPI_RESIDUAL_BF16
        elif residual.dtype != torch.float32:
            raise ValueError(f"residual is float32 or bfloat16, not {residual.dtype}")
        _have(residual, residual.dtype, shape, "residual", dev)
    if y is None:
        y = _maker(x, dev)(shape, dtype=out_dtype)
    else:
        _have(y, out_dtype, shape, "y", dev)
    return Epilogue(ACTIVATIONS[activation], flags, _ptr(bias), _ptr(gate), _ptr(residual)), y


def _scratch(need: int, workspace, dev: int):
    """(workspace, its bytes): the caller's, or a new one of `need` bytes."""
    if workspace is None:
        if need == 0:
            return None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=f"cuda:{dev}")
    else:
        _have(workspace, workspace.dtype, workspace.shape, "workspace", dev)
    return workspace, workspace.numel() * workspace.element_size()


def linear_fused_workspace_bytes(m: int, n: int, k: int, r: int = 0) -> int:
    """Workspace bytes of q2_linear_fused for a weight of n rows."""
    return int(load().q2_linear_fused_workspace_bytes(m, n, k, r))


def q2_linear_fused(x, packed, scales, A=None, B=None, bias=None, activation="none", gated=False, gate=None,
                    residual=None, out_dtype=torch.float32, y=None, workspace=None) -> torch.Tensor:
    """y = residual + gate * act(x W^T + (x A^T) B^T + bias) for Q2_0 weights, in float32 and rounded once to
    out_dtype (or y's type).

    gated: the weight holds the rows of two branches, [2 n, K], and act(first half) * second half has n columns.
    bias f32 [N]; gate f32 [n_out]; residual f32 or bf16 [M, n_out], which may be y itself; A f16 [r, K] and
    B f16 [N, r] add the rank-r branch.  activation: none, relu, gelu, gelu_tanh or silu."""
    lib = load()
    dev = _here()
    m, k = x.shape
    n = packed.shape[0]
    _have(x, torch.bfloat16, (m, k), "x", dev)
    _have(packed, torch.uint8, (n, k // 4), "packed", dev)
    _have(scales, torch.float16, (n, k // 128), "scales", dev)
    if (A is None) != (B is None):
        raise ValueError("A and B come together")
    r = 0 if A is None else A.shape[0]
    if A is not None:
        _have(A, torch.float16, (r, k), "A", dev)
        _have(B, torch.float16, (n, r), "B", dev)
    epi, y = _epilogue(n, m, (n,), bias, activation, gated, gate, residual, out_dtype, y, x, dev)
    ws, ws_bytes = _scratch(lib.q2_linear_fused_workspace_bytes(m, n, k, r), workspace, dev)
    _check(lib.q2_linear_fused(_ptr(x), _ptr(packed), _ptr(scales), _ptr(A), _ptr(B), r, ctypes.addressof(epi), _ptr(y),
                               m, n, k, _ptr(ws), ws_bytes, _stream()))
    return y


def q4_linear_fused(x, packed4, scale, zero, bias=None, activation="none", gated=False, gate=None, residual=None,
                    out_dtype=torch.float32, y=None) -> torch.Tensor:
    """q2_linear_fused (without the branch) for the 4-bit format of q4_linear."""
    lib = load()
    dev = _here()
    m, k = x.shape
    n = packed4.shape[0]
    _have(x, torch.bfloat16, (m, k), "x", dev)
    _have(packed4, torch.uint8, (n, k // 2), "packed4", dev)
    _have(scale, torch.float16, (n, k // 128), "scale", dev)
    _have(zero, torch.float16, (n, k // 128), "zero", dev)
    epi, y = _epilogue(n, m, (n,), bias, activation, gated, gate, residual, out_dtype, y, x, dev)
    _check(lib.q4_linear_fused(_ptr(x), _ptr(packed4), _ptr(scale), _ptr(zero), ctypes.addressof(epi), _ptr(y), m, n, k,
                               _stream()))
    return y


def _groups(x, offsets, experts, row_index, dev):
    """(rows, x_rows, K) of a grouped call, its integer arguments checked."""
    x_rows, k = x.shape
    _have(x, torch.bfloat16, (x_rows, k), "x", dev)
    _have(offsets, torch.int32, (experts + 1,), "offsets", dev)
    if row_index is None:
        return x_rows, x_rows, k
    rows = row_index.numel()
    _have(row_index, torch.int32, (rows,), "row_index", dev)
    return rows, x_rows, k


def linear_grouped_workspace_bytes(rows: int, experts: int, n: int, k: int) -> int:
    """Workspace bytes of q2_linear_grouped for `experts` weights of n rows."""
    return int(load().q2_linear_grouped_workspace_bytes(rows, experts, n, k))


def q2_linear_grouped(x, offsets, packed, scales, row_index=None, bias=None, activation="none", gated=False,
                      out_dtype=torch.float32, y=None, workspace=None) -> torch.Tensor:
    """Q2_0 linears of E experts over rows sorted by expert: row i in offsets[e] .. offsets[e+1] - 1 of y is
    act(x[row_index[i]] W_e^T + bias_e), or of x[i] without an index.

    packed u8 [E, N, K/4], scales f16 [E, N, K/128], offsets i32 [E+1] and row_index i32 [R] as q2_route gives
    them, bias f32 [E, N]; gated, activation and out_dtype as q2_linear_fused.  Rows that no expert has are left
    as they are in y (undefined in a y allocated here)."""
    lib = load()
    dev = _here()
    e, n = packed.shape[:2]
    rows, x_rows, k = _groups(x, offsets, e, row_index, dev)
    _have(packed, torch.uint8, (e, n, k // 4), "packed", dev)
    _have(scales, torch.float16, (e, n, k // 128), "scales", dev)
    epi, y = _epilogue(n, rows, (e, n), bias, activation, gated, None, None, out_dtype, y, x, dev)
    ws, ws_bytes = _scratch(lib.q2_linear_grouped_workspace_bytes(rows, e, n, k), workspace, dev)
    _check(lib.q2_linear_grouped(_ptr(x), x_rows, _ptr(row_index), _ptr(offsets), _ptr(packed), _ptr(scales),
                                 ctypes.addressof(epi), _ptr(y), rows, e, n, k, _ptr(ws), ws_bytes, _stream()))
    return y


def q4_linear_grouped(x, offsets, packed4, scale, zero, row_index=None, bias=None, activation="none", gated=False,
                      out_dtype=torch.float32, y=None) -> torch.Tensor:
    """q2_linear_grouped for the 4-bit format: packed4 u8 [E, N, K/2], scale and zero f16 [E, N, K/128]."""
    lib = load()
    dev = _here()
    e, n = packed4.shape[:2]
    rows, x_rows, k = _groups(x, offsets, e, row_index, dev)
    _have(packed4, torch.uint8, (e, n, k // 2), "packed4", dev)
    _have(scale, torch.float16, (e, n, k // 128), "scale", dev)
    _have(zero, torch.float16, (e, n, k // 128), "zero", dev)
    epi, y = _epilogue(n, rows, (e, n), bias, activation, gated, None, None, out_dtype, y, x, dev)
    _check(lib.q4_linear_grouped(_ptr(x), x_rows, _ptr(row_index), _ptr(offsets), _ptr(packed4), _ptr(scale), _ptr(zero),
                                 ctypes.addressof(epi), _ptr(y), rows, e, n, k, _stream()))
    return y


class Route(NamedTuple):
    """q2_route's choice and row plan."""
    expert: torch.Tensor      # i32 [T, k], -1 past the last unmasked expert
    weight: torch.Tensor      # f32 [T, k]
    offsets: torch.Tensor     # i32 [E + 1]: the rows of each expert
    row_token: torch.Tensor   # i32 [T k]: the token of each row, -1 behind the last row
    slot: torch.Tensor        # i32 [T, k]: the row of each choice, or -1


def q2_route(logits, k: int, renormalize: bool = True, workspace=None) -> Route:
    """Top-k routing of the tokens of logits [T, E] (f32 or bf16): the k largest per token (equal logits: the lower
    expert first; -inf and NaN are masked experts), their softmax weights over all unmasked experts or, with
    renormalize, over the chosen ones, and the rows sorted by expert, then token, as the grouped linears
    (offsets, row_token) and q2_combine (slot, weight) take them."""
    lib = load()
    dev = _here()
    t, e = logits.shape
    if logits.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"logits are float32 or bfloat16, not {logits.dtype}")
    _have(logits, logits.dtype, (t, e), "logits", dev)
    flags = (Q2_ROUTE_LOGITS_BF16 if logits.dtype == torch.bfloat16 else 0) | (Q2_ROUTE_RENORM if renormalize else 0)
    k = int(k)
    c = k if 0 < k <= e else 0                             # a refused k allocates nothing and reaches the library's message
    new, i32 = _maker(logits, dev), torch.int32
    expert = new((t, c), dtype=i32)
    route = Route(expert, new((t, c), dtype=torch.float32), new(e + 1, dtype=i32), new(t * c, dtype=i32),
                  torch.empty_like(expert))
    ws, ws_bytes = _scratch(lib.q2_route_workspace_bytes(t, e, k), workspace, dev)
    _check(lib.q2_route(_ptr(logits), t, e, k, flags, _ptr(route.expert), _ptr(route.weight), _ptr(route.offsets),
                        _ptr(route.row_token), _ptr(route.slot), _ptr(ws), ws_bytes, _stream()))
    return route


def q2_combine(z, slot, weight, residual=None, out_dtype=torch.float32, y=None) -> torch.Tensor:
    """y[t] = residual[t] + sum_j weight[t, j] * z[slot[t, j]]: the experts' rows z [R, N] (f32 or bf16) back on
    their tokens; slot i32 and weight f32 [T, k] as q2_route gives them, a slot outside [0, R) adds nothing;
    residual f32 or bf16 [T, N], which may be y itself."""
    lib = load()
    dev = _here()
    r, n = z.shape
    t, k = slot.shape
    if z.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"z is float32 or bfloat16, not {z.dtype}")
    _have(z, z.dtype, (r, n), "z", dev)
    _have(slot, torch.int32, (t, k), "slot", dev)
    _have(weight, torch.float32, (t, k), "weight", dev)
    if y is not None:
        out_dtype = y.dtype
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"the output is float32 or bfloat16, not {out_dtype}")
    flags = (Q2_COMBINE_Z_BF16 if z.dtype == torch.bfloat16 else 0) | \
        (Q2_COMBINE_OUT_BF16 if out_dtype == torch.bfloat16 else 0)
    if residual is not None:
        if residual.dtype == torch.bfloat16:
            flags |= Q2_COMBINE_RESIDUAL_BF16
        elif residual.dtype != torch.float32:
            raise ValueError(f"residual is float32 or bfloat16, not {residual.dtype}")
        _have(residual, residual.dtype, (t, n), "residual", dev)
    if y is None:
        y = _maker(z, dev)((t, n), dtype=out_dtype)
    else:
        _have(y, out_dtype, (t, n), "y", dev)
    _check(lib.q2_combine(_ptr(z), r, _ptr(slot), _ptr(weight), _ptr(residual), _ptr(y), t, k, n, flags, _stream()))
    return y


def q2_dequant(packed, scales, w=None) -> torch.Tensor:
    """Test export: float32 [N, K] weights (q - 1) * d."""
    lib = load()
    n, kq = packed.shape
    k = kq * 4
    _want(packed, torch.uint8, (n, kq), "packed")
    _want(scales, torch.float16, (n, k // 128), "scales")
    if w is None:
        w = torch.empty((n, k), dtype=torch.float32, device=packed.device)
    _check(lib.q2_dequant(_ptr(packed), _ptr(scales), _ptr(w), n, k, _stream()))
    return w


def set_dispatch(path: str | None = None, tile: str | None = None, ksplit: int = 0) -> None:
    """Test / profiling control of the launch choice for the whole process (q2_set_dispatch): path None,
    "auto", "gemv" or "gemm"; tile None or a GEMM configuration name; ksplit 0 (automatic), 1 or 2."""
    lib = load()
    _check(lib.q2_set_dispatch(None if path is None else path.encode(), None if tile is None else tile.encode(),
                               int(ksplit)))
