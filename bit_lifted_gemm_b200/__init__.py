"""Python binding of liblq.so, the C-ABI LiftQuant layer for B200 (sm_100a).

Argument marshalling only: every step of the layer runs in the library's
CUDA kernels. PyTorch supplies device memory and the current stream. There is
no fallback: if liblq.so is missing or cannot be loaded, import fails loudly.

    o = diag(s) . W_q . (blockdiag(M^T) . T^{-1} . a)

Entry points (same names as include/lq.h, minus the `lq_` prefix):
    lifted_dim, pack_signs, unpack_signs, lift_activations,
    lift_activations_kron, gemv_workspace_size, gemv, lift_gemv, gemm, encode,
    gemm_epilogue, gemv_epilogue, gemm_grouped, group_rows, combine_rows (and the
    workspace sizes of the first three), get_device_status
    (lq_selftest_wait_timeout is reached through `lib`)
"""

from __future__ import annotations

import contextlib
import ctypes
import functools
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
# LQ_DEBUG=1 selects the debug build (device-side bounds checks, LQ_ERR_BOUNDS)
DEBUG = os.environ.get("LQ_DEBUG", "") not in ("", "0")
LIB_PATH = os.path.join(_HERE, "liblq_debug.so" if DEBUG else "liblq.so")

LQ_OK, LQ_ERR_INVALID_ARG, LQ_ERR_UNSUPPORTED, LQ_ERR_CUDA, LQ_ERR_TIMEOUT, LQ_ERR_TOO_LARGE = 0, 1, 2, 3, 4, 5
LQ_ERR_BOUNDS = 6
LQ_F32, LQ_BF16 = 0, 1
ACTIVATIONS = {None: 0, "none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}  # lq_act
GEMV_NOALLOC_SCRATCH_BYTES = 4 << 20  # LQ_GEMV_NOALLOC_SCRATCH_BYTES of include/lq.h

SYMBOLS = ("lq_status_str", "lq_lifted_dim", "lq_pack_signs", "lq_unpack_signs", "lq_lift_activations",
           "lq_lift_activations_kron", "lq_gemv_workspace_size", "lq_gemv", "lq_gemv_noalloc", "lq_lift_gemv",
           "lq_gemm", "lq_gemm_epilogue", "lq_gemm_epilogue_workspace_size", "lq_gemv_epilogue",
           "lq_gemv_epilogue_workspace_size", "lq_gemm_grouped", "lq_gemm_grouped_workspace_size",
           "lq_gemm_grouped_in_order_workspace_size",
           "lq_group_rows", "lq_combine_rows", "lq_encode", "lq_selftest_wait_timeout", "lq_selftest_bounds", "lq_is_debug_build",
           "lq_get_device_status")


class LQError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_str(status)}")


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        how = "python bit_lifted_gemm_b200/build.py" + (" --debug" if DEBUG else "")
        raise ImportError(f"{os.path.basename(LIB_PATH)} not built at {LIB_PATH}; run `{how}`")
    lib = ctypes.CDLL(LIB_PATH)
    p, i = ctypes.c_void_p, ctypes.c_int
    lib.lq_status_str.restype = ctypes.c_char_p
    lib.lq_status_str.argtypes = [i]
    lib.lq_lifted_dim.restype = i
    lib.lq_lifted_dim.argtypes = [i, i, i]
    lib.lq_pack_signs.restype = i
    lib.lq_pack_signs.argtypes = [p, i, i, p, p]
    lib.lq_unpack_signs.restype = i
    lib.lq_unpack_signs.argtypes = [p, i, i, p, p]
    lib.lq_lift_activations.restype = i
    lib.lq_lift_activations.argtypes = [p, i, i, i, p, i, p, i, i, p, i, i, p]
    lib.lq_lift_activations_kron.restype = i
    lib.lq_lift_activations_kron.argtypes = [p, i, i, i, p, p, i, p, i, p, p, i, i, p, i, i, p]
    z = ctypes.c_size_t
    lib.lq_gemv_workspace_size.restype = z
    lib.lq_gemv_workspace_size.argtypes = [i, i, i]
    lib.lq_gemv.restype = i
    lib.lq_gemv.argtypes = [p, p, i, i, p, i, p, p, z, p]
    lib.lq_gemv_noalloc.restype = i
    lib.lq_gemv_noalloc.argtypes = [p, p, i, i, p, i, p, p]
    lib.lq_lift_gemv.restype = i
    lib.lq_lift_gemv.argtypes = [p, i, i, i, p, i, p, i, i, p, p, i, i, p, p, p, z, p]
    lib.lq_gemm.restype = i
    lib.lq_encode.restype = i
    lib.lq_selftest_wait_timeout.restype = i
    lib.lq_selftest_wait_timeout.argtypes = [ctypes.c_uint, p]
    lib.lq_selftest_bounds.restype = i
    lib.lq_selftest_bounds.argtypes = [p]
    lib.lq_is_debug_build.restype = i
    lib.lq_is_debug_build.argtypes = []
    lib.lq_encode.argtypes = [p, i, i, p, i, i, p, i, p, p]
    lib.lq_gemm.argtypes = [p, p, i, i, p, i, p, p]
    for name, argtypes in (("lq_gemm_epilogue_workspace_size", [i, i, i]), ("lq_gemv_epilogue_workspace_size", [i, i, i]),
                           ("lq_gemm_grouped_workspace_size", [i, i, i, i]),
                           ("lq_gemm_grouped_in_order_workspace_size", [i, i, i, i])):
        getattr(lib, name).restype = z
        getattr(lib, name).argtypes = argtypes
    layer = [p, p, i, i, p, i, p, i, i, p, p, i, p, z, p]
    for name, argtypes in (("lq_gemm_epilogue", layer), ("lq_gemv_epilogue", layer),
                           ("lq_gemm_grouped", [p, p, i, i, i, p, i, p, p, i, p, i, i, p, i, p, z, p]),
                           ("lq_group_rows", [p, i, i, i, p, p, p, p]),
                           ("lq_combine_rows", [p, i, i, i, p, p, i, i, p, p, p])):
        getattr(lib, name).restype = i
        getattr(lib, name).argtypes = argtypes
    lib.lq_get_device_status.restype = i
    lib.lq_get_device_status.argtypes = [p]
    return lib


lib = _load()


def status_str(status: int) -> str:
    return lib.lq_status_str(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != LQ_OK:
        raise LQError(status, where)


def lifted_dim(in_dim: int, d: int, D: int) -> int:
    return int(lib.lq_lifted_dim(in_dim, d, D))


# ------------------------------------------------------------------ torch helpers

def _stream(stream=None):
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _dev_tensor(t, name):
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    return t


def pack_signs(signs, out=None, stream=None):
    """int8 +-1 [out][K] (CUDA) -> packed words [out][K/32] (int32 storage of uint32)."""
    import torch
    _dev_tensor(signs, "signs")
    rows, K = signs.shape
    if out is None:
        out = torch.empty((rows, K // 32), dtype=torch.int32, device=signs.device)
    _check(lib.lq_pack_signs(_ptr(signs), rows, K, _ptr(out), _stream(stream)), "lq_pack_signs")
    return out


def unpack_signs(packed, K, out=None, stream=None):
    import torch
    _dev_tensor(packed, "packed")
    rows = packed.shape[0]
    if out is None:
        out = torch.empty((rows, K), dtype=torch.int8, device=packed.device)
    _check(lib.lq_unpack_signs(_ptr(packed), rows, K, _ptr(out), _stream(stream)), "lq_unpack_signs")
    return out


def lift_activations(a, M, K, tinv=None, u_dtype="f32", out=None, stream=None):
    """a [batch][in] (float32 or bfloat16) -> u [batch][K] (float32 or bfloat16)."""
    import torch
    _dev_tensor(a, "a")
    _dev_tensor(M, "M")
    batch, in_dim = a.shape
    d, D = M.shape
    a_t = LQ_BF16 if a.dtype == torch.bfloat16 else LQ_F32
    u_t = LQ_BF16 if u_dtype in ("bf16", torch.bfloat16) else LQ_F32
    if out is None:
        out = torch.empty((batch, K), dtype=torch.bfloat16 if u_t == LQ_BF16 else torch.float32, device=a.device)
    tblk = 0 if tinv is None else int(tinv.shape[-1])
    if tinv is not None:
        _dev_tensor(tinv, "tinv")
    _check(lib.lq_lift_activations(_ptr(a), a_t, batch, in_dim, _ptr(tinv), tblk, _ptr(M), d, D, _ptr(out), u_t,
                                   K, _stream(stream)), "lq_lift_activations")
    return out


def lift_activations_kron(a, q1, q2, M, K, r1=None, r2=None, u_dtype="f32", out=None, stream=None):
    """Lift with the Kronecker-factored whitening a' = diag(r2) (q1 kron q2) diag(r1) a.

    a [batch][in] (float32 or bfloat16), q1 [n1][n1], q2 [n2][n2] with in = n1 * n2,
    r1 [in] or None, r2 [in/d] or None -> u [batch][K] (float32 or bfloat16)."""
    import torch
    for t, name in ((a, "a"), (q1, "q1"), (q2, "q2"), (M, "M")):
        _dev_tensor(t, name)
    for t, name in ((r1, "r1"), (r2, "r2")):
        if t is not None:
            _dev_tensor(t, name)
    batch, in_dim = a.shape
    d, D = M.shape
    a_t = LQ_BF16 if a.dtype == torch.bfloat16 else LQ_F32
    u_t = LQ_BF16 if u_dtype in ("bf16", torch.bfloat16) else LQ_F32
    if out is None:
        out = torch.empty((batch, K), dtype=torch.bfloat16 if u_t == LQ_BF16 else torch.float32, device=a.device)
    _check(lib.lq_lift_activations_kron(_ptr(a), a_t, batch, in_dim, _ptr(r1), _ptr(q1), int(q1.shape[0]), _ptr(q2),
                                        int(q2.shape[0]), _ptr(r2), _ptr(M), d, D, _ptr(out), u_t, K,
                                        _stream(stream)), "lq_lift_activations_kron")
    return out


def gemv_workspace_size(out_rows: int, K: int, batch: int) -> int:
    """Bytes of device scratch lq_gemv / lq_lift_gemv need (0: shape not supported)."""
    return int(lib.lq_gemv_workspace_size(out_rows, K, batch))


def gemv_workspace(out_rows: int, K: int, batch: int, device=None):
    """A device scratch tensor big enough for lq_gemv / lq_lift_gemv on this shape
    (256-byte aligned: the caching allocator hands out 512-byte aligned blocks)."""
    import torch
    n = gemv_workspace_size(out_rows, K, batch)
    if n == 0:
        raise LQError(LQ_ERR_INVALID_ARG, "lq_gemv_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device if device is not None else "cuda")


def _workspace(ws, out_rows, K, batch, device):
    if ws is None:
        ws = gemv_workspace(out_rows, K, batch, device)
    _dev_tensor(ws, "workspace")
    return ws


def gemv(packed, s, u, out=None, workspace=None, stream=None):
    """Decode: packed [out][K/32], s [out], u fp32 [batch][K] (batch <= 16) -> o fp32 [batch][out].

    `workspace` (uint8 CUDA tensor of gemv_workspace_size bytes) is allocated
    when not given; calls that share one must run on the same stream."""
    import torch
    _dev_tensor(packed, "packed")
    _dev_tensor(s, "s")
    _dev_tensor(u, "u")
    rows = packed.shape[0]
    batch, K = u.shape
    if out is None:
        out = torch.empty((batch, rows), dtype=torch.float32, device=u.device)
    _dev_tensor(out, "out")
    ws = _workspace(workspace, rows, K, batch, u.device)
    _check(lib.lq_gemv(_ptr(packed), _ptr(s), rows, K, _ptr(u), batch, _ptr(out), _ptr(ws), ws.numel(),
                       _stream(stream)), "lq_gemv")
    return out


def _dev_or_pinned(t, name):
    if not t.is_contiguous() or not (t.is_cuda or t.is_pinned()):
        raise ValueError(f"{name} must be a contiguous CUDA tensor or pinned host tensor")
    return t


def lift_gemv(a, M, packed, s, K, tinv=None, u=None, out=None, workspace=None, stream=None):
    """Fused decode step: a [batch][in] (float32 or bfloat16) -> (u fp32 [batch][K], o fp32 [batch][out]).

    `a` and `out` may be pinned host tensors (zero-copy: the kernels read and
    write them across the host link); everything else lives on the device."""
    import torch
    _dev_or_pinned(a, "a")
    _dev_tensor(M, "M")
    _dev_tensor(packed, "packed")
    _dev_tensor(s, "s")
    batch, in_dim = a.shape
    d, D = M.shape
    rows = packed.shape[0]
    a_t = LQ_BF16 if a.dtype == torch.bfloat16 else LQ_F32
    if u is None:
        u = torch.empty((batch, K), dtype=torch.float32, device=M.device)
    if out is None:
        out = torch.empty((batch, rows), dtype=torch.float32, device=M.device)
    _dev_tensor(u, "u")
    _dev_or_pinned(out, "out")
    tblk = 0 if tinv is None else int(tinv.shape[-1])
    if tinv is not None:
        _dev_tensor(tinv, "tinv")
    ws = _workspace(workspace, rows, K, batch, M.device)
    _check(lib.lq_lift_gemv(_ptr(a), a_t, batch, in_dim, _ptr(tinv), tblk, _ptr(M), d, D, _ptr(packed), _ptr(s),
                            rows, K, _ptr(u), _ptr(out), _ptr(ws), ws.numel(), _stream(stream)), "lq_lift_gemv")
    return u, out


def gemm(packed, s, u, out=None, stream=None):
    """Prefill: packed [out][K/32], s [out], u bf16 [tokens][K] -> o fp32 [tokens][out]."""
    import torch
    _dev_tensor(packed, "packed")
    _dev_tensor(s, "s")
    _dev_tensor(u, "u")
    rows = packed.shape[0]
    tokens, K = u.shape
    if out is None:
        out = torch.empty((tokens, rows), dtype=torch.float32, device=u.device)
    _dev_tensor(out, "out")
    _check(lib.lq_gemm(_ptr(packed), _ptr(s), rows, K, _ptr(u), tokens, _ptr(out), _stream(stream)), "lq_gemm")
    return out


def encode(w, M, K, err=False, out=None, stream=None):
    """Encoder: weights w [rows][in] fp32, M [d][D] -> packed signs [rows][K/32]
    (int32 storage of uint32), and the per-block squared errors [rows][in/d] when
    err=True."""
    import torch
    _dev_tensor(w, "w")
    _dev_tensor(M, "M")
    rows, in_dim = w.shape
    d, D = M.shape
    if out is None:
        out = torch.empty((rows, K // 32), dtype=torch.int32, device=w.device)
    e = torch.empty((rows, in_dim // d), dtype=torch.float32, device=w.device) if err else None
    _check(lib.lq_encode(_ptr(w), rows, in_dim, _ptr(M), d, D, _ptr(out), K, _ptr(e), _stream(stream)), "lq_encode")
    return (out, e) if err else out


# ------------------------------------------------------------------ fused epilogues and grouped products
#
# At decode sizes the kernels take a few microseconds, so these calls keep their own work on
# the host small: plain comparisons, one allocation per output, addresses passed as integers.

def _on(t, stream):
    """Context in which `t`'s device is current, with `stream` (if given) as the
    current stream, so that what a call allocates belongs to the stream it runs on."""
    import torch
    if stream is not None:
        if stream.device != t.device:
            raise ValueError(f"stream is on {stream.device}, the tensors on {t.device}")
        return torch.cuda.stream(stream)
    if t.is_cuda and t.device.index != torch.cuda.current_device():
        return torch.cuda.device(t.device)
    return contextlib.nullcontext()


def _elsewhere(t, stream, name):
    """Whether a call on `t` has to enter another device or stream first (see _on)."""
    import torch
    if not t.is_cuda:
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    return stream is not None or t.get_device() != torch.cuda.current_device()


def _raw_stream(device):
    import torch
    return torch._C._cuda_getCurrentRawStream(device)


def _operand(t, name, dtype, shape, device):
    """Address of one operand: a contiguous tensor on CUDA device `device`, of this type and shape; None for None."""
    if t is None:
        return None
    if t.get_device() == device and t.dtype is dtype and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    raise ValueError(f"{name} must be {dtype} {tuple(shape)} on cuda:{device}, got {t.dtype} {tuple(t.shape)} on {t.device}")


def _result(t, name, dtype, shape, like):
    """(the output given, or a new one beside `like`; its address)."""
    if t is None:
        t = like.new_empty(shape, dtype=dtype)
        return t, t.data_ptr()
    return t, _operand(t, name, dtype, shape, like.get_device())


@functools.lru_cache(maxsize=None)
def _float_types():
    import torch
    f32, bf16 = (torch.float32, LQ_F32), (torch.bfloat16, LQ_BF16)
    return {"f32": f32, torch.float32: f32, "bf16": bf16, torch.bfloat16: bf16}


def _float_type(o_dtype, name="o_dtype"):
    found = _float_types().get(o_dtype)
    if found is None:
        raise ValueError(f"{name} must be 'f32' or 'bf16'")
    return found


def _activation(act):
    if act not in ACTIVATIONS:
        raise ValueError(f"act must be one of {sorted(k for k in ACTIVATIONS if k)} or None")
    return ACTIVATIONS[act]


_INT_MAX = 2 ** 31 - 1  # the C ABI's counts are ints, and ctypes drops the bits above without a word


def _counts(where, *counts):
    if max(counts) > _INT_MAX:
        raise LQError(LQ_ERR_INVALID_ARG, where)


def _fit(*counts):
    return -_INT_MAX <= min(counts) and max(counts) <= _INT_MAX


@functools.lru_cache(maxsize=1024)
def gemm_epilogue_workspace_size(out_rows: int, K: int, tokens: int) -> int:
    """Bytes of workspace gemm_epilogue needs (0: refused sizes)."""
    return 0 if not _fit(out_rows, K, tokens) else int(lib.lq_gemm_epilogue_workspace_size(out_rows, K, tokens))


@functools.lru_cache(maxsize=1024)
def gemv_epilogue_workspace_size(out_rows: int, K: int, batch: int) -> int:
    """Bytes of workspace gemv_epilogue needs (0: refused sizes)."""
    return 0 if not _fit(out_rows, K, batch) else int(lib.lq_gemv_epilogue_workspace_size(out_rows, K, batch))


@functools.lru_cache(maxsize=1024)
def gemm_grouped_workspace_size(experts: int, out_rows: int, K: int, n: int, rows: bool = True) -> int:
    """Bytes of workspace gemm_grouped needs, with or without `rows` (0: refused sizes)."""
    if not _fit(experts, out_rows, K, n):
        return 0
    size = lib.lq_gemm_grouped_workspace_size if rows else lib.lq_gemm_grouped_in_order_workspace_size
    return int(size(experts, out_rows, K, n))


def _scratch(ws, need, like):
    """(the workspace given, or a new one beside `like`; its bytes). The caching allocator aligns to 512 bytes."""
    import torch
    if ws is None:
        return like.new_empty(need or 1, dtype=torch.uint8), need or 1
    _dev_tensor(ws, "workspace")
    if ws.device != like.device:
        raise ValueError(f"workspace must be on {like.device}")
    return ws, ws.numel() * ws.element_size()


def _layer_epilogue(fn, size_fn, u_type, packed, s, u, bias, act, glu, residual, o_dtype, out, workspace, stream):
    import torch
    if u.dim() != 2 or packed.dim() != 2:
        raise ValueError("packed must be [out][K/32] and u [tokens][K]")
    tokens, K = u.shape
    rows = packed.shape[0]
    _counts(fn, tokens, K, rows)
    if _elsewhere(u, stream, "u"):
        with _on(u, stream):
            return _layer_epilogue(fn, size_fn, u_type, packed, s, u, bias, act, glu, residual, o_dtype, out, workspace,
                                   None)
    dev = u.get_device()
    ot, o_t = _float_type(o_dtype if out is None else out.dtype)
    width = rows // 2 if glu else rows
    out, o = _result(out, "out", ot, (tokens, width), u)
    ws, ws_bytes = _scratch(workspace, size_fn(rows, K, tokens), u)
    f32 = torch.float32
    _check(getattr(lib, fn)(_operand(packed, "packed", torch.int32, (rows, K // 32), dev), _operand(s, "s", f32, (rows,), dev),
                            rows, K, _operand(u, "u", u_type, (tokens, K), dev), tokens,
                            _operand(bias, "bias", f32, (rows,), dev), _activation(act), 1 if glu else 0,
                            _operand(residual, "residual", ot, (tokens, width), dev), o, o_t, ws.data_ptr(), ws_bytes,
                            _raw_stream(dev)), fn)
    return out


def gemm_epilogue(packed, s, u, bias=None, act=None, glu=False, residual=None, o_dtype="f32", out=None,
                  workspace=None, stream=None):
    """packed [out][K/32], s [out], u bf16 [tokens][K] -> o [tokens][width], o_dtype "f32" or "bf16".

    z = s * (W_q u) + bias; o = act(z) + residual with width = out, or with glu
    (rows 2i the gate's, rows 2i+1 the other factor's) o[i] = act(z[2i]) * z[2i+1] +
    residual[i] with width = out/2. act: None, "relu", "gelu", "gelu_tanh" or "silu";
    bias fp32 [out]; residual in o's type. `workspace` (gemm_epilogue_workspace_size
    bytes) is allocated when not given; calls that share one must be ordered."""
    import torch
    return _layer_epilogue("lq_gemm_epilogue", gemm_epilogue_workspace_size, torch.bfloat16, packed, s, u, bias, act,
                           glu, residual, o_dtype, out, workspace, stream)


def gemv_epilogue(packed, s, u, bias=None, act=None, glu=False, residual=None, o_dtype="f32", out=None,
                  workspace=None, stream=None):
    """gemm_epilogue for decode: u fp32 [batch][K], batch <= 16, at fp32 accuracy."""
    import torch
    return _layer_epilogue("lq_gemv_epilogue", gemv_epilogue_workspace_size, torch.float32, packed, s, u, bias, act,
                           glu, residual, o_dtype, out, workspace, stream)


def gemm_grouped(packed, s, u, offsets, n, rows=None, bias=None, act=None, glu=False, o_dtype="f32", out=None,
                 workspace=None, stream=None):
    """Products grouped by expert: packed [experts][out][K/32], s [experts][out], u bf16 [tokens][K],
    offsets int32 [experts+1], rows int32 [n] or None -> o [n][width].

    Slot i of expert e (offsets[e] <= i < offsets[e+1]) takes row rows[i] of u (row i
    without rows) through expert e's layer and the epilogue of gemm_epilogue (bias fp32
    [experts][out]). offsets and rows, as group_rows gives them, stay on the device.
    Slots of no expert are not written: uninitialized when `out` is allocated here."""
    import torch
    if u.dim() != 2 or packed.dim() != 3:
        raise ValueError("packed must be [experts][out][K/32] and u [tokens][K]")
    tokens, K = u.shape
    experts, out_rows = packed.shape[:2]
    n = int(n)
    _counts("lq_gemm_grouped", n, tokens, K, experts, out_rows)
    if _elsewhere(u, stream, "u"):
        with _on(u, stream):
            return gemm_grouped(packed, s, u, offsets, n, rows, bias, act, glu, o_dtype, out, workspace)
    dev = u.get_device()
    ot, o_t = _float_type(o_dtype if out is None else out.dtype)
    width = out_rows // 2 if glu else out_rows
    out, o = _result(out, "out", ot, (n, width), u)
    ws, ws_bytes = _scratch(workspace, gemm_grouped_workspace_size(experts, out_rows, K, n, rows is not None), u)
    f32, i32 = torch.float32, torch.int32
    _check(lib.lq_gemm_grouped(_operand(packed, "packed", i32, (experts, out_rows, K // 32), dev),
                               _operand(s, "s", f32, (experts, out_rows), dev), experts, out_rows, K,
                               _operand(u, "u", torch.bfloat16, (tokens, K), dev), tokens,
                               _operand(rows, "rows", i32, (n,), dev), _operand(offsets, "offsets", i32, (experts + 1,), dev),
                               n, _operand(bias, "bias", f32, (experts, out_rows), dev), _activation(act), 1 if glu else 0,
                               o, o_t, ws.data_ptr(), ws_bytes, _raw_stream(dev)), "lq_gemm_grouped")
    return out


def group_rows(expert_ids, experts, offsets=None, rows=None, slots=None, stream=None):
    """Router choices int32 [tokens][topk] -> (offsets int32 [experts+1], rows int32 [tokens*topk],
    slots int32 [tokens][topk]): expert e's slots are [offsets[e], offsets[e+1]) in (token, choice)
    order, rows the token of each slot (-1 past the last), slots the slot of each choice (-1 for
    ids outside 0..experts-1)."""
    import torch
    if expert_ids.dim() != 2:
        raise ValueError("expert_ids must be [tokens][topk]")
    tokens, topk = expert_ids.shape
    _counts("lq_group_rows", tokens, topk, experts)
    if _elsewhere(expert_ids, stream, "expert_ids"):
        with _on(expert_ids, stream):
            return group_rows(expert_ids, experts, offsets, rows, slots)
    dev, i32 = expert_ids.get_device(), torch.int32
    offsets, offsets_at = _result(offsets, "offsets", i32, (experts + 1,), expert_ids)
    rows, rows_at = _result(rows, "rows", i32, (tokens * topk,), expert_ids)
    slots, slots_at = _result(slots, "slots", i32, (tokens, topk), expert_ids)
    _check(lib.lq_group_rows(_operand(expert_ids, "expert_ids", i32, (tokens, topk), dev), tokens, topk, experts,
                             offsets_at, rows_at, slots_at, _raw_stream(dev)), "lq_group_rows")
    return offsets, rows, slots


def combine_rows(y, slots, weights, residual=None, out=None, stream=None):
    """o[t] = residual[t] + sum_j weights[t][j] * y[slots[t][j]]: y [n][width] (float32 or bfloat16), slots
    int32 [tokens][topk] (values outside 0..n-1 add nothing), weights fp32 [tokens][topk], residual and o
    [tokens][width] in y's type."""
    import torch
    if y.dim() != 2 or slots.dim() != 2:
        raise ValueError("y must be [n][width] and slots [tokens][topk]")
    n, width = y.shape
    tokens, topk = slots.shape
    _counts("lq_combine_rows", n, width, tokens, topk)
    if _elsewhere(y, stream, "y"):
        with _on(y, stream):
            return combine_rows(y, slots, weights, residual, out)
    dev = y.get_device()
    yt, y_t = _float_type(y.dtype, "y's type")
    out, o = _result(out, "out", yt, (tokens, width), y)
    _check(lib.lq_combine_rows(_operand(y, "y", yt, (n, width), dev), y_t, n, width,
                               _operand(slots, "slots", torch.int32, (tokens, topk), dev),
                               _operand(weights, "weights", torch.float32, (tokens, topk), dev), tokens, topk,
                               _operand(residual, "residual", yt, (tokens, width), dev), o, _raw_stream(dev)),
           "lq_combine_rows")
    return out


def get_device_status(stream=None) -> int:
    return int(lib.lq_get_device_status(_stream(stream)))
