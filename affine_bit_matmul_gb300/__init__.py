"""affine_bit_matmul_gb300 — affine group-wise quantized matmul on GB300.

A thin Python binding over the C ABI of ``libmxq.so`` (declared in
``include/mxq.h``).  Every step of the computation runs in the library's
sm_103a kernels; this module only checks tensors, passes their device
pointers and the current CUDA stream, and turns status codes into
exceptions.  There is no fallback: if the library is missing or the device
is not sm_103a, the calls raise.

Storage conventions (mlxcel issue #1536, Baseline section: "affine 4-bit /
group 64"):

* ``x``: bf16 ``[M, K]`` (``[K]`` for ``qmv``);
* ``w``: int32 or uint32 ``[N, K*bits/32]`` packed codes, 4-bit codes eight per
  little-endian word (lowest k in the lowest nibble), 2-bit codes sixteen per
  word, 8-bit codes four per word; 3- and 6-bit codes continue the same
  little-endian bit stream per row and may straddle words (``bits`` in 2, 3,
  4, 6, 8);
* ``scales``, ``biases``: bf16 ``[N, K/group_size]``, one pair per group of
  ``group_size`` consecutive k (32, 64 or 128; every call defaults to 64);
* result ``y``: bf16 ``[M, N]``.
"""

from __future__ import annotations

import ctypes
import importlib
import os

__all__ = [
    "lib",
    "qmv",
    "qmm",
    "qmv_kn",
    "qmm_kn",
    "gather_qmm",
    "gather_qmm_kn",
    "gather_qmm_gateup",
    "gather_workspace_bytes",
    "gather_qmm_noalloc",
    "quantize",
    "qk_norm_rope",
    "rope_inv_freq",
    "kv_block_bytes",
    "kv_append",
    "kv_read",
    "kv_attention",
    "kv_attention_workspace_bytes",
    "kv_attention_shared",
    "kv_attention_shared_workspace_bytes",
    "beam_select",
    "kv_reorder",
    "set_wait_budget",
    "NOALLOC_SCRATCH_BYTES",
    "MxqError",
    "DEV_BAD_EXPERT_ID",
    "DEV_UNSORTED_IDS",
    "DEV_BAD_ROW_SRC",
    "DEV_TIMEOUT",
    "DEV_BAD_SLOT",
    "DEV_BAD_PAGE",
    "DEV_BAD_SEQUENCE",
    "EXPORTED_SYMBOLS",
]

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmxq.so")

MXQ_OK = 0
STATUS_NAMES = {
    0: "MXQ_OK",
    1: "MXQ_ERR_INVALID_ARG",
    2: "MXQ_ERR_MISALIGNED",
    3: "MXQ_ERR_UNSUPPORTED",
    4: "MXQ_ERR_ARCH",
    5: "MXQ_ERR_CUDA",
    6: "MXQ_ERR_WORKSPACE",
    7: "MXQ_ERR_SCRATCH_LIMIT",
}
DEV_BAD_EXPERT_ID = 0x1
DEV_UNSORTED_IDS = 0x2
DEV_BAD_ROW_SRC = 0x4
DEV_TIMEOUT = 0x8
DEV_BAD_SLOT = 0x10
DEV_BAD_PAGE = 0x20
DEV_BAD_SEQUENCE = 0x40
NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024  # MXQ_NOALLOC_SCRATCH_BYTES

EXPORTED_SYMBOLS = (
    "mxq_qmv",
    "mxq_qmm",
    "mxq_qmv_kn",
    "mxq_qmm_kn",
    "mxq_gather_qmm",
    "mxq_gather_qmm_kn",
    "mxq_gather_qmm_gateup",
    "mxq_gather_workspace_bytes",
    "mxq_gather_qmm_noalloc",
    "mxq_quantize",
    "mxq_qk_norm_rope",
    "mxq_kv_block_bytes",
    "mxq_kv_append",
    "mxq_kv_read",
    "mxq_kv_attention",
    "mxq_kv_attention_workspace_bytes",
    "mxq_kv_attention_shared",
    "mxq_kv_attention_shared_workspace_bytes",
    "mxq_beam_select",
    "mxq_beam_select_workspace_bytes",
    "mxq_kv_reorder",
    "mxq_kv_reorder_workspace_bytes",
    "mxq_status_string",
    "mxq_version",
    "mxq_debug_set_wait_budget",
)


class MxqError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__("%s: %s (%s)" % (what, STATUS_NAMES.get(status, status),
                                           _status_string(status)))


_lib_handle = None


def lib():
    """The loaded ``libmxq.so`` with argument types set (raises if absent)."""
    global _lib_handle
    if _lib_handle is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                "libmxq.so is not built; run affine_bit_matmul_gb300.build.build() "
                "(needs nvcc) before using the library")
        L = ctypes.CDLL(LIB_PATH)
        P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        L.mxq_qmv.argtypes = [P, P, P, P, P, I, I, I, I, P, P]
        L.mxq_qmv.restype = I
        L.mxq_qmm.argtypes = [P, P, P, P, P, I, I, I, I, I, P, P]
        L.mxq_qmm.restype = I
        L.mxq_qmv_kn.argtypes = [P, P, P, P, P, I, I, I, I, P, P]
        L.mxq_qmv_kn.restype = I
        L.mxq_qmm_kn.argtypes = [P, P, P, P, P, I, I, I, I, I, P, P]
        L.mxq_qmm_kn.restype = I
        L.mxq_gather_qmm.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, I, P, Z, P, P]
        L.mxq_gather_qmm.restype = I
        L.mxq_gather_qmm_kn.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, I, P, Z, P, P]
        L.mxq_gather_qmm_kn.restype = I
        L.mxq_gather_qmm_gateup.argtypes = [P, P, P, P, P, P, P, P, P, P, P, I, I, I, I, I, I,
                                             I, P, Z, P, P]
        L.mxq_gather_qmm_gateup.restype = I
        L.mxq_gather_qmm_noalloc.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, I, P, P]
        L.mxq_gather_qmm_noalloc.restype = I
        L.mxq_quantize.argtypes = [P, P, P, P, I, I, I, I, P]
        L.mxq_quantize.restype = I
        J, F = ctypes.c_longlong, ctypes.c_float
        L.mxq_qk_norm_rope.argtypes = [P, J, J, P, J, J, P, P, P, P, P, J, J, P, J, J, I, I, I, I,
                                       I, I, F, F, F, P]
        L.mxq_qk_norm_rope.restype = I
        L.mxq_kv_block_bytes.argtypes = [I, I, I]
        L.mxq_kv_block_bytes.restype = Z
        L.mxq_kv_append.argtypes = [P, J, J, P, J, J, P, P, I, I, I, I, I, I, P, P]
        L.mxq_kv_append.restype = I
        L.mxq_kv_read.argtypes = [P, P, P, P, I, I, I, I, I, I, P, P]
        L.mxq_kv_read.restype = I
        L.mxq_kv_attention.argtypes = [P, J, J, P, P, P, P, P, P, I, I, I, I, I, I, I, I, I, I, F,
                                       I, I, P, Z, P, P]
        L.mxq_kv_attention.restype = I
        L.mxq_kv_attention_workspace_bytes.argtypes = [I, I, I, I, I, I]
        L.mxq_kv_attention_workspace_bytes.restype = Z
        L.mxq_kv_attention_shared.argtypes = [P, J, J] + [P] * 9 + [I] * 13 + [F, P, Z, P, P]
        L.mxq_kv_attention_shared.restype = I
        L.mxq_kv_attention_shared_workspace_bytes.argtypes = [I] * 8
        L.mxq_kv_attention_shared_workspace_bytes.restype = Z
        L.mxq_beam_select.argtypes = [P, J, I, P, P, P, P, P, P, I, I, I, I, I, P, Z, P]
        L.mxq_beam_select.restype = I
        L.mxq_beam_select_workspace_bytes.argtypes = [I] * 5
        L.mxq_beam_select_workspace_bytes.restype = Z
        L.mxq_kv_reorder.argtypes = [P] * 7 + [I] * 9 + [P, Z, P, P]
        L.mxq_kv_reorder.restype = I
        L.mxq_kv_reorder_workspace_bytes.argtypes = [I]
        L.mxq_kv_reorder_workspace_bytes.restype = Z
        L.mxq_gather_workspace_bytes.argtypes = [I, I, I, I]
        L.mxq_gather_workspace_bytes.restype = Z
        L.mxq_status_string.argtypes = [I]
        L.mxq_status_string.restype = ctypes.c_char_p
        L.mxq_version.restype = I
        L.mxq_debug_set_wait_budget.argtypes = [ctypes.c_longlong]
        L.mxq_debug_set_wait_budget.restype = ctypes.c_longlong
        _lib_handle = L
    return _lib_handle


_calls_module = None


def _direct():
    """The module that reads and checks the cache operators' tensors (``csrc/torch_calls.cpp``),
    with the library's functions; raises if it is not built."""
    global _calls_module
    if _calls_module is None:
        L = lib()
        _torch()
        try:
            module = importlib.import_module("._calls", __name__)
        except ImportError as e:
            raise RuntimeError("_calls.so is not built, or not for this Python and torch (%s); run "
                               "affine_bit_matmul_gb300.build.build() before using the cache "
                               "operators" % e) from e
        module.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
            L.mxq_qk_norm_rope, L.mxq_kv_append, L.mxq_kv_read, L.mxq_kv_attention,
            L.mxq_kv_attention_workspace_bytes, L.mxq_kv_attention_shared,
            L.mxq_kv_attention_shared_workspace_bytes, L.mxq_beam_select, L.mxq_beam_select_workspace_bytes,
            L.mxq_kv_reorder, L.mxq_kv_reorder_workspace_bytes)))
        _calls_module = module
    return _calls_module


def _status_string(status: int) -> str:
    try:
        return lib().mxq_status_string(status).decode()
    except Exception:  # library not loadable: name only
        return STATUS_NAMES.get(status, "unknown")


def _check(status: int, what: str):
    if status != MXQ_OK:
        raise MxqError(status, what)


# ---------------------------------------------------------------- torch level

_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch

        _torch_module = torch
    return _torch_module


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None else None


class _Here:
    """A context that does nothing: the tensors' device is the current one."""

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        return False


_HERE_CTX = _Here()


def _launch_on(device, stream):
    """The device context and raw stream handle for a call on ``device``.

    The library launches on the CUDA device that is current when it is
    called, so every wrapper makes the tensors' device current for the call
    (nothing is to be done where it is); ``stream`` (default: that device's
    current stream) must belong to the same device, else the launch would pair
    one device's pointers with another device's stream."""
    torch = _torch()
    if stream is None:
        handle = torch._C._cuda_getCurrentRawStream(device.index)
    elif stream.device != device:
        raise ValueError("stream is on %s but the tensors are on %s" % (stream.device, device))
    else:
        handle = stream.cuda_stream
    if torch._C._cuda_getDevice() == device.index:
        return _HERE_CTX, handle
    return torch.cuda.device(device), handle


def _require(t, name, dtypes, device=None):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dtype not in dtypes:
        raise TypeError("%s has dtype %s, expected one of %s" % (name, t.dtype, dtypes))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))


def _code_dtypes():
    torch = _torch()
    out = [torch.int32]
    if hasattr(torch, "uint32"):
        out.append(torch.uint32)
    return tuple(out)


def _check_weights(w, scales, biases, N, K, bits, device, lead=(), group_size=64):
    torch = _torch()
    _require(w, "w", _code_dtypes(), device)
    _require(scales, "scales", (torch.bfloat16,), device)
    _require(biases, "biases", (torch.bfloat16,), device)
    if tuple(w.shape) != tuple(lead) + (N, K * bits // 32):
        raise ValueError("w has shape %s, expected %s" % (tuple(w.shape), tuple(lead) + (N, K * bits // 32)))
    if group_size <= 0:
        raise ValueError("group_size must be positive")
    for t, name in ((scales, "scales"), (biases, "biases")):
        if tuple(t.shape) != tuple(lead) + (N, K // group_size):
            raise ValueError("%s has shape %s, expected %s" % (
                name, tuple(t.shape), tuple(lead) + (N, K // group_size)))


def qmv(x, w, scales, biases, bits: int, out=None, dev_status=None, stream=None,
        group_size: int = 64):
    """Decode GEMV: ``y[N] = sum_k x[k] * (s*q + b)[n, k]`` (``x`` bf16 [K]).
    ``dev_status`` (CUDA int32 [1]) receives DEV_TIMEOUT if a wait gave up."""
    torch = _torch()
    _require(x, "x", (torch.bfloat16,))
    if x.dim() != 1:
        raise ValueError("x must be 1-D [K]")
    K = x.shape[0]
    N = w.shape[0]
    _check_weights(w, scales, biases, N, K, bits, x.device, group_size=group_size)
    if out is None:
        out = torch.empty((N,), dtype=torch.bfloat16, device=x.device)
    _require(out, "out", (torch.bfloat16,), x.device)
    if dev_status is not None:
        _require(dev_status, "dev_status", (torch.int32,), x.device)
    ctx, st = _launch_on(x.device, stream)
    with ctx:
        _check(lib().mxq_qmv(_ptr(x), _ptr(w), _ptr(scales), _ptr(biases), _ptr(out), K, N, bits,
                             group_size, _ptr(dev_status), st), "mxq_qmv")
    return out


def qmv_kn(x, w, scales, biases, bits: int, out=None, dev_status=None, stream=None,
           group_size: int = 64):
    """Decode GEMV with w stored [K, N] (codes and groups along n):
    ``y[n] = sum_k x[k] * (s[k, n/G] q[k, n] + b[k, n/G])``; ``w`` int32
    [K, N*bits/32], ``scales``/``biases`` bf16 [K, N/G], ``x`` bf16 [K]."""
    torch = _torch()
    _require(x, "x", (torch.bfloat16,))
    if x.dim() != 1:
        raise ValueError("x must be 1-D [K]")
    K = x.shape[0]
    _require(w, "w", _code_dtypes(), x.device)
    _require(scales, "scales", (torch.bfloat16,), x.device)
    _require(biases, "biases", (torch.bfloat16,), x.device)
    if w.dim() != 2 or w.shape[0] != K:
        raise ValueError("w must be [K, N*bits/32]")
    N = w.shape[1] * 32 // bits
    if group_size <= 0:
        raise ValueError("group_size must be positive")
    for t, name in ((scales, "scales"), (biases, "biases")):
        if tuple(t.shape) != (K, N // group_size):
            raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape),
                                                               (K, N // group_size)))
    if out is None:
        out = torch.empty((N,), dtype=torch.bfloat16, device=x.device)
    _require(out, "out", (torch.bfloat16,), x.device)
    if dev_status is not None:
        _require(dev_status, "dev_status", (torch.int32,), x.device)
    ctx, st = _launch_on(x.device, stream)
    with ctx:
        _check(lib().mxq_qmv_kn(_ptr(x), _ptr(w), _ptr(scales), _ptr(biases), _ptr(out), K, N,
                                bits, group_size, _ptr(dev_status), st), "mxq_qmv_kn")
    return out


def qmm(x, w, scales, biases, bits: int, out=None, dev_status=None, stream=None,
        group_size: int = 64):
    """Prefill GEMM on the tensor cores: ``y[M, N] = x[M, K] . w^[N, K]^T``.

    ``dev_status`` (CUDA int32 [1]) receives DEV_TIMEOUT if a pipeline wait
    gave up.
    """
    torch = _torch()
    _require(x, "x", (torch.bfloat16,))
    if x.dim() != 2:
        raise ValueError("x must be 2-D [M, K]")
    M, K = x.shape
    N = w.shape[0]
    _check_weights(w, scales, biases, N, K, bits, x.device, group_size=group_size)
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    _require(out, "out", (torch.bfloat16,), x.device)
    if dev_status is not None:
        _require(dev_status, "dev_status", (torch.int32,), x.device)
    ctx, st = _launch_on(x.device, stream)
    with ctx:
        _check(lib().mxq_qmm(_ptr(x), _ptr(w), _ptr(scales), _ptr(biases), _ptr(out), M, K, N,
                             bits, group_size, _ptr(dev_status), st), "mxq_qmm")
    return out


def _check_weights_kn(w, scales, biases, K, N, bits, device, lead=(), group_size=64):
    """[K, N]-layout weights: ``w`` int32 [..., K, N*bits/32], ``scales`` and
    ``biases`` bf16 [..., K, N/G]."""
    torch = _torch()
    _require(w, "w", _code_dtypes(), device)
    _require(scales, "scales", (torch.bfloat16,), device)
    _require(biases, "biases", (torch.bfloat16,), device)
    if group_size <= 0:
        raise ValueError("group_size must be positive")
    if tuple(w.shape) != tuple(lead) + (K, N * bits // 32):
        raise ValueError("w has shape %s, expected %s" % (tuple(w.shape),
                                                          tuple(lead) + (K, N * bits // 32)))
    for t, name in ((scales, "scales"), (biases, "biases")):
        if tuple(t.shape) != tuple(lead) + (K, N // group_size):
            raise ValueError("%s has shape %s, expected %s" % (
                name, tuple(t.shape), tuple(lead) + (K, N // group_size)))


def qmm_kn(x, w, scales, biases, bits: int, out=None, dev_status=None, stream=None,
           group_size: int = 64):
    """Prefill GEMM with w stored [K, N] (codes and groups along n):
    ``y[m, n] = sum_k x[m, k] (s[k, n/G] q[k, n] + b[k, n/G])``; ``x`` bf16
    [M, K], ``w`` int32 [K, N*bits/32], ``scales``/``biases`` bf16 [K, N/G]."""
    torch = _torch()
    _require(x, "x", (torch.bfloat16,))
    if x.dim() != 2:
        raise ValueError("x must be 2-D [M, K]")
    M, K = x.shape
    if w.dim() != 2:
        raise ValueError("w must be [K, N*bits/32]")
    N = w.shape[1] * 32 // bits
    _check_weights_kn(w, scales, biases, K, N, bits, x.device, group_size=group_size)
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    _require(out, "out", (torch.bfloat16,), x.device)
    if tuple(out.shape) != (M, N):
        raise ValueError("out has shape %s, expected %s" % (tuple(out.shape), (M, N)))
    if dev_status is not None:
        _require(dev_status, "dev_status", (torch.int32,), x.device)
    ctx, st = _launch_on(x.device, stream)
    with ctx:
        _check(lib().mxq_qmm_kn(_ptr(x), _ptr(w), _ptr(scales), _ptr(biases), _ptr(out), M, K, N,
                                bits, group_size, _ptr(dev_status), st), "mxq_qmm_kn")
    return out


def gather_qmm_kn(x, w, scales, biases, expert_ids, row_src, bits: int, out=None, workspace=None,
                  dev_status=None, stream=None, group_size: int = 64):
    """Sorted mixture-of-experts GEMM with each expert's w stored [K, N]:
    ``w`` int32 [E, K, N*bits/32], ``scales``/``biases`` bf16 [E, K, N/G];
    sorted row r multiplies ``x[row_src[r]]`` by expert ``expert_ids[r]``."""
    torch = _torch()
    _require(x, "x", (torch.bfloat16,))
    if x.dim() != 2:
        raise ValueError("x must be 2-D [T, K]")
    T, K = x.shape
    if w.dim() != 3:
        raise ValueError("w must be [E, K, N*bits/32]")
    E = w.shape[0]
    N = w.shape[2] * 32 // bits
    _check_weights_kn(w, scales, biases, K, N, bits, x.device, lead=(E,), group_size=group_size)
    _require(expert_ids, "expert_ids", (torch.int32,), x.device)
    B = expert_ids.numel()
    if row_src is not None:
        _require(row_src, "row_src", (torch.int32,), x.device)
        if row_src.numel() != B:
            raise ValueError("row_src must have B entries")
    if out is None:
        out = torch.empty((B, N), dtype=torch.bfloat16, device=x.device)
    _require(out, "out", (torch.bfloat16,), x.device)
    if tuple(out.shape) != (B, N):
        raise ValueError("out has shape %s, expected %s" % (tuple(out.shape), (B, N)))
    if workspace is None:
        workspace = torch.empty((gather_workspace_bytes(B, E, K if row_src is not None else 0, N),),
                                dtype=torch.uint8, device=x.device)
    _require(workspace, "workspace", (torch.uint8,), x.device)
    if dev_status is not None:
        _require(dev_status, "dev_status", (torch.int32,), x.device)
    ctx, st = _launch_on(x.device, stream)
    with ctx:
        _check(lib().mxq_gather_qmm_kn(
            _ptr(x), _ptr(w), _ptr(scales), _ptr(biases), _ptr(expert_ids), _ptr(row_src),
            _ptr(out), T, B, E, K, N, bits, group_size, _ptr(workspace), workspace.numel(),
            _ptr(dev_status), st), "mxq_gather_qmm_kn")
    return out


def quantize(w, bits: int, codes=None, scales=None, biases=None, stream=None,
             group_size: int = 64):
    """Affine group-wise encoder on the GPU: float32 ``w`` [N, K] -> (codes
    int32 [N, K*bits/32], scales bf16 [N, K/G], biases bf16 [N, K/G]),
    G = ``group_size``."""
    torch = _torch()
    _require(w, "w", (torch.float32,))
    if w.dim() != 2:
        raise ValueError("w must be 2-D [N, K]")
    N, K = w.shape
    dev = w.device
    if codes is None:
        codes = torch.empty((N, K * bits // 32), dtype=torch.int32, device=dev)
    if group_size <= 0:
        raise ValueError("group_size must be positive")
    if scales is None:
        scales = torch.empty((N, K // group_size), dtype=torch.bfloat16, device=dev)
    if biases is None:
        biases = torch.empty((N, K // group_size), dtype=torch.bfloat16, device=dev)
    _check_weights(codes, scales, biases, N, K, bits, dev, group_size=group_size)
    ctx, st = _launch_on(dev, stream)
    with ctx:
        _check(lib().mxq_quantize(_ptr(w), _ptr(codes), _ptr(scales), _ptr(biases), N, K, bits,
                                  group_size, st), "mxq_quantize")
    return codes, scales, biases


def gather_workspace_bytes(B: int, E: int, K: int, N: int) -> int:
    """Workspace bytes for gather_qmm and gather_qmm_gateup; pass K = 0 when
    row_src is None."""
    return int(lib().mxq_gather_workspace_bytes(B, E, K, N))


def gather_qmm_noalloc(x, w, scales, biases, expert_ids, row_src, bits: int, out,
                       dev_status=None, stream=None, group_size: int = 64):
    """gather_qmm without any allocation: ``out`` must be given, and the
    scratch is the library's fixed MXQ_NOALLOC_SCRATCH_BYTES array (calls on
    one device must not overlap in time; see include/mxq.h)."""
    torch = _torch()
    _require(x, "x", (torch.bfloat16,))
    if x.dim() != 2:
        raise ValueError("x must be 2-D [T, K]")
    T, K = x.shape
    if w.dim() != 3:
        raise ValueError("w must be 3-D [E, N, K*bits/32]")
    E, N = w.shape[0], w.shape[1]
    _check_weights(w, scales, biases, N, K, bits, x.device, lead=(E,), group_size=group_size)
    _require(expert_ids, "expert_ids", (torch.int32,), x.device)
    B = expert_ids.numel()
    if row_src is not None:
        _require(row_src, "row_src", (torch.int32,), x.device)
        if row_src.numel() != B:
            raise ValueError("row_src must have B entries")
    _require(out, "out", (torch.bfloat16,), x.device)
    if tuple(out.shape) != (B, N):
        raise ValueError("out has shape %s, expected %s" % (tuple(out.shape), (B, N)))
    if dev_status is not None:
        _require(dev_status, "dev_status", (torch.int32,), x.device)
    ctx, st = _launch_on(x.device, stream)
    with ctx:
        _check(lib().mxq_gather_qmm_noalloc(_ptr(x), _ptr(w), _ptr(scales), _ptr(biases),
                                            _ptr(expert_ids), _ptr(row_src), _ptr(out), T, B, E, K,
                                            N, bits, group_size, _ptr(dev_status),
                                            st), "mxq_gather_qmm_noalloc")
    return out


def gather_qmm(x, w, scales, biases, expert_ids, row_src, bits: int, out=None, workspace=None,
               dev_status=None, stream=None, group_size: int = 64):
    """Sorted mixture-of-experts GEMM: sorted row r multiplies expert
    ``expert_ids[r]``'s dequantised matrix by ``x[row_src[r]]``.

    ``w`` is [E, N, K*bits/32], ``scales``/``biases`` [E, N, K/group_size],
    ``expert_ids`` int32 [B] non-decreasing, ``row_src`` int32 [B] or None
    (identity).  Returns y bf16 [B, N] in sorted row order.
    """
    torch = _torch()
    _require(x, "x", (torch.bfloat16,))
    if x.dim() != 2:
        raise ValueError("x must be 2-D [T, K]")
    T, K = x.shape
    if w.dim() != 3:
        raise ValueError("w must be 3-D [E, N, K*bits/32]")
    E, N = w.shape[0], w.shape[1]
    _check_weights(w, scales, biases, N, K, bits, x.device, lead=(E,), group_size=group_size)
    _require(expert_ids, "expert_ids", (torch.int32,), x.device)
    B = expert_ids.numel()
    if row_src is not None:
        _require(row_src, "row_src", (torch.int32,), x.device)
        if row_src.numel() != B:
            raise ValueError("row_src must have B entries")
    if out is None:
        out = torch.empty((B, N), dtype=torch.bfloat16, device=x.device)
    _require(out, "out", (torch.bfloat16,), x.device)
    if workspace is None:
        workspace = torch.empty((gather_workspace_bytes(B, E, K if row_src is not None else 0, N),),
                                dtype=torch.uint8, device=x.device)
    _require(workspace, "workspace", (torch.uint8,), x.device)
    if dev_status is not None:
        _require(dev_status, "dev_status", (torch.int32,), x.device)
    ctx, st = _launch_on(x.device, stream)
    with ctx:
        _check(lib().mxq_gather_qmm(_ptr(x), _ptr(w), _ptr(scales), _ptr(biases),
                                    _ptr(expert_ids), _ptr(row_src), _ptr(out), T, B, E, K, N,
                                    bits, group_size, _ptr(workspace), workspace.numel(),
                                    _ptr(dev_status), st), "mxq_gather_qmm")
    return out


def gather_qmm_gateup(x, w_gate, s_gate, b_gate, w_up, s_up, b_up, expert_ids, row_src,
                      bits: int, out_gate=None, out_up=None, workspace=None, dev_status=None,
                      stream=None, group_size: int = 64):
    """The gate and up projections of a mixture-of-experts layer: the same
    routed rows against two expert weight sets of one shape.  Returns
    (y_gate, y_up), each bf16 [B, N] in sorted row order; no activation
    function is applied."""
    torch = _torch()
    _require(x, "x", (torch.bfloat16,))
    if x.dim() != 2:
        raise ValueError("x must be 2-D [T, K]")
    T, K = x.shape
    if w_gate.dim() != 3 or tuple(w_up.shape) != tuple(w_gate.shape):
        raise ValueError("w_gate and w_up must both be [E, N, K*bits/32]")
    E, N = w_gate.shape[0], w_gate.shape[1]
    _check_weights(w_gate, s_gate, b_gate, N, K, bits, x.device, lead=(E,),
                   group_size=group_size)
    _check_weights(w_up, s_up, b_up, N, K, bits, x.device, lead=(E,), group_size=group_size)
    _require(expert_ids, "expert_ids", (torch.int32,), x.device)
    B = expert_ids.numel()
    if row_src is not None:
        _require(row_src, "row_src", (torch.int32,), x.device)
        if row_src.numel() != B:
            raise ValueError("row_src must have B entries")
    outs = []
    for o, name in ((out_gate, "out_gate"), (out_up, "out_up")):
        if o is None:
            o = torch.empty((B, N), dtype=torch.bfloat16, device=x.device)
        _require(o, name, (torch.bfloat16,), x.device)
        if tuple(o.shape) != (B, N):
            raise ValueError("%s has shape %s, expected %s" % (name, tuple(o.shape), (B, N)))
        outs.append(o)
    if workspace is None:
        workspace = torch.empty((gather_workspace_bytes(B, E, K if row_src is not None else 0, N),),
                                dtype=torch.uint8, device=x.device)
    _require(workspace, "workspace", (torch.uint8,), x.device)
    if dev_status is not None:
        _require(dev_status, "dev_status", (torch.int32,), x.device)
    ctx, st = _launch_on(x.device, stream)
    with ctx:
        _check(lib().mxq_gather_qmm_gateup(
            _ptr(x), _ptr(w_gate), _ptr(s_gate), _ptr(b_gate), _ptr(w_up), _ptr(s_up), _ptr(b_up),
            _ptr(expert_ids), _ptr(row_src), _ptr(outs[0]), _ptr(outs[1]), T, B, E, K, N, bits,
            group_size, _ptr(workspace), workspace.numel(), _ptr(dev_status), st),
            "mxq_gather_qmm_gateup")
    return outs[0], outs[1]


# ------------------------------------------------- 4-bit key/value cache

def _empty(shape, dtype, device, stream):
    """A tensor for a call on ``stream``, out of that stream's memory: what was freed on the
    current one may still be in use there, and a workspace goes when the call returns."""
    torch = _torch()
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if stream.device != device:
        raise ValueError("stream is on %s but the tensors are on %s" % (stream.device, device))
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _heads(t, name, index=None, out=False):
    """Checks a bf16 [T, heads, D] tensor whose heads are contiguous; returns
    its (row, head) strides in values.  ``index``: the device it has to be on."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    on = t.get_device()
    if on < 0:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dtype is not torch.bfloat16:
        raise TypeError("%s has dtype %s, expected torch.bfloat16" % (name, t.dtype))
    if t.dim() != 3:
        raise ValueError("%s must be 3-D [T, heads, D]" % name)
    if index is not None and on != index:
        raise ValueError("%s is on %s, expected cuda:%d" % (name, t.device, index))
    n, h, d = t.shape
    rs, hs, vs = t.stride()
    if vs != 1 and d > 1:
        raise ValueError("the values of a head of %s must be contiguous" % name)
    if h <= 1:
        hs = d
    if n <= 1:
        rs = h * d
    if rs % 8 or hs % 8:
        raise ValueError("the strides of %s must be multiples of 8 values" % name)
    if out and ((h > 1 and hs < d) or (n > 1 and rs < d) or
                (n > 1 and h > 1 and rs < h * hs and hs < n * rs)):
        raise ValueError("the rows of %s overlap" % name)
    return rs, hs


def _flat(t, name, dtype, index=None):
    """Checks a contiguous tensor of ``dtype`` on device ``index``; its address."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    on = t.get_device()
    if on < 0:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dtype is not dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if index is not None and on != index:
        raise ValueError("%s is on %s, expected cuda:%d" % (name, t.device, index))
    return t.data_ptr()


def rope_inv_freq(rot_dim: int, theta: float = 10000.0, scaling=None, factor: float = 1.0,
                  original_len: int = 0, low: float = 1.0, high: float = 4.0,
                  beta_fast: float = 32.0, beta_slow: float = 1.0, device=None):
    """The rotation's frequencies ``theta^(-2 j / rot_dim)`` (fp32
    [rot_dim/2]) and the factor of its cosines and sines, ``(inv_freq,
    rope_scale)`` for ``qk_norm_rope``; computed in 64 bits.

    ``scaling`` stretches them for contexts ``factor`` times as long as the
    ``original_len`` tokens that a model was trained on:

    * ``"linear"``: every frequency divided by ``factor``;
    * ``"base"``: theta raised to ``theta * factor^(rot_dim / (rot_dim - 2))``,
      which leaves the highest frequency and divides the lowest by ``factor``;
    * ``"bands"``: by the turns that a frequency makes in ``original_len``
      tokens: below ``low`` divided by ``factor``, above ``high`` kept, between
      them mixed linearly in the turns;
    * ``"yarn"``: divided by ``factor`` from the value whose frequency makes
      ``beta_slow`` turns on, kept up to the one that makes ``beta_fast``,
      mixed linearly in the index between; ``rope_scale = 0.1 ln(factor) + 1``.
    """
    import math

    torch = _torch()
    if rot_dim <= 0 or rot_dim % 2:
        raise ValueError("rot_dim must be positive and even")
    if not theta > 0 or not factor >= 1.0:
        raise ValueError("theta must be positive and factor at least 1")
    j = torch.arange(rot_dim // 2, dtype=torch.float64)
    scale = 1.0
    if scaling == "base":
        if rot_dim <= 2:
            raise ValueError("base scaling needs rot_dim > 2")
        theta = theta * factor ** (rot_dim / (rot_dim - 2.0))
    freq = theta ** (-2.0 * j / rot_dim)
    if scaling == "linear":
        freq = freq / factor
    elif scaling in ("bands", "yarn"):
        if original_len <= 0:
            raise ValueError("%s scaling needs original_len" % scaling)
        if scaling == "bands":
            if not high > low:
                raise ValueError("high must be above low")
            turns = original_len * freq / (2.0 * math.pi)
            keep = ((turns - low) / (high - low)).clamp(0.0, 1.0)
        else:
            def index(turns):
                return rot_dim * math.log(original_len / (turns * 2.0 * math.pi)) / (
                    2.0 * math.log(theta))

            first = max(math.floor(index(beta_fast)), 0)
            last = min(math.ceil(index(beta_slow)), rot_dim - 1)
            keep = 1.0 - ((j - first) / max(last - first, 0.001)).clamp(0.0, 1.0)
            scale = 0.1 * math.log(factor) + 1.0
        freq = freq * (keep + (1.0 - keep) / factor)
    elif scaling not in (None, "base"):
        raise ValueError("unknown scaling %r" % (scaling,))
    return freq.to(torch.float32).to(device if device is not None else "cpu"), scale


def qk_norm_rope(q, k, positions=None, inv_freq=None, q_weight=None, k_weight=None, eps=1e-6,
                 weight_offset=0.0, interleaved=False, rope_scale=1.0, q_out=None, k_out=None,
                 stream=None):
    """RMS norm of query and key heads (``q_weight``/``k_weight`` bf16 [D];
    None: no norm) and the rotary position (``positions`` int32 [T],
    ``inv_freq`` fp32 [rot_dim/2]; None: no rotation) in one pass.

    ``q`` bf16 [T, Hq, D] and ``k`` bf16 [T, Hk, D] or None may be slices of
    one projection's output (heads contiguous, strides multiples of 8);
    ``q_out``/``k_out`` may be ``q``/``k`` themselves.  Returns (q_out, k_out)."""
    if stream is None:
        done = _direct().qk_norm_rope(q, k, positions, inv_freq, q_weight, k_weight, eps, weight_offset,
                                     interleaved, rope_scale, q_out, k_out)
        if done is not None:
            return done
    torch = _torch()
    q_rs, q_hs = _heads(q, "q")
    dev = q.device
    on = dev.index
    T, Hq, D = q.shape
    Hk = k_rs = k_hs = k_ors = k_ohs = rot = 0
    k_at = k_out_at = pos_at = freq_at = qw_at = kw_at = None
    if k is not None:
        k_rs, k_hs = _heads(k, "k", on)
        Hk = k.shape[1]
        if k.shape[0] != T or k.shape[2] != D:
            raise ValueError("k has shape %s, expected [%d, heads, %d]" % (tuple(k.shape), T, D))
        k_at = k.data_ptr()
    elif k_weight is not None or k_out is not None:
        raise ValueError("k_weight and k_out need k")
    if inv_freq is not None:
        freq_at = _flat(inv_freq, "inv_freq", torch.float32, on)
        if positions is None:
            raise ValueError("a rotation needs positions")
        pos_at = _flat(positions, "positions", torch.int32, on)
        if positions.numel() != T:
            raise ValueError("positions must have T entries")
        rot = 2 * inv_freq.numel()
        if inv_freq.dim() != 1 or rot == 0:
            raise ValueError("inv_freq must be 1-D [rot_dim/2]")
    if q_weight is not None:
        qw_at = _flat(q_weight, "q_weight", torch.bfloat16, on)
        if q_weight.dim() != 1 or q_weight.numel() != D:
            raise ValueError("q_weight must be [D]")
    if k_weight is not None:
        kw_at = _flat(k_weight, "k_weight", torch.bfloat16, on)
        if k_weight.dim() != 1 or k_weight.numel() != D:
            raise ValueError("k_weight must be [D]")
    if q_out is None:
        q_out = _empty((T, Hq, D), torch.bfloat16, dev, stream)
        q_ors, q_ohs = Hq * D, D
    else:
        if q_out.shape != q.shape:
            raise ValueError("q_out must have the shape of q")
        q_ors, q_ohs = _heads(q_out, "q_out", on, out=True)
    if k is not None:
        if k_out is None:
            k_out = _empty((T, Hk, D), torch.bfloat16, dev, stream)
            k_ors, k_ohs = Hk * D, D
        else:
            if k_out.shape != k.shape:
                raise ValueError("k_out must have the shape of k")
            k_ors, k_ohs = _heads(k_out, "k_out", on, out=True)
        k_out_at = k_out.data_ptr()
    ctx, st = _launch_on(dev, stream)
    with ctx:
        _check(lib().mxq_qk_norm_rope(
            q.data_ptr(), q_rs, q_hs, k_at, k_rs, k_hs, pos_at, freq_at, qw_at, kw_at,
            q_out.data_ptr(), q_ors, q_ohs, k_out_at, k_ors, k_ohs, T, Hq, Hk, D, rot,
            1 if interleaved else 0, eps, weight_offset, rope_scale, st), "mxq_qk_norm_rope")
    return q_out, k_out


def _int32(x):
    """A count for the C functions, which take 32 bits and would be given the lowest ones: what is
    past them stays past every length there is."""
    return max(min(x, 2 ** 31 - 1), -2 ** 31)


def kv_block_bytes(head_dim: int, page_size: int, group_size: int = 64) -> int:
    """Bytes of one page of the 4-bit cache for one key/value head: a cache is
    a uint8 tensor ``[n_pages, kv_heads, kv_block_bytes(...)]``."""
    n = int(lib().mxq_kv_block_bytes(_int32(head_dim), _int32(page_size), _int32(group_size)))
    if n == 0:
        raise ValueError("no cache of head_dim %s, page_size %s, group_size %s" % (
            head_dim, page_size, group_size))
    return n


def _cache(pages, head_dim, group_size, index, kv_heads=None):
    """Checks a cache tensor and returns (address, n_pages, kv_heads, page_size)."""
    at = _flat(pages, "pages", _torch().uint8, index)
    if pages.dim() != 3:
        raise ValueError("pages must be [n_pages, kv_heads, block bytes]")
    n, h, block = pages.shape
    if kv_heads is not None and h != kv_heads:
        raise ValueError("pages hold %d heads, expected %d" % (h, kv_heads))
    if head_dim not in (64, 128, 256) or group_size not in (32, 64, 128) or group_size > head_dim:
        raise ValueError("no cache of head_dim %s and group_size %s" % (head_dim, group_size))
    per = head_dim + 8 * (head_dim // group_size)
    if block % per or block // per not in (16, 32, 64, 128):
        raise ValueError("a block of %d bytes is no page of head_dim %d, group_size %d" % (
            block, head_dim, group_size))
    return at, n, h, block // per


def kv_append(k, v, pages, slots, group_size: int = 64, dev_status=None, stream=None):
    """Encodes the rows ``k``, ``v`` (bf16 [T, kv_heads, D], heads contiguous)
    to 4 bits and writes row t to slot ``slots[t]`` (int32 [T], page *
    page_size + token; negative: skipped) of the cache ``pages``."""
    if stream is None and _direct().kv_append(k, v, pages, slots, group_size, dev_status) is not None:
        return pages
    torch = _torch()
    k_rs, k_hs = _heads(k, "k")
    dev = k.device
    on = dev.index
    v_rs, v_hs = _heads(v, "v", on)
    if v.shape != k.shape:
        raise ValueError("v has shape %s, expected %s" % (tuple(v.shape), tuple(k.shape)))
    T, H, D = k.shape
    at, n_pages, _, page_size = _cache(pages, D, group_size, on, H)
    slots_at = _flat(slots, "slots", torch.int32, on)
    if slots.numel() != T:
        raise ValueError("slots must have T entries")
    status = None if dev_status is None else _flat(dev_status, "dev_status", torch.int32, on)
    ctx, st = _launch_on(dev, stream)
    with ctx:
        _check(lib().mxq_kv_append(k.data_ptr(), k_rs, k_hs, v.data_ptr(), v_rs, v_hs, at, slots_at,
                                   T, H, D, n_pages, page_size, group_size, status, st),
               "mxq_kv_append")
    return pages


def kv_read(pages, slots, head_dim: int, group_size: int = 64, k_out=None, v_out=None,
            dev_status=None, stream=None):
    """The rows of ``slots`` (int32 [T]) out of the cache: (k, v) bf16 [T,
    kv_heads, head_dim]; zeros for a negative slot."""
    if stream is None:
        done = _direct().kv_read(pages, slots, head_dim, group_size, k_out, v_out, dev_status)
        if done is not None:
            return done
    torch = _torch()
    at, n_pages, H, page_size = _cache(pages, head_dim, group_size, None)
    dev = pages.device
    on = dev.index
    slots_at = _flat(slots, "slots", torch.int32, on)
    T = slots.numel()
    shape = (T, H, head_dim)
    if k_out is None:
        k_out = _empty(shape, torch.bfloat16, dev, stream)
    elif tuple(k_out.shape) != shape:
        raise ValueError("k_out has shape %s, expected %s" % (tuple(k_out.shape), shape))
    if v_out is None:
        v_out = _empty(shape, torch.bfloat16, dev, stream)
    elif tuple(v_out.shape) != shape:
        raise ValueError("v_out has shape %s, expected %s" % (tuple(v_out.shape), shape))
    k_at = _flat(k_out, "k_out", torch.bfloat16, on)
    v_at = _flat(v_out, "v_out", torch.bfloat16, on)
    status = None if dev_status is None else _flat(dev_status, "dev_status", torch.int32, on)
    ctx, st = _launch_on(dev, stream)
    with ctx:
        _check(lib().mxq_kv_read(at, slots_at, k_at, v_at, T, H, head_dim, n_pages, page_size,
                                 group_size, status, st), "mxq_kv_read")
    return k_out, v_out


def kv_attention_workspace_bytes(rows: int, seqs: int, heads: int, kv_heads: int, head_dim: int,
                                 max_q_len: int = 1) -> int:
    """Workspace bytes for kv_attention of ``rows`` query rows in ``seqs`` sequences."""
    return int(lib().mxq_kv_attention_workspace_bytes(rows, seqs, heads, kv_heads, head_dim,
                                                      _int32(max_q_len)))


def kv_attention(q, pages, page_table, ctx_lens, q_starts=None, max_q_len: int = 1,
                 group_size: int = 64, scale=None, window: int = 0, sinks: int = 0, out=None,
                 lse=None, workspace=None, dev_status=None, stream=None):
    """Causal attention of ``q`` (bf16 [T, heads, D]) over a 4-bit paged cache.

    Sequence i holds ``ctx_lens[i]`` tokens in the pages ``page_table[i]``
    (int32 [S, max_pages]); its query rows ``q_starts[i]:q_starts[i+1]``
    (int32 [S+1]; None: one row per sequence) are its last tokens, at most
    ``max_q_len`` of them.  With ``window`` a row sees the last ``window``
    tokens up to its own and the first ``sinks``.  ``scale`` defaults to
    D^-1/2.  ``lse`` (fp32 [T, heads]) receives the log sum exp.  Returns out
    bf16 [T, heads, D]; a row that sees nothing is 0."""
    if stream is None:
        done = _direct().kv_attention(q, pages, page_table, ctx_lens, q_starts, max_q_len, group_size, scale,
                                     window, sinks, out, lse, workspace, dev_status)
        if done is not None:
            return done
    torch = _torch()
    q_rs, q_hs = _heads(q, "q")
    dev = q.device
    on = dev.index
    T, Hq, D = q.shape
    at, n_pages, Hkv, page_size = _cache(pages, D, group_size, on)
    if Hq == 0 or Hkv == 0 or Hq % Hkv:
        raise ValueError("%d query heads do not divide over %d key/value heads" % (Hq, Hkv))
    table_at = _flat(page_table, "page_table", torch.int32, on)
    if page_table.dim() != 2:
        raise ValueError("page_table must be 2-D [S, max_pages]")
    S, max_pages = page_table.shape
    lens_at = _flat(ctx_lens, "ctx_lens", torch.int32, on)
    if ctx_lens.numel() != S:
        raise ValueError("ctx_lens must have S entries")
    starts_at = lse_at = status = None
    if q_starts is not None:
        starts_at = _flat(q_starts, "q_starts", torch.int32, on)
        if q_starts.numel() != S + 1:
            raise ValueError("q_starts must have S + 1 entries")
    elif T != S or max_q_len != 1:
        raise ValueError("without q_starts every sequence has one row: T must be S, max_q_len 1")
    if out is None:
        out = _empty((T, Hq, D), torch.bfloat16, dev, stream)
        out_at = out.data_ptr()
    else:
        out_at = _flat(out, "out", torch.bfloat16, on)
        if tuple(out.shape) != (T, Hq, D):
            raise ValueError("out has shape %s, expected %s" % (tuple(out.shape), (T, Hq, D)))
    if lse is not None:
        lse_at = _flat(lse, "lse", torch.float32, on)
        if tuple(lse.shape) != (T, Hq):
            raise ValueError("lse has shape %s, expected %s" % (tuple(lse.shape), (T, Hq)))
    if dev_status is not None:
        status = _flat(dev_status, "dev_status", torch.int32, on)
    if max_q_len <= 0:
        raise ValueError("max_q_len must be positive")
    max_q_len, window, sinks = _int32(max_q_len), _int32(window), _int32(sinks)
    L = lib()
    if workspace is None:
        need = L.mxq_kv_attention_workspace_bytes(T, S, Hq, Hkv, D, max_q_len)
        workspace = _empty((need,), torch.uint8, dev, stream)
    ws_at = _flat(workspace, "workspace", torch.uint8, on)
    ctx, st = _launch_on(dev, stream)
    with ctx:
        _check(L.mxq_kv_attention(
            q.data_ptr(), q_rs, q_hs, at, table_at, lens_at, starts_at, out_at, lse_at, T, S, Hq,
            Hkv, D, n_pages, max_pages, page_size, group_size, max_q_len,
            D ** -0.5 if scale is None else scale, window, sinks, ws_at, workspace.numel(), status,
            st), "mxq_kv_attention")
    return out


def kv_attention_shared_workspace_bytes(rows: int, seqs: int, groups: int, heads: int, kv_heads: int,
                                        head_dim: int, max_q_len: int = 1, max_group=None) -> int:
    """Workspace bytes for kv_attention_shared of ``rows`` query rows in ``seqs`` sequences and
    ``groups`` groups of at most ``max_group`` sequences (default: all of them)."""
    return int(lib().mxq_kv_attention_shared_workspace_bytes(*map(_int32, (
        rows, seqs, groups, heads, kv_heads, head_dim, max_q_len, max(seqs, 1) if max_group is None else max_group))))


def kv_attention_shared(q, pages, prefix_table, prefix_lens, page_table, ctx_lens, group_starts=None,
                        q_starts=None, max_q_len: int = 1, max_group=None, group_size: int = 64,
                        scale=None, out=None, lse=None, workspace=None, dev_status=None, stream=None):
    """Attention of ``q`` (bf16 [T, heads, D]) over a 4-bit paged cache for groups of sequences
    that begin with the same tokens, which are read once for a group.

    Group g shares the ``prefix_lens[g]`` tokens (int32 [N]) in the pages ``prefix_table[g]``
    (int32 [N, max_prefix_pages]); its sequences are ``group_starts[g]:group_starts[g+1]`` (int32
    [N+1], at most ``max_group`` each, default all; None: S / N each).  Sequence i has
    ``ctx_lens[i]`` tokens of its own in the pages ``page_table[i]`` (int32 [S, max_pages]); its
    query rows ``q_starts[i]:q_starts[i+1]`` (int32 [S+1], at most ``max_q_len`` each; None: one
    row per sequence) are the last of them: row j of n sees the whole prefix and the own tokens up
    to ``ctx_lens[i] - n + j``.  ``scale`` defaults to D^-1/2.  ``lse`` (fp32 [T, heads]) receives
    the log sum exp.  Returns out bf16 [T, heads, D]; a row that sees nothing is 0.

    Where groups have more than 32 rows (times query heads to a key/value head), by ``max_group`` and
    ``max_q_len``, the prefix's keys, values and weights may be rounded to 11 bits, as kv_attention does for
    prompts; else keys are as the cache holds them, and weights times value scales have 11 bits."""
    if stream is None:
        done = _direct().kv_attention_shared(q, pages, prefix_table, prefix_lens, page_table, ctx_lens, group_starts,
                                             q_starts, max_q_len, max_group, group_size, scale, out, lse, workspace,
                                             dev_status)
        if done is not None:
            return done
    torch = _torch()
    q_rs, q_hs = _heads(q, "q")
    dev = q.device
    on = dev.index
    T, Hq, D = q.shape
    at, n_pages, Hkv, page_size = _cache(pages, D, group_size, on)
    if Hq == 0 or Hkv == 0 or Hq % Hkv:
        raise ValueError("%d query heads do not divide over %d key/value heads" % (Hq, Hkv))
    prefix_at = _flat(prefix_table, "prefix_table", torch.int32, on)
    if prefix_table.dim() != 2 or prefix_table.shape[0] == 0:
        raise ValueError("prefix_table must be 2-D [N, max_prefix_pages]")
    N, max_prefix_pages = prefix_table.shape
    prefix_lens_at = _flat(prefix_lens, "prefix_lens", torch.int32, on)
    if prefix_lens.numel() != N:
        raise ValueError("prefix_lens must have N entries")
    table_at = _flat(page_table, "page_table", torch.int32, on)
    if page_table.dim() != 2:
        raise ValueError("page_table must be 2-D [S, max_pages]")
    S, max_pages = page_table.shape
    lens_at = _flat(ctx_lens, "ctx_lens", torch.int32, on)
    if ctx_lens.numel() != S:
        raise ValueError("ctx_lens must have S entries")
    groups_at = starts_at = lse_at = status = None
    if group_starts is not None:
        groups_at = _flat(group_starts, "group_starts", torch.int32, on)
        if group_starts.numel() != N + 1:
            raise ValueError("group_starts must have N + 1 entries")
        max_group = max(S, 1) if max_group is None else max_group
    elif S % N:
        raise ValueError("without group_starts the %d sequences must divide over the %d groups" % (S, N))
    else:
        max_group = max(S // N, 1) if max_group is None else max_group
        if max_group < S // N:
            raise ValueError("max_group must be at least the %d sequences of a group" % (S // N))
    if q_starts is not None:
        starts_at = _flat(q_starts, "q_starts", torch.int32, on)
        if q_starts.numel() != S + 1:
            raise ValueError("q_starts must have S + 1 entries")
    elif T != S or max_q_len != 1:
        raise ValueError("without q_starts every sequence has one row: T must be S, max_q_len 1")
    if out is None:
        out = _empty((T, Hq, D), torch.bfloat16, dev, stream)
        out_at = out.data_ptr()
    else:
        out_at = _flat(out, "out", torch.bfloat16, on)
        if tuple(out.shape) != (T, Hq, D):
            raise ValueError("out has shape %s, expected %s" % (tuple(out.shape), (T, Hq, D)))
    if lse is not None:
        lse_at = _flat(lse, "lse", torch.float32, on)
        if tuple(lse.shape) != (T, Hq):
            raise ValueError("lse has shape %s, expected %s" % (tuple(lse.shape), (T, Hq)))
    if dev_status is not None:
        status = _flat(dev_status, "dev_status", torch.int32, on)
    if max_q_len <= 0 or max_group <= 0:
        raise ValueError("max_q_len and max_group must be positive")
    max_q_len, max_group = _int32(max_q_len), _int32(max_group)
    S, N, max_prefix_pages, max_pages = map(_int32, (S, N, max_prefix_pages, max_pages))
    L = lib()
    if workspace is None:
        need = L.mxq_kv_attention_shared_workspace_bytes(T, S, N, Hq, Hkv, D, max_q_len, max_group)
        workspace = _empty((need,), torch.uint8, dev, stream)
    ws_at = _flat(workspace, "workspace", torch.uint8, on)
    ctx, st = _launch_on(dev, stream)
    with ctx:
        _check(L.mxq_kv_attention_shared(
            q.data_ptr(), q_rs, q_hs, at, prefix_at, prefix_lens_at, groups_at, table_at, lens_at,
            starts_at, out_at, lse_at, T, S, N, Hq, Hkv, D, n_pages, max_prefix_pages, max_pages,
            page_size, group_size, max_q_len, max_group, D ** -0.5 if scale is None else scale, ws_at,
            workspace.numel(), status, st), "mxq_kv_attention_shared")
    return out


# ------------------------------------------------- beams

def beam_select(logits, scores, k=None, done=None, end_token: int = 0, scores_out=None, parents_out=None,
                tokens_out=None, done_out=None, workspace=None, stream=None):
    """The ``k`` best continuations (default: as many as beams) of N prompts with W beams each:
    ``scores[w] + log_softmax(logits[w])[v]`` over a prompt's beams and tokens, the best first,
    equal ones in the order of w V + v.

    ``logits`` bf16 or fp32 [N, W, V] or [N W, V] (tokens contiguous, rows at equal distances), ``scores`` fp32
    [N, W]; -inf is a beam that is not in use, a -inf logit a token that is not allowed.  ``done``
    (bool [N, W]): beams that have ended; one has the single candidate ``end_token``, with its score
    as it is.  Returns (scores fp32, parents int32, tokens int32), each [N, k], and with ``done``
    a fourth, bool: the parent had ended or the token is ``end_token``."""
    if stream is None:
        found = _direct().beam_select(logits, scores, k, done, end_token, scores_out, parents_out, tokens_out,
                                      done_out, workspace)
        if found is not None:
            return found
    torch = _torch()
    if not isinstance(logits, torch.Tensor):
        raise TypeError("logits must be a torch.Tensor")
    if not logits.is_cuda:
        raise ValueError("logits must be a CUDA tensor")
    if logits.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError("logits has dtype %s, expected bfloat16 or float32" % logits.dtype)
    dev = logits.device
    on = dev.index
    scores_at = _flat(scores, "scores", torch.float32, on)
    if scores.dim() != 2:
        raise ValueError("scores must be 2-D [N, W]")
    N, W = scores.shape
    if logits.dim() not in (2, 3) or tuple(logits.shape[:-1]) != ((N * W,) if logits.dim() == 2 else (N, W)):
        raise ValueError("logits has shape %s, expected [%d, %d, V] or [%d, V]" % (tuple(logits.shape), N, W, N * W))
    V = logits.shape[-1]
    row = logits.stride(-2) if logits.shape[-2] > 1 else logits.stride(0)
    if V > 1 and logits.stride(-1) != 1:
        raise ValueError("the tokens of a row of logits must be contiguous")
    if logits.dim() == 3 and N > 1 and W > 1 and logits.stride(0) != W * row:
        raise ValueError("the rows of logits must be at equal distances")
    k = W if k is None else k
    if not 0 < k <= min(64, W * V) or W > 64:
        raise ValueError("%d of %d beams times %d tokens: at most 64 beams and 64 of them" % (k, W, V))
    done_at = done_out_at = None
    if done is not None:
        done_at = _flat(done, "done", torch.bool, on)
        if tuple(done.shape) != (N, W):
            raise ValueError("done has shape %s, expected %s" % (tuple(done.shape), (N, W)))
    elif done_out is not None:
        raise ValueError("done_out needs done")
    if done is not None and not 0 <= end_token < V:
        raise ValueError("end_token %d is none of %d tokens" % (end_token, V))
    outs = []
    for t, name, dtype in ((scores_out, "scores_out", torch.float32), (parents_out, "parents_out", torch.int32),
                           (tokens_out, "tokens_out", torch.int32), (done_out, "done_out", torch.bool)):
        if name == "done_out" and done is None:
            break
        if t is None:
            t = _empty((N, k), dtype, dev, stream)
        _flat(t, name, dtype, on)
        if tuple(t.shape) != (N, k):
            raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), (N, k)))
        outs.append(t)
    if done is not None:
        done_out_at = outs[3].data_ptr()
    fp32 = 1 if logits.dtype is torch.float32 else 0
    N, V = _int32(N), _int32(V)
    end = _int32(end_token) if done is not None else 0
    L = lib()
    if workspace is None:
        workspace = _empty((L.mxq_beam_select_workspace_bytes(N, W, V, k, fp32),), torch.uint8, dev, stream)
    ws_at = _flat(workspace, "workspace", torch.uint8, on)
    ctx, st = _launch_on(dev, stream)
    with ctx:
        _check(L.mxq_beam_select(logits.data_ptr(), row, fp32, scores_at, done_at, outs[0].data_ptr(),
                                 outs[1].data_ptr(), outs[2].data_ptr(), done_out_at, N, W, V, k,
                                 end, ws_at, workspace.numel(), st),
               "mxq_beam_select")
    return tuple(outs)


def kv_reorder(pages, page_table, home_table, ctx_lens, parents, head_dim: int, group_size: int = 64,
               table_out=None, lens_out=None, workspace=None, dev_status=None, stream=None):
    """The cache after a selection of beams: sequence i of a group goes on from sequence
    ``parents[i]`` of it (int32 [N, W], as beam_select gives them; groups of W sequences in a row).

    ``home_table`` (int32 [S, max_pages]) are the pages that each sequence was given; ``page_table``
    starts as a copy of it.  Full pages come to be shared, the page that is being written stays with
    the lowest sequence that goes on from it, and each other one gets one of the group's own pages
    of that column that nobody uses, into which the tokens are copied.  ``pages``: the cache, uint8
    [n_pages, kv_heads, block] or [layers, n_pages, kv_heads, block] for layers with one table.
    Returns (table, lens), the page table and ``ctx_lens`` (int32 [S]) of the sequences as they go
    on; ``table_out`` and ``lens_out`` may be ``page_table`` and ``ctx_lens`` themselves."""
    if stream is None:
        found = _direct().kv_reorder(pages, page_table, home_table, ctx_lens, parents, head_dim, group_size,
                                     table_out, lens_out, workspace, dev_status)
        if found is not None:
            return found
    torch = _torch()
    at = _flat(pages, "pages", torch.uint8)
    dev = pages.device
    on = dev.index
    if pages.dim() not in (3, 4):
        raise ValueError("pages must be [n_pages, kv_heads, block bytes] or [layers, n_pages, kv_heads, block bytes]")
    layers = pages.shape[0] if pages.dim() == 4 else 1
    if layers == 0:
        raise ValueError("pages hold no layers")
    _, n_pages, H, page_size = _cache(pages[0] if pages.dim() == 4 else pages, head_dim, group_size, on)
    table_at = _flat(page_table, "page_table", torch.int32, on)
    if page_table.dim() != 2:
        raise ValueError("page_table must be 2-D [S, max_pages]")
    S, max_pages = page_table.shape
    home_at = _flat(home_table, "home_table", torch.int32, on)
    if tuple(home_table.shape) != (S, max_pages):
        raise ValueError("home_table has shape %s, expected %s" % (tuple(home_table.shape), (S, max_pages)))
    lens_at = _flat(ctx_lens, "ctx_lens", torch.int32, on)
    parents_at = _flat(parents, "parents", torch.int32, on)
    if ctx_lens.numel() != S or parents.numel() != S or parents.dim() != 2 or not 0 < parents.shape[1] <= 64:
        raise ValueError("ctx_lens must have S entries and parents be [N, W], N W = S, W up to 64")
    if table_out is None:
        table_out = _empty((S, max_pages), torch.int32, dev, stream)
    if lens_out is None:
        lens_out = _empty((S,), torch.int32, dev, stream)
    table_out_at = _flat(table_out, "table_out", torch.int32, on)
    lens_out_at = _flat(lens_out, "lens_out", torch.int32, on)
    if tuple(table_out.shape) != (S, max_pages) or lens_out.numel() != S:
        raise ValueError("table_out must be [S, max_pages] and lens_out have S entries")
    status = None if dev_status is None else _flat(dev_status, "dev_status", torch.int32, on)
    S, max_pages, layers = map(_int32, (S, max_pages, layers))
    L = lib()
    if workspace is None:
        workspace = _empty((L.mxq_kv_reorder_workspace_bytes(S),), torch.uint8, dev, stream)
    ws_at = _flat(workspace, "workspace", torch.uint8, on)
    ctx, st = _launch_on(dev, stream)
    with ctx:
        _check(L.mxq_kv_reorder(at, table_at, home_at, lens_at, parents_at, table_out_at, lens_out_at, S,
                                parents.shape[1], layers, n_pages, H, head_dim, max_pages, page_size, group_size,
                                ws_at, workspace.numel(), status, st), "mxq_kv_reorder")
    return table_out, lens_out


def set_wait_budget(cycles: int) -> int:
    """Testing aid: the budget, in SM clock cycles, after which an on-chip
    pipeline wait of a kernel launched from now on gives up (the call's
    ``dev_status`` then gets ``DEV_TIMEOUT`` and its output is incomplete).
    ``cycles <= 0`` restores the default of 2e9 cycles.  Returns the budget in
    force.  Waits for a CTA's own copies and MMAs keep the default, so the
    next call after a timed-out one runs normally."""
    return int(lib().mxq_debug_set_wait_budget(int(cycles)))
