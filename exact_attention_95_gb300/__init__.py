"""Exact softmax attention for NVIDIA GB300 (sm_103a): Python binding.

A thin layer over the C ABI in ``include/attn.h`` (``libattn_sm103.so``, built
in-tree by ``exact_attention_95_gb300.build``): ctypes, and for the paged cache's
calls an extension module, without which they make their checks in Python and
take longer.  It only marshals arguments: PyTorch supplies device memory and the
current stream, and every step of the computation runs in the library's CUDA
kernels.  If the library is missing, every call raises; there is no fallback
implementation.

Functions carry the C names:

* ``attn_fwd(Q, K, V, scale, causal, out_dtype=None) -> (O, LSE)``
* ``attn_fwd_split(Q, K, V, scale, causal, num_splits=0, ...) -> (O, LSE)``: query
  and key lengths may differ (bottom-right causal alignment); the key range may
  be split, with the partial results merged
* ``attn_fwd_split_workspace_size(B, Hq, Hkv, Nq, Nk, d, num_splits)``
* ``attn_fwd_masked(Q, K, V, block_mask, scale, causal, out_dtype=None)`` and
  ``attn_bwd_masked(Q, K, V, O, dO, LSE, block_mask, scale, causal)``: block-sparse
  attention with a uint8 CUDA mask [1 or Hq, ceil(N/128), ceil(N/128)]
* ``attn_quantize_fp8(X, transpose=False) -> (codes, scales)`` and
  ``attn_fwd_fp8(Qc, q_scale, Kc, k_scale, Vtc, v_scale, scale, causal)``: e4m3
  codes with one fp32 scale per 128-row block (V transposed) and the FP8
  forward on them (d = 128); ``attn_fp8_vt_stride(N)``
* ``attn_kv_tables(cached, added, free_pages, block_table, page_size, T)``,
  ``attn_kv_append_fp8(K, V, slots, k_pages, k_scale, v_pages, v_scale)`` and
  ``attn_fwd_paged_fp8(Q, k_pages, k_scale, v_pages, v_scale, block_table, cu_q, kv_lens, ...)``:
  a paged e4m3 key/value cache -- its block table and slot map from the requests'
  lengths, the quantizing append, and ragged attention over it;
  ``attn_fwd_paged_workspace_size(R, T, Hq, Hkv, d)``
* ``attn_rope_freqs(rot, base=10000.0, scaling="none", ...) -> (freqs, amplitude)``,
  ``attn_rope(Q, K, freqs, positions=None, ...) -> (Q_out, K_out)`` and
  ``attn_rope_bwd(dQ, dK, freqs, positions=None, ...)``: rotary positions and their
  gradient, for ``[B, H, N, d]`` and ``[T, H, d]`` tensors of any strides;
  ``attn_kv_append_rope_fp8(Q, K, V, positions, slots, freqs, k_pages, ...) -> Q_out``:
  the paged append with them applied on the way
* ``attn_bwd(Q, K, V, O, dO, LSE, scale, causal) -> (dQ, dK, dV)``
* ``attn_bwd_workspace_size(B, Hq, Hkv, N, d)``
* ``attn_fwd_dropout(Q, K, V, p, rng, scale, causal) -> (O, LSE)`` and
  ``attn_bwd_dropout(Q, K, V, O, dO, LSE, p, rng, scale, causal) -> (dQ, dK, dV)``: with
  dropout on the softmax, from a counter-based generator (seed and offset in ``rng``);
  ``attn_bwd_dropout_workspace_size(B, Hq, Hkv, N, d, causal)``
* ``attn_last_device_status(stream=None)``, ``attn_status_string(code)``
* ``attn_selftest_wait_timeout(limit_ns)``, ``attn_selftest_paged_wait_timeout(limit_ns)``

Tensors are ``[B, H, N, d]`` contiguous CUDA tensors (bf16, or fp32 for the
fp32 forward); ``LSE`` is ``[B, Hq, N]`` fp32.
"""

from __future__ import annotations

import ctypes
import importlib.util
import math
import os
import threading
import warnings

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# ATTN_DEBUG=1 selects the debug build (python -m exact_attention_95_gb300.build
# --debug): the same kernels with explicit bounds checks on tensor-copy
# coordinates and store indices, reported through attn_last_device_status as
# ATTN_ERR_DEVICE instead of an access out of bounds.
LIB_PATH = os.path.join(_HERE, "libattn_sm103_debug.so" if os.environ.get("ATTN_DEBUG") == "1"
                        else "libattn_sm103.so")

ATTN_OK, ATTN_ERR_INVALID_ARG, ATTN_ERR_UNSUPPORTED = 0, 1, 2
ATTN_ERR_CUDA, ATTN_ERR_TIMEOUT, ATTN_ERR_DEVICE = 3, 4, 5
ATTN_BF16, ATTN_F32 = 0, 1

EXPORTED = ("attn_fwd", "attn_fwd_split", "attn_fwd_split_workspace_size", "attn_fwd_masked",
            "attn_bwd_masked", "attn_quantize_fp8", "attn_fp8_vt_stride", "attn_fwd_fp8", "attn_bwd",
            "attn_bwd_preprocess", "attn_bwd_main", "attn_bwd_convert", "attn_bwd_workspace_size",
            "attn_kv_tables", "attn_kv_append_fp8", "attn_fwd_paged_fp8", "attn_fwd_paged_workspace_size",
            "attn_fwd_dropout", "attn_bwd_dropout", "attn_bwd_dropout_workspace_size", "attn_rope_freqs", "attn_rope", "attn_rope_bwd", "attn_kv_append_rope_fp8",
            "attn_status_string", "attn_last_device_status", "attn_selftest_wait_timeout",
            "attn_selftest_paged_wait_timeout")
_BWD_STAGES = {"all": "attn_bwd", "preprocess": "attn_bwd_preprocess", "main": "attn_bwd_main",
               "convert": "attn_bwd_convert"}

_lock = threading.Lock()
_lib = None
_fast = None  # the extension module, bound to the loaded library; False where there is none


class _Rows(ctypes.Structure):
    """attn_rows: rows of d elements and the elements between them."""

    _fields_ = [("data", ctypes.c_void_p), ("batch", ctypes.c_longlong), ("head", ctypes.c_longlong),
                ("token", ctypes.c_longlong)]


class AttnError(RuntimeError):
    def __init__(self, code: int, where: str):
        self.code = code
        super().__init__(f"{where}: {attn_status_string(code)}")


def load_library(path: str = LIB_PATH):
    """Load the CUDA library (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(
                f"CUDA library {path} is missing; build it with "
                "`python -m exact_attention_95_gb300.build` (there is no CPU fallback)")
        lib = ctypes.CDLL(path)
        vp, i32, f32, sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        lib.attn_fwd.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, i32, i32, i32, vp]
        lib.attn_fwd.restype = i32
        for fname in _BWD_STAGES.values():
            fn = getattr(lib, fname)
            fn.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, f32,
                           i32, i32, vp, sz, vp]
            fn.restype = i32
        lib.attn_fwd_split.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, f32, i32, i32, i32,
                                       vp, sz, vp]
        lib.attn_fwd_split.restype = i32
        lib.attn_fwd_split_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32, i32]
        lib.attn_fwd_split_workspace_size.restype = sz
        lib.attn_fwd_masked.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, i32, vp, i32, i32, vp]
        lib.attn_fwd_masked.restype = i32
        lib.attn_bwd_masked.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, i32,
                                        vp, i32, vp, sz, vp]
        lib.attn_bwd_masked.restype = i32
        lib.attn_fp8_vt_stride.argtypes = [i32]
        lib.attn_fp8_vt_stride.restype = i32
        lib.attn_quantize_fp8.argtypes = [vp, vp, vp, ctypes.c_longlong, i32, i32, i32, vp]
        lib.attn_quantize_fp8.restype = i32
        lib.attn_fwd_fp8.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, i32, i32, vp]
        lib.attn_fwd_fp8.restype = i32
        i64, f64 = ctypes.c_longlong, ctypes.c_double
        lib.attn_kv_tables.argtypes = [vp, vp, vp, i32, vp, i32, i32, vp, vp, vp, vp, vp, i32, i32, vp]
        lib.attn_kv_tables.restype = i32
        lib.attn_kv_append_fp8.argtypes = [vp, i64, vp, i64, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp]
        lib.attn_kv_append_fp8.restype = i32
        lib.attn_fwd_paged_fp8.argtypes = [vp, i64, vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32,
                                           i32, i32, f32, i32, i32, vp, sz, vp]
        lib.attn_fwd_paged_fp8.restype = i32
        lib.attn_fwd_paged_workspace_size.argtypes = [i32, i32, i32, i32, i32]
        lib.attn_fwd_paged_workspace_size.restype = sz
        lib.attn_fwd_dropout.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, i32, f32, vp, i32, vp]
        lib.attn_fwd_dropout.restype = i32
        lib.attn_bwd_dropout.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, i32, f32, vp,
                                         vp, sz, vp]
        lib.attn_bwd_dropout.restype = i32
        lib.attn_bwd_dropout_workspace_size.argtypes = [i32, i32, i32, i32, i32, i32]
        lib.attn_bwd_dropout_workspace_size.restype = sz
        rows = ctypes.POINTER(_Rows)
        for fn in (lib.attn_rope, lib.attn_rope_bwd):
            fn.argtypes = [rows, rows, rows, rows, vp, i64, vp, i32, i32, f32, i32, i32, i32, i32, i32, i32, vp]
            fn.restype = i32
        lib.attn_rope_freqs.argtypes = [vp, vp, i32, f64, i32, f64, f64, f64, f64]
        lib.attn_rope_freqs.restype = i32
        lib.attn_kv_append_rope_fp8.argtypes = [vp, i64, vp, i64, vp, i64, vp, vp, vp, i32, i32, f32, vp, i64, vp, vp,
                                                vp, vp, i32, i32, i32, i32, i32, i32, vp]
        lib.attn_kv_append_rope_fp8.restype = i32
        lib.attn_bwd_workspace_size.argtypes = [i32, i32, i32, i32, i32]
        lib.attn_bwd_workspace_size.restype = sz
        lib.attn_status_string.argtypes = [i32]
        lib.attn_status_string.restype = ctypes.c_char_p
        lib.attn_last_device_status.argtypes = [vp]
        lib.attn_last_device_status.restype = i32
        lib.attn_selftest_wait_timeout.argtypes = [ctypes.c_ulonglong, vp]
        lib.attn_selftest_wait_timeout.restype = i32
        lib.attn_selftest_paged_wait_timeout.argtypes = [ctypes.c_ulonglong, vp]
        lib.attn_selftest_paged_wait_timeout.restype = i32
        _lib = lib
        return lib


def _bound():
    """The extension module (csrc/binding.cpp) with the library loaded, at the first call that
    uses it; False, after a warning, where it cannot be loaded."""
    global _fast
    if _fast is not None:
        return _fast
    lib = load_library()
    with _lock:
        if _fast is None:
            from .build import binding_path
            try:
                spec = importlib.util.spec_from_file_location(__name__ + "._binding", binding_path())
                module = importlib.util.module_from_spec(spec)
                spec.loader.exec_module(module)
                module.bind(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
                    lib.attn_kv_tables, lib.attn_kv_append_fp8, lib.attn_fwd_paged_fp8,
                    lib.attn_fwd_paged_workspace_size, lib.attn_rope, lib.attn_rope_bwd,
                    lib.attn_kv_append_rope_fp8, lib.attn_fwd_dropout, lib.attn_bwd_dropout,
                    lib.attn_bwd_dropout_workspace_size)))
                _fast = module
            except ImportError as e:
                _fast = False
                warnings.warn(f"the paged calls make their checks in Python, which takes longer: {e} "
                              "(python -m exact_attention_95_gb300.build makes the module)", RuntimeWarning, stacklevel=3)
    return _fast


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr())


def _check_tensor(name, t, dtype, shape, device=None):
    """Placement, dtype, shape and contiguity of a tensor handed to the library.

    Outputs are checked like inputs: a host tensor, a wrong dtype or shape
    would otherwise become a kernel's write target."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _check_workspace(ws, need, device):
    """A caller-given workspace: contiguous uint8 CUDA memory on `device`, at
    least `need` bytes."""
    if not isinstance(ws, torch.Tensor) or not ws.is_cuda:
        raise TypeError("workspace must be a CUDA tensor")
    if ws.device != device:
        raise ValueError(f"workspace is on {ws.device}, expected {device}")
    if ws.dtype != torch.uint8 or not ws.is_contiguous():
        raise TypeError("workspace must be a contiguous uint8 tensor")
    if ws.numel() < need:
        raise ValueError(f"workspace has {ws.numel()} bytes, needs {need}")


def _check_bwd_outputs(dQ, dK, dV, B, Hq, Hkv, N, d, device):
    bf = torch.bfloat16
    _check_tensor("dQ", dQ, bf, (B, Hq, N, d), device)
    _check_tensor("dK", dK, bf, (B, Hkv, N, d), device)
    _check_tensor("dV", dV, bf, (B, Hkv, N, d), device)


def attn_status_string(code: int) -> str:
    return load_library().attn_status_string(int(code)).decode()


def attn_bwd_workspace_size(B: int, Hq: int, Hkv: int, N: int, d: int) -> int:
    return int(load_library().attn_bwd_workspace_size(B, Hq, Hkv, N, d))


def attn_last_device_status(stream=None) -> int:
    return int(load_library().attn_last_device_status(_stream(stream)))


def attn_selftest_wait_timeout(limit_ns: int, stream=None) -> int:
    return int(load_library().attn_selftest_wait_timeout(int(limit_ns), _stream(stream)))


def attn_selftest_paged_wait_timeout(limit_ns: int, stream=None) -> int:
    return int(load_library().attn_selftest_paged_wait_timeout(int(limit_ns), _stream(stream)))


def attn_fwd(Q, K, V, scale=None, causal=False, out_dtype=None, O=None, LSE=None, stream=None):
    """O, LSE = softmax(scale Q K^T [+causal]) V and its row log-sum-exp."""
    lib = load_library()
    B, Hq, N, d = Q.shape
    Hkv = K.shape[1]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    in_dt = {torch.bfloat16: ATTN_BF16, torch.float32: ATTN_F32}.get(Q.dtype)
    if in_dt is None:
        raise TypeError("Q must be bf16 or fp32")
    if out_dtype is None:
        out_dtype = Q.dtype
    out_dt = {torch.bfloat16: ATTN_BF16, torch.float32: ATTN_F32}[out_dtype]
    _check_tensor("Q", Q, Q.dtype, (B, Hq, N, d))
    dev = Q.device
    _check_tensor("K", K, Q.dtype, (B, Hkv, N, d), dev)
    _check_tensor("V", V, Q.dtype, (B, Hkv, N, d), dev)
    if O is None:
        O = torch.empty((B, Hq, N, d), dtype=out_dtype, device=dev)
    if LSE is None:
        LSE = torch.empty((B, Hq, N), dtype=torch.float32, device=dev)
    _check_tensor("O", O, out_dtype, (B, Hq, N, d), dev)
    _check_tensor("LSE", LSE, torch.float32, (B, Hq, N), dev)
    with torch.cuda.device(dev):
        rc = lib.attn_fwd(_ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(LSE), B, Hq, Hkv, N, d,
                          float(scale), int(bool(causal)), in_dt, out_dt, _stream(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_fwd")
    return O, LSE


def attn_fwd_split_workspace_size(B: int, Hq: int, Hkv: int, Nq: int, Nk: int, d: int,
                                  num_splits: int = 0) -> int:
    return int(load_library().attn_fwd_split_workspace_size(B, Hq, Hkv, Nq, Nk, d, num_splits))


def attn_fwd_split(Q, K, V, scale=None, causal=False, num_splits=0, out_dtype=None, O=None, LSE=None,
                   workspace=None, stream=None):
    """O, LSE of attention with Nq = Q.shape[2] queries and Nk = K.shape[2] keys
    (bottom-right causal alignment when they differ), the key range cut into
    num_splits parts (0: chosen by the library) whose partial results are
    merged.  bf16 inputs; O bf16 (default) or fp32."""
    lib = load_library()
    B, Hq, Nq, d = Q.shape
    Hkv, Nk = K.shape[1], K.shape[2]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    bf = torch.bfloat16
    if out_dtype is None:
        out_dtype = bf
    out_dt = {torch.bfloat16: ATTN_BF16, torch.float32: ATTN_F32}[out_dtype]
    _check_tensor("Q", Q, bf, (B, Hq, Nq, d))
    dev = Q.device
    _check_tensor("K", K, bf, (B, Hkv, Nk, d), dev)
    _check_tensor("V", V, bf, (B, Hkv, Nk, d), dev)
    if O is None:
        O = torch.empty((B, Hq, Nq, d), dtype=out_dtype, device=dev)
    if LSE is None:
        LSE = torch.empty((B, Hq, Nq), dtype=torch.float32, device=dev)
    _check_tensor("O", O, out_dtype, (B, Hq, Nq, d), dev)
    _check_tensor("LSE", LSE, torch.float32, (B, Hq, Nq), dev)
    ws_bytes = attn_fwd_split_workspace_size(B, Hq, Hkv, Nq, Nk, d, num_splits)
    if workspace is None and ws_bytes > 0:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    if workspace is not None:
        _check_workspace(workspace, ws_bytes, dev)
    wptr = _ptr(workspace) if workspace is not None else ctypes.c_void_p(0)
    wbytes = workspace.numel() if workspace is not None else 0
    with torch.cuda.device(dev):
        rc = lib.attn_fwd_split(_ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(LSE), B, Hq, Hkv, Nq, Nk, d,
                                float(scale), int(bool(causal)), out_dt, int(num_splits), wptr, wbytes,
                                _stream(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_fwd_split")
    return O, LSE


def _check_mask(block_mask, Hq, N, device):
    T = (N + 127) // 128
    if not isinstance(block_mask, torch.Tensor) or not block_mask.is_cuda or block_mask.dtype != torch.uint8:
        raise TypeError("block_mask must be a uint8 CUDA tensor")
    if block_mask.device != device:
        raise ValueError(f"block_mask is on {block_mask.device}, expected {device}")
    m = block_mask if block_mask.dim() == 3 else block_mask.reshape(1, T, T)
    if tuple(m.shape[1:]) != (T, T) or m.shape[0] not in (1, Hq) or not m.is_contiguous():
        raise ValueError(f"block_mask must be contiguous [1 or {Hq}, {T}, {T}], got {tuple(block_mask.shape)}")
    return m, m.shape[0]


def attn_fwd_masked(Q, K, V, block_mask, scale=None, causal=False, out_dtype=None, O=None, LSE=None,
                    stream=None):
    """Block-sparse forward: block_mask[h, i, j] == 0 removes the 128 x 128 block
    (query tile i, key tile j) of head h (h = 0 for a mask shared by all heads)."""
    lib = load_library()
    B, Hq, N, d = Q.shape
    Hkv = K.shape[1]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    bf = torch.bfloat16
    out_dtype = bf if out_dtype is None else out_dtype
    out_dt = {torch.bfloat16: ATTN_BF16, torch.float32: ATTN_F32}[out_dtype]
    _check_tensor("Q", Q, bf, (B, Hq, N, d))
    dev = Q.device
    for name, t, H in (("K", K, Hkv), ("V", V, Hkv)):
        _check_tensor(name, t, bf, (B, H, N, d), dev)
    m, mh = _check_mask(block_mask, Hq, N, dev)
    O = torch.empty((B, Hq, N, d), dtype=out_dtype, device=dev) if O is None else O
    LSE = torch.empty((B, Hq, N), dtype=torch.float32, device=dev) if LSE is None else LSE
    _check_tensor("O", O, out_dtype, (B, Hq, N, d), dev)
    _check_tensor("LSE", LSE, torch.float32, (B, Hq, N), dev)
    with torch.cuda.device(dev):
        rc = lib.attn_fwd_masked(_ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(LSE), B, Hq, Hkv, N, d, float(scale),
                                 int(bool(causal)), _ptr(m), mh, out_dt, _stream(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_fwd_masked")
    return O, LSE


def attn_fp8_vt_stride(N: int) -> int:
    """Row length of transposed FP8 codes: N rounded up to 16."""
    return int(load_library().attn_fp8_vt_stride(int(N)))


def attn_quantize_fp8(X, transpose=False, codes=None, scales=None, stream=None):
    """Per-128-row-block e4m3 quantization of X [B, H, N, d] (bf16).

    Returns (codes, scales): codes uint8 [B, H, N, d], or with transpose
    [B, H, d, attn_fp8_vt_stride(N)]; scales fp32 [B, H, ceil(N / 128)]."""
    lib = load_library()
    B, H, N, d = X.shape
    _check_tensor("X", X, torch.bfloat16, (B, H, N, d))
    dev = X.device
    T = (N + 127) // 128
    cshape = (B, H, d, attn_fp8_vt_stride(N)) if transpose else (B, H, N, d)
    codes = torch.empty(cshape, dtype=torch.uint8, device=dev) if codes is None else codes
    scales = torch.empty((B, H, T), dtype=torch.float32, device=dev) if scales is None else scales
    _check_tensor("codes", codes, torch.uint8, cshape, dev)
    _check_tensor("scales", scales, torch.float32, (B, H, T), dev)
    with torch.cuda.device(dev):
        rc = lib.attn_quantize_fp8(_ptr(X), _ptr(codes), _ptr(scales), B * H, N, d, int(bool(transpose)),
                                   _stream(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_quantize_fp8")
    return codes, scales


def attn_fwd_fp8(Qc, q_scale, Kc, k_scale, Vtc, v_scale, scale=None, causal=False, out_dtype=None, O=None,
                 LSE=None, stream=None):
    """FP8 forward on block-quantized Q, K and transposed V (see attn_quantize_fp8)."""
    lib = load_library()
    B, Hq, N, d = Qc.shape
    Hkv = Kc.shape[1]
    T = (N + 127) // 128
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    out_dtype = torch.bfloat16 if out_dtype is None else out_dtype
    out_dt = {torch.bfloat16: ATTN_BF16, torch.float32: ATTN_F32}[out_dtype]
    u8, f32 = torch.uint8, torch.float32
    _check_tensor("Qc", Qc, u8, (B, Hq, N, d))
    dev = Qc.device
    _check_tensor("Kc", Kc, u8, (B, Hkv, N, d), dev)
    _check_tensor("Vtc", Vtc, u8, (B, Hkv, d, attn_fp8_vt_stride(N)), dev)
    _check_tensor("q_scale", q_scale, f32, (B, Hq, T), dev)
    _check_tensor("k_scale", k_scale, f32, (B, Hkv, T), dev)
    _check_tensor("v_scale", v_scale, f32, (B, Hkv, T), dev)
    O = torch.empty((B, Hq, N, d), dtype=out_dtype, device=dev) if O is None else O
    LSE = torch.empty((B, Hq, N), dtype=f32, device=dev) if LSE is None else LSE
    _check_tensor("O", O, out_dtype, (B, Hq, N, d), dev)
    _check_tensor("LSE", LSE, f32, (B, Hq, N), dev)
    with torch.cuda.device(dev):
        rc = lib.attn_fwd_fp8(_ptr(Qc), _ptr(q_scale), _ptr(Kc), _ptr(k_scale), _ptr(Vtc), _ptr(v_scale),
                              _ptr(O), _ptr(LSE), B, Hq, Hkv, N, d, float(scale), int(bool(causal)), out_dt,
                              _stream(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_fwd_fp8")
    return O, LSE


# ---------------------------------------------------------------- paged 8-bit cache
# A decoding step makes these calls once a layer, on kernels of a few
# microseconds, so the extension module checks, allocates and calls first; where
# it finds an argument that is not as it has to be it returns None, and the
# checks below say what is wrong.  A call on a named stream takes this way too.
def _cuda_device(name, t):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    return t.device


def _call(fn, *args):
    """fn(*args, current stream) of the current device."""
    rc = fn(*args, torch.cuda.current_stream().cuda_stream)
    if rc != ATTN_OK:
        raise AttnError(rc, fn.__name__)


def _on(dev, stream):
    """A context with `dev` and `stream` (None: dev's current one) current, so
    that what a call allocates belongs to the stream that it runs on."""
    if stream is None:
        return torch.cuda.device(dev)
    if stream.device != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on {dev}")
    return torch.cuda.stream(stream)


def _result(r, where):
    if type(r) is int:
        raise AttnError(r, where)
    return r


def _check_tokens(name, t, heads, d, device):
    """A bf16 [T, heads, d] tensor whose tokens may be apart (a slice of a packed
    projection); returns the elements between tokens."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16}, got {t.dtype}")
    if t.dim() != 3 or t.shape[1] != heads or t.shape[2] != d:
        raise ValueError(f"{name} must have shape (T, {heads}, {d}), got {tuple(t.shape)}")
    st = t.stride()
    apart = st[0] if t.shape[0] > 1 else heads * d  # the stride of a single token says nothing
    if st[2] != 1 or (heads > 1 and st[1] != d) or apart < heads * d or apart % 8:
        raise ValueError(f"{name}: the rows of a token must be contiguous and tokens a multiple of 8 elements apart")
    return apart


def _check_cache(k_pages, k_scale, v_pages, v_scale, device):
    """Checks the pages and scales; returns (num_pages, Hkv, page_size, d)."""
    if not isinstance(k_pages, torch.Tensor) or k_pages.dim() != 4:
        raise TypeError("k_pages must be a 4-dimensional CUDA tensor")
    shape = k_pages.shape
    scales = shape[:2]
    _check_tensor("k_pages", k_pages, torch.uint8, shape, device)
    _check_tensor("v_pages", v_pages, torch.uint8, shape, device)
    _check_tensor("k_scale", k_scale, torch.float32, scales, device)
    _check_tensor("v_scale", v_scale, torch.float32, scales, device)
    return shape


def _check_table(block_table, device):
    if not isinstance(block_table, torch.Tensor) or block_table.dim() != 2:
        raise TypeError("block_table must be a CUDA tensor [R, max_pages]")
    _check_tensor("block_table", block_table, torch.int32, block_table.shape, device)
    return block_table.shape


def attn_kv_tables(cached, added, free_pages, block_table, page_size, T, kv_lens=None, cu_tokens=None, slots=None,
                   positions=None, taken=None, stream=None):
    """Block table entries and slot map of a step from the requests' lengths.

    cached, added int32 [R]; free_pages int32 [F]; block_table int32 [R, max_pages]
    (updated in place); T places for new tokens.  Returns (kv_lens [R], cu_tokens
    [R + 1], slots [T] int64, positions [T], taken [2]: pages taken from the head
    of free_pages, requests refused).  kv_lens, cu_tokens and taken may be views of one
    storage where the call makes them."""
    fast = stream is None and _bound()
    if fast:
        r = fast.kv_tables(cached, added, free_pages, block_table, page_size, T, kv_lens, cu_tokens, slots,
                           positions, taken)
        if r is not None:
            return _result(r, "attn_kv_tables")
    lib = load_library()
    i32 = torch.int32
    dev = _cuda_device("cached", cached)
    R, max_pages = _check_table(block_table, dev)
    _check_tensor("cached", cached, i32, (R,), dev)
    _check_tensor("added", added, i32, (R,), dev)
    _cuda_device("free_pages", free_pages)
    F = free_pages.numel()
    _check_tensor("free_pages", free_pages, i32, (F,), dev)
    with _on(dev, stream):
        empty = torch.empty
        kv_lens = empty(R, dtype=i32, device=dev) if kv_lens is None else kv_lens
        cu_tokens = empty(R + 1, dtype=i32, device=dev) if cu_tokens is None else cu_tokens
        slots = empty(T, dtype=torch.int64, device=dev) if slots is None else slots
        positions = empty(T, dtype=i32, device=dev) if positions is None else positions
        taken = empty(2, dtype=i32, device=dev) if taken is None else taken
        _check_tensor("kv_lens", kv_lens, i32, (R,), dev)
        _check_tensor("cu_tokens", cu_tokens, i32, (R + 1,), dev)
        _check_tensor("slots", slots, torch.int64, (T,), dev)
        _check_tensor("positions", positions, i32, (T,), dev)
        _check_tensor("taken", taken, i32, (2,), dev)
        _call(lib.attn_kv_tables, cached.data_ptr(), added.data_ptr(), free_pages.data_ptr(), F,
              block_table.data_ptr(), max_pages, int(page_size), kv_lens.data_ptr(), cu_tokens.data_ptr(),
              slots.data_ptr(), positions.data_ptr(), taken.data_ptr(), R, int(T))
    return kv_lens, cu_tokens, slots, positions, taken


def attn_kv_append_fp8(K, V, slots, k_pages, k_scale, v_pages, v_scale, stream=None):
    """Quantizes the new tokens' K, V [T, Hkv, d] (bf16) into the pages their slots name.

    k_pages, v_pages uint8 [num_pages, Hkv, page_size, d] and k_scale, v_scale fp32
    [num_pages, Hkv] are updated in place, and returned."""
    fast = stream is None and _bound()
    if fast:
        r = fast.kv_append_fp8(K, V, slots, k_pages, k_scale, v_pages, v_scale)
        if r is not None:
            return _result(r, "attn_kv_append_fp8")
    lib = load_library()
    dev = _cuda_device("K", K)
    num_pages, Hkv, page_size, d = _check_cache(k_pages, k_scale, v_pages, v_scale, dev)
    k_stride = _check_tokens("K", K, Hkv, d, dev)
    v_stride = _check_tokens("V", V, Hkv, d, dev)
    T = K.shape[0]
    if V.shape[0] != T:
        raise ValueError(f"V has {V.shape[0]} tokens, K has {T}")
    _check_tensor("slots", slots, torch.int64, (T,), dev)
    with _on(dev, stream):
        _call(lib.attn_kv_append_fp8, K.data_ptr(), k_stride, V.data_ptr(), v_stride, slots.data_ptr(),
              k_pages.data_ptr(), k_scale.data_ptr(), v_pages.data_ptr(), v_scale.data_ptr(), T, Hkv, d, num_pages,
              page_size)
    return k_pages, k_scale, v_pages, v_scale


def attn_fwd_paged_workspace_size(R: int, T: int, Hq: int, Hkv: int, d: int) -> int:
    """Bytes of attn_fwd_paged_fp8's workspace.  A workspace for several steps has the largest
    of their sizes: a decoding step (T <= R, Hq / Hkv <= 8) needs less than one of fewer
    requests with more tokens."""
    return int(load_library().attn_fwd_paged_workspace_size(R, T, Hq, Hkv, d))


def attn_fwd_paged_fp8(Q, k_pages, k_scale, v_pages, v_scale, block_table, cu_q, kv_lens, scale=None, causal=False,
                       out_dtype=None, O=None, LSE=None, workspace=None, stream=None):
    """O [T, Hq, d], LSE [T, Hq] of ragged queries over the paged cache.

    Q bf16 [T, Hq, d]; request r's queries are tokens cu_q[r] .. cu_q[r + 1] - 1 and
    its keys the first kv_lens[r] tokens of the pages that block_table[r] names
    (bottom-right causal alignment).  Rows behind cu_q[R] are not written."""
    if out_dtype is None:
        out_dtype = torch.bfloat16
    out_dt = {torch.bfloat16: ATTN_BF16, torch.float32: ATTN_F32}[out_dtype]
    fast = stream is None and _bound()
    if fast:
        r = fast.fwd_paged_fp8(Q, k_pages, k_scale, v_pages, v_scale, block_table, cu_q, kv_lens, scale, causal,
                               out_dt, O, LSE, workspace)
        if r is not None:
            return _result(r, "attn_fwd_paged_fp8")
    lib = load_library()
    dev = _cuda_device("Q", Q)
    if Q.dim() != 3:
        raise ValueError(f"Q must have shape (T, Hq, d), got {tuple(Q.shape)}")
    T, Hq, d = Q.shape
    q_stride = _check_tokens("Q", Q, Hq, d, dev)
    num_pages, Hkv, page_size, dk = _check_cache(k_pages, k_scale, v_pages, v_scale, dev)
    if dk != d:
        raise ValueError(f"the pages have d = {dk}, Q has {d}")
    R, max_pages = _check_table(block_table, dev)
    i32 = torch.int32
    _check_tensor("cu_q", cu_q, i32, (R + 1,), dev)
    _check_tensor("kv_lens", kv_lens, i32, (R,), dev)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    with _on(dev, stream):
        O = torch.empty((T, Hq, d), dtype=out_dtype, device=dev) if O is None else O
        LSE = torch.empty((T, Hq), dtype=torch.float32, device=dev) if LSE is None else LSE
        _check_tensor("O", O, out_dtype, (T, Hq, d), dev)
        _check_tensor("LSE", LSE, torch.float32, (T, Hq), dev)
        need = int(lib.attn_fwd_paged_workspace_size(R, T, Hq, Hkv, d))
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        _check_workspace(workspace, need, dev)
        _call(lib.attn_fwd_paged_fp8, Q.data_ptr(), q_stride, k_pages.data_ptr(), k_scale.data_ptr(),
              v_pages.data_ptr(), v_scale.data_ptr(), block_table.data_ptr(), cu_q.data_ptr(), kv_lens.data_ptr(),
              O.data_ptr(), LSE.data_ptr(), R, T, Hq, Hkv, d, num_pages, page_size, max_pages, float(scale),
              int(bool(causal)), out_dt, workspace.data_ptr(), workspace.numel())
    return O, LSE


# ---------------------------------------------------------------- rotary positions
_SCALINGS = {"none": 0, "linear": 1, "base": 2, "parts": 3}


def attn_rope_freqs(rot, base=10000.0, scaling="none", factor=1.0, original_len=0.0, low=1.0, high=32.0, device="cuda"):
    """(freqs, amplitude) for attn_rope: turns a position of each of rot / 2 pairs, as int64
    in units of 2^-64 turn, and what the rotated elements are multiplied with.

    scaling: "none"; for contexts `factor` times longer "linear" (positions divided),
    "base" (the base raised), or "parts" (pairs that turn at most `low` times over
    original_len positions divided, those that turn `high` times left, a ramp between).

    Frequencies from elsewhere, w radians a position in float64 (below pi), are
    (w / (2 * math.pi) * 2.0 ** 64).round().long()."""
    lib = load_library()
    if scaling not in _SCALINGS:
        raise ValueError(f"scaling must be one of {', '.join(_SCALINGS)}, got {scaling!r}")
    rot = int(rot)
    host = torch.empty(max(rot, 0) // 2, dtype=torch.int64)
    amplitude = ctypes.c_double()
    rc = lib.attn_rope_freqs(host.data_ptr(), ctypes.addressof(amplitude), rot, float(base), _SCALINGS[scaling],
                             float(factor), float(original_len), float(low), float(high))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_rope_freqs")
    return host.to(device), amplitude.value


def _rope_rows(name, t, shape, dtype, device):
    """attn_rows of a [T, H, d] or [B, H, N, d] tensor whose rows may be anywhere."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    st = t.stride()
    return _Rows(t.data_ptr(), *((0, st[1], st[0]) if t.dim() == 3 else st[:3]))


def _check_freqs(freqs, d, device):
    if not isinstance(freqs, torch.Tensor) or freqs.dim() != 1:
        raise TypeError("freqs must be a CUDA tensor [rot / 2] (attn_rope_freqs makes it)")
    _check_tensor("freqs", freqs, torch.int64, freqs.shape, device)
    rot = 2 * freqs.shape[0]
    if rot < 1 or rot > d:
        raise ValueError(f"freqs turns {rot} elements of {d}")
    return rot


def _rope(fname, q_name, k_name, Q, K, freqs, positions, interleaved, amplitude, Q_out, K_out, stream):
    fast = stream is None and _bound()
    if fast:
        r = fast.rope(fname == "attn_rope_bwd", Q, K, freqs, positions, interleaved, amplitude, Q_out, K_out)
        if r is not None:
            return _result(r, fname)
    lib = load_library()
    dev = _cuda_device(q_name, Q)
    dtype = {torch.bfloat16: ATTN_BF16, torch.float32: ATTN_F32}.get(Q.dtype)
    if dtype is None:
        raise TypeError(f"{q_name} must be bf16 or fp32")
    if Q.dim() not in (3, 4):
        raise ValueError(f"{q_name} must have shape (T, Hq, d) or (B, Hq, N, d), got {tuple(Q.shape)}")
    tokens = Q.dim() == 3
    B, Hq, N, d = (1, Q.shape[1], Q.shape[0], Q.shape[2]) if tokens else Q.shape
    q_shape = tuple(Q.shape)
    q = _rope_rows(q_name, Q, q_shape, Q.dtype, dev)
    k, k_shape, Hkv = None, None, 0
    if K is not None:
        if not isinstance(K, torch.Tensor) or K.dim() != Q.dim():
            raise TypeError(f"{k_name} must be a {Q.dim()}-dimensional CUDA tensor or None")
        Hkv = K.shape[1]
        k_shape = (N, Hkv, d) if tokens else (B, Hkv, N, d)
        k = _rope_rows(k_name, K, k_shape, Q.dtype, dev)
    elif K_out is not None:
        raise ValueError(f"{k_name}_out without {k_name}")
    rot = _check_freqs(freqs, d, dev)
    pos_batch = 0
    if positions is not None:
        if not isinstance(positions, torch.Tensor) or not positions.is_cuda:
            raise TypeError("positions must be a CUDA tensor")
        batched = not tokens and positions.dim() == 2
        _check_tensor("positions", positions, torch.int32, (B, N) if batched else (N,), dev)
        pos_batch = N if batched else 0
    with _on(dev, stream):
        Q_out = torch.empty(q_shape, dtype=Q.dtype, device=dev) if Q_out is None else Q_out
        qo = _rope_rows(q_name + "_out", Q_out, q_shape, Q.dtype, dev)
        ko = None
        if K is not None:
            K_out = torch.empty(k_shape, dtype=Q.dtype, device=dev) if K_out is None else K_out
            ko = _rope_rows(k_name + "_out", K_out, k_shape, Q.dtype, dev)
        if Q.numel() or (K is not None and K.numel()):
            _call(getattr(lib, fname), q, k, qo, ko, positions.data_ptr() if positions is not None else None, pos_batch,
                  freqs.data_ptr(), rot, int(bool(interleaved)), float(amplitude), B, Hq, Hkv, N, d, dtype)
    return Q_out, K_out


def attn_rope(Q, K, freqs, positions=None, interleaved=False, amplitude=1.0, Q_out=None, K_out=None, stream=None):
    """Rotary positions: Q [B, Hq, N, d] and K [B, Hkv, N, d], or [T, H, d] both (bf16 or
    fp32, of any strides between rows; K may be None), rotated into Q_out and K_out.

    freqs, amplitude: from attn_rope_freqs.  positions int32 [N] ([T]) or [B, N]; None:
    0 .. N - 1.  A token with a negative position is copied.  New outputs are contiguous;
    Q_out may be Q and K_out K."""
    return _rope("attn_rope", "Q", "K", Q, K, freqs, positions, interleaved, amplitude, Q_out, K_out, stream)


def attn_rope_bwd(dQ, dK, freqs, positions=None, interleaved=False, amplitude=1.0, dQ_out=None, dK_out=None,
                  stream=None):
    """The gradient of attn_rope: from those of its outputs to those of its inputs."""
    return _rope("attn_rope_bwd", "dQ", "dK", dQ, dK, freqs, positions, interleaved, amplitude, dQ_out, dK_out, stream)


def attn_kv_append_rope_fp8(Q, K, V, positions, slots, freqs, k_pages, k_scale, v_pages, v_scale, interleaved=False,
                            amplitude=1.0, Q_out=None, stream=None):
    """attn_kv_append_fp8 with the keys rotated before they are quantized; returns the
    queries [T, Hq, d] of the same tokens, rotated too (in Q_out; new: contiguous).

    positions int32 [T] as attn_kv_tables writes them (negative: not rotated); freqs,
    interleaved and amplitude as for attn_rope."""
    fast = stream is None and _bound()
    if fast:
        r = fast.kv_append_rope_fp8(Q, K, V, positions, slots, freqs, k_pages, k_scale, v_pages, v_scale, interleaved,
                                    amplitude, Q_out)
        if r is not None:
            return _result(r, "attn_kv_append_rope_fp8")
    lib = load_library()
    dev = _cuda_device("K", K)
    num_pages, Hkv, page_size, d = _check_cache(k_pages, k_scale, v_pages, v_scale, dev)
    k_stride = _check_tokens("K", K, Hkv, d, dev)
    v_stride = _check_tokens("V", V, Hkv, d, dev)
    if not isinstance(Q, torch.Tensor) or Q.dim() != 3:
        raise TypeError("Q must be a CUDA tensor (T, Hq, d)")
    T, Hq = K.shape[0], Q.shape[1]
    q_stride = _check_tokens("Q", Q, Hq, d, dev)
    for name, t in (("Q", Q), ("V", V)):
        if t.shape[0] != T:
            raise ValueError(f"{name} has {t.shape[0]} tokens, K has {T}")
    _check_tensor("positions", positions, torch.int32, (T,), dev)
    _check_tensor("slots", slots, torch.int64, (T,), dev)
    rot = _check_freqs(freqs, d, dev)
    with _on(dev, stream):
        Q_out = torch.empty((T, Hq, d), dtype=torch.bfloat16, device=dev) if Q_out is None else Q_out
        qo_stride = _check_tokens("Q_out", Q_out, Hq, d, dev)
        if Q_out.shape[0] != T:
            raise ValueError(f"Q_out has {Q_out.shape[0]} tokens, K has {T}")
        _call(lib.attn_kv_append_rope_fp8, Q.data_ptr(), q_stride, K.data_ptr(), k_stride, V.data_ptr(), v_stride,
              positions.data_ptr(), slots.data_ptr(), freqs.data_ptr(), rot, int(bool(interleaved)), float(amplitude),
              Q_out.data_ptr(), qo_stride, k_pages.data_ptr(), k_scale.data_ptr(), v_pages.data_ptr(),
              v_scale.data_ptr(), T, Hq, Hkv, d, num_pages, page_size)
    return Q_out


def _bwd_inputs(Q, K, V, O, dO, LSE):
    """Checks the backward's inputs; returns (B, Hq, Hkv, N, d, device)."""
    B, Hq, N, d = Q.shape
    Hkv = K.shape[1]
    bf = torch.bfloat16
    _check_tensor("Q", Q, bf, (B, Hq, N, d))
    dev = Q.device
    for name, t, H in (("K", K, Hkv), ("V", V, Hkv), ("O", O, Hq), ("dO", dO, Hq)):
        _check_tensor(name, t, bf, (B, H, N, d), dev)
    _check_tensor("LSE", LSE, torch.float32, (B, Hq, N), dev)
    return B, Hq, Hkv, N, d, dev


def attn_bwd_masked(Q, K, V, O, dO, LSE, block_mask, scale=None, causal=False, dQ=None, dK=None, dV=None,
                    workspace=None, stream=None):
    """Block-sparse backward with the mask of attn_fwd_masked."""
    lib = load_library()
    B, Hq, Hkv, N, d, dev = _bwd_inputs(Q, K, V, O, dO, LSE)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    m, mh = _check_mask(block_mask, Hq, N, dev)
    dQ = torch.empty_like(Q) if dQ is None else dQ
    dK = torch.empty_like(K) if dK is None else dK
    dV = torch.empty_like(V) if dV is None else dV
    _check_bwd_outputs(dQ, dK, dV, B, Hq, Hkv, N, d, dev)
    ws_bytes = attn_bwd_workspace_size(B, Hq, Hkv, N, d)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
    _check_workspace(workspace, ws_bytes, dev)
    with torch.cuda.device(dev):
        rc = lib.attn_bwd_masked(_ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(dO), _ptr(LSE), _ptr(dQ), _ptr(dK),
                                 _ptr(dV), B, Hq, Hkv, N, d, float(scale), int(bool(causal)), _ptr(m), mh,
                                 _ptr(workspace), workspace.numel(), _stream(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_bwd_masked")
    return dQ, dK, dV


def attn_bwd(Q, K, V, O, dO, LSE, scale=None, causal=False, dQ=None, dK=None, dV=None,
             workspace=None, stream=None, stage="all"):
    """dQ, dK, dV of O = attention(Q, K, V) given dO and the forward's LSE.

    ``stage`` selects one of the C entry points: "all" (attn_bwd) or one of
    "preprocess", "main", "convert" (run in that order with the same
    workspace to obtain the same result)."""
    lib = load_library()
    B, Hq, Hkv, N, d, dev = _bwd_inputs(Q, K, V, O, dO, LSE)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dQ = torch.empty_like(Q) if dQ is None else dQ
    dK = torch.empty_like(K) if dK is None else dK
    dV = torch.empty_like(V) if dV is None else dV
    _check_bwd_outputs(dQ, dK, dV, B, Hq, Hkv, N, d, dev)
    ws_bytes = attn_bwd_workspace_size(B, Hq, Hkv, N, d)
    if workspace is None:
        workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
    _check_workspace(workspace, ws_bytes, dev)
    fname = _BWD_STAGES[stage]
    with torch.cuda.device(dev):
        rc = getattr(lib, fname)(_ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(dO), _ptr(LSE), _ptr(dQ),
                                 _ptr(dK), _ptr(dV), B, Hq, Hkv, N, d, float(scale),
                                 int(bool(causal)), ATTN_BF16, _ptr(workspace), workspace.numel(),
                                 _stream(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, fname)
    return dQ, dK, dV


# ---------------------------------------------------------------- dropout
def _check_rng(rng, device):
    if not isinstance(rng, torch.Tensor):
        raise TypeError("rng must be a CUDA tensor [2] (seed, offset)")
    _check_tensor("rng", rng, torch.int64, (2,), device)


def attn_fwd_dropout(Q, K, V, p, rng, scale=None, causal=False, out_dtype=None, O=None, LSE=None, stream=None):
    """attn_fwd (bf16) with elements of the softmax dropped with probability p, rounded to a
    multiple of 1/256 (so nothing is dropped below 1/512; from 511/512 on p is refused).

    rng int64 [2] on the device: seed, and an offset (its low 32 bits count) that tells calls of
    one seed apart; read when the kernels run.  The mask follows from them and is
    never stored; LSE is that without dropout."""
    bf = torch.bfloat16
    out_dtype = bf if out_dtype is None else out_dtype
    out_dt = {torch.bfloat16: ATTN_BF16, torch.float32: ATTN_F32}[out_dtype]
    fast = stream is None and _bound()
    if fast:
        r = fast.fwd_dropout(Q, K, V, p, rng, scale, causal, out_dt, O, LSE)
        if r is not None:
            return _result(r, "attn_fwd_dropout")
    lib = load_library()
    B, Hq, N, d = Q.shape
    Hkv = K.shape[1]
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    _check_tensor("Q", Q, bf, (B, Hq, N, d))
    dev = Q.device
    _check_tensor("K", K, bf, (B, Hkv, N, d), dev)
    _check_tensor("V", V, bf, (B, Hkv, N, d), dev)
    _check_rng(rng, dev)
    with _on(dev, stream):
        O = torch.empty((B, Hq, N, d), dtype=out_dtype, device=dev) if O is None else O
        LSE = torch.empty((B, Hq, N), dtype=torch.float32, device=dev) if LSE is None else LSE
        _check_tensor("O", O, out_dtype, (B, Hq, N, d), dev)
        _check_tensor("LSE", LSE, torch.float32, (B, Hq, N), dev)
        _call(lib.attn_fwd_dropout, Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(), LSE.data_ptr(), B, Hq, Hkv, N,
              d, float(scale), int(bool(causal)), float(p), rng.data_ptr(), out_dt)
    return O, LSE


def attn_bwd_dropout_workspace_size(B: int, Hq: int, Hkv: int, N: int, d: int, causal: bool = False) -> int:
    """Bytes for attn_bwd_dropout.  They do not grow with N throughout: a workspace for several lengths has the
    largest of their sizes."""
    return int(load_library().attn_bwd_dropout_workspace_size(B, Hq, Hkv, N, d, int(bool(causal))))


def attn_bwd_dropout(Q, K, V, O, dO, LSE, p, rng, scale=None, causal=False, dQ=None, dK=None, dV=None, workspace=None,
                     stream=None):
    """dQ, dK, dV of attn_fwd_dropout's O, given dO and the forward's O, LSE, p and numbers in rng."""
    fast = stream is None and _bound()
    if fast:
        r = fast.bwd_dropout(Q, K, V, O, dO, LSE, p, rng, scale, causal, dQ, dK, dV, workspace)
        if r is not None:
            return _result(r, "attn_bwd_dropout")
    lib = load_library()
    B, Hq, Hkv, N, d, dev = _bwd_inputs(Q, K, V, O, dO, LSE)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    _check_rng(rng, dev)
    with _on(dev, stream):
        dQ = torch.empty_like(Q) if dQ is None else dQ
        dK = torch.empty_like(K) if dK is None else dK
        dV = torch.empty_like(V) if dV is None else dV
        _check_bwd_outputs(dQ, dK, dV, B, Hq, Hkv, N, d, dev)
        ws_bytes = attn_bwd_dropout_workspace_size(B, Hq, Hkv, N, d, causal)
        if workspace is None:
            workspace = torch.empty(max(ws_bytes, 1), dtype=torch.uint8, device=dev)
        _check_workspace(workspace, ws_bytes, dev)
        _call(lib.attn_bwd_dropout, Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(), dO.data_ptr(), LSE.data_ptr(),
              dQ.data_ptr(), dK.data_ptr(), dV.data_ptr(), B, Hq, Hkv, N, d, float(scale), int(bool(causal)), float(p),
              rng.data_ptr(), workspace.data_ptr(), workspace.numel())
    return dQ, dK, dV


# ---------------------------------------------------------------- no-alloc backward
EXPORTED = EXPORTED + ("attn_bwd_noalloc",)
NOALLOC_SCRATCH_BYTES = 32 * 1024 * 1024


def attn_bwd_noalloc(Q, K, V, O, dO, LSE, scale=None, causal=False, dQ=None, dK=None, dV=None,
                     stream=None):
    """attn_bwd with the library's fixed scratch array instead of a workspace.

    For callers that cannot allocate device memory where they run the
    backward.  The C call allocates nothing; problems whose workspace would
    exceed NOALLOC_SCRATCH_BYTES are rejected (ATTN_ERR_UNSUPPORTED).  Calls on
    one device share the scratch array: do not let them overlap on the GPU.
    (Here the outputs are allocated by PyTorch unless given.)"""
    lib = load_library()
    fn = lib.attn_bwd_noalloc
    vp, i32, f32 = ctypes.c_void_p, ctypes.c_int, ctypes.c_float
    fn.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, f32, i32, i32, vp]
    fn.restype = i32
    B, Hq, Hkv, N, d, dev = _bwd_inputs(Q, K, V, O, dO, LSE)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    dQ = torch.empty_like(Q) if dQ is None else dQ
    dK = torch.empty_like(K) if dK is None else dK
    dV = torch.empty_like(V) if dV is None else dV
    _check_bwd_outputs(dQ, dK, dV, B, Hq, Hkv, N, d, dev)
    with torch.cuda.device(dev):
        rc = fn(_ptr(Q), _ptr(K), _ptr(V), _ptr(O), _ptr(dO), _ptr(LSE), _ptr(dQ), _ptr(dK), _ptr(dV),
                B, Hq, Hkv, N, d, float(scale), int(bool(causal)), ATTN_BF16, _stream(stream))
    if rc != ATTN_OK:
        raise AttnError(rc, "attn_bwd_noalloc")
    return dQ, dK, dV
