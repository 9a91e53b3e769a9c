"""GGML Q2_K weight-quantized matmul, dequantize and embedding gather on GB300.

A thin ctypes binding over the C ABI of ``libq2k.so`` (declared in
``include/q2k.h``).  It only marshals arguments: every step of the work runs in
the library's CUDA kernels on the tensors' device, on PyTorch's current stream.
PyTorch supplies device memory and streams, nothing else.  There is no CPU
fallback: if the library has not been built (``ggml_q2_quantized_gb300.build``)
or no sm_103 device is present, the calls raise.

Names follow the mlx-native page "tests/deepseek_q2_k.rs": ``matmul`` is
``quantized_matmul_ggml`` (with ``path=`` playing the role of
``dispatch_mm_for_test``), ``embedding_gather`` is ``embedding_gather_q2_k`` and
``dequantize`` is ``test_only_dequantize``.
"""

from __future__ import annotations

import collections
import ctypes
import importlib.util
import os
import re
import threading
import warnings

from . import build as _build

QK_K = 256
BLOCK_BYTES = 84
GGML_TYPE_Q2_K = 10

PATH_AUTO, PATH_GEMV, PATH_TENSOR = 0, 1, 2
FLAG_CONST_WEIGHTS = 1
FLAG_INDEPENDENT = 2
ID_SLOTTED = 1
DTYPE_F32, DTYPE_BF16 = 0, 1
ACT_SILU, ACT_GELU, ACT_NONE = 0, 1, 2
MOE_MAX_EXPERTS = 4096
_ACTS = {"silu": ACT_SILU, "gelu": ACT_GELU}
_LINEAR_ACTS = {**_ACTS, None: ACT_NONE}
_PATHS = {"auto": PATH_AUTO, "gemv": PATH_GEMV, "tensor": PATH_TENSOR,
          PATH_AUTO: PATH_AUTO, PATH_GEMV: PATH_GEMV, PATH_TENSOR: PATH_TENSOR}

STATUS = {0: "Q2K_OK", 1: "Q2K_ERR_INVALID_ARGUMENT", 2: "Q2K_ERR_BAD_ID",
          3: "Q2K_ERR_CUDA", 4: "Q2K_ERR_TIMEOUT", 5: "Q2K_ERR_NO_DEVICE", 6: "Q2K_ERR_IO"}

HEADER = os.path.join(_build.INCLUDE, "q2k.h")
LIB_PATH = _build.LIB_PATH


class Q2KError(RuntimeError):
    """A non-OK status from libq2k, with its message."""

    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status
        self.message = message


class InvalidArgument(Q2KError, ValueError):
    pass


class MatmulParams(ctypes.Structure):
    _fields_ = [("m", ctypes.c_uint32), ("n", ctypes.c_uint32), ("k", ctypes.c_uint32),
                ("ggml_type", ctypes.c_uint32)]


class MatmulIdParams(ctypes.Structure):
    _fields_ = [("n_tokens", ctypes.c_uint32), ("top_k", ctypes.c_uint32), ("n", ctypes.c_uint32),
                ("k", ctypes.c_uint32), ("n_experts", ctypes.c_uint32),
                ("ggml_type", ctypes.c_uint32), ("expert_stride", ctypes.c_uint64)]


class GgufTensor(ctypes.Structure):
    _fields_ = [("ggml_type", ctypes.c_uint32), ("n_dims", ctypes.c_uint32),
                ("dims", ctypes.c_uint64 * 4), ("n_elements", ctypes.c_uint64),
                ("offset", ctypes.c_uint64), ("byte_len", ctypes.c_uint64)]


class MatmulCall(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("x_elems", ctypes.c_size_t), ("w", ctypes.c_void_p),
                ("w_bytes", ctypes.c_size_t), ("y", ctypes.c_void_p), ("y_elems", ctypes.c_size_t),
                ("params", MatmulParams), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t), ("path", ctypes.c_uint32),
                ("flags", ctypes.c_uint32)]


class EmbeddingParams(ctypes.Structure):
    _fields_ = [("vocab_size", ctypes.c_uint32), ("embed_dim", ctypes.c_uint32),
                ("n_tokens", ctypes.c_uint32), ("ggml_type", ctypes.c_uint32)]


class GatedFfnParams(ctypes.Structure):
    _fields_ = [("m", ctypes.c_uint32), ("n", ctypes.c_uint32), ("k", ctypes.c_uint32),
                ("ggml_type", ctypes.c_uint32), ("dtype", ctypes.c_uint32),
                ("act", ctypes.c_uint32)]


class LoraParams(ctypes.Structure):
    _fields_ = [("m", ctypes.c_uint32), ("n", ctypes.c_uint32), ("k", ctypes.c_uint32),
                ("ggml_type", ctypes.c_uint32), ("dtype", ctypes.c_uint32),
                ("rank", ctypes.c_uint32), ("n_adapters", ctypes.c_uint32),
                ("reserved", ctypes.c_uint32)]


class LinearParams(ctypes.Structure):
    _fields_ = [("m", ctypes.c_uint32), ("n", ctypes.c_uint32), ("k", ctypes.c_uint32),
                ("ggml_type", ctypes.c_uint32), ("dtype", ctypes.c_uint32),
                ("act", ctypes.c_uint32), ("n_experts", ctypes.c_uint32),
                ("reserved", ctypes.c_uint32)]


class MoeParams(ctypes.Structure):
    _fields_ = [("n_tokens", ctypes.c_uint32), ("top_k", ctypes.c_uint32),
                ("n_experts", ctypes.c_uint32), ("width", ctypes.c_uint32),
                ("dtype", ctypes.c_uint32), ("reserved", ctypes.c_uint32)]


class Routes(collections.namedtuple("Routes", "rows order offsets")):
    """What ``moe_route`` returns, int32 CUDA tensors: ``rows`` ``[n_tokens, top_k]``,
    each choice's place in expert order; ``order`` ``[n_tokens * top_k]``, the choice
    ``token * top_k + slot`` at each place; ``offsets`` ``[n_experts + 1]``, where each
    expert's places begin and the last one's end (behind it: choices without one)."""

    __slots__ = ()

    @property
    def n_experts(self) -> int:
        return self.offsets.shape[0] - 1


_lock = threading.Lock()
_lib = None


def header_functions() -> list[str]:
    """Names of the functions ``include/q2k.h`` declares."""
    with open(HEADER) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return re.findall(r"^\s*(?:const\s+)?[\w]+\s*\*?\s*(q2k_\w+)\s*\(", text, flags=re.M)


def load(path: str | None = None) -> ctypes.CDLL:
    """Load the in-tree libq2k.so (built by ``build.build()``); raise if absent."""
    global _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(
                f"libq2k is not built ({p} missing): run ggml_q2_quantized_gb300.build.build() "
                "- there is no fallback implementation")
        lib = ctypes.CDLL(p)
        vp, sz, u32p = ctypes.c_void_p, ctypes.c_size_t, ctypes.POINTER(ctypes.c_uint32)
        lib.q2k_dequantize.argtypes = [vp, sz, vp, sz, vp]
        lib.q2k_embedding_gather.argtypes = [vp, sz, vp, vp, sz, ctypes.POINTER(EmbeddingParams),
                                             vp, vp]
        lib.q2k_matmul.argtypes = [vp, sz, vp, sz, vp, sz, ctypes.POINTER(MatmulParams), vp]
        lib.q2k_matmul_path.argtypes = [ctypes.c_int, vp, sz, vp, sz, vp, sz,
                                        ctypes.POINTER(MatmulParams), vp]
        lib.q2k_matmul_ex.argtypes = [ctypes.c_int, ctypes.c_uint32, vp, sz, vp, sz, vp, sz,
                                      ctypes.POINTER(MatmulParams), vp, sz, vp]
        lib.q2k_matmul_workspace_bytes.argtypes = [ctypes.POINTER(MatmulParams), ctypes.c_int]
        lib.q2k_matmul_workspace_bytes.restype = ctypes.c_size_t
        lib.q2k_matmul_batched_mv.argtypes = [vp, sz, vp, sz, vp, sz, ctypes.c_uint32,
                                              ctypes.c_uint32, ctypes.c_uint32, ctypes.c_uint32,
                                              vp, sz, vp]
        lib.q2k_matmul_id.argtypes = [vp, sz, vp, sz, vp, vp, sz, ctypes.POINTER(MatmulIdParams),
                                      vp, vp, sz, vp]
        lib.q2k_matmul_id_slotted.argtypes = lib.q2k_matmul_id.argtypes
        lib.q2k_matmul_id_pair.argtypes = [vp, sz, vp, sz, vp, sz, vp, vp, vp, sz,
                                           ctypes.POINTER(MatmulIdParams), vp, vp, sz, vp]
        lib.q2k_matmul_id_ex.argtypes = [ctypes.c_int, ctypes.c_uint32, vp, sz, vp, sz, vp, vp, sz,
                                         ctypes.POINTER(MatmulIdParams), vp, vp, sz, vp]
        lib.q2k_matmul_id_pair_ex.argtypes = [ctypes.c_int, vp, sz, vp, sz, vp, sz, vp, vp, vp, sz,
                                              ctypes.POINTER(MatmulIdParams), vp, vp, sz, vp]
        lib.q2k_matmul_id_workspace_bytes.argtypes = [ctypes.c_int, ctypes.c_uint32,
                                                      ctypes.POINTER(MatmulIdParams)]
        lib.q2k_matmul_id_workspace_bytes.restype = sz
        lib.q2k_x_planes_bytes.argtypes = [ctypes.c_uint32, ctypes.c_uint32]
        lib.q2k_x_planes_bytes.restype = sz
        lib.q2k_gguf_open.argtypes = [ctypes.c_char_p, ctypes.POINTER(vp)]
        lib.q2k_gguf_close.argtypes = [vp]
        lib.q2k_gguf_close.restype = None
        lib.q2k_gguf_tensor_count.argtypes = [vp]
        lib.q2k_gguf_tensor_count.restype = ctypes.c_uint64
        lib.q2k_gguf_tensor_name.argtypes = [vp, ctypes.c_uint64]
        lib.q2k_gguf_tensor_name.restype = ctypes.c_char_p
        lib.q2k_gguf_tensor_info.argtypes = [vp, ctypes.c_char_p, ctypes.POINTER(GgufTensor)]
        lib.q2k_gguf_read_tensor.argtypes = [vp, ctypes.c_char_p, vp, sz]
        lib.q2k_matmul_ex_batch.argtypes = [ctypes.POINTER(MatmulCall), sz, vp, sz, vp]
        lib.q2k_matmul_batch_scratch_bytes.argtypes = [ctypes.POINTER(MatmulCall), sz]
        lib.q2k_matmul_batch_scratch_bytes.restype = sz
        gfp, lop, u32 = ctypes.POINTER(GatedFfnParams), ctypes.POINTER(LoraParams), ctypes.c_uint32
        lib.q2k_gated_ffn.argtypes = [ctypes.c_int, u32, vp, sz, vp, sz, vp, sz, vp, sz, vp, vp,
                                      gfp, vp, sz, vp]
        lib.q2k_gated_ffn_workspace_bytes.argtypes = [ctypes.c_int, gfp]
        lib.q2k_gated_ffn_workspace_bytes.restype = sz
        lib.q2k_gated_ffn_backward.argtypes = [vp, vp, vp, sz, vp, sz, vp, sz, vp, sz, vp, vp,
                                               gfp, vp, sz, vp]
        lib.q2k_gated_ffn_backward_workspace_bytes.argtypes = [gfp]
        lib.q2k_gated_ffn_backward_workspace_bytes.restype = sz
        lib.q2k_matmul_lora.argtypes = [ctypes.c_int, u32, vp, sz, vp, sz, vp, sz, vp, sz, vp, vp,
                                        vp, sz, lop, vp, vp, sz, vp]
        lib.q2k_matmul_lora_workspace_bytes.argtypes = [ctypes.c_int, lop]
        lib.q2k_matmul_lora_workspace_bytes.restype = sz
        lib.q2k_gated_ffn_experts.argtypes = [ctypes.c_int, u32, vp, sz, vp, sz, vp, sz, vp, sz, vp,
                                              vp, vp, u32, gfp, vp, sz, vp]
        lib.q2k_gated_ffn_experts_workspace_bytes.argtypes = [ctypes.c_int, gfp, u32]
        lib.q2k_gated_ffn_experts_workspace_bytes.restype = sz
        lib.q2k_gated_ffn_experts_backward.argtypes = [vp, vp, vp, sz, vp, sz, vp, sz, vp, sz, vp,
                                                       vp, vp, u32, gfp, vp, sz, vp]
        lib.q2k_gated_ffn_experts_backward_workspace_bytes.argtypes = [gfp, u32]
        lib.q2k_gated_ffn_experts_backward_workspace_bytes.restype = sz
        lip = ctypes.POINTER(LinearParams)
        lib.q2k_linear.argtypes = [ctypes.c_int, u32, vp, sz, vp, sz, vp, vp, vp, sz, vp, vp, lip, vp,
                                   sz, vp]
        lib.q2k_linear_workspace_bytes.argtypes = [ctypes.c_int, lip]
        lib.q2k_linear_workspace_bytes.restype = sz
        lib.q2k_linear_backward.argtypes = [vp, sz, vp, vp, sz, vp, sz, vp, vp, vp, lip, vp, sz, vp]
        lib.q2k_linear_backward_workspace_bytes.argtypes = [lip]
        lib.q2k_linear_backward_workspace_bytes.restype = sz
        mop = ctypes.POINTER(MoeParams)
        lib.q2k_moe_route.argtypes = [vp, sz, vp, vp, vp, mop, vp, vp]
        lib.q2k_moe_sort.argtypes = [vp, sz, vp, vp, vp, sz, mop, vp]
        lib.q2k_moe_sort_backward.argtypes = lib.q2k_moe_sort.argtypes
        lib.q2k_moe_combine.argtypes = [vp, sz, vp, vp, vp, vp, vp, sz, mop, vp]
        lib.q2k_moe_combine_backward.argtypes = [vp, sz, vp, sz, vp, vp, vp, vp, vp, mop, vp]
        lib.q2k_device_error.argtypes = [u32p, vp]
        lib.q2k_selftest_wait_timeout.argtypes = [ctypes.c_uint32, vp]
        for fn in ("q2k_dequantize", "q2k_embedding_gather", "q2k_matmul", "q2k_matmul_path",
                   "q2k_matmul_ex", "q2k_matmul_ex_batch", "q2k_matmul_batched_mv", "q2k_matmul_id",
                   "q2k_matmul_id_slotted", "q2k_matmul_id_pair", "q2k_matmul_id_ex",
                   "q2k_matmul_id_pair_ex", "q2k_gated_ffn", "q2k_gated_ffn_backward",
                   "q2k_gated_ffn_experts", "q2k_gated_ffn_experts_backward", "q2k_linear",
                   "q2k_linear_backward", "q2k_matmul_lora", "q2k_moe_route", "q2k_moe_sort", "q2k_moe_sort_backward",
                   "q2k_moe_combine", "q2k_moe_combine_backward", "q2k_device_error",
                   "q2k_selftest_wait_timeout", "q2k_gguf_open", "q2k_gguf_tensor_info",
                   "q2k_gguf_read_tensor"):
            getattr(lib, fn).restype = ctypes.c_int
        lib.q2k_last_error.restype = ctypes.c_char_p
        lib.q2k_last_error.argtypes = []
        lib.q2k_abi_version.restype = ctypes.c_int
        lib.q2k_abi_version.argtypes = []
        if path is None:
            _lib = lib
        return lib


def _check(lib, status: int):
    if status != 0:
        msg = lib.q2k_last_error().decode(errors="replace")
        if status == 1:
            raise InvalidArgument(status, msg)
        raise Q2KError(status, msg)


_torch_mod = None
_raw_stream = None


def _torch():
    global _torch_mod, _raw_stream
    if _torch_mod is None:
        import torch
        # the raw handle of a device's current stream without building a
        # torch.cuda.Stream object (the per-call cost of the public accessor)
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        _torch_mod = torch
    return _torch_mod


def _stream_handle(tensor) -> int:
    torch = _torch()
    if _raw_stream is not None:
        return _raw_stream(tensor.device.index)
    return torch.cuda.current_stream(tensor.device).cuda_stream


class _on_device:
    """``torch.cuda.device(t.device)`` only when it is not already current."""

    __slots__ = ("idx", "prev")

    def __init__(self, tensor):
        self.idx = tensor.device.index
        self.prev = None

    def __enter__(self):
        torch = _torch()
        cur = torch.cuda.current_device()
        if cur != self.idx:
            self.prev = cur
            torch.cuda.set_device(self.idx)
        return self

    def __exit__(self, *exc):
        if self.prev is not None:
            _torch().cuda.set_device(self.prev)


def _require_cuda(t, name, dtype):
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def dequantize(blocks, out=None):
    """Decode a uint8 CUDA tensor of whole Q2_K blocks to float32 (256 per block)."""
    torch = _torch()
    _require_cuda(blocks, "blocks", torch.uint8)
    n_out = (blocks.numel() // BLOCK_BYTES) * QK_K
    if out is None:
        out = torch.empty(max(n_out, 1), dtype=torch.float32, device=blocks.device)[:n_out]
    _require_cuda(out, "out", torch.float32)
    lib = load()
    with _on_device(blocks):
        _check(lib, lib.q2k_dequantize(blocks.data_ptr(), blocks.numel(), out.data_ptr(),
                                       out.numel(), _stream_handle(blocks)))
    return out


def embedding_gather(table, ids, embed_dim: int, vocab_size: int | None = None, out=None,
                     check: bool = True):
    """Rows ``ids`` of a Q2_K table ``[vocab, embed_dim]`` decoded to float32.

    With ``check`` (the default) the call waits for the stream and raises
    ``InvalidArgument`` if any id was >= vocab_size, as the pages' gather does;
    with ``check=False`` it returns ``(out, bad_id_count)`` without waiting.
    """
    torch = _torch()
    _require_cuda(table, "table", torch.uint8)
    _require_cuda(ids, "ids", ids.dtype)
    if ids.element_size() != 4 or ids.is_floating_point():
        raise TypeError("ids must be a 32-bit integer tensor (read as uint32)")
    row_bytes = (embed_dim // QK_K) * BLOCK_BYTES
    if vocab_size is None:
        vocab_size = table.numel() // row_bytes if row_bytes else 0
    n_tokens = ids.numel()
    if out is None:
        out = torch.empty((n_tokens, embed_dim), dtype=torch.float32, device=table.device)
    _require_cuda(out, "out", torch.float32)
    bad = torch.zeros(1, dtype=torch.int32, device=table.device)
    p = EmbeddingParams(vocab_size, embed_dim, n_tokens, GGML_TYPE_Q2_K)
    lib = load()
    with _on_device(table):
        _check(lib, lib.q2k_embedding_gather(table.data_ptr(), table.numel(), ids.data_ptr(),
                                             out.data_ptr(), out.numel(), ctypes.byref(p),
                                             bad.data_ptr(), _stream_handle(table)))
    if not check:
        return out, bad
    n_bad = int(bad.item())
    if n_bad:
        raise InvalidArgument(1, f"{n_bad} embedding id(s) >= vocab_size {vocab_size}")
    return out


_ws_bytes_cache: dict = {}


def matmul(x, w, n: int, out=None, path="auto", const_weights: bool = False,
           workspace="auto", independent: bool = False):
    """``y[m, r] = sum_k x[m, k] * W[r, k]`` with W = ``n`` rows of Q2_K blocks.

    ``const_weights=True`` passes Q2K_FLAG_CONST_WEIGHTS: the caller promises
    that the kernel enqueued just before on the stream does not write ``w``.
    ``independent=True`` passes Q2K_FLAG_INDEPENDENT: no kernel still running
    on the stream writes ``x`` or ``w`` or touches ``out`` (e.g. several
    projections of one activation enqueued back to back), so consecutive
    m = 1 calls overlap.
    ``workspace``: "auto" allocates the tensor-core path's workspace from
    PyTorch's caching allocator; None runs without one; or a uint8 CUDA tensor.
    """
    torch = _torch()
    _require_cuda(x, "x", torch.float32)
    _require_cuda(w, "w", torch.uint8)
    if x.dim() != 2:
        raise ValueError("x must be [m, k]")
    m, k = x.shape
    if out is None:
        out = torch.empty((m, n), dtype=torch.float32, device=x.device)
    _require_cuda(out, "out", torch.float32)
    p = MatmulParams(m, n, k, GGML_TYPE_Q2_K)
    lib = _lib if _lib is not None else load()
    pcode = _PATHS[path]
    ws_ptr, ws_bytes = None, 0
    if isinstance(workspace, str):
        # the GEMV path takes no workspace: skip the query for it
        if pcode == PATH_GEMV or (pcode == PATH_AUTO and m <= 8):
            workspace = None
        else:
            key = (m, n, k, pcode)
            need = _ws_bytes_cache.get(key)
            if need is None:
                need = lib.q2k_matmul_workspace_bytes(ctypes.byref(p), pcode)
                _ws_bytes_cache[key] = need
            workspace = torch.empty(need, dtype=torch.uint8, device=x.device) if need else None
    if workspace is not None:
        _require_cuda(workspace, "workspace", torch.uint8)
        ws_ptr, ws_bytes = workspace.data_ptr(), workspace.numel()
    flags = (FLAG_CONST_WEIGHTS if const_weights else 0) | (FLAG_INDEPENDENT if independent else 0)
    with _on_device(x):
        _check(lib, lib.q2k_matmul_ex(pcode, flags, x.data_ptr(), x.numel(), w.data_ptr(),
                                      w.numel(), out.data_ptr(), out.numel(), ctypes.byref(p),
                                      ws_ptr, ws_bytes, _stream_handle(x)))
    return out


class MatmulBatch:
    """A fixed list of matmuls enqueued by one library call per ``run()``.

    ``calls`` holds dicts with the arguments of ``matmul``: ``x``, ``w``, ``n``
    and optionally ``out``, ``path``, ``const_weights``, ``independent``,
    ``workspace`` (a uint8 CUDA tensor; "auto" allocates one per distinct
    geometry, shared by its calls).  Everything is checked and packed once;
    ``run()`` enqueues all calls in order on the current stream of the first
    call's device with ``q2k_matmul_ex_batch`` (results bit-identical to
    separate ``matmul`` calls; m = 1 calls reading one x convert it once),
    except that independent tensor-path calls with m <= 64 on one x, enough
    of them to fill the GPU, share persistent grids over all of k (the tensor
    path's bound, deterministic, other bits than a separate call).  The
    tensors stay bound: update their contents in place between runs.  ``outs``
    lists the output tensors in call order.

    ``graph=True``: the first ``run()`` enqueues the calls and captures them
    into a CUDA graph; later runs replay it on the current stream, one launch
    from the host for the whole list (the same kernels and bits).
    """

    def __init__(self, calls, graph: bool = False):
        torch = _torch()
        calls = list(calls)
        self._lib = load()
        self._use_graph = bool(graph)
        self._graph = None
        self._arr = (MatmulCall * max(1, len(calls)))()
        self._keep = []
        self.outs = []
        shared_ws = {}
        for i, c in enumerate(calls):
            x, w, n = c["x"], c["w"], int(c["n"])
            _require_cuda(x, "x", torch.float32)
            _require_cuda(w, "w", torch.uint8)
            if x.dim() != 2:
                raise ValueError("x must be [m, k]")
            m, k = x.shape
            out = c.get("out")
            if out is None:
                out = torch.empty((m, n), dtype=torch.float32, device=x.device)
            _require_cuda(out, "out", torch.float32)
            pcode = _PATHS[c.get("path", "auto")]
            ws = c.get("workspace", "auto")
            p = MatmulParams(m, n, k, GGML_TYPE_Q2_K)
            if isinstance(ws, str):
                tensor_path = pcode == PATH_TENSOR or (pcode == PATH_AUTO and m > 8)
                ws = None
                if tensor_path:
                    need = self._lib.q2k_matmul_workspace_bytes(ctypes.byref(p), pcode)
                    if need:
                        key = (x.device.index, need)
                        if key not in shared_ws:
                            shared_ws[key] = torch.empty(need, dtype=torch.uint8, device=x.device)
                        ws = shared_ws[key]
            if ws is not None:
                _require_cuda(ws, "workspace", torch.uint8)
            flags = (FLAG_CONST_WEIGHTS if c.get("const_weights") else 0) | \
                    (FLAG_INDEPENDENT if c.get("independent") else 0)
            a = self._arr[i]
            a.x, a.x_elems, a.w, a.w_bytes = x.data_ptr(), x.numel(), w.data_ptr(), w.numel()
            a.y, a.y_elems, a.params = out.data_ptr(), out.numel(), p
            a.workspace = ws.data_ptr() if ws is not None else None
            a.workspace_bytes = ws.numel() if ws is not None else 0
            a.path, a.flags = pcode, flags
            self._keep.append((x, w, out, ws))
            self.outs.append(out)
        self._count = len(calls)
        # scratch for x converted once: the rows several m = 1 calls share, and
        # the bf16 image of each run of independent small-m tensor calls
        need = self._lib.q2k_matmul_batch_scratch_bytes(self._arr, self._count) if calls else 0
        self._scratch = (torch.empty(need, dtype=torch.uint8, device=calls[0]["x"].device)
                         if need else None)

    def _enqueue(self):
        with _on_device(self._keep[0][0]):
            sp = self._scratch
            _check(self._lib, self._lib.q2k_matmul_ex_batch(
                self._arr, self._count, sp.data_ptr() if sp is not None else None,
                sp.numel() if sp is not None else 0, _stream_handle(self._keep[0][0])))

    def run(self):
        if self._count == 0:
            return self.outs
        if not self._use_graph:
            self._enqueue()
            return self.outs
        if self._graph is not None:
            with _on_device(self._keep[0][0]):
                self._graph.replay()
            return self.outs
        torch = _torch()
        self._enqueue()  # this run; the graph serves the next ones
        dev = self._keep[0][0].device
        with _on_device(self._keep[0][0]):
            cur = torch.cuda.current_stream(dev)
            side = torch.cuda.Stream(dev)
            side.wait_stream(cur)
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                self._enqueue()
            cur.wait_stream(side)
        self._graph = g
        return self.outs


def _planes_scratch(lib, k, rows, device, scratch):
    """(pointer, bytes) of the x-planes scratch: "auto" allocates one."""
    if scratch is None:
        return None, 0, None
    if isinstance(scratch, str):
        need = lib.q2k_x_planes_bytes(k, rows)
        if not need:
            return None, 0, None
        scratch = _torch().empty(need, dtype=_torch().uint8, device=device)
    return scratch.data_ptr(), scratch.numel(), scratch


def matmul_batched_mv(x, w, n: int, out=None, scratch=None):
    """``batches`` matrix-vector products in one launch: ``x`` f32 ``[batches, k]``
    (or ``[batches, 1, k]``), ``w`` uint8 holding the batches' ``[n, k]`` Q2_K
    matrices back to back; returns ``[batches, n]`` (the shape of ``x`` with k
    replaced by n).  Each batch is bit-identical to ``matmul`` of it alone.
    ``scratch="auto"`` converts each batch's x once instead of per CTA (an
    extra launch; it pays for long k), or pass a uint8 tensor of
    ``q2k_x_planes_bytes(k, batches)`` bytes."""
    torch = _torch()
    _require_cuda(x, "x", torch.float32)
    _require_cuda(w, "w", torch.uint8)
    k = x.shape[-1]
    batches = x.shape[0]
    if out is None:
        out = torch.empty(tuple(x.shape[:-1]) + (n,), dtype=torch.float32, device=x.device)
    _require_cuda(out, "out", torch.float32)
    lib = load()
    sp, sb, _keep = _planes_scratch(lib, k, batches, x.device, scratch)
    with _on_device(x):
        _check(lib, lib.q2k_matmul_batched_mv(x.data_ptr(), x.numel(), w.data_ptr(), w.numel(),
                                              out.data_ptr(), out.numel(), batches, 1, n, k, sp, sb,
                                              _stream_handle(x)))
    return out


def _routed_finish(bad, check, outs, n_experts):
    if not check:
        return (*outs, bad) if len(outs) > 1 else (outs[0], bad)
    n_bad = int(bad.item())
    if n_bad:
        raise InvalidArgument(1, f"{n_bad} expert id(s) >= n_experts {n_experts}")
    return outs if len(outs) > 1 else outs[0]


def matmul_id_slotted(x, w, ids, n: int, n_experts: int, expert_stride: int | None = None,
                      out=None, check: bool = True, scratch=None):
    """Routed product with one input row per route: ``x`` f32 ``[n_tokens, top_k,
    k]``, ``ids`` ``[n_tokens, top_k]``; returns ``[n_tokens, top_k, n]``, route
    (t, s) = expert ``ids[t, s]`` times ``x[t, s]``.  ``check`` as ``matmul_id``."""
    torch = _torch()
    _require_cuda(x, "x", torch.float32)
    _require_cuda(w, "w", torch.uint8)
    _require_cuda(ids, "ids", ids.dtype)
    if ids.element_size() != 4 or ids.is_floating_point():
        raise TypeError("ids must be a 32-bit integer tensor (read as uint32)")
    n_tokens, top_k, k = x.shape
    if expert_stride is None:
        expert_stride = n * (k // QK_K) * BLOCK_BYTES
    if out is None:
        out = torch.empty((n_tokens, top_k, n), dtype=torch.float32, device=x.device)
    _require_cuda(out, "out", torch.float32)
    bad = torch.zeros(1, dtype=torch.int32, device=x.device)
    p = MatmulIdParams(n_tokens, top_k, n, k, n_experts, GGML_TYPE_Q2_K, expert_stride)
    lib = load()
    sp, sb, _keep = _planes_scratch(lib, k, n_tokens * top_k, x.device, scratch)
    with _on_device(x):
        _check(lib, lib.q2k_matmul_id_slotted(x.data_ptr(), x.numel(), w.data_ptr(), w.numel(),
                                              ids.data_ptr(), out.data_ptr(), out.numel(),
                                              ctypes.byref(p), bad.data_ptr(), sp, sb,
                                              _stream_handle(x)))
    return _routed_finish(bad, check, (out,), n_experts)


def matmul_id_pair(x, w_a, w_b, ids, n: int, n_experts: int, top_k: int,
                   expert_stride: int | None = None, check: bool = True, scratch="auto",
                   path=None, workspace=None):
    """Two routed products sharing ``x`` and ``ids`` (e.g. the gate and up
    projections) in one launch; returns ``(y_a, y_b)`` as ``matmul_id`` would.
    ``path`` ("gemv", "tensor" or "auto", as ``matmul_id_ex``) goes through
    ``q2k_matmul_id_pair_ex``; the tensor path routes and gathers x once for
    both products.  ``workspace`` as in ``matmul_id_ex``."""
    torch = _torch()
    _require_cuda(x, "x", torch.float32)
    _require_cuda(w_a, "w_a", torch.uint8)
    _require_cuda(w_b, "w_b", torch.uint8)
    _require_cuda(ids, "ids", ids.dtype)
    if ids.element_size() != 4 or ids.is_floating_point():
        raise TypeError("ids must be a 32-bit integer tensor (read as uint32)")
    n_tokens, k = x.shape
    if expert_stride is None:
        expert_stride = n * (k // QK_K) * BLOCK_BYTES
    y_a = torch.empty((ids.numel(), n), dtype=torch.float32, device=x.device)
    y_b = torch.empty((ids.numel(), n), dtype=torch.float32, device=x.device)
    bad = torch.zeros(1, dtype=torch.int32, device=x.device)
    p = MatmulIdParams(n_tokens, top_k, n, k, n_experts, GGML_TYPE_Q2_K, expert_stride)
    lib = load()
    if path is not None:
        pcode = _PATHS[path]
        if workspace is None:
            nbytes = lib.q2k_matmul_id_workspace_bytes(pcode, 0, ctypes.byref(p))
            if nbytes:
                workspace = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
        wp = workspace.data_ptr() if workspace is not None else None
        wb = workspace.numel() if workspace is not None else 0
        with _on_device(x):
            _check(lib, lib.q2k_matmul_id_pair_ex(pcode, x.data_ptr(), x.numel(), w_a.data_ptr(),
                                                  w_a.numel(), w_b.data_ptr(), w_b.numel(),
                                                  ids.data_ptr(), y_a.data_ptr(), y_b.data_ptr(),
                                                  y_a.numel(), ctypes.byref(p), bad.data_ptr(),
                                                  wp, wb, _stream_handle(x)))
        return _routed_finish(bad, check, (y_a, y_b), n_experts)
    sp, sb, _keep = _planes_scratch(lib, k, n_tokens, x.device, scratch)
    with _on_device(x):
        _check(lib, lib.q2k_matmul_id_pair(x.data_ptr(), x.numel(), w_a.data_ptr(), w_a.numel(),
                                           w_b.data_ptr(), w_b.numel(), ids.data_ptr(),
                                           y_a.data_ptr(), y_b.data_ptr(), y_a.numel(),
                                           ctypes.byref(p), bad.data_ptr(), sp, sb,
                                           _stream_handle(x)))
    return _routed_finish(bad, check, (y_a, y_b), n_experts)


def matmul_id(x, w, ids, n: int, n_experts: int, top_k: int, expert_stride: int | None = None,
              out=None, check: bool = True, scratch="auto"):
    """Expert-routed product: ``x`` f32 ``[n_tokens, k]``, ``ids`` 32-bit ints
    ``[n_tokens * top_k]`` (token-major), expert e's ``[n, k]`` Q2_K matrix at
    byte ``e * expert_stride`` of ``w`` (default: packed, ``n * k/256 * 84``).
    Returns ``[n_tokens * top_k, n]`` with row r = expert ``ids[r]`` times token
    ``r // top_k``.  With ``check`` the call waits and raises ``InvalidArgument``
    if an id was >= n_experts; with ``check=False`` it returns ``(out,
    bad_id_count)`` without waiting."""
    torch = _torch()
    _require_cuda(x, "x", torch.float32)
    _require_cuda(w, "w", torch.uint8)
    _require_cuda(ids, "ids", ids.dtype)
    if ids.element_size() != 4 or ids.is_floating_point():
        raise TypeError("ids must be a 32-bit integer tensor (read as uint32)")
    n_tokens, k = x.shape
    if expert_stride is None:
        expert_stride = n * (k // QK_K) * BLOCK_BYTES
    if out is None:
        out = torch.empty((ids.numel(), n), dtype=torch.float32, device=x.device)
    _require_cuda(out, "out", torch.float32)
    bad = torch.zeros(1, dtype=torch.int32, device=x.device)
    p = MatmulIdParams(n_tokens, top_k, n, k, n_experts, GGML_TYPE_Q2_K, expert_stride)
    lib = load()
    sp, sb, _keep = _planes_scratch(lib, k, n_tokens, x.device, scratch)
    with _on_device(x):
        _check(lib, lib.q2k_matmul_id(x.data_ptr(), x.numel(), w.data_ptr(), w.numel(),
                                      ids.data_ptr(), out.data_ptr(), out.numel(),
                                      ctypes.byref(p), bad.data_ptr(), sp, sb, _stream_handle(x)))
    if not check:
        return out, bad
    n_bad = int(bad.item())
    if n_bad:
        raise InvalidArgument(1, f"{n_bad} expert id(s) >= n_experts {n_experts}")
    return out


def matmul_id_ex(x, w, ids, n: int, n_experts: int, top_k: int = 1, path="auto",
                 slotted: bool = False, expert_stride: int | None = None, out=None,
                 check: bool = True, workspace=None):
    """``matmul_id`` (or, with ``slotted``, ``matmul_id_slotted``; then ``x`` is
    ``[n_tokens, top_k, k]`` and ``top_k`` is taken from it) on a chosen path:
    ``"gemv"`` (fp32, as ``matmul_id``), ``"tensor"`` (routes grouped per
    expert and multiplied on the bf16 tensor cores) or ``"auto"`` (tensor above
    32 tokens).  ``workspace``: a CUDA uint8 tensor of at least
    ``matmul_id_workspace_bytes`` bytes, allocated here when None."""
    torch = _torch()
    _require_cuda(x, "x", torch.float32)
    _require_cuda(w, "w", torch.uint8)
    _require_cuda(ids, "ids", ids.dtype)
    if ids.element_size() != 4 or ids.is_floating_point():
        raise TypeError("ids must be a 32-bit integer tensor (read as uint32)")
    if slotted:
        n_tokens, top_k, k = x.shape
        shape = (n_tokens, top_k, n)
    else:
        n_tokens, k = x.shape
        shape = (n_tokens * top_k, n)
    if expert_stride is None:
        expert_stride = n * (k // QK_K) * BLOCK_BYTES
    if out is None:
        out = torch.empty(shape, dtype=torch.float32, device=x.device)
    _require_cuda(out, "out", torch.float32)
    bad = torch.zeros(1, dtype=torch.int32, device=x.device)
    p = MatmulIdParams(n_tokens, top_k, n, k, n_experts, GGML_TYPE_Q2_K, expert_stride)
    pcode = _PATHS[path]
    flags = ID_SLOTTED if slotted else 0
    lib = load()
    if workspace is None:
        nbytes = lib.q2k_matmul_id_workspace_bytes(pcode, flags, ctypes.byref(p))
        if nbytes:
            workspace = torch.empty(nbytes, dtype=torch.uint8, device=x.device)
    wp = workspace.data_ptr() if workspace is not None else None
    wb = workspace.numel() if workspace is not None else 0
    with _on_device(x):
        _check(lib, lib.q2k_matmul_id_ex(pcode, flags, x.data_ptr(), x.numel(), w.data_ptr(),
                                         w.numel(), ids.data_ptr(), out.data_ptr(), out.numel(),
                                         ctypes.byref(p), bad.data_ptr(), wp, wb,
                                         _stream_handle(x)))
    return _routed_finish(bad, check, (out,), n_experts)


def matmul_id_workspace_bytes(n_tokens: int, top_k: int, n: int, k: int, n_experts: int,
                              path="auto", slotted: bool = False,
                              expert_stride: int | None = None) -> int:
    """Bytes of workspace ``matmul_id_ex`` takes on ``path`` (0: none or invalid)."""
    if expert_stride is None:
        expert_stride = n * (k // QK_K) * BLOCK_BYTES
    p = MatmulIdParams(n_tokens, top_k, n, k, n_experts, GGML_TYPE_Q2_K, expert_stride)
    return int(load().q2k_matmul_id_workspace_bytes(_PATHS[path], ID_SLOTTED if slotted else 0,
                                                    ctypes.byref(p)))


def _need_activations(t, name, dtype=None):
    """Raise unless ``t`` is a contiguous f32 or bf16 CUDA tensor (of ``dtype``)."""
    torch = _torch()
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _need_like(x, **tensors):
    """Raise unless every tensor (dtype, shape or None, tensor) fits and is on x's device."""
    for name, (dtype, shape, t) in tensors.items():
        _require_cuda(t, name, dtype)
        if shape is not None and tuple(t.shape) != tuple(shape):
            raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
        if t.device != x.device:
            raise ValueError(f"{name} is on {t.device}, expected {x.device}")


def _fits(dev, dtype, *tensors):
    """Whether every tensor is a contiguous ``dtype`` tensor on CUDA device ``dev``
    (the quick form of ``_need_like``, which says what is wrong)."""
    try:
        for t in tensors:
            if t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous():
                return False
    except AttributeError:
        return False
    return dev >= 0


# A call's parameter block (by reference), workspace bytes and path code, by its
# geometry: what depends on neither the tensors nor their contents.
_ffn_plans: dict = {}


def _ffn_plan(key):
    """``key``: (kind, path, dtype, m, n, k, act, n_experts), kind "gated", "backward",
    "linear" or "linear_backward", or ("lora", path, dtype, m, n, k, rank, n_adapters)."""
    lib, torch = load(), _torch()
    kind, path, dtype, m, n, k = key[:6]
    acts = _LINEAR_ACTS if kind.startswith("linear") else _ACTS
    for name, value, known in (("path", path, _PATHS), ("act", "silu" if kind == "lora" else key[6], acts)):
        if value not in known:
            raise KeyError(f"{name} must be one of {', '.join(map(repr, known))}, got {value!r}")
    pcode, code = _PATHS[path], DTYPE_F32 if dtype == torch.float32 else DTYPE_BF16
    if kind == "lora":
        p = LoraParams(m, n, k, GGML_TYPE_Q2_K, code, *key[6:], 0)
        need = lib.q2k_matmul_lora_workspace_bytes(pcode, ctypes.byref(p))
    elif kind.startswith("linear"):
        p = LinearParams(m, n, k, GGML_TYPE_Q2_K, code, acts[key[6]], key[7], 0)
        need = (lib.q2k_linear_backward_workspace_bytes(ctypes.byref(p))
                if kind == "linear_backward"
                else lib.q2k_linear_workspace_bytes(pcode, ctypes.byref(p)))
    else:
        p = GatedFfnParams(m, n, k, GGML_TYPE_Q2_K, code, _ACTS[key[6]])
        experts = key[7]
        if kind == "backward":
            need = (lib.q2k_gated_ffn_experts_backward_workspace_bytes(ctypes.byref(p), experts)
                    if experts else lib.q2k_gated_ffn_backward_workspace_bytes(ctypes.byref(p)))
        else:
            need = (lib.q2k_gated_ffn_experts_workspace_bytes(pcode, ctypes.byref(p), experts)
                    if experts else lib.q2k_gated_ffn_workspace_bytes(pcode, ctypes.byref(p)))
    if len(_ffn_plans) >= 4096:  # (geometries, not tensors: a bound for long runs)
        _ffn_plans.clear()
    plan = _ffn_plans[key] = (ctypes.byref(p), need, pcode)
    return plan


def _segments(x, routes):
    """(pointer of the offsets or None, n_experts or 0) of a call's tokens."""
    if routes is None:
        return None, 0
    torch = _torch_mod or _torch()
    offsets = routes.offsets
    if not _fits(x.get_device(), torch.int32, offsets):
        _need_like(x, offsets=(torch.int32, None, offsets))
    if offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError("routes.offsets must be [n_experts + 1]")
    return offsets.data_ptr(), offsets.shape[0] - 1


def _ffn_workspace(workspace, need, x):
    """(tensor, pointer, bytes) of a call's workspace: "auto" takes one from
    PyTorch's allocator."""
    if workspace is None or (need == 0 and isinstance(workspace, str)):
        return None, None, 0
    torch = _torch()
    if isinstance(workspace, str):
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    else:
        _need_like(x, workspace=(torch.uint8, None, workspace))
    return workspace, workspace.data_ptr(), workspace.numel()


def _ffn_call(dev, fn, *args):
    """Call ``fn`` with the current stream of CUDA device ``dev``, ``dev`` current."""
    cuda = _torch_mod.cuda
    if cuda.current_device() == dev:
        status = fn(*args, _raw_stream(dev) if _raw_stream else cuda.current_stream(dev).cuda_stream)
    else:
        with cuda.device(dev):
            status = fn(*args, cuda.current_stream(dev).cuda_stream)
    if status:
        _check(_lib, status)


_quick_mod = None


def _quick():
    """The compiled module for ordinary calls (q2k_torch), or False without it."""
    global _quick_mod
    if _quick_mod is None:
        lib, torch = load(), _torch()
        path = _build.torch_module_path(torch.__version__)
        if not os.path.exists(path):
            _quick_mod = False
            return False
        spec = importlib.util.spec_from_file_location("q2k_torch", path)
        try:
            mod = importlib.util.module_from_spec(spec)
            spec.loader.exec_module(mod)
        except ImportError as e:
            warnings.warn(f"the PyTorch module does not load; feed-forward calls go through ctypes: {e}",
                          RuntimeWarning, stacklevel=3)
            _quick_mod = False
            return False
        mod.bind(*(ctypes.cast(getattr(lib, f), ctypes.c_void_p).value for f in (
            "q2k_gated_ffn", "q2k_gated_ffn_workspace_bytes", "q2k_gated_ffn_backward",
            "q2k_gated_ffn_backward_workspace_bytes", "q2k_matmul_lora",
            "q2k_matmul_lora_workspace_bytes")))
        mod.bind_experts(*(ctypes.cast(getattr(lib, f), ctypes.c_void_p).value for f in (
            "q2k_linear", "q2k_linear_workspace_bytes", "q2k_linear_backward",
            "q2k_linear_backward_workspace_bytes", "q2k_gated_ffn_experts",
            "q2k_gated_ffn_experts_workspace_bytes", "q2k_gated_ffn_experts_backward",
            "q2k_gated_ffn_experts_backward_workspace_bytes", "q2k_moe_route", "q2k_moe_sort",
            "q2k_moe_sort_backward", "q2k_moe_combine", "q2k_moe_combine_backward")))
        _quick_mod = mod
    return _quick_mod


def gated_ffn(x, w_gate, w_up, n: int, act="silu", save: bool = False, out=None, path="auto",
              const_weights: bool = False, workspace="auto", routes=None):
    """The gated feed-forward block ``h = act(x Wg^T) * (x Wu^T)``: both
    projections, the activation and the product in one kernel.

    ``x`` f32 or bf16 ``[m, k]``; ``w_gate``, ``w_up`` uint8, ``n`` rows of Q2_K
    blocks each; ``act`` "silu" or "gelu" (the tanh form).  Returns h ``[m, n]``
    in x's dtype, or with ``save`` ``(h, gate, up)`` with the two projections
    that ``gated_ffn_backward`` reads.  ``path``, ``const_weights`` and
    ``workspace`` as in ``matmul``: up to 16 bf16 or 8 f32 tokens the weights
    are exact, above that x and W are rounded to bf16 for the tensor cores.
    Nothing is recorded for autograd: h does not require a gradient, even where
    x does.

    ``routes`` (of ``moe_route``): x holds rows in expert order, as ``moe_sort`` makes
    them, and each row is multiplied by its own expert's matrices; ``w_gate`` and
    ``w_up`` then hold ``n_experts`` matrices each, one after another.  Rows behind the
    last expert's reach no result, and theirs are not written.  The weights are exact
    up to eight bf16 or four f32 tokens for each expert.
    """
    if out is None and workspace.__class__ is str:
        quick = _quick_mod or _quick()
        done = (quick.gated(x, w_gate, w_up, n, act, save, path, const_weights,
                            routes if routes is None else routes.offsets)
                if quick else None)
        if done.__class__ is int:
            _check(_lib, done)
        elif done is not None:
            return done
    torch = _torch_mod or _torch()
    _need_activations(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be [m, k]")
    m, k = x.shape
    dt, dev = x.dtype, x.get_device()
    if not _fits(dev, torch.uint8, w_gate, w_up):
        _need_like(x, w_gate=(torch.uint8, None, w_gate), w_up=(torch.uint8, None, w_up))
    if out is None:
        out = torch.empty((m, n), dtype=dt, device=x.device)
    else:
        _need_like(x, out=(dt, (m, n), out))
    gate = torch.empty_like(out) if save else None
    up = torch.empty_like(out) if save else None
    segments = _segments(x, routes)
    key = ("gated", path, dt, m, n, k, act, segments[1])
    params, need, pcode = _ffn_plans.get(key) or _ffn_plan(key)
    _keep, ws, ws_bytes = _ffn_workspace(workspace, need, x)
    fn, where = ((_lib.q2k_gated_ffn, ()) if routes is None
                 else (_lib.q2k_gated_ffn_experts, segments))
    _ffn_call(dev, fn, pcode, FLAG_CONST_WEIGHTS if const_weights else 0,
              x.data_ptr(), m * k, w_gate.data_ptr(), w_gate.numel(), w_up.data_ptr(),
              w_up.numel(), out.data_ptr(), m * n, gate.data_ptr() if save else None,
              up.data_ptr() if save else None, *where, params, ws, ws_bytes)
    return (out, gate, up) if save else out


def gated_ffn_backward(dh, gate, up, w_gate, w_up, k: int, act="silu", workspace="auto",
                       routes=None):
    """The backward pass of ``gated_ffn`` with its weights frozen, bf16 only.

    ``dh``, ``gate``, ``up`` bf16 ``[m, n]`` (the gradient of h and the saved
    projections); returns ``(dx, dgate, dup)``: ``dx = dgate Wg + dup Wu``
    ``[m, k]`` and the gradients ``[m, n]`` of the two projections.  ``routes`` as in
    ``gated_ffn``.  dx's product takes dgate, dup and the weights rounded to bf16.
    """
    if workspace.__class__ is str:
        quick = _quick_mod or _quick()
        done = (quick.backward(dh, gate, up, w_gate, w_up, k, act,
                               routes if routes is None else routes.offsets)
                if quick else None)
        if done.__class__ is int:
            _check(_lib, done)
        elif done is not None:
            return done
    torch = _torch_mod or _torch()
    bf16, u8 = torch.bfloat16, torch.uint8
    _need_activations(dh, "dh", bf16)
    if dh.dim() != 2:
        raise ValueError("dh must be [m, n]")
    m, n = shape = dh.shape
    dev = dh.get_device()
    if not (_fits(dev, bf16, gate, up) and gate.shape == shape == up.shape
            and _fits(dev, u8, w_gate, w_up)):
        _need_like(dh, gate=(bf16, shape, gate), up=(bf16, shape, up),
                   w_gate=(u8, None, w_gate), w_up=(u8, None, w_up))
    dx = torch.empty((m, k), dtype=bf16, device=dh.device)
    dgate, dup = torch.empty_like(dh), torch.empty_like(dh)
    segments = _segments(dh, routes)
    key = ("backward", "auto", bf16, m, n, k, act, segments[1])
    params, need, _ = _ffn_plans.get(key) or _ffn_plan(key)
    _keep, ws, ws_bytes = _ffn_workspace(workspace, need, dh)
    fn, where = ((_lib.q2k_gated_ffn_backward, ()) if routes is None
                 else (_lib.q2k_gated_ffn_experts_backward, segments))
    _ffn_call(dev, fn, dh.data_ptr(), gate.data_ptr(), up.data_ptr(),
              m * n, w_gate.data_ptr(), w_gate.numel(), w_up.data_ptr(), w_up.numel(),
              dx.data_ptr(), m * k, dgate.data_ptr(), dup.data_ptr(), *where, params, ws, ws_bytes)
    return dx, dgate, dup


def linear(x, w, n: int, bias=None, act=None, residual=None, save: bool = False, out=None,
           path="auto", const_weights: bool = False, workspace="auto", routes=None):
    """A projection with its epilogue: ``y = act(x W^T + bias) + residual`` in one kernel.

    ``x`` f32 or bf16 ``[m, k]``; ``w`` uint8, ``n`` rows of Q2_K blocks; ``bias`` f32
    ``[n]`` or None; ``act`` None, "silu" or "gelu" (the tanh form); ``residual`` ``[m,
    n]`` in x's dtype or None.  Returns y ``[m, n]`` in x's dtype, or with ``save`` ``(y,
    z)`` with ``z = x W^T + bias``, which ``linear_backward`` reads.  ``path``,
    ``const_weights`` and ``workspace`` as in ``gated_ffn``; nothing is recorded for
    autograd.  ``routes`` as in ``gated_ffn``: ``w`` then holds ``n_experts`` matrices
    and ``bias`` is ``[n_experts, n]``.

    Above 16 bf16 or 8 f32 tokens "auto" rounds x and W to bf16, also where x is f32;
    ``path="gemv"`` keeps the weights exact, in a time that grows with every 16 (8)
    tokens (4096 x 4096, 64 f32 tokens: 61 us against 16).
    """
    if out is None and workspace.__class__ is str:
        quick = _quick_mod or _quick()
        done = (quick.linear(x, w, n, bias, act, residual, save, path, const_weights,
                             routes if routes is None else routes.offsets)
                if quick else None)
        if done.__class__ is int:
            _check(_lib, done)
        elif done is not None:
            return done
    torch = _torch_mod or _torch()
    _need_activations(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be [m, k]")
    m, k = x.shape
    dt, dev = x.dtype, x.get_device()
    if not _fits(dev, torch.uint8, w):
        _need_like(x, w=(torch.uint8, None, w))
    offsets, experts = _segments(x, routes)
    if bias is not None:
        _need_like(x, bias=(torch.float32, (experts, n) if experts else (n,), bias))
    if residual is not None:
        _need_like(x, residual=(dt, (m, n), residual))
    if out is None:
        out = torch.empty((m, n), dtype=dt, device=x.device)
    else:
        _need_like(x, out=(dt, (m, n), out))
    z = torch.empty_like(out) if save else None
    key = ("linear", path, dt, m, n, k, act, experts)
    params, need, pcode = _ffn_plans.get(key) or _ffn_plan(key)
    _keep, ws, ws_bytes = _ffn_workspace(workspace, need, x)
    _ffn_call(dev, _lib.q2k_linear, pcode, FLAG_CONST_WEIGHTS if const_weights else 0, x.data_ptr(),
              m * k, w.data_ptr(), w.numel(), bias.data_ptr() if bias is not None else None,
              residual.data_ptr() if residual is not None else None, out.data_ptr(), m * n,
              z.data_ptr() if save else None, offsets, params, ws, ws_bytes)
    return (out, z) if save else out


def linear_backward(dy, w, k: int, z=None, act=None, bias: bool = False, workspace="auto",
                    routes=None):
    """The backward pass of ``linear`` with its weights frozen, bf16 only.

    ``dy`` bf16 ``[m, n]``; ``z`` the saved ``[m, n]``, read where there is an
    activation.  Returns ``(dx, dz, dbias)``: ``dx = dz W`` ``[m, k]``, ``dz = dy
    act'(z)`` (without an activation ``dy`` itself) and with ``bias`` the sum of dz over
    the tokens, f32 ``[n]`` (with ``routes`` over each expert's, ``[n_experts, n]``), else
    None.  The residual's gradient is ``dy``.  ``routes`` as in ``gated_ffn``.  dx's product
    takes dz and W rounded to bf16 (dx within 8e-3 of the sum of ``|dz w|``); dbias sums
    dz before it is rounded.
    """
    if workspace.__class__ is str:
        quick = _quick_mod or _quick()
        done = (quick.linear_backward(dy, w, k, z, act, bias,
                                      routes if routes is None else routes.offsets)
                if quick else None)
        if done.__class__ is int:
            _check(_lib, done)
        elif done is not None:
            if act is not None:
                return done if bias else (*done, None)
            return (done[0], dy, done[1]) if bias else (done, dy, None)
    torch = _torch_mod or _torch()
    bf16 = torch.bfloat16
    _need_activations(dy, "dy", bf16)
    if dy.dim() != 2:
        raise ValueError("dy must be [m, n]")
    m, n = dy.shape
    dev = dy.get_device()
    if not _fits(dev, torch.uint8, w):
        _need_like(dy, w=(torch.uint8, None, w))
    if act is None:
        z = None
    else:
        _need_like(dy, z=(bf16, (m, n), z))
    offsets, experts = _segments(dy, routes)
    dx = torch.empty((m, k), dtype=bf16, device=dy.device)
    dz = dy if act is None else torch.empty_like(dy)
    dbias = (torch.empty((experts, n) if experts else (n,), dtype=torch.float32, device=dy.device)
             if bias else None)
    key = ("linear_backward", "auto", bf16, m, n, k, act, experts)
    params, need, _ = _ffn_plans.get(key) or _ffn_plan(key)
    _keep, ws, ws_bytes = _ffn_workspace(workspace, need, dy)
    _ffn_call(dev, _lib.q2k_linear_backward, dy.data_ptr(), m * n,
              z.data_ptr() if z is not None else None, w.data_ptr(), w.numel(), dx.data_ptr(), m * k,
              dz.data_ptr() if z is not None else None, dbias.data_ptr() if bias else None, offsets,
              params, ws, ws_bytes)
    return dx, dz, dbias


def matmul_lora(x, w, n: int, lora_a, lora_b, ids, scales=None, out=None, path="auto",
                const_weights: bool = False, workspace="auto", check: bool = True):
    """A shared projection with low-rank adapters of many requests at once:
    ``y_i = W x_i + s_a B_a (A_a x_i)`` with ``a = ids[i]``, -1 for none.

    ``x`` f32 or bf16 ``[m, k]``; ``w`` uint8, ``n`` rows of Q2_K blocks;
    ``lora_a`` bf16 ``[n_adapters, rank, k]``, ``lora_b`` bf16 ``[n_adapters, n,
    rank]`` (rank a multiple of 8, lower ranks padded with zeros); ``ids`` int32
    ``[m]``; ``scales`` f32 ``[n_adapters]`` or None.  Returns ``[m, n]`` in x's
    dtype.  With ``check`` the call waits and raises ``InvalidArgument`` if an
    id was neither -1 nor below n_adapters; with ``check=False`` it returns
    ``(out, bad_id_count)`` without waiting (such a token's row is zero).
    ``path``, ``const_weights`` and ``workspace`` as in ``gated_ffn``.
    """
    if out is None and workspace.__class__ is str:
        quick = _quick_mod or _quick()
        done = (quick.lora(x, w, n, lora_a, lora_b, ids, scales, path, const_weights)
                if quick else None)
        if done.__class__ is int:
            _check(_lib, done)
        elif done is not None:
            return _lora_result(*done, lora_a.shape[0], check)
    torch = _torch_mod or _torch()
    _need_activations(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be [m, k]")
    m, k = x.shape
    bf16, dt, dev = torch.bfloat16, x.dtype, x.get_device()
    if not isinstance(lora_a, torch.Tensor) or lora_a.dim() != 3:
        raise ValueError("lora_a must be [n_adapters, rank, k]")
    n_adapters, rank, _ = lora_a.shape
    if not (_fits(dev, bf16, lora_a, lora_b) and lora_a.shape == (n_adapters, rank, k)
            and lora_b.shape == (n_adapters, n, rank) and _fits(dev, torch.int32, ids)
            and ids.shape == (m,) and _fits(dev, torch.uint8, w)):
        _need_like(x, w=(torch.uint8, None, w), lora_a=(bf16, (n_adapters, rank, k), lora_a),
                   lora_b=(bf16, (n_adapters, n, rank), lora_b), ids=(torch.int32, (m,), ids))
    if scales is not None:
        if not (_fits(dev, torch.float32, scales) and scales.shape == (n_adapters,)):
            _need_like(x, scales=(torch.float32, (n_adapters,), scales))
    if out is None:
        out = torch.empty((m, n), dtype=dt, device=x.device)
    else:
        _need_like(x, out=(dt, (m, n), out))
    bad = torch.empty(1, dtype=torch.int32, device=x.device)
    key = ("lora", path, dt, m, n, k, rank, n_adapters)
    params, need, pcode = _ffn_plans.get(key) or _ffn_plan(key)
    _keep, ws, ws_bytes = _ffn_workspace(workspace, need, x)
    _ffn_call(dev, _lib.q2k_matmul_lora, pcode, FLAG_CONST_WEIGHTS if const_weights else 0,
              x.data_ptr(), m * k, w.data_ptr(), w.numel(), lora_a.data_ptr(),
              lora_a.numel(), lora_b.data_ptr(), lora_b.numel(),
              scales.data_ptr() if scales is not None else None, ids.data_ptr(), out.data_ptr(),
              m * n, params, bad.data_ptr(), ws, ws_bytes)
    return _lora_result(out, bad, n_adapters, check)


def _lora_result(out, bad, n_adapters, check):
    if not check:
        return out, bad
    n_bad = int(bad.item())
    if n_bad:
        raise InvalidArgument(1, f"{n_bad} adapter id(s) outside -1..{n_adapters - 1}")
    return out


def moe_route(ids, n_experts: int, check: bool = True):
    """Where a router's choices land in expert order: ``Routes(rows, order, offsets)``.

    ``ids`` int32 ``[n_tokens, top_k]``, each token's experts, -1 for none; the choices
    of one expert keep their order, those without an expert come last.  With ``check``
    the call waits and raises ``InvalidArgument`` if an id was neither -1 nor below
    n_experts; with ``check=False`` it returns ``(routes, bad_id_count)`` without
    waiting (such a choice has no expert).
    """
    quick = _quick_mod or _quick()
    done = quick.route(ids, n_experts) if quick else None
    if done.__class__ is int:
        _check(_lib, done)
    elif done is not None:
        return _routed(Routes(*done[:3]), done[3], n_experts, check)
    torch = _torch_mod or _torch()
    i32 = torch.int32
    _require_cuda(ids, "ids", i32)
    if ids.dim() != 2:
        raise ValueError("ids must be [n_tokens, top_k]")
    if not 1 <= n_experts <= MOE_MAX_EXPERTS:
        raise ValueError(f"n_experts must be in 1..{MOE_MAX_EXPERTS}, got {n_experts}")
    n_tokens, top_k = ids.shape
    choices = n_tokens * top_k
    # (one buffer: each part starts at a whole 16 bytes)
    part = (choices + 3) // 4 * 4
    buf = torch.empty(2 * part + n_experts + 2, dtype=i32, device=ids.device)
    rows, order = buf[:choices].view(n_tokens, top_k), buf[part:part + choices]
    offsets, bad = buf[2 * part:2 * part + n_experts + 1], buf[2 * part + n_experts + 1:]
    p = MoeParams(n_tokens, top_k, n_experts, 0, 0, 0)
    lib = _lib if _lib is not None else load()
    _ffn_call(ids.get_device(), lib.q2k_moe_route, ids.data_ptr(), choices, rows.data_ptr(),
              order.data_ptr(), offsets.data_ptr(), ctypes.byref(p), bad.data_ptr())
    return _routed(Routes(rows, order, offsets), bad, n_experts, check)


def _routed(routes, bad, n_experts, check):
    if not check:
        return routes, bad
    n_bad = int(bad.item())
    if n_bad:
        raise InvalidArgument(1, f"{n_bad} expert id(s) outside -1..{n_experts - 1}")
    return routes


def _moe_params(t, routes, name, rows_of):
    """(params, rows, offsets) of a move whose activations ``t`` have a row for each
    token (``rows_of`` "tokens") or each choice ("choices")."""
    torch = _torch_mod or _torch()
    _need_activations(t, name)
    rows, _, offsets = routes
    dev, i32 = t.get_device(), torch.int32
    if not _fits(dev, i32, rows, offsets):
        _need_like(t, rows=(i32, None, rows), offsets=(i32, None, offsets))
    if rows.dim() != 2 or offsets.dim() != 1 or offsets.shape[0] < 2:
        raise ValueError("routes must hold rows [n_tokens, top_k] and offsets [n_experts + 1]")
    n_tokens, top_k = rows.shape
    first = n_tokens if rows_of == "tokens" else n_tokens * top_k
    if t.dim() != 2 or t.shape[0] != first:
        raise ValueError(f"{name} must be [{first}, width], got {list(t.shape)}")
    code = DTYPE_F32 if t.dtype == torch.float32 else DTYPE_BF16
    return MoeParams(n_tokens, top_k, offsets.shape[0] - 1, t.shape[1], code, 0), rows, offsets


def _moe_out(out, like, shape):
    if out is None:
        return _torch_mod.empty(shape, dtype=like.dtype, device=like.device)
    _need_like(like, out=(like.dtype, shape, out))
    return out


def moe_sort(x, routes, out=None):
    """The tokens' rows in expert order: ``xs[routes.rows[t, s]] = x[t]``.

    ``x`` f32 or bf16 ``[n_tokens, width]``; returns ``[n_tokens * top_k, width]``, the
    rows of expert e at ``routes.offsets[e]`` up to ``offsets[e + 1]``, ready for
    ``linear`` and ``gated_ffn`` with ``routes``; rows behind the last are zeros.
    """
    if out is None:
        quick = _quick_mod or _quick()
        done = quick.sort(x, routes.rows, routes.offsets) if quick else None
        if done.__class__ is int:
            _check(_lib, done)
        elif done is not None:
            return done
    p, rows, offsets = _moe_params(x, routes, "x", "tokens")
    out = _moe_out(out, x, (p.n_tokens * p.top_k, p.width))
    lib = _lib if _lib is not None else load()
    _ffn_call(x.get_device(), lib.q2k_moe_sort, x.data_ptr(), x.numel(), rows.data_ptr(),
              offsets.data_ptr(), out.data_ptr(), out.numel(), ctypes.byref(p))
    return out


def moe_sort_backward(dxs, routes, out=None):
    """The gradient of ``moe_sort``'s x from that of its result: ``dx[t]``, the sum of
    ``dxs[routes.rows[t, s]]`` over the token's choices that have an expert."""
    if out is None:
        quick = _quick_mod or _quick()
        done = quick.sort_backward(dxs, routes.rows, routes.offsets) if quick else None
        if done.__class__ is int:
            _check(_lib, done)
        elif done is not None:
            return done
    p, rows, offsets = _moe_params(dxs, routes, "dxs", "choices")
    out = _moe_out(out, dxs, (p.n_tokens, p.width))
    lib = _lib if _lib is not None else load()
    _ffn_call(dxs.get_device(), lib.q2k_moe_sort_backward, dxs.data_ptr(), dxs.numel(),
              rows.data_ptr(), offsets.data_ptr(), out.data_ptr(), out.numel(), ctypes.byref(p))
    return out


def moe_combine(ys, routes, weights=None, residual=None, out=None):
    """The experts' rows back to their tokens: ``y[t] = residual[t] + sum_s weights[t, s]
    ys[routes.rows[t, s]]`` over the choices that have an expert.

    ``ys`` f32 or bf16 ``[n_tokens * top_k, width]``; ``weights`` f32 ``[n_tokens,
    top_k]`` or None (all 1); ``residual`` ``[n_tokens, width]`` in ys' dtype or None.
    The gradients are ``moe_combine_backward``'s; without weights ys' is ``moe_sort`` of
    y's.
    """
    if out is None:
        quick = _quick_mod or _quick()
        done = quick.combine(ys, routes.rows, routes.offsets, weights, residual) if quick else None
        if done.__class__ is int:
            _check(_lib, done)
        elif done is not None:
            return done
    torch = _torch_mod or _torch()
    p, rows, offsets = _moe_params(ys, routes, "ys", "choices")
    if weights is not None:
        _need_like(ys, weights=(torch.float32, rows.shape, weights))
    if residual is not None:
        _need_like(ys, residual=(ys.dtype, (p.n_tokens, p.width), residual))
    out = _moe_out(out, ys, (p.n_tokens, p.width))
    lib = _lib if _lib is not None else load()
    _ffn_call(ys.get_device(), lib.q2k_moe_combine, ys.data_ptr(), ys.numel(), rows.data_ptr(),
              offsets.data_ptr(), weights.data_ptr() if weights is not None else None,
              residual.data_ptr() if residual is not None else None, out.data_ptr(), out.numel(),
              ctypes.byref(p))
    return out


def moe_combine_backward(dy, ys, routes, weights):
    """The gradients of ``moe_combine``: ``(dys, dweights)`` from that of y.  ``dys`` as
    ``ys`` (zeros in rows without an expert), ``dweights`` f32 as ``weights``.  The
    residual's gradient is ``dy``.  Where ``moe_combine`` had no weights, ``dys`` is
    ``moe_sort(dy, routes)``."""
    quick = _quick_mod or _quick()
    done = quick.combine_backward(dy, ys, routes.rows, routes.offsets, weights) if quick else None
    if done.__class__ is int:
        _check(_lib, done)
    elif done is not None:
        return done
    torch = _torch_mod or _torch()
    p, rows, offsets = _moe_params(ys, routes, "ys", "choices")
    _need_like(ys, dy=(ys.dtype, (p.n_tokens, p.width), dy),
               weights=(torch.float32, rows.shape, weights))
    dys, dweights = torch.empty_like(ys), torch.empty_like(weights)
    lib = _lib if _lib is not None else load()
    _ffn_call(ys.get_device(), lib.q2k_moe_combine_backward, dy.data_ptr(), dy.numel(),
              ys.data_ptr(), ys.numel(), rows.data_ptr(), offsets.data_ptr(), weights.data_ptr(),
              dys.data_ptr(), dweights.data_ptr(), ctypes.byref(p))
    return dys, dweights


class GgufFile:
    """An open GGUF file (host only): ``names``, ``info(name)`` (a ``GgufTensor``:
    ggml_type, n_dims, dims innermost first, n_elements, offset, byte_len),
    ``read(name)`` (the bytes as a numpy uint8 array) and ``to_device(name)``
    (those bytes in a CUDA uint8 tensor, ready for ``matmul`` when the type is
    Q2_K).  Use as a context manager or call ``close``."""

    def __init__(self, path):
        self._lib = load()
        h = ctypes.c_void_p()
        _check(self._lib, self._lib.q2k_gguf_open(os.fsencode(path), ctypes.byref(h)))
        self._h = h

    def close(self):
        if self._h is not None and self._h.value:
            self._lib.q2k_gguf_close(self._h)
        self._h = None

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @property
    def names(self) -> list[str]:
        n = self._lib.q2k_gguf_tensor_count(self._h)
        return [self._lib.q2k_gguf_tensor_name(self._h, i).decode() for i in range(n)]

    def info(self, name: str) -> GgufTensor:
        out = GgufTensor()
        _check(self._lib, self._lib.q2k_gguf_tensor_info(self._h, name.encode(), ctypes.byref(out)))
        return out

    def read(self, name: str):
        import numpy as np
        n = self.info(name).byte_len
        buf = np.empty(n, dtype=np.uint8)
        _check(self._lib, self._lib.q2k_gguf_read_tensor(self._h, name.encode(),
                                                         buf.ctypes.data, n))
        return buf

    def to_device(self, name: str, device="cuda"):
        torch = _torch()
        return torch.from_numpy(self.read(name)).to(device)


def selftest_wait_timeout(limit_us: int = 2000, device=None) -> None:
    """Enqueue the library's bounded-wait self-test on the current stream: a kernel
    waits ~limit_us on a barrier nothing completes, gives up and sets the time-out
    bit that ``device_error()`` then returns."""
    torch = _torch()
    dev = torch.device("cuda", torch.cuda.current_device() if device is None else device)
    lib = load()
    with torch.cuda.device(dev):
        _check(lib, lib.q2k_selftest_wait_timeout(int(limit_us),
                                                  torch.cuda.current_stream(dev).cuda_stream))


def device_error(device=None) -> int:
    """Read and clear the device error word (nonzero: a kernel gave up waiting)."""
    torch = _torch()
    dev = torch.device("cuda", torch.cuda.current_device() if device is None else device)
    v = ctypes.c_uint32(0)
    lib = load()
    with torch.cuda.device(dev):
        _check(lib, lib.q2k_device_error(ctypes.byref(v),
                                         torch.cuda.current_stream(dev).cuda_stream))
    return int(v.value)
