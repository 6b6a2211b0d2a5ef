"""Thin Python binding of ``libspear.so`` (C ABI in ``include/spear.h``).

Argument marshalling only: every step of the layer runs in the library's
CUDA kernels.  Torch provides device memory and streams.  There is no CPU
fallback -- if the library cannot be loaded every call raises.

Function names follow the C ABI:
  spear_pack_w4, spear_linear_decode, spear_linear_prefill,
  spear_layer_select_mask, the paged key/value cache (spear_kv_*) and its
  attention (spear_attn_*), plus the workspace / status helpers.
"""
from __future__ import annotations

import ctypes
import os
import threading
from dataclasses import dataclass
from typing import Optional

import numpy as np
import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "lib", "libspear.so")

SPEAR_OK = 0
STATUS_NAMES = {0: "SPEAR_OK", 1: "SPEAR_ERR_INVALID_ARG", 2: "SPEAR_ERR_UNSUPPORTED",
                3: "SPEAR_ERR_WORKSPACE", 4: "SPEAR_ERR_CUDA", 5: "SPEAR_ERR_TIMEOUT", 6: "SPEAR_ERR_BOUNDS"}
PREFILL_AUTO, PREFILL_FUSED, PREFILL_STREAM = 0, 1, 2
OUT_BF16, OUT_F32 = 0, 1
DT_BF16, DT_F16 = 0, 1

# every symbol include/spear.h declares
EXPORTS = ["spear_pack_w4_sizes", "spear_pack_w4", "spear_decode_workspace_bytes",
           "spear_linear_decode", "spear_linear_decode_noalloc", "spear_prefill_workspace_bytes", "spear_linear_prefill",
           "spear_workspace_init", "spear_set_launch_overlap", "spear_set_wait_limit_ns", "spear_layer_select_mask",
           "spear_chunk_select",
           "spear_linear_cka", "spear_cka_damage",
           "spear_kv_append", "spear_attn_decode_workspace_bytes", "spear_attn_decode",
           "spear_attn_prefill_workspace_bytes", "spear_attn_prefill", "spear_kv_reserve", "spear_kv_fork",
           "spear_kv_free", "spear_kv_compact", "spear_kv_copy_pages",
           "spear_get_device_status", "spear_status_string", "spear_last_error", "spear_version"]


class SpearError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}: {detail}")
        self.status = status


class _Layer(ctypes.Structure):
    _fields_ = [("N", ctypes.c_int), ("K", ctypes.c_int), ("group_size", ctypes.c_int),
                ("symmetric", ctypes.c_int), ("qweight", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("zeros", ctypes.c_void_p), ("rank", ctypes.c_int), ("A", ctypes.c_void_p),
                ("B", ctypes.c_void_p), ("w_g", ctypes.c_void_p), ("b_g", ctypes.c_float),
                ("alpha", ctypes.c_float), ("comp_enabled", ctypes.c_int), ("gate_hidden", ctypes.c_int),
                ("gate_w1", ctypes.c_void_p), ("gate_c1", ctypes.c_void_p), ("gate_w2", ctypes.c_void_p),
                ("gate_c2", ctypes.c_void_p)]


class _Cache(ctypes.Structure):
    _fields_ = [("num_pages", ctypes.c_int), ("page_size", ctypes.c_int), ("num_kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("dtype", ctypes.c_int), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
                ("page_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64), ("slot_stride", ctypes.c_int64)]


class _Seqs(ctypes.Structure):
    _fields_ = [("num_seqs", ctypes.c_int), ("max_pages", ctypes.c_int), ("table_rows", ctypes.c_int),
                ("table_stride", ctypes.c_int64), ("block_table", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
                ("seq_ids", ctypes.c_void_p), ("refused", ctypes.c_void_p)]


class _Attn(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("q_token_stride", ctypes.c_int64), ("q_head_stride", ctypes.c_int64),
                ("num_q_heads", ctypes.c_int), ("scale", ctypes.c_float), ("window", ctypes.c_int),
                ("sinks", ctypes.c_int), ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p)]


class _Pool(ctypes.Structure):
    _fields_ = [("num_pages", ctypes.c_int), ("page_size", ctypes.c_int), ("max_seqs", ctypes.c_int),
                ("max_pages", ctypes.c_int), ("refs", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
                ("block_table", ctypes.c_void_p), ("moves", ctypes.c_void_p)]


_lock = threading.Lock()
_lib = None


def load(path: str = LIB_PATH):
    """Loads the CUDA library (once).  Raises if it is missing."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(f"libspear.so not found at {path}: build it first "
                               "(python -m quantized_gemm_error_gb300.build)")
        lib = ctypes.CDLL(path)
        P, I, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        LP = ctypes.POINTER(_Layer)
        sig = {
            "spear_pack_w4_sizes": [I, I, I, I, ctypes.POINTER(S), ctypes.POINTER(S), ctypes.POINTER(S)],
            "spear_pack_w4": [P, I, I, I, I, P, P, P, P],
            "spear_decode_workspace_bytes": [LP, I, ctypes.POINTER(S)],
            "spear_linear_decode": [LP, P, I, P, I, P, S, P],
            "spear_linear_decode_noalloc": [LP, P, I, P, I, P],
            "spear_prefill_workspace_bytes": [LP, I, I, ctypes.POINTER(S)],
            "spear_linear_prefill": [LP, P, I, P, I, I, P, S, P, P],
            "spear_workspace_init": [P, S, P],
            "spear_layer_select_mask": [P, P, I, ctypes.c_double, I, I, P, P],
            "spear_chunk_select": [P, P, I, I, P, I, ctypes.c_double, ctypes.POINTER(I), ctypes.POINTER(ctypes.c_double)],
            "spear_linear_cka": [P, P, I, I, I, ctypes.POINTER(ctypes.c_double)],
            "spear_cka_damage": [P, P, I, I, I, ctypes.POINTER(ctypes.c_double)],
            "spear_kv_append": [P, P, P, I, P, ctypes.c_int64, ctypes.c_int64, P, ctypes.c_int64, ctypes.c_int64, P],
            "spear_attn_decode_workspace_bytes": [P, I, I, P],
            "spear_attn_decode": [P, P, P, P, S, P],
            "spear_attn_prefill_workspace_bytes": [P, I, I, I, P],
            "spear_attn_prefill": [P, P, P, I, P, P, S, P],
            "spear_kv_reserve": [P, P, P, I, P],
            "spear_kv_fork": [P, P, I, P, P, I, P],
            "spear_kv_free": [P, P, I, P],
            "spear_kv_compact": [P, P, I, P],
            "spear_kv_copy_pages": [P, I, P, I, P],
            "spear_get_device_status": [ctypes.POINTER(I), P],
            "spear_set_launch_overlap": [I],
            "spear_set_wait_limit_ns": [ctypes.c_uint64],
        }
        for name, args in sig.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = I
        lib.spear_status_string.argtypes = [I]
        lib.spear_status_string.restype = ctypes.c_char_p
        lib.spear_last_error.argtypes = []
        lib.spear_last_error.restype = ctypes.c_char_p
        lib.spear_version.argtypes = []
        lib.spear_version.restype = ctypes.c_char_p
        _lib = lib
        return lib


def _check(rc: int, where: str):
    if rc != SPEAR_OK:
        detail = load().spear_last_error().decode(errors="replace")
        raise SpearError(rc, where, detail)


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return ctypes.c_void_p(t.data_ptr())


def _raw_stream(stream) -> int:
    if stream is None:                                # the current one, without making a Stream object of it
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _stream(stream) -> ctypes.c_void_p:
    return ctypes.c_void_p(_raw_stream(stream))


def _made_on(stream, make, *args, **kw) -> torch.Tensor:
    """make(*args, **kw), a tensor of the stream that a call runs on: memory of the current stream's could still be in use
    there by work that is queued.  It may be used on the current stream as well (once that waits for the call)."""
    if stream is None or _raw_stream(stream) == _raw_stream(None):
        return make(*args, **kw)
    here = torch.cuda.current_stream()
    with torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream) else
                           torch.cuda.ExternalStream(_raw_stream(stream))):
        t = make(*args, **kw)
    t.record_stream(here)
    return t


@dataclass
class W4Layer:
    """A packed layer plus its compensator (all tensors on the same CUDA device)."""
    N: int
    K: int
    group_size: int
    symmetric: bool
    qweight: torch.Tensor                 # uint8 [N][K/2]
    scales: torch.Tensor                  # fp16  [N][K/G]
    zeros: Optional[torch.Tensor] = None  # uint8 [N][ceil(K/G/2)]
    rank: int = 0
    A: Optional[torch.Tensor] = None      # bf16 [rank][K]
    B: Optional[torch.Tensor] = None      # bf16 [N][rank]
    w_g: Optional[torch.Tensor] = None    # bf16 [K]
    b_g: float = 0.0
    alpha: float = 1.0
    comp_enabled: bool = True
    # the vector gate gamma(A x) = sigmoid(W2 relu(W1 (A x) + c1) + c2), fp32 device
    # tensors W1 [h][rank], c1 [h], W2 [rank][h], c2 [rank]; None: the scalar gate
    gate_w1: Optional[torch.Tensor] = None
    gate_c1: Optional[torch.Tensor] = None
    gate_w2: Optional[torch.Tensor] = None
    gate_c2: Optional[torch.Tensor] = None

    def check(self):
        """Shapes and dtypes of the layer's tensors, which the C ABI (plain
        pointers) cannot see; the library checks the rest (shape rules, rank,
        hidden width, alignment)."""
        N, K, G, r = self.N, self.K, self.group_size, self.rank
        if G <= 0 or K % G:
            raise ValueError(f"group_size={G} must divide K={K}")

        def need(t, name, dtype, shape):
            if t is None:
                raise ValueError(f"{name} is missing")
            if t.dtype != dtype or tuple(t.shape) != tuple(shape):
                raise ValueError(f"{name} must be {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")

        need(self.qweight, "qweight", torch.uint8, (N, K // 2))
        need(self.scales, "scales", torch.float16, (N, K // G))
        if not self.symmetric:
            need(self.zeros, "zeros", torch.uint8, (N, (K // G + 1) // 2))
        if self.comp_enabled and r > 0:
            need(self.A, "A", torch.bfloat16, (r, K))
            need(self.B, "B", torch.bfloat16, (N, r))
            if self.gate_w1 is None:
                need(self.w_g, "w_g", torch.bfloat16, (K,))
            else:
                h = int(self.gate_w1.shape[0]) if self.gate_w1.dim() == 2 else -1
                need(self.gate_w1, "gate_w1", torch.float32, (h, r))
                need(self.gate_c1, "gate_c1", torch.float32, (h,))
                need(self.gate_w2, "gate_w2", torch.float32, (r, h))
                need(self.gate_c2, "gate_c2", torch.float32, (r,))

    def c_struct(self) -> _Layer:
        self.check()
        h = int(self.gate_w1.shape[0]) if self.gate_w1 is not None else 0
        return _Layer(self.N, self.K, self.group_size, int(self.symmetric), _ptr(self.qweight),
                      _ptr(self.scales), _ptr(self.zeros), int(self.rank), _ptr(self.A), _ptr(self.B),
                      _ptr(self.w_g), float(self.b_g), float(self.alpha), int(self.comp_enabled), h,
                      _ptr(self.gate_w1), _ptr(self.gate_c1), _ptr(self.gate_w2), _ptr(self.gate_c2))

    def with_comp(self, enabled: bool) -> "W4Layer":
        d = dict(self.__dict__)
        d["comp_enabled"] = enabled
        return W4Layer(**d)


# ------------------------------------------------------------------ pack

def spear_pack_w4_sizes(N: int, K: int, group_size: int, symmetric: bool):
    q, s, z = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
    _check(load().spear_pack_w4_sizes(N, K, group_size, int(symmetric), ctypes.byref(q), ctypes.byref(s),
                                      ctypes.byref(z)), "spear_pack_w4_sizes")
    return q.value, s.value, z.value


def spear_pack_w4(W: torch.Tensor, group_size: int, symmetric: bool, *, out=None, stream=None):
    """Quantise + pack W (CUDA fp32 [N][K]); returns (qweight, scales, zeros)."""
    if W.dtype != torch.float32 or W.dim() != 2:
        raise ValueError("W must be a 2-D float32 CUDA tensor")
    N, K = W.shape
    qb, sb, zb = spear_pack_w4_sizes(N, K, group_size, symmetric)
    if out is None:
        make = lambda n, dtype: _made_on(stream, torch.empty, (N, n), dtype=dtype, device=W.device)
        q, s = make(K // 2, torch.uint8), make(K // group_size, torch.float16)
        z = None if symmetric else make(zb // N, torch.uint8)
    else:
        q, s, z = out
    _check(load().spear_pack_w4(_ptr(W), N, K, group_size, int(symmetric), _ptr(q), _ptr(s), _ptr(z),
                                _stream(stream)), "spear_pack_w4")
    return q, s, z


# ---------------------------------------------------------------- layer

def spear_decode_workspace_bytes(layer: W4Layer, M: int) -> int:
    n = ctypes.c_size_t()
    L = layer.c_struct()
    _check(load().spear_decode_workspace_bytes(ctypes.byref(L), M, ctypes.byref(n)),
           "spear_decode_workspace_bytes")
    return n.value


def spear_prefill_workspace_bytes(layer: W4Layer, M: int, mode: int = PREFILL_AUTO) -> int:
    n = ctypes.c_size_t()
    L = layer.c_struct()
    _check(load().spear_prefill_workspace_bytes(ctypes.byref(L), M, mode, ctypes.byref(n)),
           "spear_prefill_workspace_bytes")
    return n.value


def new_workspace(nbytes: int, device, zero: bool = True) -> torch.Tensor:
    """A 256-byte aligned device buffer (torch allocations are) of at least nbytes."""
    ws = torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)
    if zero:
        spear_workspace_init(ws)
    return ws


# Workspaces of the calls made without one: one per (kind, device, stream),
# grown when a call needs more and otherwise reused.  Calls on one stream run
# in order, so they never use it at the same time; a decode workspace is left
# ready for the next call by the kernel itself.
_default_ws = {}


def _default_workspace(kind: str, nbytes: int, device, stream, zero: bool) -> torch.Tensor:
    dev = device if isinstance(device, torch.device) else torch.device(device)
    idx = dev.index if dev.index is not None else torch.cuda.current_device()
    key = (kind, idx, _raw_stream(stream))
    ws = _default_ws.get(key)
    if ws is None or ws.numel() < nbytes:
        ws = _made_on(stream, torch.empty, max(int(nbytes), 256), dtype=torch.uint8, device=torch.device("cuda", idx))
        if zero:
            spear_workspace_init(ws, stream)          # on the stream the calls use
        _default_ws[key] = ws
    return ws


def reset_default_workspaces() -> None:
    """Drops the workspaces kept for calls made without one (the next call
    makes a zeroed one): after spear_get_device_status reports
    SPEAR_ERR_TIMEOUT, or to release the memory."""
    _default_ws.clear()


def spear_workspace_init(ws: torch.Tensor, stream=None):
    _check(load().spear_workspace_init(_ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "spear_workspace_init")


def _check_io(layer: W4Layer, x: torch.Tensor, y: Optional[torch.Tensor], out_dtype: int):
    """Shapes and dtypes the C ABI cannot see: x bf16 [M][K]; y, when given,
    [M][N] in the requested output type (a wrong type would be written past
    its end)."""
    if x.dtype != torch.bfloat16 or x.dim() != 2 or x.shape[1] != layer.K:
        raise ValueError(f"x must be a bfloat16 [M][{layer.K}] tensor, got {x.dtype} {tuple(x.shape)}")
    if out_dtype not in (OUT_BF16, OUT_F32):
        raise ValueError(f"out_dtype must be OUT_BF16 or OUT_F32, got {out_dtype}")
    if y is not None:
        want = torch.float32 if out_dtype == OUT_F32 else torch.bfloat16
        if y.dtype != want or tuple(y.shape) != (x.shape[0], layer.N):
            raise ValueError(f"y must be a {want} [{x.shape[0]}][{layer.N}] tensor, got {y.dtype} "
                             f"{tuple(y.shape)}")


def _out(y, M, N, out_dtype, device, stream):
    if y is not None:
        return y
    return _made_on(stream, torch.empty, (M, N), dtype=torch.float32 if out_dtype == OUT_F32 else torch.bfloat16,
                    device=device)


def spear_linear_decode(layer: W4Layer, x: torch.Tensor, *, y=None, out_dtype: int = OUT_BF16,
                        workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """y = dequant(Wq) x + alpha g(x) B (A x) for M <= 64 tokens, one kernel launch.
    Without `workspace` the call uses the binding's workspace for this device
    and stream (made once, zeroed, then reused; see reset_default_workspaces)."""
    _check_io(layer, x, y, out_dtype)
    M = x.shape[0]
    y = _out(y, M, layer.N, out_dtype, x.device, stream)
    if workspace is None:
        workspace = _default_workspace("decode", spear_decode_workspace_bytes(layer, M), x.device, stream, True)
    L = layer.c_struct()
    _check(load().spear_linear_decode(ctypes.byref(L), _ptr(x), M, _ptr(y), out_dtype, _ptr(workspace),
                                      workspace.numel(), _stream(stream)), "spear_linear_decode")
    return y


def spear_linear_decode_noalloc(layer: W4Layer, x: torch.Tensor, *, y: torch.Tensor,
                                out_dtype: int = OUT_BF16, stream=None) -> torch.Tensor:
    """Decode for callers that cannot allocate device memory: the library keeps
    the scratch in a fixed 8 MiB array of its own, so the caller passes only
    inputs and the output buffer.  Calls that overlap on the GPU race."""
    _check_io(layer, x, y, out_dtype)
    L = layer.c_struct()
    _check(load().spear_linear_decode_noalloc(ctypes.byref(L), _ptr(x), x.shape[0], _ptr(y), out_dtype,
                                              _stream(stream)), "spear_linear_decode_noalloc")
    return y


def spear_linear_prefill(layer: W4Layer, x: torch.Tensor, *, y=None, out_dtype: int = OUT_BF16,
                         mode: int = PREFILL_AUTO, workspace: Optional[torch.Tensor] = None,
                         stream=None, stream_aux=None) -> torch.Tensor:
    """Same layer for large M on the tcgen05 tensor-core path."""
    _check_io(layer, x, y, out_dtype)
    M = x.shape[0]
    y = _out(y, M, layer.N, out_dtype, x.device, stream)
    if workspace is None:
        workspace = _default_workspace("prefill", spear_prefill_workspace_bytes(layer, M, mode), x.device, stream,
                                       False)
    L = layer.c_struct()
    aux = None if stream_aux is None else _stream(stream_aux)
    _check(load().spear_linear_prefill(ctypes.byref(L), _ptr(x), M, _ptr(y), out_dtype, mode,
                                       _ptr(workspace), workspace.numel(), _stream(stream), aux),
           "spear_linear_prefill")
    return y


# ------------------------------------- paged key/value cache and attention

_INT_MIN, _INT_MAX = -0x80000000, 0x7fffffff
_DT_OF = {torch.bfloat16: DT_BF16, torch.float16: DT_F16}


class KVCache:
    """One layer's cache: K and V, CUDA bf16 or fp16 [num_pages][kv_heads][page_size][head_dim] of equal strides
    (views are fine as long as a row's head_dim elements are contiguous; [pages][slots][heads][d] memory is a
    transposed view).  Keeps the tensors and the C description of them."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor):
        if k.dtype not in _DT_OF or v.dtype != k.dtype:
            raise ValueError(f"k and v must both be bfloat16 or float16, got {k.dtype} and {v.dtype}")
        if k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride():
            raise ValueError(f"k and v must be [pages][heads][slots][d] of equal strides, got {tuple(k.shape)} "
                             f"{k.stride()} and {tuple(v.shape)} {v.stride()}")
        if k.stride(3) != 1:
            raise ValueError("a cache row's elements must be contiguous")
        if not k.is_cuda or k.device != v.device:
            raise ValueError("k and v must be on one CUDA device")
        self.k, self.v, self.index = k, v, k.get_device()
        self.num_pages, self.num_kv_heads, self.page_size, self.head_dim = k.shape
        self.dtype, self.device = k.dtype, k.device
        self.c = _Cache(self.num_pages, self.page_size, self.num_kv_heads, self.head_dim, _DT_OF[k.dtype],
                        k.data_ptr(), v.data_ptr(), k.stride(0), k.stride(1), k.stride(2))
        self.ref = ctypes.byref(self.c)
        self._ws_bytes = {}                           # workspace bytes by call: the head size and the device make them

    def _workspace(self, kind: str, sizes: tuple, fn, zero: bool, stream) -> torch.Tensor:
        """The binding's workspace for a call on this cache (see _default_workspace)."""
        n = self._ws_bytes.get(kind)
        if n is None:
            n = self._ws_bytes[kind] = fn(self, *sizes)
        return _default_workspace(kind, n, self.device, stream, zero)


def new_kv_cache(num_pages: int, page_size: int, num_kv_heads: int, head_dim: int, device,
                 dtype: torch.dtype = torch.bfloat16) -> KVCache:
    """A zeroed cache of its own memory."""
    k, v = (torch.zeros(num_pages, num_kv_heads, page_size, head_dim, dtype=dtype, device=device) for _ in range(2))
    return KVCache(k, v)


class PagePool:
    """The pages' bookkeeping, shared by every layer's cache: page reference counts, block table and lengths on the
    device, in one int32 buffer `state` = [refs | seq_lens | block_table]."""

    def __init__(self, num_pages: int, page_size: int, max_seqs: int, max_pages: int, device):
        self.num_pages, self.page_size, self.max_seqs, self.max_pages = num_pages, page_size, max_seqs, max_pages
        self.state = torch.zeros(num_pages + max_seqs + max_seqs * max_pages, dtype=torch.int32, device=device)
        self.refs = self.state[:num_pages]
        self.seq_lens = self.state[num_pages:num_pages + max_seqs]
        self.block_table = self.state[num_pages + max_seqs:].view(max_seqs, max_pages)
        self.block_table.fill_(-1)
        # page moves of the last fork or compact: [0] their number, pairs (source, destination) from [2]; [1] is odd
        # while the last reserve was refused
        self.moves = torch.zeros(2 + 3 * num_pages, dtype=torch.int32, device=device)
        self.device, self.index = self.state.device, self.state.get_device()
        self.c = _Pool(num_pages, page_size, max_seqs, max_pages, self.refs.data_ptr(), self.seq_lens.data_ptr(),
                       self.block_table.data_ptr(), self.moves.data_ptr())
        self.ref = ctypes.byref(self.c)

    def snapshot(self) -> torch.Tensor:
        return self.state.clone()

    def restore(self, saved: torch.Tensor) -> None:
        if saved.dtype != torch.int32 or saved.shape != self.state.shape:
            raise ValueError(f"saved must be int32 {tuple(self.state.shape)}, got {saved.dtype} {tuple(saved.shape)}")
        self.state.copy_(saved)


# The tensors of a call are on the device of its cache or pool (`dev`, an index), which is the current one: the library
# launches there.

def _stream_on(dev: int, stream) -> int:
    if torch._C._cuda_getDevice() != dev:
        raise ValueError(f"the call's tensors are on cuda:{dev}, the current device is cuda:{torch.cuda.current_device()}")
    if stream is not None and getattr(stream, "device_index", dev) != dev:
        raise ValueError(f"the call's tensors are on cuda:{dev}, its stream on cuda:{stream.device_index}")
    return _raw_stream(stream)


def _bytes_ptr(t: torch.Tensor, dev: int) -> int:
    if t.dtype is not torch.uint8 or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"workspace must be a contiguous uint8 tensor on cuda:{dev}, got {t.dtype} on {t.device}")
    return t.data_ptr()


def _i32(t: torch.Tensor, name: str, n: Optional[int] = None, dev: Optional[int] = None) -> int:
    if dev is not None and t.get_device() != dev:
        raise ValueError(f"{name} must be on cuda:{dev}, got {t.device}")
    if t.dtype is not torch.int32 or t.dim() != 1 or not t.is_cuda or (n is not None and t.shape[0] != n):
        raise ValueError(f"{name} must be a 1-D int32 CUDA tensor{'' if n is None else f' of {n}'}, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _seqs(table: torch.Tensor, lens: torch.Tensor, ids: Optional[torch.Tensor], n: int, dev: int) -> _Seqs:
    if table.dtype is not torch.int32 or table.dim() != 2 or table.get_device() != dev or table.stride(1) != 1:
        raise ValueError(f"block_table must be an int32 [rows][max_pages] tensor on cuda:{dev} with contiguous rows")
    rows, cols = table.shape
    if ids is None and n > rows:
        raise ValueError(f"{n} sequences, but block_table has {rows} rows")
    return _Seqs(n, cols, rows, table.stride(0) if rows > 1 else cols, table.data_ptr(), _i32(lens, "seq_lens", rows, dev),
                 None if ids is None else _i32(ids, "seq_ids", n, dev))


def _token_rows(t: torch.Tensor, name: str, dtype, heads: Optional[int], D: int, dev: int):
    """(tokens, heads, token stride, head stride) of q or of new K/V rows; the stride of an extent of one counts as 0."""
    if t.dim() != 3 or t.dtype is not dtype or t.shape[2] != D or (heads is not None and t.shape[1] != heads):
        raise ValueError(f"{name} must be {dtype} [tokens][{'heads' if heads is None else heads}][{D}], got {t.dtype} "
                         f"{tuple(t.shape)}")
    st, sh, sd = t.stride()
    if sd != 1 or t.get_device() != dev:
        raise ValueError(f"{name} must be a tensor on cuda:{dev} whose rows of {D} elements are contiguous, got {t.device}")
    T, H, _ = t.shape
    return T, H, st if T > 1 else 0, sh if H > 1 else 0


def _attn(q, cache, scale, window, sinks, out, lse, stream):
    if not (_INT_MIN <= window <= _INT_MAX and _INT_MIN <= sinks <= _INT_MAX):         # ctypes would cut them to 32 bits
        raise ValueError(f"window and sinks are 32-bit numbers, got {window} and {sinks}")
    D, dev = cache.head_dim, cache.index
    T, H, st, sh = _token_rows(q, "q", cache.dtype, None, D, dev)
    if out is None:
        out = _made_on(stream, torch.empty_like, q, memory_format=torch.contiguous_format)
    elif out.dtype is not q.dtype or out.shape != q.shape or not out.is_contiguous() or out.get_device() != dev:
        raise ValueError(f"out must be a contiguous {q.dtype} {tuple(q.shape)} tensor on cuda:{dev}, got {out.dtype} "
                         f"{tuple(out.shape)} on {out.device}")
    if lse is None:
        p_lse = None
    elif lse.dtype is torch.float32 and lse.shape == (T, H) and lse.is_contiguous() and lse.get_device() == dev:
        p_lse = lse.data_ptr()
    else:
        raise ValueError(f"lse must be a contiguous float32 [{T}][{H}] tensor on cuda:{dev}, got {lse.dtype} "
                         f"{tuple(lse.shape)} on {lse.device}")
    return out, _Attn(q.data_ptr(), st, sh, H, D ** -0.5 if scale is None else scale, window, sinks, out.data_ptr(),
                      p_lse)


def spear_kv_append(cache: KVCache, k_new: torch.Tensor, v_new: torch.Tensor, block_table: torch.Tensor,
                    seq_lens: torch.Tensor, starts: torch.Tensor, *, seq_ids: Optional[torch.Tensor] = None,
                    pool: Optional[PagePool] = None, stream=None) -> None:
    """Writes the new tokens' rows k_new, v_new [tokens][kv_heads][head_dim] into their pages: rows [starts[b],
    starts[b + 1]) are the last tokens of sequence b, whose length seq_lens counts them already.  Pass the `pool`
    whose spear_kv_reserve made room for them: where it was refused the call then writes nothing and reports
    SPEAR_ERR_INVALID_ARG (without it the rows would replace the sequences' last cached ones)."""
    dev = cache.index
    T, _, kt, kh = _token_rows(k_new, "k_new", cache.dtype, cache.num_kv_heads, cache.head_dim, dev)
    Tv, _, vt, vh = _token_rows(v_new, "v_new", cache.dtype, cache.num_kv_heads, cache.head_dim, dev)
    if T != Tv:
        raise ValueError(f"k_new has {T} tokens, v_new {Tv}")
    p_starts, n = _i32(starts, "starts", None, dev), starts.shape[0] - 1
    s = _seqs(block_table, seq_lens, seq_ids, n, dev)
    if pool is not None:
        if pool.index != dev:
            raise ValueError(f"pool must be on cuda:{dev}, got {pool.device}")
        s.refused = pool.c.moves + 4
    _check(load().spear_kv_append(cache.ref, ctypes.byref(s), p_starts, T, k_new.data_ptr(), kt, kh,
                                  v_new.data_ptr(), vt, vh, _stream_on(dev, stream)), "spear_kv_append")


def spear_attn_decode_workspace_bytes(cache: KVCache, num_seqs: int, num_q_heads: int) -> int:
    n = ctypes.c_size_t()
    _check(load().spear_attn_decode_workspace_bytes(cache.ref, num_seqs, num_q_heads, ctypes.byref(n)),
           "spear_attn_decode_workspace_bytes")
    return n.value


def spear_attn_decode(q: torch.Tensor, cache: KVCache, block_table: torch.Tensor, seq_lens: torch.Tensor, *,
                      seq_ids: Optional[torch.Tensor] = None, scale: Optional[float] = None, window: int = 0,
                      sinks: int = 0, out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Attention of one new token of each sequence, q [seqs][q_heads][head_dim], over its cached keys (its own among
    them); scale defaults to head_dim ** -0.5.  `lse`, when given, receives the rows' log sums (fp32)."""
    raw, dev = _stream_on(cache.index, stream), cache.index
    out, a = _attn(q, cache, scale, window, sinks, out, lse, stream)
    s = _seqs(block_table, seq_lens, seq_ids, q.shape[0], dev)
    if workspace is None:
        workspace = cache._workspace("attn_decode", (s.num_seqs, a.num_q_heads), spear_attn_decode_workspace_bytes, True,
                                     stream)
    _check(load().spear_attn_decode(cache.ref, ctypes.byref(s), ctypes.byref(a), _bytes_ptr(workspace, dev),
                                    workspace.numel(), raw), "spear_attn_decode")
    return out


def spear_attn_prefill_workspace_bytes(cache: KVCache, num_seqs: int, num_tokens: int, num_q_heads: int) -> int:
    n = ctypes.c_size_t()
    _check(load().spear_attn_prefill_workspace_bytes(cache.ref, num_seqs, num_tokens, num_q_heads, ctypes.byref(n)),
           "spear_attn_prefill_workspace_bytes")
    return n.value


def spear_attn_prefill(q: torch.Tensor, cache: KVCache, block_table: torch.Tensor, seq_lens: torch.Tensor,
                       starts: torch.Tensor, *, seq_ids: Optional[torch.Tensor] = None,
                       scale: Optional[float] = None, window: int = 0, sinks: int = 0,
                       out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Causal attention of a ragged batch of new tokens, q [tokens][q_heads][head_dim], rows [starts[b],
    starts[b + 1]) the last tokens of sequence b; their K and V rows are in the cache already."""
    raw, dev = _stream_on(cache.index, stream), cache.index
    out, a = _attn(q, cache, scale, window, sinks, out, lse, stream)
    p_starts, n = _i32(starts, "starts", None, dev), starts.shape[0] - 1
    s = _seqs(block_table, seq_lens, seq_ids, n, dev)
    T = out.shape[0]
    if workspace is None:
        workspace = cache._workspace("attn_prefill", (n, T, a.num_q_heads), spear_attn_prefill_workspace_bytes, False,
                                     stream)
    _check(load().spear_attn_prefill(cache.ref, ctypes.byref(s), p_starts, T, ctypes.byref(a), _bytes_ptr(workspace, dev),
                                     workspace.numel(), raw), "spear_attn_prefill")
    return out


def spear_kv_reserve(pool: PagePool, rows: torch.Tensor, tokens: torch.Tensor, *, stream=None) -> None:
    """Lengthens each listed sequence by tokens[i], taking the pages it needs (the lowest free ones, in order)."""
    p_rows, n, dev = _i32(rows, "rows", None, pool.index), rows.shape[0], pool.index
    _check(load().spear_kv_reserve(pool.ref, p_rows, _i32(tokens, "tokens", n, dev), n, _stream_on(dev, stream)),
           "spear_kv_reserve")


def _caches(caches, dev: int):
    """(C array, count) of one cache or a list of them."""
    for c in (caches,) if isinstance(caches, KVCache) else caches:
        if c.index != dev:
            raise ValueError(f"the caches must be on cuda:{dev}, got {c.device}")
    if isinstance(caches, KVCache):
        return caches.ref, 1
    return (_Cache * max(1, len(caches)))(*[c.c for c in caches]), len(caches)


def spear_kv_fork(pool: PagePool, caches, parents: torch.Tensor, children: torch.Tensor, *, stream=None) -> None:
    """Makes each empty sequence children[i] a copy of parents[i]: whole pages shared, a partly filled one copied in
    every cache (one KVCache, or the list of all layers')."""
    p_par, n, dev = _i32(parents, "parents", None, pool.index), parents.shape[0], pool.index
    arr, count = _caches(caches, dev)
    _check(load().spear_kv_fork(pool.ref, arr, count, p_par, _i32(children, "children", n, dev), n,
                                _stream_on(dev, stream)), "spear_kv_fork")


def spear_kv_free(pool: PagePool, rows: torch.Tensor, *, stream=None) -> None:
    """Empties the listed sequences and gives up their references to pages."""
    _check(load().spear_kv_free(pool.ref, _i32(rows, "rows", None, pool.index), rows.shape[0],
                                _stream_on(pool.index, stream)), "spear_kv_free")


def spear_kv_compact(pool: PagePool, caches, *, stream=None) -> None:
    """Moves the live pages of every cache to the front of the pool and renames them in the block table."""
    arr, count = _caches(caches, pool.index)
    _check(load().spear_kv_compact(pool.ref, arr, count, _stream_on(pool.index, stream)), "spear_kv_compact")


def spear_kv_copy_pages(caches, moves: torch.Tensor, max_moves: Optional[int] = None, *, stream=None) -> None:
    """Copies moves[0] pages in every cache: pairs (source, destination) from moves[2]."""
    p_moves, room = _i32(moves, "moves"), (moves.shape[0] - 2) // 2
    if room < 0 or (max_moves is not None and max_moves > room):
        raise ValueError(f"moves holds {moves.shape[0]} words: 2, and 2 for each of up to {max_moves} pairs")
    dev = moves.get_device()
    arr, count = _caches(caches, dev)
    _check(load().spear_kv_copy_pages(arr, count, p_moves, room if max_moves is None else max_moves,
                                      _stream_on(dev, stream)), "spear_kv_copy_pages")


# ------------------------------------------------------- module selection

def spear_layer_select_mask(damage, cost, budget_bytes: float, rank_min: int, rank_max: int):
    d = np.ascontiguousarray(damage, dtype=np.float32)
    c = np.ascontiguousarray(cost, dtype=np.float32)
    mask = np.zeros(d.shape[0], np.uint8)
    rank = np.zeros(d.shape[0], np.int32)
    _check(load().spear_layer_select_mask(d.ctypes.data_as(ctypes.c_void_p), c.ctypes.data_as(ctypes.c_void_p),
                                          d.shape[0], float(budget_bytes), int(rank_min), int(rank_max),
                                          mask.ctypes.data_as(ctypes.c_void_p),
                                          rank.ctypes.data_as(ctypes.c_void_p)), "spear_layer_select_mask")
    return mask, rank


def spear_linear_cka(X, Y) -> float:
    """Linear CKA of two host activation matrices [n][dx], [n][dy] (fp32)."""
    x = np.ascontiguousarray(X, dtype=np.float32)
    y = np.ascontiguousarray(Y, dtype=np.float32)
    if x.ndim != 2 or y.ndim != 2 or x.shape[0] != y.shape[0]:
        raise ValueError("X and Y must be [n][d] with the same n")
    out = ctypes.c_double()
    _check(load().spear_linear_cka(x.ctypes.data_as(ctypes.c_void_p), y.ctypes.data_as(ctypes.c_void_p),
                                   x.shape[0], x.shape[1], y.shape[1], ctypes.byref(out)), "spear_linear_cka")
    return out.value


def spear_cka_damage(X_ref, Y_quant) -> float:
    """1 - CKA(X_ref, Y_quant) of two host matrices [n][dx], [n][dy] (fp32),
    computed by the library: one module's damage score."""
    x = np.ascontiguousarray(X_ref, dtype=np.float32)
    y = np.ascontiguousarray(Y_quant, dtype=np.float32)
    if x.ndim != 2 or y.ndim != 2 or x.shape[0] != y.shape[0]:
        raise ValueError("X_ref and Y_quant must be [n][d] with the same n")
    out = ctypes.c_double()
    _check(load().spear_cka_damage(x.ctypes.data_as(ctypes.c_void_p), y.ctypes.data_as(ctypes.c_void_p),
                                   x.shape[0], x.shape[1], y.shape[1], ctypes.byref(out)), "spear_cka_damage")
    return out.value


def cka_damage(reference_outputs, quantised_outputs):
    """Per-module damage scores for the module-selection rule (one
    spear_cka_damage call per module); each argument a list of host [n][d]
    matrices."""
    return np.array([spear_cka_damage(a, b) for a, b in zip(reference_outputs, quantised_outputs)],
                    dtype=np.float32)


class _Curve(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int), ("M", ctypes.c_void_p), ("us", ctypes.c_void_p)]


def spear_chunk_select(prefill_curves, decode_curves, decode_tokens: int, choices, itl_target_us: float):
    """prefill_curves / decode_curves: per layer, a pair (M list, microseconds list).
    Returns (chunk, predicted step microseconds)."""
    keep = []

    def curves(cs):
        arr = (_Curve * len(cs))()
        for i, (Ms, us) in enumerate(cs):
            m = np.ascontiguousarray(Ms, dtype=np.int32)
            u = np.ascontiguousarray(us, dtype=np.float32)
            keep.extend([m, u])
            arr[i] = _Curve(m.shape[0], m.ctypes.data, u.ctypes.data)
        return arr
    pre, dec = curves(prefill_curves), curves(decode_curves)
    ch = np.ascontiguousarray(choices, dtype=np.int32)
    out = ctypes.c_int()
    step = ctypes.c_double()
    _check(load().spear_chunk_select(ctypes.cast(pre, ctypes.c_void_p), ctypes.cast(dec, ctypes.c_void_p),
                                     len(prefill_curves), int(decode_tokens), ch.ctypes.data_as(ctypes.c_void_p),
                                     ch.shape[0], float(itl_target_us), ctypes.byref(out), ctypes.byref(step)),
           "spear_chunk_select")
    return out.value, step.value


# ------------------------------------------------------------ status

def spear_get_device_status(stream=None) -> int:
    out = ctypes.c_int()
    _check(load().spear_get_device_status(ctypes.byref(out), _stream(stream)), "spear_get_device_status")
    return out.value


def spear_set_launch_overlap(enable: bool) -> None:
    """Process-wide: decode launches may start while the previous kernel on
    their stream finishes (programmatic dependent launch).  The caller
    guarantees that the kernel right before a decode call does not write that
    layer's weights; see include/spear.h."""
    _check(load().spear_set_launch_overlap(1 if enable else 0), "spear_set_launch_overlap")


def spear_set_wait_limit_ns(ns: int) -> None:
    """Process-wide limit of the device-side waits on other thread blocks (0:
    the defaults); a wait that runs out records SPEAR_ERR_TIMEOUT.  For tests
    and diagnostics; see include/spear.h."""
    _check(load().spear_set_wait_limit_ns(int(ns)), "spear_set_wait_limit_ns")


def version() -> str:
    return load().spear_version().decode()
