"""Thin torch wrappers over the libmoe calls (router projection, gate,
permutation, grouped FFN, combine, statistics).

Argument marshalling only: shapes, dtypes and contiguity are checked, outputs
and workspaces are allocated with torch on the input's device, and the call is
enqueued on torch's current stream.  Every step of the path runs in libmoe's
HIP kernels; there is no fallback.
"""
from __future__ import annotations

import ctypes
from typing import Dict, Optional

import torch

from . import _lib
from ._lib import MOE_BF16, MOE_F32, check


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _stream(dev: torch.device) -> int:
    return torch.cuda.current_stream(dev).cuda_stream


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype == torch.bfloat16:
        return MOE_BF16
    if t.dtype == torch.float32:
        return MOE_F32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _need(t: torch.Tensor, name: str, dtype=None, ndim=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims")


def _out(t: torch.Tensor, name: str, dtype, shape):
    """A caller-supplied output: a contiguous GPU tensor of exactly this dtype and shape."""
    _need(t, name, dtype, len(shape))
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _same_device(first: torch.Tensor, **others: Optional[torch.Tensor]):
    for name, t in others.items():
        if t is not None and t.device != first.device:
            raise ValueError(f"{name} must be on {first.device}, got {t.device}")


def _ok(t: torch.Tensor, index: int, dtype, shape) -> bool:
    """A contiguous tensor of this dtype and shape on GPU `index` (the checks of
    _out and _same_device in one cheap test: a small call's time is its host side)."""
    return t.dtype is dtype and t.get_device() == index and t.shape == shape and t.is_contiguous()


def _new(rows: int, cols: int, dtype, index: int) -> torch.Tensor:
    """torch.empty((rows, cols)) on GPU `index`, in three quarters of its time."""
    return torch.empty_strided((rows, cols), (cols, 1), dtype=dtype, device=index)


def _int32_rows(x: torch.Tensor, d: int) -> None:
    """The C calls take rows and columns as int32, and ctypes would pass on the low 32 bits of more."""
    if d > 2 ** 31 - 1 or x.numel() > (2 ** 31 - 1) * d:
        raise ValueError("x must have fewer than 2^31 rows and columns")


def _call(name: str, index: int, fn, *args) -> None:
    """fn(*args, stream) on GPU `index` and its current stream."""
    if torch._C._cuda_getDevice() == index:
        status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(index))
    if status != _lib.MOE_OK:
        raise _lib.MoeError(name, status)


def _workspace(fn, args_before_ws, dev) -> torch.Tensor:
    """Query a call's workspace size (NULL workspace) and allocate it."""
    n = ctypes.c_size_t(0)
    check(fn.__name__, fn(*args_before_ws, None, ctypes.byref(n), None))
    return torch.empty(max(int(n.value), 256), dtype=torch.uint8, device=dev)


def router(x: torch.Tensor, w_router: torch.Tensor, logits: Optional[torch.Tensor] = None) -> torch.Tensor:
    """fp32 router logits [T][E] = x [T][d] . w_router [E][d]^T (bf16 or fp32 inputs)."""
    _need(x, "x", None, 2)
    _need(w_router, "w_router", x.dtype, 2)
    T, d = x.shape
    E = w_router.shape[0]
    if w_router.shape[1] != d:
        raise ValueError("w_router must be [E][d]")
    dev = x.device
    if logits is None:
        logits = torch.empty((T, E), dtype=torch.float32, device=dev)
    _out(logits, "logits", torch.float32, (T, E))
    lib = _lib.load()
    check("moe_router", lib.moe_router(_ptr(x), _ptr(w_router), T, d, E, _dtype_code(x), _ptr(logits),
                                       _stream(dev)))
    return logits


def gate(logits: torch.Tensor, k: int, renormalize: bool = True,
         topk_ids: Optional[torch.Tensor] = None, topk_w: Optional[torch.Tensor] = None):
    _need(logits, "logits", torch.float32, 2)
    T, E = logits.shape
    dev = logits.device
    if topk_ids is None:
        topk_ids = torch.empty((T, k), dtype=torch.int32, device=dev)
    if topk_w is None:
        topk_w = torch.empty((T, k), dtype=torch.float32, device=dev)
    _out(topk_ids, "topk_ids", torch.int32, (T, k))
    _out(topk_w, "topk_w", torch.float32, (T, k))
    lib = _lib.load()
    check("moe_gate", lib.moe_gate(_ptr(logits), T, E, k, int(bool(renormalize)), _ptr(topk_ids),
                                   _ptr(topk_w), _stream(dev)))
    return topk_ids, topk_w


def gate_record(logits: torch.Tensor, k: int, block_tokens: int, layer: int, block_counts: torch.Tensor,
                renormalize: bool = True, topk_ids: Optional[torch.Tensor] = None,
                topk_w: Optional[torch.Tensor] = None):
    """gate() that also fills row `layer` of the KV-block record block_counts
    [ceil(T / block_tokens)][L][E] int32 (moe_gate_record)."""
    _need(logits, "logits", torch.float32, 2)
    T, E = logits.shape
    dev = logits.device
    if block_tokens < 1:
        raise ValueError("block_tokens must be >= 1")
    nb = -(-T // block_tokens)
    _need(block_counts, "block_counts", torch.int32, 3)
    L = block_counts.shape[1]
    _out(block_counts, "block_counts", torch.int32, (nb, L, E))
    if topk_ids is None:
        topk_ids = torch.empty((T, k), dtype=torch.int32, device=dev)
    if topk_w is None:
        topk_w = torch.empty((T, k), dtype=torch.float32, device=dev)
    _out(topk_ids, "topk_ids", torch.int32, (T, k))
    _out(topk_w, "topk_w", torch.float32, (T, k))
    lib = _lib.load()
    check("moe_gate_record", lib.moe_gate_record(_ptr(logits), T, E, k, int(bool(renormalize)), _ptr(topk_ids),
                                                 _ptr(topk_w), block_tokens, layer, L, _ptr(block_counts),
                                                 _stream(dev)))
    return topk_ids, topk_w


def route(logits: torch.Tensor, k: int, score: str = "softmax", bias: Optional[torch.Tensor] = None,
          n_groups: int = 1, top_groups: Optional[int] = None, group_rank: str = "max", renormalize: bool = True,
          scale: float = 1.0, topk_ids: Optional[torch.Tensor] = None, topk_w: Optional[torch.Tensor] = None):
    """k experts and weights per token from scores (moe_route): softmax or
    sigmoid of the logits [T][E] (fp32 or bf16), `bias` ([E] fp32) added for the
    selection only, the experts in `n_groups` groups of which the `top_groups`
    best stay (all, if not given), weights renormalised and scaled."""
    _need(logits, "logits", None, 2)
    T, E = logits.shape
    index = logits.get_device()
    if score not in _lib.SCORES:
        raise ValueError(f"score must be one of {sorted(_lib.SCORES)}")
    if group_rank not in _lib.GROUP_RANKS:
        raise ValueError(f"group_rank must be one of {sorted(_lib.GROUP_RANKS)}")
    if bias is not None and not _ok(bias, index, torch.float32, (E,)):
        _out(bias, "bias", torch.float32, (E,))
        _same_device(logits, bias=bias)
    if topk_ids is None:
        topk_ids = _new(T, k, torch.int32, index)
    elif not _ok(topk_ids, index, torch.int32, (T, k)):
        _out(topk_ids, "topk_ids", torch.int32, (T, k))
        _same_device(logits, topk_ids=topk_ids)
    if topk_w is None:
        topk_w = _new(T, k, torch.float32, index)
    elif not _ok(topk_w, index, torch.float32, (T, k)):
        _out(topk_w, "topk_w", torch.float32, (T, k))
        _same_device(logits, topk_w=topk_w)
    _call("moe_route", index, _lib.load().moe_route, logits.data_ptr(), _dtype_code(logits), _ptr(bias), T, E, k,
          _lib.SCORES[score], n_groups, n_groups if top_groups is None else top_groups, _lib.GROUP_RANKS[group_rank],
          1 if renormalize else 0, scale, topk_ids.data_ptr(), topk_w.data_ptr())
    return topk_ids, topk_w


def stage_to_host(src: torch.Tensor, dst: torch.Tensor) -> torch.Tensor:
    """Enqueue the copy of GPU tensor `src` into the pinned host tensor `dst`
    (same dtype and shape) on the current stream (moe_stage_to_host); read
    `dst` after synchronising that stream."""
    _need(src, "src")
    if dst.is_cuda or not dst.is_contiguous():
        raise ValueError("dst must be a contiguous host tensor")
    if dst.dtype != src.dtype or dst.shape != src.shape:
        raise ValueError("dst must match src in dtype and shape")
    lib = _lib.load()
    check("moe_stage_to_host", lib.moe_stage_to_host(_ptr(src), ctypes.c_void_p(dst.data_ptr()),
                                                     src.numel() * src.element_size(), _stream(src.device)))
    return dst


def permute_workspace_bytes(T, E, k, n_shared=0, n_priority=0) -> int:
    lib = _lib.load()
    n = ctypes.c_size_t(0)
    check("moe_permute", lib.moe_permute(None, T, E, k, n_shared, n_priority, None, MOE_BF16, 8,
                                         None, None, None, None, None, None, ctypes.byref(n), None))
    return int(n.value)


def permute(topk_ids: torch.Tensor, E: int, n_shared: int = 0, n_priority: int = 0,
            x: Optional[torch.Tensor] = None, out: Optional[Dict[str, torch.Tensor]] = None,
            workspace: Optional[torch.Tensor] = None, sorted_token: bool = True) -> Dict[str, torch.Tensor]:
    """Counting sort of the assignments; `sorted_token` also writes the token
    of every sorted row (the row list moe_grouped_ffn can read x through)."""
    _need(topk_ids, "topk_ids", torch.int32, 2)
    T, k = topk_ids.shape
    dev = topk_ids.device
    nseg = 2 if n_priority > 0 else 1
    G = nseg * E + n_shared
    N = T * (k + n_shared)
    d = 8
    dt = MOE_BF16
    if x is not None:
        _need(x, "x", None, 2)
        if x.shape[0] != T:
            raise ValueError(f"x must have {T} rows, one per token")
        d = x.shape[1]
        dt = _dtype_code(x)
    o = {} if out is None else out
    if "group_offsets" not in o:
        o["group_offsets"] = torch.empty(G + 1, dtype=torch.int32, device=dev)
    if "sorted_to_flat" not in o:
        o["sorted_to_flat"] = torch.empty(N, dtype=torch.int32, device=dev)
    if "flat_to_sorted" not in o:
        o["flat_to_sorted"] = torch.empty(N, dtype=torch.int32, device=dev)
    if sorted_token and "sorted_token" not in o:
        o["sorted_token"] = torch.empty(N, dtype=torch.int32, device=dev)
    if x is not None and "x_sorted" not in o:
        o["x_sorted"] = torch.empty((N, d), dtype=x.dtype, device=dev)
    _out(o["group_offsets"], "group_offsets", torch.int32, (G + 1,))
    for key in ("sorted_to_flat", "flat_to_sorted") + (("sorted_token",) if sorted_token else ()):
        _out(o[key], key, torch.int32, (N,))
    if x is not None:
        _out(o["x_sorted"], "x_sorted", x.dtype, (N, d))
    if workspace is None:
        workspace = torch.empty(max(permute_workspace_bytes(T, E, k, n_shared, n_priority), 256),
                                dtype=torch.uint8, device=dev)
    lib = _lib.load()
    nbytes = ctypes.c_size_t(workspace.numel())
    check("moe_permute", lib.moe_permute(
        _ptr(topk_ids), T, E, k, n_shared, n_priority, _ptr(x), dt, d,
        _ptr(o["group_offsets"]), _ptr(o["sorted_to_flat"]), _ptr(o["flat_to_sorted"]),
        _ptr(o.get("sorted_token")) if sorted_token else None,
        _ptr(o.get("x_sorted")) if x is not None else None,
        _ptr(workspace), ctypes.byref(nbytes), _stream(dev)))
    return o


def ffn_workspace_bytes(n_rows, E, n_shared, nseg, d, I, dtype=torch.bfloat16) -> int:
    lib = _lib.load()
    n = ctypes.c_size_t(0)
    code = MOE_BF16 if dtype == torch.bfloat16 else MOE_F32
    check("moe_grouped_ffn", lib.moe_grouped_ffn(None, None, 0, None, n_rows, E, n_shared, nseg, d, I, None, None,
                                                 None, code, None, None, ctypes.byref(n), None))
    return int(n.value)


def grouped_ffn(x_sorted: torch.Tensor, group_offsets: torch.Tensor, E: int, n_shared: int, nseg: int,
                w_gate: torch.Tensor, w_up: torch.Tensor, w_down: torch.Tensor,
                h_sorted: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None,
                x_rows: Optional[torch.Tensor] = None,
                trace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Grouped SwiGLU FFN.  With `x_rows` ([N] int32, e.g. permute's
    sorted_token) `x_sorted` is the unsorted token matrix and sorted row n
    reads its row x_rows[n].  With `trace` ([R][4] int64, zero-filled by the
    caller) the persistent-queue path records one line per tile
    (moe_grouped_ffn_traced)."""
    _need(x_sorted, "x_sorted", None, 2)
    _need(group_offsets, "group_offsets", torch.int32, 1)
    for name, w in (("w_gate", w_gate), ("w_up", w_up), ("w_down", w_down)):
        _need(w, name, x_sorted.dtype, 3)
    n_x, d = x_sorted.shape
    N = n_x
    if x_rows is not None:
        _need(x_rows, "x_rows", torch.int32, 1)
        N = x_rows.numel()
    I = w_gate.shape[1]
    if w_gate.shape != (E + n_shared, I, d) or w_up.shape != w_gate.shape or w_down.shape != (E + n_shared, d, I):
        raise ValueError("expert weight shapes do not match [E+S][I][d] / [E+S][d][I]")
    if group_offsets.numel() != nseg * E + n_shared + 1:
        raise ValueError("group_offsets must have nseg*E + n_shared + 1 entries")
    dev = x_sorted.device
    if h_sorted is None:
        h_sorted = torch.empty((N, d), dtype=x_sorted.dtype, device=dev)
    _need(h_sorted, "h_sorted", x_sorted.dtype, 2)
    if h_sorted.shape != (N, d):
        raise ValueError(f"h_sorted must be [{N}][{d}]")
    if workspace is None:
        workspace = torch.empty(max(ffn_workspace_bytes(N, E, n_shared, nseg, d, I, x_sorted.dtype), 256),
                                dtype=torch.uint8, device=dev)
    lib = _lib.load()
    nbytes = ctypes.c_size_t(workspace.numel())
    args = (_ptr(x_sorted), _ptr(x_rows), n_x, _ptr(group_offsets), N, E, n_shared, nseg, d, I, _ptr(w_gate),
            _ptr(w_up), _ptr(w_down), _dtype_code(x_sorted), _ptr(h_sorted), _ptr(workspace), ctypes.byref(nbytes))
    if trace is None:
        check("moe_grouped_ffn", lib.moe_grouped_ffn(*args, _stream(dev)))
    else:
        _need_trace(trace)
        check("moe_grouped_ffn_traced", lib.moe_grouped_ffn_traced(*args, _ptr(trace), trace.shape[0], 0,
                                                                   _stream(dev)))
    return h_sorted


def _need_trace(trace: torch.Tensor):
    _need(trace, "trace", torch.int64, 2)
    if trace.shape[1] != 4:
        raise ValueError("trace must be [records][4] int64")


def ffn_combine_workspace_bytes(N, E, n_shared, nseg, d, I, T, k, packed=False) -> int:
    """Workspace of moe_grouped_ffn_combine (raises MoeError for a batch it
    does not serve)."""
    lib = _lib.load()
    n = ctypes.c_size_t(0)
    check("moe_grouped_ffn_combine", lib.moe_grouped_ffn_combine(
        None, None, 0, None, N, E, n_shared, nseg, d, I, None, None, None, int(bool(packed)), None, None, T, k,
        None, None, ctypes.byref(n), None))
    return int(n.value)


def grouped_ffn_combine(x_sorted: torch.Tensor, group_offsets: torch.Tensor, E: int, n_shared: int, nseg: int,
                        w_gate: torch.Tensor, w_up: torch.Tensor, w_down: torch.Tensor,
                        sorted_to_flat: torch.Tensor, topk_w: torch.Tensor, y: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, x_rows: Optional[torch.Tensor] = None,
                        packed: bool = False) -> torch.Tensor:
    """grouped_ffn then combine in one call, the combine folded into the down
    projection (moe_grouped_ffn_combine; bf16, decode-sized batches).  With
    `packed` the weights come from pack_weights."""
    _need(x_sorted, "x_sorted", torch.bfloat16, 2)
    _need(group_offsets, "group_offsets", torch.int32, 1)
    for name, w in (("w_gate", w_gate), ("w_up", w_up), ("w_down", w_down)):
        _need(w, name, torch.bfloat16, 3)
    _need(sorted_to_flat, "sorted_to_flat", torch.int32, 1)
    _need(topk_w, "topk_w", torch.float32, 2)
    n_x, d = x_sorted.shape
    N = sorted_to_flat.numel()
    if x_rows is not None:
        _need(x_rows, "x_rows", torch.int32, 1)
        if x_rows.numel() != N:
            raise ValueError("x_rows and sorted_to_flat must have one entry per sorted row")
    elif n_x != N:
        raise ValueError("x_sorted must have one row per sorted row")
    T, k = topk_w.shape
    I = w_gate.shape[1]
    if w_gate.shape != (E + n_shared, I, d) or w_up.shape != w_gate.shape or w_down.shape != (E + n_shared, d, I):
        raise ValueError("expert weight shapes do not match [E+S][I][d] / [E+S][d][I]")
    if group_offsets.numel() != nseg * E + n_shared + 1:
        raise ValueError("group_offsets must have nseg*E + n_shared + 1 entries")
    dev = x_sorted.device
    if y is None:
        y = torch.empty((T, d), dtype=torch.bfloat16, device=dev)
    _out(y, "y", torch.bfloat16, (T, d))
    if workspace is None:
        workspace = torch.empty(max(ffn_combine_workspace_bytes(N, E, n_shared, nseg, d, I, T, k, packed), 256),
                                dtype=torch.uint8, device=dev)
    lib = _lib.load()
    nbytes = ctypes.c_size_t(workspace.numel())
    check("moe_grouped_ffn_combine", lib.moe_grouped_ffn_combine(
        _ptr(x_sorted), _ptr(x_rows), n_x, _ptr(group_offsets), N, E, n_shared, nseg, d, I, _ptr(w_gate),
        _ptr(w_up), _ptr(w_down), int(bool(packed)), _ptr(sorted_to_flat), _ptr(topk_w), T, k, _ptr(y),
        _ptr(workspace), ctypes.byref(nbytes), _stream(dev)))
    return y


NOALLOC_SCRATCH_BYTES = 64 << 20


def grouped_ffn_noalloc(x_sorted: torch.Tensor, group_offsets: torch.Tensor, E: int, n_shared: int, nseg: int,
                        w_gate: torch.Tensor, w_up: torch.Tensor, w_down: torch.Tensor, h_sorted: torch.Tensor,
                        x_rows: Optional[torch.Tensor] = None) -> torch.Tensor:
    """grouped_ffn on the library's per-device scratch array
    (moe_grouped_ffn_noalloc): no workspace, nothing allocated by the call.
    The caller passes the output; calls on one GPU must not overlap."""
    _need(x_sorted, "x_sorted", None, 2)
    _need(group_offsets, "group_offsets", torch.int32, 1)
    for name, w in (("w_gate", w_gate), ("w_up", w_up), ("w_down", w_down)):
        _need(w, name, x_sorted.dtype, 3)
    n_x, d = x_sorted.shape
    N = n_x
    if x_rows is not None:
        _need(x_rows, "x_rows", torch.int32, 1)
        N = x_rows.numel()
    I = w_gate.shape[1]
    if w_gate.shape != (E + n_shared, I, d) or w_up.shape != w_gate.shape or w_down.shape != (E + n_shared, d, I):
        raise ValueError("expert weight shapes do not match [E+S][I][d] / [E+S][d][I]")
    if group_offsets.numel() != nseg * E + n_shared + 1:
        raise ValueError("group_offsets must have nseg*E + n_shared + 1 entries")
    _out(h_sorted, "h_sorted", x_sorted.dtype, (N, d))
    lib = _lib.load()
    check("moe_grouped_ffn_noalloc", lib.moe_grouped_ffn_noalloc(
        _ptr(x_sorted), _ptr(x_rows), n_x, _ptr(group_offsets), N, E, n_shared, nseg, d, I, _ptr(w_gate),
        _ptr(w_up), _ptr(w_down), _dtype_code(x_sorted), _ptr(h_sorted), _stream(x_sorted.device)))
    return h_sorted


def pack_weights(w: torch.Tensor) -> torch.Tensor:
    """Expert matrices [..][R][K] in the layout moe_grouped_ffn_packed reads:
    blocks of 16 rows x 32 K values, block (r/16, k/32) at element offset
    ((r/16) * (K/32) + k/32) * 512 of each matrix, and W[r][k] at
    (((k%32)/8) * 16 + r%16) * 8 + k%8 inside its block.  The result keeps the
    input's shape (and each matrix its place); a one-time weight preparation."""
    *lead, R, K = w.shape
    if R % 16 != 0 or K % 32 != 0:
        raise ValueError("packing needs rows % 16 == 0 and K % 32 == 0")
    v = w.reshape(*lead, R // 16, 16, K // 32, 4, 8)       # r = 16 rb + r16, k = 32 kb + 8 q + t
    n = len(lead)
    return v.permute(*range(n), n, n + 2, n + 3, n + 1, n + 4).contiguous().reshape(w.shape)


def grouped_ffn_packed(x_sorted: torch.Tensor, group_offsets: torch.Tensor, E: int, n_shared: int, nseg: int,
                       w_gate: torch.Tensor, w_up: torch.Tensor, w_down: torch.Tensor,
                       h_sorted: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                       x_rows: Optional[torch.Tensor] = None,
                       trace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """grouped_ffn (bf16, any batch size) with weights from pack_weights;
    `trace` as in grouped_ffn (moe_grouped_ffn_traced with packed weights)."""
    _need(x_sorted, "x_sorted", torch.bfloat16, 2)
    _need(group_offsets, "group_offsets", torch.int32, 1)
    for name, w in (("w_gate", w_gate), ("w_up", w_up), ("w_down", w_down)):
        _need(w, name, torch.bfloat16, 3)
    n_x, d = x_sorted.shape
    N = n_x
    if x_rows is not None:
        _need(x_rows, "x_rows", torch.int32, 1)
        N = x_rows.numel()
    I = w_gate.shape[1]
    if w_gate.shape != (E + n_shared, I, d) or w_up.shape != w_gate.shape or w_down.shape != (E + n_shared, d, I):
        raise ValueError("expert weight shapes do not match [E+S][I][d] / [E+S][d][I]")
    if group_offsets.numel() != nseg * E + n_shared + 1:
        raise ValueError("group_offsets must have nseg*E + n_shared + 1 entries")
    dev = x_sorted.device
    if h_sorted is None:
        h_sorted = torch.empty((N, d), dtype=torch.bfloat16, device=dev)
    _out(h_sorted, "h_sorted", torch.bfloat16, (N, d))
    if workspace is None:
        workspace = torch.empty(max(ffn_workspace_bytes(N, E, n_shared, nseg, d, I, torch.bfloat16), 256),
                                dtype=torch.uint8, device=dev)
    lib = _lib.load()
    nbytes = ctypes.c_size_t(workspace.numel())
    if trace is None:
        check("moe_grouped_ffn_packed", lib.moe_grouped_ffn_packed(
            _ptr(x_sorted), _ptr(x_rows), n_x, _ptr(group_offsets), N, E, n_shared, nseg, d, I, _ptr(w_gate),
            _ptr(w_up), _ptr(w_down), _ptr(h_sorted), _ptr(workspace), ctypes.byref(nbytes), _stream(dev)))
    else:
        _need_trace(trace)
        check("moe_grouped_ffn_traced", lib.moe_grouped_ffn_traced(
            _ptr(x_sorted), _ptr(x_rows), n_x, _ptr(group_offsets), N, E, n_shared, nseg, d, I, _ptr(w_gate),
            _ptr(w_up), _ptr(w_down), _dtype_code(x_sorted), _ptr(h_sorted), _ptr(workspace), ctypes.byref(nbytes),
            _ptr(trace), trace.shape[0], 1, _stream(dev)))
    return h_sorted


def ffn_fp8w_workspace_bytes(n_rows, I, E=1, n_shared=0, nseg=1, d=64, packed=False) -> int:
    """Workspace of the FP8-weight FFN (the SwiGLU intermediate, plus the
    persistent queue's state for the batches that may run on it)."""
    lib = _lib.load()
    n = ctypes.c_size_t(0)
    name = "moe_grouped_ffn_fp8w_packed" if packed else "moe_grouped_ffn_fp8w"
    check(name, getattr(lib, name)(None, None, 0, None, n_rows, E, n_shared, nseg, d, I, None, None, None, None,
                                   None, None, None, None, ctypes.byref(n), None))
    return int(n.value)


def quantize_fp8_rows(w: torch.Tensor):
    """Per-row E4M3 quantisation of [..][rows][cols] weights: scale = max|row| / 448
    (1 for an all-zero row), codes = round-to-nearest-even(w / scale).  Input
    preparation for moe_grouped_ffn_fp8w; returns (codes uint8, scales fp32)."""
    wf = w.float()
    s = wf.abs().amax(dim=-1) / 448.0
    s = torch.where(s > 0, s, torch.ones_like(s))
    q = (wf / s.unsqueeze(-1)).to(torch.float8_e4m3fn).view(torch.uint8)
    return q.contiguous(), s.contiguous()


def pack_fp8_codes(q: torch.Tensor) -> torch.Tensor:
    """E4M3 code matrices [..][R][K] (uint8 or float8_e4m3fn) in the layout
    moe_grouped_ffn_fp8w_packed and the FP8 products read: blocks of 16 rows x 64 codes, block
    (r/16, k/64) at byte ((r/16) * (K/64) + k/64) * 1024 of each matrix and
    C[r][k] at (((k%64)/16) * 16 + r%16) * 16 + k%16 inside it; same shape."""
    *lead, R, K = q.shape
    if R % 16 != 0 or K % 64 != 0:
        raise ValueError("packing needs rows % 16 == 0 and K % 64 == 0")
    v = q.reshape(*lead, R // 16, 16, K // 64, 4, 16)      # r = 16 rb + r16, k = 64 kb + 16 j + t
    n = len(lead)
    return v.permute(*range(n), n, n + 2, n + 3, n + 1, n + 4).contiguous().reshape(q.shape)


def grouped_ffn_fp8w(x: torch.Tensor, group_offsets: torch.Tensor, E: int, n_shared: int, nseg: int,
                     w_gate: torch.Tensor, s_gate: torch.Tensor, w_up: torch.Tensor, s_up: torch.Tensor,
                     w_down: torch.Tensor, s_down: torch.Tensor, h_sorted: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, x_rows: Optional[torch.Tensor] = None,
                     packed: bool = False) -> torch.Tensor:
    """The expert FFN with E4M3 weight codes (uint8) and fp32 per-row scales;
    bf16 token rows, read directly or through `x_rows`.  packed: the codes come
    from pack_fp8_codes (moe_grouped_ffn_fp8w_packed)."""
    _need(x, "x", torch.bfloat16, 2)
    for t, n in ((w_gate, "w_gate"), (w_up, "w_up"), (w_down, "w_down")):
        _need(t, n, torch.uint8, 3)
    for t, n in ((s_gate, "s_gate"), (s_up, "s_up"), (s_down, "s_down")):
        _need(t, n, torch.float32, 2)
    _need(group_offsets, "group_offsets", torch.int32, 1)
    if x_rows is not None:
        _need(x_rows, "x_rows", torch.int32, 1)
    n_rows = int(x_rows.numel()) if x_rows is not None else x.shape[0]
    d = x.shape[1]
    I = w_gate.shape[1]
    G = E + n_shared
    if w_gate.shape != (G, I, d) or w_up.shape != w_gate.shape or w_down.shape != (G, d, I):
        raise ValueError("expert weight codes must be [E+S][I][d] (gate, up) and [E+S][d][I] (down)")
    if s_gate.shape != (G, I) or s_up.shape != (G, I) or s_down.shape != (G, d):
        raise ValueError("row scales must be [E+S][I] (gate, up) and [E+S][d] (down)")
    if group_offsets.numel() != nseg * E + n_shared + 1:
        raise ValueError("group_offsets must have nseg*E + n_shared + 1 entries")
    dev = x.device
    if h_sorted is None:
        h_sorted = torch.empty((n_rows, d), dtype=torch.bfloat16, device=dev)
    _need(h_sorted, "h_sorted", torch.bfloat16, 2)
    if h_sorted.shape != (n_rows, d):
        raise ValueError(f"h_sorted must be [{n_rows}][{d}]")
    if workspace is None:
        workspace = torch.empty(max(ffn_fp8w_workspace_bytes(n_rows, I, E, n_shared, nseg, d, packed), 256),
                                dtype=torch.uint8, device=dev)
    lib = _lib.load()
    nbytes = ctypes.c_size_t(workspace.numel())
    name = "moe_grouped_ffn_fp8w_packed" if packed else "moe_grouped_ffn_fp8w"
    check(name, getattr(lib, name)(
        _ptr(x), _ptr(x_rows), x.shape[0] if x_rows is not None else 0, _ptr(group_offsets), n_rows, E, n_shared,
        nseg, d, I, _ptr(w_gate), _ptr(s_gate), _ptr(w_up), _ptr(s_up), _ptr(w_down), _ptr(s_down), _ptr(h_sorted),
        _ptr(workspace), ctypes.byref(nbytes), _stream(dev)))
    return h_sorted


def quantize_rows_i8(x: torch.Tensor, q: Optional[torch.Tensor] = None, s: Optional[torch.Tensor] = None):
    """int8 codes [..][d] and fp32 scales [..] of the rows of x [..][d] (bf16 or
    fp32): scale = max|row| * fl(1/127), codes to the nearest, halves to even
    (moe_quantize_rows_i8).  Serves token rows and, once, weights."""
    _need(x, "x")
    if x.dim() < 1:
        raise ValueError("x must have at least one dim")
    index = x.get_device()
    *rows, d = shape = x.shape
    _int32_rows(x, d)
    if q is None:
        q = _new(*rows, d, torch.int8, index) if len(rows) == 1 else torch.empty(shape, dtype=torch.int8, device=index)
    elif not _ok(q, index, torch.int8, shape):
        _out(q, "q", torch.int8, shape)
        _same_device(x, q=q)
    if s is None:
        s = torch.empty_strided(rows, (1,), dtype=torch.float32, device=index) if len(rows) == 1 else \
            torch.empty(rows, dtype=torch.float32, device=index)
    elif not _ok(s, index, torch.float32, shape[:-1]):
        _out(s, "s", torch.float32, shape[:-1])
        _same_device(x, s=s)
    _call("moe_quantize_rows_i8", index, _lib.load().moe_quantize_rows_i8, x.data_ptr(), _dtype_code(x), s.numel(),
          d, q.data_ptr(), s.data_ptr())
    return q, s


def pack_i8_codes(q: torch.Tensor) -> torch.Tensor:
    """int8 matrices [..][R][K] in the layout the int8 products read (blocks of
    16 rows x 64 codes, the layout of pack_fp8_codes); same shape."""
    if q.dtype != torch.int8:
        raise TypeError(f"q must be {torch.int8}, got {q.dtype}")
    return pack_fp8_codes(q)


def _i8_batch(x, x_rows, group_offsets, E, n_shared, nseg):
    """Checks of a grouped int8 call's row list and offsets; its sorted rows."""
    index, entries = x.get_device(), nseg * E + n_shared + 1
    if not _ok(group_offsets, index, torch.int32, (entries,)):
        _need(group_offsets, "group_offsets", torch.int32, 1)
        if group_offsets.numel() != entries:
            raise ValueError("group_offsets must have nseg*E + n_shared + 1 entries")
        _same_device(x, group_offsets=group_offsets)
    if x_rows is None:
        return x.shape[0]
    if not _ok(x_rows, index, torch.int32, (x_rows.numel(),)):
        _need(x_rows, "x_rows", torch.int32, 1)
        _same_device(x, x_rows=x_rows)
    return x_rows.numel()


def grouped_linear_i8(xq: torch.Tensor, x_scale: torch.Tensor, group_offsets: torch.Tensor, E: int, n_shared: int,
                      nseg: int, w: torch.Tensor, w_scale: torch.Tensor, y: Optional[torch.Tensor] = None,
                      x_rows: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """y[n] = x_scale * w_scale * (xq . w[expert of row n]) with int8 rows
    [n_x][K] and packed int8 matrices [E+S][O][K] (pack_i8_codes); bf16 or fp32
    out (y's dtype, or `out_dtype`).  E = 1 with offsets [0, N] is a plain
    linear map (moe_grouped_linear_i8)."""
    _need(xq, "xq", torch.int8, 2)
    if w.dim() != 3:
        _need(w, "w", torch.int8, 3)
    n_x, K = xq.shape
    G, O = E + n_shared, w.size(1)
    index = xq.get_device()
    N = _i8_batch(xq, x_rows, group_offsets, E, n_shared, nseg)
    if not (_ok(x_scale, index, torch.float32, (n_x,)) and _ok(w, index, torch.int8, (G, O, K)) and
            _ok(w_scale, index, torch.float32, (G, O))):
        _out(x_scale, "x_scale", torch.float32, (n_x,))
        _out(w, "w", torch.int8, (G, O, K))
        _out(w_scale, "w_scale", torch.float32, (G, O))
        _same_device(xq, x_scale=x_scale, w=w, w_scale=w_scale)
    if y is None:
        y = _new(N, O, out_dtype, index)
    elif not _ok(y, index, y.dtype, (N, O)):
        _out(y, "y", y.dtype, (N, O))
        _same_device(xq, y=y)
    _call("moe_grouped_linear_i8", index, _lib.load().moe_grouped_linear_i8, xq.data_ptr(), x_scale.data_ptr(),
          _ptr(x_rows), n_x, group_offsets.data_ptr(), N, E, n_shared, nseg, K, O, w.data_ptr(), w_scale.data_ptr(),
          _dtype_code(y), y.data_ptr())
    return y


def ffn_i8_workspace_bytes(n_rows, n_x, d, I, E=1, n_shared=0, nseg=1) -> int:
    """Workspace of grouped_ffn_i8: the int8 token rows (n_x of them; n_rows
    without a row list), the int8 SwiGLU product, and their scales."""
    lib = _lib.load()
    n = ctypes.c_size_t(0)
    check("moe_grouped_ffn_i8", lib.moe_grouped_ffn_i8(None, None, n_x, None, n_rows, E, n_shared, nseg, d, I, None,
                                                       None, None, None, None, None, None, None, ctypes.byref(n),
                                                       None))
    return int(n.value)


def _need_i8_weights(like: torch.Tensor, G: int, d: int, I: int, weights) -> None:
    """The six tensors (codes, scales of gate, up, down) of an int8 FFN over G experts."""
    index = like.get_device()
    shapes = (("w_gate", torch.int8, (G, I, d)), ("s_gate", torch.float32, (G, I)),
              ("w_up", torch.int8, (G, I, d)), ("s_up", torch.float32, (G, I)),
              ("w_down", torch.int8, (G, d, I)), ("s_down", torch.float32, (G, d)))
    if len(weights) != len(shapes):
        raise ValueError("int8 weights are codes and scales of gate, up and down")
    for t, (name, dtype, shape) in zip(weights, shapes):
        if not _ok(t, index, dtype, shape):
            _out(t, name, dtype, shape)
            _same_device(like, **{name: t})


def grouped_ffn_i8(x: torch.Tensor, group_offsets: torch.Tensor, E: int, n_shared: int, nseg: int,
                   w_gate: torch.Tensor, s_gate: torch.Tensor, w_up: torch.Tensor, s_up: torch.Tensor,
                   w_down: torch.Tensor, s_down: torch.Tensor, h_sorted: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, x_rows: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The expert FFN with packed int8 weights (pack_i8_codes), fp32 channel
    scales and int8 activations; bf16 token rows, read directly or through
    `x_rows`, bf16 out (moe_grouped_ffn_i8)."""
    _need(x, "x", torch.bfloat16, 2)
    _need(w_gate, "w_gate", torch.int8, 3)
    n_x, d = x.shape
    I, G = w_gate.shape[1], E + n_shared
    index = x.get_device()
    N = _i8_batch(x, x_rows, group_offsets, E, n_shared, nseg)
    i8, f32, ins, outs = torch.int8, torch.float32, (G, I), (G, d)
    if not (_ok(w_gate, index, i8, (G, I, d)) and _ok(w_up, index, i8, (G, I, d)) and _ok(w_down, index, i8, (G, d, I)) and
            _ok(s_gate, index, f32, ins) and _ok(s_up, index, f32, ins) and _ok(s_down, index, f32, outs)):
        _need_i8_weights(x, G, d, I, (w_gate, s_gate, w_up, s_up, w_down, s_down))
    if h_sorted is None:
        h_sorted = _new(N, d, torch.bfloat16, index)
    elif not _ok(h_sorted, index, torch.bfloat16, (N, d)):
        _out(h_sorted, "h_sorted", torch.bfloat16, (N, d))
        _same_device(x, h_sorted=h_sorted)
    if workspace is None:
        workspace = torch.empty(max(ffn_i8_workspace_bytes(N, n_x, d, I, E, n_shared, nseg), 256), dtype=torch.uint8,
                                device=index)
    elif not _ok(workspace, index, torch.uint8, (workspace.numel(),)):
        _out(workspace, "workspace", torch.uint8, (workspace.numel(),))
        _same_device(x, workspace=workspace)
    nbytes = ctypes.c_size_t(workspace.numel())
    _call("moe_grouped_ffn_i8", index, _lib.load().moe_grouped_ffn_i8, x.data_ptr(), _ptr(x_rows), n_x,
          group_offsets.data_ptr(), N, E, n_shared, nseg, d, I, w_gate.data_ptr(), s_gate.data_ptr(), w_up.data_ptr(),
          s_up.data_ptr(), w_down.data_ptr(), s_down.data_ptr(), h_sorted.data_ptr(), workspace.data_ptr(),
          ctypes.byref(nbytes))
    return h_sorted


FP8_BLOCK = 128       # columns of a row, and rows and columns of a matrix, that share a scale (MOE_FP8_BLOCK)


def _blocks(n: int) -> int:
    return -(-n // FP8_BLOCK)


def _code_out(q, s, shape, fp8, like, index):
    """Codes of `shape` and scales of a quantising call: the caller's, checked, or new ones."""
    dtype = torch.float8_e4m3fn if fp8 else torch.int8
    scales = shape[:-1] + (_blocks(shape[-1]),) if fp8 else shape[:-1]
    if q is None:
        q = torch.empty(shape, dtype=dtype, device=index)
    elif not (q.dtype is dtype and q.shape == shape and q.get_device() == index and q.is_contiguous()):
        _out(q, "q", dtype, shape)
        _same_device(like, q=q)
    if s is None:
        s = torch.empty(scales, dtype=torch.float32, device=index)
    elif not (s.dtype is torch.float32 and s.shape == scales and s.get_device() == index and s.is_contiguous()):
        _out(s, "s", torch.float32, scales)
        _same_device(like, s=s)
    return q, s


def _rows_of(x: torch.Tensor):
    """GPU, shape and columns of rows x [..][d] of a supported type; the checks of _need."""
    index, shape = x.get_device(), x.shape
    if index < 0 or not shape or not x.is_contiguous():
        _need(x, "x")
        raise ValueError("x must have at least one dim")
    _int32_rows(x, shape[-1])
    return index, shape, shape[-1]


_TYPES = {torch.float32: MOE_F32, torch.bfloat16: MOE_BF16}


def rmsnorm(x: torch.Tensor, weight: torch.Tensor, eps: float = 1e-6, residual: Optional[torch.Tensor] = None,
            residual_out: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None, codes: Optional[str] = None,
            q: Optional[torch.Tensor] = None, s: Optional[torch.Tensor] = None, want_y: bool = True):
    """Root-mean-square norm of the rows of x [..][d] times `weight` [d], the residual added first
    (moe_rmsnorm).  Returns (y, q, s), None where not asked for.

    residual: [..][d] bf16 or fp32; the sum goes to `residual_out` (`residual` itself, if not given) and the
    norm is taken of it as stored there.  y has its own type or, if not given, x's; want_y=False leaves it
    out.  codes: None, "i8" (int8 codes and a scale per row, for grouped_linear_i8) or "fp8" (E4M3 codes and
    a scale for each 128 columns, for grouped_linear_fp8 and grouped_ffn_fp8)."""
    index, shape, d = _rows_of(x)
    code = _lib.CODES.get(codes)
    if code is None:
        raise ValueError('codes must be None, "i8" or "fp8"')
    # a small call's time is its host side: each tensor's checks in one expression, the messages where it fails
    xt, wt, rt, yt, rp, op, yp, qp, sp = _TYPES.get(x.dtype), _TYPES.get(weight.dtype), 0, 0, None, None, None, None, None
    if xt is None or wt is None:
        _dtype_code(x)
        _dtype_code(weight)
    if not (weight.shape == (d,) and weight.get_device() == index and weight.is_contiguous()):
        _out(weight, "weight", weight.dtype, (d,))
        _same_device(x, weight=weight)
    if residual is not None:
        if residual_out is None:
            residual_out = residual
        rt = _TYPES.get(residual.dtype)
        if rt is None:
            _dtype_code(residual)
        if not (residual.shape == shape and residual.get_device() == index and residual.is_contiguous() and
                (residual_out is residual or (residual_out.dtype is residual.dtype and residual_out.shape == shape and
                                              residual_out.get_device() == index and residual_out.is_contiguous()))):
            for name, t in (("residual", residual), ("residual_out", residual_out)):
                _out(t, name, residual.dtype, shape)
                _same_device(x, **{name: t})
        rp, op = residual.data_ptr(), residual_out.data_ptr()
    elif residual_out is not None:
        raise ValueError("residual_out goes with residual")
    if want_y:
        if y is None:
            y = torch.empty(shape, dtype=x.dtype, device=index)
        yt = _TYPES.get(y.dtype)
        if yt is None:
            _dtype_code(y)
        if not (y.shape == shape and y.get_device() == index and y.is_contiguous()):
            _out(y, "y", y.dtype, shape)
            _same_device(x, y=y)
        yp = y.data_ptr()
    elif codes is None or y is not None:
        raise ValueError("want_y=False goes with codes and without y")
    if code:
        q, s = _code_out(q, s, shape, code == 2, x, index)
        qp, sp = q.data_ptr(), s.data_ptr()
    elif q is not None or s is not None:
        raise ValueError("q and s go with codes")
    _call("moe_rmsnorm", index, _lib.load().moe_rmsnorm, x.data_ptr(), xt, rp, rt, weight.data_ptr(), wt,
          x.numel() // d if d else 0, d, eps, op, yp, yt, code, qp, sp)
    return y, q, s


def quantize_blocks_fp8(x: torch.Tensor, q: Optional[torch.Tensor] = None, s: Optional[torch.Tensor] = None):
    """E4M3 codes [..][d] and fp32 scales [..][ceil(d / 128)] of the rows of x [..][d] (bf16 or fp32), a scale
    for each 128 columns: max|block| * fl(1/448), codes to the nearest (moe_quantize_blocks_fp8)."""
    index, shape, d = _rows_of(x)
    xt = _TYPES.get(x.dtype)
    if xt is None:
        _dtype_code(x)
    q, s = _code_out(q, s, shape, True, x, index)
    _call("moe_quantize_blocks_fp8", index, _lib.load().moe_quantize_blocks_fp8, x.data_ptr(), xt,
          x.numel() // d if d else 0, d, q.data_ptr(), s.data_ptr())
    return q, s


def quantize_fp8_blocks(w: torch.Tensor):
    """E4M3 quantisation of [..][R][K] weights with a scale for each 128 x 128 block (the last ones may be
    smaller): scale = max|block| * fl(1/448) (1 where that is below 2^-100), codes = w / scale to the nearest; scale NaN
    and codes 0 for a block that is not all finite.
    Input preparation for the FP8 products, like quantize_fp8_rows; returns (codes float8_e4m3fn [..][R][K],
    scales fp32 [..][ceil(R / 128)][ceil(K / 128)])."""
    *lead, R, K = w.shape
    rb, kb = _blocks(R), _blocks(K)
    wf = w.float()
    p = torch.nn.functional.pad(wf, (0, kb * FP8_BLOCK - K, 0, rb * FP8_BLOCK - R))
    s = p.reshape(*lead, rb, FP8_BLOCK, kb, FP8_BLOCK).abs().amax(dim=(-3, -1)) * (1.0 / 448.0)
    s = torch.where(s < 2.0 ** -100, torch.ones_like(s), s)
    s = s.masked_fill(~torch.isfinite(s), float("nan"))
    wide = s.repeat_interleave(FP8_BLOCK, -2).repeat_interleave(FP8_BLOCK, -1)[..., :R, :K]
    codes = (wf / wide).masked_fill_(torch.isnan(wide), 0.0)
    return codes.to(torch.float8_e4m3fn).contiguous(), s.contiguous()


def _need_fp8_rows(xq: torch.Tensor, x_scale: torch.Tensor, index: int) -> None:
    scales = (xq.size(0), _blocks(xq.size(1)))
    if not _ok(x_scale, index, torch.float32, scales):
        _out(x_scale, "x_scale", torch.float32, scales)
        _same_device(xq, x_scale=x_scale)


def grouped_linear_fp8(xq: torch.Tensor, x_scale: torch.Tensor, group_offsets: torch.Tensor, E: int, n_shared: int,
                       nseg: int, w: torch.Tensor, w_scale: torch.Tensor, y: Optional[torch.Tensor] = None,
                       x_rows: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16) -> torch.Tensor:
    """y[n] = xq . w[expert of row n] over blocks of 128 columns, each times its row's and its matrix's scale:
    E4M3 rows [n_x][K] with x_scale [n_x][ceil(K/128)], packed E4M3 matrices [E+S][O][K] (quantize_fp8_blocks,
    pack_fp8_codes) with w_scale [E+S][ceil(O/128)][ceil(K/128)]; bf16 or fp32 out (y's dtype, or `out_dtype`).
    E = 1 with offsets [0, N] is a plain linear map (moe_grouped_linear_fp8)."""
    f8, f32 = torch.float8_e4m3fn, torch.float32
    if xq.dtype is not f8 or xq.dim() != 2 or w.dim() != 3 or not xq.is_contiguous():
        _need(xq, "xq", f8, 2)
        _need(w, "w", f8, 3)
    (n_x, K), G, O, index = xq.shape, E + n_shared, w.size(1), xq.get_device()
    if index < 0:
        _need(xq, "xq")
    N = _i8_batch(xq, x_rows, group_offsets, E, n_shared, nseg)
    kb, ob = (K + 127) // FP8_BLOCK, (O + 127) // FP8_BLOCK
    if not (x_scale.dtype is f32 and x_scale.shape == (n_x, kb) and x_scale.get_device() == index and
            x_scale.is_contiguous() and w.dtype is f8 and w.shape == (G, O, K) and w.get_device() == index and
            w.is_contiguous() and w_scale.dtype is f32 and w_scale.shape == (G, ob, kb) and
            w_scale.get_device() == index and w_scale.is_contiguous()):
        _out(x_scale, "x_scale", f32, (n_x, kb))
        _out(w, "w", f8, (G, O, K))
        _out(w_scale, "w_scale", f32, (G, ob, kb))
        _same_device(xq, x_scale=x_scale, w=w, w_scale=w_scale)
    if y is None:
        y = _new(N, O, out_dtype, index)
    elif not (y.shape == (N, O) and y.get_device() == index and y.is_contiguous()):
        _out(y, "y", y.dtype, (N, O))
        _same_device(xq, y=y)
    _call("moe_grouped_linear_fp8", index, _lib.load().moe_grouped_linear_fp8, xq.data_ptr(), x_scale.data_ptr(),
          None if x_rows is None else x_rows.data_ptr(), n_x, group_offsets.data_ptr(), N, E, n_shared, nseg, K, O,
          w.data_ptr(), w_scale.data_ptr(), _dtype_code(y), y.data_ptr())
    return y


def ffn_fp8_workspace_bytes(n_rows, I, E=1, n_shared=0, nseg=1, d=64) -> int:
    """Workspace of grouped_ffn_fp8: the SwiGLU product's codes and their block scales."""
    lib = _lib.load()
    n = ctypes.c_size_t(0)
    check("moe_grouped_ffn_fp8", lib.moe_grouped_ffn_fp8(None, None, None, 0, None, n_rows, E, n_shared, nseg, d, I, None,
                                                         None, None, None, None, None, None, None, ctypes.byref(n),
                                                         None))
    return int(n.value)


def _need_fp8_weights(like: torch.Tensor, G: int, d: int, I: int, weights) -> None:
    """The six tensors (codes, block scales of gate, up, down) of an FP8 FFN over G experts."""
    if len(weights) != 6:
        raise ValueError("FP8 weights are codes and block scales of gate, up and down")
    index, f8, f32 = like.get_device(), torch.float8_e4m3fn, torch.float32
    ins, outs = (G, _blocks(I), _blocks(d)), (G, _blocks(d), _blocks(I))
    w_gate, s_gate, w_up, s_up, w_down, s_down = weights
    if (_ok(w_gate, index, f8, (G, I, d)) and _ok(w_up, index, f8, (G, I, d)) and _ok(w_down, index, f8, (G, d, I)) and
            _ok(s_gate, index, f32, ins) and _ok(s_up, index, f32, ins) and _ok(s_down, index, f32, outs)):
        return
    for t, name, dtype, shape in ((w_gate, "w_gate", f8, (G, I, d)), (s_gate, "s_gate", f32, ins),
                                  (w_up, "w_up", f8, (G, I, d)), (s_up, "s_up", f32, ins),
                                  (w_down, "w_down", f8, (G, d, I)), (s_down, "s_down", f32, outs)):
        _out(t, name, dtype, shape)
        _same_device(like, **{name: t})


def grouped_ffn_fp8(xq: torch.Tensor, x_scale: torch.Tensor, group_offsets: torch.Tensor, E: int, n_shared: int,
                    nseg: int, w_gate: torch.Tensor, s_gate: torch.Tensor, w_up: torch.Tensor, s_up: torch.Tensor,
                    w_down: torch.Tensor, s_down: torch.Tensor, h_sorted: Optional[torch.Tensor] = None,
                    workspace: Optional[torch.Tensor] = None, x_rows: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The expert FFN on E4M3 rows [n_x][d] with x_scale [n_x][ceil(d/128)] (rmsnorm(codes="fp8") or
    quantize_blocks_fp8) and packed E4M3 weights with 128 x 128 block scales (quantize_fp8_blocks,
    pack_fp8_codes); rows read directly or through `x_rows`, bf16 out (moe_grouped_ffn_fp8)."""
    _need(xq, "xq", torch.float8_e4m3fn, 2)
    _need(w_gate, "w_gate", torch.float8_e4m3fn, 3)
    n_x, d = xq.shape
    I = w_gate.size(1)
    index = xq.get_device()
    N = _i8_batch(xq, x_rows, group_offsets, E, n_shared, nseg)
    _need_fp8_rows(xq, x_scale, index)
    _need_fp8_weights(xq, E + n_shared, d, I, (w_gate, s_gate, w_up, s_up, w_down, s_down))
    if h_sorted is None:
        h_sorted = _new(N, d, torch.bfloat16, index)
    elif not _ok(h_sorted, index, torch.bfloat16, (N, d)):
        _out(h_sorted, "h_sorted", torch.bfloat16, (N, d))
        _same_device(xq, h_sorted=h_sorted)
    if workspace is None:
        workspace = torch.empty(max(ffn_fp8_workspace_bytes(N, I, E, n_shared, nseg, d), 256), dtype=torch.uint8,
                                device=index)
    elif not _ok(workspace, index, torch.uint8, (workspace.numel(),)):
        _out(workspace, "workspace", torch.uint8, (workspace.numel(),))
        _same_device(xq, workspace=workspace)
    nbytes = ctypes.c_size_t(workspace.numel())
    _call("moe_grouped_ffn_fp8", index, _lib.load().moe_grouped_ffn_fp8, xq.data_ptr(), x_scale.data_ptr(), _ptr(x_rows),
          n_x, group_offsets.data_ptr(), N, E, n_shared, nseg, d, I, w_gate.data_ptr(), s_gate.data_ptr(),
          w_up.data_ptr(), s_up.data_ptr(), w_down.data_ptr(), s_down.data_ptr(), h_sorted.data_ptr(),
          workspace.data_ptr(), ctypes.byref(nbytes))
    return h_sorted


def combine(h_sorted: torch.Tensor, flat_to_sorted: torch.Tensor, topk_w: torch.Tensor, n_shared: int = 0,
            y: Optional[torch.Tensor] = None) -> torch.Tensor:
    _need(h_sorted, "h_sorted", None, 2)
    _need(flat_to_sorted, "flat_to_sorted", torch.int32, 1)
    _need(topk_w, "topk_w", torch.float32, 2)
    T, k = topk_w.shape
    d = h_sorted.shape[1]
    if flat_to_sorted.numel() != T * (k + n_shared) or h_sorted.shape[0] != T * (k + n_shared):
        raise ValueError("h_sorted / flat_to_sorted must have T*(k+n_shared) rows")
    dev = h_sorted.device
    if y is None:
        y = torch.empty((T, d), dtype=h_sorted.dtype, device=dev)
    lib = _lib.load()
    check("moe_combine", lib.moe_combine(_ptr(h_sorted), _ptr(flat_to_sorted), _ptr(topk_w), T, k, n_shared,
                                         d, _dtype_code(h_sorted), _ptr(y), _stream(dev)))
    return y


def stats_workspace_bytes(L, T, k, E, R) -> int:
    lib = _lib.load()
    n = ctypes.c_size_t(0)
    check("moe_stats", lib.moe_stats(None, L, T, k, E, None, R, None, None, None, None, None, None, None,
                                     None, ctypes.byref(n), None))
    return int(n.value)


def stats(topk_ids: torch.Tensor, E: int, req_offsets: Optional[torch.Tensor] = None,
          idf: Optional[torch.Tensor] = None, affinity: bool = True, signature: bool = True,
          out: Optional[Dict[str, torch.Tensor]] = None,
          workspace: Optional[torch.Tensor] = None) -> Dict[str, torch.Tensor]:
    _need(topk_ids, "topk_ids", torch.int32, 3)
    L, T, k = topk_ids.shape
    dev = topk_ids.device
    R = 0
    if req_offsets is not None:
        _need(req_offsets, "req_offsets", torch.int32, 1)
        R = req_offsets.numel() - 1
    if idf is not None:
        _out(idf, "idf", torch.float32, (L, E))
    o = {} if out is None else out
    o.setdefault("counts", torch.empty((L, E), dtype=torch.int32, device=dev))
    o.setdefault("union_size", torch.empty(L, dtype=torch.int32, device=dev))
    o.setdefault("union_mask", torch.empty((L, E), dtype=torch.uint8, device=dev))
    if affinity:
        o.setdefault("affinity", torch.empty((L, E, E), dtype=torch.int32, device=dev))
    if R > 0:
        o.setdefault("req_counts", torch.empty((R, L, E), dtype=torch.int32, device=dev))
        if signature:
            o.setdefault("signature", torch.empty((R, L, E), dtype=torch.float32, device=dev))
    shapes = {"counts": ((L, E), torch.int32), "union_size": ((L,), torch.int32),
              "union_mask": ((L, E), torch.uint8), "affinity": ((L, E, E), torch.int32),
              "req_counts": ((R, L, E), torch.int32), "signature": ((R, L, E), torch.float32)}
    for key, (shape, dt) in shapes.items():
        if key in o and (R > 0 or key not in ("req_counts", "signature")):
            _out(o[key], key, dt, shape)
    if workspace is None:
        workspace = torch.empty(max(stats_workspace_bytes(L, T, k, E, R), 256), dtype=torch.uint8, device=dev)
    lib = _lib.load()
    nbytes = ctypes.c_size_t(workspace.numel())
    check("moe_stats", lib.moe_stats(
        _ptr(topk_ids), L, T, k, E, _ptr(req_offsets), R, _ptr(idf), _ptr(o["counts"]),
        _ptr(o["union_size"]), _ptr(o["union_mask"]), _ptr(o.get("affinity")), _ptr(o.get("req_counts")),
        _ptr(o.get("signature")), _ptr(workspace), ctypes.byref(nbytes), _stream(dev)))
    return o


def prob_signature(logits: torch.Tensor, req_offsets: torch.Tensor,
                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Continuous request signature [R][L][E]: per request, the sum of its
    tokens' full-E softmax probabilities, from fp32 logits [L][T][E]."""
    _need(logits, "logits", torch.float32, 3)
    _need(req_offsets, "req_offsets", torch.int32, 1)
    L, T, E = logits.shape
    R = req_offsets.numel() - 1
    dev = logits.device
    if out is None:
        out = torch.empty((R, L, E), dtype=torch.float32, device=dev)
    _out(out, "out", torch.float32, (R, L, E))
    lib = _lib.load()
    check("moe_prob_signature", lib.moe_prob_signature(_ptr(logits), L, T, E, _ptr(req_offsets), R, _ptr(out),
                                                       _stream(dev)))
    return out


class MoeLayer:
    """One MoE layer's expert path with every buffer allocated up front.

    `forward()` enqueues gate -> permute -> grouped FFN -> combine and, when
    `stats_ids` is given, the statistics over that [L][T][k] id stack (the
    routing layer's own ids are written into stats_ids[0] by the gate).  With
    `w_router` ([E][d], the input dtype) the router projection runs first and
    the gate reads its logits; `forward` then ignores the logits argument.
    With `norm` ((weight [d], eps)) the layer starts with the RMS norm of its
    input, to which `forward` and `bound_calls` then add a residual, if given one,
    in place; the router and the experts read the normalised rows.
    Nothing is allocated per call.
    """

    def __init__(self, E, k, d, I, T, dtype, w_gate, w_up, w_down, n_shared=0, n_priority=0,
                 renormalize=True, stats_layers=0, req_offsets=None, device="cuda", topk_ids=None,
                 fused_gather=True, w_router=None, fp8_weights=None, packed_weights=False, fused_combine=False,
                 int8_weights=None, routing=None, fp8_block_weights=None, norm=None):
        dev = torch.device(device)
        # fp8_weights = (codes_gate, scales_gate, codes_up, scales_up, codes_down, scales_down):
        # the FFN runs moe_grouped_ffn_fp8w on them instead of w_gate / w_up / w_down
        self.fp8_weights = fp8_weights
        # packed_weights: w_gate / w_up / w_down come from pack_weights and the FFN
        # runs moe_grouped_ffn_packed (bf16, decode-sized batches); with
        # fp8_weights, the codes come from pack_fp8_codes (moe_grouped_ffn_fp8w_packed)
        self.packed = bool(packed_weights)
        # fused_combine: the FFN and the combine run as one moe_grouped_ffn_combine
        # call (bf16 decode-sized batches; h_sorted is then not written)
        self.fused_combine = bool(fused_combine)
        if self.fused_combine and (fp8_weights is not None or dtype != torch.bfloat16):
            raise ValueError("fused_combine serves bf16 expert weights only")
        # int8_weights = (codes_gate, scales_gate, codes_up, scales_up, codes_down, scales_down), codes from
        # pack_i8_codes: the FFN runs moe_grouped_ffn_i8 on them instead of w_gate / w_up / w_down
        self.int8_weights = int8_weights
        if int8_weights is not None and (fp8_weights is not None or self.fused_combine or dtype != torch.bfloat16):
            raise ValueError("int8_weights serve bf16 tokens, without fp8_weights or fused_combine")
        # fp8_block_weights = (codes_gate, scales_gate, codes_up, scales_up, codes_down, scales_down) of
        # quantize_fp8_blocks, codes from pack_fp8_codes: the FFN runs moe_grouped_ffn_fp8 on E4M3 codes of the
        # tokens, which the norm makes, or moe_quantize_blocks_fp8 without one
        self.fp8_block_weights = fp8_block_weights
        if fp8_block_weights is not None and (fp8_weights is not None or int8_weights is not None or self.fused_combine or
                                              not fused_gather or dtype != torch.bfloat16):
            raise ValueError("fp8_block_weights serve bf16 tokens read through the row list (fused_gather), without "
                             "fp8_weights, int8_weights or fused_combine")
        self.norm = None if norm is None else tuple(norm)
        # routing: None (moe_gate), or a dict of route()'s score, bias, n_groups, top_groups, group_rank, scale:
        # the layer's gate is moe_route
        self.routing = None if routing is None else dict(routing)
        unknown = set(self.routing or ()) - {"score", "bias", "n_groups", "top_groups", "group_rank", "scale"}
        if unknown:
            raise ValueError(f"unknown routing options {sorted(unknown)}")
        if self.routing and self.routing.get("score", "softmax") not in _lib.SCORES:
            raise ValueError(f"score must be one of {sorted(_lib.SCORES)}")
        if self.routing and self.routing.get("group_rank", "max") not in _lib.GROUP_RANKS:
            raise ValueError(f"group_rank must be one of {sorted(_lib.GROUP_RANKS)}")
        if self.routing and self.routing.get("bias") is not None:
            _out(self.routing["bias"], "bias", torch.float32, (E,))
        if int8_weights is not None:
            _need_i8_weights(int8_weights[0], E + n_shared, d, I, int8_weights)
        if fp8_block_weights is not None:
            _need_fp8_weights(fp8_block_weights[0], E + n_shared, d, I, fp8_block_weights)
        self.xn = self.xq = self.xs = None
        if self.norm is not None:
            self._need_norm(d)
            if fp8_block_weights is None or w_router is not None:
                self.xn = torch.empty((T, d), dtype=dtype, device=dev)
        if fp8_block_weights is not None:
            self.xq = torch.empty((T, d), dtype=torch.float8_e4m3fn, device=dev)
            self.xs = torch.empty((T, _blocks(d)), dtype=torch.float32, device=dev)
        self.w_router = w_router
        self.logits = torch.empty((T, E), dtype=torch.float32, device=dev) if w_router is not None else None
        self.E, self.k, self.d, self.I, self.T = E, k, d, I, T
        self.S, self.P = n_shared, n_priority
        self.nseg = 2 if n_priority > 0 else 1
        self.renormalize = renormalize
        self.w_gate, self.w_up, self.w_down = w_gate, w_up, w_down
        N = T * (k + n_shared)
        G = self.nseg * E + n_shared
        self.N, self.G = N, G
        # the gate may write straight into a caller buffer (e.g. one layer of a
        # statistics id stack)
        self.topk_ids = torch.empty((T, k), dtype=torch.int32, device=dev) if topk_ids is None else topk_ids
        self.topk_w = torch.empty((T, k), dtype=torch.float32, device=dev)
        # fused_gather: the permutation writes only the row list and the FFN
        # reads the token rows through it; otherwise x_sorted is materialised
        self.fused_gather = fused_gather
        self.perm = {"group_offsets": torch.empty(G + 1, dtype=torch.int32, device=dev),
                     "sorted_to_flat": torch.empty(N, dtype=torch.int32, device=dev),
                     "flat_to_sorted": torch.empty(N, dtype=torch.int32, device=dev),
                     "sorted_token": torch.empty(N, dtype=torch.int32, device=dev)}
        if not fused_gather:
            self.perm["x_sorted"] = torch.empty((N, d), dtype=dtype, device=dev)
        self.perm_ws = torch.empty(max(permute_workspace_bytes(T, E, k, n_shared, n_priority), 256),
                                   dtype=torch.uint8, device=dev)
        self.h_sorted = torch.empty((N, d), dtype=dtype, device=dev)
        if self.fused_combine:
            ws_bytes = ffn_combine_workspace_bytes(N, E, n_shared, self.nseg, d, I, T, k, self.packed)
        elif int8_weights is not None:
            ws_bytes = ffn_i8_workspace_bytes(N, T if fused_gather else 0, d, I, E, n_shared, self.nseg)
        elif fp8_block_weights is not None:
            ws_bytes = ffn_fp8_workspace_bytes(N, I, E, n_shared, self.nseg, d)
        elif fp8_weights is not None:
            ws_bytes = ffn_fp8w_workspace_bytes(N, I, E, n_shared, self.nseg, d, self.packed)
        else:
            ws_bytes = ffn_workspace_bytes(N, E, n_shared, self.nseg, d, I, dtype)
        self.ffn_ws = torch.empty(max(ws_bytes, 256), dtype=torch.uint8, device=dev)
        self.y = torch.empty((T, d), dtype=dtype, device=dev)
        self.stats_out = None
        self.req_offsets = req_offsets
        if stats_layers:
            R = 0 if req_offsets is None else req_offsets.numel() - 1
            self.stats_out = {}
            self.stats_ws = torch.empty(max(stats_workspace_bytes(stats_layers, T, k, E, R), 256),
                                        dtype=torch.uint8, device=dev)

    def _need_norm(self, d):
        weight, eps = self.norm
        if weight.dtype not in _TYPES or not eps > 0:
            raise ValueError("norm is a bf16 or fp32 weight and a positive eps")
        _out(weight, "the norm's weight", weight.dtype, (d,))

    def prepare(self, x, residual=None):
        """The rows that the router and the experts read: the norm's, if there is one, and the experts' FP8 codes."""
        if self.norm is not None:
            rmsnorm(x, self.norm[0], self.norm[1], residual=residual, y=self.xn, want_y=self.xn is not None,
                    codes=None if self.xq is None else "fp8", q=self.xq, s=self.xs)
            return x if self.xn is None else self.xn
        if residual is not None:
            raise ValueError("a residual goes with a norm")
        if self.xq is not None:
            _out(x, "x", torch.bfloat16, (self.T, self.d))
            quantize_blocks_fp8(x, self.xq, self.xs)
        return x

    def route(self, x):
        return router(x, self.w_router, self.logits)

    def gate(self, logits):
        if self.routing is not None:
            return route(logits, self.k, renormalize=self.renormalize, topk_ids=self.topk_ids, topk_w=self.topk_w,
                         **self.routing)
        return gate(logits, self.k, self.renormalize, self.topk_ids, self.topk_w)

    def permute(self, x):
        return permute(self.topk_ids, self.E, self.S, self.P, None if self.fused_gather else x, out=self.perm,
                       workspace=self.perm_ws)

    def ffn_combine(self, x):
        src = x if self.fused_gather else self.perm["x_sorted"]
        return grouped_ffn_combine(src, self.perm["group_offsets"], self.E, self.S, self.nseg, self.w_gate,
                                   self.w_up, self.w_down, self.perm["sorted_to_flat"], self.topk_w, self.y,
                                   self.ffn_ws, x_rows=self.perm["sorted_token"] if self.fused_gather else None,
                                   packed=self.packed)

    def ffn(self, x):
        if self.fp8_block_weights is not None:
            return grouped_ffn_fp8(self.xq, self.xs, self.perm["group_offsets"], self.E, self.S, self.nseg,
                                   *self.fp8_block_weights, h_sorted=self.h_sorted, workspace=self.ffn_ws,
                                   x_rows=self.perm["sorted_token"])
        if self.int8_weights is not None:
            src = x if self.fused_gather else self.perm["x_sorted"]
            return grouped_ffn_i8(src, self.perm["group_offsets"], self.E, self.S, self.nseg, *self.int8_weights,
                                  h_sorted=self.h_sorted, workspace=self.ffn_ws,
                                  x_rows=self.perm["sorted_token"] if self.fused_gather else None)
        if self.fp8_weights is not None:
            src = x if self.fused_gather else self.perm["x_sorted"]
            return grouped_ffn_fp8w(src, self.perm["group_offsets"], self.E, self.S, self.nseg, *self.fp8_weights,
                                    h_sorted=self.h_sorted, workspace=self.ffn_ws,
                                    x_rows=self.perm["sorted_token"] if self.fused_gather else None,
                                    packed=self.packed)
        if self.packed:
            src = x if self.fused_gather else self.perm["x_sorted"]
            return grouped_ffn_packed(src, self.perm["group_offsets"], self.E, self.S, self.nseg, self.w_gate,
                                      self.w_up, self.w_down, self.h_sorted, self.ffn_ws,
                                      x_rows=self.perm["sorted_token"] if self.fused_gather else None)
        if self.fused_gather:
            return grouped_ffn(x, self.perm["group_offsets"], self.E, self.S, self.nseg, self.w_gate, self.w_up,
                               self.w_down, self.h_sorted, self.ffn_ws, x_rows=self.perm["sorted_token"])
        return grouped_ffn(self.perm["x_sorted"], self.perm["group_offsets"], self.E, self.S, self.nseg,
                           self.w_gate, self.w_up, self.w_down, self.h_sorted, self.ffn_ws)

    def combine(self):
        return combine(self.h_sorted, self.perm["flat_to_sorted"], self.topk_w, self.S, self.y)

    def stats(self, stats_ids):
        return stats(stats_ids, self.E, self.req_offsets, out=self.stats_out, workspace=self.stats_ws)

    def bound_calls(self, logits, x, stats_ids=None, stream=None, stats_stream=None, residual=None):
        """Pre-marshalled raw C calls for one forward over fixed buffers.

        Returns a list of (name, fn, args) whose arguments are plain integers,
        so a timing loop pays only the ctypes call per step.  Each entry is one
        of the libmoe calls, in path order (the norm first when the layer has one, then
        the router when it has router weights; the gate then reads the router's
        logits).  `stats_stream` (a raw stream
        handle) puts the statistics call on its own stream; the caller orders it
        after the gate.
        """
        lib = _lib.load()
        dev = logits.device
        st = _stream(dev) if stream is None else stream
        k, T, E = self.k, self.T, self.E
        dt = _dtype_code(x)
        fused = self.fused_gather
        n_perm = ctypes.c_size_t(self.perm_ws.numel())
        n_ffn = ctypes.c_size_t(self.ffn_ws.numel())
        calls = []
        prepare = self._prepare_call(lib, x, residual, st)
        if self.norm is not None:
            calls.append(prepare)
            x = x if self.xn is None else self.xn
            dt = _dtype_code(self.h_sorted)
        if self.w_router is not None:
            _out(self.w_router, "w_router", x.dtype, (E, self.d))
            logits = self.logits
            calls.append(("moe_router", lib.moe_router, (x.data_ptr(), self.w_router.data_ptr(), T, self.d, E, dt,
                                                         logits.data_ptr(), st)))
        calls += [
            self._gate_call(lib, logits, st),
            ("moe_permute", lib.moe_permute, (self.topk_ids.data_ptr(), T, E, k, self.S, self.P,
                                              None if fused else x.data_ptr(), dt,
                                              self.d, self.perm["group_offsets"].data_ptr(),
                                              self.perm["sorted_to_flat"].data_ptr(),
                                              self.perm["flat_to_sorted"].data_ptr(),
                                              self.perm["sorted_token"].data_ptr(),
                                              None if fused else self.perm["x_sorted"].data_ptr(),
                                              self.perm_ws.data_ptr(), ctypes.byref(n_perm), st)),
        ]
        if self.norm is None and prepare is not None:
            calls.append(prepare)
        if self.fused_combine:
            src = x.data_ptr() if fused else self.perm["x_sorted"].data_ptr()
            calls.append(("moe_grouped_ffn_combine", lib.moe_grouped_ffn_combine, (
                src, self.perm["sorted_token"].data_ptr() if fused else None, T, self.perm["group_offsets"].data_ptr(),
                self.N, E, self.S, self.nseg, self.d, self.I, self.w_gate.data_ptr(), self.w_up.data_ptr(),
                self.w_down.data_ptr(), int(self.packed), self.perm["sorted_to_flat"].data_ptr(),
                self.topk_w.data_ptr(), T, k, self.y.data_ptr(), self.ffn_ws.data_ptr(), ctypes.byref(n_ffn), st)))
        else:
            calls += [
                self._ffn_call(lib, x, fused, dt, n_ffn, st),
                ("moe_combine", lib.moe_combine, (self.h_sorted.data_ptr(), self.perm["flat_to_sorted"].data_ptr(),
                                                  self.topk_w.data_ptr(), T, k, self.S, self.d, dt,
                                                  self.y.data_ptr(), st)),
            ]
        if stats_ids is not None and self.stats_out is not None:
            o = self.stats(stats_ids)          # allocates the outputs once
            L = stats_ids.shape[0]
            R = 0 if self.req_offsets is None else self.req_offsets.numel() - 1
            n_st = ctypes.c_size_t(self.stats_ws.numel())

            def p(key):
                return o[key].data_ptr() if key in o else None
            calls.append(("moe_stats", lib.moe_stats, (
                stats_ids.data_ptr(), L, T, k, E,
                self.req_offsets.data_ptr() if self.req_offsets is not None else None, R, None,
                p("counts"), p("union_size"), p("union_mask"), p("affinity"), p("req_counts"), p("signature"),
                self.stats_ws.data_ptr(), ctypes.byref(n_st), st if stats_stream is None else stats_stream)))
        self._keep = (n_perm, n_ffn, n_st if stats_ids is not None and self.stats_out is not None else None)
        return calls

    def _prepare_call(self, lib, x, residual, st):
        if self.norm is None and residual is not None:
            raise ValueError("a residual goes with a norm")
        if self.norm is None and self.xq is None:
            return None
        if x.dtype not in _TYPES:
            raise TypeError("x must be bf16 or fp32")
        _out(x, "x", torch.bfloat16 if self.norm is None else x.dtype, (self.T, self.d))
        _same_device(self.h_sorted, x=x, residual=residual)
        q, s = (None, None) if self.xq is None else (self.xq.data_ptr(), self.xs.data_ptr())
        if self.norm is None:
            return ("moe_quantize_blocks_fp8", lib.moe_quantize_blocks_fp8, (
                x.data_ptr(), _TYPES[x.dtype], self.T, self.d, q, s, st))
        self._need_norm(self.d)
        weight, eps = self.norm
        if residual is not None:
            if residual.dtype not in _TYPES:
                raise TypeError("the residual must be bf16 or fp32")
            _out(residual, "residual", residual.dtype, (self.T, self.d))
        _same_device(x, weight=weight)
        return ("moe_rmsnorm", lib.moe_rmsnorm, (
            x.data_ptr(), _TYPES[x.dtype], _ptr(residual), 0 if residual is None else _TYPES[residual.dtype],
            weight.data_ptr(), _TYPES[weight.dtype], self.T, self.d, eps, _ptr(residual), _ptr(self.xn),
            0 if self.xn is None else _TYPES[self.xn.dtype], _lib.CODES["fp8" if q else None], q, s, st))

    def _gate_call(self, lib, logits, st):
        if self.routing is None:
            return ("moe_gate", lib.moe_gate, (logits.data_ptr(), self.T, self.E, self.k, int(bool(self.renormalize)),
                                               self.topk_ids.data_ptr(), self.topk_w.data_ptr(), st))
        o = {"score": "softmax", "bias": None, "n_groups": 1, "top_groups": None, "group_rank": "max", "scale": 1.0,
             **self.routing}
        groups = o["n_groups"]
        _need(logits, "logits", None, 2)
        if tuple(logits.shape) != (self.T, self.E):
            raise ValueError(f"logits must have shape {(self.T, self.E)}, got {tuple(logits.shape)}")
        _same_device(logits, bias=o["bias"], topk_ids=self.topk_ids)
        return ("moe_route", lib.moe_route, (
            logits.data_ptr(), _dtype_code(logits), _ptr(o["bias"]), self.T, self.E, self.k, _lib.SCORES[o["score"]],
            groups, groups if o["top_groups"] is None else o["top_groups"], _lib.GROUP_RANKS[o["group_rank"]],
            int(bool(self.renormalize)), float(o["scale"]), self.topk_ids.data_ptr(), self.topk_w.data_ptr(), st))

    def _ffn_call(self, lib, x, fused, dt, n_ffn, st):
        src = x.data_ptr() if fused else self.perm["x_sorted"].data_ptr()
        rows = self.perm["sorted_token"].data_ptr() if fused else None
        offs = self.perm["group_offsets"].data_ptr()
        if self.fp8_block_weights is not None:
            _need_fp8_weights(self.h_sorted, self.E + self.S, self.d, self.I, self.fp8_block_weights)
            qg, sg, qu, su, qd, sd = (t.data_ptr() for t in self.fp8_block_weights)
            return ("moe_grouped_ffn_fp8", lib.moe_grouped_ffn_fp8, (
                self.xq.data_ptr(), self.xs.data_ptr(), rows, self.T, offs, self.N, self.E, self.S, self.nseg, self.d,
                self.I, qg, sg, qu, su, qd, sd, self.h_sorted.data_ptr(), self.ffn_ws.data_ptr(), ctypes.byref(n_ffn),
                st))
        if self.int8_weights is not None:
            _need_i8_weights(self.h_sorted, self.E + self.S, self.d, self.I, self.int8_weights)
            _out(x, "x", torch.bfloat16, (self.T, self.d))
            _same_device(self.h_sorted, x=x)
            qg, sg, qu, su, qd, sd = (t.data_ptr() for t in self.int8_weights)
            return ("moe_grouped_ffn_i8", lib.moe_grouped_ffn_i8, (
                src, rows, self.T, offs, self.N, self.E, self.S, self.nseg, self.d, self.I, qg, sg, qu, su, qd, sd,
                self.h_sorted.data_ptr(), self.ffn_ws.data_ptr(), ctypes.byref(n_ffn), st))
        if self.fp8_weights is not None:
            qg, sg, qu, su, qd, sd = (t.data_ptr() for t in self.fp8_weights)
            name = "moe_grouped_ffn_fp8w_packed" if self.packed else "moe_grouped_ffn_fp8w"
            return (name, getattr(lib, name), (
                src, rows, self.T, offs, self.N, self.E, self.S, self.nseg, self.d, self.I, qg, sg, qu, su, qd, sd,
                self.h_sorted.data_ptr(), self.ffn_ws.data_ptr(), ctypes.byref(n_ffn), st))
        if self.packed:
            return ("moe_grouped_ffn_packed", lib.moe_grouped_ffn_packed, (
                src, rows, self.T, offs, self.N, self.E, self.S, self.nseg, self.d, self.I, self.w_gate.data_ptr(),
                self.w_up.data_ptr(), self.w_down.data_ptr(), self.h_sorted.data_ptr(), self.ffn_ws.data_ptr(),
                ctypes.byref(n_ffn), st))
        return ("moe_grouped_ffn", lib.moe_grouped_ffn, (
            src, rows, self.T, offs, self.N, self.E, self.S, self.nseg, self.d, self.I, self.w_gate.data_ptr(),
            self.w_up.data_ptr(), self.w_down.data_ptr(), dt, self.h_sorted.data_ptr(), self.ffn_ws.data_ptr(),
            ctypes.byref(n_ffn), st))

    def forward(self, logits, x, stats_ids=None, stats_stream=None, residual=None):
        """Enqueue the layer on the current stream.  With `stats_stream` (a
        torch stream) the statistics run there, concurrently with the permute /
        FFN / combine chain; the current stream waits for them at the end."""
        x = self.prepare(x, residual)
        if self.w_router is not None:
            logits = self.route(x)
        self.gate(logits)
        side = stats_ids is not None and self.stats_out is not None
        if side and stats_stream is not None:
            main = torch.cuda.current_stream(logits.device)
            stats_stream.wait_stream(main)
            with torch.cuda.stream(stats_stream):
                self.stats(stats_ids)
            side = False
        self.permute(x)
        if self.fused_combine:
            self.ffn_combine(x)
        else:
            self.ffn(x)
            self.combine()
        if side:
            self.stats(stats_ids)
        elif stats_ids is not None and self.stats_out is not None:
            torch.cuda.current_stream(logits.device).wait_stream(stats_stream)
        return self.y
