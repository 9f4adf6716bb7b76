"""Thin ctypes binding of ``libmoe_route.so`` (C ABI in ``include/moe_route.h``
and ``include/moe_recv.h``; the test-support library of
``include/moe_harness.h`` has its own binding, ``harness.py``).

Same names as the C entry points; each function only checks that torch
tensors have the dtype, device and contiguity the ABI expects, passes their
device pointers and the stream handle, and raises ``MoeError`` on a non-zero
status.  Every step of the path runs in the HIP kernels; there is no CPU or
PyTorch fallback, and a missing library is an error.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import NamedTuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoe_route.so")

MOE_QUANT_BF16 = 0
MOE_QUANT_INT8 = 1
MOE_QUANT_INT4 = 2
MOE_QUANT_FP8 = 3
MOE_PACK_STREAM = 0x100  # OR into the quant of the pack calls: streaming row stores

EXPORTS = ("moe_route_topk", "moe_dispatch_layout", "moe_dispatch_layout_chunks",
           "moe_route_layout_chunks", "moe_route_layout_chunks_noalloc",
           "moe_dispatch_pack", "moe_combine", "moe_combine_pack", "moe_status_string",
           "moe_row_bytes", "moe_recv_layout", "moe_recv_regroup", "moe_recv_ungroup",
           "moe_balance_loss", "moe_route_grad", "moe_combine_grad", "moe_expert_matmul",
           "moe_expert_matmul_dx", "moe_expert_matmul_dw", "moe_add_norm", "moe_add_norm_grad",
           "moe_quant_rows", "moe_quant_weights", "moe_expert_matmul_fp8",
           "moe_expert_matmul_fp8_dx")

MOE_ACT_NONE, MOE_ACT_RELU, MOE_ACT_SILU, MOE_ACT_GELU, MOE_ACT_SWIGLU = range(5)
MOE_GRAD_FP32, MOE_GRAD_BF16, MOE_GRAD_ACCUMULATE = 0, 1, 0x100
MOE_BLOCK_ROW, MOE_BLOCK_128 = 0, 128  # what a scale of E4M3 codes stands for
MOE_ROUTE_MASKED_GATES = 0x100  # OR into the k of moe_route_grad's entry point

_lib = None


class MoeError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn}: {status_string(status)} (status {status})")
        self.status = status


def load() -> ctypes.CDLL:
    """Load the built library (never builds, never falls back)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built; run __graft_entry__.build() first")
    lib = ctypes.CDLL(LIB_PATH)
    P, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    lib.moe_route_topk.argtypes = [P, i64, i32, i32, P, P, P]
    lib.moe_dispatch_layout.argtypes = [P, i64, i32, i32, i32, i32, P, P, P, P, P, P, P,
                                        ctypes.POINTER(sz), P]
    lib.moe_dispatch_layout_chunks.argtypes = [P, i64, i64, i32, i32, i32, i32, P, P, P, P, P, P,
                                               P, P, ctypes.POINTER(sz), P]
    lib.moe_route_layout_chunks.argtypes = [P, i64, i64, i32, i32, i32, i32, P, P, P, P, P, P,
                                            P, P, P, P, ctypes.POINTER(sz), P]
    lib.moe_route_layout_chunks_noalloc.argtypes = [P, i64, i64, i32, i32, i32, i32, P, P, P, P,
                                                    P, P, P, P, P, P]
    lib.moe_dispatch_pack.argtypes = [P, i64, i32, i32, P, i32, P, P, P]
    lib.moe_combine.argtypes = [P, P, i32, P, P, i64, i32, i32, P, P]
    lib.moe_combine_pack.argtypes = [P, P, P, P, i64, P, P, P, i64, P, P, i32, i32, i32, P]
    lib.moe_recv_layout.argtypes = [P, i32, i32, i64, P, P, P, P, P, P]
    lib.moe_recv_regroup.argtypes = [P, P, i64, i32, i32, P, P, P, P]
    lib.moe_recv_ungroup.argtypes = [P, P, i64, i32, i32, P, P, P, P]
    lib.moe_balance_loss.argtypes = [P, P, P, i64, i64, i32, i32, P, P, P, P, P, P, P]
    lib.moe_route_grad.argtypes = [P, P, P, P, P, P, P, P, i64, i64, i32, i32, P, P]
    lib.moe_combine_grad.argtypes = [P, P, P, i32, P, P, i64, i32, i32, P, P, P]
    lib.moe_expert_matmul.argtypes = [P, P, P, P, i32, P, i32, i64, i32, i32, P, P, P,
                                      ctypes.POINTER(sz), P]
    lib.moe_expert_matmul_dx.argtypes = [P, P, P, i32, P, i32, i64, i32, i32, P, P,
                                         ctypes.POINTER(sz), P]
    lib.moe_expert_matmul_dw.argtypes = [P, P, P, i32, i64, i32, i32, i32, P, P, P,
                                         ctypes.POINTER(sz), P]
    f32 = ctypes.c_float
    lib.moe_add_norm.argtypes = [P, P, P, f32, i64, i32, P, P, i32, P, P, P]
    lib.moe_add_norm_grad.argtypes = [P, P, P, P, f32, i64, i32, P, P, i32, P, ctypes.POINTER(sz),
                                      P]
    lib.moe_quant_rows.argtypes = [P, P, i32, i64, i32, i32, P, P, P]
    lib.moe_quant_weights.argtypes = [P, i32, i32, i32, i32, P, P, P, P, P]
    lib.moe_expert_matmul_fp8.argtypes = [P, P, i32, P, P, P, P, i32, P, i32, i64, i32, i32, P, P,
                                          P, P, P, ctypes.POINTER(sz), P]
    lib.moe_expert_matmul_fp8_dx.argtypes = [P, P, P, P, P, i32, i32, P, i32, i64, i32, i32, P, P,
                                             P, P, ctypes.POINTER(sz), P]
    lib.moe_status_string.argtypes = [i32]
    lib.moe_status_string.restype = ctypes.c_char_p
    lib.moe_row_bytes.argtypes = [i32, i32]
    lib.moe_row_bytes.restype = i64
    for n in EXPORTS:
        if n not in ("moe_status_string", "moe_row_bytes"):
            getattr(lib, n).restype = i32
    _lib = lib
    return lib


def status_string(status: int) -> str:
    return load().moe_status_string(int(status)).decode()


def moe_row_bytes(H: int, quant: int) -> int:
    """Bytes per row of a row buffer (quantised formats: the codes only; the
    fp32 scale of each row lives in a separate scale array)."""
    return int(load().moe_row_bytes(int(H), int(quant)))


def alloc_rows(rows: int, H: int, quant: int, device) -> tuple[torch.Tensor, torch.Tensor | None]:
    """A row buffer for `rows` rows of format `quant`: (uint8 [rows, row
    bytes], fp32 [rows] scales, or None for bf16)."""
    data = torch.empty((max(rows, 1), moe_row_bytes(H, quant)), dtype=torch.uint8,
                       device=device)[:rows]
    scales = (torch.empty(max(rows, 1), dtype=torch.float32, device=device)[:rows]
              if quant else None)
    return data, scales


def _ptr(t: torch.Tensor | None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("expected a device tensor")
    if not t.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        stream = stream.cuda_stream
    return ctypes.c_void_p(int(stream))


def _check(fn: str, status: int):
    if status != 0:
        raise MoeError(fn, status)


def _want(t: torch.Tensor, dtype, name: str):
    if t.dtype != dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")


def moe_route_topk(logits: torch.Tensor, k: int, topk_idx: torch.Tensor,
                   topk_w: torch.Tensor, stream=None) -> None:
    """logits fp32 [T, E] -> topk_idx int32 [T, k], topk_w fp32 [T, k]."""
    _want(logits, torch.float32, "logits")
    _want(topk_idx, torch.int32, "topk_idx")
    _want(topk_w, torch.float32, "topk_w")
    T, E = logits.shape
    if topk_idx.numel() != T * k or topk_w.numel() != T * k:
        raise ValueError("topk outputs must hold T*k elements")
    _check("moe_route_topk", load().moe_route_topk(_ptr(logits), T, E, k, _ptr(topk_idx),
                                                   _ptr(topk_w), _stream(stream)))


def layout_workspace_bytes(T: int, E: int, k: int, R: int) -> int:
    n = ctypes.c_size_t(0)
    _check("moe_dispatch_layout",
           load().moe_dispatch_layout(None, T, E, k, R, 0, None, None, None, None, None, None,
                                      None, ctypes.byref(n), None))
    return int(n.value)


class Layout(NamedTuple):
    expert_counts: torch.Tensor   # [E]
    expert_offsets: torch.Tensor  # [E+1]
    rank_counts: torch.Tensor     # [R]
    rank_offsets: torch.Tensor    # [R+1]
    pos: torch.Tensor             # [T*k]
    row_src: torch.Tensor         # [T*k]
    workspace: torch.Tensor       # uint8 scratch


def alloc_layout(T: int, E: int, k: int, R: int, device) -> Layout:
    i32 = dict(dtype=torch.int32, device=device)
    ws = layout_workspace_bytes(T, E, k, R)
    return Layout(torch.empty(E, **i32), torch.empty(E + 1, **i32), torch.empty(R, **i32),
                  torch.empty(R + 1, **i32), torch.empty(max(T * k, 1), **i32),
                  torch.empty(max(T * k, 1), **i32),
                  torch.empty(ws, dtype=torch.uint8, device=device))


def moe_dispatch_layout(topk_idx: torch.Tensor, T: int, E: int, k: int, R: int, capacity: int,
                        out: Layout, stream=None) -> Layout:
    _want(topk_idx, torch.int32, "topk_idx")
    if topk_idx.numel() < T * k or out.pos.numel() < T * k or out.row_src.numel() < T * k:
        raise ValueError("layout buffers smaller than T*k")
    n = ctypes.c_size_t(out.workspace.numel())
    _check("moe_dispatch_layout",
           load().moe_dispatch_layout(_ptr(topk_idx), T, E, k, R, int(capacity),
                                      _ptr(out.expert_counts), _ptr(out.expert_offsets),
                                      _ptr(out.rank_counts), _ptr(out.rank_offsets),
                                      _ptr(out.pos), _ptr(out.row_src), _ptr(out.workspace),
                                      ctypes.byref(n), _stream(stream)))
    return out


def layout_chunks_workspace_bytes(T: int, chunk_tokens: int, E: int, k: int, R: int) -> int:
    n = ctypes.c_size_t(0)
    _check("moe_dispatch_layout_chunks",
           load().moe_dispatch_layout_chunks(None, T, chunk_tokens, E, k, R, 0, None, None, None,
                                             None, None, None, None, None, ctypes.byref(n), None))
    return int(n.value)


def route_layout_workspace_bytes(T: int, chunk_tokens: int, E: int, k: int, R: int) -> int:
    n = ctypes.c_size_t(0)
    _check("moe_route_layout_chunks",
           load().moe_route_layout_chunks(None, T, chunk_tokens, E, k, R, 0, None, None, None,
                                          None, None, None, None, None, None, None,
                                          ctypes.byref(n), None))
    return int(n.value)


class ChunkLayouts(NamedTuple):
    """Outputs of moe_dispatch_layout_chunks for C chunks of chunk_tokens."""
    expert_counts: torch.Tensor   # [C, E]
    expert_offsets: torch.Tensor  # [C, E+1]
    rank_counts: torch.Tensor     # [C, R]
    rank_offsets: torch.Tensor    # [C, R+1]
    pos: torch.Tensor             # [T*k], chunk-relative rows
    row_src: torch.Tensor         # [T*k], chunk-relative slots
    workspace: torch.Tensor
    chunk_tokens: int
    k: int


def alloc_layout_chunks(T: int, chunk_tokens: int, E: int, k: int, R: int, device,
                        chunks: int = 1) -> ChunkLayouts:
    """Room for ceil(T / chunk_tokens) chunks (at least `chunks` rows); the
    workspace serves moe_dispatch_layout_chunks and moe_route_layout_chunks
    over the whole batch, over its first chunk alone and over the remaining
    chunks (the calls a two-stream driver makes; the fused call's workspace
    depends on the number of tokens it is given)."""
    chunk_tokens = max(1, min(chunk_tokens, max(T, 1)))
    C = max(1, chunks, -(-T // chunk_tokens))
    i32 = dict(dtype=torch.int32, device=device)
    spans = {T, min(T, chunk_tokens), max(T - chunk_tokens, 0)}
    ws = max(max(layout_chunks_workspace_bytes(t, chunk_tokens, E, k, R),
                 route_layout_workspace_bytes(t, chunk_tokens, E, k, R)) for t in spans)
    return ChunkLayouts(torch.empty((C, E), **i32), torch.empty((C, E + 1), **i32),
                        torch.empty((C, R), **i32), torch.empty((C, R + 1), **i32),
                        torch.empty(max(T * k, 1), **i32), torch.empty(max(T * k, 1), **i32),
                        torch.empty(ws, dtype=torch.uint8, device=device), chunk_tokens, k)


def layout_view(lay: ChunkLayouts, c: int, T: int) -> Layout:
    """Chunk c of a ChunkLayouts as a one-chunk Layout (views, no copy)."""
    s0 = c * lay.chunk_tokens * lay.k
    s1 = min(T, (c + 1) * lay.chunk_tokens) * lay.k
    return Layout(lay.expert_counts[c], lay.expert_offsets[c], lay.rank_counts[c],
                  lay.rank_offsets[c], lay.pos[s0:max(s1, s0 + 1)],
                  lay.row_src[s0:max(s1, s0 + 1)], lay.workspace)


def layout_chunks_from(lay: ChunkLayouts, c0: int) -> ChunkLayouts:
    """Chunks c0.. of a ChunkLayouts as their own ChunkLayouts (views)."""
    s0 = c0 * lay.chunk_tokens * lay.k
    return ChunkLayouts(lay.expert_counts[c0:], lay.expert_offsets[c0:], lay.rank_counts[c0:],
                        lay.rank_offsets[c0:], lay.pos[s0:], lay.row_src[s0:], lay.workspace,
                        lay.chunk_tokens, lay.k)


def moe_dispatch_layout_chunks(topk_idx: torch.Tensor, T: int, E: int, k: int, R: int,
                               capacity: int, chunk_capacity: torch.Tensor | None,
                               out: ChunkLayouts, stream=None) -> ChunkLayouts:
    _want(topk_idx, torch.int32, "topk_idx")
    if topk_idx.numel() < T * k or out.pos.numel() < T * k:
        raise ValueError("layout buffers smaller than T*k")
    if chunk_capacity is not None:
        _want(chunk_capacity, torch.int32, "chunk_capacity")
    n = ctypes.c_size_t(out.workspace.numel())
    _check("moe_dispatch_layout_chunks",
           load().moe_dispatch_layout_chunks(
               _ptr(topk_idx), T, out.chunk_tokens, E, k, R, int(capacity), _ptr(chunk_capacity),
               _ptr(out.expert_counts), _ptr(out.expert_offsets), _ptr(out.rank_counts),
               _ptr(out.rank_offsets), _ptr(out.pos), _ptr(out.row_src), _ptr(out.workspace),
               ctypes.byref(n), _stream(stream)))
    return out


def moe_route_layout_chunks(logits: torch.Tensor, k: int, R: int, capacity: int,
                            chunk_capacity: torch.Tensor | None, topk_idx: torch.Tensor,
                            topk_w: torch.Tensor, out: ChunkLayouts, stream=None) -> ChunkLayouts:
    """logits fp32 [T, E] -> topk_idx / topk_w [T, k] and every chunk's layout."""
    _want(logits, torch.float32, "logits")
    _want(topk_idx, torch.int32, "topk_idx")
    _want(topk_w, torch.float32, "topk_w")
    T, E = logits.shape
    if topk_idx.numel() < T * k or topk_w.numel() < T * k or out.pos.numel() < T * k:
        raise ValueError("route / layout buffers smaller than T*k")
    if chunk_capacity is not None:
        _want(chunk_capacity, torch.int32, "chunk_capacity")
    n = ctypes.c_size_t(out.workspace.numel())
    _check("moe_route_layout_chunks",
           load().moe_route_layout_chunks(
               _ptr(logits), T, out.chunk_tokens, E, k, R, int(capacity), _ptr(chunk_capacity),
               _ptr(topk_idx), _ptr(topk_w), _ptr(out.expert_counts), _ptr(out.expert_offsets),
               _ptr(out.rank_counts), _ptr(out.rank_offsets), _ptr(out.pos), _ptr(out.row_src),
               _ptr(out.workspace), ctypes.byref(n), _stream(stream)))
    return out


MOE_NOALLOC_SCRATCH_BYTES = 4 << 20  # static scratch of moe_route_layout_chunks_noalloc


def moe_route_layout_chunks_noalloc(logits: torch.Tensor, k: int, R: int, capacity: int,
                                    chunk_capacity: torch.Tensor | None, topk_idx: torch.Tensor,
                                    topk_w: torch.Tensor, out: ChunkLayouts,
                                    stream=None) -> ChunkLayouts:
    """As moe_route_layout_chunks, with the histogram scratch in the
    library's static device buffer: out.workspace is not used."""
    _want(logits, torch.float32, "logits")
    _want(topk_idx, torch.int32, "topk_idx")
    _want(topk_w, torch.float32, "topk_w")
    T, E = logits.shape
    if topk_idx.numel() < T * k or topk_w.numel() < T * k or out.pos.numel() < T * k:
        raise ValueError("route / layout buffers smaller than T*k")
    if chunk_capacity is not None:
        _want(chunk_capacity, torch.int32, "chunk_capacity")
    _check("moe_route_layout_chunks_noalloc",
           load().moe_route_layout_chunks_noalloc(
               _ptr(logits), T, out.chunk_tokens, E, k, R, int(capacity), _ptr(chunk_capacity),
               _ptr(topk_idx), _ptr(topk_w), _ptr(out.expert_counts), _ptr(out.expert_offsets),
               _ptr(out.rank_counts), _ptr(out.rank_offsets), _ptr(out.pos), _ptr(out.row_src),
               _stream(stream)))
    return out


def _want_scales(t: torch.Tensor | None, rows: int, quant: int, name: str):
    """A quantised row buffer's scale array: fp32, at least `rows` entries."""
    if quant == MOE_QUANT_BF16:
        return
    if t is None:
        raise ValueError(f"{name}: a quantised payload needs its fp32 scale array")
    _want(t, torch.float32, name)
    if t.numel() < rows:
        raise ValueError(f"{name} must hold {rows} scales")


def moe_dispatch_pack(x: torch.Tensor, T: int, H: int, k: int, pos: torch.Tensor, quant: int,
                      send: torch.Tensor, send_scales: torch.Tensor | None = None,
                      stream=None) -> None:
    """x bf16 [T, H] (or its int16/uint16 bits); send uint8 [rows, row_bytes];
    send_scales fp32 [rows] for the quantised formats.  quant may carry
    MOE_PACK_STREAM."""
    if x.element_size() != 2:
        raise ValueError("x must hold bf16 bits")
    _want(pos, torch.int32, "pos")
    if x.numel() < T * H or pos.numel() < T * k:
        raise ValueError("x / pos too small")
    _want_scales(send_scales, 0, quant & ~MOE_PACK_STREAM, "send_scales")
    _check("moe_dispatch_pack", load().moe_dispatch_pack(_ptr(x), T, H, k, _ptr(pos), quant,
                                                         _ptr(send), _ptr(send_scales),
                                                         _stream(stream)))


def moe_combine(recv: torch.Tensor, recv_scales: torch.Tensor | None, quant: int,
                pos: torch.Tensor, topk_w: torch.Tensor, T: int, H: int, k: int,
                out: torch.Tensor, stream=None) -> None:
    _want(pos, torch.int32, "pos")
    _want(topk_w, torch.float32, "topk_w")
    if out.element_size() != 2 or out.numel() < T * H:
        raise ValueError("out must hold T*H bf16 values")
    _want_scales(recv_scales, 0, quant, "recv_scales")
    _check("moe_combine", load().moe_combine(_ptr(recv), _ptr(recv_scales), quant, _ptr(pos),
                                             _ptr(topk_w), T, H, k, _ptr(out), _stream(stream)))


def moe_combine_pack(recv: torch.Tensor | None, recv_scales: torch.Tensor | None,
                     pos_c: torch.Tensor | None, topk_w: torch.Tensor | None, Tc: int,
                     out: torch.Tensor | None, x: torch.Tensor | None,
                     pos_p: torch.Tensor | None, Tp: int, send: torch.Tensor | None,
                     send_scales: torch.Tensor | None, H: int, k: int, quant: int,
                     stream=None) -> None:
    """moe_combine of Tc tokens and moe_dispatch_pack of Tp tokens in one
    launch; the tensors of a half with no tokens may be None (and the scale
    arrays are None for bf16).  quant may carry MOE_PACK_STREAM (pack half)."""
    fmt = quant & ~MOE_PACK_STREAM
    if Tc > 0:
        _want(pos_c, torch.int32, "pos_c")
        _want(topk_w, torch.float32, "topk_w")
        if out.element_size() != 2 or out.numel() < Tc * H:
            raise ValueError("out must hold Tc*H bf16 values")
        _want_scales(recv_scales, 0, fmt, "recv_scales")
    if Tp > 0:
        if x.element_size() != 2:
            raise ValueError("x must hold bf16 bits")
        _want(pos_p, torch.int32, "pos_p")
        if x.numel() < Tp * H or pos_p.numel() < Tp * k:
            raise ValueError("x / pos_p too small")
        _want_scales(send_scales, 0, fmt, "send_scales")
    _check("moe_combine_pack",
           load().moe_combine_pack(_ptr(recv), _ptr(recv_scales), _ptr(pos_c), _ptr(topk_w), Tc,
                                   _ptr(out), _ptr(x), _ptr(pos_p), Tp, _ptr(send),
                                   _ptr(send_scales), H, k, quant, _stream(stream)))


class RecvLayout(NamedTuple):
    recv_offsets: torch.Tensor   # [R, R+1] int32: segment starts per receiver (flat rows)
    group_offsets: torch.Tensor  # [E+1] int32: first grouped row per expert; [E] = N
    group_seg: torch.Tensor      # [E, R] int32: first grouped row of (expert, source)
    group_pos: torch.Tensor      # [max_rows] int32: grouped row of receive row q, -1 past N
    group_src: torch.Tensor      # [max_rows] int32: receive row of grouped row p, -1 past N

    @property
    def max_rows(self) -> int:
        return self.group_pos.numel()


def alloc_recv_layout(E: int, R: int, max_rows: int, device) -> RecvLayout:
    i32 = dict(dtype=torch.int32, device=device)
    return RecvLayout(torch.empty((R, R + 1), **i32), torch.empty(E + 1, **i32),
                      torch.empty((E, R), **i32), torch.empty(max(max_rows, 1), **i32)[:max_rows],
                      torch.empty(max(max_rows, 1), **i32)[:max_rows])


def _want_offsets(src_offsets: torch.Tensor, E: int, R: int):
    _want(src_offsets, torch.int32, "src_offsets")
    if src_offsets.numel() < R * (E + 1):
        raise ValueError("src_offsets must hold [R, E+1] int32")


def _want_rows(t: torch.Tensor, scales: torch.Tensor | None, rows: int, H: int, quant: int,
               name: str):
    if not t.is_contiguous() or t.numel() * t.element_size() < rows * moe_row_bytes(H, quant):
        raise ValueError(f"{name} must be contiguous and hold {rows} rows")
    _want_scales(scales, rows, quant, name + " scales")


def moe_recv_layout(src_offsets: torch.Tensor, E: int, R: int, out: RecvLayout,
                    stream=None) -> RecvLayout:
    _want_offsets(src_offsets, E, R)
    if (out.recv_offsets.numel() < R * (R + 1) or out.group_offsets.numel() < E + 1 or
            out.group_seg.numel() < E * R or out.group_src.numel() != out.max_rows):
        raise ValueError("RecvLayout buffers too small")
    _check("moe_recv_layout",
           load().moe_recv_layout(_ptr(src_offsets), E, R, out.max_rows, _ptr(out.recv_offsets),
                                  _ptr(out.group_offsets), _ptr(out.group_seg),
                                  _ptr(out.group_pos), _ptr(out.group_src), _stream(stream)))
    return out


def moe_recv_regroup(recv: torch.Tensor, recv_scales: torch.Tensor | None, max_rows: int,
                     H: int, quant: int, group_src: torch.Tensor, grouped: torch.Tensor,
                     grouped_scales: torch.Tensor | None, stream=None) -> None:
    _want(group_src, torch.int32, "group_src")
    if group_src.numel() < max_rows:
        raise ValueError("group_src shorter than max_rows")
    _want_rows(recv, recv_scales, max_rows, H, quant, "recv")
    _want_rows(grouped, grouped_scales, max_rows, H, quant, "grouped")
    _check("moe_recv_regroup",
           load().moe_recv_regroup(_ptr(recv), _ptr(recv_scales), max_rows, H, quant,
                                   _ptr(group_src), _ptr(grouped), _ptr(grouped_scales),
                                   _stream(stream)))


def moe_recv_ungroup(grouped: torch.Tensor, grouped_scales: torch.Tensor | None, max_rows: int,
                     H: int, quant: int, group_pos: torch.Tensor, recv: torch.Tensor,
                     recv_scales: torch.Tensor | None, stream=None) -> None:
    _want(group_pos, torch.int32, "group_pos")
    if group_pos.numel() < max_rows:
        raise ValueError("group_pos shorter than max_rows")
    _want_rows(recv, recv_scales, max_rows, H, quant, "recv")
    _want_rows(grouped, grouped_scales, max_rows, H, quant, "grouped")
    _check("moe_recv_ungroup",
           load().moe_recv_ungroup(_ptr(grouped), _ptr(grouped_scales), max_rows, H, quant,
                                   _ptr(group_pos), _ptr(recv), _ptr(recv_scales),
                                   _stream(stream)))


# torch's own calls behind current_stream() and current_device(), without the
# Stream object and the check for a first use: 1.3 us less a call
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda device: torch.cuda.current_stream(device).cuda_stream)
_raw_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _call(name: str, stream, *args) -> None:
    """Entry point `name` on `args`, its tensors as their addresses, and the
    stream: `stream`, or the current stream of the tensors' device.  The
    tensors must be contiguous and share one device, which is current during
    the call (a null stream is the current device's).  Plain ints and the
    argtypes rather than c_void_p objects: half the cost of a call."""
    device, raw, tensor = None, [], torch.Tensor
    for a in args:
        if isinstance(a, tensor):
            d = a.get_device()
            if d != device:
                if d < 0:
                    raise ValueError("expected a device tensor")
                if device is not None:
                    raise ValueError(f"tensors on different devices: cuda:{device}, cuda:{d}")
                device = d
            if not a.is_contiguous():
                raise ValueError("expected a contiguous tensor")
            a = a.data_ptr()
        raw.append(a)
    if stream is None:
        stream = _raw_stream(device)
    elif isinstance(stream, torch.cuda.Stream):
        if stream.device_index != device:
            raise ValueError(f"a stream of cuda:{stream.device_index}, tensors on cuda:{device}")
        stream = stream.cuda_stream
    else:
        stream = int(stream)
    entry = getattr(_lib or load(), name)
    if device == _raw_device():
        status = entry(*raw, stream)
    else:
        with torch.cuda.device(device):
            status = entry(*raw, stream)
    if status:
        _check(name, status)


def stream_handle(stream, device: torch.device) -> int:
    """The handle of `stream`: a torch stream, a handle, or None for the device's
    current one."""
    if stream is None:
        return _raw_stream(device.index)
    return stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)


def stream_of(stream, device: torch.device) -> torch.cuda.Stream:
    """The same as torch's stream."""
    if isinstance(stream, torch.cuda.Stream):
        return stream
    if stream is None:
        return torch.cuda.current_stream(device)
    handle = int(stream)
    return (torch.cuda.ExternalStream(handle, device=device) if handle else
            torch.cuda.default_stream(device))


_BF16_TYPES = (torch.bfloat16, torch.int16, torch.uint16)  # values, or their bits


def _want_bf16(t: torch.Tensor, shape, name: str):
    """bf16 values (or their int16/uint16 bits) of exactly `shape`."""
    if t.dtype not in _BF16_TYPES:
        raise ValueError(f"{name} must hold bf16 values or their bits, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {shape}, got {tuple(t.shape)}")


class Balance(NamedTuple):
    """Outputs of moe_balance_loss for S segments of seg_tokens tokens."""
    loss: torch.Tensor           # [S] fp32
    expert_counts: torch.Tensor  # [S, E] int32
    prob_sums: torch.Tensor      # [S, E] fp32
    tokens: torch.Tensor         # [S] int32: live tokens
    workspace: torch.Tensor      # uint8 scratch
    seg_tokens: int


def balance_workspace_bytes(T: int, seg_tokens: int, E: int, k: int) -> int:
    n = ctypes.c_size_t(0)
    _check("moe_balance_loss",
           load().moe_balance_loss(None, None, None, T, seg_tokens, E, k, None, None, None, None,
                                   None, ctypes.byref(n), None))
    return int(n.value)


def alloc_balance(T: int, seg_tokens: int, E: int, k: int, device) -> Balance:
    """Outputs and workspace for T tokens in segments of seg_tokens."""
    seg_tokens = max(1, min(seg_tokens, max(T, 1)))
    S = max(1, -(-T // seg_tokens))
    f32, i32 = dict(dtype=torch.float32, device=device), dict(dtype=torch.int32, device=device)
    ws = balance_workspace_bytes(T, seg_tokens, E, k)
    return Balance(torch.empty(S, **f32), torch.empty((S, E), **i32), torch.empty((S, E), **f32),
                   torch.empty(S, **i32), torch.empty(ws, dtype=torch.uint8, device=device),
                   seg_tokens)


def _want_mask(mask: torch.Tensor | None, T: int):
    if mask is not None:
        if mask.element_size() != 1:
            raise ValueError("token_mask: expected one byte per token (uint8 or bool)")
        if mask.numel() != T:
            raise ValueError("token_mask must hold one byte per token")


def _want_segments(b: Balance, T: int, E: int):
    loss, counts, sums, tokens, _, seg_tokens = b
    S = max(1, -(-T // seg_tokens))
    _want(loss, torch.float32, "loss")
    _want(counts, torch.int32, "expert_counts")
    _want(sums, torch.float32, "prob_sums")
    _want(tokens, torch.int32, "tokens")
    if (loss.numel() < S or tokens.numel() < S or counts.numel() < S * E or
            sums.numel() < S * E):
        raise ValueError("Balance buffers too small")


def moe_balance_loss(logits: torch.Tensor, topk_idx: torch.Tensor,
                     token_mask: torch.Tensor | None, out: Balance, stream=None) -> Balance:
    """logits fp32 [T, E], topk_idx int32 [T, k], token_mask uint8 [T] or
    None -> out.loss, expert_counts, prob_sums and tokens per segment."""
    _want(logits, torch.float32, "logits")
    _want(topk_idx, torch.int32, "topk_idx")
    T, E = logits.shape
    if topk_idx.dim() != 2 or topk_idx.shape[0] != T:
        raise ValueError("topk_idx must be [T, k]")
    _want_mask(token_mask, T)
    _want_segments(out, T, E)
    n = ctypes.c_size_t(out.workspace.numel())
    _call("moe_balance_loss", stream, logits, topk_idx, token_mask, T, out.seg_tokens, E,
          topk_idx.shape[1], out.loss, out.expert_counts, out.prob_sums, out.tokens,
          out.workspace, ctypes.byref(n))
    return out


def moe_route_grad(logits: torch.Tensor | None, topk_idx: torch.Tensor,
                   topk_w: torch.Tensor | None, d_topk_w: torch.Tensor | None,
                   token_mask: torch.Tensor | None, d_loss: torch.Tensor | None,
                   balance: Balance | None, d_logits: torch.Tensor, stream=None,
                   masked_gates: bool = False) -> torch.Tensor:
    """Gradient of the router's logits [T, E] from that of the gate weights
    (d_topk_w [T, k] or None) and of the balance loss (d_loss [S] with the
    forward call's Balance, or None for both).  A masked token's row is zero;
    with masked_gates it keeps the part through the gate weights."""
    _want(d_logits, torch.float32, "d_logits")
    _want(topk_idx, torch.int32, "topk_idx")
    T, E = d_logits.shape
    if topk_idx.dim() != 2 or topk_idx.shape[0] != T:
        raise ValueError("topk_idx must be [T, k]")
    k = topk_idx.shape[1]
    _want_mask(token_mask, T)
    if d_topk_w is not None:
        if topk_w is None:
            raise ValueError("d_topk_w needs topk_w")
        for t, name in ((topk_w, "topk_w"), (d_topk_w, "d_topk_w")):
            _want(t, torch.float32, name)
            if t.numel() != T * k:
                raise ValueError(f"{name} must hold T*k elements")
    if d_loss is not None:
        if logits is None or balance is None:
            raise ValueError("d_loss needs logits and the forward call's Balance")
        _want(logits, torch.float32, "logits")
        if tuple(logits.shape) != (T, E):
            raise ValueError("logits and d_logits differ in shape")
        _want_segments(balance, T, E)
        _want(d_loss, torch.float32, "d_loss")
        if d_loss.numel() < max(1, -(-T // balance.seg_tokens)):
            raise ValueError("d_loss must hold one value per segment")
    counts = balance.expert_counts if d_loss is not None else None
    live = balance.tokens if d_loss is not None else None
    seg = balance.seg_tokens if d_loss is not None else max(T, 1)
    _call("moe_route_grad", stream, logits, topk_idx, topk_w, d_topk_w, token_mask, d_loss, counts,
          live, T, seg, E, k | MOE_ROUTE_MASKED_GATES if masked_gates else k, d_logits)
    return d_logits


def moe_combine_grad(d_out: torch.Tensor, recv: torch.Tensor | None,
                     recv_scales: torch.Tensor | None, quant: int, pos: torch.Tensor,
                     topk_w: torch.Tensor, T: int, H: int, k: int, d_recv: torch.Tensor | None,
                     d_topk_w: torch.Tensor | None, stream=None) -> None:
    """Gradient of moe_combine: d_out bf16 [T, H] -> d_recv (bf16 rows, as
    [rows, H] or as the bytes of a bf16 payload) and d_topk_w fp32 [T*k];
    either output may be None.  d_recv has fewer than T*k rows only where its
    shape says that they are whole ones."""
    if d_out.dtype not in _BF16_TYPES or d_out.numel() < T * H:
        raise ValueError("d_out must hold T*H bf16 values")
    if d_recv is not None:
        if d_recv.dtype not in _BF16_TYPES and d_recv.dtype != torch.uint8:
            raise ValueError(f"d_recv takes rows of bf16, not {d_recv.dtype}")
        if d_recv.nbytes < T * k * H * 2 and (
                d_recv.dim() != 2 or d_recv.shape[1] * d_recv.element_size() != 2 * H):
            raise ValueError("d_recv must hold rows of 2*H bytes, whatever the payload of recv")
    _want(pos, torch.int32, "pos")
    _want(topk_w, torch.float32, "topk_w")
    if pos.numel() < T * k or topk_w.numel() < T * k:
        raise ValueError("pos / topk_w too small")
    if d_topk_w is not None:
        _want(d_topk_w, torch.float32, "d_topk_w")
        if d_topk_w.numel() < T * k:
            raise ValueError("d_topk_w must hold T*k values")
        if recv is not None and recv.element_size() > (2 if quant == MOE_QUANT_BF16 else 1):
            raise ValueError(f"recv: {recv.dtype} does not hold rows of this payload")
        _want_scales(recv_scales, 0, quant, "recv_scales")
    _call("moe_combine_grad", stream, d_out, recv, recv_scales, quant, pos, topk_w, T, H, k, d_recv,
          d_topk_w)


def _want_weights(w: torch.Tensor, offsets: torch.Tensor):
    if w.dim() != 3:
        raise ValueError("weights must be [E, N, K]")
    _want(offsets, torch.int32, "offsets")
    if offsets.numel() != w.shape[0] + 1:
        raise ValueError("offsets must hold E+1 int32")


@functools.lru_cache(maxsize=4096)
def expert_workspace_bytes(name: str, E: int, rows: int, K: int, N: int,
                           act: int = MOE_ACT_NONE) -> int:
    """Workspace of moe_expert_matmul, _dx or _dw (`name`) for these sizes."""
    n, i, none = ctypes.c_size_t(0), ctypes.byref, None
    if name == "moe_expert_matmul":
        status = load().moe_expert_matmul(none, none, none, none, act, none, E, rows, K, N, none,
                                          none, none, i(n), none)
    elif name == "moe_expert_matmul_dx":
        status = load().moe_expert_matmul_dx(none, none, none, 0, none, E, rows, K, N, none, none,
                                             i(n), none)
    else:
        status = load().moe_expert_matmul_dw(none, none, none, E, rows, K, N, 0, none, none, none,
                                             i(n), none)
    _check(name, status)
    return int(n.value)


def _call_sharing(name: str, stream, workspace: torch.Tensor | None, sizes: tuple,
                  like: torch.Tensor, *args) -> None:
    """A product's call with its workspace: `workspace`, or one allocated for the
    call (torch's allocator, in the stream's order) when the sizes want one."""
    _call_with_room(name, stream, workspace, expert_workspace_bytes(name, *sizes), like, *args)


def _call_with_room(name: str, stream, workspace: torch.Tensor | None, need: int,
                    like: torch.Tensor, *args) -> None:
    """A call with its workspace of `need` bytes, `workspace` or one allocated
    for the call."""
    if not need:
        _call(name, stream, *args, None, None)
        return
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=like.device)
        if stream is not None and workspace.is_cuda:
            # allocated in the current stream's order, used in this one's
            current = torch.cuda.current_stream(like.device)
            if stream_handle(stream, like.device) != current.cuda_stream:
                user = stream_of(stream, like.device)
                user.wait_stream(current)
                workspace.record_stream(user)
    n = ctypes.c_size_t(workspace.numel() * workspace.element_size())
    _call(name, stream, *args, workspace, ctypes.byref(n))


def moe_expert_matmul(x: torch.Tensor, offsets: torch.Tensor, w: torch.Tensor,
                      bias: torch.Tensor | None, act: int, residual: torch.Tensor | None,
                      out: torch.Tensor, preact: torch.Tensor | None = None, stream=None,
                      workspace: torch.Tensor | None = None) -> torch.Tensor:
    """x bf16 [rows, K] in runs of offsets int32 [E+1], w bf16 [E, N, K]
    ([E, 2N, K] for MOE_ACT_SWIGLU) -> out bf16 [rows, N]; bias fp32 [E, N]
    ([E, 2N]); preact bf16 [rows, N] ([rows, 2N]) keeps z for the gradient;
    workspace: scratch of expert_workspace_bytes, else allocated where wanted."""
    _want_weights(w, offsets)
    E, wide_n, K = w.shape
    wide = 2 if act == MOE_ACT_SWIGLU else 1
    if wide_n % wide:
        raise ValueError("MOE_ACT_SWIGLU takes an even number of weight rows")
    rows, N = x.shape[0], wide_n // wide
    _want_bf16(w, (E, wide_n, K), "w")
    _want_bf16(x, (rows, K), "x")
    _want_bf16(out, (rows, N), "out")
    if residual is not None:
        _want_bf16(residual, (rows, N), "residual")
    if preact is not None:
        _want_bf16(preact, (rows, wide_n), "preact")
    if bias is not None:
        _want(bias, torch.float32, "bias")
        if bias.numel() != E * wide_n:
            raise ValueError("bias must hold one value per weight row")
    _call_sharing("moe_expert_matmul", stream, workspace, (E, rows, K, N, act), x, x, offsets, w,
                  bias, act, residual, E, rows, K, N, out, preact)
    return out


def moe_expert_matmul_dx(dy: torch.Tensor, offsets: torch.Tensor, w: torch.Tensor, act: int,
                         preact: torch.Tensor | None, dx: torch.Tensor, stream=None,
                         workspace: torch.Tensor | None = None) -> torch.Tensor:
    """dy bf16 [rows, N], w bf16 [E, N, K] -> dx bf16 [rows, K], through the
    activation before the product when act says so (preact and dx [rows, K],
    or [rows, 2K] for MOE_ACT_SWIGLU).  workspace: as moe_expert_matmul."""
    _want_weights(w, offsets)
    E, N, K = w.shape
    rows, wide = dy.shape[0], 2 if act == MOE_ACT_SWIGLU else 1
    _want_bf16(w, (E, N, K), "w")
    _want_bf16(dy, (rows, N), "dy")
    _want_bf16(dx, (rows, wide * K), "dx")
    if act == MOE_ACT_NONE:
        preact = None
    elif preact is None:
        raise ValueError("an activation's gradient needs preact")
    else:
        _want_bf16(preact, (rows, wide * K), "preact")
    _call_sharing("moe_expert_matmul_dx", stream, workspace, (E, rows, K, N), dy, dy, offsets, w,
                  act, preact, E, rows, K, N, dx)
    return dx


def moe_expert_matmul_dw(dy: torch.Tensor, x: torch.Tensor, offsets: torch.Tensor,
                         dw: torch.Tensor, dbias: torch.Tensor | None = None,
                         accumulate: bool = False, stream=None,
                         workspace: torch.Tensor | None = None) -> torch.Tensor:
    """dy bf16 [rows, N], x bf16 [rows, K] -> dw [E, N, K] (fp32, or bf16 by
    its dtype) and dbias fp32 [E, N]; accumulate adds to what they hold
    (fp32 dw only).  workspace: as moe_expert_matmul."""
    _want_weights(dw, offsets)
    E, N, K = dw.shape
    rows = dy.shape[0]
    _want_bf16(dy, (rows, N), "dy")
    _want_bf16(x, (rows, K), "x")
    if dw.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError(f"dw: expected float32 or bfloat16, got {dw.dtype}")
    if dbias is not None:
        _want(dbias, torch.float32, "dbias")
        if dbias.numel() != E * N:
            raise ValueError("dbias must hold E*N values")
    flags = MOE_GRAD_FP32 if dw.dtype == torch.float32 else MOE_GRAD_BF16
    if accumulate:
        flags |= MOE_GRAD_ACCUMULATE
    _call_sharing("moe_expert_matmul_dw", stream, workspace, (E, rows, K, N), dy, dy, x, offsets,
                  E, rows, K, N, flags, dw, dbias)
    return dw


# ---- the norm in front of a layer, E4M3 codes and their products

_CODE_TYPES = (torch.float8_e4m3fn, torch.uint8)  # E4M3 values, or their bits


def code_blocks(n: int) -> int:
    """Blocks of 128 values with a scale each."""
    return -(-n // MOE_BLOCK_128)


def _want_codes(t: torch.Tensor, shape, name: str):
    if t.dtype not in _CODE_TYPES:
        raise ValueError(f"{name} must hold E4M3 codes, not {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")


def _want_floats(t: torch.Tensor, shapes, name: str):
    """fp32 of one of `shapes`."""
    if t.dtype is not torch.float32:
        _want(t, torch.float32, name)
    if t.shape not in shapes:
        raise ValueError(f"{name}: expected shape {shapes[0]}, got {tuple(t.shape)}")


def _want_coded(codes: torch.Tensor | None, scales: torch.Tensor | None, rows: int, n: int,
                halves: int, name: str = "codes"):
    """Codes [rows, halves * n] with their scales [rows, halves, blocks of n] (one
    half: [rows, blocks] too), or neither."""
    if (codes is None) != (scales is None):
        raise ValueError(f"{name} and their scales come together")
    if codes is not None:
        _want_codes(codes, (rows, halves * n), name)
        flat = ((rows, code_blocks(n)),) if halves == 1 else ()
        _want_floats(scales, ((rows, halves, code_blocks(n)),) + flat, f"the scales of {name}")


def moe_add_norm(x: torch.Tensor, residual: torch.Tensor | None, weight: torch.Tensor | None,
                 eps: float, sum: torch.Tensor | None, y: torch.Tensor | None,
                 codes: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                 stream=None) -> None:
    """s = x + residual (bf16 [T, H] each; residual may be None) and its
    root-mean-square norm by weight fp32 [H] -> sum and y bf16 [T, H], codes
    E4M3 [T, H] with scales fp32 [T] (one a row) or [T, ceil(H / 128)]; any output
    may be None, but not both y and codes."""
    shape = x.shape
    if len(shape) != 2:
        raise ValueError("x must be [T, H]")
    T, H = shape
    _want_bf16(x, shape, "x")
    if residual is not None:
        _want_bf16(residual, shape, "residual")
    if sum is not None:
        _want_bf16(sum, shape, "sum")
    if y is not None:
        _want_bf16(y, shape, "y")
    if weight is not None:
        _want_floats(weight, ((H,),), "weight")
    if (codes is None) != (scales is None):
        raise ValueError("codes and scales come together")
    if codes is not None:
        _want_codes(codes, shape, "codes")
        _want_floats(scales, ((T, code_blocks(H)), (T,)), "scales")
    block = MOE_BLOCK_ROW if scales is None or scales.dim() == 1 else MOE_BLOCK_128
    _call("moe_add_norm", stream, x, residual, weight, float(eps), T, H, sum, y, block, codes, scales)


@functools.lru_cache(maxsize=4096)
def add_norm_grad_workspace_bytes(T: int, H: int) -> int:
    """Workspace of moe_add_norm_grad with d_weight."""
    n = ctypes.c_size_t(0)
    _check("moe_add_norm_grad",
           load().moe_add_norm_grad(None, None, None, None, 0.0, T, H, None, None, 0, None,
                                    ctypes.byref(n), None))
    return int(n.value)


def moe_add_norm_grad(d_y: torch.Tensor, d_sum: torch.Tensor | None, sum: torch.Tensor,
                      weight: torch.Tensor | None, eps: float, d_x: torch.Tensor,
                      d_weight: torch.Tensor | None = None, accumulate: bool = False, stream=None,
                      workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Gradient of moe_add_norm at `sum` bf16 [T, H] from those of y (d_y) and of
    the sum (d_sum or None): d_x bf16 [T, H], of x and of the residual, and
    d_weight fp32 [H] (which accumulate adds to) or None.  workspace: scratch of
    add_norm_grad_workspace_bytes, else allocated where wanted."""
    shape = d_y.shape
    if len(shape) != 2:
        raise ValueError("d_y must be [T, H]")
    T, H = shape
    _want_bf16(d_y, shape, "d_y")
    if d_sum is not None:
        _want_bf16(d_sum, shape, "d_sum")
    _want_bf16(sum, shape, "sum")
    _want_bf16(d_x, shape, "d_x")
    if weight is not None:
        _want_floats(weight, ((H,),), "weight")
    if d_weight is not None:
        _want_floats(d_weight, ((H,),), "d_weight")
    need = 0 if d_weight is None else add_norm_grad_workspace_bytes(T, H)
    _call_with_room("moe_add_norm_grad", stream, workspace, need, d_y, d_y, d_sum, sum, weight,
                    float(eps), T, H, d_x, d_weight, int(accumulate))
    return d_x


def moe_quant_rows(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                   offsets: torch.Tensor | None = None, halves: int = 1, stream=None) -> None:
    """bf16 x [rows, H] -> E4M3 codes [rows, H] and scales fp32 [rows, ceil(H / 128)]
    (halves 2: [rows, 2, ceil(H / 2 / 128)]); with offsets int32 [E+1] of the rows of
    runs alone."""
    if x.dim() != 2 or halves not in (1, 2) or x.shape[1] % halves:
        raise ValueError("x must be [rows, H], in 1 or 2 halves")
    rows, H = x.shape
    _want_bf16(x, (rows, H), "x")
    _want_coded(codes, scales, rows, H // halves, halves)
    E = 0
    if offsets is not None:
        _want(offsets, torch.int32, "offsets")
        E = offsets.numel() - 1
        if E < 1:
            raise ValueError("offsets must hold E+1 int32")
    _call("moe_quant_rows", stream, x, offsets, E, rows, H, halves, codes, scales)


def moe_quant_weights(w: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                      codes_t: torch.Tensor | None = None, scales_t: torch.Tensor | None = None,
                      halves: int = 1, stream=None) -> None:
    """bf16 w [E, halves * N, K] -> E4M3 codes of its shape with scales fp32 [E, halves,
    ceil(N / 128), ceil(K / 128)], and codes_t [E, K, halves * N] with scales_t [E, ceil(K /
    128), halves, ceil(N / 128)] (or None)."""
    if w.dim() != 3 or halves not in (1, 2) or w.shape[1] % halves:
        raise ValueError("w must be [E, N, K], in 1 or 2 halves of N")
    E, wide_n, K = w.shape
    N = wide_n // halves
    nbn, nbk = code_blocks(N), code_blocks(K)
    _want_bf16(w, (E, wide_n, K), "w")
    _want_codes(codes, (E, wide_n, K), "codes")
    _want_floats(scales, ((E, halves, nbn, nbk),) + (((E, nbn, nbk),) if halves == 1 else ()), "scales")
    if (codes_t is None) != (scales_t is None):
        raise ValueError("codes_t and scales_t come together")
    if codes_t is not None:
        _want_codes(codes_t, (E, K, wide_n), "codes_t")
        _want_floats(scales_t, ((E, nbk, halves, nbn),) + (((E, nbk, nbn),) if halves == 1 else ()),
                     "scales_t")
    _call("moe_quant_weights", stream, w, E, N, K, halves, codes, scales, codes_t, scales_t)


@functools.lru_cache(maxsize=4096)
def expert_fp8_workspace_bytes(name: str, E: int, rows: int, K: int, N: int,
                               act: int = MOE_ACT_NONE, halves: int = 1) -> int:
    """Workspace of moe_expert_matmul_fp8 or _fp8_dx (`name`) for these sizes."""
    n, i, none = ctypes.c_size_t(0), ctypes.byref, None
    if name == "moe_expert_matmul_fp8":
        status = load().moe_expert_matmul_fp8(none, none, 1, none, none, none, none, act, none, E,
                                              rows, K, N, none, none, none, none, none, i(n), none)
    else:
        status = load().moe_expert_matmul_fp8_dx(none, none, none, none, none, halves, act, none, E,
                                                 rows, K, N, none, none, none, none, i(n), none)
    _check(name, status)
    return int(n.value)


def moe_expert_matmul_fp8(x: torch.Tensor, x_scales: torch.Tensor, offsets: torch.Tensor,
                          w: torch.Tensor, w_scales: torch.Tensor, bias: torch.Tensor | None,
                          act: int, residual: torch.Tensor | None, out: torch.Tensor | None,
                          codes: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                          preact: torch.Tensor | None = None, stream=None,
                          workspace: torch.Tensor | None = None) -> None:
    """moe_expert_matmul of E4M3 x [rows, K] with x_scales fp32 [rows, ceil(K / 128)]
    or [rows] (one a row) and w E4M3 [E, N, K] with w_scales [E, ceil(N / 128), ceil(K /
    128)] (MOE_ACT_SWIGLU: [E, 2N, K], [E, 2, ...]) -> out bf16 [rows, N], codes [rows,
    N] with scales [rows, ceil(N / 128)], or both; preact as there; workspace: for
    codes, scratch of expert_fp8_workspace_bytes, else allocated where wanted."""
    _want_weights(w, offsets)
    E, wide_n, K = w.shape
    wide = 2 if act == MOE_ACT_SWIGLU else 1
    if wide_n % wide:
        raise ValueError("MOE_ACT_SWIGLU takes an even number of weight rows")
    rows, N = x.shape[0], wide_n // wide
    nbn, nbk = code_blocks(N), code_blocks(K)
    _want_codes(w, (E, wide_n, K), "w")
    _want_floats(w_scales, ((E, wide, nbn, nbk),) + (((E, nbn, nbk),) if wide == 1 else ()), "w_scales")
    _want_codes(x, (rows, K), "x")
    _want_floats(x_scales, ((rows, nbk), (rows,), (rows, 1)), "x_scales")
    _want_coded(codes, scales, rows, N, 1)
    for t, n, name in ((out, N, "out"), (residual, N, "residual"), (preact, wide_n, "preact")):
        if t is not None:
            _want_bf16(t, (rows, n), name)
    if bias is not None:
        _want(bias, torch.float32, "bias")
        if bias.numel() != E * wide_n:
            raise ValueError("bias must hold one value per weight row")
    name = "moe_expert_matmul_fp8"  # whose workspace is for coded results
    need = 0 if codes is None else expert_fp8_workspace_bytes(name, E, rows, K, N, act)
    cols = 1 if x_scales.dim() == 1 else x_scales.shape[1]
    _call_with_room(name, stream, workspace, need, x, x, x_scales, cols, offsets, w, w_scales, bias,
                    act, residual, E, rows, K, N, out, codes, scales, preact)


def moe_expert_matmul_fp8_dx(dy: torch.Tensor, dy_scales: torch.Tensor, offsets: torch.Tensor,
                             w_t: torch.Tensor, w_t_scales: torch.Tensor, act: int,
                             preact: torch.Tensor | None, dx: torch.Tensor | None,
                             codes: torch.Tensor | None = None, scales: torch.Tensor | None = None,
                             stream=None, workspace: torch.Tensor | None = None) -> None:
    """moe_expert_matmul_dx of E4M3 dy [rows, N] with dy_scales fp32 [rows, ceil(N /
    128)] (two halves: [rows, 2N], [rows, 2, ceil(N / 128)]) and moe_quant_weights' codes_t
    and scales_t -> dx bf16 [rows, K] ([rows, 2K] for MOE_ACT_SWIGLU), its codes with scales
    [rows, ceil(K / 128)] ([rows, 2, ceil(K / 128)]), or both; workspace as there."""
    if w_t.dim() != 3:
        raise ValueError("w_t must be [E, K, N]")
    _want_weights(w_t, offsets)
    E, K, wide_n = w_t.shape
    halves = dy_scales.shape[1] if dy_scales.dim() == 3 else 1
    if halves not in (1, 2) or wide_n % halves:
        raise ValueError("dy comes in 1 or 2 halves")
    rows, N, wide = dy.shape[0], wide_n // halves, 2 if act == MOE_ACT_SWIGLU else 1
    nbn, nbk = code_blocks(N), code_blocks(K)
    _want_codes(w_t, (E, K, wide_n), "w_t")
    _want_floats(w_t_scales, ((E, nbk, halves, nbn),) + (((E, nbk, nbn),) if halves == 1 else ()),
                 "w_t_scales")
    _want_coded(dy, dy_scales, rows, N, halves, "dy")
    _want_coded(codes, scales, rows, K, wide)
    if dx is not None:
        _want_bf16(dx, (rows, wide * K), "dx")
    if act == MOE_ACT_NONE:
        preact = None
    elif preact is None:
        raise ValueError("an activation's gradient needs preact")
    else:
        _want_bf16(preact, (rows, wide * K), "preact")
    name = "moe_expert_matmul_fp8_dx"  # whose workspace is for coded results
    need = 0 if codes is None else expert_fp8_workspace_bytes(name, E, rows, K, N, act, halves)
    _call_with_room(name, stream, workspace, need, dy, dy, dy_scales, offsets, w_t, w_t_scales,
                    halves, act, preact, E, rows, K, N, dx, codes, scales)
