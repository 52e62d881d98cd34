"""Operators on pages of grouped heads, held in 8 bits (include/hs_heads.h).

  append_heads  quantise the keys and values of new tokens into their pages, a scale for each page, head and side
  read_heads    read tokens of requests back, in 16 or 32 bits
  attend_heads  attention of grouped query heads over the pages: single tokens, verify positions, prompt chunks and prompts

A pool for kv_heads heads of head_dim has page_size 64 and row_bytes = heads_row_bytes(kv_heads, head_dim).  Thin marshalling like
the rest of the binding: no CPU fallback, every refusal of the library raises.  All tensors of a call must be on the current
device."""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import Pool, _check, lib
from .latent import _DTYPES, _I32, _empty, _here, _on, _tensor, _whole

HEADS_PAGE = 64

_i32, _i64, _p, _f = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float


class HeadsAppendC(ctypes.Structure):
    _fields_ = [("kv_heads", _i32), ("head_dim", _i32), ("dtype", _i32), ("R", _i32), ("max_pages", _i32), ("n", _i64),
                ("block_table", _p), ("ctx_len", _p), ("cu", _p), ("k", _p), ("k_token_stride", _i64),
                ("k_head_stride", _i64), ("v", _p), ("v_token_stride", _i64), ("v_head_stride", _i64), ("status", _p)]


class HeadsReadC(ctypes.Structure):
    _fields_ = [("kv_heads", _i32), ("head_dim", _i32), ("dtype", _i32), ("R", _i32), ("max_pages", _i32), ("n", _i64),
                ("block_table", _p), ("start", _p), ("cu", _p), ("k", _p), ("k_token_stride", _i64),
                ("k_head_stride", _i64), ("v", _p), ("v_token_stride", _i64), ("v_head_stride", _i64), ("status", _p)]


class HeadsAttendC(ctypes.Structure):
    _fields_ = [("kv_heads", _i32), ("head_dim", _i32), ("q_heads", _i32), ("dtype", _i32), ("causal", _i32), ("scale", _f),
                ("R", _i32), ("max_pages", _i32), ("n", _i64), ("block_table", _p), ("ctx_len", _p), ("cu_q", _p),
                ("q", _p), ("q_token_stride", _i64), ("q_head_stride", _i64), ("out", _p), ("out_token_stride", _i64),
                ("out_head_stride", _i64), ("lse", _p), ("status", _p)]


_bound = None


def _lib():
    global _bound
    if _bound is None:
        L = lib()
        L.hs_heads_row_bytes.restype = _i32
        L.hs_heads_row_bytes.argtypes = [_i32, _i32]
        L.hs_append_heads.restype = _i32
        L.hs_append_heads.argtypes = [_p, _i32, ctypes.POINTER(HeadsAppendC), _p]
        L.hs_read_heads.restype = _i32
        L.hs_read_heads.argtypes = [_p, _i32, ctypes.POINTER(HeadsReadC), _p]
        L.hs_heads_workspace_bytes.restype = ctypes.c_size_t
        L.hs_heads_workspace_bytes.argtypes = []
        L.hs_attend_heads.restype = _i32
        L.hs_attend_heads.argtypes = [_p, _i32, ctypes.POINTER(HeadsAttendC), _p, ctypes.c_size_t, _p]
        _bound = L
    return _bound


def heads_row_bytes(kv_heads: int, head_dim: int) -> int:
    """row_bytes of a pool for these heads; raises where there is none."""
    n = int(_lib().hs_heads_row_bytes(int(kv_heads), int(head_dim)))
    if n == 0:
        raise ValueError(f"no pages for {kv_heads} heads of {head_dim}: head_dim is 64 or 128, kv_heads 1 to 128")
    return n


def _pages(pool: Pool, block_table: torch.Tensor, cu, n: int, head_dim: int, dev: int) -> tuple:
    """(kv_heads, R, max_pages, table address, cu address) of a call; cu None: the n tokens fall to the requests evenly."""
    if block_table.dim() != 2:
        raise ValueError("block_table must be [requests][max_pages]")
    R, max_pages = block_table.shape
    if cu is None:
        if n % max(R, 1) or (R == 0 and n):
            raise ValueError(f"{n} tokens do not fall to {R} requests evenly: give their offsets")
    elif cu.numel() != R + 1:
        raise ValueError("the token offsets must have one entry more than there are requests")
    kv_heads = (pool.row_bytes - 16) // (2 * head_dim)
    return (kv_heads, R, max_pages, _whole(block_table, "block_table", _I32, dev),
            None if cu is None else _whole(cu, "cu", _I32, dev))


def _status(status, dev: int):
    return None if status is None else _whole(status, "status", _I32, dev)


def append_heads(pool: Pool, block_table: torch.Tensor, ctx_len: torch.Tensor, k: torch.Tensor, v: torch.Tensor, *,
                 cu: Optional[torch.Tensor] = None, layer: int = 0, status: Optional[torch.Tensor] = None,
                 stream=None) -> None:
    """Quantises the keys and values of new tokens into their pages: block_table int32 [R][max_pages], ctx_len int32 [R] (new
    tokens included), k and v [n][kv_heads][head_dim] (bf16, fp16 or fp32), cu int32 [R + 1] offsets of the requests'
    tokens in them (None: n / R each).  The new tokens are the last of each request's."""
    if k.dim() != 3:
        raise ValueError("k must be [tokens][kv_heads][head_dim]")
    n, heads, dim = k.shape
    dev = _here(k, "k")
    dt = _DTYPES.get(k.dtype)
    if dt is None:
        raise TypeError("k must be bf16, fp16 or fp32")
    sk, sv = _tensor(k, "k", (n, heads, dim), dev, k.dtype), _tensor(v, "v", (n, heads, dim), dev, k.dtype)
    if dim not in (64, 128):
        raise ValueError("head_dim must be 64 or 128")
    kv_heads, R, max_pages, table, offsets = _pages(pool, block_table, cu, n, dim, dev)
    if kv_heads != heads:
        raise ValueError(f"the pool's rows of {pool.row_bytes} bytes are not of {heads} heads of {dim}")
    a = HeadsAppendC(heads, dim, dt, R, max_pages, n, table, _whole(ctx_len, "ctx_len", _I32, dev, (R,)), offsets, k.data_ptr(),
                     sk[0], sk[1], v.data_ptr(), sv[0], sv[1], _status(status, dev))
    _check(_lib().hs_append_heads(pool.handle, int(layer), ctypes.byref(a), _on(stream, k)), "hs_append_heads")


def read_heads(pool: Pool, block_table: torch.Tensor, start: Optional[torch.Tensor], cu: Optional[torch.Tensor], tokens: int,
               head_dim: int, *, layer: int = 0, dtype: torch.dtype = torch.bfloat16, k: Optional[torch.Tensor] = None,
               v: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None, stream=None):
    """Keys and values of requests' tokens, start[r] and on (int32 [R]; None: 0), into rows cu[r] .. cu[r + 1] - 1 (int32
    [R + 1]; None: tokens / R each) of (k, v), each [tokens][kv_heads][head_dim] in dtype (bf16, fp16 or fp32, or that
    of k and v where they are given)."""
    dev = _here(block_table, "block_table")
    if k is not None or v is not None:
        dtype = (k if k is not None else v).dtype
    dt = _DTYPES.get(dtype)
    if dt is None:
        raise TypeError("k and v must be bf16, fp16 or fp32")
    if head_dim not in (64, 128):
        raise ValueError("head_dim must be 64 or 128")
    tokens = int(tokens)
    heads, R, max_pages, table, offsets = _pages(pool, block_table, cu, tokens, head_dim, dev)
    shape = (tokens, heads, head_dim)
    if k is None:
        k = _empty(shape, dtype, block_table.device, stream)
    if v is None:
        v = _empty(shape, dtype, block_table.device, stream)
    sk, sv = _tensor(k, "k", shape, dev, dtype), _tensor(v, "v", shape, dev, dtype)
    a = HeadsReadC(heads, head_dim, dt, R, max_pages, tokens, table,
                   None if start is None else _whole(start, "start", _I32, dev, (R,)), offsets, k.data_ptr(), sk[0], sk[1],
                   v.data_ptr(), sv[0], sv[1], _status(status, dev))
    _check(_lib().hs_read_heads(pool.handle, int(layer), ctypes.byref(a), _on(stream, block_table)), "hs_read_heads")
    return k, v


def heads_workspace_bytes() -> int:
    return int(_lib().hs_heads_workspace_bytes())


def alloc_heads_workspace(device="cuda") -> torch.Tensor:
    """Workspace of attend_heads, for any shape; calls that share one must be ordered on one stream."""
    with torch.cuda.device(device):
        return torch.empty(max(16, heads_workspace_bytes()), dtype=torch.uint8, device=device)


def attend_heads(pool: Pool, block_table: torch.Tensor, ctx_len: torch.Tensor, q: torch.Tensor, scale: float, *,
                 cu_q: Optional[torch.Tensor] = None, causal: bool = True, layer: int = 0,
                 out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                 status: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """Attention of query tokens over their requests' pages: block_table int32 [R][max_pages], ctx_len int32 [R], q [n][q_heads]
    [head_dim] (bf16 or fp16), cu_q int32 [R + 1] offsets of the requests' query tokens (None: n / R each) -> (out like q,
    lse fp32 [n][q_heads]).  causal: the queries are the last tokens of their contexts, else they see all of them."""
    if q.dim() != 3:
        raise ValueError("q must be [tokens][q_heads][head_dim]")
    n, q_heads, dim = q.shape
    dev = _here(q, "q")
    if q.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError("q must be bf16 or fp16")
    if dim not in (64, 128):
        raise ValueError("head_dim must be 64 or 128")
    sq = _tensor(q, "q", (n, q_heads, dim), dev, q.dtype)
    kv_heads, R, max_pages, table, offsets = _pages(pool, block_table, cu_q, n, dim, dev)
    if out is None:
        out = _empty((n, q_heads, dim), q.dtype, q.device, stream)
    so = _tensor(out, "out", (n, q_heads, dim), dev, q.dtype)
    if lse is None:
        lse = _empty((n, q_heads), torch.float32, q.device, stream)
    if workspace is None:
        workspace = _empty((max(16, heads_workspace_bytes()),), torch.uint8, q.device, stream)
    a = HeadsAttendC(kv_heads, dim, q_heads, _DTYPES[q.dtype], bool(causal), scale, R, max_pages, n, table,
                     _whole(ctx_len, "ctx_len", _I32, dev, (R,)), offsets, q.data_ptr(), sq[0], sq[1], out.data_ptr(), so[0],
                     so[1], _whole(lse, "lse", torch.float32, dev, (n, q_heads)), _status(status, dev))
    _check(_lib().hs_attend_heads(pool.handle, int(layer), ctypes.byref(a), _whole(workspace, "workspace", torch.uint8, dev),
                                  workspace.numel(), _on(stream, q)), "hs_attend_heads")
    return out, lse
