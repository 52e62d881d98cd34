"""Operators on the latent rows of the paged KV pool (include/hs_latent.h).

  append_rows      write the rows of new tokens (rotation + quantisation + store, one launch)
  read_rows        read rows back by id, in 16 or 32 bits
  attend_rows      absorbed latent attention over row ids (resolve_topk's out_rows)
  attend_pages     absorbed latent attention over whole contexts through a block table
  attend_expanded  attention over keys and values expanded to every head (prompts)

Thin marshalling like the rest of the binding: no CPU fallback, every refusal of the library raises.  All tensors of a call
must be on the current device."""
from __future__ import annotations

import ctypes
from typing import Optional

import torch

from . import Pool, _check, lib

LATENT_DIM, ROPE_DIM, NOPE_DIM, VALUE_DIM = 512, 64, 128, 128
ROW_BYTES_FP8, ROW_BYTES_BF16 = 656, 1152
_I32 = torch.int32
_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}

_i32, _i64, _p, _f = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_float


class AppendC(ctypes.Structure):
    _fields_ = [("n", _i64), ("rows", _p), ("positions", _p), ("rotation", _p), ("num_positions", _i32),
                ("interleaved", _i32), ("dtype", _i32), ("heads", _i32), ("latent", _p), ("latent_stride", _i64),
                ("rope", _p), ("rope_stride", _i64), ("q_rope", _p), ("q_token_stride", _i64), ("q_head_stride", _i64),
                ("q_out", _p), ("q_out_token_stride", _i64), ("q_out_head_stride", _i64), ("status", _p)]


class ReadLatentC(ctypes.Structure):
    _fields_ = [("n", _i64), ("rows", _p), ("dtype", _i32), ("latent", _p), ("latent_stride", _i64), ("rope", _p),
                ("rope_stride", _i64), ("status", _p)]


class AttendC(ctypes.Structure):
    _fields_ = [("heads", _i32), ("scale", _f), ("q_latent", _p), ("ql_token_stride", _i64), ("ql_head_stride", _i64),
                ("q_rope", _p), ("qr_token_stride", _i64), ("qr_head_stride", _i64), ("out", _p),
                ("out_token_stride", _i64), ("out_head_stride", _i64), ("lse", _p), ("status", _p)]


class ExpandedC(ctypes.Structure):
    _fields_ = [("seqs", _i32), ("heads", _i32), ("causal", _i32), ("scale", _f), ("q_tokens", _i64),
                ("k_tokens", _i64), ("cu_q", _p), ("cu_k", _p), ("q_nope", _p), ("qn_token_stride", _i64),
                ("qn_head_stride", _i64), ("q_rope", _p), ("qr_token_stride", _i64), ("qr_head_stride", _i64),
                ("k_nope", _p), ("kn_token_stride", _i64), ("kn_head_stride", _i64), ("k_rope", _p),
                ("kr_token_stride", _i64), ("v", _p), ("v_token_stride", _i64), ("v_head_stride", _i64), ("out", _p),
                ("out_token_stride", _i64), ("out_head_stride", _i64), ("lse", _p), ("status", _p)]


_bound = None


def _lib():
    global _bound
    if _bound is None:
        L = lib()
        L.hs_append_rows.restype = _i32
        L.hs_append_rows.argtypes = [_p, _i32, ctypes.POINTER(AppendC), _p]
        L.hs_read_rows.restype = _i32
        L.hs_read_rows.argtypes = [_p, _i32, ctypes.POINTER(ReadLatentC), _p]
        L.hs_attend_workspace_bytes.restype = ctypes.c_size_t
        L.hs_attend_workspace_bytes.argtypes = []
        L.hs_attend_rows.restype = _i32
        L.hs_attend_rows.argtypes = [_p, _i32, _p, _i64, _i32, ctypes.POINTER(AttendC), _p, ctypes.c_size_t, _p]
        L.hs_attend_pages.restype = _i32
        L.hs_attend_pages.argtypes = [_p, _i32, _p, _p, _i32, _i32, _i32, ctypes.POINTER(AttendC), _p, ctypes.c_size_t, _p]
        L.hs_attend_expanded.restype = _i32
        L.hs_attend_expanded.argtypes = [ctypes.POINTER(ExpandedC), _p]
        _bound = L
    return _bound


_current_device = torch._C._cuda_getDevice


def _here(t: torch.Tensor, name: str) -> int:
    """The device that all of a call's tensors must be on: that of its first one, which must be the current device (the
    kernels are launched there)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    dev = t.get_device()
    if dev != _current_device():
        raise ValueError(f"{name} is on device {dev}, but device {_current_device()} is current")
    return dev


def _refuse(t, name: str, dev: int, dtype):
    """Raises what is wrong with the type or the device of a tensor, if it is one of these."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or not t.is_cuda:
        raise TypeError(f"{name} must be a {dtype} CUDA tensor")
    if t.get_device() != dev:
        raise ValueError(f"{name} is on device {t.get_device()}, not on device {dev} with the other tensors")


def _tensor(t: torch.Tensor, name: str, shape: tuple, dev: int, dtype=torch.bfloat16) -> tuple:
    """The strides of a tensor of this shape, type and device whose last dimension is contiguous."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != dev:
        _refuse(t, name, dev, dtype)
        raise ValueError(f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    strides = t.stride()
    if strides[-1] != 1 and t.numel():
        raise ValueError(f"{name}'s last dimension must be contiguous")
    return strides


def _whole(t: torch.Tensor, name: str, dtype, dev: int, shape=None) -> int:
    """The address of a contiguous tensor of this type and device (and shape)."""
    if t.dtype is not dtype or t.get_device() != dev or not t.is_contiguous() or (shape is not None and t.shape != shape):
        _refuse(t, name, dev, dtype)
        raise TypeError(f"{name} must be contiguous" + (f" and have shape {tuple(shape)}" if shape is not None else ""))
    return t.data_ptr()


def _on(stream, t: torch.Tensor):
    """The raw stream to launch on: the given one, or the current one of the tensor's device."""
    return stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(t.get_device())


def _empty(shape: tuple, dtype, device, stream) -> torch.Tensor:
    """An output or workspace made here belongs to the stream that the call launches on: memory of another stream could
    still be in use there, or be handed out again before this call's kernels are done with it."""
    if isinstance(stream, torch.cuda.Stream):
        with torch.cuda.stream(stream):
            return torch.empty(shape, dtype=dtype, device=device)
    return torch.empty(shape, dtype=dtype, device=device)


def append_rows(pool: Pool, rows: torch.Tensor, latent: torch.Tensor, rope: torch.Tensor, positions: torch.Tensor,
                rotation: torch.Tensor, *, layer: int = 0, q_rope: Optional[torch.Tensor] = None,
                q_out: Optional[torch.Tensor] = None, interleaved: bool = False,
                status: Optional[torch.Tensor] = None, stream=None) -> Optional[torch.Tensor]:
    """Writes the pool rows of n new tokens of one layer: rows int32 [n] (-1: none), latent [n][512], rope
    [n][64] (not yet rotated), positions int32 [n], rotation fp32 [num_positions][64] (32 cosines, 32 sines).
    q_rope [n][heads][64], of the same type, is rotated into q_out (a new tensor, or q_rope itself) in the
    same launch; returns q_out.  latent, rope and q_rope share a type: bf16, fp16 or fp32."""
    n = int(rows.numel())
    dt = _DTYPES.get(latent.dtype)
    if dt is None:
        raise TypeError("latent must be bf16, fp16 or fp32")
    dtype = latent.dtype
    dev = _here(latent, "latent")
    latent_stride = _tensor(latent, "latent", (n, LATENT_DIM), dev, dtype)[0]
    rope_stride = _tensor(rope, "rope", (n, ROPE_DIM), dev, dtype)[0]
    if positions.numel() != n:
        raise ValueError("positions must have one entry per row")
    if rotation.dim() != 2 or rotation.shape[1] != ROPE_DIM:
        raise ValueError("rotation must be [num_positions][64]")
    heads, q, qo = 0, (None, 0, 0), (None, 0, 0)
    if q_rope is not None:
        heads = int(q_rope.shape[1]) if q_rope.dim() == 3 else -1
        st = _tensor(q_rope, "q_rope", (n, heads, ROPE_DIM), dev, dtype)
        q = (q_rope.data_ptr(), st[0], st[1])
        if q_out is None:
            q_out = _empty((n, heads, ROPE_DIM), dtype, q_rope.device, stream)
        st = _tensor(q_out, "q_out", (n, heads, ROPE_DIM), dev, dtype)
        qo = (q_out.data_ptr(), st[0], st[1])
    elif q_out is not None:
        raise ValueError("q_out without q_rope")
    a = AppendC(n, _whole(rows, "rows", _I32, dev), _whole(positions, "positions", _I32, dev),
                _whole(rotation, "rotation", torch.float32, dev), rotation.shape[0], bool(interleaved), dt, heads,
                latent.data_ptr(), latent_stride, rope.data_ptr(), rope_stride, *q, *qo,
                status if status is None else _whole(status, "status", _I32, dev))
    _check(_lib().hs_append_rows(pool.handle, int(layer), ctypes.byref(a), _on(stream, latent)), "hs_append_rows")
    return q_out


def read_rows(pool: Pool, rows: torch.Tensor, *, layer: int = 0, dtype: torch.dtype = torch.bfloat16,
              latent: Optional[torch.Tensor] = None, rope: Optional[torch.Tensor] = None,
              status: Optional[torch.Tensor] = None, stream=None):
    """The latents and rotated keys of pool rows: rows int32 [n] (-1: zeros) -> (latent [n][512], rope [n][64]) in dtype:
    bf16, fp16 or fp32, or that of latent and rope where they are given."""
    n = int(rows.numel())
    dev = _here(rows, "rows")
    if latent is not None or rope is not None:
        dtype = (latent if latent is not None else rope).dtype
    dt = _DTYPES.get(dtype)
    if dt is None:
        raise TypeError("latent and rope must be bf16, fp16 or fp32")
    if latent is None:
        latent = _empty((n, LATENT_DIM), dtype, rows.device, stream)
    if rope is None:
        rope = _empty((n, ROPE_DIM), dtype, rows.device, stream)
    a = ReadLatentC(n, _whole(rows, "rows", _I32, dev), dt, latent.data_ptr(), _tensor(latent, "latent", (n, LATENT_DIM), dev, dtype)[0],
                    rope.data_ptr(), _tensor(rope, "rope", (n, ROPE_DIM), dev, dtype)[0],
                    status if status is None else _whole(status, "status", _I32, dev))
    _check(_lib().hs_read_rows(pool.handle, int(layer), ctypes.byref(a), _on(stream, rows)), "hs_read_rows")
    return latent, rope


def attend_workspace_bytes() -> int:
    return int(_lib().hs_attend_workspace_bytes())


def alloc_attend_workspace(device="cuda") -> torch.Tensor:
    """Workspace of attend_rows and attend_pages, for any shape; calls that share one must be ordered on one
    stream."""
    with torch.cuda.device(device):
        return torch.empty(max(16, attend_workspace_bytes()), dtype=torch.uint8, device=device)


def _attend(lead: tuple, q_latent, q_rope, scale, out, lse, status, workspace, stream):
    """Marshals an absorbed call whose query tensors have the leading dimensions `lead` (tokens) and heads."""
    k = len(lead)
    heads = q_latent.shape[k] if q_latent.dim() == k + 2 else -1
    dev = _here(q_latent, "q_latent")
    shape, device = (*lead, heads, LATENT_DIM), q_latent.device
    sl = _tensor(q_latent, "q_latent", shape, dev)
    sr = _tensor(q_rope, "q_rope", (*lead, heads, ROPE_DIM), dev)
    if out is None:
        out = _empty(shape, torch.bfloat16, device, stream)
    so = _tensor(out, "out", shape, dev)
    if lse is None:
        lse = _empty((*lead, heads), torch.float32, device, stream)
    if workspace is None:
        workspace = _empty((max(16, attend_workspace_bytes()),), torch.uint8, device, stream)
    ws = (_whole(workspace, "workspace", torch.uint8, dev), workspace.numel())
    token = (sl[0], sr[0], so[0])
    if k == 2 and lead[1] > 1:  # [requests][positions]: the two must merge into one dimension of tokens
        if lead[0] > 1 and (sl[0] != lead[1] * sl[1] or sr[0] != lead[1] * sr[1] or so[0] != lead[1] * so[1]):
            raise ValueError("the two leading dimensions of q_latent, q_rope and out must merge into one")
        token = (sl[1], sr[1], so[1])
    a = AttendC(heads, scale, q_latent.data_ptr(), token[0], sl[k], q_rope.data_ptr(), token[1], sr[k], out.data_ptr(),
                token[2], so[k], _whole(lse, "lse", torch.float32, dev, (*lead, heads)),
                status if status is None else _whole(status, "status", _I32, dev))
    return a, out, lse, ws, dev


def attend_rows(pool: Pool, rows: torch.Tensor, q_latent: torch.Tensor, q_rope: torch.Tensor, scale: float, *,
                layer: int = 0, out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                status: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """Absorbed attention of n query tokens over their own rows: rows int32 [n][K] (-1: skipped), q_latent bf16
    [n][heads][512], q_rope bf16 [n][heads][64] (rotated) -> (out bf16 [n][heads][512], lse fp32 [n][heads])."""
    if rows.dim() != 2:
        raise ValueError("rows must be [tokens][K]")
    n, K = rows.shape
    a, out, lse, ws, dev = _attend((n,), q_latent, q_rope, scale, out, lse, status, workspace, stream)
    _check(_lib().hs_attend_rows(pool.handle, int(layer), _whole(rows, "rows", _I32, dev), n, K, ctypes.byref(a),
                                 *ws, _on(stream, q_latent)), "hs_attend_rows")
    return out, lse


def attend_pages(pool: Pool, block_table: torch.Tensor, ctx_len: torch.Tensor, q_latent: torch.Tensor,
                 q_rope: torch.Tensor, scale: float, *, layer: int = 0, out: Optional[torch.Tensor] = None,
                 lse: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None, stream=None):
    """Absorbed attention over whole contexts: block_table int32 [R][max_pages], ctx_len int32 [R], q_latent bf16
    [R][P][heads][512], q_rope bf16 [R][P][heads][64]; position p of request r sees its first
    ctx_len[r] - P + 1 + p tokens -> (out bf16 [R][P][heads][512], lse fp32 [R][P][heads])."""
    if q_latent.dim() != 4 or block_table.dim() != 2:
        raise ValueError("q_latent must be [R][P][heads][512] and block_table [R][max_pages]")
    R, P = int(q_latent.shape[0]), int(q_latent.shape[1])
    if block_table.shape[0] != R or ctx_len.numel() != R:
        raise ValueError("block_table and ctx_len must have one entry per request")
    a, out, lse, ws, dev = _attend((R, P), q_latent, q_rope, scale, out, lse, status, workspace, stream)
    _check(_lib().hs_attend_pages(pool.handle, int(layer), _whole(block_table, "block_table", _I32, dev),
                                  _whole(ctx_len, "ctx_len", _I32, dev), R, P, int(block_table.shape[1]), ctypes.byref(a),
                                  *ws, _on(stream, q_latent)), "hs_attend_pages")
    return out, lse


def attend_expanded(q_nope: torch.Tensor, q_rope: torch.Tensor, k_nope: torch.Tensor, k_rope: torch.Tensor,
                    v: torch.Tensor, cu_q: torch.Tensor, cu_k: torch.Tensor, scale: float, *, causal: bool = True,
                    out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                    status: Optional[torch.Tensor] = None, stream=None):
    """Attention of ragged sequences over expanded keys and values: q_nope bf16 [Tq][heads][128], q_rope bf16
    [Tq][heads][64] and k_rope bf16 [Tk][64] (rotated; the key part is shared by the heads), k_nope and v bf16
    [Tk][heads][128], cu_q and cu_k int32 [seqs + 1] -> (out bf16 [Tq][heads][128], lse fp32 [Tq][heads]).
    causal: the queries are the last tokens of their sequence."""
    if q_nope.dim() != 3 or k_rope.dim() != 2:
        raise ValueError("q_nope must be [Tq][heads][128] and k_rope [Tk][64]")
    Tq, H, Tk = int(q_nope.shape[0]), int(q_nope.shape[1]), int(k_rope.shape[0])
    dev = _here(q_nope, "q_nope")
    sqn = _tensor(q_nope, "q_nope", (Tq, H, NOPE_DIM), dev)
    sqr = _tensor(q_rope, "q_rope", (Tq, H, ROPE_DIM), dev)
    skn = _tensor(k_nope, "k_nope", (Tk, H, NOPE_DIM), dev)
    skr = _tensor(k_rope, "k_rope", (Tk, ROPE_DIM), dev)
    sv = _tensor(v, "v", (Tk, H, VALUE_DIM), dev)
    if cu_q.numel() < 1 or cu_q.numel() != cu_k.numel():
        raise ValueError("cu_q and cu_k must both have one entry more than there are sequences")
    if out is None:
        out = _empty((Tq, H, VALUE_DIM), torch.bfloat16, q_nope.device, stream)
    so = _tensor(out, "out", (Tq, H, VALUE_DIM), dev)
    if lse is None:
        lse = _empty((Tq, H), torch.float32, q_nope.device, stream)
    a = ExpandedC(cu_q.numel() - 1, H, bool(causal), scale, Tq, Tk, _whole(cu_q, "cu_q", _I32, dev),
                  _whole(cu_k, "cu_k", _I32, dev),
                  q_nope.data_ptr(), sqn[0], sqn[1], q_rope.data_ptr(), sqr[0], sqr[1], k_nope.data_ptr(), skn[0], skn[1],
                  k_rope.data_ptr(), skr[0], v.data_ptr(), sv[0], sv[1], out.data_ptr(), so[0], so[1],
                  _whole(lse, "lse", torch.float32, dev, (Tq, H)),
                  status if status is None else _whole(status, "status", _I32, dev))
    _check(_lib().hs_attend_expanded(ctypes.byref(a), _on(stream, q_nope)), "hs_attend_expanded")
    return out, lse
