"""Python entry points of the attention layers' paged cache, with the C-ABI's names.

As in ``decode``: each function checks what the pointers cannot show (types, shapes,
strides, devices), gathers them, and calls the matching ``gdn_*`` function of libgdn on the
current stream. All tensors of a call live on the current device, on which libgdn launches. Where
a tensor is wrong the call raises ``ValueError`` before anything is launched; what libgdn refuses
raises ``GDNError``.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import _abi
from ._abi import GDN_OK, check

# A decode step makes one call a layer, so what these functions spend before the launch counts:
# conditions are written out (no helper call for each), and the C structs are packed in one go.
_pack_kv = struct.Struct("=QQ6q5i4x").pack       # gdn_paged_kv
_pack_attn = struct.Struct("=5if4q4Q").pack      # gdn_attn
_pack_strides = struct.Struct("=2q").pack
_BF16, _FP32, _I32, _I64 = torch.bfloat16, torch.float32, torch.int32, torch.int64
# absent where torch has no CUDA
_raw_stream, _current_device = (getattr(torch._C, name, None) for name in ("_cuda_getCurrentRawStream", "_cuda_getDevice"))


class PagedKV:
    """The cache of one layer, as make_paged_kv() describes it to the calls; it keeps its pages alive."""

    __slots__ = ("packed", "dk", "dv", "heads", "latent", "device", "k", "v")

    def __init__(self, packed, dk, dv, heads, latent, k, v):
        self.packed, self.dk, self.dv, self.heads, self.latent, self.k, self.v = packed, dk, dv, heads, latent, k, v
        self.device = k.get_device()


def _not_here(device: int, what: str):
    """The error of tensors that are not on the current device (get_device() is -1 on the host)."""
    got = "the host" if device < 0 else f"cuda:{device}"
    return ValueError(f"{what}: on the GPU that is the current device, got {got}")


def _status(t, device: int):
    if t.dtype is not _I32 or t.numel() < 1 or t.get_device() != device:
        raise ValueError(f"status: int32 on the GPU beside the others, got {t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _stream(stream, device: int):
    """The given stream, or the current one."""
    if stream is None:
        return _raw_stream(device)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _ints(t, n: int, what: str, device: int, dtype=_I32) -> int:
    if t.dtype is not dtype or t.numel() != n or not t.is_contiguous() or t.get_device() != device:
        raise ValueError(f"{what}: contiguous {dtype} on the GPU beside the others with {n} entries, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _table(t, batch: int, device: int) -> int:
    shape = t.shape
    if t.dtype is not _I32 or len(shape) != 2 or shape[0] != batch or not t.is_contiguous() or t.get_device() != device:
        raise ValueError("block_table: contiguous int32 [batch, max_pages] on the GPU beside the others")
    return shape[1]


def make_paged_kv(k, v=None, dv=None) -> PagedKV:
    """The cache of one layer: bf16 pages k [pages, page_size, kv heads, dk] and v [.., dv], in any
    strides whose last is 1; without v a latent cache whose value is the first dv of each key row."""
    if k.dtype is not _BF16 or k.dim() != 4 or k.stride(3) != 1 or not k.is_cuda:
        raise ValueError("k: bf16 [pages, page_size, heads, dk] on the GPU, its last stride 1")
    pages, page_size, heads, dk = k.shape
    k0, k1, k2, _ = k.stride()
    if v is None:
        if dv is None:
            raise ValueError("a latent cache needs dv, the part of a row that is the value")
        packed = _pack_kv(k.data_ptr(), 0, k0, k1, k2, 0, 0, 0, pages, page_size, heads, dk, dv)
        return PagedKV(packed, dk, dv, heads, True, k, None)
    if v.dtype is not _BF16 or v.dim() != 4 or v.stride(3) != 1 or v.device != k.device:
        raise ValueError("v: bf16 [pages, page_size, heads, dv] beside k, its last stride 1")
    v_pages, v_size, v_heads, size = v.shape
    if v_pages != pages or v_size != page_size or v_heads != heads or (dv is not None and dv != size):
        raise ValueError("v: as many pages, positions and heads as k; dv is its last size")
    v0, v1, v2, _ = v.stride()
    packed = _pack_kv(k.data_ptr(), v.data_ptr(), k0, k1, k2, v0, v1, v2, pages, page_size, heads, dk, size)
    return PagedKV(packed, dk, size, heads, False, k, v)


def kv_plan(cached_len, new_len, held, block_table, free_list, free_count, *, kv_len, cu_new, slot_map, held_out,
            free_count_out, page_size: int, num_pages: int, status=None, stream=None):
    """Pages and slots for the new tokens of a step, from the requests' lengths (new_len None: one
    token each). Writes block_table, kv_len, cu_new, slot_map, held_out and free_count_out; kv_len,
    held_out and free_count_out may be cached_len, held and free_count themselves. A cached length of
    LEN_PADDING marks a row that takes no part and stays so; -1 does for one step only. An empty
    batch is no call: nothing is written."""
    batch, capacity, free = cached_len.numel(), slot_map.numel(), free_list.numel()
    at = cached_len.get_device()
    if at < 0 or at != _current_device():
        raise _not_here(at, "cached_len")
    cached = _ints(cached_len, batch, "cached_len", at)
    check(_abi.load().gdn_kv_plan(
        batch, _table(block_table, batch, at), page_size, num_pages, free, capacity, cached,
        None if new_len is None else _ints(new_len, batch, "new_len", at), _ints(held, batch, "held", at),
        block_table.data_ptr(), _ints(free_list, free, "free_list", at), _ints(free_count, 1, "free_count", at),
        _ints(kv_len, batch, "kv_len", at), _ints(cu_new, batch + 1, "cu_new", at),
        _ints(slot_map, capacity, "slot_map", at, _I64), _ints(held_out, batch, "held_out", at),
        _ints(free_count_out, 1, "free_count_out", at), None if status is None else _status(status, at),
        _stream(stream, at)), "gdn_kv_plan")


def kv_release(requests, held, block_table, free_list, free_count, *, status=None, stream=None):
    """Pushes the pages of the given requests (rows of block_table) on free_list, which has room for
    every page of the cache; held of those rows becomes 0 and free_count grows."""
    batch, n, free = held.numel(), requests.numel(), free_list.numel()
    at = requests.get_device()
    if at < 0 or at != _current_device():
        raise _not_here(at, "requests")
    finished = _ints(requests, n, "requests", at)
    check(_abi.load().gdn_kv_release(
        batch, _table(block_table, batch, at), free, finished, n, block_table.data_ptr(),
        _ints(held, batch, "held", at), _ints(free_list, free, "free_list", at), _ints(free_count, 1, "free_count", at),
        None if status is None else _status(status, at), _stream(stream, at)), "gdn_kv_release")


def kv_append(kv: PagedKV, k, v, slot_map, *, status=None, stream=None):
    """Rows of new tokens to their slots: k [n, heads, dk] and v [n, heads, dv]; for a latent cache the
    latent part [n, 1, dv] and the tail [n, 1, dk - dv] (None if dk == dv). bf16 or fp32."""
    n, heads, dv, dtype = slot_map.numel(), kv.heads, kv.dv, k.dtype
    width, tail = (dv, kv.dk - dv) if kv.latent else (kv.dk, dv)
    at = kv.device
    if at < 0 or at != _current_device():
        raise _not_here(at, "the pages")
    slots = _ints(slot_map, n, "slot_map", at, _I64)
    k_row, k_head, k_last = k.stride() if k.dim() == 3 else (0, 0, 0)
    if k_last != 1 or (dtype is not _BF16 and dtype is not _FP32) or k.shape != (n, heads, width) or k.get_device() != at:
        raise ValueError(f"k: bf16 or fp32 [{n}, {heads}, {width}] on the GPU beside the pages, its last stride 1")
    v_ptr = v_strides = None
    if tail:
        if v is None or v.dtype is not dtype or v.shape != (n, heads, tail) or v.get_device() != at or v.stride(2) != 1:
            raise ValueError(f"v: of k's type [{n}, {heads}, {tail}] on the GPU beside the pages, its last stride 1")
        v_row, v_head, _ = v.stride()
        v_ptr, v_strides = v.data_ptr(), _pack_strides(v_row, v_head)
    check(_abi.load().gdn_kv_append(kv.packed, n, k.data_ptr(), _pack_strides(k_row, k_head), v_ptr, v_strides, slots,
                                    1 if dtype is _BF16 else 0, None if status is None else _status(status, at),
                                    _stream(stream, at)), "gdn_kv_append")


def attn_workspace_bytes(kv: PagedKV, batch: int, num_tokens: int, num_heads: int) -> int:
    """Bytes of workspace that attn_decode / latent_decode need."""
    out = ctypes.c_size_t()
    check(_abi.load().gdn_attn_workspace(kv.packed, batch, num_tokens, num_heads, ctypes.byref(out)), "gdn_attn_workspace")
    return out.value


def _attend(call, name, kv, q, block_table, kv_len, o, workspace, lse, scale, window, status, stream):
    at = kv.device
    if at < 0 or at != _current_device():
        raise _not_here(at, "the pages")
    if q.dtype is not _BF16 or q.dim() != 4 or q.get_device() != at:
        raise ValueError("q: bf16 [batch, tokens, heads, dk] on the GPU beside the pages")
    batch, tokens, heads, dk = q.shape
    s0, s1, s2, s3 = q.stride()
    if dk != kv.dk or s3 != 1:
        raise ValueError("q: heads of dk elements, its last stride 1")
    if o.dtype is not _BF16 or o.shape != (batch, tokens, heads, kv.dv) or not o.is_contiguous() or o.get_device() != at:
        raise ValueError("o: contiguous bf16 [batch, tokens, heads, dv] on the GPU beside the pages")
    if lse is not None and (lse.dtype is not _FP32 or lse.shape != (batch, tokens, heads) or not lse.is_contiguous()
                            or lse.get_device() != at):
        raise ValueError("lse: contiguous fp32 [batch, tokens, heads] on the GPU beside the pages")
    if workspace.get_device() != at or not workspace.is_contiguous():
        raise ValueError("workspace: contiguous, on the GPU beside the pages")
    a = _pack_attn(batch, tokens, heads, _table(block_table, batch, at), window, dk ** -0.5 if scale is None else scale,
                   q.data_ptr(), s0, s1, s2, block_table.data_ptr(), _ints(kv_len, batch, "kv_len", at), o.data_ptr(),
                   0 if lse is None else lse.data_ptr())
    rc = call(kv.packed, a, workspace.data_ptr(), workspace.nbytes, None if status is None else _status(status, at),
              _stream(stream, at))
    if rc != GDN_OK:
        check(rc, name)


def attn_decode(kv: PagedKV, q, block_table, kv_len, o, workspace, *, lse=None, scale=None, window=0, status=None,
                stream=None):
    """Attention of the newest T positions of every request (q [B, T, H, dk]) over its pages;
    o [B, T, H, dv], lse [B, T, H]. scale None: dk ** -0.5; window 0: the whole request."""
    _attend(_abi.load().gdn_attn_decode, "gdn_attn_decode", kv, q, block_table, kv_len, o, workspace, lse, scale, window, status, stream)


def latent_decode(kv: PagedKV, q, block_table, kv_len, o, workspace, *, lse=None, scale=None, window=0, status=None,
                  stream=None):
    """The same over a latent cache (one shared row a token; absorbed queries of dk elements)."""
    _attend(_abi.load().gdn_latent_decode, "gdn_latent_decode", kv, q, block_table, kv_len, o, workspace, lse, scale, window, status, stream)
