"""Python entry points of the attention layers' paged cache, with the C-ABI's names.

As in ``decode``: each function checks what the pointers cannot show (types, shapes,
strides, devices), gathers them, and calls the matching ``gdn_*`` function of libgdn on the
current stream. Where a tensor is wrong the call raises ``ValueError`` before anything is
launched; what libgdn refuses raises ``GDNError``.
"""
from __future__ import annotations

import ctypes

import torch

from . import _abi
from ._abi import Attn, PagedKV, check
from .decode import _ptr

_I2 = ctypes.c_int64 * 2
_I3 = ctypes.c_int64 * 3


def _stream(stream, beside):
    """The given stream, or the current one of the device that tensor `beside` lives on."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(beside.get_device())
    return stream if isinstance(stream, int) else stream.cuda_stream


def _want(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _ints(t, n: int, what: str, dtype=torch.int32) -> None:
    if t.dtype is not dtype or t.numel() != n or not t.is_contiguous() or not t.is_cuda:
        raise ValueError(f"{what}: contiguous {dtype} on the GPU with {n} entries, got {t.dtype} {tuple(t.shape)} "
                         f"on {t.device}")


def _table(t, batch: int) -> None:
    _want(t.dtype is torch.int32 and t.dim() == 2 and t.shape[0] == batch and t.is_contiguous() and t.is_cuda,
          "block_table: contiguous int32 [batch, max_pages] on the GPU")


def make_paged_kv(k, v=None, dv=None) -> PagedKV:
    """The cache of one layer: bf16 pages k [pages, page_size, kv heads, dk] and v [.., dv], in any
    strides whose last is 1; without v a latent cache whose value is the first dv of each key row."""
    _want(k.dtype is torch.bfloat16 and k.dim() == 4 and k.stride(3) == 1 and k.is_cuda,
          "k: bf16 [pages, page_size, heads, dk] on the GPU, its last stride 1")
    pages, page_size, heads, dk = k.shape
    kv = PagedKV()
    kv.k, kv.k_strides = k.data_ptr(), _I3(*k.stride()[:3])
    if v is None:
        _want(dv is not None, "a latent cache needs dv, the part of a row that is the value")
    else:
        _want(v.dtype is torch.bfloat16 and v.dim() == 4 and v.stride(3) == 1 and v.shape[:3] == k.shape[:3]
              and v.device == k.device, "v: bf16 [pages, page_size, heads, dv] beside k")
        _want(dv is None or dv == v.shape[3], "dv is v's last size")
        dv = v.shape[3]
        kv.v, kv.v_strides = v.data_ptr(), _I3(*v.stride()[:3])
    kv.num_pages, kv.page_size, kv.num_kv_heads, kv.dk, kv.dv = pages, page_size, heads, dk, dv
    kv._keep = (k, v)  # the struct keeps the pages alive for as long as it holds their addresses
    return kv


def kv_plan(cached_len, new_len, held, block_table, free_list, free_count, *, kv_len, cu_new, slot_map, held_out,
            free_count_out, page_size: int, num_pages: int, status=None, stream=None):
    """Pages and slots for the new tokens of a step, from the requests' lengths (new_len None: one
    token each). Writes block_table, kv_len, cu_new, slot_map, held_out and free_count_out; the
    last three of kv_len / held_out / free_count_out may be the input arrays themselves."""
    batch = cached_len.numel()
    _ints(cached_len, batch, "cached_len")
    if new_len is not None:
        _ints(new_len, batch, "new_len")
    _ints(held, batch, "held")
    _ints(kv_len, batch, "kv_len")
    _ints(held_out, batch, "held_out")
    _ints(cu_new, batch + 1, "cu_new")
    _ints(free_count, 1, "free_count")
    _ints(free_count_out, 1, "free_count_out")
    _ints(slot_map, slot_map.numel(), "slot_map", torch.int64)
    _table(block_table, batch)
    _ints(free_list, free_list.numel(), "free_list")
    _want(free_list.numel() <= num_pages, "free_list: at most num_pages entries")
    check(_abi.load().gdn_kv_plan(batch, block_table.shape[1], page_size, num_pages, slot_map.numel(),
                                  _ptr(cached_len), _ptr(new_len), _ptr(held), _ptr(block_table), _ptr(free_list),
                                  _ptr(free_count), _ptr(kv_len), _ptr(cu_new), _ptr(slot_map), _ptr(held_out),
                                  _ptr(free_count_out), _ptr(status), _stream(stream, cached_len)), "gdn_kv_plan")


def kv_release(requests, held, block_table, free_list, free_count, *, status=None, stream=None):
    """Pushes the pages of the given requests (rows of block_table) on free_list, which has room for
    every page of the cache; held of those rows becomes 0 and free_count grows."""
    batch = held.numel()
    _ints(requests, requests.numel(), "requests")
    _ints(held, batch, "held")
    _ints(free_count, 1, "free_count")
    _ints(free_list, free_list.numel(), "free_list")
    _table(block_table, batch)
    check(_abi.load().gdn_kv_release(batch, block_table.shape[1], free_list.numel(), _ptr(requests),
                                     requests.numel(), _ptr(block_table), _ptr(held), _ptr(free_list),
                                     _ptr(free_count), _ptr(status), _stream(stream, held)), "gdn_kv_release")


def kv_append(kv: PagedKV, k, v, slot_map, *, status=None, stream=None):
    """Rows of new tokens to their slots: k [n, heads, dk] and v [n, heads, dv]; for a latent cache the
    latent part [n, 1, dv] and the tail [n, 1, dk - dv] (None if dk == dv). bf16 or fp32."""
    latent = kv.v is None
    n, heads = slot_map.numel(), kv.num_kv_heads
    tail = kv.dk - kv.dv if latent else kv.dv
    _ints(slot_map, n, "slot_map", torch.int64)
    _want(k.dtype in (torch.bfloat16, torch.float32) and k.shape == (n, heads, kv.dv if latent else kv.dk)
          and k.stride(2) == 1 and k.is_cuda, "k: bf16 or fp32 [n, heads, size] on the GPU, its last stride 1")
    v_strides = None
    if tail:
        _want(v is not None and v.dtype is k.dtype and v.shape == (n, heads, tail) and v.stride(2) == 1
              and v.is_cuda, "v: of k's type [n, heads, size], its last stride 1")
        v_strides = _I2(v.stride(0), v.stride(1))
    check(_abi.load().gdn_kv_append(kv, n, k.data_ptr(), _I2(k.stride(0), k.stride(1)), _ptr(v) if tail else None,
                                    v_strides, slot_map.data_ptr(),
                                    _abi.QKV_BF16 if k.dtype is torch.bfloat16 else 0, _ptr(status),
                                    _stream(stream, k)), "gdn_kv_append")


def attn_workspace_bytes(kv: PagedKV, batch: int, num_tokens: int, num_heads: int) -> int:
    """Bytes of workspace that attn_decode / latent_decode need."""
    out = ctypes.c_size_t()
    check(_abi.load().gdn_attn_workspace(kv, batch, num_tokens, num_heads, out), "gdn_attn_workspace")
    return out.value


def _attend(name, kv, q, block_table, kv_len, o, workspace, lse, scale, window, status, stream):
    _want(q.dtype is torch.bfloat16 and q.dim() == 4 and q.shape[3] == kv.dk and q.stride(3) == 1 and q.is_cuda,
          "q: bf16 [batch, tokens, heads, dk] on the GPU, its last stride 1")
    batch, tokens, heads, dk = q.shape
    _want(o.dtype is torch.bfloat16 and o.shape == (batch, tokens, heads, kv.dv) and o.is_contiguous() and o.is_cuda,
          "o: contiguous bf16 [batch, tokens, heads, dv] on the GPU")
    _want(lse is None or (lse.dtype is torch.float32 and lse.shape == (batch, tokens, heads) and lse.is_contiguous()
                            and lse.is_cuda), "lse: contiguous fp32 [batch, tokens, heads] on the GPU")
    _want(workspace.is_cuda and workspace.is_contiguous(), "workspace: contiguous, on the GPU")
    _table(block_table, batch)
    _ints(kv_len, batch, "kv_len")
    s = q.stride()
    a = Attn(batch, tokens, heads, block_table.shape[1], window, dk ** -0.5 if scale is None else scale, q.data_ptr(),
             _I3(s[0], s[1], s[2]), block_table.data_ptr(), kv_len.data_ptr(), o.data_ptr(), _ptr(lse))
    check(getattr(_abi.load(), name)(kv, a, workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                     _ptr(status), _stream(stream, q)), name)


def attn_decode(kv: PagedKV, q, block_table, kv_len, o, workspace, *, lse=None, scale=None, window=0, status=None,
                stream=None):
    """Attention of the newest T positions of every request (q [B, T, H, dk]) over its pages;
    o [B, T, H, dv], lse [B, T, H]. scale None: dk ** -0.5; window 0: the whole request."""
    _attend("gdn_attn_decode", kv, q, block_table, kv_len, o, workspace, lse, scale, window, status, stream)


def latent_decode(kv: PagedKV, q, block_table, kv_len, o, workspace, *, lse=None, scale=None, window=0, status=None,
                  stream=None):
    """The same over a latent cache (one shared row a token; absorbed queries of dk elements)."""
    _attend("gdn_latent_decode", kv, q, block_table, kv_len, o, workspace, lse, scale, window, status, stream)
