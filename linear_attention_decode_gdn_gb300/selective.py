"""Python entry points of selective state space layers, with the C-ABI's names.

As in ``paged``: each function checks what the pointers cannot show (types, shapes, strides,
devices), packs them into the C struct and calls the matching ``gdn_*`` function of libgdn on the
current stream. All tensors of a call live on the current device. Where a tensor is wrong the call
raises ``ValueError`` before anything is launched; what libgdn refuses raises ``GDNError``: outputs
that overlap inputs among it, but for o in place of x (norm) and y in place of u, dt or z (scan, step).
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import _abi
from ._abi import GDN_OK, check
from .paged import _current_device, _ints, _not_here, _status, _stream

_pack_norm = struct.Struct("=6if4xQqQqQQQ").pack        # gdn_norm
_pack_conv = struct.Struct("=4iI4xQ2q6Q").pack          # gdn_conv
_pack_ssm = struct.Struct("=6iI4xQ2qQ2qQ3qQ3qQ2q7Q").pack  # gdn_ssm
_BF16, _FP32, _E4M3 = torch.bfloat16, torch.float32, torch.float8_e4m3fn
_TYPES = {_BF16: _abi.TYPE_BF16, _FP32: _abi.TYPE_FP32, _E4M3: _abi.TYPE_E4M3}


def _rows(t, shape, dtype, what: str, device: int):
    """Address and leading strides of an operand whose last dimension is contiguous."""
    strides = t.stride()
    if t.dtype is not dtype or t.shape != shape or strides[-1] != 1 or t.get_device() != device:
        raise ValueError(f"{what}: {dtype} {tuple(shape)} on the GPU beside the others, its last stride 1, got {t.dtype} "
                         f"{tuple(t.shape)} in strides {tuple(strides)} on {t.device}")
    return t.data_ptr(), *strides[:-1]


def _whole(t, shape, dtype, what: str, device: int) -> int:
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.get_device() != device:
        raise ValueError(f"{what}: contiguous {dtype} {tuple(shape)} on the GPU beside the others, got {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    return t.data_ptr()


# A decode step makes one call a layer: conditions are written out, as in ``paged``, and gone through
# again one by one only for the error of a call that they refuse.
def _refuse(at, x, what, dims, wide, whole):
    """Raises the error of what a call found wrong: x is its first operand, `wide` the others of its kind,
    `whole` those that are contiguous."""
    if at < 0 or at != _current_device():
        raise _not_here(at, what)
    if (x.dtype is not _BF16 and x.dtype is not _FP32) or x.dim() not in dims:
        raise ValueError(f"{what}: bf16 or fp32, with {' or '.join(map(str, dims))} dimensions, got {x.dtype} {tuple(x.shape)}")
    for t, shape, dtype, name in ((x, x.shape, x.dtype, what), *wide):
        if t is not None:
            _rows(t, shape, dtype, name, at)
    for t, shape, dtype, name in whole:
        if t is not None:
            _whole(t, shape, dtype, name, at)
    raise ValueError("tensors of other types, shapes, strides or devices than the call takes")


def add_rms_norm(x, o, *, residual=None, weight=None, eps=1e-6, scales=None, group=0, stream=None):
    """residual += x, and o = RMSNorm of that sum (of x without a residual) times weight [width]. x, residual
    [rows, width] bf16 or fp32, in rows of any distance; o [rows, width] bf16, fp32 or float8_e4m3fn, which needs
    scales: fp32 [rows, ceil(width / 128)] with group=128, [rows, 1] or [rows] with group=0."""
    at, dtype, shape, out = x.get_device(), x.dtype, x.shape, o.dtype
    x_type, o_type = _TYPES.get(dtype), _TYPES.get(out)
    ok = at >= 0 and at == _current_device() and len(shape) == 2 and x_type is not None and x_type != _abi.TYPE_E4M3 and o_type is not None
    if ok:
        rows, width = shape
        x_row, x_last = x.stride()
        ok = x_last == 1 and o.shape == shape and o.is_contiguous() and o.get_device() == at
    r_type, r_ptr, r_row, w_ptr, scale_ptr = x_type, 0, 0, 0, 0
    if ok and residual is not None:
        r_type = _TYPES.get(residual.dtype)
        ok = r_type is not None and r_type != _abi.TYPE_E4M3 and residual.shape == shape and residual.get_device() == at
        if ok:
            r_row, r_last = residual.stride()
            ok, r_ptr = r_last == 1, residual.data_ptr()
    if ok and weight is not None:
        ok = weight.dtype is _FP32 and weight.dim() == 1 and weight.numel() == width and weight.is_contiguous() and weight.get_device() == at
        w_ptr = weight.data_ptr()
    if not ok:
        if out not in _TYPES:
            raise ValueError(f"o: bf16, fp32 or float8_e4m3fn, got {out}")
        if residual is not None and residual.dtype is not _BF16 and residual.dtype is not _FP32:
            raise ValueError(f"residual: bf16 or fp32, got {residual.dtype}")
        _refuse(at, x, "x", (2,), () if residual is None else ((residual, shape, residual.dtype, "residual"),),
                ((weight, shape[-1:], _FP32, "weight"), (o, shape, out, "o")))
    if out is _E4M3:
        if scales is None:
            raise ValueError("o in 8 bits needs scales")
        want = (rows, -(-width // group)) if group else (rows, 1)
        scale_ptr = _whole(scales, (rows,) if not group and scales.dim() == 1 else want, _FP32, "scales", at)
    elif scales is not None or group:
        raise ValueError("scales and group belong to an output in 8 bits")
    rc = _abi.load().gdn_add_rms_norm(_pack_norm(rows, width, x_type, r_type, o_type, group, eps, x.data_ptr(), x_row, r_ptr, r_row, w_ptr,
                                                 o.data_ptr(), scale_ptr), _stream(stream, at))
    if rc != GDN_OK:
        check(rc, "gdn_add_rms_norm")


def causal_conv(x, weight, pool, slot, o, *, bias=None, silu=True, seq_lens=None, status=None, stream=None):
    """o = the causal convolution of x [batch, T, channels] (or [batch, channels]: one token each) with weight
    [channels, 4], plus bias [channels], through SiLU. pool [slots, channels, 3], of x's type, holds the three inputs
    before each request's first position in row slot[b] and is left with the last three."""
    at, dtype, shape, rows = x.get_device(), x.dtype, x.shape, pool.shape
    ok = at >= 0 and at == _current_device() and (dtype is _BF16 or dtype is _FP32)
    if ok:
        if len(shape) == 2:
            (batch, channels), tokens, (x0, last), x1 = shape, 1, x.stride(), 0
        elif len(shape) == 3:
            (batch, tokens, channels), (x0, x1, last) = shape, x.stride()
        else:
            ok = False
    ok = (ok and last == 1 and len(rows) == 3 and rows[1] == channels and rows[2] == 3 and pool.dtype is dtype and o.dtype is dtype
          and weight.dtype is _FP32 and weight.shape == (channels, 4) and o.shape == shape
          and weight.is_contiguous() and pool.is_contiguous() and o.is_contiguous()
          and weight.get_device() == pool.get_device() == o.get_device() == at)
    bias_ptr = 0
    if ok and bias is not None:
        ok = bias.dtype is _FP32 and bias.dim() == 1 and bias.numel() == channels and bias.is_contiguous() and bias.get_device() == at
        bias_ptr = bias.data_ptr()
    if not ok:
        last = shape[-1:]
        _refuse(at, x, "x", (2, 3), (), ((weight, (*last, 4), _FP32, "weight"), (bias, last, _FP32, "bias"),
                                         (pool, (*rows[:1], *last, 3), dtype, "pool"), (o, shape, dtype, "o")))
    rc = _abi.load().gdn_causal_conv(
        _pack_conv(batch, tokens, channels, rows[0], (_abi.QKV_BF16 if dtype is _BF16 else 0) | (_abi.CONV_SILU if silu else 0), x.data_ptr(),
                   x0, x1, weight.data_ptr(), bias_ptr, pool.data_ptr(), _ints(slot, batch, "slot", at),
                   0 if seq_lens is None else _ints(seq_lens, batch, "seq_lens", at), o.data_ptr()),
        None if status is None else _status(status, at), _stream(stream, at))
    if rc != GDN_OK:
        check(rc, "gdn_causal_conv")


def ssm_workspace_bytes(batch: int, num_tokens: int, channels: int, state_size: int) -> int:
    """Bytes of workspace for every ssm_scan of these channels and states with no more requests and positions."""
    out = ctypes.c_size_t()
    check(_abi.load().gdn_ssm_workspace(batch, num_tokens, channels, state_size, ctypes.byref(out)), "gdn_ssm_workspace")
    return out.value


def _refuse_ssm(dims, at, u, dt, a, b, c, state, y, z, skip, dt_bias):
    dtype, shape, narrow, pool = u.dtype, u.shape, b.shape, state.shape
    if len(shape) != dims:
        _refuse(at, u, "u", (dims,), (), ())
    if len(narrow) != dims + 1:
        raise ValueError(f"b: {dims + 1} dimensions [.., groups, state size], got {tuple(narrow)}")
    if len(pool) != 3:
        raise ValueError(f"state: [slots, channels, state size], got {tuple(pool)}")
    few, channels, n = (*shape[:-1], *narrow[-2:]), shape[-1], narrow[-1]
    _refuse(at, u, "u", (dims,), ((dt, shape, dtype, "dt"), (z, shape, dtype, "z"), (b, few, dtype, "b"), (c, few, dtype, "c")),
            ((a, (channels, n), _FP32, "a"), (skip, (channels,), _FP32, "skip"), (dt_bias, (channels,), _FP32, "dt_bias"),
             (state, (pool[0], channels, n), _FP32, "state"), (y, shape, dtype, "y")))


def _pack(dims, u, dt, a, b, c, state, slot, y, z, skip, dt_bias, softplus, seq_lens):
    """The C struct of a scan (dims 3) or a step (dims 2), and the device."""
    at, dtype, shape, narrow, pool = u.get_device(), u.dtype, u.shape, b.shape, state.shape
    if (at < 0 or at != _current_device() or (dtype is not _BF16 and dtype is not _FP32) or len(shape) != dims or len(narrow) != dims + 1
            or len(pool) != 3):
        _refuse_ssm(dims, at, u, dt, a, b, c, state, y, z, skip, dt_bias)
    batch, channels, groups, n = shape[0], shape[-1], narrow[-2], narrow[-1]
    z_ptr = z0 = z1 = 0
    try:
        if dims == 2:  # no stride between the tokens of one
            tokens = 1
            (u0, ul), (t0, tl), (b0, b2, bl), (c0, c2, cl) = u.stride(), dt.stride(), b.stride(), c.stride()
            u1 = t1 = b1 = c1 = 0
            ok = narrow[0] == batch
            if z is not None:
                z0, zl = z.stride()
        else:
            tokens = shape[1]
            (u0, u1, ul), (t0, t1, tl), (b0, b1, b2, bl), (c0, c1, c2, cl) = u.stride(), dt.stride(), b.stride(), c.stride()
            ok = narrow[0] == batch and narrow[1] == tokens
            if z is not None:
                z0, z1, zl = z.stride()
    except ValueError:  # another number of dimensions
        ok = False
    ok = (ok and ul == tl == bl == cl == 1 and dt.dtype is dtype and b.dtype is dtype and c.dtype is dtype and y.dtype is dtype
          and dt.shape == shape and c.shape == narrow and y.shape == shape and a.shape == (channels, n) and pool[1] == channels and pool[2] == n
          and a.dtype is _FP32 and state.dtype is _FP32 and y.is_contiguous() and a.is_contiguous() and state.is_contiguous()
          and dt.get_device() == b.get_device() == c.get_device() == a.get_device() == state.get_device() == y.get_device() == at)
    if ok and z is not None:
        ok = zl == 1 and z.dtype is dtype and z.shape == shape and z.get_device() == at
        z_ptr = z.data_ptr()
    if ok and skip is not None:
        ok = skip.dtype is _FP32 and skip.dim() == 1 and skip.numel() == channels and skip.is_contiguous() and skip.get_device() == at
    if ok and dt_bias is not None:
        ok = dt_bias.dtype is _FP32 and dt_bias.dim() == 1 and dt_bias.numel() == channels and dt_bias.is_contiguous() and dt_bias.get_device() == at
    if not ok:
        _refuse_ssm(dims, at, u, dt, a, b, c, state, y, z, skip, dt_bias)
    return _pack_ssm(
        batch, tokens, channels, n, groups, pool[0], (_abi.QKV_BF16 if dtype is _BF16 else 0) | (_abi.DT_SOFTPLUS if softplus else 0),
        u.data_ptr(), u0, u1, dt.data_ptr(), t0, t1, b.data_ptr(), b0, b1, b2, c.data_ptr(), c0, c1, c2, z_ptr, z0, z1, a.data_ptr(),
        0 if skip is None else skip.data_ptr(), 0 if dt_bias is None else dt_bias.data_ptr(), state.data_ptr(), _ints(slot, batch, "slot", at),
        0 if seq_lens is None else _ints(seq_lens, batch, "seq_lens", at), y.data_ptr()), at


def ssm_scan(u, dt, a, b, c, state, slot, y, workspace=None, *, z=None, skip=None, dt_bias=None, softplus=True, seq_lens=None,
             status=None, stream=None):
    """The selective recurrence over prompts: u, dt, z, y [batch, T, channels], b, c [batch, T, groups, N], a [channels, N],
    skip, dt_bias [channels]; state [slots, channels, N] fp32 advances in place in the rows slot. workspace: a tensor
    of ssm_workspace_bytes() or more."""
    s, at = _pack(3, u, dt, a, b, c, state, slot, y, z, skip, dt_bias, softplus, seq_lens)
    room = 0
    if workspace is not None:
        if workspace.get_device() != at or not workspace.is_contiguous():
            raise ValueError("workspace: contiguous, on the GPU beside the others")
        room = workspace.nbytes
    rc = _abi.load().gdn_ssm_scan(s, workspace.data_ptr() if room else None, room, None if status is None else _status(status, at),
                                  _stream(stream, at))
    if rc != GDN_OK:
        check(rc, "gdn_ssm_scan")


def ssm_step(u, dt, a, b, c, state, slot, y, *, z=None, skip=None, dt_bias=None, softplus=True, status=None, stream=None):
    """One token of every request: as ssm_scan, without the dimension of the positions."""
    s, at = _pack(2, u, dt, a, b, c, state, slot, y, z, skip, dt_bias, softplus, None)
    rc = _abi.load().gdn_ssm_step(s, None if status is None else _status(status, at), _stream(stream, at))
    if rc != GDN_OK:
        check(rc, "gdn_ssm_step")
