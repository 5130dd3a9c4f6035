"""Python binding of the layer operators of libengram.so (include/
engram_layer.h; ctypes, the C ABI's names): the residual norm and its
backward, 8-bit activation checkpoints, the convolution's backward and its
single-token form, the scaled token embedding and its gradient.

As ``engram.py``: argument marshalling only, every step in the library's HIP
kernels, asynchronous on the current stream of the tensors' device, or on the
stream of that device passed as ``stream``.  Outputs and workspaces are torch tensors, allocated when
they are not passed in.  What each call computes stands in the header.

A tensor that is freed while work on another stream still reads it has to be
kept (or ``record_stream``-ed) by the caller, as everywhere in torch.
"""
from __future__ import annotations

import ctypes
import functools
import struct
from typing import NamedTuple, Optional

import torch

from . import abi
from .abi import ACT_BLOCK, BF16, F32, NORM_MAX_GROUP  # noqa: F401
from .engram import EngramError, _lib

abi.declare_layer(_lib)

_TYPES = {torch.bfloat16: BF16, torch.float32: F32}
_BAD_SIZE = (1 << 64) - 1


# The checks below run on every call, and a small call's time is its host
# time: the whole test of a good tensor comes first, and only one that fails it
# is looked at further for the message.
def _tensor(t, dtype, numel, what, index):
    """The address of a contiguous tensor on device `index` with `numel` values of `dtype`."""
    try:
        if (t.dtype is dtype and t.numel() == numel and t.get_device() == index
                and t.is_contiguous()):
            return t.data_ptr()
    except AttributeError:
        pass
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{what} must be a device (cuda) tensor")
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if t.get_device() != index:
        raise ValueError(f"{what} must be on cuda:{index}, is on {t.device}")
    if t.numel() != numel:
        raise ValueError(f"{what} must hold {numel} values, holds {t.numel()}")
    raise ValueError(f"{what} must be contiguous")


def _optional(t, dtype, numel, what, index):
    return 0 if t is None else _tensor(t, dtype, numel, what, index)


def _check_rows(t, lead, widths, what):
    """Raises when `t`, which has the right number of values, has them in another order of axes:
    it keeps the axes `lead` in front, or is flattened to rows of one of `widths` or to one axis
    (or the rows of `lead` are one axis themselves).  Axes of one do not count."""
    have, want = ([d for d in axes if d != 1] for axes in (t.shape, lead))
    if have[:len(want)] == want or len(have) <= 1:
        return
    if have[-1] in widths and (len(have) == 2 or len(want) <= 1):
        return
    raise ValueError(f"{what} must have the leading axes {tuple(lead)}, or be flattened to rows; "
                     f"has the shape {tuple(t.shape)}")


def _device_of(t, what):
    """(device, its index) of a device tensor."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{what} must be a device (cuda) tensor")
    return t.device, t.get_device()


def _stream_of(index):
    """The handle of the device's current stream (torch.cuda.current_stream's, without the
    object that it makes)."""
    return torch._C._cuda_getCurrentRawStream(index)


def _bytes(workspace, need, device, index, what):
    """A workspace of at least `need` bytes, allocated when none is given."""
    if need == _BAD_SIZE:
        raise EngramError(abi.ENGRAM_EINVAL, what)
    if workspace is None:
        return torch.empty(max(need, 16), dtype=torch.uint8, device=device)
    if workspace.numel() < need:
        raise ValueError(f"workspace must hold {need} bytes, holds {workspace.numel()}")
    _tensor(workspace, torch.uint8, workspace.numel(), "workspace", index)
    return workspace


def _run(index, name, *args):
    """The library's call `name` with device `index` current; raises on a status."""
    if torch.cuda.current_device() == index:
        status = getattr(_lib, name)(*args)
    else:
        with torch.cuda.device(index):
            status = getattr(_lib, name)(*args)
    if status != abi.ENGRAM_OK:
        raise EngramError(status, name)


def _streamed(call):
    """Adds the argument `stream`: the call runs, and what it allocates is allocated, with
    that stream current (so the memory is never given away while that stream still uses it)."""
    @functools.wraps(call)
    def on_stream(*args, stream=None, **kwargs):
        if stream is None:
            return call(*args, **kwargs)
        # (a stream of another device would leave the call on its tensors' device's own stream)
        for t in (*args, *kwargs.values()):
            if isinstance(t, torch.Tensor) and t.is_cuda:
                if t.get_device() != stream.device.index:
                    raise ValueError(f"the stream is on {stream.device}, the tensors on {t.device}")
                break
        with torch.cuda.stream(stream):
            return call(*args, **kwargs)
    return on_stream


def code_blocks(channels: int) -> int:
    """Scales a row of `channels` values takes (ENGRAM_ACT_BLOCK values each)."""
    return -(-channels // ACT_BLOCK)


# ------------------------------------------------------------- residual norm --
class ResidualNorm(NamedTuple):
    """What engram_residual_norm wrote; what was not asked for is None."""
    out: Optional[torch.Tensor]
    next: Optional[torch.Tensor]
    rstd_post: Optional[torch.Tensor]
    rstd_next: Optional[torch.Tensor]
    y_codes: Optional[torch.Tensor] = None
    y_scales: Optional[torch.Tensor] = None
    next_codes: Optional[torch.Tensor] = None
    next_scales: Optional[torch.Tensor] = None


class ResidualNormGrads(NamedTuple):
    """The gradients engram_residual_norm_backward wrote."""
    residual: Optional[torch.Tensor]
    y: Optional[torch.Tensor]
    gate: Optional[torch.Tensor]
    w_post: Optional[torch.Tensor]
    scale: Optional[torch.Tensor]
    w_next: Optional[torch.Tensor]


# struct engram_norm_args, packed in one go
_NORM = struct.Struct("=4q2f2i" + 25 * "Q")
assert _NORM.size == ctypes.sizeof(abi.EngramNormArgs)


def _norm_shape(like, groups):
    """(rows, channels, type) of rows like `like` [..., channels]."""
    kind = _TYPES.get(like.dtype)
    if kind is None:
        raise TypeError(f"the residual must be bfloat16 or float32, is {like.dtype}")
    channels = like.shape[-1] if like.dim() else 0
    if channels < 1 or groups < 1 or channels % (8 * groups):
        raise ValueError("channels must be a positive multiple of 8 * groups")
    return like.numel() // channels, channels, kind


def _gate_of(gate, like, rows, channels, groups, index):
    """(width, address) of a gate [..., groups] or [..., channels] of the rows of `like`, or of
    none."""
    if gate is None:
        return 0, 0
    width = gate.shape[-1] if gate.dim() else 0
    if width != groups and width != channels:
        raise ValueError("gate must be [..., groups] or [..., channels]")
    address = _tensor(gate, torch.bfloat16, rows * width, "gate", index)
    if gate.dim() > 2:  # (of two axes the first is the rows)
        _check_rows(gate, like.shape[:-1], (width,), "gate")
    return width, address


def _codes(rows, channels, groups, device):
    return (torch.empty((rows, channels), dtype=torch.int8, device=device),
            torch.empty((rows, groups * code_blocks(channels // groups)), dtype=torch.float32,
                        device=device))


@_streamed
def engram_residual_norm(residual, y=None, *, gate=None, w_post=None, scale=None, w_next=None,
                         groups=1, eps=1e-6, residual_scale=1.0, save_codes=False,
                         next_codes=False, out=None, next_out=None, rstd_post=None,
                         rstd_next=None):
    """out = residual_scale * residual + scale * sigmoid(gate) * w_post * norm(y), and the
    next block's norm of it; without y, the norm of the residual alone (w_next).

    residual bf16 or fp32 [..., channels], y bf16 of its shape.  save_codes keeps y's 8-bit
    checkpoint, next_codes that of the next norm's output.  out may be the residual."""
    device, index = _device_of(residual, "residual")
    rows, channels, kind = _norm_shape(residual, groups)
    n, stats, rt, bf = rows * channels, rows * groups, residual.dtype, torch.bfloat16
    width, gate_p = _gate_of(gate, residual, rows, channels, groups, index)
    y_p = out_p = post_p = next_p = rnext_p = yc_p = ys_p = nc_p = ns_p = 0
    yc = ys = nc = ns = None
    if y is not None:
        y_p = _tensor(y, bf, n, "y", index)
        if y.shape != residual.shape:
            raise ValueError("y must have the residual's shape")
        if out is None:
            out = torch.empty_like(residual)
        out_p = _tensor(out, rt, n, "out", index)
        if rstd_post is None:
            rstd_post = torch.empty((rows, groups), dtype=torch.float32, device=device)
        post_p = _tensor(rstd_post, torch.float32, stats, "rstd_post", index)
    elif out is not None or rstd_post is not None or save_codes:
        raise ValueError("out, rstd_post and save_codes need y")
    if w_next is not None:
        if next_out is None:
            next_out = torch.empty(residual.shape, dtype=bf, device=device)
        next_p = _tensor(next_out, bf, n, "next_out", index)
        if rstd_next is None:
            rstd_next = torch.empty((rows, groups), dtype=torch.float32, device=device)
        rnext_p = _tensor(rstd_next, torch.float32, stats, "rstd_next", index)
    elif next_out is not None or rstd_next is not None or next_codes:
        raise ValueError("next_out, rstd_next and next_codes need w_next")
    if save_codes:
        yc, ys = _codes(rows, channels, groups, device)
        yc_p, ys_p = yc.data_ptr(), ys.data_ptr()
    if next_codes:
        nc, ns = _codes(rows, channels, groups, device)
        nc_p, ns_p = nc.data_ptr(), ns.data_ptr()
    _run(index, "engram_residual_norm", _NORM.pack(
        rows, channels, groups, width, eps, residual_scale, kind, 0,
        _tensor(residual, rt, n, "residual", index), y_p, gate_p,
        _optional(w_post, bf, channels, "w_post", index),
        _optional(scale, bf, channels, "scale", index),
        _optional(w_next, bf, channels, "w_next", index), out_p, next_p, post_p, rnext_p,
        yc_p, ys_p, nc_p, ns_p, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, _stream_of(index)))
    return ResidualNorm(out, next_out, rstd_post, rstd_next, yc, ys, nc, ns)


@_streamed
def engram_residual_norm_backward(grad_out, grad_next=None, *, out=None, rstd_post=None,
                                  rstd_next=None, y=None, y_codes=None, y_scales=None, gate=None,
                                  w_post=None, scale=None, w_next=None, groups=1,
                                  residual_scale=1.0, grad_residual=None, workspace=None):
    """Gradients of engram_residual_norm from what it kept: out, the two rstds, and y or its
    8-bit checkpoint.  grad_out (of the residual's type) or grad_next may be None when nothing
    reads that output.  grad_residual may be grad_out, which is then overwritten."""
    like = grad_out if grad_out is not None else out
    if like is None:
        raise ValueError("grad_out or out must be given")
    device, index = _device_of(like, "grad_out" if grad_out is not None else "out")
    rows, channels, kind = _norm_shape(like, groups)
    n, stats, rt = rows * channels, rows * groups, like.dtype
    bf, f32 = torch.bfloat16, torch.float32
    width, gate_p = _gate_of(gate, like, rows, channels, groups, index)
    if (w_next is None) != (grad_next is None):
        raise ValueError("grad_next goes with w_next")
    out_p = dn_p = rnext_p = post_p = y_p = yc_p = ys_p = 0
    if w_next is not None:
        dn_p = _tensor(grad_next, bf, n, "grad_next", index)
        if grad_next.shape != like.shape:
            raise ValueError("grad_next must have the shape of grad_out (or of out)")
        out_p = _tensor(out, rt, n, "out", index)
        if out.shape != like.shape:
            _check_rows(out, like.shape[:-1], (channels,), "out")
        rnext_p = _tensor(rstd_next, f32, stats, "rstd_next", index)
    branch = y is not None or y_codes is not None
    if branch:
        post_p = _tensor(rstd_post, f32, stats, "rstd_post", index)
        y_p = _optional(y, bf, n, "y", index)
        if y is not None and y.shape != like.shape:
            _check_rows(y, like.shape[:-1], (channels,), "y")
        yc_p = _optional(y_codes, torch.int8, n, "y_codes", index)
        if y_codes is not None:
            _check_rows(y_codes, like.shape[:-1], (channels, channels // groups), "y_codes")
        ys_p = _optional(y_scales, f32, stats * code_blocks(channels // groups), "y_scales",
                         index)
    if grad_residual is None:
        grad_residual = torch.empty_like(like)
    gy = gz = gp = gs = gn = None
    gy_p = gz_p = gp_p = gs_p = gn_p = ws_p = size = 0
    if branch:
        gy = torch.empty_like(y) if y is not None else torch.empty(like.shape, dtype=bf,
                                                                   device=device)
        gy_p = gy.data_ptr()
        if gate is not None:
            gz = torch.empty_like(gate)
            gz_p = gz.data_ptr()
        if w_post is not None:
            gp = torch.empty((channels,), dtype=f32, device=device)
            gp_p = gp.data_ptr()
        if scale is not None:
            gs = torch.empty((channels,), dtype=f32, device=device)
            gs_p = gs.data_ptr()
    if w_next is not None:
        gn = torch.empty((channels,), dtype=f32, device=device)
        gn_p = gn.data_ptr()
    if gp_p or gs_p or gn_p:
        need = _lib.engram_residual_norm_backward_workspace(rows, channels, groups)
        workspace = _bytes(workspace, need, device, index,
                           "engram_residual_norm_backward_workspace")
        ws_p, size = workspace.data_ptr(), workspace.numel()
    _run(index, "engram_residual_norm_backward", _NORM.pack(
        rows, channels, groups, width, 0.0, residual_scale, kind, 0, 0, y_p, gate_p,
        _optional(w_post, bf, channels, "w_post", index),
        _optional(scale, bf, channels, "scale", index),
        _optional(w_next, bf, channels, "w_next", index), out_p, 0, post_p, rnext_p, yc_p,
        ys_p, 0, 0, _optional(grad_out, rt, n, "grad_out", index), dn_p,
        _tensor(grad_residual, rt, n, "grad_residual", index), gy_p, gz_p, gp_p, gs_p, gn_p,
        ws_p, size, _stream_of(index)))
    return ResidualNormGrads(grad_residual, gy, gz, gp, gs, gn)


def engram_residual_norm_backward_workspace(rows, channels, groups=1) -> int:
    need = _lib.engram_residual_norm_backward_workspace(rows, channels, groups)
    if need == _BAD_SIZE:
        raise EngramError(abi.ENGRAM_EINVAL, "engram_residual_norm_backward_workspace")
    return need


# --------------------------------------------------------- 8-bit checkpoints --
@_streamed
def engram_act_encode(x, codes=None, scales=None):
    """The 8-bit checkpoint of x bf16 [..., channels]: (codes int8 of its shape, scales fp32
    [..., ceil(channels / 128)])."""
    device, index = _device_of(x, "x")
    channels = x.shape[-1] if x.dim() else 0
    if channels < 1:
        raise ValueError("x must be [..., channels]")
    rows = x.numel() // channels
    xp = _tensor(x, torch.bfloat16, rows * channels, "x", index)
    if codes is None:
        codes = torch.empty(x.shape, dtype=torch.int8, device=device)
    if scales is None:
        scales = torch.empty((*x.shape[:-1], code_blocks(channels)), dtype=torch.float32,
                             device=device)
    cp = _tensor(codes, torch.int8, rows * channels, "codes", index)
    sp = _tensor(scales, torch.float32, rows * code_blocks(channels), "scales", index)
    _run(index, "engram_act_encode", xp, rows, channels, cp, sp, _stream_of(index))
    return codes, scales


@_streamed
def engram_act_decode(codes, scales, out=None):
    """The values (bf16) of an 8-bit checkpoint."""
    device, index = _device_of(codes, "codes")
    channels = codes.shape[-1] if codes.dim() else 0
    if channels < 1:
        raise ValueError("codes must be [..., channels]")
    rows = codes.numel() // channels
    cp = _tensor(codes, torch.int8, rows * channels, "codes", index)
    sp = _tensor(scales, torch.float32, rows * code_blocks(channels), "scales", index)
    if out is None:
        out = torch.empty(codes.shape, dtype=torch.bfloat16, device=device)
    op = _tensor(out, torch.bfloat16, rows * channels, "out", index)
    _run(index, "engram_act_decode", cp, sp, rows, channels, op, _stream_of(index))
    return out


# --------------------------------------------------------------- convolution --
def _taps(weight, dilation):
    """(kernel_size, dilation) as the 32-bit numbers of the call, which would take a larger
    one's low half."""
    kernel, dilation = weight.shape[1], int(dilation)
    if not -1 << 31 <= dilation < 1 << 31 or kernel >= 1 << 31:
        raise ValueError("kernel_size and dilation must fit 32 bits")
    return kernel, dilation


class ConvGrads(NamedTuple):
    """The gradients engram_ple_conv_backward wrote."""
    x: Optional[torch.Tensor]
    weight: Optional[torch.Tensor]
    bias: Optional[torch.Tensor]
    halo: Optional[torch.Tensor]


@_streamed
def engram_ple_conv_backward(grad_out, weight, dilation, x=None, x_codes=None, x_scales=None,
                             code_width=0, seq_ids=None, halo=None, need_x=True,
                             need_weight=True, need_bias=True, workspace=None):
    """Gradients of engram_ple_conv: of x (and the halo), of the weight (fp32, needs x or its
    8-bit checkpoint; code_width: the row width it was made with, 0 for all channels) and of
    the bias (fp32)."""
    device, index = _device_of(grad_out, "grad_out")
    if grad_out.dim() != 3:
        raise ValueError("grad_out must be [batch, seq, channels]")
    batch, seq, channels = grad_out.shape
    if weight.dim() != 2 or weight.shape[0] != channels:
        raise ValueError("weight must be [channels, kernel_size]")
    kernel, dilation = _taps(weight, dilation)
    n, halo_len = grad_out.numel(), 0
    gp = _tensor(grad_out, torch.bfloat16, n, "grad_out", index)
    wp = _tensor(weight, torch.bfloat16, channels * kernel, "weight", index)
    hp = None
    if halo is not None:
        if halo.dim() != 3 or halo.shape[0] != batch or halo.shape[2] != channels:
            raise ValueError("halo must be [batch, halo_len, channels]")
        halo_len = halo.shape[1]
        hp = _tensor(halo, torch.bfloat16, batch * halo_len * channels, "halo", index)
    ids = _optional(seq_ids, torch.int64, batch * (halo_len + seq), "seq_ids", index)
    if seq_ids is not None and seq_ids.shape != (batch, halo_len + seq):
        _check_rows(seq_ids, (batch, halo_len + seq), (), "seq_ids")
    xp = cp = sp = None
    if need_weight:
        if (x is None) == (x_codes is None):
            raise ValueError("the weight's gradient needs x, or x_codes and x_scales")
        xp = _optional(x, torch.bfloat16, n, "x", index)
        if x is not None and x.shape != grad_out.shape:
            _check_rows(x, (batch, seq), (channels,), "x")
        cp = _optional(x_codes, torch.int8, n, "x_codes", index)
        if x_codes is not None:
            width = code_width or channels
            if width < 1 or channels % width:
                raise ValueError("code_width must divide channels")
            _check_rows(x_codes, (batch, seq), (channels, width), "x_codes")
            sp = _tensor(x_scales, torch.float32,
                         batch * seq * (channels // width) * code_blocks(width), "x_scales", index)
    gx = torch.empty_like(grad_out) if need_x else None
    gh = torch.empty_like(halo) if need_x and halo_len else None
    gw = gb = None
    if need_weight:
        gw = torch.empty((channels, kernel), dtype=torch.float32, device=device)
    if need_bias:
        gb = torch.empty((channels,), dtype=torch.float32, device=device)
    size = 0
    if need_weight or need_bias:
        need = _lib.engram_ple_conv_backward_workspace(batch, seq, halo_len, channels, kernel,
                                                       dilation)
        workspace = _bytes(workspace, need, device, index, "engram_ple_conv_backward_workspace")
        size = workspace.numel()

    def ptr(t):
        return None if t is None else t.data_ptr()

    _run(index, "engram_ple_conv_backward", gp, xp, cp, sp, code_width,
         hp if halo_len else None, halo_len, ids, wp, batch, seq, channels, kernel, dilation,
         ptr(gx), ptr(gh), ptr(gw), ptr(gb), ptr(workspace) if size else None, size,
         _stream_of(index))
    if need_x and halo is not None and gh is None:
        gh = torch.empty_like(halo)  # a halo of no positions
    return ConvGrads(gx, gw, gb, gh)


@_streamed
def engram_ple_conv_step(x, ring, weight, dilation, positions, slots=None, bias=None, out=None,
                         write_only=False, err_count=None):
    """engram_ple_conv for the next tokens of each sequence: x bf16 [batch, tokens, channels]
    (or [batch, channels], one token), ring bf16 [ring_count, ring_rows, channels] updated in
    place, positions int64 [batch] of each sequence's first token here within its segment,
    slots int64 [batch] the ring of each (None: ring b; -1: unused).  write_only: the ring is
    written and nothing computed (a prompt's last inputs)."""
    device, index = _device_of(x, "x")
    if x.dim() == 2:
        (batch, channels), tokens = x.shape, 1
    elif x.dim() == 3:
        batch, tokens, channels = x.shape
    else:
        raise ValueError("x must be [batch, tokens, channels] or [batch, channels]")
    if ring.dim() != 3 or ring.shape[2] != channels:
        raise ValueError("ring must be [ring_count, ring_rows, channels]")
    if weight.dim() != 2 or weight.shape[0] != channels:
        raise ValueError("weight must be [channels, kernel_size]")
    kernel, dilation = _taps(weight, dilation)
    n = batch * tokens * channels
    xp = _tensor(x, torch.bfloat16, n, "x", index)
    rp = _tensor(ring, torch.bfloat16, ring.numel(), "ring", index)
    wp = _tensor(weight, torch.bfloat16, channels * kernel, "weight", index)
    pp = _tensor(positions, torch.int64, batch, "positions", index)
    ip = _optional(slots, torch.int64, batch, "slots", index)
    bp = _optional(bias, torch.bfloat16, channels, "bias", index)
    ep = _optional(err_count, torch.int64, 1, "err_count", index)
    op = None
    if not write_only:
        if out is None:
            out = torch.empty(x.shape, dtype=torch.bfloat16, device=device)
        op = _tensor(out, torch.bfloat16, n, "out", index)
    elif out is not None:
        raise ValueError("write_only computes no out")
    _run(index, "engram_ple_conv_step", xp, rp, ring.shape[0], ring.shape[1], ip, pp, wp, bp,
         batch, tokens, channels, kernel, dilation, op, ep, _stream_of(index))
    return out


# ----------------------------------------------------------------- embedding --
@_streamed
def engram_embed(tokens, table, scale=1.0, out=None, out_dtype=torch.bfloat16, err_count=None):
    """scale * table[tokens]: tokens int64 of any shape (-1: a zero row), table bf16
    [table_rows, channels]; out of out_dtype (bf16 or fp32) [..., channels]."""
    device, index = _device_of(tokens, "tokens")
    if table.dim() != 2:
        raise ValueError("table must be [table_rows, channels]")
    table_rows, channels = table.shape
    n = tokens.numel()
    tp = _tensor(tokens, torch.int64, n, "tokens", index)
    bp = _tensor(table, torch.bfloat16, table.numel(), "table", index)
    if out is None:
        out = torch.empty((*tokens.shape, channels), dtype=out_dtype, device=device)
    if out.dtype not in _TYPES:
        raise TypeError(f"out must be bfloat16 or float32, is {out.dtype}")
    op = _tensor(out, out.dtype, n * channels, "out", index)
    ep = _optional(err_count, torch.int64, 1, "err_count", index)
    _run(index, "engram_embed", tp, n, bp, table_rows, channels, float(scale),
         _TYPES[out.dtype], op, ep, _stream_of(index))
    return out


@_streamed
def engram_embed_grad(tokens, grads, table_rows, scale=1.0, grad_table=None,
                      grad_dtype=torch.float32, accumulate=False, workspace=None, err_count=None):
    """The gradient of engram_embed, from grads bf16 or fp32 [..., channels], into the whole
    table [table_rows, channels] (grad_dtype: fp32 or bf16): rows without a token get zeros;
    with accumulate (fp32, grad_table given) the sums are added to the rows that have tokens.
    Should a bounded wait of the sort (of more than 65,536 tokens) expire, err_count receives
    ERR_STALLED and the gradient is NaN; accumulated, the table is left as it was, and only
    err_count tells."""
    device, index = _device_of(grads, "grads")
    n = tokens.numel()
    channels = grads.shape[-1] if grads.dim() else 0
    if channels < 1:
        raise ValueError("grads must be [..., channels]")
    tp = _tensor(tokens, torch.int64, n, "tokens", index)
    if grads.dtype not in _TYPES:
        raise TypeError(f"grads must be bfloat16 or float32, is {grads.dtype}")
    gp = _tensor(grads, grads.dtype, n * channels, "grads", index)
    if grads.dim() > 2 and tokens.dim() > 1 and grads.shape[:-1] != tokens.shape:
        _check_rows(grads, tokens.shape, (channels,), "grads")
    if grad_table is None:
        if accumulate:
            raise ValueError("accumulate needs grad_table")
        grad_table = torch.empty((table_rows, channels), dtype=grad_dtype, device=device)
    if grad_table.dtype not in _TYPES:
        raise TypeError(f"grad_table must be bfloat16 or float32, is {grad_table.dtype}")
    op = _tensor(grad_table, grad_table.dtype, table_rows * channels, "grad_table", index)
    if grad_table.dim() == 2 and grad_table.shape[1] != channels:
        raise ValueError("grad_table must be [table_rows, channels]")
    ep = _optional(err_count, torch.int64, 1, "err_count", index)
    need = _lib.engram_embed_grad_workspace(n, channels, table_rows)
    workspace = _bytes(workspace, need, device, index, "engram_embed_grad_workspace")
    _run(index, "engram_embed_grad", tp, n, gp, _TYPES[grads.dtype], channels, float(scale),
         table_rows, _TYPES[grad_table.dtype], int(accumulate), op, workspace.data_ptr(),
         workspace.numel(), ep, _stream_of(index))
    return grad_table
