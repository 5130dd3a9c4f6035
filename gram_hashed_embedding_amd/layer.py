"""Python binding of the layer operators of libengram.so (include/
engram_layer.h; ctypes, the C ABI's names): the residual norm and its
backward, 8-bit activation checkpoints, the convolution's backward and its
single-token form, the scaled token embedding and its gradient.

As ``engram.py``: argument marshalling only, every step in the library's HIP
kernels, asynchronous on the current stream of the tensors' device, or on the
stream passed as ``stream``.  Outputs and workspaces are torch tensors, allocated when
they are not passed in.  What each call computes stands in the header.

A tensor that is freed while work on another stream still reads it has to be
kept (or ``record_stream``-ed) by the caller, as everywhere in torch.
"""
from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple, Optional

import torch

from . import abi
from .abi import ACT_BLOCK, BF16, F32, NORM_MAX_GROUP  # noqa: F401
from .engram import EngramError, _check, _lib, _on  # noqa: F401

abi.declare_layer(_lib)

_TYPES = {torch.bfloat16: BF16, torch.float32: F32}
_BAD_SIZE = (1 << 64) - 1


def _tensor(t, dtype, numel, what, device):
    """A contiguous tensor of `device` with `numel` elements of `dtype`."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{what} must be a device (cuda) tensor")
    if t.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{what} must be on {device}, is on {t.device}")
    if t.numel() != numel:
        raise ValueError(f"{what} must hold {numel} values, holds {t.numel()}")
    if not t.is_contiguous():
        raise ValueError(f"{what} must be contiguous")
    return t.data_ptr()


def _optional(t, dtype, numel, what, device):
    return None if t is None else _tensor(t, dtype, numel, what, device)


def _stream_of(device):
    return torch.cuda.current_stream(device).cuda_stream


def _streamed(call):
    """Adds the argument `stream`: the call runs, and what it allocates is allocated, with
    that stream current (so the memory is never given away while that stream still uses it)."""
    @functools.wraps(call)
    def on_stream(*args, stream=None, **kwargs):
        if stream is None:
            return call(*args, **kwargs)
        with torch.cuda.stream(stream):
            return call(*args, **kwargs)
    return on_stream


def _device_of(t, what):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{what} must be a device (cuda) tensor")
    return t.device


def _bytes(workspace, need, device, what):
    """A workspace of at least `need` bytes, allocated when none is given."""
    if need == _BAD_SIZE:
        raise EngramError(abi.ENGRAM_EINVAL, what)
    if workspace is None:
        return torch.empty(max(need, 16), dtype=torch.uint8, device=device)
    if workspace.numel() < need:
        raise ValueError(f"workspace must hold {need} bytes, holds {workspace.numel()}")
    _tensor(workspace, torch.uint8, workspace.numel(), "workspace", device)
    return workspace


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


def _norm_args(like, groups, gate, w_post, scale, w_next, residual_scale, device):
    """The fields both directions share, for rows like `like` [..., channels]."""
    channels = like.shape[-1] if like.dim() else 0
    if like.dtype not in _TYPES:
        raise TypeError(f"the residual must be bfloat16 or float32, is {like.dtype}")
    if channels < 1 or groups < 1 or channels % (8 * groups):
        raise ValueError("channels must be a positive multiple of 8 * groups")
    rows = like.numel() // channels
    a = abi.EngramNormArgs()
    a.rows, a.channels, a.groups = rows, channels, groups
    a.residual_scale, a.residual_type = residual_scale, _TYPES[like.dtype]
    if gate is not None:
        width = gate.shape[-1] if gate.dim() else 0
        if width not in (groups, channels):
            raise ValueError("gate must be [..., groups] or [..., channels]")
        a.gate_width = width
        a.d_gate = _tensor(gate, torch.bfloat16, rows * width, "gate", device)
    a.d_w_post = _optional(w_post, torch.bfloat16, channels, "w_post", device)
    a.d_scale = _optional(scale, torch.bfloat16, channels, "scale", device)
    a.d_w_next = _optional(w_next, torch.bfloat16, channels, "w_next", device)
    return a, rows, channels


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
    device = _device_of(residual, "residual")
    a, rows, channels = _norm_args(residual, groups, gate, w_post, scale, w_next,
                                   residual_scale, device)
    a.eps = eps
    n = rows * channels
    a.d_residual = _tensor(residual, residual.dtype, n, "residual", device)
    shape = residual.shape
    if y is not None:
        a.d_y = _tensor(y, torch.bfloat16, n, "y", device)
        if out is None:
            out = torch.empty(shape, dtype=residual.dtype, device=device)
        a.d_out = _tensor(out, residual.dtype, n, "out", device)
        if rstd_post is None:
            rstd_post = torch.empty((rows, groups), dtype=torch.float32, device=device)
        a.d_rstd_post = _tensor(rstd_post, torch.float32, rows * groups, "rstd_post", device)
    elif out is not None or rstd_post is not None or save_codes:
        raise ValueError("out, rstd_post and save_codes need y")
    if w_next is not None:
        if next_out is None:
            next_out = torch.empty(shape, dtype=torch.bfloat16, device=device)
        a.d_next = _tensor(next_out, torch.bfloat16, n, "next_out", device)
        if rstd_next is None:
            rstd_next = torch.empty((rows, groups), dtype=torch.float32, device=device)
        a.d_rstd_next = _tensor(rstd_next, torch.float32, rows * groups, "rstd_next", device)
    elif next_out is not None or rstd_next is not None or next_codes:
        raise ValueError("next_out, rstd_next and next_codes need w_next")
    yc = ys = nc = ns = None
    if save_codes:
        yc, ys = _codes(rows, channels, groups, device)
        a.d_y_codes, a.d_y_scales = yc.data_ptr(), ys.data_ptr()
    if next_codes:
        nc, ns = _codes(rows, channels, groups, device)
        a.d_next_codes, a.d_next_scales = nc.data_ptr(), ns.data_ptr()
    with _on(device):
        a.stream = _stream_of(device)
        status = _lib.engram_residual_norm(ctypes.byref(a))
    _check(status, "engram_residual_norm")
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
    device = _device_of(like, "grad_out" if grad_out is not None else "out")
    a, rows, channels = _norm_args(like, groups, gate, w_post, scale, w_next, residual_scale,
                                   device)
    n, rt = rows * channels, like.dtype
    if (w_next is None) != (grad_next is None):
        raise ValueError("grad_next goes with w_next")
    a.d_grad_out = _optional(grad_out, rt, n, "grad_out", device)
    if w_next is not None:
        a.d_grad_next = _tensor(grad_next, torch.bfloat16, n, "grad_next", device)
        a.d_out = _tensor(out, rt, n, "out", device)
        a.d_rstd_next = _tensor(rstd_next, torch.float32, rows * groups, "rstd_next", device)
    branch = y is not None or y_codes is not None
    if branch:
        a.d_rstd_post = _tensor(rstd_post, torch.float32, rows * groups, "rstd_post", device)
        a.d_y = _optional(y, torch.bfloat16, n, "y", device)
        a.d_y_codes = _optional(y_codes, torch.int8, n, "y_codes", device)
        a.d_y_scales = _optional(y_scales, torch.float32,
                                 rows * groups * code_blocks(channels // groups), "y_scales",
                                 device)
    shape = like.shape
    if grad_residual is None:
        grad_residual = torch.empty(shape, dtype=rt, device=device)
    a.d_grad_residual = _tensor(grad_residual, rt, n, "grad_residual", device)
    gy = gz = gp = gs = gn = None
    if branch:
        gy = torch.empty(shape, dtype=torch.bfloat16, device=device)
        a.d_grad_y = gy.data_ptr()
        if gate is not None:
            gz = torch.empty_like(gate)
            a.d_grad_gate = gz.data_ptr()

    def sums():
        return torch.empty((channels,), dtype=torch.float32, device=device)

    if branch and w_post is not None:
        gp = sums()
        a.d_grad_w_post = gp.data_ptr()
    if branch and scale is not None:
        gs = sums()
        a.d_grad_scale = gs.data_ptr()
    if w_next is not None:
        gn = sums()
        a.d_grad_w_next = gn.data_ptr()
    if gp is not None or gs is not None or gn is not None:
        need = _lib.engram_residual_norm_backward_workspace(rows, channels, groups)
        workspace = _bytes(workspace, need, device, "engram_residual_norm_backward_workspace")
        a.d_workspace, a.workspace_bytes = workspace.data_ptr(), workspace.numel()
    with _on(device):
        a.stream = _stream_of(device)
        status = _lib.engram_residual_norm_backward(ctypes.byref(a))
    _check(status, "engram_residual_norm_backward")
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
    device = _device_of(x, "x")
    channels = x.shape[-1] if x.dim() else 0
    if channels < 1:
        raise ValueError("x must be [..., channels]")
    rows = x.numel() // channels
    xp = _tensor(x, torch.bfloat16, rows * channels, "x", device)
    if codes is None:
        codes = torch.empty(x.shape, dtype=torch.int8, device=device)
    if scales is None:
        scales = torch.empty((*x.shape[:-1], code_blocks(channels)), dtype=torch.float32,
                             device=device)
    cp = _tensor(codes, torch.int8, rows * channels, "codes", device)
    sp = _tensor(scales, torch.float32, rows * code_blocks(channels), "scales", device)
    with _on(device):
        status = _lib.engram_act_encode(xp, rows, channels, cp, sp, _stream_of(device))
    _check(status, "engram_act_encode")
    return codes, scales


@_streamed
def engram_act_decode(codes, scales, out=None):
    """The values (bf16) of an 8-bit checkpoint."""
    device = _device_of(codes, "codes")
    channels = codes.shape[-1] if codes.dim() else 0
    if channels < 1:
        raise ValueError("codes must be [..., channels]")
    rows = codes.numel() // channels
    cp = _tensor(codes, torch.int8, rows * channels, "codes", device)
    sp = _tensor(scales, torch.float32, rows * code_blocks(channels), "scales", device)
    if out is None:
        out = torch.empty(codes.shape, dtype=torch.bfloat16, device=device)
    op = _tensor(out, torch.bfloat16, rows * channels, "out", device)
    with _on(device):
        status = _lib.engram_act_decode(cp, sp, rows, channels, op, _stream_of(device))
    _check(status, "engram_act_decode")
    return out


# --------------------------------------------------------------- convolution --
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
    device = _device_of(grad_out, "grad_out")
    if grad_out.dim() != 3:
        raise ValueError("grad_out must be [batch, seq, channels]")
    batch, seq, channels = grad_out.shape
    if weight.dim() != 2 or weight.shape[0] != channels:
        raise ValueError("weight must be [channels, kernel_size]")
    kernel = weight.shape[1]
    n, halo_len = grad_out.numel(), 0
    gp = _tensor(grad_out, torch.bfloat16, n, "grad_out", device)
    wp = _tensor(weight, torch.bfloat16, channels * kernel, "weight", device)
    hp = None
    if halo is not None:
        if halo.dim() != 3 or halo.shape[0] != batch or halo.shape[2] != channels:
            raise ValueError("halo must be [batch, halo_len, channels]")
        halo_len = halo.shape[1]
        hp = _tensor(halo, torch.bfloat16, batch * halo_len * channels, "halo", device)
    ids = _optional(seq_ids, torch.int64, batch * (halo_len + seq), "seq_ids", device)
    xp = cp = sp = None
    if need_weight:
        if (x is None) == (x_codes is None):
            raise ValueError("the weight's gradient needs x, or x_codes and x_scales")
        xp = _optional(x, torch.bfloat16, n, "x", device)
        cp = _optional(x_codes, torch.int8, n, "x_codes", device)
        if cp is not None:
            width = code_width or channels
            if width < 1 or channels % width:
                raise ValueError("code_width must divide channels")
            sp = _tensor(x_scales, torch.float32,
                         batch * seq * (channels // width) * code_blocks(width), "x_scales",
                         device)
    gx = torch.empty(grad_out.shape, dtype=torch.bfloat16, device=device) if need_x else None
    gh = torch.empty_like(halo) if need_x and halo_len else None
    gw = gb = None
    if need_weight:
        gw = torch.empty((channels, kernel), dtype=torch.float32, device=device)
    if need_bias:
        gb = torch.empty((channels,), dtype=torch.float32, device=device)
    size = 0
    if need_weight or need_bias:
        need = _lib.engram_ple_conv_backward_workspace(batch, seq, halo_len, channels, kernel,
                                                       int(dilation))
        workspace = _bytes(workspace, need, device, "engram_ple_conv_backward_workspace")
        size = workspace.numel()

    def ptr(t):
        return None if t is None else t.data_ptr()

    with _on(device):
        status = _lib.engram_ple_conv_backward(
            gp, xp, cp, sp, code_width, hp if halo_len else None, halo_len, ids, wp, batch, seq,
            channels, kernel, int(dilation), ptr(gx), ptr(gh), ptr(gw), ptr(gb),
            ptr(workspace) if size else None, size, _stream_of(device))
    _check(status, "engram_ple_conv_backward")
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
    device = _device_of(x, "x")
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
    kernel, n = weight.shape[1], batch * tokens * channels
    xp = _tensor(x, torch.bfloat16, n, "x", device)
    rp = _tensor(ring, torch.bfloat16, ring.numel(), "ring", device)
    wp = _tensor(weight, torch.bfloat16, channels * kernel, "weight", device)
    pp = _tensor(positions, torch.int64, batch, "positions", device)
    ip = _optional(slots, torch.int64, batch, "slots", device)
    bp = _optional(bias, torch.bfloat16, channels, "bias", device)
    ep = _optional(err_count, torch.int64, 1, "err_count", device)
    op = None
    if not write_only:
        if out is None:
            out = torch.empty(x.shape, dtype=torch.bfloat16, device=device)
        op = _tensor(out, torch.bfloat16, n, "out", device)
    elif out is not None:
        raise ValueError("write_only computes no out")
    with _on(device):
        status = _lib.engram_ple_conv_step(xp, rp, ring.shape[0], ring.shape[1], ip, pp, wp, bp,
                                           batch, tokens, channels, kernel, int(dilation), op, ep,
                                           _stream_of(device))
    _check(status, "engram_ple_conv_step")
    return out


# ----------------------------------------------------------------- embedding --
@_streamed
def engram_embed(tokens, table, scale=1.0, out=None, out_dtype=torch.bfloat16, err_count=None):
    """scale * table[tokens]: tokens int64 of any shape (-1: a zero row), table bf16
    [table_rows, channels]; out of out_dtype (bf16 or fp32) [..., channels]."""
    device = _device_of(tokens, "tokens")
    if table.dim() != 2:
        raise ValueError("table must be [table_rows, channels]")
    table_rows, channels = table.shape
    n = tokens.numel()
    tp = _tensor(tokens, torch.int64, n, "tokens", device)
    bp = _tensor(table, torch.bfloat16, table.numel(), "table", device)
    if out is None:
        out = torch.empty((*tokens.shape, channels), dtype=out_dtype, device=device)
    if out.dtype not in _TYPES:
        raise TypeError(f"out must be bfloat16 or float32, is {out.dtype}")
    op = _tensor(out, out.dtype, n * channels, "out", device)
    ep = _optional(err_count, torch.int64, 1, "err_count", device)
    with _on(device):
        status = _lib.engram_embed(tp, n, bp, table_rows, channels, float(scale),
                                   _TYPES[out.dtype], op, ep, _stream_of(device))
    _check(status, "engram_embed")
    return out


@_streamed
def engram_embed_grad(tokens, grads, table_rows, scale=1.0, grad_table=None,
                      grad_dtype=torch.float32, accumulate=False, workspace=None, err_count=None):
    """The gradient of engram_embed into the whole table [table_rows, channels] (grad_dtype:
    fp32 or bf16): rows without a token get zeros; with accumulate (fp32, grad_table given) the
    sums are added to the rows that have tokens."""
    device = _device_of(grads, "grads")
    n = tokens.numel()
    channels = grads.shape[-1] if grads.dim() else 0
    if channels < 1:
        raise ValueError("grads must be [..., channels]")
    tp = _tensor(tokens, torch.int64, n, "tokens", device)
    gp = _tensor(grads, torch.bfloat16, n * channels, "grads", device)
    if grad_table is None:
        if accumulate:
            raise ValueError("accumulate needs grad_table")
        grad_table = torch.empty((table_rows, channels), dtype=grad_dtype, device=device)
    if grad_table.dtype not in _TYPES:
        raise TypeError(f"grad_table must be bfloat16 or float32, is {grad_table.dtype}")
    op = _tensor(grad_table, grad_table.dtype, table_rows * channels, "grad_table", device)
    ep = _optional(err_count, torch.int64, 1, "err_count", device)
    need = _lib.engram_embed_grad_workspace(n, channels, table_rows)
    workspace = _bytes(workspace, need, device, "engram_embed_grad_workspace")
    with _on(device):
        status = _lib.engram_embed_grad(tp, n, gp, channels, float(scale), table_rows,
                                        _TYPES[grad_table.dtype], int(accumulate), op,
                                        workspace.data_ptr(), workspace.numel(), ep,
                                        _stream_of(device))
    _check(status, "engram_embed_grad")
    return grad_table
