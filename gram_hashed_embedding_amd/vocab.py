"""Python binding of the operators at the vocabulary's end of the layer
(include/engram_vocab.h; ctypes, the C ABI's names): distillation from a
teacher's top logits, the selection of a beam search, and the reordering of the
decoding states after it.

As ``layer.py``: argument marshalling only, every step in the library's HIP
kernels, asynchronous on the current stream of the tensors' device, or on the
stream of that device passed as ``stream``.  Outputs and workspaces are torch
tensors, allocated when they are not passed in.  What each call computes stands
in the header.
"""
from __future__ import annotations

import ctypes
import math
import struct
from typing import NamedTuple, Optional

import torch

from . import abi
from .abi import BEAM_MAX, DISTILL_MAX_TOP, FORK_MAX_POOLS  # noqa: F401
from .engram import EngramError, _lib
from .layer import (_BAD_SIZE, _TYPES, _bytes, _check_rows, _device_of, _optional, _run,
                    _stream_of, _streamed, _tensor)

abi.declare_vocab(_lib)


def _row_stride(t, what):
    """The distance, in values, of the rows [..., n] of `t`, which lie equally far apart."""
    shape, stride = t.shape, t.stride()
    if shape[-1] > 1 and stride[-1] != 1:
        raise ValueError(f"{what} must have adjacent values along its last axis")
    rows = [(n, s) for n, s in zip(shape[:-1], stride[:-1]) if n != 1]
    for (_, outer), (n, inner) in zip(rows, rows[1:]):
        if outer != n * inner:
            raise ValueError(f"{what} must have rows that lie equally far apart")
    if not rows or t.numel() == 0:
        return shape[-1]
    if rows[-1][1] < shape[-1]:
        raise ValueError(f"{what} must have rows that do not overlap")
    return rows[-1][1]


def _logits(t, what):
    """(device index, rows, vocab, stride, type) of device logits [..., vocab]."""
    _, index = _device_of(t, what)
    kind = _TYPES.get(t.dtype)
    if kind is None:
        raise TypeError(f"{what} must be bfloat16 or float32, is {t.dtype}")
    shape = t.shape
    vocab = shape[-1] if shape else 0
    if vocab < 1:
        raise ValueError(f"{what} must be [..., vocab]")
    stride = vocab if t.is_contiguous() else _row_stride(t, what)
    return index, t.numel() // vocab, vocab, stride, kind


# New tensors are made from a given one where that has the shape already: the call that takes a
# shape, a type and a device takes twice as long, and a small call's time is its host time.
def _new_rows(like, lead, logits):
    """fp32 [lead], as `like` where that is so already."""
    if like is not None and like.shape == lead:
        return torch.empty_like(like)
    return logits.new_empty(lead, dtype=torch.float32)


def _workspace(workspace, need, like, index, what):
    """The address and size of a workspace of at least `need` bytes; the tensor too, which has to
    live until the call was made."""
    if need == _BAD_SIZE:
        raise EngramError(abi.ENGRAM_EINVAL, what)
    if workspace is None:
        workspace = like.new_empty((need + 15) // 4, dtype=torch.float32)
        return workspace, workspace.data_ptr(), need
    workspace = _bytes(workspace, need, like.device, index, what)
    return workspace, workspace.data_ptr(), workspace.numel()


# -------------------------------------------------------------- distillation --
class Distill(NamedTuple):
    """What engram_distill wrote; lse_rest with rest, grad with grad_loss."""
    loss: torch.Tensor
    lse: torch.Tensor
    lse_rest: Optional[torch.Tensor]
    grad: Optional[torch.Tensor]


# struct engram_distill_args, packed in one go
_DISTILL = struct.Struct("=5qd4i" + 13 * "Q")
assert _DISTILL.size == ctypes.sizeof(abi.EngramDistillArgs)


def _entries(logits, ids, teacher, teacher_lse, rows, index):
    """(top, the teacher's type, addresses of ids, teacher and its lse)."""
    lead = logits.shape[:-1]
    if not isinstance(ids, torch.Tensor) or not isinstance(teacher, torch.Tensor):
        raise TypeError("ids and teacher must be device (cuda) tensors")
    top = ids.shape[-1] if ids.dim() else 0
    if top < 1 or teacher.dim() < 1 or teacher.shape[-1] != top:
        raise ValueError("ids and teacher must be [..., top]")
    kind = _TYPES.get(teacher.dtype)
    if kind is None:
        raise TypeError(f"teacher must be bfloat16 or float32, is {teacher.dtype}")
    ids_p = _tensor(ids, torch.int64, rows * top, "ids", index)
    teacher_p = _tensor(teacher, teacher.dtype, rows * top, "teacher", index)
    for t, what in ((ids, "ids"), (teacher, "teacher")):
        if t.shape[:-1] != lead:
            _check_rows(t, lead, (top,), what)
    return top, kind, ids_p, teacher_p, _per_row(teacher_lse, lead, rows, "teacher_lse", index)


def _per_row(t, lead, rows, what, index):
    """The address of one float a row, or 0 for None."""
    if t is None:
        return 0
    p = _tensor(t, torch.float32, rows, what, index)
    if t.shape != lead:
        _check_rows(t, lead, (), what)
    return p


def _grad_of(logits, grad, index):
    """(the gradient's tensor, its stride): a new one, or one of the logits' shape."""
    if grad is None:
        grad = torch.empty(logits.shape, dtype=logits.dtype, device=logits.device)
        return grad, grad.shape[-1]
    if not isinstance(grad, torch.Tensor) or not grad.is_cuda:
        raise TypeError("grad must be a device (cuda) tensor")
    if grad.dtype != logits.dtype or grad.shape != logits.shape:
        raise ValueError("grad must have the shape and type of logits")
    if grad.get_device() != index:
        raise ValueError(f"grad must be on cuda:{index}, is on {grad.device}")
    return grad, _row_stride(grad, "grad")


@_streamed
def engram_distill(logits, ids, teacher, *, teacher_lse=None, rest=False, temperature=1.0,
                   grad_loss=None, grad=None, loss=None, lse=None, lse_rest=None,
                   workspace=None, err_count=None):
    """The loss of each row of logits (bf16 or fp32 [..., vocab]; rows may lie apart) against
    the teacher's entries: ids int64 [..., top] (-1: unused) and logits teacher (bf16 or fp32
    [..., top]).  Without teacher_lse the teacher's probabilities are a softmax over the
    entries; with it (fp32 [...]) they are the true ones, and with rest what they leave is one
    class more.  With grad_loss (fp32 [...], the loss' gradients; 0 where a row does not count)
    the gradient is written too, into grad, which may be logits."""
    index, rows, vocab, stride, kind = _logits(logits, "logits")
    lead = logits.shape[:-1]
    top, teacher_kind, ids_p, teacher_p, tlse_p = _entries(logits, ids, teacher, teacher_lse,
                                                           rows, index)
    if rest and teacher_lse is None:
        raise ValueError("rest needs teacher_lse")
    if lse_rest is not None and not rest:
        raise ValueError("lse_rest needs rest")
    weight_p = grad_p = grad_stride = rest_p = ws_p = 0
    if grad_loss is not None:
        weight_p = _per_row(grad_loss, lead, rows, "grad_loss", index)
        grad, grad_stride = _grad_of(logits, grad, index)
        grad_p = grad.data_ptr()
    elif grad is not None:
        raise ValueError("grad needs grad_loss")
    if loss is None:
        loss = _new_rows(grad_loss if grad_loss is not None else teacher_lse, lead, logits)
        loss_p = loss.data_ptr()
    else:
        loss_p = _per_row(loss, lead, rows, "loss", index)
    if lse is None:
        lse = _new_rows(loss, lead, logits)
        lse_p = lse.data_ptr()
    else:
        lse_p = _per_row(lse, lead, rows, "lse", index)
    if rest:
        if lse_rest is None:
            lse_rest = _new_rows(loss, lead, logits)
        rest_p = _per_row(lse_rest, lead, rows, "lse_rest", index)
    err_p = 0 if err_count is None else _tensor(err_count, torch.int64, 1, "err_count", index)
    size = _lib.engram_distill_workspace(rows, vocab, 1 if grad_p else 0)
    if size:
        workspace, ws_p, size = _workspace(workspace, size, logits, index,
                                           "engram_distill_workspace")
    _run(index, "engram_distill", _DISTILL.pack(
        rows, vocab, top, stride, grad_stride, temperature, kind, teacher_kind, int(bool(rest)), 0,
        logits.data_ptr(), ids_p, teacher_p, tlse_p, weight_p, loss_p, lse_p, rest_p, grad_p,
        err_p, ws_p, size, _stream_of(index)))
    return Distill(loss, lse, lse_rest, grad)


@_streamed
def engram_distill_backward(grad_loss, logits, ids, teacher, lse, *, teacher_lse=None,
                            lse_rest=None, temperature=1.0, grad=None, err_count=None):
    """The gradient of engram_distill's loss from the lse that it wrote (and lse_rest, which
    stands for rest), for grad_loss fp32 [...] (0: the row does not count).  grad may be
    logits.  Rows whose lse or lse_rest fp32 holds too coarsely (64 or more in size, for bf16
    logits 1024) are summed again, which takes two to six times as long."""
    index, rows, vocab, stride, kind = _logits(logits, "logits")
    lead = logits.shape[:-1]
    top, teacher_kind, ids_p, teacher_p, tlse_p = _entries(logits, ids, teacher, teacher_lse,
                                                           rows, index)
    if lse_rest is not None and teacher_lse is None:
        raise ValueError("lse_rest needs teacher_lse")
    if grad_loss is None or lse is None:
        raise TypeError("grad_loss and lse must be device (cuda) tensors")
    weight_p = _per_row(grad_loss, lead, rows, "grad_loss", index)
    lse_p = _per_row(lse, lead, rows, "lse", index)
    rest_p = _per_row(lse_rest, lead, rows, "lse_rest", index)
    grad, grad_stride = _grad_of(logits, grad, index)
    err_p = _optional(err_count, torch.int64, 1, "err_count", index)
    _run(index, "engram_distill_backward", _DISTILL.pack(
        rows, vocab, top, stride, grad_stride, temperature, kind, teacher_kind,
        int(lse_rest is not None), 0, logits.data_ptr(), ids_p, teacher_p, tlse_p, weight_p, 0,
        lse_p, rest_p, grad.data_ptr(), err_p, 0, 0, _stream_of(index)))
    return grad


def engram_distill_workspace(rows, vocab, grad=False) -> int:
    need = _lib.engram_distill_workspace(rows, vocab, int(bool(grad)))
    if need == _BAD_SIZE:
        raise EngramError(abi.ENGRAM_EINVAL, "engram_distill_workspace")
    return need


# --------------------------------------------------------------- beam search --
class Beams(NamedTuple):
    """What engram_beam_select chose, [batch, count] each."""
    scores: torch.Tensor
    parents: torch.Tensor
    tokens: torch.Tensor
    finished: torch.Tensor


@_streamed
def engram_beam_select(logits, scores, count=None, *, finished=None, eos=-1, out_scores=None,
                       parents=None, tokens=None, out_finished=None, workspace=None):
    """The `count` (default: beams) best continuations of each sequence's beams: logits bf16 or
    fp32 [batch * beams, vocab] or [batch, beams, vocab] (rows may lie apart), scores fp32
    [batch, beams] the beams' log-probabilities so far (-inf: no beam), finished bool [batch,
    beams] those that `eos` has ended.  Entries that nothing is left for have score -inf and
    parent and token -1.  With as many as there are beams out_scores may be scores and
    out_finished finished."""
    index, rows, vocab, stride, kind = _logits(logits, "logits")
    if not isinstance(scores, torch.Tensor) or scores.dim() != 2:
        raise ValueError("scores must be [batch, beams]")
    batch, beams = lead = scores.shape
    if rows != batch * beams or logits.dim() not in (2, 3) or \
            (logits.dim() == 3 and logits.shape[:2] != lead):
        raise ValueError("logits must be [batch * beams, vocab] or [batch, beams, vocab]")
    count = beams if count is None else int(count)
    if not 1 <= count <= BEAM_MAX or not 1 <= beams <= BEAM_MAX:
        raise ValueError(f"beams and count must be 1 to {BEAM_MAX}")
    scores_p = _tensor(scores, torch.float32, rows, "scores", index)
    finished_p = 0
    if finished is not None:
        finished_p = _tensor(finished, torch.bool, rows, "finished", index)
        if finished.shape != lead:
            _check_rows(finished, lead, (), "finished")
    shape = (batch, count)
    if out_scores is None:
        out_scores = torch.empty_like(scores) if count == beams else scores.new_empty(shape)
        os_p = out_scores.data_ptr()
    else:
        os_p = _chosen(out_scores, torch.float32, shape, "out_scores", index)
    if parents is None:
        parents = torch.empty_like(out_scores, dtype=torch.int64)
        op_p = parents.data_ptr()
    else:
        op_p = _chosen(parents, torch.int64, shape, "parents", index)
    if tokens is None:
        tokens = torch.empty_like(out_scores, dtype=torch.int64)
        ot_p = tokens.data_ptr()
    else:
        ot_p = _chosen(tokens, torch.int64, shape, "tokens", index)
    if out_finished is None:
        out_finished = torch.empty_like(out_scores, dtype=torch.bool)
        of_p = out_finished.data_ptr()
    else:
        of_p = _chosen(out_finished, torch.bool, shape, "out_finished", index)
    need = _lib.engram_beam_select_workspace(batch, beams, vocab)
    workspace, ws_p, size = _workspace(workspace, need, scores, index,
                                       "engram_beam_select_workspace")
    _run(index, "engram_beam_select", logits.data_ptr(), kind, stride, scores_p, finished_p,
         int(eos), batch, beams, vocab, count, os_p, op_p, ot_p, of_p, ws_p, size,
         _stream_of(index))
    return Beams(out_scores, parents, tokens, out_finished)


def _chosen(t, dtype, shape, what, index):
    """The address of an output [batch, count]."""
    p = _tensor(t, dtype, shape[0] * shape[1], what, index)
    if t.shape != shape:
        _check_rows(t, shape, (), what)
    return p


def engram_beam_select_workspace(batch, beams, vocab) -> int:
    need = _lib.engram_beam_select_workspace(batch, beams, vocab)
    if need == _BAD_SIZE:
        raise EngramError(abi.ENGRAM_EINVAL, "engram_beam_select_workspace")
    return need


_LISTS = [struct.Struct(f"={n}Q") for n in range(FORK_MAX_POOLS + 1)]  # 64-bit numbers


class Fork(NamedTuple):
    """What engram_beam_fork wrote: the new beams' slots and (with history) histories."""
    slots: torch.Tensor
    history: Optional[torch.Tensor]


@_streamed
def engram_beam_fork(parents, pools=(), *, slots=None, tokens=None, history=None, new_len=None,
                     new_slots=None, new_history=None, err_count=None):
    """The states of the beams that a selection kept: parents int64 [batch, beams] (-1:
    unused), pools up to 8 tensors [slot_count, ...] of states (16-byte multiples a slot;
    rings of engram_ple_conv_step, say), in which those that are needed twice are copied,
    slots int64 [batch, beams] of the old beams (None: 0, 1, ...).  With tokens int64 [batch,
    beams] and history int64 [batch, beams, n] also each new beam's history: the last new_len
    (default n) of its parent's and its token."""
    _, index = _device_of(parents, "parents")
    if parents.dim() != 2:
        raise ValueError("parents must be [batch, beams]")
    batch, beams = parents.shape
    n = batch * beams
    parents_p = _tensor(parents, torch.int64, n, "parents", index)
    slots_p = _optional(slots, torch.int64, n, "slots", index)
    if slots is not None and slots.shape != parents.shape:
        _check_rows(slots, parents.shape, (), "slots")
    pools = (pools,) if isinstance(pools, torch.Tensor) else tuple(pools)
    if len(pools) > FORK_MAX_POOLS:
        raise ValueError(f"at most {FORK_MAX_POOLS} pools")
    count, addresses, sizes = 0, [], []
    for i, pool in enumerate(pools):
        if not isinstance(pool, torch.Tensor) or pool.dim() < 1:
            raise TypeError("a pool must be a device (cuda) tensor [slot_count, ...]")
        numel = pool.numel()
        addresses.append(_tensor(pool, pool.dtype, numel, "a pool", index))
        slots_here = pool.shape[0]
        if i and slots_here != count:
            raise ValueError("pools must have the same number of slots")
        count = slots_here
        if slots_here:
            sizes.append(numel // slots_here * pool.element_size())
        else:
            sizes.append(math.prod(pool.shape[1:]) * pool.element_size())
    if new_slots is None:
        new_slots = torch.empty_like(parents)
        new_p = new_slots.data_ptr()
    else:
        new_p = _tensor(new_slots, torch.int64, n, "new_slots", index)
        if new_slots.shape != parents.shape:
            _check_rows(new_slots, parents.shape, (), "new_slots")
    tokens_p = history_p = out_p = have = 0
    if history is not None:
        if tokens is None:
            raise ValueError("history goes with tokens")
        if history.dim() != 3 or history.shape[:2] != parents.shape:
            raise ValueError("history must be [batch, beams, n]")
        have = history.shape[2]
        new_len = have if new_len is None else int(new_len)
        if not 1 <= new_len <= have + 1:
            raise ValueError("new_len must be 1 to the history's length and one")
        tokens_p = _tensor(tokens, torch.int64, n, "tokens", index)
        if tokens.shape != parents.shape:
            _check_rows(tokens, parents.shape, (), "tokens")
        history_p = _tensor(history, torch.int64, n * have, "history", index)
        if new_history is None:
            new_history = (torch.empty_like(history) if new_len == have
                           else history.new_empty((batch, beams, new_len)))
            out_p = new_history.data_ptr()
        else:
            out_p = _tensor(new_history, torch.int64, n * new_len, "new_history", index)
            if new_history.shape != (batch, beams, new_len):
                _check_rows(new_history, (batch, beams, new_len), (new_len,), "new_history")
    elif tokens is not None or new_history is not None or new_len is not None:
        raise ValueError("tokens, new_history and new_len need history")
    err_p = _optional(err_count, torch.int64, 1, "err_count", index)
    lists = _LISTS[len(pools)]
    _run(index, "engram_beam_fork", parents_p, slots_p, batch, beams, lists.pack(*addresses),
         lists.pack(*sizes), len(pools), count, new_p, tokens_p, history_p, have, out_p,
         new_len or 0, err_p, _stream_of(index))
    return Fork(new_slots, new_history)
