"""Host-side checks of the vocabulary operators' entry points (include/engram_vocab.h), against
any loaded copy of them: the HIP build or the CPU build of the same host code under sanitizers.
No case reaches a kernel; every device pointer is a fake address.  Plain ctypes, no torch."""
import ctypes
import struct

from gram_hashed_embedding_amd import abi

OK, INVALID, ALIGN, WORKSPACE = (abi.ENGRAM_OK, abi.ENGRAM_EINVAL, abi.ENGRAM_EALIGN,
                                 abi.ENGRAM_EWORKSPACE)
A, B, C = 0x10000, 0x20000, 0x30000  # aligned, never dereferenced
ODD = 0x10008
BAD_SIZE = (1 << 64) - 1


def distill(call, **fields):
    """A full call with some fields replaced."""
    a = abi.EngramDistillArgs(rows=4, vocab=50, top=3, logits_stride=64, grad_stride=50,
                              temperature=1.0, d_logits=A, d_ids=A, d_teacher=A, d_teacher_lse=A,
                              rest=1, d_grad_loss=A + 64, d_loss=C, d_lse=C + 64,
                              d_lse_rest=C + 128, d_grad=B)
    for k, v in fields.items():
        setattr(a, k, v)
    return call(ctypes.byref(a))


SHARED = [
    dict(rows=-1), dict(vocab=0), dict(vocab=(1 << 30) + 1, logits_stride=1 << 31), dict(top=0),
    dict(top=abi.DISTILL_MAX_TOP + 1), dict(logits_stride=49), dict(grad_stride=49),
    dict(rows=1 << 58), dict(logits_type=2), dict(logits_type=-1), dict(teacher_type=2),
    dict(rest=2), dict(rest=-1), dict(reserved=1), dict(temperature=0.0), dict(temperature=-1.0),
    dict(temperature=float("nan")), dict(temperature=float("inf")), dict(temperature=2.0 ** -65),
    dict(temperature=2.0 ** 65), dict(d_logits=None), dict(d_ids=None), dict(d_teacher=None),
    dict(d_teacher_lse=None), dict(rest=0), dict(d_grad_loss=None),
    dict(d_grad=A),  # in place with another stride
]


def case_distill_rejects(lib):
    for fields in SHARED + [dict(d_grad=None), dict(d_loss=A), dict(d_lse=A + 64),
                            dict(d_lse_rest=A), dict(d_lse=C), dict(d_lse_rest=C),
                            dict(d_lse_rest=C + 64)]:
        assert distill(lib.engram_distill, **fields) == INVALID, fields
    assert distill(lib.engram_distill, d_loss=None, d_lse=None, d_lse_rest=None, d_grad=None,
                   d_grad_loss=None) == INVALID
    assert lib.engram_distill(None) == INVALID


def case_distill_backward_rejects(lib):
    call = lib.engram_distill_backward
    for fields in SHARED:
        assert distill(call, **{"d_loss": None, **fields}) == INVALID, fields
    for fields in (dict(), dict(d_loss=None, d_grad=None, d_grad_loss=None),
                   dict(d_loss=None, d_lse=None), dict(d_loss=None, d_lse_rest=None)):
        assert distill(call, **fields) == INVALID, fields
    assert call(None) == INVALID


def case_distill_nothing_to_do(lib):
    assert distill(lib.engram_distill, rows=0, d_logits=None) == OK
    assert distill(lib.engram_distill_backward, rows=0, d_loss=None) == OK
    assert distill(lib.engram_distill, rows=0, vocab=0) == INVALID


def case_distill_workspace(lib):
    need = lib.engram_distill_workspace
    assert need(4, 50, 1) == 0 and need(0, 1 << 20, 1) == 0
    for args in ((-1, 5, 0), (1, 0, 0), (1, 5, 2), (1, 5, -1), (1, (1 << 30) + 1, 0),
                 (1 << 60, 8, 0)):
        assert need(*args) == BAD_SIZE, args
    # a vocabulary that no block marks
    assert need(4, 1 << 20, 0) > 0
    big = dict(vocab=1 << 20, logits_stride=1 << 20, grad_stride=1 << 20)
    size = need(4, 1 << 20, 1)
    call = lib.engram_distill
    assert distill(call, **big) == WORKSPACE
    assert distill(call, **big, d_workspace=C, workspace_bytes=size - 1) == WORKSPACE
    assert distill(call, **big, d_workspace=ODD, workspace_bytes=size) == WORKSPACE


def select(call, **fields):
    a = dict(logits=A, type=abi.BF16, stride=64, scores=A, finished=A, eos=3, batch=2, beams=3,
             vocab=50, count=4, out_scores=B, parents=B, tokens=B, out_finished=B, workspace=C,
             size=1 << 20, stream=None)
    a.update(fields)
    return call(*a.values())


def case_select_rejects(lib):
    call = lib.engram_beam_select
    for fields in (dict(type=2), dict(stride=49), dict(batch=-1), dict(beams=0),
                   dict(beams=abi.BEAM_MAX + 1), dict(vocab=0), dict(vocab=1 << 31, stride=1 << 31),
                   dict(count=0), dict(count=abi.BEAM_MAX + 1), dict(eos=-1), dict(eos=-2),
                   dict(eos=50), dict(logits=None), dict(scores=None), dict(out_scores=None),
                   dict(parents=None), dict(tokens=None), dict(batch=1 << 60),
                   dict(out_scores=A), dict(out_finished=A)):
        assert select(call, **fields) == INVALID, fields
    for fields in (dict(workspace=None), dict(workspace=ODD), dict(size=16)):
        assert select(call, **fields) == WORKSPACE, fields
    assert select(call, batch=0, logits=None, workspace=None) == OK
    need = lib.engram_beam_select_workspace
    assert need(0, 3, 50) == 0 and need(2, 3, 50) > 0
    for args in ((-1, 3, 50), (1, 0, 50), (1, 65, 50), (1, 3, 0), (1 << 60, 3, 50)):
        assert need(*args) == BAD_SIZE, args


def fork(call, held=((B, 64),), **fields):
    a = dict(parents=A, slots=C, batch=2, beams=3,
             pools=struct.pack(f"={len(held)}Q", *(p or 0 for p, _ in held)),
             sizes=struct.pack(f"={len(held)}q", *(n for _, n in held)), n=len(held),
             slot_count=8, new_slots=A + 64, tokens=A, history=A, history_len=4,
             new_history=B + 64, new_len=4, err=None, stream=None)
    a.update(fields)
    return call(*a.values())


def case_fork_rejects(lib):
    call = lib.engram_beam_fork
    for fields in (dict(parents=None), dict(new_slots=None), dict(new_slots=C), dict(new_slots=A),
                   dict(batch=-1), dict(beams=0), dict(beams=abi.BEAM_MAX + 1), dict(slot_count=-1), dict(n=-1),
                   dict(n=abi.FORK_MAX_POOLS + 1), dict(pools=None), dict(sizes=None),
                   dict(tokens=None), dict(history=None), dict(new_history=None),
                   dict(new_history=A), dict(new_len=0), dict(new_len=6), dict(history_len=-1),
                   dict(slots=None, slot_count=5), dict(batch=1 << 60)):
        assert fork(call, **fields) == INVALID, fields
    for held in (((None, 64),), ((B, 0),), ((B, 24),), ((B, -16),), ((B, 1 << 62),),
                  ((B, 64), (B, 32))):
        assert fork(call, held=held) == INVALID, held
    assert fork(call, held=((B + 8, 64),)) == ALIGN
    assert fork(call, batch=0, parents=None, new_slots=None) == OK


CASES = [v for k, v in sorted(globals().items()) if k.startswith("case_")]
