"""Host-side checks of the layer operators' entry points (include/
engram_layer.h), against any loaded copy of them: the HIP build or the CPU
build of the same host code under sanitizers.  No case reaches a kernel; every
device pointer is a fake address.  Plain ctypes, no torch."""
import ctypes

from gram_hashed_embedding_amd import abi

OK, INVALID, ALIGN, WORKSPACE = (abi.ENGRAM_OK, abi.ENGRAM_EINVAL, abi.ENGRAM_EALIGN,
                                 abi.ENGRAM_EWORKSPACE)
A = 0x10000                # aligned, never dereferenced
ODD = 0x10008
BAD_SIZE = (1 << 64) - 1
HUGE = 1 << 62


def norm(call, **fields):
    """A full forward (or backward) call with some fields replaced."""
    a = abi.EngramNormArgs(rows=4, channels=64, groups=2, gate_width=2, eps=1e-6,
                           residual_scale=1.0, d_gate=A, d_w_post=A, d_scale=A, d_w_next=A)
    for k in ("d_out", "d_rstd_post", "d_rstd_next"):
        setattr(a, k, A)
    for k, v in fields.items():
        setattr(a, k, v)
    return call(ctypes.byref(a))


FORWARD = dict(d_residual=A, d_y=A, d_next=A)
BACKWARD = dict(d_y=A, d_grad_out=A, d_grad_next=A, d_grad_residual=A, d_grad_y=A, d_grad_gate=A,
                d_grad_w_post=A, d_grad_scale=A, d_grad_w_next=A, d_workspace=A,
                workspace_bytes=1 << 20)

SHARED_REJECTS = [
    dict(rows=-1), dict(channels=0), dict(channels=60), dict(groups=0), dict(groups=3),
    dict(groups=16), dict(channels=1 << 31), dict(rows=1 << 60),
    dict(channels=abi.NORM_MAX_GROUP * 2 + 16, groups=2), dict(reserved=1),
    dict(residual_type=2), dict(residual_type=-1),
    dict(residual_scale=float("inf")), dict(residual_scale=float("nan")),
    dict(gate_width=3), dict(gate_width=0), dict(d_gate=None),
    dict(d_y_codes=A, d_y_scales=None), dict(d_next_scales=A, d_next_codes=None),
]
FORWARD_REJECTS = SHARED_REJECTS + [
    dict(eps=0.0), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
    dict(d_residual=None), dict(d_out=None), dict(d_next=None),
    dict(d_w_next=None), dict(d_w_next=None, d_next=None),         # rstd_next left over
    dict(d_y=None),                                                # a branch without y
    dict(d_y=None, d_out=None, d_gate=None, gate_width=0, d_w_post=None, d_scale=None,
         d_rstd_post=None, residual_scale=2.0),
]
BACKWARD_REJECTS = SHARED_REJECTS + [
    dict(d_grad_next=None), dict(d_w_next=None), dict(d_out=None), dict(d_rstd_next=None),
    dict(d_rstd_post=None), dict(d_y_codes=A, d_y_scales=A), dict(d_y=None),
    dict(d_w_post=None), dict(d_scale=None),
    dict(d_grad_out=None, d_grad_next=None, d_w_next=None, d_grad_w_next=None),
]


def case_norm_rejects(lib):
    for bad in FORWARD_REJECTS:
        assert norm(lib.engram_residual_norm, **{**FORWARD, **bad}) == INVALID, bad
    assert lib.engram_residual_norm(None) == INVALID
    for k in ("d_residual", "d_y", "d_w_post", "d_scale", "d_w_next", "d_out", "d_next"):
        assert norm(lib.engram_residual_norm, **{**FORWARD, k: ODD}) == ALIGN, k
    for k in ("d_y", "d_next"):
        codes = {f"{k}_codes": ODD, f"{k}_scales": A}
        assert norm(lib.engram_residual_norm, **FORWARD, **codes) == ALIGN, k
    assert norm(lib.engram_residual_norm, **FORWARD, gate_width=64, d_gate=ODD) == ALIGN
    assert norm(lib.engram_residual_norm, rows=0, d_gate=None) == OK


def case_norm_backward_rejects(lib):
    call = lib.engram_residual_norm_backward
    for bad in BACKWARD_REJECTS:
        assert norm(call, **{**BACKWARD, **bad}) == INVALID, bad
    assert call(None) == INVALID
    for k in BACKWARD:
        if k.startswith("d_") and k not in ("d_grad_gate", "d_workspace"):
            assert norm(call, **{**BACKWARD, k: ODD}) == ALIGN, k
    need = lib.engram_residual_norm_backward_workspace(4, 64, 2)
    assert 0 < need < 1 << 20
    for bad in (dict(d_workspace=None), dict(d_workspace=ODD), dict(workspace_bytes=need - 1)):
        assert norm(call, **{**BACKWARD, **bad}) == WORKSPACE, bad
    nothing = {k: None for k in BACKWARD if k.startswith("d_grad_")}
    assert norm(call, **{**BACKWARD, **nothing, "d_grad_out": A, "d_grad_next": A}) == OK


def case_norm_workspace(lib):
    w = lib.engram_residual_norm_backward_workspace
    for bad in ((-1, 64, 1), (4, 60, 1), (4, 64, 3), (4, 0, 1), (1 << 60, 64, 1),
                (4, 1 << 20, 1)):
        assert w(*bad) == BAD_SIZE, bad
    assert w(0, 64, 1) == 0
    # two fp32 rows for every block of rows, never many more than the rows themselves
    for rows, channels, groups in ((1, 8, 1), (100, 6144, 24), (65536, 6144, 24), (10 ** 7, 64, 1)):
        size = w(rows, channels, groups)
        assert size % (8 * channels) == 0 and 0 < size <= 8 * channels * max(rows, 1)


def case_act_rejects(lib):
    for f in (lambda *a: lib.engram_act_encode(a[0], a[3], a[4], a[1], a[2], None),
              lambda *a: lib.engram_act_decode(a[1], a[2], a[3], a[4], a[0], None)):
        for bad in ((A, A, A, -1, 64), (A, A, A, 4, 0), (A, A, A, 4, 60), (A, A, A, HUGE, 64),
                    (None, A, A, 4, 64), (A, None, A, 4, 64), (A, A, None, 4, 64)):
            assert f(*bad) == INVALID, bad
        assert f(ODD, A, A, 4, 64) == ALIGN and f(A, ODD, A, 4, 64) == ALIGN
        assert f(None, None, None, 0, 64) == OK


CONV = dict(g=A, x=A, codes=None, scales=None, width=0, halo=A, halo_len=3, seg=None, w=A, batch=2,
            seq=9, channels=16, K=4, d=2, gx=A, gh=A, gw=A, gb=A, ws=A, size=1 << 20)
CONV_REJECTS = [
    dict(batch=-1), dict(seq=-1), dict(channels=0), dict(channels=12), dict(halo_len=-1),
    dict(K=0), dict(K=17), dict(d=0), dict(seq=HUGE), dict(batch=HUGE), dict(channels=1 << 31),
    dict(width=-8), dict(width=12), dict(width=24), dict(codes=A), dict(scales=A),
    dict(codes=A, scales=A), dict(x=None), dict(halo=None), dict(halo_len=0), dict(g=None),
    dict(w=None), dict(halo_len=0, halo=None),
]


def conv(lib, **fields):
    v = {**CONV, **fields}
    return lib.engram_ple_conv_backward(
        v["g"], v["x"], v["codes"], v["scales"], v["width"], v["halo"], v["halo_len"], v["seg"],
        v["w"], v["batch"], v["seq"], v["channels"], v["K"], v["d"], v["gx"], v["gh"], v["gw"],
        v["gb"], v["ws"], v["size"], None)


def case_conv_backward_rejects(lib):
    for bad in CONV_REJECTS:
        assert conv(lib, **bad) == INVALID, bad
    for k in ("g", "x", "halo", "w", "gx", "gh", "gw", "gb"):
        assert conv(lib, **{k: ODD}) == ALIGN, k
    assert conv(lib, x=None, codes=ODD, scales=A) == ALIGN
    w = lib.engram_ple_conv_backward_workspace
    need = w(2, 9, 3, 16, 4, 2)
    assert need % (5 * 16 * 4) == 0 and 0 < need < 1 << 20
    for bad in (dict(ws=None), dict(ws=ODD), dict(size=need - 1)):
        assert conv(lib, **bad) == WORKSPACE, bad
    assert conv(lib, gx=None, gh=None, gw=None, gb=None, ws=None) == OK
    for bad in ((-1, 9, 3, 16, 4, 2), (2, 9, 3, 12, 4, 2), (2, 9, 3, 16, 17, 2),
                (2, HUGE, 3, 16, 4, 2), (2, 9, HUGE, 16, 4, 2)):
        assert w(*bad) == BAD_SIZE, bad
    assert w(0, 9, 3, 16, 4, 2) == 0


STEP = dict(x=A, ring=A, count=8, rows=9, ids=A, pos=A, w=A, b=A, batch=4, tokens=1, channels=16,
            K=4, d=3, out=A)
STEP_REJECTS = [
    dict(batch=-1), dict(tokens=-1), dict(channels=12), dict(K=0), dict(K=17), dict(d=0),
    dict(rows=8), dict(rows=0, K=1), dict(count=-1), dict(count=HUGE), dict(ids=None, count=3),
    dict(x=None), dict(ring=None), dict(pos=None), dict(w=None), dict(tokens=HUGE),
]


def step(lib, **fields):
    v = {**STEP, **fields}
    return lib.engram_ple_conv_step(v["x"], v["ring"], v["count"], v["rows"], v["ids"], v["pos"],
                                    v["w"], v["b"], v["batch"], v["tokens"], v["channels"], v["K"],
                                    v["d"], v["out"], None, None)


def case_conv_step_rejects(lib):
    for bad in STEP_REJECTS:
        assert step(lib, **bad) == INVALID, bad
    for k in ("x", "ring", "w", "b", "out"):
        assert step(lib, **{k: ODD}) == ALIGN, k
    assert step(lib, batch=0, x=None, ids=None, pos=None) == OK
    assert step(lib, tokens=0, x=None) == OK


def case_embed_rejects(lib):
    def e(tokens=A, n=5, table=A, rows=10, channels=16, kind=abi.BF16, out=A):
        return lib.engram_embed(tokens, n, table, rows, channels, 1.0, kind, out, None, None)
    for bad in (dict(n=-1), dict(rows=-1), dict(channels=12), dict(channels=0), dict(kind=2),
                dict(tokens=None), dict(table=None), dict(out=None), dict(n=HUGE),
                dict(rows=HUGE)):
        assert e(**bad) == INVALID, bad
    assert e(table=ODD) == ALIGN and e(out=ODD) == ALIGN
    assert e(n=0, tokens=None, out=None) == OK


def case_embed_grad_rejects(lib):
    need = lib.engram_embed_grad_workspace(500, 16, 10)
    assert need >= 500 // 64 * 16 * 8

    def e(tokens=A, n=500, grads=A, channels=16, rows=10, kind=abi.F32, acc=0, out=A, ws=A,
          size=need, given=abi.BF16):
        return lib.engram_embed_grad(tokens, n, grads, given, channels, 1.0, rows, kind, acc, out,
                                     ws, size, None, None)
    for bad in (dict(n=-1), dict(rows=-1), dict(channels=12), dict(kind=2), dict(acc=2),
                dict(acc=1, kind=abi.BF16), dict(tokens=None), dict(grads=None), dict(out=None),
                dict(n=1 << 32), dict(rows=(1 << 32) - 1),
                dict(given=2)):
        assert e(**bad) == INVALID, bad
    assert e(grads=ODD) == ALIGN and e(out=ODD) == ALIGN
    for bad in (dict(ws=None), dict(ws=ODD), dict(size=need - 1)):
        assert e(**bad) == WORKSPACE, bad
    assert e(n=0, acc=1, out=None, ws=None) == OK
    assert e(n=0, rows=0, out=None, ws=None) == OK
    for bad in ((-1, 16, 10), (500, 12, 10), (500, 16, 1 << 32), (1 << 32, 16, 10)):
        assert lib.engram_embed_grad_workspace(*bad) == BAD_SIZE, bad


CASES = [f for name, f in sorted(globals().items()) if name.startswith("case_")]
