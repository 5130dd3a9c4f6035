"""The residual norm with one wide group a row and blocks that take several rows, in
the forms with one norm only (the norm before a block; a last block's branch) and with
both, against the 64-bit reference.  Bounds as in test_gpu_norm.py."""
import numpy as np
import pytest
import torch

from tests import layer_reference as ref
from tests import norm_shapes
from tests.gpu_helpers import needs_gpu, release
from tests.test_gpu_norm import EPS, L, check_backward, check_forward, make, weights

pytestmark = needs_gpu

FORMS = ["next only", "branch only", "both"]


def inputs(rows, channels, residual, form, seed):
    """test_gpu_norm's, each row of its own size, without what the form lacks."""
    v = make(rows, channels, 1, None if form == "next only" else "group", residual, seed)
    size = torch.exp2((torch.arange(rows, device="cuda") % 7).float() - 3).view(-1, 1)
    for k in ("residual", "y"):
        v[k] = (v[k].float() * size).to(v[k].dtype)
    if form == "next only":
        v["y"] = v["w_post"] = v["scale"] = None
    if form == "branch only":
        v["w_next"] = v["d_next"] = None
    return v


def forward(v, rows=slice(None)):
    gate = None if v["gate"] is None else v["gate"][rows]
    return L.engram_residual_norm(v["residual"][rows], None if v["y"] is None else v["y"][rows],
                                  eps=EPS, **{**weights(v), "gate": gate})


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("residual", ["bf16", "f32"])
@pytest.mark.parametrize("rows,channels", norm_shapes.FORWARD)
def test_forward(rows, channels, residual, form):
    """All rows: the bits that the same rows give in calls with a block to each; some of them
    against the reference."""
    print(f"forward [{rows}, {channels}] {residual}, {form}", flush=True)
    v = inputs(rows, channels, residual, form, rows)
    f, again = forward(v), forward(v)
    step = 4000  # rows of a call: a block each, of the same lanes and chunks
    for r in range(0, rows, step):
        part = slice(r, min(rows, r + step)) if rows - r >= step else slice(rows - step, rows)
        g = forward(v, part)
        for k in ("out", "next", "rstd_post", "rstd_next"):
            whole = getattr(f, k)
            if whole is not None:
                assert torch.equal(whole[part], getattr(g, k)), (k, part)
                assert torch.equal(whole, getattr(again, k)), k
    some = torch.cat([torch.arange(0, rows, 500), torch.arange(rows - 20, rows)]).cuda()
    per_row = ("residual", "y", "gate", "d_out", "d_next")
    few = {k: t[some] if t is not None and k in per_row else t for k, t in v.items()}
    got = L.ResidualNorm(*(None if t is None else t[some] for t in f[:4]))
    check_forward(few, 1, 1.0, got, y=v["y"] is not None)
    del v, f, again, g
    release()


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("residual", ["bf16", "f32"])
@pytest.mark.parametrize("rows,channels", norm_shapes.BACKWARD)
def test_backward(rows, channels, residual, form):
    print(f"backward [{rows}, {channels}] {residual}, {form}", flush=True)
    v = inputs(rows, channels, residual, form, rows)
    f = forward(v)
    kept = dict(out=v["residual"] if f.out is None else f.out, y=v["y"], rstd_post=f.rstd_post,
                rstd_next=f.rstd_next)
    b, again = (L.engram_residual_norm_backward(v["d_out"], v["d_next"], **kept, **weights(v))
                for _ in range(2))
    for x, y in zip(b, again):
        assert x is None or torch.equal(x, y)
    check_backward(v, 1, 1.0, f, b, None if v["y"] is None else ref.f64(v["y"]))
    assert np.isfinite(ref.f64(b.residual)).all()
    release()
