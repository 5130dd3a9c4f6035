"""Arguments of the layer operators that have the right number of values in another
order of axes are refused: they would be read as other rows.  Flattened ones are not."""
import pytest
import torch

from gram_hashed_embedding_amd import workloads
from tests.gpu_helpers import needs_gpu

pytestmark = needs_gpu
L = pytest.importorskip("gram_hashed_embedding_amd.layer")

B, S, C, G = 2, 6, 64, 4
N = C // G
F32, I8, I64 = torch.float32, torch.int8, torch.int64


def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype, device="cuda")


def draw(*shape):
    return workloads.make_bf16(shape, sum(shape), "cuda")


# ------------------------------------------------------------- residual norm --
@pytest.mark.parametrize("name,shape", [("y", (S, B, C)), ("y", (C, B * S)), ("out", (S, B, C)),
                                        ("gate", (S, B, G)), ("gate", (S, B, C)),
                                        ("y_codes", (S, B, C)), ("y_codes", (C, B * S)),
                                        ("y_codes", (S, B, G, N))])
def test_norm_backward_refuses(name, shape):
    args = dict(out=z(B, S, C), rstd_post=z(B * S, G, dtype=F32), rstd_next=z(B * S, G, dtype=F32),
                y=z(B, S, C), gate=z(B, S, G), w_next=z(C), groups=G)
    if name == "y_codes":
        args.update(y=None, y_scales=z(B * S, G, dtype=F32), y_codes=z(*shape, dtype=I8))
    else:
        args[name] = z(*shape)
    with pytest.raises(ValueError):
        L.engram_residual_norm_backward(z(B, S, C), z(B, S, C), **args)


@pytest.mark.parametrize("shape", [(S, B, G), (S, B, C)])
def test_norm_refuses_a_gate(shape):
    with pytest.raises(ValueError):
        L.engram_residual_norm(z(B, S, C), z(B, S, C), gate=z(*shape), groups=G)


def test_norm_takes_flattened_rows():
    """Codes and gates of rows [B * S, ...], as the forward and a product of rows leave them;
    and every argument flattened, or only the rows that the shape is taken of."""
    r, y, gate, d = draw(B, S, C), draw(B, S, C), draw(B, S, G), draw(B, S, C)
    f, flat = (L.engram_residual_norm(r, y, gate=g, groups=G, save_codes=True)
               for g in (gate, gate.view(-1, G)))
    assert torch.equal(f.out, flat.out) and f.y_codes.shape == (B * S, C)
    stats = dict(rstd_post=f.rstd_post, groups=G)
    codes = [L.engram_residual_norm_backward(dd, y_codes=c, y_scales=f.y_scales, gate=g, **stats)
             for c in (f.y_codes, f.y_codes.view(B, S, C), f.y_codes.view(-1, N),
                       f.y_codes.view(B, S, G, N), f.y_codes.view(-1))
             for g in (gate, gate.view(-1, G)) for dd in (d, d.view(-1, C))]
    plain = [L.engram_residual_norm_backward(dd, y=yy, gate=gate, **stats)
             for dd in (d, d.view(-1, C)) for yy in (y, y.view(-1, C))]
    for results in (codes, plain):
        for b in results[1:]:
            for k in ("y", "residual", "gate"):
                assert torch.equal(getattr(b, k).view(-1), getattr(results[0], k).view(-1))


# --------------------------------------------------------------- convolution --
def conv_backward(**other):
    return L.engram_ple_conv_backward(z(B, S, C), z(C, 4), 1, **{"x": z(B, S, C), **other})


@pytest.mark.parametrize("shape", [(S, B, C), (B, C, S), (C, B * S)])
def test_conv_backward_refuses_x(shape):
    with pytest.raises(ValueError):
        conv_backward(x=z(*shape))


@pytest.mark.parametrize("shape,width", [((S, B, C), 0), ((C, B * S), 0), ((S, B, G, N), N),
                                         ((B * S * G // 2, 2 * N), N)])
def test_conv_backward_refuses_codes(shape, width):
    with pytest.raises(ValueError):
        conv_backward(x=None, x_codes=z(*shape, dtype=I8), code_width=width,
                      x_scales=z(B * S * (G if width else 1), dtype=F32))


def test_conv_backward_refuses_segment_ids():
    with pytest.raises(ValueError):
        conv_backward(seq_ids=z(S, B, dtype=I64))


def test_conv_backward_takes_flattened_rows():
    x, g, w = draw(B, S, C), draw(B, S, C), draw(C, 4)
    ids = torch.tensor([[0, 0, 1, 1, 1, 2], [3, 3, 3, 3, 4, 4]], device="cuda")
    codes, scales = L.engram_act_encode(x.view(-1, N))
    kept = [dict(x_codes=c, x_scales=scales, code_width=N)
            for c in (codes, codes.view(B, S, C), codes.view(B * S, C), codes.view(B, S, G, N),
                      codes.view(-1))]
    for forms in (kept, [dict(x=x), dict(x=x.view(-1, C))]):
        results = [L.engram_ple_conv_backward(g, w, 2, seq_ids=i, **k)
                   for k in forms for i in (ids, ids.view(-1))]
        for b in results[1:]:
            assert torch.equal(b.weight, results[0].weight) and torch.equal(b.x, results[0].x)


# ----------------------------------------------------------------- embedding --
@pytest.mark.parametrize("tokens,grads", [((S, B), (B, S, C)), ((B, S), (S, B, C))])
def test_embed_grad_refuses_other_axes(tokens, grads):
    with pytest.raises(ValueError):
        L.engram_embed_grad(z(*tokens, dtype=I64), z(*grads), 9)


def test_embed_grad_refuses_a_table_of_other_rows():
    with pytest.raises(ValueError):
        L.engram_embed_grad(z(B, S, dtype=I64), z(B, S, C), 9, grad_table=z(C, 9, dtype=F32))


def test_embed_grad_takes_flattened_rows():
    t, g = torch.arange(B * S, device="cuda").view(B, S) % 7, draw(B, S, C)
    want = L.engram_embed_grad(t, g, 9)
    for a in (t, t.view(-1), t.view(-1, 1)):
        for b in (g, g.view(-1, C)):
            assert torch.equal(L.engram_embed_grad(a, b, 9), want)
    table = torch.empty((9 * C,), device="cuda")
    assert torch.equal(L.engram_embed_grad(t, g, 9, grad_table=table).view(9, C), want)


# --------------------------------------------------------------------- sizes --
@pytest.mark.parametrize("dilation", [2 ** 32 + 1, 2 ** 31, -2 ** 32 + 1])
def test_dilations_past_32_bits_are_refused(dilation):
    """Their low halves are dilations."""
    with pytest.raises(ValueError):
        L.engram_ple_conv_backward(z(1, 3, 8), z(8, 4), dilation, x=z(1, 3, 8))
    with pytest.raises(ValueError):
        L.engram_ple_conv_step(z(1, 8), z(1, 3, 8), z(8, 4), dilation, z(1, dtype=I64))


def test_the_largest_dilation():
    """No tap but a position's own lies inside the row."""
    g, x, w = draw(1, 5, 8), draw(1, 5, 8), draw(8, 4)
    b = L.engram_ple_conv_backward(g, w, 2 ** 31 - 1, x=x)
    assert torch.equal(b.x, (g.float() * w[:, 3].float()).to(torch.bfloat16))
    assert bool((b.weight[:, :3] == 0).all()) and bool((b.weight[:, 3] != 0).any())
