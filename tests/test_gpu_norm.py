"""The residual norm and its backward on the GPU against the 64-bit reference.

Bounds, in fp32 roundings (2^-24 of the sum of the terms' magnitudes), from the
kernels' sums: a group's mean is at most 32 additions in a lane and 10 across
lanes and wavefronts, halved by the square root; the gate's exponential adds
1.5 |gate| + 2.  So 64 cover a forward value and the stream's gradient, 160 a
gradient behind the second mean; a sum over rows adds at most 256 in a lane and
64 across a block: 512.  bf16 outputs add half a step (and the step that a
value next to a rounding boundary may take)."""
import numpy as np
import pytest
import torch

from gram_hashed_embedding_amd import workloads
from tests import layer_reference as ref
from tests.gpu_helpers import needs_gpu, release

pytestmark = needs_gpu
L = pytest.importorskip("gram_hashed_embedding_amd.layer")

FORWARD, DEEP, SUMS = 64, 160, 512
EPS = 1e-5


def make(rows, channels, groups, gate, residual, seed, weights=True):
    rt = torch.float32 if residual == "f32" else torch.bfloat16
    n = (rows, channels)
    v = dict(residual=workloads.make_bf16(n, seed, "cuda", std=2.0).to(rt),
             y=workloads.make_bf16(n, seed + 1, "cuda", std=0.5),
             d_out=workloads.make_bf16(n, seed + 2, "cuda", std=1.0).to(rt),
             d_next=workloads.make_bf16(n, seed + 3, "cuda", std=1.0))
    if rt == torch.float32:  # not only values that bf16 holds
        v["residual"] = v["residual"] * 1.2345
    width = {None: 0, "group": groups, "channel": channels}[gate]
    v["gate"] = workloads.make_bf16((rows, width), seed + 4, "cuda", std=1.5) if width else None
    for i, k in enumerate(("w_post", "scale", "w_next")):
        v[k] = workloads.make_bf16((channels,), seed + 5 + i, "cuda", std=0.5) if weights else None
    return v


def reference_inputs(v, channels):
    one = np.ones(channels)
    return {k: ref.f64(v[k]) if v[k] is not None else (one if k in ("w_post", "scale") else None)
            for k in v}


def check_forward(v, groups, alpha, f, y=True):
    h = reference_inputs(v, v["residual"].shape[1])
    rounding = ref.BF16_ROUNDING if v["residual"].dtype == torch.bfloat16 else 0.0
    out = h["residual"]
    if y:
        out, u, mag = ref.norm_out(h["residual"], h["y"], h["gate"], h["w_post"], h["scale"],
                                   groups, EPS, alpha)
        ref.within(ref.f64(f.out), out, mag, FORWARD, rounding)
        ref.within(ref.f64(f.rstd_post), u, u, FORWARD)
        out = ref.f64(f.out)  # the next norm is of what was stored
    if v["w_next"] is not None:
        nxt, s = ref.norm_next(out, h["w_next"], groups, EPS)
        ref.within(ref.f64(f.next), nxt, np.abs(nxt), FORWARD, ref.BF16_ROUNDING)
        ref.within(ref.f64(f.rstd_next), s, s, FORWARD)


def check_backward(v, groups, alpha, f, b, y, d_out=True):
    """y: the values the backward read as y, or None without a branch."""
    h = reference_inputs(v, v["residual"].shape[1])
    stream = ref.f64(f.out) if f.out is not None else h["residual"]
    grads, mags = ref.norm_grads(
        h["d_out"] if d_out else None, h["d_next"], stream,
        None if f.rstd_next is None else ref.f64(f.rstd_next), y,
        None if f.rstd_post is None else ref.f64(f.rstd_post), h["gate"], h["w_post"],
        h["scale"], h["w_next"], groups, alpha)
    bf = ref.BF16_ROUNDING
    steps = dict(residual=FORWARD, y=DEEP, gate=DEEP, w_post=SUMS, scale=SUMS, w_next=SUMS)
    for k, got in b._asdict().items():
        if got is None:
            continue
        rounding = bf if got.dtype == torch.bfloat16 else 0.0
        want = grads[k] if grads[k].shape == tuple(got.shape) else grads[k].reshape(got.shape)
        ref.within(ref.f64(got), want, mags[k].reshape(want.shape), steps[k], rounding)


def weights(v):
    return dict(gate=v["gate"], w_post=v["w_post"], scale=v["scale"], w_next=v["w_next"])


def run_case(rows, channels, groups, gate, residual, codes, seed, with_weights=True, alpha=0.75):
    v = make(rows, channels, groups, gate, residual, seed, with_weights)
    if not with_weights:
        v["w_next"] = workloads.make_bf16((channels,), seed + 9, "cuda", std=0.5)
    f = L.engram_residual_norm(v["residual"], v["y"], groups=groups, eps=EPS,
                               residual_scale=alpha, save_codes=codes, next_codes=codes,
                               **weights(v))
    kept, y = dict(y=v["y"]), ref.f64(v["y"])
    if codes:
        n = channels // groups
        for values, c, s in ((v["y"], f.y_codes, f.y_scales), (f.next, f.next_codes,
                                                               f.next_scales)):
            want_c, want_s = ref.encode(values.float().cpu().numpy().reshape(-1, n))
            assert np.array_equal(c.cpu().numpy().reshape(-1, n), want_c)
            assert np.array_equal(s.cpu().numpy().reshape(want_s.shape), want_s)
        kept = dict(y_codes=f.y_codes, y_scales=f.y_scales)
        y = ref.decode(*ref.encode(y.reshape(-1, n))).reshape(y.shape).astype(np.float64)
    b = L.engram_residual_norm_backward(v["d_out"], v["d_next"], out=f.out,
                                        rstd_post=f.rstd_post, rstd_next=f.rstd_next,
                                        groups=groups, residual_scale=alpha, **kept, **weights(v))
    torch.cuda.synchronize()
    check_forward(v, groups, alpha, f)
    check_backward(v, groups, alpha, f, b, y)


# every way a group is held: 4 to 64 lanes, several chunks a lane, whole blocks
SHAPES = [(1, 8, 1), (3, 32, 1), (70, 120, 5), (9, 128, 1), (33, 1024, 16), (65, 6144, 24),
          (5, 504, 1), (2, 1536, 3), (4097, 520, 1), (1400, 3000, 3), (4098, 1040, 1),
          (4099, 2048, 1), (1026, 6144, 1),
          (7, 1000, 1), (8, 6144, 1), (40, 4104, 1), (1030, 4096, 1), (1025, 8192, 1),
          (5, 8200, 1), (3, 16384, 1), (2, 32768, 2), (700, 64, 1), (1, 2048, 64)]


@pytest.mark.parametrize("rows,channels,groups", SHAPES)
@pytest.mark.parametrize("gate,residual,codes", [("group", "bf16", True), ("channel", "f32", False),
                                                 (None, "f32", True)])
def test_shapes(rows, channels, groups, gate, residual, codes):
    run_case(rows, channels, groups, gate, residual, codes, rows * 7 + channels)
    release()


@pytest.mark.parametrize("gate", [None, "group", "channel"])
def test_without_weights(gate):
    run_case(130, 384, 3, gate, "bf16", False, 5, with_weights=False, alpha=-1.5)


@pytest.mark.parametrize("residual", ["bf16", "f32"])
@pytest.mark.parametrize("rows,channels,groups", [(1, 8, 1), (37, 520, 1), (300, 1024, 4)])
def test_norm_before_a_block(rows, channels, groups, residual):
    """Without a block's output: the norm of the residual, and its backward with and without a
    gradient of the residual itself."""
    v = make(rows, channels, groups, None, residual, rows)
    v["w_post"] = v["scale"] = v["y"] = None
    f = L.engram_residual_norm(v["residual"], w_next=v["w_next"], groups=groups, eps=EPS)
    assert f.out is None and f.rstd_post is None
    check_forward(v, groups, 1.0, f, y=False)
    for d_out in (v["d_out"], None):
        b = L.engram_residual_norm_backward(d_out, v["d_next"], out=v["residual"],
                                            rstd_next=f.rstd_next, w_next=v["w_next"],
                                            groups=groups)
        assert b.y is None and b.gate is None and b.w_post is None
        check_backward(v, groups, 1.0, f, b, None, d_out is not None)


def test_without_a_next_norm():
    v = make(50, 768, 3, "group", "bf16", 8)
    v["w_next"] = v["d_next"] = None
    f = L.engram_residual_norm(v["residual"], v["y"], groups=3, eps=EPS, **weights(v))
    assert f.next is None and f.rstd_next is None
    check_forward(v, 3, 1.0, f)
    b = L.engram_residual_norm_backward(v["d_out"], y=v["y"], rstd_post=f.rstd_post, groups=3,
                                        **weights(v))
    assert b.w_next is None
    check_backward(v, 3, 1.0, f, b, ref.f64(v["y"]))


def test_many_rows_of_one_column():
    """Sums over more rows than one lane adds in fp32 (they go on in fp64)."""
    run_case(400_003, 8, 1, "group", "f32", False, 3)
    release()


def test_gradient_against_differences_of_the_forward():
    """The kernel's gradients along a direction against differences of the 64-bit forward."""
    rows, channels, groups, alpha = 12, 256, 2, 0.75
    v = make(rows, channels, groups, "channel", "f32", 77)
    f = L.engram_residual_norm(v["residual"], v["y"], groups=groups, eps=EPS,
                               residual_scale=alpha, **weights(v))
    b = L.engram_residual_norm_backward(v["d_out"], v["d_next"], out=f.out, y=v["y"],
                                        rstd_post=f.rstd_post, rstd_next=f.rstd_next,
                                        groups=groups, residual_scale=alpha, **weights(v))
    h = reference_inputs(v, channels)
    rng = np.random.default_rng(1)
    for k in ("residual", "y", "gate", "w_post", "scale", "w_next"):
        direction = rng.normal(size=h[k].shape)

        def loss(x):
            a = {**h, k: x}
            out, _, _ = ref.norm_out(a["residual"], a["y"], a["gate"], a["w_post"], a["scale"],
                                     groups, EPS, alpha)
            nxt, _ = ref.norm_next(out, a["w_next"], groups, EPS)
            return (out * h["d_out"]).sum() + (nxt * h["d_next"]).sum()

        step = 1e-5
        want = (loss(h[k] + step * direction) - loss(h[k] - step * direction)) / (2 * step)
        got = ref.f64(getattr(b, k))
        # each value is off by its type's half step (bf16: 2^-8) and roundings that add up at
        # random; 6 standard deviations
        part = 2.0 ** -8 if getattr(b, k).dtype == torch.bfloat16 else 2.0 ** -15
        slack = 6 * part * np.sqrt(((got * direction) ** 2).sum()) + 1e-5 * (1 + abs(want))
        assert abs((got * direction).sum() - want) < slack, k


def test_rows_of_zeros():
    """A group of zeros: its branch is zero, its reciprocal root 1 / sqrt(eps)."""
    v = make(6, 128, 2, "group", "f32", 4)
    v["y"][2] = 0
    v["residual"][2:4] = 0
    v["y"][3, :64] = 0
    f = L.engram_residual_norm(v["residual"], v["y"], groups=2, eps=EPS, save_codes=True,
                               **weights(v))
    b = L.engram_residual_norm_backward(v["d_out"], v["d_next"], out=f.out, y_codes=f.y_codes,
                                        y_scales=f.y_scales, rstd_post=f.rstd_post,
                                        rstd_next=f.rstd_next, groups=2, **weights(v))
    assert bool((f.out[2] == 0).all()) and bool((f.next[2] == 0).all())
    assert bool((f.y_codes[2] == 0).all()) and bool((f.y_scales[2] == 0).all())
    check_forward(v, 2, 1.0, f)
    y = ref.f64(v["y"]).astype(np.float32).reshape(-1, 64)
    check_backward(v, 2, 1.0, f, b, ref.decode(*ref.encode(y)).reshape(6, 128).astype(float))


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("rows,channels,groups", [(40, 512, 8), (9, 2048, 1), (5, 9000, 1)])
def test_non_finite_values_stay_in_their_group(bad, rows, channels, groups):
    """One bad value makes its group of its row non-finite and changes no other bit."""
    v = make(rows, channels, groups, "group", "f32", 6)
    clean = L.engram_residual_norm(v["residual"], v["y"], groups=groups, eps=EPS, save_codes=True,
                                   **weights(v))
    n, row = channels // groups, rows // 2
    group = groups - 1
    v["y"][row, group * n + 3] = bad
    f = L.engram_residual_norm(v["residual"], v["y"], groups=groups, eps=EPS, save_codes=True,
                               **weights(v))
    mask = torch.ones((rows, groups), dtype=torch.bool, device="cuda")
    mask[row, group] = False
    for got, want in ((f.out, clean.out), (f.next, clean.next)):
        got, want = got.view(rows, groups, n), want.view(rows, groups, n)
        assert torch.equal(got[mask], want[mask])
    assert not bool(torch.isfinite(f.out.view(rows, groups, n)[row, group]).all())
    blocks = L.code_blocks(n)
    s = f.y_scales.view(rows, groups, blocks)
    assert bool(torch.isnan(s[row, group, 0])) and bool(torch.isfinite(s[mask]).all())
    assert bool((f.y_codes.view(rows, groups, n)[row, group, :128] == 0).all())
    gate_grad = L.engram_residual_norm_backward(
        v["d_out"], v["d_next"], out=f.out, y=v["y"], rstd_post=f.rstd_post,
        rstd_next=f.rstd_next, groups=groups, **weights(v))
    assert bool(torch.isfinite(gate_grad.y.view(rows, groups, n)[mask]).all())


@pytest.mark.parametrize("gate", ["group", "channel"])
def test_extreme_gates(gate):
    """Gates at infinity and at the type's ends shut or open exactly, with no gradient."""
    v = make(8, 128, 2, gate, "f32", 9)
    ends = [float("-inf"), float("inf"), torch.finfo(torch.bfloat16).min,
            torch.finfo(torch.bfloat16).max]
    for i, e in enumerate(ends):
        v["gate"][i] = e
    f = L.engram_residual_norm(v["residual"], v["y"], groups=2, eps=EPS, **weights(v))
    b = L.engram_residual_norm_backward(v["d_out"], v["d_next"], out=f.out, y=v["y"],
                                        rstd_post=f.rstd_post, rstd_next=f.rstd_next, groups=2,
                                        **weights(v))
    for i in (0, 2):
        assert torch.equal(f.out[i], v["residual"][i]) and bool((b.y[i] == 0).all())
    assert bool((b.gate[:4] == 0).all()) and bool((b.gate[4:] != 0).any())
    check_forward(v, 2, 1.0, f)
    check_backward(v, 2, 1.0, f, b, ref.f64(v["y"]))


def test_in_place_and_repeated():
    """out over the residual, the gradient over grad_out, on another stream: the same bits; two
    runs give the same bits."""
    v = make(3000, 1536, 6, "channel", "bf16", 10)
    args = dict(groups=6, eps=EPS, residual_scale=0.5, **weights(v))
    f = L.engram_residual_norm(v["residual"], v["y"], **args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    over = v["residual"].clone()
    side.wait_stream(torch.cuda.current_stream())
    g = L.engram_residual_norm(over, v["y"], out=over, stream=side, **args)
    torch.cuda.current_stream().wait_stream(side)
    assert g.out is over and torch.equal(g.out, f.out) and torch.equal(g.next, f.next)
    back = dict(out=f.out, y=v["y"], rstd_post=f.rstd_post, rstd_next=f.rstd_next, groups=6,
                residual_scale=0.5, **weights(v))
    b = L.engram_residual_norm_backward(v["d_out"], v["d_next"], **back)
    again = L.engram_residual_norm_backward(v["d_out"], v["d_next"], **back)
    for x, y in zip(b, again):
        assert torch.equal(x, y)
    over = v["d_out"].clone()
    c = L.engram_residual_norm_backward(over, v["d_next"], grad_residual=over, **back)
    assert c.residual is over
    for x, y in zip(b, c):
        assert torch.equal(x, y)


def test_no_rows():
    v = make(0, 64, 2, "group", "bf16", 1)
    f = L.engram_residual_norm(v["residual"], v["y"], groups=2, **weights(v))
    assert f.out.shape == (0, 64)
    b = L.engram_residual_norm_backward(v["d_out"], v["d_next"], out=f.out, y=v["y"],
                                        rstd_post=f.rstd_post, rstd_next=f.rstd_next, groups=2,
                                        **weights(v))
    assert b.residual.shape == (0, 64)
    for k in (b.w_post, b.scale, b.w_next):
        assert bool((k == 0).all())


def test_offsets_past_32_bits():
    """The last rows of an array of more than 2^31 values: the bits of the rows alone."""
    rows, channels = 2 ** 31 // 8192 + 6, 8192
    print(f"residual norm of [{rows}, {channels}]", flush=True)
    tail = make(8, channels, 32, "group", "bf16", 12)
    big = {k: torch.zeros((rows, *tail[k].shape[1:]), dtype=tail[k].dtype, device="cuda")
           for k in ("residual", "y", "gate", "d_out", "d_next")}
    for k in big:
        big[k][-8:] = tail[k]
    v = {**tail, **big}
    f, g = (L.engram_residual_norm(x["residual"], x["y"], groups=32, save_codes=True,
                                   **weights(x)) for x in (v, tail))
    for k in f._fields:
        if getattr(f, k) is not None:
            assert torch.equal(getattr(f, k)[-8:], getattr(g, k)), k
    b, c = (L.engram_residual_norm_backward(
        x["d_out"], x["d_next"], out=h.out, rstd_post=h.rstd_post, rstd_next=h.rstd_next,
        y_codes=h.y_codes, y_scales=h.y_scales, groups=32, **weights(x))
        for x, h in ((v, f), (tail, g)))
    for k in ("residual", "y", "gate"):
        assert torch.equal(getattr(b, k)[-8:], getattr(c, k)), k
    del f, g, b, c, big, v
    release()
