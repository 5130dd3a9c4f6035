"""The PLE convolution's gradients on the GPU against the 64-bit reference.

Bounds: an input's gradient is at most 16 products added in turn (18 roundings)
and one rounding to bf16.  The weight's and the bias's are fp32 sums of at most
1024 positions a lane (other shapes than the register window's: of a slice,
here at most 240), then fp64: 1026 roundings of the sum of magnitudes."""
import numpy as np
import pytest
import torch

from gram_hashed_embedding_amd import engram as E
from gram_hashed_embedding_amd import workloads
from tests import layer_reference as ref
from tests.gpu_helpers import dev, needs_gpu, release

pytestmark = needs_gpu
L = pytest.importorskip("gram_hashed_embedding_amd.layer")

STEPS = dict(x=18, halo=18, weight=1026, bias=1026)


def inputs(B, S, C, K, seed, halo_len=0, seg_mean=None):
    x = workloads.make_bf16((B, S, C), seed, "cuda")
    g = workloads.make_bf16((B, S, C), seed + 1, "cuda")
    w = workloads.make_bf16((C, K), seed + 2, "cuda", std=0.5)
    halo = workloads.make_bf16((B, halo_len, C), seed + 3, "cuda") if halo_len else None
    seg = workloads.random_segments((B, halo_len + S), seg_mean, seed) if seg_mean else None
    return x, g, w, halo, seg


def compare(b, g, x, w, d, seg, halo):
    grads, mags = ref.conv_grads(ref.f64(g), x, ref.f64(w), d, seg,
                                 None if halo is None else ref.f64(halo))
    for k, got in b._asdict().items():
        if got is not None:
            rounding = ref.BF16_ROUNDING if got.dtype == torch.bfloat16 else 0.0
            ref.within(ref.f64(got), grads[k], mags[k], STEPS[k], rounding)


def check(B, S, C, K, d, seed, halo_len=0, seg_mean=None, codes=False, width=0):
    x, g, w, halo, seg = inputs(B, S, C, K, seed, halo_len, seg_mean)
    ids = None if seg is None else dev(seg)
    if codes:
        cw = width or C
        c, s = L.engram_act_encode(x.view(-1, cw))
        kept = dict(x_codes=c, x_scales=s, code_width=width)
        values = ref.decode(c.cpu().numpy(), s.cpu().numpy()).reshape(B, S, C).astype(float)
    else:
        kept, values = dict(x=x), ref.f64(x)
    b = L.engram_ple_conv_backward(g, w, d, seq_ids=ids, halo=halo, **kept)
    torch.cuda.synchronize()
    assert (b.halo is not None) == (halo_len > 0)
    compare(b, g, values, w, d, seg, halo)
    return b


@pytest.mark.parametrize("d", range(1, 9))
@pytest.mark.parametrize("seg_mean,codes", [(None, False), (3, False), (40, True)])
def test_kernel4_every_dilation(d, seg_mean, codes):
    check(2, 77, 48, 4, d, 10 * d, seg_mean=seg_mean, codes=codes)


@pytest.mark.parametrize("S", [1, 2, 7, 8, 9, 31, 33, 150])
@pytest.mark.parametrize("C", [8, 264, 1032])
@pytest.mark.parametrize("codes", [False, True])
def test_shapes(S, C, codes):
    """Lengths around a tile and a slice, channels around a wave's 256."""
    check(2, S, C, 4, 3, S * 7 + C, seg_mean=20, codes=codes)


@pytest.mark.parametrize("halo_len,seg_mean", [(9, None), (9, 5), (12, 4), (3, 7), (1, None),
                                               (70, 30)])
@pytest.mark.parametrize("codes", [False, True])
def test_halo(halo_len, seg_mean, codes):
    """The context-parallel form: the halo's own gradient, a halo longer than any tap reaches
    and than a slice, and one shorter than the history."""
    check(2, 50, 40, 4, 3, 300 + halo_len, halo_len=halo_len, seg_mean=seg_mean, codes=codes)


@pytest.mark.parametrize("K,d", [(1, 1), (3, 2), (5, 3), (4, 9), (2, 12), (16, 1), (2, 100)])
@pytest.mark.parametrize("codes", [False, True])
def test_other_kernel_sizes(K, d, codes):
    check(2, 60, 16, K, d, K * 31 + d, halo_len=5, seg_mean=9, codes=codes)


@pytest.mark.parametrize("K,d,S,halo_len,seg_mean", [(3, 300, 1500, 0, 700), (2, 70, 2300, 90, 90),
                                                     (4, 9, 1200, 27, 40), (3, 2000, 1500, 0, 300),
                                                     (2, 1, 70, 200, None)])
def test_other_shapes_over_many_slices(K, d, S, halo_len, seg_mean):
    """Taps that reach past slices and boundaries, and a halo of several slices."""
    check(1, S, 8, K, d, K + d, halo_len=halo_len, seg_mean=seg_mean)


@pytest.mark.parametrize("C,width", [(512, 64), (400, 200), (1024, 256)])
def test_codes_of_groups(C, width):
    """Codes made group by group (as the norm before the convolution makes them)."""
    check(2, 40, C, 4, 2, C, seg_mean=11, codes=True, width=width)


def test_many_slices():
    """A row longer than a slice, in several batches: the slices' sums are joined."""
    check(3, 4500, 8, 4, 4, 5, halo_len=12, seg_mean=600)


def test_a_split_row_gives_the_whole_rows_gradients():
    """Two context-parallel halves: the second's halo gradient belongs to the first's last
    positions, the weight's gradients add up."""
    x, g, w, _, seg = inputs(2, 64, 64, 4, 9, seg_mean=15)
    ids = dev(seg)
    whole = L.engram_ple_conv_backward(g, w, 3, x=x, seq_ids=ids)
    parts = [(x[:, :30], g[:, :30], ids[:, :30], None),
             (x[:, 30:], g[:, 30:], ids[:, 21:], x[:, 21:30])]
    a, b = (L.engram_ple_conv_backward(gg.contiguous(), w, 3, x=xx.contiguous(),
                                       seq_ids=ii.contiguous(),
                                       halo=None if hh is None else hh.contiguous())
            for xx, gg, ii, hh in parts)
    assert torch.equal(b.x, whole.x[:, 30:])
    joined = a.x.double()
    joined[:, 21:] += b.halo.double()
    grads, mags = ref.conv_grads(ref.f64(g), ref.f64(x), ref.f64(w), 3, seg)
    # two bf16 roundings instead of one
    ref.within(joined.cpu().numpy(), grads["x"][:, :30], mags["x"][:, :30], 18 + 2 ** 17)
    for k in ("weight", "bias"):
        ref.within(ref.f64(getattr(a, k)) + ref.f64(getattr(b, k)), grads[k], mags[k], STEPS[k])


def test_gradient_against_differences_of_the_forward():
    x, g, w, halo, seg = inputs(2, 40, 16, 4, 21, halo_len=6, seg_mean=9)
    b = L.engram_ple_conv_backward(g, w, 2, x=x, seq_ids=dev(seg), halo=halo)
    h = dict(x=ref.f64(x), weight=ref.f64(w), halo=ref.f64(halo), bias=np.zeros(16))
    rng = np.random.default_rng(2)
    for k in h:
        direction = rng.normal(size=h[k].shape)

        def loss(v):
            a = {**h, k: v}
            return (ref.f64(g) * ref.conv_forward(a["x"], a["weight"], 2, a["bias"], seg,
                                                  a["halo"])).sum()

        want = (loss(h[k] + direction) - loss(h[k] - direction)) / 2  # it is linear
        got = ref.f64(getattr(b, k))
        part = 2.0 ** -8 if getattr(b, k).dtype == torch.bfloat16 else 2.0 ** -15
        slack = 6 * part * np.sqrt(((got * direction) ** 2).sum()) + 1e-9 * (1 + abs(want))
        assert abs((got * direction).sum() - want) < slack, k


def test_non_finite_values_stay_behind_boundaries():
    """A NaN in one segment's gradient, input or halo reaches no other segment's values; and a
    position whose every later tap is cut adds nothing for those taps."""
    B, S, C = 1, 48, 8
    x, g, w, halo, _ = inputs(B, S, C, 4, 33, halo_len=6)
    seg = np.zeros((B, 6 + S), np.int64)
    seg[:, 6:] = 1          # the halo is another segment
    seg[:, 6 + 20:] = 2
    halo[:] = float("nan")
    g[:, 20:] = float("nan")
    b = L.engram_ple_conv_backward(g, w, 2, x=x, seq_ids=dev(seg), halo=halo)
    assert bool((b.halo == 0).all()) and bool(torch.isfinite(b.x[:, :20]).all())
    assert bool(torch.isnan(b.x[:, 20:]).all())
    g[:, 20:] = 1.0
    x[:, 19] = float("nan")  # its segment's last position: only its own tap counts
    b = L.engram_ple_conv_backward(g, w, 2, x=x, seq_ids=dev(seg), halo=halo)
    assert bool(torch.isnan(b.weight[:, 3]).all()) and bool(torch.isfinite(b.weight[:, :3]).all())
    assert bool(torch.isfinite(b.bias).all()) and bool(torch.isfinite(b.x).all())


def test_only_what_is_asked_for():
    x, g, w, halo, seg = inputs(2, 50, 24, 4, 40, halo_len=4, seg_mean=9)
    full = L.engram_ple_conv_backward(g, w, 3, x=x, seq_ids=dev(seg), halo=halo)
    only = L.engram_ple_conv_backward(g, w, 3, seq_ids=dev(seg), halo=halo, need_weight=False,
                                      need_bias=False)
    assert only.weight is None and only.bias is None
    assert torch.equal(only.x, full.x) and torch.equal(only.halo, full.halo)
    sums = L.engram_ple_conv_backward(g, w, 3, x=x, seq_ids=dev(seg), halo=halo, need_x=False)
    assert sums.x is None and sums.halo is None
    assert torch.equal(sums.weight, full.weight) and torch.equal(sums.bias, full.bias)
    bias = L.engram_ple_conv_backward(g, w, 3, halo=halo, need_x=False, need_weight=False)
    ref.within(ref.f64(bias.bias), ref.f64(g).sum((0, 1)), np.abs(ref.f64(g)).sum((0, 1)), 1026)


def test_empty():
    for B, S in ((0, 5), (3, 0)):
        g = torch.empty((B, S, 16), dtype=torch.bfloat16, device="cuda")
        w = torch.ones((16, 4), dtype=torch.bfloat16, device="cuda")
        halo = torch.ones((B, 7, 16), dtype=torch.bfloat16, device="cuda")
        b = L.engram_ple_conv_backward(g, w, 2, x=g, halo=halo)
        assert b.x.shape == g.shape and bool((b.halo == 0).all())
        assert bool((b.weight == 0).all()) and bool((b.bias == 0).all())


def test_repeated_runs_give_the_same_bits():
    x, g, w, _, seg = inputs(4, 1500, 520, 4, 50, seg_mean=100)
    a = L.engram_ple_conv_backward(g, w, 4, x=x, seq_ids=dev(seg))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b = L.engram_ple_conv_backward(g, w, 4, x=x, seq_ids=dev(seg), stream=side)
    torch.cuda.synchronize()
    for p, q in zip(a[:3], b[:3]):
        assert torch.equal(p, q)


def test_transpose_of_the_forward_at_the_workloads_shape():
    """<g, conv(x)> = <conv^T(g), x> on the benchmark's [8, 8192, 8192] (dilation 4, packed
    documents), and the weight's gradient through <weight, grad_weight>."""
    wl = workloads.ple_conv()
    B, S, C = wl.batch, wl.seq, wl.channels
    x = workloads.make_bf16((B, S, C), 1, "cuda")
    g = workloads.make_bf16((B, S, C), 2, "cuda")
    w = workloads.make_bf16((C, 4), 3, "cuda", std=0.5)
    seg = dev(wl.segments())
    out = E.engram_ple_conv(x, w, wl.dilation, seq_ids=seg)
    b = L.engram_ple_conv_backward(g, w, wl.dilation, x=x, seq_ids=seg)

    def dot(p, q):
        return sum(float((p[i].double() * q[i].double()).sum()) for i in range(p.shape[0]))

    forward = dot(g, out)
    # rounding errors of 2^-9 a value at random: 6 standard deviations of each side
    size = 6 * 2.0 ** -9 * (dot(out * out, g * g) ** 0.5 + dot(b.x * b.x, x * x) ** 0.5)
    assert abs(dot(b.x, x) - forward) < size
    assert abs(float((b.weight.double() * w.double()).sum()) - forward) < size
    del x, g, out, b
    release()


def test_offsets_past_32_bits():
    S, C = 2 ** 31 // 8192 + 40, 8192
    print(f"convolution's gradients of [1, {S}, {C}]", flush=True)
    x, g, w, _, _ = inputs(1, 64, C, 4, 60)
    big_x, big_g = (torch.zeros((1, S, C), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    big_x[:, -64:], big_g[:, -64:] = x, g
    a = L.engram_ple_conv_backward(big_g, w, 4, x=big_x)
    b = L.engram_ple_conv_backward(g, w, 4, x=x)
    assert torch.equal(a.x[:, -64:], b.x)
    # the same terms in other slices, beside zeros; 12 positions before it are zero in x
    ref.within(ref.f64(a.weight), ref.f64(b.weight), np.full((C, 4), 64.0 * 16), 130)
    del big_x, big_g, a
    release()
