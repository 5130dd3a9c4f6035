"""Distillation from a teacher's top logits against the definition in 64 bits: every kernel
(a block of each size to a row, rows cut into segments, gradients from the statistics), types, odd
sizes, strides and addresses, rows that a mask leaves nothing of, what does not count, and
refusals.  The tolerances are derived in vocab_reference."""
import math

import pytest
import torch

from tests import vocab_reference as R
from tests.gpu_helpers import needs_gpu

pytestmark = needs_gpu
V = pytest.importorskip("gram_hashed_embedding_amd.vocab")

BF, F32 = torch.bfloat16, torch.float32


def problem(rows, vocab, top, dtype=BF, teacher_dtype=F32, target="rest", temperature=1.0, seed=0,
            std=3.0):
    """Logits, a teacher near them, its top entries in rising rows with unused ones at the end."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, s=1.0):
        return torch.empty(shape, device="cuda").normal_(0.0, s, generator=g)

    z = normal(rows, vocab, s=std).to(dtype)
    y = z.float() * 0.8 + normal(rows, vocab, s=1.0)
    best = torch.topk(y, min(top, vocab), dim=1)
    ids = torch.full((rows, top), -1, dtype=torch.int64, device="cuda")
    values = torch.zeros((rows, top), device="cuda", dtype=teacher_dtype)
    ids[:, :best.indices.shape[1]] = best.indices
    values[:, :best.values.shape[1]] = best.values.to(teacher_dtype)
    used = torch.randint(1, top + 1, (rows, 1), generator=g, device="cuda")
    used[::2] = top
    ids = torch.where(torch.arange(top, device="cuda") < used, ids, -1)
    lse = None if target == "kept" else torch.logsumexp(y.double() / temperature, 1).float()
    weight = torch.rand(rows, generator=g, device="cuda") + 0.5
    return dict(logits=z, ids=ids, teacher=values, teacher_lse=lse, rest=target == "rest",
                temperature=temperature), weight


def reference(p, weight=None):
    return R.distill(p["logits"], p["ids"], p["teacher"], p["teacher_lse"], p["rest"],
                     p["temperature"], weight)


def forward(p, weight=None, **kw):
    return V.engram_distill(p["logits"], p["ids"], p["teacher"], teacher_lse=p["teacher_lse"],
                            rest=p["rest"], temperature=p["temperature"], grad_loss=weight, **kw)


def backward(p, weight, d, **kw):
    return V.engram_distill_backward(weight, p["logits"], p["ids"], p["teacher"], d.lse,
                                     lse_rest=d.lse_rest, teacher_lse=p["teacher_lse"],
                                     temperature=p["temperature"], **kw)


def check_all(p, weight):
    """The loss alone, loss and gradient, and the gradient from what the loss kept."""
    want = reference(p, weight)
    d = forward(p)
    assert d.grad is None and (d.lse_rest is not None) == p["rest"]
    R.check_distill(d._asdict(), want)
    R.check_distill(forward(p, weight)._asdict(), want)
    R.check_distill(dict(grad=backward(p, weight, d)), want)
    return d


@pytest.mark.parametrize("target", ["kept", "part", "rest"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("vocab", [1, 2, 7, 8, 9, 15, 100, 1003, 2048, 2049, 16383, 16384, 16385])
def test_vocabularies(vocab, dtype, target):
    p, weight = problem(5, vocab, min(6, vocab + 2), dtype, target=target, seed=vocab)
    check_all(p, weight)


# a few rows, around whole steps of a block and the lengths from which rows are cut
@pytest.mark.parametrize("rows, vocab, dtype", [
    (3, 32768, BF), (3, 32769, BF), (131, 65537, BF), (3, 81921, BF), (130, 81920, BF),
    (130, 81921, BF), (129, 163840, BF), (129, 163841, BF), (3, 16385, F32), (3, 40961, F32),
    (130, 81920, F32), (130, 81921, F32), (2, 262144, BF), (2, 262145, F32), (2, 300001, BF)])
def test_long_rows(rows, vocab, dtype):
    p, weight = problem(rows, vocab, 9, dtype, seed=vocab)
    check_all(p, weight)


@pytest.mark.parametrize("rows, vocab", [(1, 5000), (513, 3001), (1100, 2500), (2100, 700)])
def test_many_rows(rows, vocab):
    """More rows than blocks stay on the GPU."""
    p, weight = problem(rows, vocab, 7, BF, seed=rows)
    check_all(p, weight)


# rows up to 256 by blocks of 256, 512 and 1024 threads (12,000, 48,000 bytes), up to 2048 by 64
# and 256 (4000), more by 64, 128 and 256 (9000 and 20,000 with a gradient, 20,000 and 40,000
# without); with a gradient longer ones by 512 and 1024 (55,000, 110,000); gradients from the
# statistics by 64 and 256 (8192); up to 128 rows of 65,536 values or more cut, and all past 2^18
@pytest.mark.parametrize("rows, vocab, dtype", [
    (7, 4096, BF), (7, 4097, BF), (7, 6000, BF), (7, 6001, BF), (7, 24000, BF), (7, 24001, BF),
    (256, 3000, F32), (256, 3001, F32), (257, 2000, BF), (257, 2001, BF), (2048, 1000, F32),
    (2048, 1001, F32), (2049, 4500, BF), (2049, 4501, BF), (2049, 2250, F32), (2049, 2251, F32),
    (2049, 10000, BF), (2049, 10001, BF), (2049, 20000, BF), (2049, 20001, BF), (2049, 10001, F32),
    (256, 2049, BF), (257, 2049, BF), (257, 27500, BF), (257, 27501, BF), (257, 55000, BF),
    (257, 55001, BF), (257, 13750, F32), (257, 13751, F32), (257, 27500, F32), (257, 27501, F32),
    (128, 65535, BF), (128, 65536, BF), (129, 65536, BF), (128, 65537, F32), (129, 65537, F32),
    (129, 262144, BF), (129, 262145, BF), (1, 262144, F32)])
def test_rows_that_a_rule_divides(rows, vocab, dtype):
    p, weight = problem(rows, vocab, 5, dtype, seed=rows + vocab)
    check_all(p, weight)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows, vocab", [(3, 1), (3, 3), (3, 63), (3, 64), (3, 65), (3, 130),
                                         (257, 131), (2, 2049), (3, 65600), (1, 262150)])
def test_every_place_in_a_cache_line(rows, vocab, dtype):
    """Logits from every value of a cache line on, the gradient elsewhere in one; what lies
    around it stays."""
    p, weight = problem(rows, vocab, min(4, vocab), dtype, seed=vocab)
    p["ids"][0, 0], p["ids"][rows - 1, 0] = 0, vocab - 1
    want = reference(p, weight)
    z, stride = p["logits"], vocab + 3
    line = 128 // dtype.itemsize
    for first in range(line if vocab < 3000 else 5):
        wide = torch.full((first + rows * stride + line,), math.nan, dtype=dtype, device="cuda")
        p["logits"] = wide.as_strided((rows, vocab), (stride, 1), first)
        p["logits"].copy_(z)
        around = torch.full((line + rows * stride,), 7.0, dtype=dtype, device="cuda")
        at = (5 * first + 2) % line
        grad = around.as_strided((rows, vocab), (stride, 1), at)
        d = forward(p)
        R.check_distill(d._asdict(), want)
        for call in (lambda: forward(p, weight, grad=grad).grad,
                     lambda: backward(p, weight, d, grad=grad)):
            around.fill_(7.0)
            R.check_distill(dict(grad=call()), want)
            grad.fill_(7.0)
            assert bool((around == 7.0).all())


@pytest.mark.parametrize("top", [1, 2, 63, 64, 65, 255, 256, 257, 1000, 1024])
@pytest.mark.parametrize("teacher_dtype", [BF, F32])
def test_entries(top, teacher_dtype):
    p, weight = problem(4, 3000, top, BF, teacher_dtype, seed=top)
    check_all(p, weight)


@pytest.mark.parametrize("temperature", [0.25, 0.7, 1.5, 8.0, 1000.0])
@pytest.mark.parametrize("target", ["kept", "rest"])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_temperatures(temperature, target, dtype):
    p, weight = problem(6, 2500, 12, dtype, target=target, temperature=temperature, seed=3)
    check_all(p, weight)


@pytest.mark.parametrize("target", ["kept", "part", "rest"])
@pytest.mark.parametrize("vocab", [600, 70000])
def test_repeated_and_invalid_ids(target, vocab):
    p, weight = problem(8, vocab, 40, BF, target=target, seed=4)
    p["ids"][:, 20:30] = p["ids"][:, 3:13]          # twice
    p["ids"][:, 30:33] = p["ids"][:, 3:4]           # one of them five times
    p["ids"][1] = p["ids"][1, :1]                   # one id only
    p["ids"][2, 5], p["ids"][2, 6], p["ids"][3, 0] = vocab, -2, 1 << 40
    p["ids"][4] = -1                                # no target
    p["ids"][5] = vocab + 1                         # none either: 40 invalid ones
    want = reference(p, weight)
    for call in (lambda e: forward(p, err_count=e), lambda e: forward(p, weight, err_count=e)):
        err = torch.zeros(1, dtype=torch.int64, device="cuda")
        d = call(err)
        R.check_distill(d._asdict(), want)
        assert int(err) == 43
        assert d.loss[4] == 0 and d.loss[5] == 0
    err.zero_()
    grad = backward(p, weight, d, err_count=err)
    R.check_distill(dict(grad=grad), want)
    assert int(err) == 43 and not bool(grad[4:6].any())


@pytest.mark.parametrize("vocab", [900, 70000])
@pytest.mark.parametrize("kinds", [1, 7, 500])
def test_many_repeated_ids(kinds, vocab):
    p, weight = problem(5, vocab, 1000, BF, target="part", seed=kinds)
    g = torch.Generator(device="cuda").manual_seed(kinds)
    some = torch.randint(0, vocab, (kinds,), generator=g, device="cuda")
    p["ids"] = some[torch.randint(0, kinds, (5, 1000), generator=g, device="cuda")].contiguous()
    p["ids"][2, ::3] = -1
    p["teacher_lse"] = p["teacher_lse"] + 8.0
    check_all(p, weight)


MASKS = [-math.inf, torch.finfo(BF).min, torch.finfo(F32).min]


@pytest.mark.parametrize("mask", MASKS)
@pytest.mark.parametrize("target", ["kept", "part", "rest"])
@pytest.mark.parametrize("vocab", [500, 70000])
def test_masked_logits(mask, target, vocab):
    """A mask over most of a row, over all of it but one value, over the teacher's ids."""
    dtype = F32 if mask == torch.finfo(F32).min else BF
    p, weight = problem(6, vocab, 5, dtype, target=target, seed=6)
    z = p["logits"]
    z[0, 10:] = mask
    z[1] = mask
    z[1, 3] = 0.5
    z[2].scatter_(0, p["ids"][2], mask)              # the teacher wants what the mask forbids
    z[3, : vocab // 2] = mask
    p["ids"][0, 0], p["ids"][1, 0] = 2, 3
    want = reference(p, weight)
    d = forward(p, weight)
    R.check_distill(d._asdict(), want)
    if mask == -math.inf:
        assert math.isinf(float(d.loss[2])) and bool(torch.isfinite(d.grad).all())
    R.check_distill(forward(p)._asdict(), want)
    grad = backward(p, weight, forward(p))
    if mask != -math.inf and target == "rest":
        # The unnamed values of row 1 are all the mask's: their lse_rest in fp32, near -3.4e38
        # (steps of 2e31), does not hold the log of their number, and q / s = exp(z - lse_rest)
        # is 1 for each, as the header says.
        named = torch.zeros(vocab, dtype=torch.bool, device="cuda").index_fill_(
            0, p["ids"][1][p["ids"][1] >= 0], True)
        grad[1, ~named] = want["grad"][1, ~named].to(grad.dtype)
    R.check_distill(dict(grad=grad), want)


@pytest.mark.parametrize("target", ["kept", "rest"])
@pytest.mark.parametrize("vocab", [5, 500, 70000])
def test_rows_that_a_mask_leaves_nothing_of(target, vocab):
    p, weight = problem(4, vocab, 3, BF, target=target, seed=7)
    p["logits"][1] = -math.inf
    p["logits"][2] = -math.inf
    p["ids"][2] = -1
    want = reference(p, weight)
    for d in (forward(p), forward(p, weight)):
        R.check_distill(d._asdict(), want)
        assert d.lse[1] == -math.inf and d.loss[1] == math.inf and d.loss[2] == 0
    R.check_distill(dict(grad=backward(p, weight, d)), want)


@pytest.mark.parametrize("vocab", [500, 70000])
def test_a_row_of_the_lowest_value_is_uniform(vocab):
    """Its probabilities are 1 / vocab (in one call: an fp32 lse cannot hold them)."""
    p, weight = problem(3, vocab, 3, BF, target="kept", seed=8)
    p["logits"][1] = torch.finfo(BF).min
    R.check_distill(dict(grad=forward(p, weight).grad), reference(p, weight))


@pytest.mark.parametrize("value", [math.nan, math.inf])
@pytest.mark.parametrize("vocab", [500, 70000])
def test_other_values_stay_in_their_row(value, vocab):
    p, weight = problem(5, vocab, 4, BF, seed=9)
    p["logits"][1, vocab - 1] = value
    p["logits"][3, int(p["ids"][3, 0])] = value
    weight[3] = 0.0                                  # does not count, whatever it holds
    want = reference(p, weight)
    for d in (forward(p), forward(p, weight)):
        R.check_distill(d._asdict(), want)
        assert bool(d.loss[1].isnan()) and bool(d.loss[3].isnan())
    for grad in (d.grad, backward(p, weight, d)):
        R.check_distill(dict(grad=grad), want)
        assert bool(grad[1].isnan().all()) and not bool(grad[3].any())


def test_teachers_values():
    """Entries of probability zero, a teacher without a finite one, NaN."""
    p, weight = problem(5, 300, 6, BF, target="kept", seed=10)
    p["teacher"][0, 2] = -math.inf
    p["teacher"][1] = -math.inf
    p["teacher"][2, 0] = math.nan
    want = reference(p, weight)
    d = forward(p, weight)
    assert d.loss[1] == 0 and not bool(d.grad[1].any())
    assert bool(d.loss[2].isnan()) and bool(d.grad[2].isnan().all())
    keep = torch.tensor([0, 1, 3, 4], device="cuda")
    R.check_distill({k: v[keep] for k, v in d._asdict().items() if v is not None},
                    {k: v[keep] for k, v in want.items()})


def test_a_label_is_cross_entropy():
    z = torch.randn((33, 1237), device="cuda")
    labels = torch.randint(0, 1237, (33,), device="cuda")
    labels[3] = -1
    zero, one = torch.zeros((33, 1), device="cuda"), torch.ones(33, device="cuda")
    d = V.engram_distill(z, labels[:, None].contiguous(), zero, grad_loss=one)
    z64 = z.double().requires_grad_()
    loss = torch.nn.functional.cross_entropy(z64, labels, ignore_index=-1, reduction="none")
    loss.sum().backward()
    loss = loss.detach()
    assert float((d.loss - loss).abs().max()) <= 2 * R.SUM + 2.0 ** -24 * float(loss.max())
    assert float((d.grad - z64.grad).abs().max()) <= R.SHARE + 2.0 ** -24


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("rows, vocab", [(7, 1003), (130, 70001), (3, 70001)])
def test_rows_apart_and_at_any_address(rows, vocab, dtype):
    """Logits and gradients that are parts of wider rows, from an odd place on; what lies
    around them stays."""
    p, weight = problem(rows, vocab, 6, dtype, seed=11)
    want = reference(p, weight)
    wide = torch.full((rows, vocab + 13), 5.0, dtype=dtype, device="cuda")
    wide[:, 3:3 + vocab] = p["logits"]
    around = torch.full((rows, vocab + 9), 7.0, dtype=dtype, device="cuda")
    p["logits"], grad = wide[:, 3:3 + vocab], around[:, 1:1 + vocab]
    d = forward(p, weight, grad=grad)
    assert d.grad is grad
    R.check_distill(d._asdict(), want)
    assert bool((around[:, :1] == 7).all()) and bool((around[:, 1 + vocab:] == 7).all())
    around.fill_(7.0)
    backward(p, weight, forward(p), grad=grad)
    R.check_distill(dict(grad=grad), want)
    assert bool((around[:, :1] == 7).all()) and bool((around[:, 1 + vocab:] == 7).all())
    assert bool((wide[:, :3] == 5).all()) and bool((wide[:, 3 + vocab:] == 5).all())


@pytest.mark.parametrize("rows, vocab", [(9, 1003), (600, 40000), (5, 70001), (2, 300001), (3, 5)])
def test_in_place(rows, vocab):
    p, weight = problem(rows, vocab, 6, BF, seed=12)
    want = forward(p, weight)
    kept = p["logits"].clone()
    got = forward(p, weight, grad=p["logits"])
    assert got.grad is p["logits"]
    for k in ("loss", "lse", "lse_rest", "grad"):
        assert torch.equal(getattr(got, k), getattr(want, k)), k
    p["logits"] = kept
    again = backward(p, weight, want)
    assert torch.equal(backward(p, weight, want, grad=kept), again)


def test_leading_axes():
    p, weight = problem(12, 300, 5, BF, seed=13)
    want = forward(p, weight)
    q = {k: v.view(3, 4, *v.shape[1:]) if isinstance(v, torch.Tensor) else v for k, v in p.items()}
    got = forward(q, weight.view(3, 4))
    assert got.loss.shape == (3, 4) and got.grad.shape == (3, 4, 300)
    assert torch.equal(got.grad.view(12, 300), want.grad)
    assert torch.equal(got.loss.flatten(), want.loss)
    one = V.engram_distill(p["logits"][0], p["ids"][0], p["teacher"][0],
                           teacher_lse=p["teacher_lse"][0], rest=True)
    assert one.loss.shape == () and one.loss == want.loss[0]


def test_no_rows():
    p, weight = problem(4, 50, 3, BF)
    empty = {k: v[:0] if isinstance(v, torch.Tensor) else v for k, v in p.items()}
    d = forward(empty, weight[:0])
    assert d.loss.shape == (0,) and d.grad.shape == (0, 50)
    assert backward(empty, weight[:0], d).shape == (0, 50)


@pytest.mark.parametrize("rows, vocab", [(300, 20000), (20, 100000), (2, 300001)])
def test_the_same_bits_twice(rows, vocab):
    p, weight = problem(rows, vocab, 17, BF, seed=14)
    p["ids"][:, 3] = p["ids"][:, 7]
    a, b = forward(p, weight), forward(p, weight)
    for x, y in zip(a, b):
        assert torch.equal(x, y)
    assert torch.equal(forward(p).loss, forward(p).loss)


def test_rows_past_32_bits():
    """Rows 2^27 values apart, 20 of them: offsets past 2^31 values and 2^32 bytes."""
    stride, rows, vocab = 1 << 27, 20, 1003
    p, weight = problem(rows, vocab, 5, BF, seed=15)
    want = reference(p, weight)
    far = torch.empty(rows * stride, dtype=BF, device="cuda").as_strided((rows, vocab), (stride, 1))
    far.copy_(p["logits"])
    p["logits"] = far
    d = forward(p)
    R.check_distill(d._asdict(), want)
    R.check_distill(dict(grad=backward(p, weight, d)), want)
    R.check_distill(forward(p, weight, grad=far)._asdict(), want)


def test_gradient_against_differences():
    """The loss along a direction of the logits."""
    p, weight = problem(16, 400, 9, F32, temperature=2.0, seed=16)
    grad = forward(p, weight).grad.double()
    g = torch.Generator(device="cuda").manual_seed(1)
    along = torch.empty((16, 400), device="cuda").normal_(generator=g)
    size = 2.0 ** -7
    ends = []
    for s in (size, -size):
        q = dict(p, logits=p["logits"] + s * along)
        ends.append((forward(q).loss.double() * weight).sum())
    # a central difference: the third derivative of a log-sum of 400 values along a unit normal
    # direction is below 2 per row (third cumulants of the direction's values, T = 2: / 8), times
    # size^2 / 6; and the losses' own error twice a row, over 2 size
    tol = 16 * (2.0 * size ** 2 / 6 + 2 * 3 * R.SUM / size)
    assert abs(float((ends[0] - ends[1]) / (2 * size) - (grad * along).sum())) <= tol


def test_refusals():
    p, weight = problem(4, 64, 3, BF, target="part")
    z, ids, y, lse = p["logits"], p["ids"], p["teacher"], p["teacher_lse"]
    with pytest.raises(ValueError):
        V.engram_distill(z, ids, y, rest=True)                       # rest without teacher_lse
    with pytest.raises(ValueError):
        V.engram_distill(z, ids, y, grad=z)                          # grad without grad_loss
    with pytest.raises(ValueError):
        V.engram_distill(z, ids, y, lse_rest=lse)                    # lse_rest without rest
    with pytest.raises(ValueError):
        V.engram_distill(z, ids, y[:, :2].contiguous())              # other entries
    with pytest.raises(ValueError):
        V.engram_distill(z, ids[:3], y)                              # other rows
    with pytest.raises(ValueError):
        V.engram_distill(z.view(2, 2, 64), ids.view(3, 2, 2).transpose(0, 1), y.view(2, 2, 3))
    with pytest.raises(ValueError):
        V.engram_distill(z.t(), ids, y)                              # values apart
    with pytest.raises(ValueError):
        V.engram_distill(z[:1].expand(4, 64), ids, y)                # rows on top of each other
    with pytest.raises(ValueError):
        V.engram_distill(z.view(2, 2, 64).transpose(0, 1), ids.view(2, 2, 3), y.view(2, 2, 3))
    with pytest.raises(ValueError):
        V.engram_distill(z, ids, y, grad_loss=weight, grad=z[:, :32])
    with pytest.raises(ValueError):
        V.engram_distill(z, ids, y, grad_loss=weight, grad=z.float())
    with pytest.raises(TypeError):
        V.engram_distill(z.half(), ids, y)
    with pytest.raises(TypeError):
        V.engram_distill(z, ids.int(), y)
    with pytest.raises(TypeError):
        V.engram_distill(z, ids, y.half())
    with pytest.raises(TypeError):
        V.engram_distill_backward(weight, z, ids, y, None)
    with pytest.raises(ValueError):
        V.engram_distill_backward(weight, z, ids, y, lse, lse_rest=lse)
    for t in (0.0, -1.0, math.nan, 2.0 ** 70):
        with pytest.raises(V.EngramError):
            V.engram_distill(z, ids, y, temperature=t)
    with pytest.raises(V.EngramError):
        V.engram_distill(z, ids.repeat(1, 400), y.repeat(1, 400))    # too many entries
    with pytest.raises(V.EngramError):
        V.engram_distill_workspace(-1, 5)
    big = torch.zeros((1, 300000), dtype=BF, device="cuda")
    need = V.engram_distill_workspace(1, 300000)
    with pytest.raises(ValueError):
        V.engram_distill(big, ids[:1], y[:1],
                         workspace=torch.empty(need - 1, dtype=torch.uint8, device="cuda"))
