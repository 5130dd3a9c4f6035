"""The distillation gradient from kept statistics where their fp32 logarithms are coarse: rows under
a mask's large finite value at temperatures that do not divide it, low temperatures, logits far
from 0.  Held to the definition in 64 bits like the gradient of the one call."""
import math

import pytest
import torch

from tests import vocab_reference as R
from tests.gpu_helpers import needs_gpu
from tests.test_gpu_distill import backward, forward, problem

pytestmark = needs_gpu
V = pytest.importorskip("gram_hashed_embedding_amd.vocab")

BF, F32 = torch.bfloat16, torch.float32

# SHARE allows for two statistics of up to 64; a bf16 gradient's are used up to 1024, where half a
# step of fp32 is 2^-15.
KEPT = {F32: 1.0, BF: 1.0 + 2.0 ** -14 / R.SHARE}

# one wavefront to a row, a block to a row, several blocks to a row, rows cut in the other call
SIZES = [500, 12000, 20000, 70000]


def losses(p, want):
    """want's losses with each row's largest logit taken off first: beside a mask's lowest value
    the reference's lse_rest - lse holds nothing of the logarithms of their numbers."""
    out = want.clone()
    for t in range(out.numel()):
        P, named, m, r, none = R.target(p["ids"][t], p["teacher"][t], p["logits"].shape[1],
                                        p["temperature"],
                                        None if p["teacher_lse"] is None else p["teacher_lse"][t],
                                        p["rest"])
        z = p["logits"][t].double()
        if none or r == 0.0 or not math.isfinite(float(z.max())):
            continue
        z = (z - z.max()) / p["temperature"]
        lse, on = torch.logsumexp(z, 0), P != 0
        out[t] = (P[on] * (P[on].log() - (z[on] - lse))).sum()
        out[t] += r * (math.log(r) - (torch.logsumexp(z[~named], 0) - lse))
    return out


def check(p, weight, loss=True):
    """The loss and gradient of one call, the gradient of kept statistics, and of these in the
    logits' place.  loss: what fp32 can hold."""
    want = R.distill(p["logits"], p["ids"], p["teacher"], p["teacher_lse"], p["rest"],
                     p["temperature"], weight)
    want["loss"] = losses(p, want["loss"])
    d = forward(p, weight)
    R.check_distill(d._asdict() if loss else dict(grad=d.grad), want)
    if loss:
        R.check_distill(forward(p)._asdict(), want)
    want["slack"] = want["slack"] * KEPT[p["logits"].dtype]
    grad = backward(p, weight, d)
    R.check_distill(dict(grad=grad), want)
    q = dict(p, logits=p["logits"].clone())
    assert torch.equal(backward(q, weight, d, grad=q["logits"]), grad)


@pytest.mark.parametrize("temperature", [0.7, 1.0, 1.1, 1.3, 1.8, 2.7, 3.1])
@pytest.mark.parametrize("mask, dtype", [(torch.finfo(BF).min, BF), (torch.finfo(F32).min, F32),
                                         (-1e30, BF), (-1e30, F32), (-1e4, F32),
                                         (-math.inf, BF), (-math.inf, F32)])
@pytest.mark.parametrize("vocab", SIZES)
def test_masks(vocab, mask, dtype, temperature):
    for target in ("kept", "part", "rest"):
        p, weight = problem(8, vocab, 5, dtype, target=target, temperature=temperature, seed=21)
        z, ids = p["logits"], p["ids"]
        names = torch.zeros((8, vocab + 1), dtype=torch.bool, device="cuda")
        names.scatter_(1, torch.where(ids >= 0, ids, vocab), True)
        for row in (0, 1, 2):                         # masked to what the teacher names
            z[row, ~names[row, :-1]] = mask
        z[3] = mask                                   # nothing left
        z[4, names[4, :-1]] = mask                    # the teacher wants what the mask forbids
        z[5, : vocab // 2] = mask
        z[6] = mask
        weight[6] = 0.0
        if target != "kept":                          # no rest: r = 0
            y = torch.where(ids >= 0, p["teacher"].double() / temperature, -math.inf)
            p["teacher_lse"][1:3] = torch.logsumexp(y, 1)[1:3].float()
        check(p, weight, loss=temperature >= 1.0)


@pytest.mark.parametrize("temperature", [2.0 ** -64, 1e-12, 1e-6, 1e-3, 0.01, 0.05, 0.2, 4e4,
                                         2.0 ** 64])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("vocab", [500, 20000])
def test_temperatures(vocab, dtype, temperature):
    p, weight = problem(6, vocab, 9, dtype, target="kept", temperature=temperature, seed=22)
    check(p, weight)


@pytest.mark.parametrize("temperature", [0.01, 0.05, 0.2])
@pytest.mark.parametrize("target", ["part", "rest"])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_temperatures_with_true_probabilities(dtype, target, temperature):
    p, weight = problem(6, 20000, 9, dtype, target=target, temperature=temperature, seed=23)
    check(p, weight)


# on both sides of where a statistic is coarse
@pytest.mark.parametrize("offset", [-3000.0, -1100.0, -1000.0, -90.0, -60.0, 40.0, 60.0, 900.0,
                                    1100.0, 3000.0])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_logits_far_from_zero(dtype, offset):
    for vocab in (500, 20000):
        p, weight = problem(6, vocab, 9, dtype, seed=24)
        p["logits"] = (p["logits"].float() + offset).to(dtype)
        check(p, weight)


@pytest.mark.parametrize("rows", [65, 1024, 1025, 65537, 70000])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_coarse_rows(rows, dtype):
    """More rows than blocks for coarse ones; some that are not, some that do not count."""
    p, weight = problem(rows, 24, 1, dtype, target="kept", temperature=0.5, seed=28)
    p["logits"][::3] -= 2000.0
    p["logits"][1::7] = torch.finfo(dtype).min
    weight[2::5] = 0.0
    z = p["logits"].double()
    q = torch.softmax((z - z.amax(1, keepdim=True)) / 0.5, 1)
    share = (weight.double() / 0.5)[:, None]
    want = share * (q - torch.nn.functional.one_hot(p["ids"][:, 0], 24))
    grad = backward(p, weight, forward(p))
    off = (grad.double() - want).abs()
    tol = R.half_step(dtype) * 1.01 * want.abs() + KEPT[dtype] * R.SHARE * share * q + 2.0 ** -125
    assert bool((off <= tol).all()), float((off - tol).max())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_long_coarse_rows(dtype):
    """More values than a block has bits for at a time, ids that repeat across and within parts."""
    p, weight = problem(2, (1 << 20) + 3, 70, dtype, target="part", temperature=0.02, seed=29)
    p["ids"][:, 40:60] = p["ids"][:, 3:23]
    p["teacher_lse"] += 2.0
    check(p, weight)


def test_errors_are_counted_once():
    p, weight = problem(3, 40000, 6, BF, target="kept", temperature=0.001, seed=25)
    p["ids"][0, 1], p["ids"][2, 3] = 40000, -7
    d = forward(p, weight)
    err = torch.zeros(1, dtype=torch.int64, device="cuda")
    grad = backward(p, weight, d, err_count=err)
    assert int(err) == 2 and torch.equal(backward(p, weight, d), grad)


def test_rows_at_any_address():
    """Rows that are summed again, beside rows that are not; what lies around them stays."""
    for dtype in (BF, F32):
        for vocab in (700, 33001):
            p, weight = problem(6, vocab, 6, dtype, seed=26)
            p["logits"][1::2] = torch.finfo(dtype).min
            want = R.distill(p["logits"], p["ids"], p["teacher"], p["teacher_lse"], True, 1.0,
                             weight)
            wide = torch.full((6, vocab + 13), 5.0, dtype=dtype, device="cuda")
            wide[:, 3:3 + vocab] = p["logits"]
            p["logits"] = wide[:, 3:3 + vocab]
            d = forward(p)
            around = torch.full((6, vocab + 9), 7.0, dtype=dtype, device="cuda")
            for grad, lot, lead in ((around[:, 1:1 + vocab], around, 1),
                                    (p["logits"], wide, 3)):
                edge = lot[:, 0].clone()
                R.check_distill(dict(grad=backward(p, weight, d, grad=grad)), want)
                assert bool((lot[:, :lead] == edge[0]).all())
                assert bool((lot[:, lead + vocab:] == edge[0]).all())


@pytest.mark.parametrize("rows, vocab", [(9, 1003), (600, 40000), (5, 70001), (2, 300001), (3, 5)])
def test_in_place_in_fp32(rows, vocab):
    p, weight = problem(rows, vocab, 6, F32, seed=27)
    want = forward(p, weight)
    kept = p["logits"].clone()
    got = forward(p, weight, grad=p["logits"])
    for k in ("loss", "lse", "lse_rest", "grad"):
        assert torch.equal(getattr(got, k), getattr(want, k)), k
    p["logits"] = kept
    again = backward(p, weight, want)
    assert torch.equal(backward(p, weight, want, grad=kept), again)


@pytest.mark.parametrize("vocab", [700, 33001])
def test_captured_and_replayed(vocab):
    """A captured gradient follows its inputs: none, some and all of the rows coarse."""
    p, weight = problem(9, vocab, 6, BF, seed=30)
    d, grad = forward(p), torch.empty_like(p["logits"])
    backward(p, weight, d, grad=grad)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        backward(p, weight, d, grad=grad)
    for turn, rows in enumerate((0, 4, 9, 0, 9)):
        fresh, _ = problem(9, vocab, 6, BF, seed=31 + turn)
        fresh["logits"][:rows] = torch.finfo(BF).min
        for name in ("logits", "ids", "teacher", "teacher_lse"):
            p[name].copy_(fresh[name])
        for old, new in zip((d.lse, d.lse_rest), forward(fresh)[1:3]):
            old.copy_(new)
        grad.fill_(7.0)
        g.replay()
        if turn % 2:
            torch.cuda.synchronize()
        want = R.distill(fresh["logits"], fresh["ids"], fresh["teacher"], fresh["teacher_lse"],
                         True, 1.0, weight)
        R.check_distill(dict(grad=grad), want)
        assert torch.equal(backward(fresh, weight, d), grad)
