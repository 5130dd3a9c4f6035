"""The selection of a beam search and the reordering of states against plain ones: the chosen
beams and tokens exactly, ties by place, masks, beams that are dead or finished, candidates that
run out; slots, copies and histories exactly."""
import math
import random

import pytest
import torch

from tests import vocab_reference as R
from tests.gpu_helpers import needs_gpu

pytestmark = needs_gpu
V = pytest.importorskip("gram_hashed_embedding_amd.vocab")

BF, F32 = torch.bfloat16, torch.float32


def logits(batch, beams, vocab, dtype=BF, seed=0, std=3.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = torch.empty((batch, beams, vocab), device="cuda").normal_(0.0, std, generator=g).to(dtype)
    scores = -20.0 - 5.0 * torch.rand((batch, beams), generator=g, device="cuda")
    return z, scores


def check(z, scores, count, finished=None, eos=-1, got=None):
    want = R.beam_select(z, scores, count, finished, eos)
    if got is None:
        got = V.engram_beam_select(z, scores, count, finished=finished, eos=eos)
    other = (got.parents != want[1]) | (got.tokens != want[2])
    if bool(other.any()):
        # A value is off by its beam's lse, at most SUM (in 64 bits otherwise), so those of two
        # beams may change places where they are no more than twice that apart; those of one
        # beam have the same lse and may not.
        every = torch.stack(list(R.beam_values(z, scores, finished, eos)))
        for b, k in other.nonzero().tolist():
            w, v = int(got.parents[b, k]), int(got.tokens[b, k])
            assert w >= 0 and v >= 0 and w != int(want[1][b, k]), (b, k, w, v)
            assert abs(float(every[b, w, v] - want[0][b, k])) <= 2 * R.SUM, (b, k, w, v)
        for b in range(got.parents.shape[0]):
            pairs = [x for x in zip(got.parents[b].tolist(), got.tokens[b].tolist())
                     if x != (-1, -1)]
            assert len(set(pairs)) == len(pairs)
            for w in range(z.shape[1]):
                # a beam's own, in their order
                values = [float(every[b, p, t]) for p, t in pairs if p == w]
                assert values == sorted(values, reverse=True)
    assert torch.equal(got.finished[~other], want[3][~other])
    none = want[0] == -math.inf
    assert torch.equal(got.scores == -math.inf, none)
    off = (got.scores.double() - want[0])[~none].abs()
    # (SUM, and where candidates changed places twice that)
    assert bool((off <= 3 * R.SUM + 2.0 ** -24 * want[0][~none].abs()).all())
    assert bool((off[~other[~none]] <= R.SUM + 2.0 ** -24 * want[0][~none & ~other].abs()).all())
    return got


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("vocab", [1, 2, 7, 8, 127, 128, 129, 1003, 2048, 2049, 8193, 50257])
def test_vocabularies(vocab, dtype):
    z, s = logits(3, 4, vocab, dtype, seed=vocab)
    check(z, s, 4)
    check(z, s, 8)


@pytest.mark.parametrize("batch, beams, count", [
    (1, 1, 1), (1, 1, 64), (2, 64, 64), (5, 3, 7), (70, 2, 4), (1, 16, 32), (9, 33, 1)])
def test_shapes(batch, beams, count):
    z, s = logits(batch, beams, 3001, seed=beams)
    check(z, s, count)


@pytest.mark.parametrize("vocab", [151936, 262145, 600001])
def test_long_rows(vocab):
    z, s = logits(2, 3, vocab, F32, seed=5)
    check(z, s, 6)


def test_many_rows():
    z, s = logits(300, 4, 2500, seed=6)
    check(z, s, 8)


@pytest.mark.parametrize("vocab", [5, 400, 40000])
def test_equal_values_by_place(vocab):
    """Constant rows, beams that are alike, values that are equal across beams, both zeros."""
    z = torch.zeros((4, 3, vocab), dtype=BF, device="cuda")
    s = torch.full((4, 3), -1.0, device="cuda")
    z[1] = 2.0
    s[1] = torch.tensor([-3.0, -1.0, -1.0])
    z[2, :, 1::2] = -0.0
    z[3] = logits(1, 1, vocab, seed=7)[0].expand(1, 3, vocab)
    for count in (1, 4, 64):
        check(z, s, count)


def test_runs_of_equal_values():
    """More equal candidates than are listed at a time, in some of the beams."""
    z, s = logits(2, 4, 30000, seed=8)
    z[0, 1] = z[0, 1].clamp(max=2.0)
    z[0, 2] = 1.0
    s[0] = torch.tensor([-30.0, -20.0, -19.0, -31.0])
    z[1] = z[1].clamp(max=0.5)
    check(z, s, 20)
    check(z, s, 64)


@pytest.mark.parametrize("mask", [-math.inf, torch.finfo(BF).min])
@pytest.mark.parametrize("allowed", [1, 3, 200])
def test_masks(mask, allowed):
    z, s = logits(4, 3, 5000, seed=9)
    keep = torch.zeros((4, 3, 5000), dtype=torch.bool, device="cuda")
    for b in range(4):
        for w in range(3):
            keep[b, w, torch.randperm(5000)[:allowed]] = True
    if mask == -math.inf:
        keep[1, 0] = False                         # nothing left of a beam
        keep[2] = False                            # nothing left of a sequence
    z = torch.where(keep, z, torch.full_like(z, mask))
    got = check(z, s, 8) if mask == -math.inf else check(z, s, min(8, 3 * allowed))
    if mask == -math.inf:
        assert bool((got.parents[2] == -1).all()) and bool((got.tokens[2] == -1).all())


def test_beams_that_are_no_beams():
    """Scores of -inf, NaN and +inf; rows with NaN or +inf."""
    z, s = logits(5, 4, 700, seed=10)
    s[0, 1:] = -math.inf                           # a search's first step
    s[1, 2], s[1, 3] = math.nan, math.inf
    z[2, 1, 699], z[2, 2, 0] = math.nan, math.inf
    s[3] = -math.inf
    z[4, :, :] = math.nan
    got = check(z, s, 6)
    assert bool((got.parents[0] == 0).all())
    assert bool((got.parents[3:] == -1).all())


@pytest.mark.parametrize("vocab", [3, 900, 20000])
def test_finished_beams(vocab):
    z, s = logits(6, 4, vocab, seed=11)
    f = torch.zeros((6, 4), dtype=torch.bool, device="cuda")
    f[0, 1], f[1], f[2, 0], f[2, 3] = True, True, True, True
    z[0, 1] = math.nan                             # not read
    s[0, 1] = -1.0                                 # the best there is
    s[1] = torch.tensor([-4.0, -4.0, -math.inf, -2.0])
    s[3] = -2.0
    z[3, :, 1] = 30.0                              # these end now
    for eos in (0, 1, vocab - 1):
        got = check(z, s, 6, f, eos)
        assert got.parents[0, 0] == 1 and got.tokens[0, 0] == eos and got.scores[0, 0] == -1.0
        assert got.parents[1].tolist() == [3, 0, 1, -1, -1, -1]
    # a finished beam level with a live one, on either side of it
    z, s = logits(2, 3, vocab, seed=12)
    live = R.beam_select(z[:, 1:2], s[:, 1:2], 1)[0][:, 0].float()
    s[:, 0], s[:, 2] = live, live
    f = torch.tensor([[True, False, True]] * 2, device="cuda")
    got = V.engram_beam_select(z, s, 3, finished=f, eos=0)
    assert set(got.parents[0, :3].tolist()) <= {0, 1, 2}
    assert got.parents[0].tolist().index(0) < got.parents[0].tolist().index(2)


def test_scores_and_flags_in_place():
    z, s = logits(5, 6, 900, seed=15)
    f = torch.rand((5, 6), device="cuda") < 0.4
    want = V.engram_beam_select(z, s, finished=f, eos=3)
    got = V.engram_beam_select(z, s, finished=f, eos=3, out_scores=s, out_finished=f)
    assert got.scores is s and got.finished is f
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    with pytest.raises(V.EngramError):                # another sequence's are read later
        V.engram_beam_select(z, s, 5, out_scores=s.flatten()[:25].view(5, 5))


def test_rows_apart_and_outputs():
    z, s = logits(3, 4, 1003, seed=13)
    wide = torch.full((12, 1040), 99.0, dtype=BF, device="cuda")
    wide[:, 5:1008] = z.view(12, 1003)
    part = wide[:, 5:1008]
    out = dict(out_scores=torch.empty((3, 5), device="cuda"),
               parents=torch.empty((3, 5), dtype=torch.int64, device="cuda"),
               tokens=torch.empty((3, 5), dtype=torch.int64, device="cuda"),
               out_finished=torch.empty((3, 5), dtype=torch.bool, device="cuda"),
               workspace=torch.full((V.engram_beam_select_workspace(3, 4, 1003),), 255,
                                    dtype=torch.uint8, device="cuda"))
    got = V.engram_beam_select(part, s, 5, **out)
    assert got.scores is out["out_scores"] and got.tokens is out["tokens"]
    check(z, s, 5, got=got)
    assert V.engram_beam_select(z, s).scores.shape == (3, 4)   # as many as there are beams
    empty = V.engram_beam_select(z[:0], s[:0], 5)
    assert empty.scores.shape == (0, 5)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("vocab", [1, 3, 63, 64, 65, 127, 128, 129, 130, 191, 192, 193, 2300])
def test_every_place_in_a_cache_line(vocab, dtype):
    """Logits from every value of a cache line on, the best first, last, and level at both."""
    z, s = logits(2, 3, vocab, dtype, seed=vocab)
    z[0, 0, 0], z[0, 1, vocab - 1] = 9.0, 9.5
    z[1, 0, 0] = z[1, 0, vocab - 1] = z[1, 0, vocab // 2] = 9.0
    finished = torch.zeros((2, 3), dtype=torch.bool, device="cuda")
    finished[1, 2] = True
    line = 128 // dtype.itemsize
    for first in range(line):
        wide = torch.full((first + 6 * (vocab + 1) + line,), math.inf, dtype=dtype, device="cuda")
        part = wide.as_strided((6, vocab), (vocab + 1, 1), first)
        part.copy_(z.view(6, vocab))
        workspace = torch.full((V.engram_beam_select_workspace(2, 3, vocab),), 127,
                               dtype=torch.uint8, device="cuda")
        check(z, s, 5, finished, vocab - 1,
              got=V.engram_beam_select(part, s, 5, finished=finished, eos=vocab - 1,
                                       workspace=workspace))


def test_rows_past_32_bits():
    stride = 1 << 27
    z, s = logits(5, 4, 700, seed=14)
    far = torch.empty(20 * stride, dtype=BF, device="cuda").as_strided((20, 700), (stride, 1))
    far.copy_(z.view(20, 700))
    check(z, s, 6, got=V.engram_beam_select(far, s, 6))


def test_select_refusals():
    z, s = logits(2, 3, 50)
    for bad in (dict(count=0), dict(count=65)):
        with pytest.raises(ValueError):
            V.engram_beam_select(z, s, **bad)
    with pytest.raises(ValueError):
        V.engram_beam_select(z, s[0])
    with pytest.raises(ValueError):
        V.engram_beam_select(z[:1], s)
    with pytest.raises(ValueError):
        V.engram_beam_select(z.transpose(0, 1), s)
    with pytest.raises(TypeError):
        V.engram_beam_select(z, s.double())
    f = torch.zeros((2, 3), dtype=torch.bool, device="cuda")
    with pytest.raises(TypeError):
        V.engram_beam_select(z, s, finished=f.int(), eos=1)
    with pytest.raises(TypeError):
        V.engram_beam_select(z, s, 2, parents=torch.empty((2, 2, 1), device="cuda"))
    for bad in (dict(finished=f), dict(eos=50), dict(eos=-2)):
        with pytest.raises(V.EngramError):
            V.engram_beam_select(z, s, **bad)
    with pytest.raises(ValueError):
        V.engram_beam_select(z, s, workspace=torch.empty(8, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        V.engram_beam_select(torch.zeros((65, 9), device="cuda"),
                             torch.zeros((1, 65), device="cuda"))


# ------------------------------------------------------------- reordering --
def fork_case(batch, beams, slot_count, seed, invalid=True):
    rng = random.Random(seed)
    slots = rng.sample(range(slot_count), batch * beams)
    slots = [slots[b * beams:(b + 1) * beams] for b in range(batch)]
    parents = [[rng.randrange(beams) for _ in range(beams)] for _ in range(batch)]
    if invalid:
        for row in parents[::2]:
            row[rng.randrange(beams)] = rng.choice([-1, -1, beams, -5, 1 << 40])
    return parents, slots


@pytest.mark.parametrize("batch, beams", [(1, 1), (1, 2), (3, 5), (40, 8), (7, 64), (2, 63)])
@pytest.mark.parametrize("shape, dtype", [((8,), BF), ((9, 1000), BF), ((3, 4), torch.int32),
                                          ((5000,), F32)])
def test_states(batch, beams, shape, dtype):
    count = batch * beams + 5
    parents, slots = fork_case(batch, beams, count, seed=batch * 100 + beams)
    g = torch.Generator(device="cuda").manual_seed(1)
    pool = torch.randint(-99, 99, (count, *shape), generator=g, device="cuda").to(dtype)
    before = pool.clone()
    err = torch.zeros(1, dtype=torch.int64, device="cuda")
    got = V.engram_beam_fork(torch.tensor(parents, device="cuda"), pool,
                             slots=torch.tensor(slots, device="cuda"), err_count=err)
    new, copies, bad = R.beam_fork(parents, slots, count)
    assert got.slots.tolist() == new and got.history is None
    want = before.clone()
    for to, source in copies.items():
        want[to] = before[source]
    assert torch.equal(pool, want)
    assert int(err) == bad


def test_several_pools_and_the_plain_slots():
    pools = [torch.randn((12, n), device="cuda") for n in (4, 3000, 64, 20000)]
    before = [p.clone() for p in pools]
    parents = [[2, 2, 0, 0], [1, 1, 1, 1], [0, 1, 2, 3]]
    slots = [[4 * b + w for w in range(4)] for b in range(3)]
    got = V.engram_beam_fork(torch.tensor(parents, device="cuda"), pools)
    new, copies, _ = R.beam_fork(parents, slots, 12)
    assert got.slots.tolist() == new
    for p, old in zip(pools, before):
        want = old.clone()
        for to, source in copies.items():
            want[to] = old[source]
        assert torch.equal(p, want)


def test_slots_that_are_none():
    """Unused slots are handed on, others outside the pool counted; nothing is copied."""
    parents = torch.tensor([[0, 0, 0], [1, 1, 2]], device="cuda")
    slots = torch.tensor([[-1, 3, 9], [0, 8, -7]], device="cuda")
    pool = torch.randn((4, 16), device="cuda")
    before, err = pool.clone(), torch.zeros(1, dtype=torch.int64, device="cuda")
    got = V.engram_beam_fork(parents, pool, slots=slots, err_count=err)
    assert got.slots.tolist() == [[-1, 3, 9], [8, 0, -7]]
    assert torch.equal(pool, before) and int(err) == 3


@pytest.mark.parametrize("have, new_len", [(1, 1), (4, 4), (4, 5), (4, 2), (4, 1), (0, 1),
                                           (700, 701)])
def test_histories(have, new_len):
    parents, slots = fork_case(6, 5, 30, seed=have)
    history = torch.randint(0, 1 << 40, (6, 5, have), device="cuda")
    tokens = torch.randint(-1, 1 << 40, (6, 5), device="cuda")
    got = V.engram_beam_fork(torch.tensor(parents, device="cuda"), tokens=tokens, history=history,
                             new_len=new_len)
    for b in range(6):
        for j in range(5):
            p = parents[b][j]
            row = history[b, p if 0 <= p < 5 else j].tolist() + [int(tokens[b, j])]
            assert got.history[b, j].tolist() == row[len(row) - new_len:]
    assert got.slots.shape == (6, 5)


def test_no_sequences():
    none = torch.empty((0, 4), dtype=torch.int64, device="cuda")
    got = V.engram_beam_fork(none, torch.zeros((4, 8), device="cuda"), tokens=none,
                             history=torch.empty((0, 4, 3), dtype=torch.int64, device="cuda"))
    assert got.slots.shape == (0, 4) and got.history.shape == (0, 4, 3)


def test_a_large_pool():
    """Slots past 2^32 bytes: 9 of 1 GiB, the last copied over the first."""
    pool = torch.empty((9, 1 << 28), dtype=torch.int32, device="cuda")
    for w in range(9):
        pool[w].fill_(w)
        pool[w, -1] = 100 + w
    slots = torch.tensor([[0, 8]], device="cuda")
    V.engram_beam_fork(torch.tensor([[1, 1]], device="cuda"), pool, slots=slots)
    for w in range(9):
        want = 8 if w == 0 else w
        assert bool((pool[w, :-1] == want).all()) and int(pool[w, -1]) == 100 + want


def test_fork_refusals():
    parents = torch.zeros((2, 3), dtype=torch.int64, device="cuda")
    pool = torch.zeros((6, 8), device="cuda")
    with pytest.raises(ValueError):
        V.engram_beam_fork(parents[0], pool)
    with pytest.raises(TypeError):
        V.engram_beam_fork(parents.int(), pool)
    with pytest.raises(ValueError):
        V.engram_beam_fork(parents, [pool] * 9)
    with pytest.raises(ValueError):
        V.engram_beam_fork(parents, [pool, torch.zeros((7, 8), device="cuda")])
    with pytest.raises(ValueError):
        V.engram_beam_fork(parents, pool.t())
    with pytest.raises(ValueError):
        V.engram_beam_fork(parents, pool, history=torch.zeros((2, 3, 4), dtype=torch.int64,
                                                              device="cuda"))
    with pytest.raises(ValueError):
        V.engram_beam_fork(parents, pool, tokens=parents, new_len=2,
                           history=torch.zeros((2, 3, 0), dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        V.engram_beam_fork(parents, pool, tokens=parents)             # without a history
    with pytest.raises(V.EngramError):
        V.engram_beam_fork(parents, [pool, pool])                     # one pool twice
    with pytest.raises(V.EngramError):
        V.engram_beam_fork(parents, pool, new_slots=parents)
    with pytest.raises(V.EngramError):
        V.engram_beam_fork(parents, pool[:5])                         # fewer slots than beams
    with pytest.raises(V.EngramError):
        V.engram_beam_fork(parents, torch.zeros((6, 3), device="cuda"))   # 12 bytes a slot
    with pytest.raises(V.EngramError):
        V.engram_beam_fork(parents, pool, slots=parents, new_slots=parents)
