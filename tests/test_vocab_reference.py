"""The plain implementations that the vocabulary operators are compared with: the gradient against
differences of the loss, a label's cross entropy, a beam search's choice against a sorted list,
and a reordering against copies made one by one."""
import math
import random

import pytest
import torch

from tests import vocab_reference as R


@pytest.mark.parametrize("target", ["kept", "part", "rest"])
@pytest.mark.parametrize("temperature", [1.0, 0.5, 3.0])
def test_gradient_against_differences(target, temperature):
    g = torch.Generator().manual_seed(5)
    rows, vocab, top = 3, 11, 4
    z = torch.randn((rows, vocab), generator=g, dtype=torch.float64)
    ids = torch.tensor([[1, 4, 4, -1], [0, 10, 3, 2], [-1, -1, -1, -1]])
    y = torch.randn((rows, top), generator=g, dtype=torch.float64)
    lse = None if target == "kept" else torch.logsumexp(y / temperature, 1) + 0.7
    kw = dict(teacher_lse=lse, rest=target == "rest", temperature=temperature)
    w = torch.tensor([0.7, -1.3, 2.0])
    grad = R.distill(z, ids, y, grad_loss=w, **kw)["grad"]
    for v in range(vocab):
        step = torch.zeros_like(z)
        step[:, v] = 1e-5
        up, down = (R.distill(z + s, ids, y, **kw)["loss"] for s in (step, -step))
        # (a central difference is off by a sixth of the third derivative times 1e-10, and by
        # the rounding of the losses, 1e-15 / 1e-5)
        assert torch.allclose(grad[:, v], w * (up - down) / 2e-5, rtol=0, atol=1e-8)


def test_one_entry_is_cross_entropy():
    z = torch.randn((5, 9), dtype=torch.float64)
    labels = torch.tensor([0, 8, 3, 3, 5])
    got = R.distill(z, labels[:, None], torch.zeros((5, 1)), grad_loss=torch.ones(5))
    want = torch.nn.functional.cross_entropy(z, labels, reduction="none")
    assert torch.allclose(got["loss"], want, rtol=1e-12)
    q = torch.softmax(z, 1)
    q[torch.arange(5), labels] -= 1
    assert torch.allclose(got["grad"], q, atol=1e-14)


def test_a_teacher_that_is_the_student_loses_nothing():
    z = torch.randn((4, 20), dtype=torch.float64)
    top = torch.topk(z, 6, dim=1)
    got = R.distill(z, top.indices, top.values, teacher_lse=torch.logsumexp(z, 1), rest=True,
                    grad_loss=torch.ones(4))
    assert float(got["loss"].abs().max()) < 1e-14 and float(got["grad"].abs().max()) < 1e-14


def test_choice_and_its_ties():
    z = torch.zeros((1, 3, 4))
    scores = torch.tensor([[0.0, 0.0, -1.0]])
    s, p, t, e = R.beam_select(z, scores, 5, eos=1)
    assert p.tolist() == [[0, 0, 0, 0, 1]] and t.tolist() == [[0, 1, 2, 3, 0]]
    assert e.tolist() == [[False, True, False, False, False]]
    assert torch.allclose(s, torch.full((1, 5), -math.log(4), dtype=torch.float64))
    s, p, t, e = R.beam_select(z, scores, 3, finished=torch.tensor([[True, False, True]]), eos=2)
    assert p.tolist() == [[0, 2, 1]]
    assert t[0, 0] == 2 and bool(e[0, 0]) and s[0, 0] == 0.0


def test_reordering():
    rng = random.Random(3)
    for _ in range(50):
        beams = rng.randint(1, 8)
        slots = [rng.sample(range(40), beams)]
        parents = [[rng.randint(-1, beams) for _ in range(beams)]]
        new, copies, bad = R.beam_fork(parents, slots, 40)
        assert sorted(new[0]) == sorted(slots[0])
        state = {s: s for s in range(40)}
        for to, source in copies.items():
            state[to] = source
            assert source not in copies  # nothing is read that is written
        for p, s in zip(parents[0], new[0]):
            if 0 <= p < beams:
                assert state[s] == slots[0][p]
        assert bad == sum(p == beams for p in parents[0])
