"""The selection of a beam search where a mask's large finite value is among what it chooses from:
beams with nothing else, fewer allowed ids than are asked for."""
import math

import pytest
import torch

from tests import vocab_reference as R
from tests.gpu_helpers import needs_gpu
from tests.test_gpu_beam import check, logits

pytestmark = needs_gpu
V = pytest.importorskip("gram_hashed_embedding_amd.vocab")

BF, F32 = torch.bfloat16, torch.float32


def beam_values(z, scores, finished=None, eos=-1):
    """R.beam_values with the largest logit taken off before the sum's logarithm, which 1e30 and
    more would not hold."""
    for b in range(z.shape[0]):
        x = z[b].double()
        most = x.amax(1, keepdim=True)
        ok = torch.isfinite(most) & torch.isfinite(scores[b].double())[:, None]
        every = scores[b].double()[:, None] + ((x - most) - (x - most).exp().sum(1, True).log())
        every = torch.where(ok, every, -math.inf)
        if finished is not None:
            for w in finished[b].nonzero().flatten().tolist():
                every[w] = -math.inf
                every[w, eos] = scores[b, w]
        yield every


@pytest.fixture(autouse=True)
def reference(monkeypatch):
    monkeypatch.setattr(R, "beam_values", beam_values)


MASKS = [(torch.finfo(BF).min, BF), (torch.finfo(F32).min, F32), (-1e30, BF), (-1e30, F32),
         (-1e9, F32)]


@pytest.mark.parametrize("mask, dtype", MASKS)
@pytest.mark.parametrize("vocab", [1, 5, 700, 40000])
def test_masked_beams(vocab, mask, dtype):
    z, s = logits(4, 3, vocab, dtype, seed=vocab)
    s = s * 0.05 - torch.arange(3, device="cuda")     # beams apart by less than log(vocab)
    z[0, 1] = mask
    z[1, 0] = z[1, 2] = mask
    z[2] = mask
    z[3, 1, : vocab // 2] = mask
    finished = torch.zeros((4, 3), dtype=torch.bool, device="cuda")
    finished[1, 1] = True
    for count in (1, 7, 64):
        check(z, s, count)
        check(z, s, count, finished, vocab - 1)
    if vocab > 100:
        got = V.engram_beam_select(z, s, 3)
        # (a third of a beam's probability is more than 1 / vocab of another's)
        assert int(got.parents[0, 0]) != 1
        assert got.parents[2].tolist() == [0, 0, 0] and got.tokens[2].tolist() == [0, 1, 2]


@pytest.mark.parametrize("mask, dtype", MASKS)
@pytest.mark.parametrize("vocab, beams", [(300, 4), (30000, 4), (3001, 64), (151936, 5)])
def test_fewer_allowed_than_asked_for(vocab, beams, mask, dtype):
    """The rest is the mask's, equal ones by place: more of them than are listed at a time."""
    z, s = logits(2, beams, vocab, dtype, seed=beams)
    keep = torch.rand((2, beams, vocab), device="cuda") < 2.0 / vocab
    keep[:, :, vocab // 3] = True
    z = torch.where(keep, z, torch.full_like(z, mask))
    check(z, s, 64)
    check(z, s, 10)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("vocab, stride", [(400, 400), (1003, 1003), (1003, 1024), (50257, 50257),
                                           (151936, 151941)])
def test_beams_that_are_copies(vocab, stride, dtype):
    """Equal beams tie to the last bit wherever their rows lie: the lower one comes first."""
    z, _ = logits(2, 1, vocab, dtype, seed=vocab)
    wide = torch.zeros((13 * stride + 64,), dtype=dtype, device="cuda")
    s = torch.full((2, 6), -3.0, device="cuda")
    for first in (0, 1, 7, 32):
        part = wide.as_strided((12, vocab), (stride, 1), first)
        part.copy_(z.expand(2, 6, vocab).reshape(12, vocab))
        got = V.engram_beam_select(part, s, 16)
        for b in range(2):
            order = torch.sort(z[b].float().expand(6, vocab).flatten(), descending=True,
                               stable=True).indices[:16]
            assert torch.equal(got.parents[b], order // vocab)
            assert torch.equal(got.tokens[b], order % vocab)
