"""The example's use of the vocabulary operators together: a distillation step's gradients, and
a beam search whose beams carry the rings and histories that their tokens say."""

import pytest
import torch

from tests import vocab_reference as R
from tests.gpu_helpers import needs_gpu
from tests.test_gpu_layer_example import load

pytestmark = needs_gpu
pytest.importorskip("gram_hashed_embedding_amd.vocab")


def net_and_tokens(seed):
    m = load()
    from gram_hashed_embedding_amd import workloads
    wl = workloads.tiny()
    net = m.NgramLayer(wl, vocab=1000, seed=seed)
    return net, torch.from_numpy(wl.tokens(seed)).cuda()


def test_distillation_step():
    """The step takes the embedding's rows and the layer where the definition's gradient, put
    through the same products, takes them."""
    net, tokens = net_and_tokens(4)
    hidden, _ = net.forward(tokens)
    z = net.logits(hidden)
    g = torch.Generator(device="cuda").manual_seed(2)
    y = z.float() + torch.empty(z.shape, device="cuda").normal_(0.0, 1.0, generator=g)
    top = torch.topk(y, 8, dim=-1)
    ids, values, lse = top.indices.contiguous(), top.values.contiguous(), torch.logsumexp(y, -1)
    n = tokens.numel()
    weight = torch.full((n,), 1.0 / n)
    want = R.distill(z.view(n, -1), ids.view(n, -1), values.view(n, -1), lse.view(n), True, 1.0,
                     weight)
    before = {k: v.clone() for k, v in net.master.items()}
    rows = (want["grad"].to(torch.bfloat16).t().contiguous() @ hidden.view(n, -1)).float()
    loss = net.distill(tokens, ids, values, 1.0, 0.0, teacher_lse=lse, rest=True)
    # (a mean of n: their own error and the mean's rounding)
    assert abs(float(loss) - float(want["loss"].mean())) <= \
        2 * R.SUM + 2.0 ** -23 * float(want["loss"].abs().max())
    moved = {k: before[k] - v for k, v in net.master.items()}
    for k in ("w_post", "scale", "w_next", "conv", "w_in", "gate"):
        assert bool(moved[k].abs().max() > 0) and bool(torch.isfinite(moved[k]).all()), k
    # rows of tokens that the batch does not hold have the vocabulary's part alone
    held = torch.zeros(1000, dtype=torch.bool, device="cuda").index_fill_(0, tokens.flatten(), True)
    a, b = moved["embed"][~held], rows[~held]
    assert a.shape[0] > 0
    # Each product sums n terms of bf16 gradients that may differ by a step of bf16 (2^-8 of the
    # larger), of values below |hidden|; the update is rounded at the size of the master.
    bound = (want["grad"].abs().t() @ hidden.view(n, -1).abs().double())[~held] * 2.0 ** -7
    size = before["embed"][~held].abs().double() * 2.0 ** -23
    rounding = b.abs().double() * 2.0 ** -7  # the products' own bf16 results
    assert bool(((a - b).abs().double() <= bound + size + rounding + 1e-9).all())


@pytest.mark.parametrize("eos", [-1, 17])
def test_beams_carry_their_states(eos):
    """Every beam's score is the sum of its tokens' log-probabilities in a whole-sequence forward
    of them: so every ring and history went with its beam."""
    net, tokens = net_and_tokens(6)
    beams, steps = 5, 9
    first = tokens[:, 0].contiguous()
    found, scores, finished = net.search(first, beams, steps, eos)
    batch = first.shape[0]
    assert found.shape == (batch, beams, steps + 1) and bool((found[:, :, 0] == first[:, None]).all())
    assert bool((scores[:, 1:] <= scores[:, :-1]).all())
    assert bool(torch.isfinite(scores).all()) and bool((found >= 0).all())
    flat = found.view(batch * beams, steps + 1)
    whole, _ = net.forward(flat[:, :-1].contiguous())
    one = torch.log_softmax(net.logits(whole).double(), -1).gather(2, flat[:, 1:, None])[..., 0]
    if eos >= 0:
        # after its end a beam's tokens are eos and cost nothing
        ended = (flat[:, 1:] == eos).cumsum(1)
        assert bool((((flat[:, 1:] == eos) == (ended > 0)))[ended > 0].all())
        one = torch.where(ended > 1, 0.0, one)
        assert torch.equal(finished.view(-1), ended[:, -1] > 0)
    # The layer one token at a time agrees with the whole sequence within a step of bf16 (2^-5 at
    # values below 8); a logit is a product of 64 channels of these with rows of about 0.02, and a
    # bf16 value below 8, off by 2^-6 more; a log-probability twice that a step.
    width = float(net.w["embed"].float().abs().sum(1).max())
    tol = steps * 2 * (2.0 ** -5 * width + 2.0 ** -6)
    off = (one.sum(1).view(batch, beams) - scores.double()).abs()
    assert float(off.max()) <= tol
    # distinct hypotheses
    for b in range(batch):
        assert len({tuple(r) for r in found[b].tolist()}) == beams
