"""The example that runs the layer operators together: training lowers the
loss, and serving token by token gives what the whole sequence gives."""
import importlib.util
import os

import pytest
import torch

from tests.gpu_helpers import needs_gpu

pytestmark = needs_gpu
pytest.importorskip("gram_hashed_embedding_amd.layer")

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "ngram_layer.py")


def load():
    spec = importlib.util.spec_from_file_location("ngram_layer", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def test_trains_and_serves():
    losses, worst = load().main(["--steps", "12"])
    assert all(b < a for a, b in zip(losses, losses[1:])) and losses[-1] < 0.97 * losses[0]
    # a token's norms lie in single lanes' groups either way, and the gate's
    # product may be taken in another order: a step of bf16
    assert worst <= 2.0 ** -5


def test_gradients_of_the_whole_layer_against_differences():
    """A directional difference of the loss in 64 bits of the loss alone: the layer's weights
    moved along their gradients change it as the gradients say (within bf16's noise)."""
    m = load()
    from gram_hashed_embedding_amd import workloads
    wl = workloads.tiny()
    net = m.NgramLayer(wl, vocab=1000, seed=3)
    tokens = torch.from_numpy(wl.tokens(1)).cuda()
    target = workloads.make_bf16((*tokens.shape, net.channels), 8, "cuda")

    def loss():
        out, kept = net.forward(tokens)
        return out.double() - target.double(), kept

    diff, kept = loss()
    before = float(0.5 * diff.square().sum())
    start = {k: v.clone() for k, v in net.master.items()}
    table = net.table.clone()
    net.backward(diff.to(torch.bfloat16), kept, 1.0, 0.0)
    assert torch.equal(net.table, table)           # a zero learning rate moves nothing
    grads = {k: start[k] - v for k, v in net.master.items()}
    for k in ("w_post", "scale", "w_next", "conv", "w_in"):
        # a step along the gradient that should lower the loss by about 1% of it
        size = 0.01 * before / float(grads[k].double().square().sum())
        net.master = {n: v.clone() for n, v in start.items()}
        net.master[k] -= size * grads[k]
        moved = start[k].to(torch.bfloat16).double() - net.master[k].to(torch.bfloat16).double()
        net.cast()
        after = float(0.5 * loss()[0].square().sum())
        predicted = float((moved * grads[k].double()).sum())
        assert abs((before - after) - predicted) < 0.25 * predicted, k
