"""Every gradient of the example's layer against one of its forward in 64 bits.

Bound, of the whole gradient's size (its root sum of squares): what the backward
reads as x and y are 8-bit codes, off by m / 127 / sqrt(12) at random, 0.8% of a
block's spread where its largest of 128 values is 3.5 spreads; x and y enter each
gradient at most twice between them, and some six roundings to bf16 add 0.11%
each: 1.2% together.  3% leaves the rest to chance, and the gate's share of the
stream's gradient, which a missing term would take, is over 10%."""
import math

import pytest
import torch

from tests.gpu_helpers import needs_gpu
from tests.test_gpu_layer_example import load

pytestmark = needs_gpu

SHARE = 0.03


def reference(net, tokens, e, target, gate_moves=True):
    """float64 gradients of 0.5 * sum((next - target)^2), from the layer's formulas; e: the looked
    up rows.  gate_moves false: without the gate's part of the stream's gradient."""
    w = {k: v.double().requires_grad_() for k, v in net.w.items()}
    e = e.double().requires_grad_()
    C, G = net.channels, net.heads

    def norm(x, weight):
        g = x.unflatten(-1, (G, C // G))
        return (g / (g.square().mean(-1, keepdim=True) + 1e-6).sqrt()).flatten(-2) * weight

    r = math.sqrt(C) * w["embed"][tokens]
    x = norm(e, w["w_in"])
    taps = w["conv"].shape[1]
    back = (taps - 1) * net.dilation
    past = torch.nn.functional.pad(x, (0, 0, back, 0))
    y = w["bias"] + sum(past[:, k * net.dilation:k * net.dilation + x.shape[1]] * w["conv"][:, k]
                        for k in range(taps))
    stream = r if gate_moves else r.detach()
    gate = torch.sigmoid((stream.flatten(0, 1) @ w["gate"]).view(*r.shape[:2], G))
    out = r + w["scale"] * gate.repeat_interleave(C // G, -1) * norm(y, w["w_post"])
    nxt = norm(out, w["w_next"])
    names = list(w)
    grads = torch.autograd.grad(0.5 * (nxt - target).square().sum(), [w[k] for k in names] + [e])
    return dict(zip(names + ["looked_up"], grads))


def off(got, want):
    return float((got.double() - want).square().sum().sqrt() / want.square().sum().sqrt())


def test_every_gradient_of_the_layer(monkeypatch):
    m = load()
    from gram_hashed_embedding_amd import workloads
    wl = workloads.tiny()
    net = m.NgramLayer(wl, vocab=1000, seed=5)
    net.master["gate"] *= 10  # so that the gate's part of the stream's gradient is a large one
    net.cast()
    tokens = torch.from_numpy(wl.tokens(2)).cuda()
    target = workloads.make_bf16((*tokens.shape, net.channels), 9, "cuda").double()
    start = {k: v.clone() for k, v in net.master.items()}
    seen = {}
    monkeypatch.setattr(m.E, "engram_scatter_apply_signsgd",
                        lambda grads, *a, **k: seen.update(looked_up=grads.clone()))
    out, kept = net.forward(tokens)
    want = reference(net, tokens, kept["e"], target)
    fixed = reference(net, tokens, kept["e"], target, gate_moves=False)
    net.backward((out.double() - target).to(torch.bfloat16), kept, 1.0, 0.0)
    got = {k: start[k] - v for k, v in net.master.items()}
    got["looked_up"] = seen["looked_up"].view(want["looked_up"].shape)
    assert set(got) == set(want)
    for k in want:
        share = off(got[k], want[k])
        print(f"{k}: {share:.4f}")
        assert share < SHARE, k
    print("the gate's share:", off(fixed["embed"], want["embed"]))
    assert off(fixed["embed"], want["embed"]) > 0.1
