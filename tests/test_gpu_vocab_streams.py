"""The vocabulary operators on another stream than the current one, on a stream of another
device, and captured into HIP graphs that are replayed with new inputs beside eager work."""
import contextlib
import types

import pytest
import torch

from tests.gpu_helpers import needs_gpu

pytestmark = needs_gpu
V = pytest.importorskip("gram_hashed_embedding_amd.vocab")

BF = torch.bfloat16


def make(seed, vocab=3001):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.empty(shape, device="cuda").normal_(0.0, 2.0, generator=g)

    z = normal(12, vocab).to(BF)
    y = z.float() + normal(12, vocab)
    top = torch.topk(y, 6, dim=1)
    return dict(z=z, ids=top.indices.contiguous(), y=top.values.contiguous(),
                lse=torch.logsumexp(y, 1), w=torch.rand(12, generator=g, device="cuda"),
                scores=normal(3, 4) - 9.0,
                history=torch.randint(0, 999, (3, 4, 5), generator=g, device="cuda"),
                pool=normal(14, 40, 8).to(BF),
                slots=torch.randperm(14, generator=g, device="cuda")[:12].view(3, 4).contiguous())


def distill(s, **kw):
    return V.engram_distill(s["z"], s["ids"], s["y"], teacher_lse=s["lse"], rest=True,
                            grad_loss=s["w"], **kw)


def backward(s, d, **kw):
    return V.engram_distill_backward(s["w"], s["z"], s["ids"], s["y"], d.lse, lse_rest=d.lse_rest,
                                     teacher_lse=s["lse"], **kw)


def step(s, stream=None):
    """Everything, as a program calls it; the pool is put back first."""
    pool = s["pool"].clone()
    d = distill(s, stream=stream)
    b = V.engram_beam_select(s["z"], s["scores"], eos=7, stream=stream)
    f = V.engram_beam_fork(b.parents, pool, slots=s["slots"], tokens=b.tokens,
                           history=s["history"], stream=stream)
    return [d.loss, d.lse, d.lse_rest, d.grad, backward(s, d, stream=stream), *b, *f, pool]


CALLS = ["distill", "backward", "select", "fork"]


def call(name, s, stream):
    if name == "distill":
        return distill(s, stream=stream)
    if name == "backward":
        lse = torch.ones(12, device="cuda")
        return backward(s, V.Distill(lse, lse, lse, None), stream=stream)
    if name == "select":
        return V.engram_beam_select(s["z"], s["scores"], stream=stream)
    return V.engram_beam_fork(s["slots"] % 4, s["pool"], slots=s["slots"], stream=stream)


@pytest.mark.parametrize("name", CALLS)
def test_a_stream_of_another_device_is_refused(name, monkeypatch):
    """A stand-in for a stream of a second device, which this machine may not have."""
    s = make(1)
    torch.cuda.synchronize()
    other = torch.device("cuda", torch.cuda.current_device() + 1)
    stream = types.SimpleNamespace(device=other, device_index=other.index, cuda_stream=0)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    with pytest.raises(ValueError, match="stream"):
        call(name, s, stream)


@pytest.mark.parametrize("vocab", [3001, 100003])
def test_a_stream_of_the_tensors_device(vocab):
    s = make(2, vocab)
    want = step(s)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        pool = s["pool"]
        s["pool"] = pool.clone()
    got = step(s, stream=None)
    with torch.cuda.stream(side):
        more = step(s)
    side.synchronize()
    torch.cuda.synchronize()
    for x, y, z in zip(want, got, more):
        assert torch.equal(x, y) and torch.equal(x, z)
    d = distill(s, stream=side)
    side.synchronize()
    assert torch.equal(d.grad, want[3])


def test_two_streams_at_once():
    """Calls of different inputs side by side do not meet."""
    a, b = make(3, 100003), make(4, 100003)
    want = step(a), step(b)
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for k, (s, stream) in enumerate(zip((a, b), streams)):
            with torch.cuda.stream(stream):
                got[k].append(step(s))
    torch.cuda.synchronize()
    for k in range(2):
        for run in got[k]:
            assert all(torch.equal(x, y) for x, y in zip(run, want[k]))


@pytest.mark.parametrize("vocab", [3001, 100003])
def test_captured_and_replayed(vocab):
    """Two graphs that share a workspace, replayed in turn with new inputs, eager calls and
    synchronizations between."""
    need = max(V.engram_distill_workspace(12, vocab, grad=True),
               V.engram_beam_select_workspace(3, 4, vocab), 16)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    sets = [make(5, vocab), make(6, vocab)]
    graphs = []

    def run(s):
        pool = s["pool"].clone()
        d = distill(s, workspace=ws)
        b = V.engram_beam_select(s["z"], s["scores"], eos=7, workspace=ws)
        f = V.engram_beam_fork(b.parents, pool, slots=s["slots"], tokens=b.tokens,
                               history=s["history"])
        return [d.loss, d.lse, d.lse_rest, d.grad, backward(s, d), *b, *f, pool]

    for s in sets:
        run(s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = run(s)
        graphs.append((g, out))
    for turn in range(4):
        for k, (s, (g, out)) in enumerate(zip(sets, graphs)):
            fresh = make(10 + 7 * turn + k, vocab)
            for name, t in s.items():
                t.copy_(fresh[name])
            g.replay()
            if turn % 2:
                torch.cuda.synchronize()
            want = step(fresh)
            for x, y in zip(out, want):
                assert torch.equal(x, y)
