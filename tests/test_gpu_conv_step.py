"""The PLE convolution for single tokens on the GPU: bit for bit what
engram_ple_conv gives for the whole sequence."""
import pytest
import torch

from gram_hashed_embedding_amd import engram as E
from gram_hashed_embedding_amd import workloads
from tests.gpu_helpers import needs_gpu, release

pytestmark = needs_gpu
L = pytest.importorskip("gram_hashed_embedding_amd.layer")


def setup(B, S, C, K, seed, bias=True):
    x = workloads.make_bf16((B, S, C), seed, "cuda")
    w = workloads.make_bf16((C, K), seed + 1, "cuda", std=0.5)
    return x, w, workloads.make_bf16((C,), seed + 2, "cuda") if bias else None


def garbage(*shape):
    return torch.full(shape, float("nan"), dtype=torch.bfloat16, device="cuda")


@pytest.mark.parametrize("K,d", [(4, 1), (4, 3), (4, 8), (1, 1), (2, 5), (5, 2), (16, 1)])
@pytest.mark.parametrize("more", [0, 3])
@pytest.mark.parametrize("tokens", [1, 2, 5])
def test_a_sequence_token_by_token(K, d, more, tokens):
    """From an empty ring (its contents never read) to past its end, with and without rows to
    spare."""
    B, S, C = 3, 30, 40
    x, w, bias = setup(B, S, C, K, 100 * K + d)
    want = E.engram_ple_conv(x, w, d, bias=bias)
    ring = garbage(B, max(1, (K - 1) * d + more), C)
    for t in range(0, S, tokens):
        pos = torch.full((B,), t, dtype=torch.int64, device="cuda")
        got = L.engram_ple_conv_step(x[:, t:t + tokens].contiguous(), ring, w, d, pos, bias=bias)
        assert torch.equal(got, want[:, t:t + tokens]), t


@pytest.mark.parametrize("S", [1, 5, 9, 40])
def test_from_a_prompt(S):
    """The prompt in one call of the convolution, its last inputs written to the ring, then
    tokens one at a time."""
    B, C, K, d, more = 2, 264, 4, 3, 6
    x, w, bias = setup(B, S + more, C, K, S)
    want = E.engram_ple_conv(x, w, d, bias=bias)
    ring = garbage(B, 9, C)
    first = max(0, S - 9)
    pos = torch.full((B,), first, dtype=torch.int64, device="cuda")
    assert L.engram_ple_conv_step(x[:, first:S].contiguous(), ring, w, d, pos,
                                  write_only=True) is None
    for t in range(S, S + more):
        pos = torch.full((B,), t, dtype=torch.int64, device="cuda")
        got = L.engram_ple_conv_step(x[:, t].contiguous(), ring, w, d, pos, bias=bias)
        assert torch.equal(got, want[:, t])


def test_slots_positions_and_unused_entries():
    """Sequences at different positions in scattered rings; an entry of -1 gives zeros and
    touches nothing; a bad ring or position does the same and is counted."""
    B, C, K, d = 6, 24, 4, 2
    x, w, bias = setup(B, 20, C, K, 3)
    want = E.engram_ple_conv(x, w, d, bias=bias)
    ring = workloads.make_bf16((9, 8, C), 50, "cuda")
    before = ring.clone()
    slots = torch.tensor([7, -1, 2, 9, 0, 5], device="cuda")
    at = [13, 4, 0, 3, 6, -2]
    for b in (0, 2, 4):  # the inputs before each position, where the ring keeps them
        for t in range(max(0, at[b] - 8), at[b]):
            ring[slots[b], t % 8] = x[b, t]
    filled = ring.clone()
    token = torch.stack([x[b, max(at[b], 0)] for b in range(B)])
    err = torch.zeros(1, dtype=torch.int64, device="cuda")
    out = L.engram_ple_conv_step(token, ring, w, d, torch.tensor(at, device="cuda"), slots=slots,
                                 bias=bias, err_count=err)
    for b in range(B):
        if b in (0, 2, 4):
            assert torch.equal(out[b], want[b, at[b]])
            filled[slots[b], at[b] % 8] = token[b]
        else:
            assert bool((out[b] == 0).all())
    assert torch.equal(ring, filled) and int(err) == 2
    for s in (1, 3, 4, 6, 8, 5):
        assert torch.equal(ring[s], before[s])


@pytest.mark.parametrize("pos", [2 ** 63 - 1, 2 ** 63 - 3, 2 ** 63 - 4, -1, -2 ** 63])
def test_positions_out_of_range(pos):
    """Positions whose tokens would pass the largest number touch nothing and are counted; the
    last ones that do not are as good as any."""
    x, w, bias = setup(2, 3, 16, 4, 70)
    ring = garbage(2, 8, 16)
    err = torch.zeros(1, dtype=torch.int64, device="cuda")
    at = torch.tensor([pos, 2 ** 63 - 1 - 3], device="cuda")
    out = L.engram_ple_conv_step(x, ring, w, 2, at, bias=bias, err_count=err)
    good = pos == 2 ** 63 - 1 - 3
    assert int(err) == (0 if good else 1)
    assert bool(torch.isnan(ring[0]).all()) != good and not bool(torch.isnan(ring[1]).all())
    assert good or bool((out[0] == 0).all())


def test_tokens_taken_back():
    """With rows to spare, drafted tokens are overwritten by the accepted ones."""
    B, C, d = 2, 16, 3
    x, w, bias = setup(B, 20, C, 4, 9)
    want = E.engram_ple_conv(x, w, d, bias=bias)
    ring = garbage(B, 9 + 4, C)
    pos = torch.zeros((B,), dtype=torch.int64, device="cuda")
    L.engram_ple_conv_step(x[:, :10].contiguous(), ring, w, d, pos, bias=bias)
    draft = garbage(B, 4, C)
    L.engram_ple_conv_step(draft, ring, w, d, pos + 10, bias=bias)
    for t in range(10, 20):
        got = L.engram_ple_conv_step(x[:, t:t + 1].contiguous(), ring, w, d, pos + t, bias=bias)
        assert torch.equal(got, want[:, t:t + 1])


def test_empty():
    w = torch.ones((16, 4), dtype=torch.bfloat16, device="cuda")
    ring = garbage(2, 3, 16)
    for shape in ((0, 1, 16), (2, 0, 16)):
        x = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        pos = torch.zeros((shape[0],), dtype=torch.int64, device="cuda")
        assert L.engram_ple_conv_step(x, ring, w, 1, pos).shape == shape
    assert bool(torch.isnan(ring).all())


def test_replayed_graph():
    """A decoding step captured once and replayed with new tokens and positions in place."""
    B, S, C, d = 4, 25, 136, 4
    x, w, bias = setup(B, S, C, 4, 30)
    want = E.engram_ple_conv(x, w, d, bias=bias)
    ring, token = garbage(B, 16, C), x[:, 0].clone()
    pos, out = torch.zeros((B,), dtype=torch.int64, device="cuda"), torch.empty_like(token)
    L.engram_ple_conv_step(token, ring, w, d, pos, bias=bias, out=out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.engram_ple_conv_step(token, ring, w, d, pos, bias=bias, out=out)
    for t in range(S):
        token.copy_(x[:, t])
        pos.fill_(t)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[:, t]), t


def test_offsets_past_32_bits():
    C, rows = 2048, 16
    count = 2 ** 31 // (C * rows) + 3
    print(f"rings [{count}, {rows}, {C}]", flush=True)
    x, w, bias = setup(1, 14, C, 4, 40)
    want = E.engram_ple_conv(x, w, 4, bias=bias)
    ring = torch.empty((count, rows, C), dtype=torch.bfloat16, device="cuda")
    slot = torch.tensor([count - 1], device="cuda")
    for t in range(14):
        pos = torch.full((1,), t, dtype=torch.int64, device="cuda")
        got = L.engram_ple_conv_step(x[:, t].contiguous(), ring, w, 4, pos, slots=slot, bias=bias)
        assert torch.equal(got, want[:, t])
    del ring
    release()
