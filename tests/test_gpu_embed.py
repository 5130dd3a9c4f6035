"""The scaled token embedding and its gradient on the GPU, bit for bit: the
forward is one product rounded once; the gradient's sums are exact in fp64 for
these gradients, and rounded once (to bf16: once more)."""
import numpy as np
import pytest
import torch

from gram_hashed_embedding_amd import workloads
from tests import layer_reference as ref
from tests.gpu_helpers import dev, needs_gpu, release

pytestmark = needs_gpu
L = pytest.importorskip("gram_hashed_embedding_amd.layer")


def tokens(n, rows, seed, hot=0.0, bad=0.01):
    rng = np.random.default_rng(seed)
    t = rng.integers(0, rows, n)
    t[rng.random(n) < hot] = rows // 2
    t[rng.random(n) < bad] = -1
    if n > 3:
        t[0], t[n - 1] = rows - 1, 0
    return t.astype(np.int64)


def check_forward(n, rows, channels, dtype, seed, scale=np.sqrt(77.0)):
    t = tokens(n, rows, seed)
    table = workloads.make_bf16((rows, channels), seed, "cuda", std=0.02)
    out = L.engram_embed(dev(t), table, scale, out_dtype=dtype)
    h = table.float().cpu().numpy()
    want = h[np.maximum(t, 0)] * np.float32(scale)
    want[t < 0] = 0
    if dtype == torch.bfloat16:
        want = ref.bf16(want)
    assert np.array_equal(ref.f64(out), want.astype(np.float64))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,rows,channels", [(1, 5, 8), (3, 1, 16), (1000, 300, 24),
                                             (77, 5000, 1000), (513, 999, 2048), (9, 40, 8200)])
def test_forward(n, rows, channels, dtype):
    check_forward(n, rows, channels, dtype, n + channels)


def test_forward_invalid_ids():
    """Invalid ids give zero rows and are counted, padding is not; rows of NaN that no token
    names stay out."""
    table = torch.full((10, 16), float("nan"), dtype=torch.bfloat16, device="cuda")
    table[3] = 1
    t = torch.tensor([[3, -1, 10, -2], [2 ** 40, 3, -2 ** 63, 3]], device="cuda")
    err = torch.zeros(1, dtype=torch.int64, device="cuda")
    out = L.engram_embed(t, table, 2.0, err_count=err)
    assert out.shape == (2, 4, 16) and int(err) == 4
    assert bool((out[t == 3] == 2).all()) and bool((out[t != 3] == 0).all())


def grad_case(n, rows, channels, seed, hot=0.0, dtype=torch.float32, scale=3.7):
    t = tokens(n, rows, seed, hot)
    g = workloads.make_bf16((n, channels), seed + 1, "cuda")
    got = L.engram_embed_grad(dev(t), g, rows, scale, grad_dtype=dtype)
    want = ref.embed_grad(t, ref.f64(g), rows, scale).astype(np.float64)
    if dtype == torch.bfloat16:
        want = ref.bf16(want)
    assert got.shape == (rows, channels) and np.array_equal(ref.f64(got), want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,rows,channels", [(1, 5, 8), (1, 30000, 64), (5, 1, 24), (63, 7, 8),
                                             (64, 1, 16), (65, 2, 16), (4099, 4062, 32),
                                             (9000, 700, 136), (700, 9001, 1000),
                                             (300, 50, 4104)])
def test_gradient(n, rows, channels, dtype):
    grad_case(n, rows, channels, n + rows, dtype=dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("n,rows,channels,hot", [(1, 5, 8, 0), (4099, 300, 136, 0.5),
                                                 (20000, 900, 2056, 0.3)])
def test_float_gradients(n, rows, channels, hot, dtype):
    """Float gradients (of a float stream), of values that bf16 does not hold: their 24 bits over
    a factor of 2^11 and up to 2^13 terms leave the fp64 sums exact."""
    t = tokens(n, rows, n, hot)
    g = torch.randn((n, channels), generator=torch.Generator("cuda").manual_seed(n),
                    device="cuda").clamp_(-8, 8)
    g[g.abs() < 2.0 ** -8] = 0
    got = L.engram_embed_grad(dev(t), g, rows, 0.7, grad_dtype=dtype)
    want = ref.embed_grad(t, ref.f64(g), rows, 0.7).astype(np.float64)
    if dtype == torch.bfloat16:
        want = ref.bf16(want)
    assert np.array_equal(ref.f64(got), want)


@pytest.mark.parametrize("n", [128, 1000, 8192, 8193, 20000, 65536, 65537, 70000])
@pytest.mark.parametrize("hot", [0.3, 0.95, 1.0])
@pytest.mark.parametrize("channels", [8, 264])
def test_frequent_tokens(n, hot, channels):
    """Runs of thousands of one token, and a batch of nothing else."""
    grad_case(n, 1000, channels, n, hot)


def test_gradient_all_padding():
    t = torch.full((300,), -1, dtype=torch.int64, device="cuda")
    g = torch.full((300, 16), float("nan"), dtype=torch.bfloat16, device="cuda")
    got = L.engram_embed_grad(t, g, 40, 2.0)
    assert bool((got == 0).all())


def test_gradient_invalid_ids():
    """Rows of NaN whose token is padding or invalid reach nothing."""
    t = torch.tensor([4, -1, 7, 7, -5, 4], device="cuda")
    g = torch.ones((6, 8), dtype=torch.bfloat16, device="cuda")
    g[1] = g[2] = g[3] = g[4] = float("nan")
    err = torch.zeros(1, dtype=torch.int64, device="cuda")
    got = L.engram_embed_grad(t, g, 7, 0.5, err_count=err)
    want = torch.zeros((7, 8), device="cuda")
    want[4] = 1.0
    assert torch.equal(got, want) and int(err) == 3


def test_non_finite_gradients_stay_in_their_row():
    t = tokens(5000, 100, 3, hot=0.5, bad=0.0)
    g = workloads.make_bf16((5000, 24), 1, "cuda")
    g[int(np.nonzero(t == 50)[0][70]), 5] = float("nan")
    g[int(np.nonzero(t == 7)[0][0]), 6] = float("inf")
    got = L.engram_embed_grad(dev(t), g, 100, 1.0)
    bad = torch.zeros((100, 24), dtype=torch.bool, device="cuda")
    bad[50, 5] = bad[7, 6] = True
    assert torch.equal(~torch.isfinite(got), bad)


def test_accumulate():
    """Added to the rows that have tokens, the others untouched, NaN among them."""
    t = tokens(3000, 500, 5)
    t[t == 123] = -1
    g = workloads.make_bf16((3000, 40), 6, "cuda")
    start = torch.randn((500, 40), device="cuda")
    start[123] = float("nan")
    got = L.engram_embed_grad(dev(t), g, 500, 0.3, grad_table=start.clone(), accumulate=True)
    add = ref.embed_grad(t, ref.f64(g), 500, 0.3)
    want = start.cpu().numpy()
    named = np.isin(np.arange(500), t)
    want[named] = want[named] + add[named]
    assert np.array_equal(got.cpu().numpy(), want, equal_nan=True)
    with pytest.raises(L.EngramError):
        L.engram_embed_grad(dev(t), g, 500, 0.3, accumulate=True,
                            grad_table=torch.zeros((500, 40), dtype=torch.bfloat16, device="cuda"))


def test_empty():
    t = torch.empty((0,), dtype=torch.int64, device="cuda")
    table = torch.ones((3, 8), dtype=torch.bfloat16, device="cuda")
    assert L.engram_embed(t, table, 2.0).shape == (0, 8)
    g = torch.empty((0, 8), dtype=torch.bfloat16, device="cuda")
    full = torch.full((3, 8), 5.0, device="cuda")
    assert bool((L.engram_embed_grad(t, g, 3, grad_table=full.clone()) == 0).all())
    kept = L.engram_embed_grad(t, g, 3, grad_table=full.clone(), accumulate=True)
    assert torch.equal(kept, full)
    some = torch.tensor([0, 1], device="cuda")
    none = L.engram_embed_grad(some, torch.ones((2, 8), dtype=torch.bfloat16, device="cuda"), 0)
    assert none.shape == (0, 8)
    assert bool((L.engram_embed(some, table[:0], 1.0) == 0).all())


def test_against_differences():
    """The gradient along a direction against differences of the 64-bit forward."""
    t = tokens(400, 60, 8)
    table = workloads.make_bf16((60, 16), 1, "cuda")
    g = workloads.make_bf16((400, 16), 2, "cuda")
    got = ref.f64(L.engram_embed_grad(dev(t), g, 60, 1.5))
    h, gg = ref.f64(table), ref.f64(g)
    direction = np.random.default_rng(0).normal(size=h.shape)

    def loss(v):
        rows = v[np.maximum(t, 0)] * 1.5
        rows[t < 0] = 0
        return (rows * gg).sum()

    want = (loss(h + direction) - loss(h - direction)) / 2
    assert abs((got * direction).sum() - want) < 2.0 ** -20 * np.abs(got * direction).sum()


def test_side_stream_and_repeats():
    t = dev(tokens(30000, 2000, 4, hot=0.2))
    g = workloads.make_bf16((30000, 128), 5, "cuda")
    side = torch.cuda.Stream()
    a = L.engram_embed_grad(t, g, 2000, 2.0)
    side.wait_stream(torch.cuda.current_stream())
    b = L.engram_embed_grad(t, g, 2000, 2.0, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(a, b)


def test_replayed_graph():
    t = dev(tokens(5000, 800, 6, hot=0.3))
    g = workloads.make_bf16((5000, 64), 7, "cuda")
    out = torch.empty((800, 64), device="cuda")
    ws = torch.empty(L._lib.engram_embed_grad_workspace(5000, 64, 800), dtype=torch.uint8,
                     device="cuda")
    L.engram_embed_grad(t, g, 800, 2.0, grad_table=out, workspace=ws)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.engram_embed_grad(t, g, 800, 2.0, grad_table=out, workspace=ws)
    for i in range(4):
        t.copy_(dev(tokens(5000, 800, 60 + i, hot=0.3)))
        want = L.engram_embed_grad(t, g, 800, 2.0)
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), i


def test_offsets_past_32_bits():
    rows, channels = 2 ** 31 // 4096 + 9, 4096
    print(f"embedding of [{rows}, {channels}]", flush=True)
    table = torch.zeros((rows, channels), dtype=torch.bfloat16, device="cuda")
    table[-4:] = workloads.make_bf16((4, channels), 1, "cuda")
    t = torch.tensor([rows - 1, 3, rows - 4, rows - 2, rows - 2], device="cuda")
    out = L.engram_embed(t, table, 0.5, out_dtype=torch.float32)
    assert torch.equal(out, table[t].float() * 0.5)
    g = workloads.make_bf16((5, channels), 2, "cuda")
    grad = L.engram_embed_grad(t, g, rows, 1.0)
    assert torch.equal(grad[rows - 1], g[0].float()) and torch.equal(grad[3], g[1].float())
    assert torch.equal(grad[rows - 2], g[3].float() + g[4].float())
    assert int((grad != 0).any(1).sum()) == 4
    del table, grad
    release()
