"""The embedding's gradient into a table past 128 GB, more rows than one launch has
blocks for at the usual rows a block: every row written."""
import pytest
import torch

from gram_hashed_embedding_amd import workloads
from tests.gpu_helpers import needs_gpu, release

pytestmark = needs_gpu
L = pytest.importorskip("gram_hashed_embedding_amd.layer")


def test_table_past_128_gb():
    rows, channels = 2 ** 26 + 5, 1024
    need = rows * channels * 2
    release()
    if torch.cuda.mem_get_info()[0] < need + (8 << 30):
        pytest.skip("needs 146 GB of free device memory")
    print(f"embedding gradient into [{rows}, {channels}] bf16", flush=True)
    t = torch.tensor([rows - 1, 3, -1, 2 ** 25, rows - 1], device="cuda")
    g = workloads.make_bf16((5, channels), 2, "cuda")
    grad = torch.empty((rows, channels), dtype=torch.bfloat16, device="cuda")
    grad.fill_(float("nan"))
    L.engram_embed_grad(t, g, rows, 2.0, grad_table=grad)
    want = {3: 2 * g[1].float(), 2 ** 25: 2 * g[3].float(), rows - 1: 2 * (g[0].float() + g[4])}
    nonzero = 0
    for r in range(0, rows, 2 ** 20):
        nonzero += int(torch.count_nonzero(grad[r:r + 2 ** 20].view(torch.int16)))
    total = 0
    for r, v in want.items():
        assert torch.equal(grad[r], v.to(torch.bfloat16)), r
        total += int(torch.count_nonzero(grad[r].view(torch.int16)))
    assert nonzero == total  # NaN left anywhere would count
    del grad
    release()
