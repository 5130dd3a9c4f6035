"""What the layer operators' binding refuses of device tensors: types, shapes,
strides and sizes that the kernels do not take raise before anything runs."""
import pytest
import torch

from tests.gpu_helpers import needs_gpu

pytestmark = needs_gpu
L = pytest.importorskip("gram_hashed_embedding_amd.layer")


def z(*shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype, device="cuda")


I64 = torch.int64
REFUSED = [
    lambda: L.engram_residual_norm(z(4, 32, dtype=torch.float16), w_next=z(32)),
    lambda: L.engram_residual_norm(z(4, 36), w_next=z(36)),
    lambda: L.engram_residual_norm(z(4, 32), w_next=z(32), groups=8),
    lambda: L.engram_residual_norm(z(4, 64)[:, :32], w_next=z(32)),
    lambda: L.engram_residual_norm(z(4, 32), z(4, 24), w_next=z(32)),
    lambda: L.engram_residual_norm(z(4, 32), z(4, 32).float()),
    lambda: L.engram_residual_norm(z(4, 32), z(8, 16)),
    lambda: L.engram_residual_norm_backward(z(4, 32), z(8, 16), out=z(4, 32), w_next=z(32),
                                            rstd_next=z(4, 1, dtype=torch.float32)),
    lambda: L.engram_residual_norm(z(4, 32), z(4, 32), gate=z(4, 5)),
    lambda: L.engram_residual_norm(z(4, 32), z(4, 32), gate=z(3, 32)),
    lambda: L.engram_residual_norm(z(4, 32), z(4, 32), eps=0.0),
    lambda: L.engram_residual_norm(z(4, 32), z(4, 32), next_codes=True),
    lambda: L.engram_residual_norm(z(4, 32), w_next=z(32), save_codes=True),
    lambda: L.engram_residual_norm(z(4, 32), gate=z(4, 32), w_next=z(32)),
    lambda: L.engram_residual_norm(z(1, 32768), w_next=z(32768)),
    lambda: L.engram_residual_norm(z(133)[5:].view(4, 32), w_next=z(32)),   # not 16-byte aligned
    lambda: L.engram_residual_norm_backward(z(4, 32), z(4, 32)),
    lambda: L.engram_residual_norm_backward(z(4, 32), y=z(4, 32)),
    lambda: L.engram_act_encode(z(4, 12)),
    lambda: L.engram_act_encode(z(4, 16).float()),
    lambda: L.engram_act_encode(z(16, 4).t()),
    lambda: L.engram_act_decode(z(4, 256, dtype=torch.int8), z(4, 1, dtype=torch.float32)),
    lambda: L.engram_ple_conv_backward(z(2, 9, 16), z(16, 4), 1),
    lambda: L.engram_ple_conv_backward(z(2, 9, 16), z(16, 17), 1, x=z(2, 9, 16)),
    lambda: L.engram_ple_conv_backward(z(2, 9, 16), z(16, 4), 0, x=z(2, 9, 16)),
    lambda: L.engram_ple_conv_backward(z(2, 9, 16), z(8, 4), 1, x=z(2, 9, 16)),
    lambda: L.engram_ple_conv_backward(z(2, 9, 16), z(16, 4), 1, x=z(2, 9, 16),
                                       seq_ids=z(2, 8, dtype=I64)),
    lambda: L.engram_ple_conv_backward(z(2, 9, 16), z(16, 4), 1, x=z(2, 9, 16), halo=z(1, 3, 16)),
    lambda: L.engram_ple_conv_step(z(2, 1, 16), z(2, 8, 16), z(16, 4), 3, z(2, dtype=I64)),
    lambda: L.engram_ple_conv_step(z(3, 1, 16), z(2, 9, 16), z(16, 4), 3, z(3, dtype=I64)),
    lambda: L.engram_ple_conv_step(z(2, 1, 16), z(2, 9, 16), z(16, 4), 3, z(2, dtype=torch.int32)),
    lambda: L.engram_embed(z(4, dtype=torch.int32), z(5, 16)),
    lambda: L.engram_embed(z(4, dtype=I64), z(5, 12)),
    lambda: L.engram_embed(z(4, dtype=I64), z(5, 16), out_dtype=torch.float16),
    lambda: L.engram_embed_grad(z(4, dtype=I64), z(3, 16), 5),
    lambda: L.engram_embed_grad(z(4, dtype=I64), z(4, 16), 5, accumulate=True),
    lambda: L.engram_embed_grad(z(4, dtype=I64), z(4, 16), 5,
                                workspace=z(16, dtype=torch.uint8)),
]


@pytest.mark.parametrize("call", range(len(REFUSED)))
def test_refused(call):
    with pytest.raises((TypeError, ValueError, L.EngramError)):
        REFUSED[call]()
