"""8-bit activation checkpoints on the GPU: codes and scales bit for bit as the
definition gives them, and the values read back."""
import numpy as np
import pytest
import torch

from gram_hashed_embedding_amd import workloads
from tests import layer_reference as ref
from tests.gpu_helpers import needs_gpu, release

pytestmark = needs_gpu
L = pytest.importorskip("gram_hashed_embedding_amd.layer")


def check(x):
    codes, scales = L.engram_act_encode(x)
    back = L.engram_act_decode(codes, scales)
    h = x.float().cpu().numpy().reshape(-1, x.shape[-1])
    want_c, want_s = ref.encode(h)
    assert np.array_equal(codes.cpu().numpy().reshape(want_c.shape), want_c)
    assert np.array_equal(scales.cpu().numpy().reshape(want_s.shape), want_s, equal_nan=True)
    want = ref.bf16(ref.decode(want_c, want_s))
    assert np.array_equal(ref.f64(back).reshape(want.shape), want, equal_nan=True)
    return back


@pytest.mark.parametrize("rows", [1, 2, 63, 1031])
@pytest.mark.parametrize("channels", [8, 56, 128, 136, 1000, 2056])
def test_shapes(rows, channels):
    x = workloads.make_bf16((rows, channels), rows + channels, "cuda")
    size = torch.exp(workloads.make_bf16((channels,), 3, "cuda", std=2.0).float())
    check((x.float() * size).to(torch.bfloat16))


def test_more_axes():
    check(workloads.make_bf16((3, 5, 7, 264), 1, "cuda"))


def test_special_blocks():
    """Zeros, the type's ends, values too small for a scale, infinities and NaN: each stays in
    its own block of its own row."""
    x = workloads.make_bf16((12, 384), 2, "cuda")
    x[0] = 0
    x[1, :128] = 0
    x[2, 5] = float("nan")
    x[3, 130] = float("inf")
    x[4, 383] = float("-inf")
    x[5] *= torch.finfo(torch.bfloat16).max / 16
    x[6, 0], x[6, 1] = torch.finfo(torch.bfloat16).max, torch.finfo(torch.bfloat16).min
    x[7] = (x[7].float() * 2.0 ** -126).to(torch.bfloat16)
    x[8] = 2.0 ** -120
    x[9] = -(2.0 ** -121)
    x[10, :128] = -0.0
    back = check(x)
    assert bool(torch.isnan(back[2, :128]).all()) and bool(torch.isfinite(back[2, 128:]).all())
    assert bool(torch.isnan(back[3, 128:256]).all()) and bool(torch.isfinite(back[3, :128]).all())
    assert bool(torch.isfinite(back[6]).all())
    assert bool((back[9] == 0).all()) and bool((back[0] == 0).all())


def test_empty():
    codes, scales = L.engram_act_encode(torch.empty((0, 16), dtype=torch.bfloat16, device="cuda"))
    assert codes.shape == (0, 16) and scales.shape == (0, 1)
    assert L.engram_act_decode(codes, scales).shape == (0, 16)


def test_offsets_past_32_bits():
    rows, channels = 2 ** 32 // 8192 + 5, 8192
    print(f"checkpoint of [{rows}, {channels}]", flush=True)
    tail = workloads.make_bf16((4, channels), 1, "cuda")
    x = torch.zeros((rows, channels), dtype=torch.bfloat16, device="cuda")
    x[-4:] = tail
    codes, scales = L.engram_act_encode(x)
    want_c, want_s = L.engram_act_encode(tail)
    assert torch.equal(codes[-4:], want_c) and torch.equal(scales[-4:], want_s)
    assert int(torch.count_nonzero(codes[-8:-4])) == 0
    back = L.engram_act_decode(codes, scales, out=x)
    assert torch.equal(back[-4:], L.engram_act_decode(want_c, want_s))
    del x, codes, scales, back
    release()
