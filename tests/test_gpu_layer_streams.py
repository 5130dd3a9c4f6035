"""The stream that a layer operator is given: its calls run on it, and one of another
device is refused (before, the call ran on the tensors' device's current stream)."""
import contextlib
import types

import pytest
import torch

from tests.gpu_helpers import needs_gpu

pytestmark = needs_gpu
L = pytest.importorskip("gram_hashed_embedding_amd.layer")


def calls():
    def z(*shape, dtype=torch.bfloat16):
        return torch.ones(shape, dtype=dtype, device="cuda")

    # (made before, on the current stream: the calls make nothing but their outputs)
    x, t, wn = z(4, 32), torch.arange(4, device="cuda"), z(32)
    f = L.engram_residual_norm(x, w_next=wn)
    codes, scales = L.engram_act_encode(x)
    g, w, table = z(2, 3, 16), z(16, 4), z(4, 16)
    one, ring = z(4, 16), z(4, 3, 16)  # (the ring's new rows are as its old ones)
    return dict(
        norm=lambda s: L.engram_residual_norm(x, w_next=wn, stream=s).next,
        norm_backward=lambda s: L.engram_residual_norm_backward(
            None, x, out=x, rstd_next=f.rstd_next, w_next=wn, stream=s).residual,
        encode=lambda s: L.engram_act_encode(x, stream=s)[0],
        decode=lambda s: L.engram_act_decode(codes, scales, stream=s),
        conv_backward=lambda s: L.engram_ple_conv_backward(g, w, 1, x=g, stream=s).x,
        conv_step=lambda s: L.engram_ple_conv_step(one, ring, w, 1, t, stream=s),
        embed=lambda s: L.engram_embed(t, table, stream=s),
        embed_grad=lambda s: L.engram_embed_grad(t, x, 4, stream=s))


NAMES = ["norm", "norm_backward", "encode", "decode", "conv_backward", "conv_step", "embed",
         "embed_grad"]


@pytest.mark.parametrize("name", NAMES)
def test_a_stream_of_another_device_is_refused(name, monkeypatch):
    """A stand-in for a stream of a second device, which this machine may not have."""
    call = calls()[name]
    torch.cuda.synchronize()
    other = torch.device("cuda", torch.cuda.current_device() + 1)
    stream = types.SimpleNamespace(device=other, device_index=other.index, cuda_stream=0)
    monkeypatch.setattr(torch.cuda, "stream", lambda s: contextlib.nullcontext())
    with pytest.raises(ValueError, match="stream"):
        call(stream)


@pytest.mark.parametrize("name", NAMES)
def test_a_stream_of_the_tensors_device(name):
    call = calls()[name]
    want = call(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = call(side)
    side.synchronize()
    assert torch.equal(got, want)
