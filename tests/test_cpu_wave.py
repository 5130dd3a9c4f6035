"""Kernels of the layer operators built as ordinary C++ (tests/cpu_wave/hip stands
in for HIP's header) and run on the CPU in the worst order of their wavefronts."""
import os
import subprocess

import pytest

from tests import norm_shapes
from tests.test_abi_sanitized import CSRC, INCLUDE, ROOT

HERE = os.path.join(ROOT, "tests", "cpu_wave")
CLANG = "/opt/rocm/llvm/bin/clang++"


def build(tmp_path, name, *more):
    """The program cpu_wave/<name>.cpp, a kernel source included in it."""
    if not os.path.exists(CLANG):
        pytest.skip("the kernel sources need ROCm's clang++")
    exe = tmp_path / name
    subprocess.run([CLANG, "-x", "c++", "-std=c++17", "-O1", "-ffp-contract=off", f"-I{HERE}",
                    f"-I{CSRC}", f"-I{INCLUDE}", os.path.join(HERE, name + ".cpp"),
                    *more, "-o", str(exe)], check=True)
    return str(exe)


def test_norm_blocks_of_several_rows(tmp_path):
    """A block's wavefronts may be a whole sum apart: no row's mean is another row's, whichever
    of the two norms a call has."""
    res = subprocess.run([build(tmp_path, "norm_rows")], capture_output=True, text=True,
                         timeout=300)
    assert res.returncode == 0, res.stdout + res.stderr
    assert res.stdout.count(": same") == 36


def test_shapes_of_several_rows_a_block(tmp_path):
    """The sizes that the GPU tests run for blocks of several rows are such sizes."""
    exe = build(tmp_path, "norm_shapes", os.path.join(CSRC, "engram_host.cpp"),
                os.path.join(CSRC, "engram_layer_host.cpp"),
                os.path.join(ROOT, "tests", "host_launch_stub.cpp"),
                os.path.join(ROOT, "tests", "layer_launch_stub.cpp"))
    for way, shapes in (("forward", norm_shapes.FORWARD), ("backward", norm_shapes.BACKWARD)):
        for rows, channels in shapes:
            out = subprocess.run([exe, way, str(rows), str(channels), "1"], check=True,
                                 capture_output=True, text=True).stdout
            lanes, at_once, blocks = map(int, out.split())
            assert lanes > 64 and at_once * blocks < rows, (way, rows, channels, out)


def test_embedding_gradient_of_a_stalled_sort(tmp_path):
    """A sort whose wait expired leaves NaN in a gradient, not what the memory held, whether or
    not the caller counts errors."""
    exe = build(tmp_path, "embed_stall", os.path.join(CSRC, "engram_host.cpp"),
                os.path.join(ROOT, "tests", "host_launch_stub.cpp"))
    res = subprocess.run([exe], capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, res.stdout + res.stderr
    assert res.stdout.count(": ok") == 6
