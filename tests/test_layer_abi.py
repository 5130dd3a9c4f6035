"""CPU checks of the layer operators' C ABI: the library exports what
include/engram_layer.h declares, the binding's struct has the header's layout,
bad arguments are refused on the host before any launch (in the HIP build and
in a CPU build of the same host code under ASan and UBSan), and the binding
refuses what is not a device tensor."""
import ctypes
import os
import re
import subprocess
import sys

import pytest

layer = pytest.importorskip("gram_hashed_embedding_amd.layer")

from gram_hashed_embedding_amd import abi  # noqa: E402
from tests import layer_abi_cases  # noqa: E402
from tests.test_abi_sanitized import CSRC, INCLUDE, ROOT, _runtime  # noqa: E402

HEADER = os.path.join(INCLUDE, "engram_layer.h")


def test_every_declared_symbol_is_exported():
    names = set(re.findall(r"^(?:int|size_t) (engram_\w+)\(", open(HEADER).read(), re.MULTILINE))
    assert names == {"engram_residual_norm", "engram_residual_norm_backward_workspace",
                     "engram_residual_norm_backward", "engram_act_encode", "engram_act_decode",
                     "engram_ple_conv_backward_workspace", "engram_ple_conv_backward",
                     "engram_ple_conv_step", "engram_embed", "engram_embed_grad_workspace",
                     "engram_embed_grad"}
    for name in names:
        assert getattr(layer._lib, name).argtypes, name


@pytest.mark.parametrize("case", layer_abi_cases.CASES, ids=lambda f: f.__name__[5:])
def test_abi_case(case):
    case(layer._lib)


def test_struct_layout_and_constants_match_the_header(tmp_path):
    fields = [f for f, _ in abi.EngramNormArgs._fields_]
    names = ["ENGRAM_BF16", "ENGRAM_F32", "ENGRAM_ACT_BLOCK", "ENGRAM_NORM_MAX_GROUP"]
    src = tmp_path / "layout.c"
    src.write_text("#include <stddef.h>\n#include <stdio.h>\n#include \"engram_layer.h\"\n"
                   "int main(void) {\n  printf(\"%zu\\n\", sizeof(engram_norm_args));\n"
                   + "".join(f'  printf("%zu\\n", offsetof(engram_norm_args, {f}));\n'
                             for f in fields)
                   + "".join(f'  printf("%d\\n", {n});\n' for n in names)
                   + "  return 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-I", INCLUDE, str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True,
                                          text=True).stdout.split()]
    assert got[0] == ctypes.sizeof(abi.EngramNormArgs)
    assert got[1:1 + len(fields)] == [getattr(abi.EngramNormArgs, f).offset for f in fields]
    assert got[1 + len(fields):] == [abi.BF16, abi.F32, abi.ACT_BLOCK, abi.NORM_MAX_GROUP]


CHILD = r"""
import ctypes, sys
sys.path.insert(0, {root!r})
from gram_hashed_embedding_amd import abi
from tests import layer_abi_cases
lib = abi.declare_layer(ctypes.CDLL({lib!r}))
for case in layer_abi_cases.CASES:
    case(lib)
print("sanitized-ok", len(layer_abi_cases.CASES))
"""


def test_host_checks_under_asan_and_ubsan(tmp_path):
    asan = _runtime("libasan.so")
    if asan is None:
        pytest.skip("g++ has no AddressSanitizer runtime here")
    lib = tmp_path / "libengram_layercheck.so"
    sources = [os.path.join(CSRC, "engram_host.cpp"), os.path.join(CSRC, "engram_layer_host.cpp"),
               os.path.join(ROOT, "tests", "host_launch_stub.cpp"),
               os.path.join(ROOT, "tests", "layer_launch_stub.cpp")]
    subprocess.run(["g++", "-std=c++17", "-O1", "-g", "-fno-omit-frame-pointer", "-shared", "-fPIC",
                    "-Wall", "-Wextra", "-fsanitize=address,undefined",
                    "-fno-sanitize-recover=all", f"-I{INCLUDE}", f"-I{CSRC}", *sources, "-o",
                    str(lib)], check=True)
    env = dict(os.environ, LD_PRELOAD=asan, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    res = subprocess.run([sys.executable, "-c", CHILD.format(root=ROOT, lib=str(lib))],
                         capture_output=True, text=True, timeout=300, env=env)
    assert res.returncode == 0 and "sanitized-ok" in res.stdout, \
        (res.stdout[-2000:], res.stderr[-4000:])


def test_the_binding_refuses_host_tensors():
    import torch
    x = torch.zeros((2, 16), dtype=torch.bfloat16)
    t = torch.zeros((2,), dtype=torch.int64)
    for call in (lambda: layer.engram_residual_norm(x, w_next=x[0]),
                 lambda: layer.engram_residual_norm_backward(x),
                 lambda: layer.engram_act_encode(x),
                 lambda: layer.engram_act_decode(x, x),
                 lambda: layer.engram_ple_conv_backward(x[None], x, 1, x=x[None]),
                 lambda: layer.engram_ple_conv_step(x, x[None], x, 1, t),
                 lambda: layer.engram_embed(t, x),
                 lambda: layer.engram_embed_grad(t, x, 4)):
        with pytest.raises(TypeError):
            call()
