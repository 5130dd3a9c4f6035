"""CPU checks of the vocabulary operators' C ABI: the library exports what include/
engram_vocab.h declares, the binding's struct has the header's layout, bad arguments are refused
on the host before any launch (in the HIP build and in a CPU build of the same host code under
ASan and UBSan), rows are cut into segments that cover them, and the binding refuses what is not
a device tensor."""
import ctypes
import os
import re
import subprocess
import sys

import pytest

vocab = pytest.importorskip("gram_hashed_embedding_amd.vocab")

from gram_hashed_embedding_amd import abi  # noqa: E402
from tests import vocab_abi_cases  # noqa: E402
from tests.test_abi_sanitized import CSRC, INCLUDE, ROOT, _runtime  # noqa: E402

HEADER = os.path.join(INCLUDE, "engram_vocab.h")


def test_every_declared_symbol_is_exported():
    names = set(re.findall(r"^(?:int|size_t) (engram_\w+)\(", open(HEADER).read(), re.MULTILINE))
    assert names == {"engram_distill_workspace", "engram_distill", "engram_distill_backward",
                     "engram_beam_select_workspace", "engram_beam_select", "engram_beam_fork"}
    for name in names:
        assert getattr(vocab._lib, name).argtypes, name


@pytest.mark.parametrize("case", vocab_abi_cases.CASES, ids=lambda f: f.__name__[5:])
def test_abi_case(case):
    case(vocab._lib)


def test_struct_layout_and_constants_match_the_header(tmp_path):
    fields = [f for f, _ in abi.EngramDistillArgs._fields_]
    names = ["ENGRAM_DISTILL_MAX_TOP", "ENGRAM_BEAM_MAX", "ENGRAM_FORK_MAX_POOLS"]
    src = tmp_path / "layout.c"
    src.write_text("#include <stddef.h>\n#include <stdio.h>\n#include \"engram_vocab.h\"\n"
                   "int main(void) {\n  printf(\"%zu\\n\", sizeof(engram_distill_args));\n"
                   + "".join(f'  printf("%zu\\n", offsetof(engram_distill_args, {f}));\n'
                             for f in fields)
                   + "".join(f'  printf("%d\\n", {n});\n' for n in names)
                   + "  return 0;\n}\n")
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-std=c99", "-I", INCLUDE, str(src), "-o", str(exe)], check=True)
    got = [int(x) for x in subprocess.run([str(exe)], check=True, capture_output=True,
                                          text=True).stdout.split()]
    assert got[0] == ctypes.sizeof(abi.EngramDistillArgs)
    assert got[1:1 + len(fields)] == [getattr(abi.EngramDistillArgs, f).offset for f in fields]
    assert got[1 + len(fields):] == [abi.DISTILL_MAX_TOP, abi.BEAM_MAX, abi.FORK_MAX_POOLS]


CHILD = r"""
import ctypes, sys
sys.path.insert(0, {root!r})
from gram_hashed_embedding_amd import abi
from tests import vocab_abi_cases as V
lib = abi.declare_vocab(ctypes.CDLL({lib!r}))
for case in V.CASES:
    case(lib)
# calls that pass: the stand-in launchers check that rows are covered
for rows in (1, 3, 127, 129, 5000):
    for n in (1, 7, 8, 9, 2047, 2048, 2049, 65535, 65536, 163840, 163841, 1 << 18, (1 << 18) + 1,
              1 << 30):
        for grad in (0, 1):
            for kind in (abi.BF16, abi.F32):
                need = lib.engram_distill_workspace(rows, n, grad)
                more = dict(d_grad=V.B, d_grad_loss=V.A) if grad else \
                    dict(d_grad=None, d_grad_loss=None)
                assert V.distill(lib.engram_distill, rows=rows, vocab=n, logits_stride=n,
                                 grad_stride=n, logits_type=kind, d_workspace=V.C,
                                 workspace_bytes=need, **more) == V.OK, (rows, n)
        need = lib.engram_beam_select_workspace(rows, 2, n)
        assert V.select(lib.engram_beam_select, batch=rows, beams=2, vocab=n, stride=n, eos=0,
                        size=need) == V.OK, (rows, n)
assert V.distill(lib.engram_distill_backward, d_loss=None) == V.OK
assert V.fork(lib.engram_beam_fork) == V.OK
assert V.fork(lib.engram_beam_fork, held=(), slots=None, slot_count=0) == V.OK
assert V.fork(lib.engram_beam_fork, history=None, history_len=0, new_len=1) == V.OK
print("sanitized-ok", len(V.CASES))
"""


def test_host_checks_under_asan_and_ubsan(tmp_path):
    asan = _runtime("libasan.so")
    if asan is None:
        pytest.skip("g++ has no AddressSanitizer runtime here")
    lib = tmp_path / "libengram_vocabcheck.so"
    sources = [os.path.join(CSRC, "engram_host.cpp"), os.path.join(CSRC, "engram_vocab_host.cpp"),
               os.path.join(ROOT, "tests", "host_launch_stub.cpp"),
               os.path.join(ROOT, "tests", "vocab_launch_stub.cpp")]
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
    z = torch.zeros((2, 16), dtype=torch.bfloat16)
    ids = torch.zeros((2, 3), dtype=torch.int64)
    y, one = torch.zeros((2, 3)), torch.zeros((2,))
    for call in (lambda: vocab.engram_distill(z, ids, y),
                 lambda: vocab.engram_distill_backward(one, z, ids, y, one),
                 lambda: vocab.engram_beam_select(z, y[:1, :2]),
                 lambda: vocab.engram_beam_fork(ids, [z], tokens=ids)):
        with pytest.raises(TypeError):
            call()
