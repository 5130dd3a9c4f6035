"""The vocabulary operators' kernels on the CPU: what their sources may not hold, and the beams'
choice built as ordinary C++ (as in test_cpu_wave)."""
import glob
import os
import re
import subprocess

from tests.test_abi_sanitized import CSRC, ROOT
from tests.test_cpu_wave import build


def test_no_instruction_is_written_by_hand():
    """The compiler puts wait states between a vector instruction and a move of its result across
    lanes, but for an instruction in inline assembly it does not have to know that one is due."""
    for path in glob.glob(os.path.join(CSRC, "*")):
        if path.endswith((".hip", ".h", ".cpp")):
            code = re.sub(r"//[^\n]*", "", open(path).read())
            assert not re.search(r"\b(?:__)?asm(?:__)?\b", code), path


def run(tmp_path, which):
    res = subprocess.run([build(tmp_path, "beam_choice", os.path.join(CSRC, "engram_host.cpp"),
                                os.path.join(CSRC, "engram_vocab_host.cpp"),
                                os.path.join(ROOT, "tests", "host_launch_stub.cpp")), which],
                         capture_output=True, text=True, timeout=300)
    assert res.returncode == 0, (res.returncode, res.stdout, res.stderr)
    return res.stdout.count(": ok")


def test_finished_beams_are_not_read(tmp_path):
    """Their rows' pages are taken away."""
    assert run(tmp_path, "finished") == 24


def test_beams_of_a_masks_lowest_value(tmp_path):
    """Their ids share the beam's probability, whose logarithm a logit of 1e30 does not hold."""
    assert run(tmp_path, "masked") == 8
