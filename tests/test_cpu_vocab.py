"""The vocabulary operators' kernels on the CPU: what their sources may not hold, and the beams'
choice built as ordinary C++ (as in test_cpu_wave)."""
import glob
import os
import re
import subprocess

import pytest

from tests.test_abi_sanitized import CSRC, ROOT
from tests.test_cpu_wave import build


def test_no_instruction_is_written_by_hand():
    """The compiler puts wait states between a vector instruction and a move of its result across
    lanes, but for an instruction in inline assembly it does not have to know that one is due."""
    for path in glob.glob(os.path.join(CSRC, "*")):
        if path.endswith((".hip", ".h", ".cpp")):
            code = re.sub(r"//[^\n]*", "", open(path).read())
            assert not re.search(r"\b(?:__)?asm(?:__)?\b", code), path


@pytest.fixture(scope="module")
def run(tmp_path_factory):
    """A check of the beams' choice by its name: how many cases of it were right."""
    exe = build(tmp_path_factory.mktemp("beams"), "beam_choice",
                os.path.join(CSRC, "engram_host.cpp"), os.path.join(CSRC, "engram_vocab_host.cpp"),
                os.path.join(ROOT, "tests", "host_launch_stub.cpp"))

    def check(which):
        res = subprocess.run([exe, which], capture_output=True, text=True, timeout=300)
        assert res.returncode == 0, (res.returncode, res.stdout, res.stderr)
        return res.stdout.count(": ok")
    return check


def test_finished_beams_are_not_read(run):
    """Their rows' pages are taken away."""
    assert run("finished") == 24


def test_beams_of_a_masks_lowest_value(run):
    """Their ids share the beam's probability, whose logarithm a logit of 1e30 does not hold."""
    assert run("masked") == 8


def test_equal_beams_by_place(run):
    """A sum's order does not go by its row's address."""
    assert run("equal") == 24
