"""The vocabulary operators' kernels on the CPU: what their sources may not hold."""
import glob
import os
import re

from tests.test_abi_sanitized import CSRC


def test_no_instruction_is_written_by_hand():
    """The compiler puts wait states between a vector instruction and a move of its result across
    lanes, but for an instruction in inline assembly it does not have to know that one is due."""
    for path in glob.glob(os.path.join(CSRC, "*")):
        if path.endswith((".hip", ".h", ".cpp")):
            code = re.sub(r"//[^\n]*", "", open(path).read())
            assert not re.search(r"\b(?:__)?asm(?:__)?\b", code), path
