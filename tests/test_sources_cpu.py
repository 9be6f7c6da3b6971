"""Rules that the kernels' sources keep."""

import glob
import os
import re

from tests.conftest import ROOT

CSRC = os.path.join(ROOT, "quantization_aware_sparse_amd", "csrc")


def asm_statements():
    for path in sorted(glob.glob(os.path.join(CSRC, "*"))):
        with open(path, encoding="utf-8") as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for m in re.finditer(r"\basm\b\s*(?:volatile\s*)?\(((?:[^()\"]|\"[^\"]*\"|\([^()]*\))*)\)", text):
            yield os.path.basename(path), m.group(1)


def test_the_scan_finds_the_statements():
    assert len(list(asm_statements())) >= 3


def test_no_vector_instruction_in_inline_asm():
    # the compiler puts wait states between a vector instruction and a matrix
    # instruction that reads its result, but does not look into inline asm
    for name, body in asm_statements():
        template = "".join(re.findall(r"\"([^\"]*)\"", body.split(":")[0]))
        assert not re.search(r"\bv_", template), (name, body)


def test_inline_asm_writes_no_register():
    # a load's output would count as written at once; what an empty statement
    # keeps in a register is read and written by nothing in it
    for name, body in asm_statements():
        if re.findall(r"\"([^\"]*)\"", body)[0]:
            outputs = body.split(":")[1] if body.count(":") else ""
            assert not outputs.strip(), (name, body)
