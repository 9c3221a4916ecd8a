"""What the sources of the kernels whose weights depend on the token must not hold."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp4_quantized_prep_amd", "csrc")


@pytest.mark.parametrize("name", ["fp8_grouped.hip", "lora.hip", "moe_route.hip", "row_groups.h"])
def test_no_instruction_in_inline_asm(name):
    """The compiler counts neither wait states nor outstanding loads of instructions
    in inline asm: these kernels hold barriers to its scheduling alone."""
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    asm = re.findall(r"\basm\b\s*(?:volatile)?\s*\(\s*(\"[^\"]*\")", text)
    assert len(asm) == len(re.findall(r"\basm\b\s*(?:volatile\s*)?\(", text))
    assert [a for a in asm if a != '""'] == []
