"""What the sources of the attention layer's kernels must not hold."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp4_quantized_prep_amd", "csrc")
LAYER = ["attention_common.h", "attention_decode.hip", "attention_prefill.hip", "attention_rows.h", "fp8_gemm.hip",
         "kv_cache_fp8.hip", "layer_common.h", "qk_norm_rope.hip"]


@pytest.mark.parametrize("name", LAYER)
def test_no_instruction_in_inline_asm(name):
    """The compiler does not count the wait states that an instruction must keep
    from an MFMA whose result it reads where that instruction is inline asm;
    statements without one (barriers to its scheduling) are all that these
    kernels may hold."""
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    asm = re.findall(r"\basm\b\s*(?:volatile)?\s*\(\s*(\"[^\"]*\")", text)
    assert len(asm) == len(re.findall(r"\basm\b\s*(?:volatile\s*)?\(", text))
    assert [a for a in asm if a != '""'] == []
