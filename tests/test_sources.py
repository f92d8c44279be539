"""Rules that the kernels' sources keep, checked on their text."""
import os
import re

import pytest

import routing_dispatch_expert_amd as moe

CSRC = os.path.join(moe.HERE, "csrc")
SOURCES = sorted(f for f in os.listdir(CSRC) if f.endswith((".h", ".hip")))


@pytest.mark.parametrize("name", SOURCES)
def test_inline_assembly_holds_no_instruction_on_registers(name):
    """The compiler keeps no wait states between an instruction written in inline assembly and the matrix
    instructions around it. Assembly without text (a mark for the compiler) and waits take no registers."""
    text = open(os.path.join(CSRC, name)).read()
    found = re.findall(r'\basm\s*(?:volatile\s*)?\(\s*"([^"]*)"', text)
    assert len(found) == len(re.findall(r"\b(?:asm|__asm__)\b", re.sub(r"//.*|/\*[\s\S]*?\*/", "", text)))
    for code in found:
        assert code == "" or re.fullmatch(r"s_waitcnt [a-z]+cnt\(0\)", code), f"{name}: {code}"
