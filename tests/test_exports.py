"""What the built library exports."""
import shutil
import subprocess

import pytest

import routing_dispatch_expert_amd as moe


def test_plain_names_are_the_documented_ones():
    """Every unmangled function that the library exports is an entry point of moe.h: a helper of a common name would
    collide with the program's own."""
    nm = shutil.which("nm")
    if nm is None:
        pytest.skip("no nm here")
    text = subprocess.run([nm, "-D", "--defined-only", moe.LIB_PATH], capture_output=True, text=True, check=True).stdout
    names = [line.split()[-1] for line in text.splitlines() if " T " in line]
    plain = {n for n in names if not n.startswith("_")}
    assert plain == set(moe.EXPORTS)
