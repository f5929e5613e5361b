"""Properties of the sources and of their code that no run shows: every load in assembly carries the wait states that it
needs after a vector instruction wrote a scalar operand of it, whatever the compiler puts before the statement, and gets
its buffer in scalar registers (the compiler would put the numbers of vector registers there without a word)."""
import glob
import os
import re
import subprocess

import pytest

from quantized_two_stage_amd import build

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_two_stage_amd", "csrc")


def test_loads_in_assembly_wait_for_their_scalar_operands():
    seen = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"\basm\b[^;]*?\);", text, re.S):
            code = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', m.group(0).split(":")[0]))
            lines = [x.strip() for x in code.replace("\\t", " ").split("\\n")]
            for at, line in enumerate(lines):
                if re.match(r"(buffer|global|flat)_load", line):
                    seen += 1
                    nops = [int(x.split()[1]) + 1 for x in lines[:at] if re.match(r"s_nop \d+$", x)]
                    assert sum(nops) >= 5, (os.path.basename(path), line)
    assert seen >= 3


@pytest.mark.parametrize("source", ["qr_gemm.hip", "qr_gemm_f8.hip"])
def test_loads_to_lds_take_scalar_buffers(source, tmp_path):
    """in the code that the build's compiler and flags make"""
    out = tmp_path / "device.s"
    flags = [f for f in build.FLAGS if f not in ("-shared", "-fPIC")]
    subprocess.run(["hipcc", *flags, "--cuda-device-only", "-S", os.path.join(CSRC, source), "-o", str(out)], check=True,
                   capture_output=True)
    seen = 0
    for line in out.read_text().splitlines():
        if re.match(r"\s*buffer_load\S*\s.*\blds\s*$", line):
            seen += 1
            assert re.match(r"\s*buffer_load_dword(x4)? v\d+, s\[\d+:\d+\], (s\d+|0) offen( nt)? lds\s*$", line), line
    assert seen > 100
