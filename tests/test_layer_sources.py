"""Properties of the kernels' sources that no run shows: what the assembly statements tell the compiler."""
import glob
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_two_stage_amd", "csrc")


def asm_statements():
    for path in sorted(glob.glob(os.path.join(CSRC, "*"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"\basm\b[^;]*?\);", text, re.S):
            yield os.path.basename(path), m.group(0)


def test_no_assembly_writes_m0_behind_the_compiler():
    """m0 is set by the compiler, as an input: it cannot be told of a change by the statement itself"""
    seen = 0
    for name, statement in asm_statements():
        lines = [x.strip() for text in re.findall(r'"((?:[^"\\]|\\.)*)"', statement.split(":")[0])
                 for x in text.replace("\\t", " ").split("\\n")]
        for line in lines:
            assert not re.match(r"\S+\s+m0\b", line), (name, line)
            if re.match(r"buffer_load\S*\s.*\blds$", line):
                seen += 1
                assert '"{m0}"' in statement, (name, statement)
    assert seen > 0
