"""Inline PTX that all lanes of a warp (or all threads of a barrier) have to execute together is
``asm volatile``: a plain ``asm`` may be moved into a branch that uses its result, where only some
of the lanes would reach it (CPU only: reads the sources)."""
import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
TOGETHER = re.compile(r"\.sync\b|\bbar\.|\bbarrier\.|griddepcontrol")


def _asm_statements():
    for path in sorted(glob.glob(os.path.join(ROOT, "pose_retrieved_kv_b200", "csrc", "*.cu*"))):
        src = re.sub(r"//[^\n]*", "", open(path).read())
        for m in re.finditer(r"\basm\b(\s+volatile\b)?\s*\(", src):
            depth, i = 1, m.end()
            while depth:
                depth += {"(": 1, ")": -1}.get(src[i], 0)
                i += 1
            text = "".join(re.findall(r'"((?:[^"\\]|\\.)*)"', src[m.end():i]))
            yield os.path.basename(path), text, bool(m.group(1))


def test_collective_instructions_are_volatile():
    found = [(name, text, volatile) for name, text, volatile in _asm_statements()
             if TOGETHER.search(text)]
    assert len(found) > 10
    assert [x[:2] for x in found if not x[2]] == []
