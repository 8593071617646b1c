"""Inline assembly in the kernels' sources names the registers that it writes by
name, so that the compiler keeps nothing in them across it. No GPU."""
import glob
import os
import re

import rank_gradient_sketching_sketch_amd as L

CSRC = os.path.join(os.path.dirname(L.__file__), "csrc")
# an instruction's destination that is not an operand (%0 ...): m0, vcc, exec or a register's number
WRITES = re.compile(r'(?:"|\\n|\\t)\s*[sv]_\w+ (m0|vcc|exec|[sva]\d+|[sva]\[\d+:\d+\])\s*,')


def _statements(text):
    for m in re.finditer(r"\basm\b\s*(?:volatile)?\s*\(", text):
        depth, at = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(text[at], 0)
            at += 1
        yield text[m.end():at - 1]


def test_registers_written_by_name_are_clobbered():
    seen = 0
    for path in sorted(glob.glob(os.path.join(CSRC, "*.h*"))):
        for body in _statements(open(path).read()):
            for reg in WRITES.findall(body):
                seen += 1
                assert '"%s"' % reg in body.rsplit(":", 1)[1], (path, reg, body)
    assert seen >= 2                    # the loads into LDS
