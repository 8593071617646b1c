"""8-bit products whose x has no rows (a rank without tokens): nothing of x is
looked at, least of all divided by. No GPU."""
import os
import subprocess
import sys

import rank_gradient_sketching_sketch_amd as L

UNSUP = 2

# a call that the library refuses after it has looked at x (too many tiles), in a process of its own
CALL = """
import ctypes, sys
sys.path.insert(0, %r)
from rank_gradient_sketching_sketch_amd import binding as B
p = ctypes.c_void_p(0x10000)
print(B.load_library().logra_fp8_matmul(1 << 26, 1 << 22, 32, 4, p, p, 1, None, %d, 0, None, p, 32, p, 1, p, 1 << 22, None))
"""


def _run(ldx):
    root = os.path.dirname(os.path.dirname(L.__file__))
    return subprocess.run([sys.executable, "-c", CALL % (root, ldx)], capture_output=True, text=True, timeout=120)


def test_row_stride_is_not_looked_at():
    L.load_library()
    for ldx in (0, 7, 1 << 30):
        p = _run(ldx)
        assert p.returncode == 0 and p.stdout.split() == [str(UNSUP)], (ldx, p.returncode, p.stderr[-300:])
