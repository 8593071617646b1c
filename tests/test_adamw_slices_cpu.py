"""Which arrays of an AdamW list count as overlapping: those that share bytes, not
those whose address ranges do. Against a set of every array's bytes. No GPU."""
import ctypes
import random

import numpy as np
import pytest

from rank_gradient_sketching_sketch_amd import binding as B

OK, BAD, UNSUP = 0, 1, 2
FAR = 1 << 30


def _pack(arrays):
    """arrays: (address, rows, cols, ld, type) of parameters; their gradients lie elsewhere."""
    lib = B.load_library()
    n = len(arrays)
    items = (B._AdamWTensor * n)(*[B._AdamWTensor(p, FAR + (i << 20), None, r, c, ld, c, 0, t, 0, 0, 0)
                                   for i, (p, r, c, ld, t) in enumerate(arrays)])
    host = np.zeros(int(lib.logra_adamw_table_bytes(n)) // 8, np.uint64)
    return lib.logra_adamw_list_pack(n, items, host.ctypes.data_as(ctypes.c_void_p), host.nbytes, ctypes.byref(B._AdamWListDesc()))


def _bytes(p, rows, cols, ld, t):
    el = 2 if t else 4
    return {p + el * (r * ld + c) + b for r in range(rows) for c in range(cols) for b in range(el)}


def _share(arrays):
    seen = set()
    for a in arrays:
        own = _bytes(*a)
        if own & seen:
            return True
        seen |= own
    return False


AT = 0x100000


def test_slices_of_one_buffer():
    # 8 rows of 48 floats: three column slices, one of bf16, one of a single row in a gap
    cols = [(AT, 8, 16, 48, 0), (AT + 64, 8, 20, 48, 0), (AT + 144, 8, 8, 96, 1), (AT + 192 + 160, 1, 8, 8, 0)]
    assert not _share(cols) and _pack(cols) == OK and _pack(cols[::-1]) == OK
    # of an upper and a lower half, beside a slice of all rows
    parts = [(AT, 4, 16, 48, 0), (AT + 4 * 192, 4, 16, 48, 0), (AT + 64, 8, 32, 48, 0)]
    assert _pack(parts) == OK
    for more in ((AT + 60, 8, 4, 48, 0), (AT + 188, 2, 2, 48, 0), (AT + 7 * 192 + 60, 1, 1, 1, 0), (AT, 400, 1, 1, 0), (AT + 176, 1, 5, 5, 0)):
        assert _share(cols + [more]) and _pack(cols + [more]) == BAD, more
    # other strides are not told apart
    assert _pack([(AT, 4, 1, 16, 0), (AT + 4, 4, 1, 17, 0)]) == BAD


def test_as_many_as_are_looked_at():
    slices = [(AT + 4 * i, 3, 1, 300, 0) for i in range(256)]
    assert _pack(slices) == OK
    assert _pack(slices + [(AT + 4 * 256, 3, 1, 300, 0)]) == UNSUP
    assert _pack(slices + [(AT + 4 * 900, 3, 1, 300, 0)]) == OK         # behind them


@pytest.mark.parametrize("seed", range(4))
def test_against_sets_of_bytes(seed):
    """Arrays of one row stride, or of one row, thrown into a small buffer."""
    rng = random.Random(seed)
    said = {OK: 0, BAD: 0}
    for _ in range(4000):
        stride = rng.choice((8, 12, 16, 24))             # in bf16 elements
        arrays = []
        for _ in range(rng.randint(2, 5)):
            t = rng.randint(0, 1)
            ld = stride if t else stride // 2
            rows, cols = rng.randint(1, 5), rng.randint(1, max(1, ld // 2))
            if rng.random() < 0.2:
                rows, cols = 1, rng.randint(1, 2 * ld)
            arrays.append((AT + (2 if t else 4) * rng.randrange(0, 40), rows, cols, max(ld, cols), t))
        want = BAD if _share(arrays) else OK
        assert _pack(arrays) == want, arrays
        said[want] += 1
    assert min(said.values()) > 200
