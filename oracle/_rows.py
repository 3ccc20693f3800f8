"""Row-wise steps of the oracle on all host cores (TEST INFRASTRUCTURE).

numpy runs elementwise arithmetic on one core; large cases spend most of their
time there. A step whose rows do not depend on one another is run piece by
piece on threads (numpy releases the interpreter lock in its loops): the same
operations on the same numbers, so the same bits as in one piece.
"""
from __future__ import annotations

import os
from concurrent.futures import ThreadPoolExecutor

_CORES = os.cpu_count() or 1
_pool = None


def by_rows(step, rows: int, columns: int) -> None:
    """step(lo, hi) over [0, rows) in contiguous pieces; at once for small arrays."""
    global _pool
    pieces = min(_CORES, rows, rows * columns // 65536)
    if pieces <= 1:
        step(0, rows)
        return
    if _pool is None:
        _pool = ThreadPoolExecutor(_CORES)
    cut = [rows * i // pieces for i in range(pieces + 1)]
    for done in [_pool.submit(step, a, b) for a, b in zip(cut[:-1], cut[1:])]:
        done.result()
