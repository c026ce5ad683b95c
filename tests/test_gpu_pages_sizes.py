"""Compacting pools of sizes beside those where one block ranks their pages."""
import numpy as np
import pytest

from tests.test_gpu_pages import Both

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("pages", [1023, 1025, 4096, 4097, 8191, 8192, 8193, 12289])
@pytest.mark.parametrize("live", [0.0, 0.3, 0.66, 1.0])
def test_compact(pages, live):
    rng = np.random.default_rng(pages)
    refs = (rng.random(pages) < live).astype(np.int64) * rng.integers(1, 4, pages)
    held = rng.permutation(np.flatnonzero(refs))
    rows = np.array_split(held, 5)
    table = np.full((5, max(1, max(len(r) for r in rows))), -1)
    for t, r in zip(table, rows):
        t[:len(r)] = r
    b = Both(table, [len(r) for r in rows], refs)
    b.compact(room=3)
    b.compact()
