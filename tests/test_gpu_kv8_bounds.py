"""Results over an 8-bit cache do not depend on max_seq_len, the bound that a
call is given for its requests' lengths."""
import numpy as np
import pytest
import torch

from tests import vc_harness as H
from tests.test_gpu_kv8 import cache, check, q_of, run, vc

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [100, 960])
@pytest.mark.parametrize("hq,n_q,d", [(4, 1, 64), (2, 7, 128), (8, 4, 64), (4, 16, 128), (8, 13, 64), (8, 32, 128), (5, 64, 64),
                                      (8, 64, 128)])
def test_the_same_bits_whatever_the_bound(hq, n_q, d, n):
    rng = np.random.default_rng(n + n_q)
    c8, h = cache(rng, [n] * 3, 1, d, "e4m3")
    qn, q = q_of(rng, (3, n_q, hq, d))
    out, st = run(q, c8, 0.1, n)
    assert st == 0
    check(out, h, qn, 0.1)
    for bound in (n + 13, 4 * n, 100000, (1 << 31) - 1):
        again, st = run(q, c8, 0.1, bound)
        assert st == 0 and torch.equal(out, again)


def test_pages_are_written_alike_whatever_the_bound():
    m, rng = vc(), np.random.default_rng(1)
    full, _ = H.full_cache(rng, [100, 33, 0], 2, 64)
    got = []
    for bound in (100, 5000, (1 << 31) - 1):
        c8 = m.PagedKV8.allocate(full.num_pages, 2, 64, torch.int8, full.block_table, full.seq_lens)
        m.kv8_write(full, None, c8, bound)
        got.append([x.cpu() for x in (c8.k_codes, c8.v_codes, c8.k_scales, c8.v_scales)])
    assert all(torch.equal(a, b) for g in got[1:] for a, b in zip(got[0], g)) and got[0][2].any()
