"""vc_kv8_attn's results do not depend on max_seq_len, the bound that a call is
given for its requests' lengths."""
import pytest
import torch

import numpy as np

from tests.test_gpu_kv8 import cache, check, q_of, run

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
    for bound in (n + 13, 4 * n, 100000):
        again, st = run(q, c8, 0.1, bound)
        assert st == 0 and torch.equal(out, again)
