"""vc_kv8_attn where a row's factor beside K's scale leaves fp32's range."""
import numpy as np
import pytest
import torch

from tests import vc_harness as H
from tests.test_gpu_kv8 import CODES, cache, check, q_of, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,n_q,d", [(4, 1, 64), (2, 5, 128), (8, 4, 64), (8, 16, 128), (4, 20, 64), (8, 32, 128), (5, 64, 64),
                                      (8, 64, 128)])
@pytest.mark.parametrize("scale,up", [(0.125, 100), (1e30, 60), (1e-30, -100), (0.125, -100)])
def test_scores_of_zero_stay_zero(hq, n_q, d, scale, up):
    """Pages of zeros in K whose scale, beside q, is beyond fp32: scores of 0, so V's mean."""
    rng = np.random.default_rng(n_q)
    k_scale = 2.0 ** 122 if up > 0 else 2.0 ** -126
    c8, h = cache(rng, [333, 70], 1, d, "int8", k_scale=lambda s: np.full_like(s, k_scale), junk=0)
    h["k"][:] = 0
    c8.k_codes.copy_(H.to_dev(h["k"]).view(CODES["int8"]))
    qn, q = q_of(rng, (2, n_q, hq, d))
    out, st = run((q.float() * 2.0 ** up).to(torch.bfloat16), c8, scale, 333)
    assert st == 0 and torch.isfinite(out).all()
    check(out, h, qn * 2.0 ** up, scale)
