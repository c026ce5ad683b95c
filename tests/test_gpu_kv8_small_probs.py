"""vc_kv8_attn where a few keys outweigh all others: the small probabilities
keep their own precision in the second product (fp16, half a step 2^-11)."""
import numpy as np
import pytest
import torch

import synth
from tests import vc_harness as H
from tests.test_gpu_kv8 import CODES, cache, check, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("hq,n_q,d", [(4, 1, 64), (2, 5, 128), (8, 4, 64), (8, 16, 128), (4, 20, 64), (8, 32, 128), (5, 64, 64),
                                      (8, 64, 128)])
def test_a_strong_key_in_every_page(hq, n_q, d, code):
    """One key of each page has the largest score and a V of zeros; the others lie 2^14 to 2^20 below it, row
    by row, and make up the result."""
    rng = np.random.default_rng(n_q)
    c8, h = cache(rng, [3000], 1, d, code, k_scale=lambda s: np.full_like(s, 2.0 ** -5), v_scale=lambda s: np.full_like(s, 2.0 ** -3))
    one = {"int8": 32, "e4m3": 0x60}[code]                        # code 32: the value 1
    h["k"][:], h["k"][:, :, 5, 0], h["v"][:, :, 5] = 0, one, 0
    c8.k_codes.copy_(H.to_dev(h["k"]).view(CODES[code]))
    c8.v_codes.copy_(H.to_dev(h["v"]).view(CODES[code]))
    qb = synth.bf16_bits(np.zeros((1, n_q, hq, d), np.float32))
    below = 14 + 6 * np.arange(n_q * hq).reshape(1, n_q, hq) / (n_q * hq)
    qb[..., 0] = synth.bf16_bits((below * np.log(2.0) * 8).astype(np.float32))
    qn = synth.bf16_to_f32(qb).astype(np.float64)
    out, st = run(H.to_dev(qb.view(np.int16)).view(torch.bfloat16), c8, 0.125, 3000)
    assert st == 0
    check(out, h, qn, 0.125)
