"""vc_kv8_write where requests share pages of both caches (forked rows): a
shared page is made from the longest of those that hold it, bit for bit."""
import numpy as np
import pytest
import torch

import synth
from oracle import kv8 as K
from tests import vc_harness as H
from tests.test_gpu_kv8 import CODES, i32, status, vc

pytestmark = pytest.mark.gpu


def shared_case(rng, lens, groups, hkv, d):
    """Rows of a group hold the same pages, in both caches: (full, pools, table of each cache)."""
    width = max(-(-n // 16) for n in lens)
    perm = rng.permutation(len(groups) * width).astype(np.int32)
    table = np.full((len(lens), width), -1, np.int32)
    for g, rows in enumerate(groups):
        table[rows] = perm[g * width:(g + 1) * width]
    k, v = synth.kv_pools(rng, len(perm), hkv, d, [3], 6.0)
    full = vc().PagedKV(*(H.to_dev(x.view(np.uint8).reshape(len(perm), -1)) for x in (k, v)), H.to_dev(table), i32(lens),
                        hkv, d, 16)
    table8 = rng.permutation(len(perm)).astype(np.int32)[table]
    return full, k, v, table, table8


LENS = {"equal": ([25, 25, 25], [[0, 1, 2]]),
        "unequal": ([25, 20, 17, 31, 16], [[0, 1, 2, 3, 4]]),
        "ends": ([31, 32, 48, 33, 33, 1], [[0, 1, 2], [3, 5], [4]]),
        "many": ([18 + (7 * i) % 14 for i in range(90)] + [5] * 10, [list(range(0, 90, 2)), list(range(1, 90, 2)), list(range(90, 100))])}


@pytest.mark.parametrize("d,code,hkv", [(64, "e4m3", 2), (128, "int8", 3)])
@pytest.mark.parametrize("first", ["all", "in the page", "some"])
@pytest.mark.parametrize("which", list(LENS))
def test_a_shared_page_is_that_of_the_longest(which, first, d, code, hkv):
    m, rng = vc(), np.random.default_rng(len(which) + d)
    lens, groups = LENS[which]
    full, k, v, table, table8 = shared_case(rng, lens, groups, hkv, d)
    start = {"all": [0] * len(lens), "in the page": [max(0, n - 1) for n in lens],
             "some": [n if i % 3 else 0 for i, n in enumerate(lens)]}[first]
    for _ in range(3):
        c8 = m.PagedKV8.allocate(table.max() + 1, hkv, d, CODES[code], H.to_dev(table8), i32([0] * len(lens)))
        for t in (c8.k_scales, c8.v_scales):
            t.fill_(-3.0)
        st = status()
        m.kv8_write(full, None if first == "all" else i32(start), c8, max(lens), status=st)
        torch.cuda.synchronize()
        assert st.item() == 0
        for codes, scales, pool in ((c8.k_codes, c8.k_scales, k), (c8.v_codes, c8.v_scales, v)):
            ref = np.zeros(codes.shape, np.uint8)
            rs = np.full(scales.shape, -3.0, np.float32)
            for rows in groups:
                for j in range(table.shape[1]):
                    tokens = min(16, max(lens[b] - 16 * j for b in rows))
                    if tokens > 0 and any(start[b] < lens[b] and start[b] // 16 <= j < -(-lens[b] // 16) for b in rows):
                        x = synth.bf16_to_f32(pool[table[rows[0], j]]).copy()
                        x[:, tokens:] = 0.0
                        for h in range(hkv):
                            at = table8[rows[0], j], h
                            ref[at], rs[at], _ = K.block(x[h], code)
            assert np.array_equal(scales.cpu().numpy(), rs)
            assert np.array_equal(K.decode(codes.view(torch.uint8).cpu().numpy(), code), K.decode(ref, code))


def test_a_row_beyond_the_call_is_no_holder():
    """Row 1 is longer than max_seq_len: it is left out, and the page is row 0's."""
    m, rng = vc(), np.random.default_rng(3)
    full, k, _, table, table8 = shared_case(rng, [20, 25], [[0, 1]], 1, 64)
    c8 = m.PagedKV8.allocate(2, 1, 64, CODES["int8"], H.to_dev(table8), i32([0, 0]))
    st = status()
    m.kv8_write(full, None, c8, 24, status=st)
    torch.cuda.synchronize()
    assert st.item() == 3
    x = synth.bf16_to_f32(k[table[0, 1]]).copy()
    x[:, 4:] = 0.0
    ref, s, _ = K.block(x[0], "int8")
    assert c8.k_scales[table8[0, 1], 0].item() == s
    assert np.array_equal(c8.k_codes[table8[0, 1], 0].view(torch.uint8).cpu().numpy(), ref)
