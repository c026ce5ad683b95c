"""The plain definitions of the 8-bit cache and of the page operations against
worked examples and a library's own conversion."""
import numpy as np
import pytest
import torch

from oracle import kv8 as K
from oracle import pages as P


def test_e4m3_codes_are_the_types():
    every = torch.arange(256, dtype=torch.uint8)
    there = every.view(torch.float8_e4m3fn).float().double().numpy()
    mine = K.decode(every.numpy(), "e4m3")
    assert np.array_equal(np.isnan(there), np.isnan(mine)) and np.array_equal(there[~np.isnan(there)], mine[~np.isnan(mine)])
    x = np.concatenate([np.random.default_rng(1).uniform(-448, 448, 20000), np.ldexp(1.0, np.arange(-14, 9)),
                        (K.e4m3_values()[:-1] + K.e4m3_values()[1:]) / 2]).astype(np.float32)
    assert np.array_equal(K.encode(x, "e4m3"), torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy())


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_block(code):
    rng = np.random.default_rng(2)
    x = rng.standard_normal((16, 64)).astype(np.float32)
    c, s, odd = K.block(x, code)
    y = K.decode(c, code) * s
    assert not odd and abs(np.abs(y).max() / np.abs(x).max() - 1) < 1e-6
    step = np.abs(x) * 2.0 ** -4 + s * 2.0 ** -10 if code == "e4m3" else s * 0.5001
    assert (np.abs(y - x) <= step * 1.0001).all()
    c, s, _ = K.block(np.zeros((16, 64)), code)
    assert not c.any() and s == np.float32(2.0 ** -126)
    x[3, 4], x[5, 6], x[7, 8] = np.nan, np.inf, -np.inf
    c, s, odd = K.block(x, code)
    v = K.decode(c, code)
    assert odd and v[3, 4] == 0 and v[5, 6] == K.TOP[code] and v[7, 8] == -K.TOP[code]


def test_attention_definition():
    rng = np.random.default_rng(3)
    q, k, v = rng.standard_normal((3, 8)), rng.standard_normal((5, 8)), rng.standard_normal((5, 8))
    seen = np.ones((3, 5), bool)
    seen[1, 2:] = False
    seen[2] = False
    out, _ = K.attn(q, k, v, seen, 0.5, 1.0)
    w = np.exp(0.5 * (k[:2] @ q[1]))
    assert np.allclose(out[1], (w[:, None] * v[:2]).sum(0) / w.sum()) and not out[2].any()


def test_pages_worked_example():
    """Two forks of a prompt of 20 tokens: both write to its second page."""
    m = P.Map(np.full((3, 4), -1), [2, 0, 0], [1, 0, 1, 0, 0, 0])
    m.table[0, :2] = [2, 0]
    lens = [20, 0, 0]
    m.fork(lens, [0, 0], [1, 2])
    assert lens == [20, 20, 20] and m.refs.tolist() == [3, 0, 3, 0, 0, 0]
    g, s, d = m.reserve(lens, [0, 21, 40])
    assert g == [1, 1, 1] and s == [-1, 0, 0] and d == [-1, 1, 3]
    assert m.table[1].tolist() == [2, 1, -1, -1] and m.table[2].tolist() == [2, 3, 4, -1]
    assert m.refs.tolist() == [1, 1, 3, 1, 1, 0]
    m.free([0, -1, -1])
    assert m.refs.tolist() == [0, 1, 2, 1, 1, 0] and m.table[0].tolist() == [-1] * 4
    moves, remap = m.compact()
    assert moves == [(4, 0)] and remap == [-1, 1, 2, 3, 0, -1] and m.table[2].tolist() == [2, 3, 0, -1] and not m.bad


def test_pages_the_last_of_all_writers_keeps_its_page():
    m = P.Map([[0, -1], [0, -1], [0, -1]], [1, 1, 1], [3, 0, 0])
    assert m.reserve([5, 5, 5], [6, 6, 6]) == ([1, 1, 1], [0, 0, -1], [1, 2, -1])
    assert m.refs.tolist() == [1, 1, 1]
    m = P.Map([[0, -1], [0, -1], [0, -1]], [1, 1, 1], [3, 0, 0])
    assert m.reserve([5, 5, 5], [6, 0, 33])[0] == [1, 1, 0]    # no room for two more: the last row stays as it was
    assert m.table.tolist() == [[1, -1], [0, -1], [0, -1]] and m.refs.tolist() == [2, 1, 0]
