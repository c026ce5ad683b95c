"""The 64-bit definitions of the tree-drafting operations, pinned by closed
forms and by the chain operations they generalise."""
import math

import numpy as np
import pytest

import oracle
from oracle import tree as T


def test_rotary_pairs_turn_and_keep_their_length():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((3, 2, 8))
    f = T.rotary_frequencies(100.0, 8)
    assert np.allclose(f, [1.0, 100 ** -0.25, 0.1, 100 ** -0.75])
    for inter in (False, True):
        y = T.rotary(x, [0, 1, 7], f, inter)
        assert np.allclose(y[0], x[0])
        assert np.allclose(np.linalg.norm(y, axis=-1), np.linalg.norm(x, axis=-1))
        # scores depend on the distance of positions alone
        a, b = T.rotary(x[:1], [11], f, inter), T.rotary(x[1:2], [4], f, inter)
        c, d = T.rotary(x[:1], [7], f, inter), T.rotary(x[1:2], [0], f, inter)
        assert np.allclose((a * b).sum(-1), (c * d).sum(-1))
    # the two layouts are the same rotation on permuted channels
    perm = [0, 4, 1, 5, 2, 6, 3, 7]
    assert np.allclose(T.rotary(x, [1, 2, 3], f, False)[..., perm], T.rotary(x[..., perm], [1, 2, 3], f, True))


def test_rotary_scaling_blends_between_the_two_ends():
    f = T.rotary_frequencies(10000.0, 64)
    s = T.rotary_frequencies(10000.0, 64, 8.0, 4096, 1.0, 32.0)
    turns = 4096 * f / (2 * math.pi)
    assert np.allclose(s[turns >= 32], f[turns >= 32]) and np.allclose(s[turns <= 1], f[turns <= 1] / 8)
    mid = (turns > 1) & (turns < 32)
    assert mid.any() and (s[mid] < f[mid]).all() and (s[mid] > f[mid] / 8).all()
    assert np.allclose(T.rotary_frequencies(10000.0, 64, 4.0), f / 4)


def test_plan_of_a_chain_and_of_a_tree():
    masks, pos, bad = T.tree_plan([-1, 0, 1, 2], 10)
    assert (masks, pos, bad) == ([1, 3, 7, 15], [6, 7, 8, 9], False)
    masks, pos, bad = T.tree_plan([-1, 0, 0, 2, -2], 5)
    assert (masks, pos, bad) == ([1, 3, 5, 13, 0], [0, 1, 1, 2, -1], False)
    masks, pos, bad = T.tree_plan([-1, 1, 5, -2, 3, 0], 6)
    assert (masks, pos, bad) == ([1, 0, 0, 0, 0, 33], [0, -1, -1, -1, -1, 1], True)
    assert T.tree_plan([-1, 0], 1) == ([0, 0], [-1, -1], True)


def test_walk_of_a_chain_is_the_chain_rule():
    rng = np.random.default_rng(1)
    for _ in range(50):
        x = int(rng.integers(1, 8))
        drafts, ver = rng.integers(0, 2, x), rng.integers(0, 2, x + 1)
        a = next((i for i in range(x) if drafts[i] != ver[i]), x)
        got = T.tree_accept([-1] + list(range(x)), np.concatenate([[9], drafts]), ver)
        assert got == (a, list(range(a + 1)), [int(t) for t in drafts[:a]] + [int(ver[a])])
    assert T.tree_accept([-1, 0, 0, 2], [5, 6, 7, 8], [7, 1, 8, 3]) == (2, [0, 2, 3], [7, 8, 3])
    assert T.tree_accept([-1, 0, 0], [5, 6, 6], [6, 1, 2]) == (1, [0, 1], [6, 1])   # twins: the first
    assert T.tree_accept([-2, -2], [0, 0], [0, 0]) == (-1, [], [])


def test_tree_attention_of_a_chain_is_causal_block_attention():
    rng = np.random.default_rng(2)
    n_q, L, hkv, g, d = 5, 23, 2, 2, 64
    import synth
    qb = synth.normal_bf16(rng, (n_q, hkv * g, d))
    kb, vb = synth.normal_bf16(rng, (L, hkv, d)), synth.normal_bf16(rng, (L, hkv, d))
    ref = oracle.verify_attn_block(qb, kb, vb, 0.125)
    masks, _, _ = T.tree_plan([-1, 0, 1, 2, 3], L)
    q, k, v = (synth.bf16_to_f32(t).astype(np.float64) for t in (qb, kb, vb))
    out, spread, _ = T.tree_attn(q, k, v, masks, 0.125)
    assert np.abs(out - ref).max() < 1e-6 and (spread >= np.abs(out) - 1e-12).all()
    out, _, _ = T.tree_attn(q, k, v, [0] * n_q, 0.125)
    assert (out == 0).all()


@pytest.mark.parametrize("tau", [1.0, 0.5])
def test_logprobs_closed_forms(tau):
    lp, ent, top, tlp = T.token_logprobs([2.0] * 8, [3, -1, 9], tau, 3)
    assert lp[0] == pytest.approx(-math.log(8)) and lp[1:] == [0.0, 0.0] and ent == pytest.approx(math.log(8))
    assert top == [0, 1, 2] and tlp == pytest.approx([-math.log(8)] * 3)
    lp, ent, top, tlp = T.token_logprobs([0.0, math.log(3) * tau, -np.inf], [0, 1, 2], tau, 4)
    assert lp[0] == pytest.approx(math.log(0.25)) and lp[1] == pytest.approx(math.log(0.75)) and lp[2] == -np.inf
    assert ent == pytest.approx(-0.25 * math.log(0.25) - 0.75 * math.log(0.75))
    assert top == [1, 0, -1, -1] and tlp[2:] == [-np.inf, -np.inf]
    lp, ent, top, tlp = T.token_logprobs([-np.inf] * 3, [1], tau, 1)
    assert lp == [-np.inf] and ent == 0.0 and top == [-1]
    lp, ent, top, tlp = T.token_logprobs([0.0, np.nan], [0], tau, 1)
    assert math.isnan(lp[0]) and math.isnan(ent) and top == [-1] and math.isnan(tlp[0])
