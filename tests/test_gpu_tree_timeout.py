"""The bounded waits of vc_tree_attn, made to run out (host-side fault
injection, no GPU fault), for every kernel: one to four tiles of 128 rows,
both head sizes.  A row whose keys did not all come in time is zeros; the
others are what they always are, and the next call is clean."""
import numpy as np
import pytest
import torch

from oracle import tree as T
from tests import vc_harness as H
from tests.test_gpu_tree import check_attn, q_bf16, random_parents, to_mask

pytestmark = pytest.mark.gpu

TIMEOUT, SMS, TILE = 6, 152, 128
# n_q, query heads (two kv heads): 112, 128, 140, 256, 280, 320, 448 and 512 rows, so one to four tiles
KERNELS = [(16, 14), (32, 8), (20, 14), (32, 16), (40, 14), (40, 16), (64, 14), (64, 16)]


def vc():
    import lossless_compressed_kv_gb300 as m
    return m


@pytest.fixture
def fault():
    yield vc().debug_set_wait_fault
    vc().debug_set_wait_fault(0, 0)


class Call:
    """A call whose output and workspace stay from one time to the next."""

    def __init__(self, n_q, hq, d, lens, dtype):
        rng = np.random.default_rng([n_q, hq, d, len(lens)])
        self.n_q, self.hq, self.hkv, self.d, self.lens = n_q, hq, 2, d, lens
        self.full, self.hf = H.full_cache(rng, lens, 2, d)
        self.qn, self.q = q_bf16(rng, (len(lens), n_q, hq, d))
        self.masks = [T.tree_plan(random_parents(rng, n_q), n)[0] for n in lens]
        self.mask = to_mask(self.masks)
        self.out = torch.full(self.q.shape, 3.0, dtype=dtype, device="cuda")
        n = vc().tree_workspace_bytes(self.full, n_q, hq, max(lens))
        self.ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")

    def run(self):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        vc().tree_attn(self.q, self.full, self.mask, self.d ** -0.5, self.out, max(self.lens), self.ws, status=st)
        torch.cuda.synchronize()
        return int(st.item()), self.out.clone()

    def rows(self, out):
        """[request][kv head][row of the unit][channel]: rows are nodes x query heads of the group."""
        b, grp = len(self.lens), self.hq // self.hkv
        return out.view(b, self.n_q, self.hkv, grp, self.d).permute(0, 2, 1, 3, 4).reshape(b, self.hkv, -1, self.d)

    def lost_in_odd_blocks(self):
        """Per row of a unit: whether a block of odd index has some of its keys.
        The units' blocks of keys, laid end to end, are dealt out in equal ranges
        to the groups; a group is a block, or for four tiles two of two each."""
        rows = self.n_q * (self.hq // self.hkv)
        tiles = -(-rows // TILE)
        lanes, keys = 2 if tiles == 4 else 1, 128 if tiles in (2, 4) else 64
        most = (2 * SMS if tiles == 1 else SMS) // lanes
        units = len(self.lens) * self.hkv
        groups = min(most, units * -(-max(self.lens) // 64))
        n = [-(-x // keys) for x in self.lens for _ in range(self.hkv)]
        total = sum(n)
        start = [g * (total // groups) + min(g, total % groups) for g in range(groups + 1)]
        lost = torch.zeros((units, rows), dtype=torch.bool)
        u0 = 0
        for u, m in enumerate(n):
            for g in range(groups):
                if start[g] < u0 + m and start[g + 1] > u0:
                    for lane in range(lanes):
                        if (g * lanes + lane) % 2:
                            lost[u, lane * 2 * TILE:(lane + 1) * 2 * TILE if lanes == 2 else rows] = True
            u0 += m
        return lost.view(len(self.lens), self.hkv, rows).cuda()


@pytest.mark.parametrize("n_q,hq", KERNELS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("requests,longest", [(1, 9000), (3, 9000), (120, 400)])
def test_every_other_block_without_copies(fault, n_q, hq, d, requests, longest):
    """Rows joined of ranges of which some came and some did not, rows of one
    range, and both in one batch."""
    rng = np.random.default_rng(requests)
    lens = [int(x) for x in rng.integers(max(n_q, longest // 3), longest, requests)]
    c = Call(n_q, hq, d, lens, torch.float32)
    st, clean = c.run()
    assert st == 0 and not bool((clean == 0).all(-1).any())
    lost = c.lost_in_odd_blocks()
    assert bool(lost.any()) and (requests < 100 or not bool(lost.all()))
    fault(2_000_000, 2)
    st, out = c.run()
    got, want = c.rows(out), c.rows(clean)
    assert st == TIMEOUT
    assert torch.equal((got == 0).all(-1), lost)
    assert torch.equal(got[~lost], want[~lost])
    fault(0, 0)
    st, out = c.run()
    assert st == 0 and torch.equal(out, clean)
    check_attn(out, c.hf, c.qn, c.masks[0], float(np.float32(d ** -0.5)), 0)


@pytest.mark.parametrize("n_q,hq", KERNELS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_no_copy_at_all(fault, n_q, hq, d, dtype):
    """20 and 40 nodes of 14 heads are two and three tiles; one tile (Q in TMEM,
    two blocks to an SM) takes 16 of them or fewer."""
    c = Call(n_q, hq, d, [n_q, 3000, 900], dtype)
    st, clean = c.run()
    assert st == 0
    for b in range(3):
        check_attn(clean, c.hf, c.qn, c.masks[b], float(np.float32(d ** -0.5)), b)
    fault(20_000, 1)
    st, out = c.run()
    assert st == TIMEOUT and bool((out == 0).all())
    fault(0, 0)
    st, out = c.run()
    assert st == 0 and torch.equal(out, clean)


@pytest.mark.parametrize("n_q,hq", KERNELS)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("requests", [1, 40])
def test_a_limit_that_runs_out_while_copies_are_under_way(fault, n_q, hq, d, requests):
    """Each row is whole or zeros, and blocks end after their copies and products."""
    rng = np.random.default_rng(requests)
    c = Call(n_q, hq, d, [int(x) for x in rng.integers(n_q, 4000, requests)], torch.float32)
    _, clean = c.run()
    fault(1, 0)
    for _ in range(3):
        st, out = c.run()
        got, want = c.rows(out), c.rows(clean)
        zero, same = (got == 0).all(-1), (got == want).all(-1)
        assert bool((zero ^ same).all()) and (st == TIMEOUT or not bool(zero.any()))
    fault(0, 0)
    st, out = c.run()
    assert st == 0 and torch.equal(out, clean)
