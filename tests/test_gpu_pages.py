"""GPU page operations (vc_pages_free, _fork, _reserve, _compact, _copy)
against their sequential definitions: whole numbers and copies, all equal."""
import numpy as np
import pytest
import torch

from oracle import pages as P
from tests import vc_harness as H

pytestmark = pytest.mark.gpu


def vc():
    import lossless_compressed_kv_gb300 as m
    return m


def i32(x):
    return H.to_dev(np.array(x, dtype=np.int32))


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


class Both:
    """The same map on the GPU and in the oracle."""

    def __init__(self, table, blocks, refs):
        self.o = P.Map(table, blocks, refs)
        self.m = vc().PageMap(i32(table), i32(blocks), i32(refs))
        self.ws = torch.full((vc().pages_workspace_bytes(self.m),), 0x5A, dtype=torch.uint8, device="cuda")
        self.st = status()

    def same(self):
        torch.cuda.synchronize()
        for a, b in ((self.m.table, self.o.table), (self.m.blocks, self.o.blocks), (self.m.refs, self.o.refs)):
            assert np.array_equal(a.cpu().numpy(), b)
        assert int(self.st.item()) == (3 if self.o.bad else 0)

    def reserve(self, lens, want):
        n = len(lens)
        g, s, d = (torch.full((n,), 77, dtype=torch.int32, device="cuda") for _ in range(3))
        vc().pages_reserve(self.m, i32(lens), i32(want), g, s, d, self.ws, status=self.st)
        ref = self.o.reserve(lens, want)
        self.same()
        assert [x.tolist() for x in (g, s, d)] == [list(r) for r in ref]
        return s, d

    def fork(self, lens, src, dst):
        t = i32(lens)
        vc().pages_fork(self.m, t, i32(src), i32(dst), status=self.st)
        self.o.fork(lens, src, dst)
        self.same()
        assert t.tolist() == list(lens)

    def free(self, keep):
        vc().pages_free(self.m, i32(keep), status=self.st)
        self.o.free(keep)
        self.same()

    def compact(self, room=0):
        n = len(self.o.refs)
        s, d = (torch.full((n // 2 + room,), 9, dtype=torch.int32, device="cuda") for _ in range(2))
        k, remap = torch.full((1,), 9, dtype=torch.int32, device="cuda"), torch.full((n,), 9, dtype=torch.int32, device="cuda")
        vc().pages_compact(self.m, s, d, k, remap, self.ws, status=self.st)
        moves, ref = self.o.compact()
        self.same()
        pad = [-1] * (n // 2 + room - len(moves))
        assert k.item() == len(moves) and remap.tolist() == ref
        assert s.tolist() == [a for a, _ in moves] + pad and d.tolist() == [b for _, b in moves] + pad
        return s, d, k


def empty(pages, rows, width):
    return Both(np.full((rows, width), -1), np.zeros(rows), np.zeros(pages))


@pytest.mark.parametrize("seed,pages,rows,width", [(1, 40, 6, 8), (2, 300, 40, 20), (3, 9000, 70, 60), (4, 70000, 33, 400),
                                                   (5, 33, 1100, 5), (6, 1, 1, 1)])
def test_a_life_of_a_pool(seed, pages, rows, width):
    """Rows come, fork, go on, give back and go, in random order, the pool at times full."""
    rng = np.random.default_rng(seed)
    b = empty(pages, rows, width)
    lens = [0] * rows
    for step in range(14):
        what = step % 5
        if what in (0, 2):
            grow = rng.integers(0, 2 if rows > 100 else 4, rows)
            most = min(width * 16, max(1, 32 * pages // rows))
            want = [int(min(width * 16, n + rng.integers(1, most + 1))) if g else int(rng.integers(0, n + 1))
                    for n, g in zip(lens, grow)]
            before = b.o.blocks.copy()
            b.reserve(lens, want)
            lens = [w if w > n and 16 * b.o.blocks[i] >= w and (b.o.blocks[i] > before[i] or 16 * before[i] >= w) else n
                    for i, (n, w) in enumerate(zip(lens, want))]
        elif what == 1:
            idle = [i for i in range(rows) if b.o.blocks[i] == 0]
            busy = [i for i in range(rows) if b.o.blocks[i] > 0]
            k = min(len(idle), 20) if busy else 0
            src, dst = [int(rng.choice(busy)) for _ in range(k)], [int(x) for x in rng.permutation(idle)[:k]]
            b.fork(lens, src + [-1], dst + [-1])
        elif what == 3:
            keep = [int(rng.integers(-1, n + 1)) if rng.random() < 0.6 else -1 for n in lens]
            b.free(keep)
            lens = [k if k >= 0 else n for k, n in zip(keep, lens)]
        else:
            b.compact(room=int(rng.integers(0, 3)))


def test_writers_that_share_pages():
    """All, some and one of a page's rows write to it; whole pages behind a cut row; a fork of a fork."""
    b = empty(64, 6, 6)
    lens = [0] * 6
    b.reserve(lens, [70, 0, 0, 0, 0, 0])
    lens[0] = 70
    b.fork(lens, [0, 0, 0], [1, 2, 3])
    b.reserve(lens, [71, 72, 80, 81, 0, 0])       # all four write to page 4: the last keeps it
    b.fork(lens, [2, 2], [4, 5])
    b.reserve(lens, [70, 70, 75, 70, 90, 0])      # two of three
    cut = [0, 0, 0, 0, 0, 17]                     # row 5 shortened: writes where three whole pages are shared
    b.reserve(cut, [0, 0, 0, 0, 0, 96])
    b.free([0, 0, 0, 0, 0, 0])
    assert not b.o.refs.any()


def test_what_is_refused_is_left_as_it_was():
    b = Both([[0, 1, -1], [2, 99, -1], [3, -1, -1], [-1, -1, -1], [-1, -1, -1]], [2, 2, 1, 0, 0], [1, 1, 1, 1, 0, 0, 0, 0])
    lens = [20, 20, 5, 0, 0]
    b.fork(lens, [0, 0, 1, 7, 0, -1, 2], [3, 3, 4, 4, 9, 2, 0])   # twice, bad page, no such rows, half a pair, held
    b.st.zero_()
    b.o.bad = False
    b.fork(lens, [0, 3], [3, 4])                                  # a target that is a source
    b.st.zero_()
    b.o.bad = False
    b.reserve([20, 20, 40, -1, 0], [21, 21, 41, 5, 49])           # bad page, too few pages, negative, too long
    b.st.zero_()
    b.o.bad = False
    b.reserve([20, 0, 5, 0, 0], [21, 0, 16, 0, 0])
    assert not b.o.bad
    b.free([0, 0, -1, -1, -1])                                    # a bad page among those given back
    assert b.o.bad


def test_pages_that_nobody_holds():
    b = Both([[0, 1], [1, -1]], [2, 1], [1, 1, 0])
    b.free([0, 0])                                # page 1 is held once and given back twice
    assert b.o.bad
    b = Both([[0, 1]], [2], [1, 0, 0])
    b.reserve([20], [25])
    assert b.o.bad
    b.st.zero_()
    b.o.bad = False
    b.compact()
    assert b.o.bad


def test_no_rows_and_nothing_to_do():
    m = vc()
    e = torch.empty(0, dtype=torch.int32, device="cuda")
    none = m.PageMap(e.view(0, 4), e, i32([0] * 5))
    m.pages_free(none, e)
    m.pages_fork(none, e, e, e)
    m.pages_reserve(none, e, e, e, e, e, torch.empty(0, dtype=torch.uint8, device="cuda"))
    b = Both([[4, 2]], [2], [0, 0, 1, 0, 1])
    b.compact()
    b.compact()                                   # nothing moves
    Both([[-1]], [0], [0] * 5).compact()
    m.pages_copy(m.PageArrays([]), e, e)
    m.pages_copy(m.PageArrays([torch.zeros((4, 8), device="cuda")]), e, e)


@pytest.mark.parametrize("n", [1, 3, 500])
def test_copy(n):
    """Pools of several formats, scales, an array off the 16-byte grid; with a count, pairs of -1 and bad pages."""
    m, rng = vc(), np.random.default_rng(n)
    pages = 2 * n + 7
    g = torch.Generator(device="cuda").manual_seed(n)
    arrays = [torch.randint(0, 256, (pages, w), generator=g, device="cuda", dtype=torch.uint8)
              for w in (16 * 128 * 2, 4 * 16 * 64, 32, 16)]
    arrays += [torch.randn((pages, 3), device="cuda"), torch.randn((pages + 1, 4), device="cuda")[:, :].reshape(-1)[1:1 + 4 * pages].view(pages, 4)]
    perm = rng.permutation(pages)
    src, dst = perm[:n].astype(np.int32), perm[n:2 * n].astype(np.int32)
    if n > 3:
        src[5], dst[5] = -1, -1
        src[8], dst[9] = pages, -2
    for count in (None, 0, n // 2, n + 5):
        ref = [a.clone() for a in arrays]
        st = status()
        m.pages_copy(m.PageArrays(arrays), i32(src), i32(dst), count=None if count is None else i32([count]), status=st)
        torch.cuda.synchronize()
        k = n if count is None else min(count, n)
        ok = [(s, d) for s, d in zip(src[:k], dst[:k]) if 0 <= s < pages and 0 <= d < pages]
        for a, r in zip(arrays, ref):
            for s, d in ok:
                r[d] = r[s]
            assert torch.equal(a, r)
        assert st.item() == (3 if n > 3 and k > 8 else 0)


def test_many_arrays():
    m = vc()
    arrays = [torch.arange(6, device="cuda", dtype=torch.int32).repeat_interleave(4 + (i % 2)).view(6, -1).contiguous() + 10 * i
              for i in range(150)]
    m.pages_copy(m.PageArrays(arrays), i32([0, 5]), i32([3, 1]))
    torch.cuda.synchronize()
    for i, a in enumerate(arrays):
        assert a[:, 0].tolist() == [10 * i + x for x in (0, 5, 2, 0, 4, 5)]


def test_arrays_that_moved_are_read_anew():
    m = vc()
    t = torch.zeros((4, 8), device="cuda")
    a = m.PageArrays([t])
    t.set_(torch.arange(32, device="cuda", dtype=torch.float32).view(4, 8))
    m.pages_copy(a, i32([3]), i32([0]))
    torch.cuda.synchronize()
    assert t[0].tolist() == t[3].tolist() == list(range(24, 32))


def test_captured_and_replayed_on_another_stream():
    """A graph of fork, reserve and copy is replayed from other lengths."""
    m = vc()
    b = empty(50, 4, 8)
    b.reserve([0] * 4, [37, 0, 0, 0])
    lens, want = i32([37, 0, 0, 0]), i32([0, 40, 70, 0])
    pool = torch.randn((50, 8), device="cuda")
    arrays = m.PageArrays([pool])
    src, dst = i32([0, 0]), i32([1, 2])
    g, s, d = (torch.zeros(4, dtype=torch.int32, device="cuda") for _ in range(3))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        m.pages_fork(b.m, lens, src, dst, status=b.st)
        m.pages_reserve(b.m, lens, want, g, s, d, b.ws, status=b.st)
        m.pages_copy(arrays, s, d, status=b.st)
    for n in (37, 30):
        b.free([-1, 0, 0, -1])
        lens.copy_(i32([n, 0, 0, 0]))
        want.copy_(i32([0, n + 3, n + 33, 0]))
        torch.cuda.synchronize()
        ref = pool.clone()
        graph.replay()
        ol = [n, 0, 0, 0]
        b.o.fork(ol, [0, 0], [1, 2])
        og, os_, od = b.o.reserve(ol, [0, n + 3, n + 33, 0])
        b.same()
        assert [g.tolist(), s.tolist(), d.tolist(), lens.tolist()] == [og, os_, od, ol]
        for x, y in zip(os_, od):
            if x >= 0:
                ref[y] = ref[x]
        assert torch.equal(pool, ref)
