"""KVLayers follows its caches: whatever tensors they carry at the time of a
tree_commit are the ones that the call gets.  The library is replaced by a
recorder, so these run without a GPU."""
import gc

import pytest
import torch


@pytest.fixture(scope="module")
def m():
    import __graft_entry__
    __graft_entry__._builder().build()
    import lossless_compressed_kv_gb300 as vc
    return vc


class Recorder:
    """vc_tree_commit's arguments: per layer what its struct says."""

    def __init__(self):
        self.layers = None

    def vc_tree_commit(self, structs, n, n_q, accept_len, path, status, stream):
        assert len(structs) == n
        self.layers = [{f: getattr(s, f) for f in ("k_pages", "v_pages", "block_table", "seq_lens", "batch", "num_pages",
                                                   "max_blocks")} for s in structs]
        return 0


@pytest.fixture
def lib(m, monkeypatch):
    r = Recorder()
    monkeypatch.setattr(m, "_lib", r)
    monkeypatch.setattr(m, "_device", lambda: -1)          # where CPU tensors are
    monkeypatch.setattr(m, "_on", lambda stream, dev: None)
    return r


HKV, D = 2, 64


def pool(n=6):
    return torch.zeros((n, HKV * 16 * D * 2), dtype=torch.uint8)


def caches(m, layers=3, batch=4):
    table, lens = torch.zeros((batch, 5), dtype=torch.int32), torch.full((batch,), 20, dtype=torch.int32)
    return [m.PagedKV(pool(), pool(), table, lens, HKV, D, 16) for _ in range(layers)]


def commit(m, lib, layers, batch=4):
    lib.layers = None
    m.tree_commit(layers, torch.zeros(batch, dtype=torch.int32), torch.zeros((batch, 3), dtype=torch.int32))
    return lib.layers


def live(cs):
    return [dict(k_pages=c.k_pages.data_ptr(), v_pages=c.v_pages.data_ptr(), block_table=c.block_table.data_ptr(),
                 seq_lens=c.seq_lens.data_ptr(), batch=c.block_table.shape[0], num_pages=c.k_pages.shape[0],
                 max_blocks=c.block_table.shape[1]) for c in cs]


def test_untouched_caches(m, lib):
    cs = caches(m)
    layers = m.KVLayers(cs)
    assert len(layers) == 3
    for _ in range(2):
        assert commit(m, lib, layers) == live(cs)


@pytest.mark.parametrize("name", ["seq_lens", "block_table", "k_pages", "v_pages"])
@pytest.mark.parametrize("which", [[0, 1, 2], [2]])
def test_a_rebound_tensor_is_the_one_that_is_passed(m, lib, name, which):
    cs = caches(m)
    layers = m.KVLayers(cs)
    new = getattr(cs[0], name).clone()
    for i in which:
        setattr(cs[i], name, pool(9) if name in ("k_pages", "v_pages") else new)
        if name in ("k_pages", "v_pages"):                 # both pools of a cache are of one size
            setattr(cs[i], "v_pages" if name == "k_pages" else "k_pages", pool(9))
    gc.collect()
    assert commit(m, lib, layers) == live(cs)
    assert commit(m, lib, layers) == live(cs)


def test_lengths_shortened_as_after_a_commit(m, lib):
    """The update that a round ends with, written out of place; every round's."""
    cs = caches(m)
    layers = m.KVLayers(cs)
    for _ in range(4):
        commit(m, lib, layers)
        lens = cs[0].seq_lens - 2
        for c in cs:
            c.seq_lens = lens
        gc.collect()
    assert commit(m, lib, layers) == live(cs)


def test_a_smaller_batch(m, lib):
    """accept_len and path are those of the batch that is launched."""
    cs = caches(m)
    layers = m.KVLayers(cs)
    table, lens = cs[0].block_table[:2], cs[0].seq_lens[:2]        # (the same addresses)
    for c in cs:
        c.block_table, c.seq_lens = table, lens
    with pytest.raises(ValueError, match="path"):
        commit(m, lib, layers, batch=4)
    assert lib.layers is None
    assert commit(m, lib, layers, batch=2) == live(cs)


@pytest.mark.parametrize("name", ["seq_lens", "block_table", "k_pages"])
def test_a_tensor_given_other_storage_in_place(m, lib, name):
    cs = caches(m)
    layers = m.KVLayers(cs)
    t = getattr(cs[0], name)
    old = t.data                                           # (the old storage lives on: the new one's address differs)
    t.data = t.data.clone()
    assert t.data_ptr() != old.data_ptr()
    assert commit(m, lib, layers) == live(cs)


def test_a_table_that_grows_in_place(m, lib):
    cs = caches(m)
    layers = m.KVLayers(cs)
    cs[0].block_table.resize_(4, 5000).zero_()
    assert commit(m, lib, layers) == live(cs)


def test_what_a_cache_may_not_carry_is_refused(m, lib):
    cs = caches(m)
    layers = m.KVLayers(cs)
    good = cs[1].seq_lens
    for bad in (good.long(), good[:3], torch.zeros(8, dtype=torch.int32)[::2]):
        cs[1].seq_lens = bad
        for _ in range(2):
            with pytest.raises(ValueError):
                commit(m, lib, layers)
            assert lib.layers is None
    cs[1].seq_lens = good
    assert commit(m, lib, layers) == live(cs)
    cs[2].k_pages = pool(7)                                # not the size of v_pages
    with pytest.raises(ValueError):
        commit(m, lib, layers)


def test_the_caches_of_a_handle_are_fixed(m, lib):
    cs = caches(m)
    layers = m.KVLayers(cs)
    cs.append(cs[0])                                       # the caller's list is not the handle's
    assert len(layers) == 3 and len(commit(m, lib, layers)) == 3
    with pytest.raises((TypeError, AttributeError)):
        layers.caches.append(cs[0])
    assert len(m.KVLayers([])) == 0
    assert commit(m, lib, m.KVLayers([])) == []
