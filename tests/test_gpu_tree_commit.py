"""vc_tree_commit through the Python handle of the layers: what is moved after
the caches carry other tensors than when the handle was built."""
import gc

import numpy as np
import pytest
import torch

import synth
from tests import vc_harness as H

pytestmark = pytest.mark.gpu


def vc():
    import lossless_compressed_kv_gb300 as m
    return m


def layers_of(rng, lens, hkv, d, n_layers):
    """Caches of random bytes that share a table and lengths."""
    table, total = synth.block_tables(rng, np.asarray(lens, np.int32))
    td, ld = H.to_dev(table), H.to_dev(np.asarray(lens, np.int32))
    kvs = []
    for _ in range(n_layers):
        p = [torch.randint(0, 256, (total, hkv * 16 * d * 2), dtype=torch.uint8, device="cuda") for _ in range(2)]
        kvs.append(vc().PagedKV(*p, td, ld, hkv, d, 16))
    return kvs, table


def moved(pool, table, hkv, d, lens, n_q, paths, skip=()):
    """A pool after the commit of `paths`; entries (request, j) in `skip` stay."""
    was = pool.view(-1, hkv, 16, 2 * d)
    want = was.clone()
    for b, p in enumerate(paths):
        base = int(lens[b]) - n_q
        for j, i in enumerate(p):
            if (b, j) not in skip:
                want[table[b, (base + j) // 16], :, (base + j) % 16] = \
                    was[table[b, (base + i) // 16], :, (base + i) % 16]
    return want.view(pool.shape)


def commit(layers, paths, n_q):
    al = np.array([len(p) - 1 for p in paths], np.int32)
    pa = np.array([p + [-1] * (n_q - len(p)) for p in paths], np.int32)
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    vc().tree_commit(layers, H.to_dev(al), H.to_dev(pa), status=st)
    torch.cuda.synchronize()
    return int(st.item())


def test_commits_after_rebound_lengths_and_tables():
    """One handle over several rounds, as a loop keeps it: the lengths written
    out of place, a table with more columns, a smaller batch, pools that grew."""
    rng = np.random.default_rng(5)
    hkv, d, n_q = 2, 64, 9
    lens = np.array([40, 70, 33, 25], np.int32)
    kvs, table = layers_of(rng, [96] * 4, hkv, d, 3)
    for kv in kvs:
        kv.seq_lens = H.to_dev(lens)                       # a tensor of its own for each layer ...
    paths = [[0, 2, 5], [0, 1, 2, 8], [0], [0, 7]]

    def step(layers, lens, paths):
        want = [[moved(p, table, hkv, d, lens, n_q, paths) for p in (kv.k_pages, kv.v_pages)] for kv in kvs]
        assert commit(layers, paths, n_q) == 0
        for kv, (k, v) in zip(kvs, want):
            assert torch.equal(kv.k_pages, k) and torch.equal(kv.v_pages, v)

    layers = vc().KVLayers(kvs)
    with pytest.raises(vc().VCError):                      # ... is refused
        commit(layers, paths, n_q)
    shared = H.to_dev(lens)
    for kv in kvs:
        kv.seq_lens = shared
    step(layers, lens, paths)
    for _ in range(3):
        kept = np.array([len(p) for p in paths], np.int32)  # what stays of the tree; the next one follows it
        lens, shared = lens + kept, shared + H.to_dev(kept)
        for kv in kvs:
            kv.seq_lens = shared
        gc.collect()
        step(layers, lens, paths)
    wide = H.to_dev(np.concatenate([table, table[:, :1]], 1))
    for kv in kvs:
        kv.block_table = wide
    step(layers, lens, paths)
    for kv in kvs:
        kv.block_table, kv.seq_lens = wide[:2], shared[:2]
    with pytest.raises(ValueError):
        commit(layers, paths, n_q)
    two = kvs[0].block_table, kvs[0].seq_lens
    for kv in kvs:
        kv.block_table, kv.seq_lens = two
    step(layers, lens[:2], paths[:2])
    for kv in kvs:
        kv.k_pages, kv.v_pages = (torch.cat([p, p[:3]]) for p in (kv.k_pages, kv.v_pages))
    gc.collect()
    step(layers, lens[:2], paths[:2])


def test_refused_requests_keep_both_pools():
    rng = np.random.default_rng(1)
    n_q, hkv, d = 6, 2, 64
    lens = np.array([20, 20, 20, 5, 20, 20, 20], np.int32)
    kvs, _ = layers_of(rng, np.maximum(lens, 20), hkv, d, 2)
    kvs[0].seq_lens.copy_(H.to_dev(lens))
    good = [0, 2, 5, -1, -1, -1]
    pa = H.to_dev(np.array([good, [0, 3, 2, -1, -1, -1], [0, 2, 6, -1, -1, -1], good, [1, 2, 5, -1, -1, -1], good, good],
                           np.int32))
    before = [(kv.k_pages.clone(), kv.v_pages.clone()) for kv in kvs]
    layers = vc().KVLayers(kvs)
    for only, a in enumerate([2, 2, 2, 2, 6, -2], 1):
        al = np.full(7, -1, np.int32)
        al[only] = a
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        vc().tree_commit(layers, H.to_dev(al), pa, status=st)
        torch.cuda.synchronize()
        assert st.item() == 3, only
        for kv, (k, v) in zip(kvs, before):
            assert torch.equal(kv.k_pages, k) and torch.equal(kv.v_pages, v), only


@pytest.mark.parametrize("page", [-1, 1 << 20, "count"])
@pytest.mark.parametrize("column,skipped", [(0, [(0, 1)]), (1, [(0, 1), (0, 2), (0, 3)]), (2, [(0, 3)])])
def test_a_bad_page_stops_its_entries_alone(page, column, skipped):
    """The tree of request 0 lies in positions 14 to 35, its path's moves are 16
    -> 15, 20 -> 16 and 33 -> 17: a bad page of either end stops a move, the
    others and the other requests are served."""
    rng = np.random.default_rng(2)
    n_q, hkv, d, lens = 22, 2, 64, np.array([36, 50, 36], np.int32)
    kvs, table = layers_of(rng, lens, hkv, d, 2)
    paths = [[0, 2, 6, 19], [0, 4, 21], [0, 1, 3]]
    kvs[0].block_table[0, column] = kvs[0].num_pages if page == "count" else page
    want = [[moved(p, table, hkv, d, lens, n_q, paths, skipped) for p in (kv.k_pages, kv.v_pages)] for kv in kvs]
    assert commit(vc().KVLayers(kvs), paths, n_q) == 3
    for kv, (k, v) in zip(kvs, want):
        assert torch.equal(kv.k_pages, k) and torch.equal(kv.v_pages, v)
