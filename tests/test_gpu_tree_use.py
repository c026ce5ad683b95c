"""The tree operations as a serving loop uses them: waits that run out,
several calls at once, graphs that share a workspace, side streams, and
arguments at the ends of their ranges."""
import numpy as np
import pytest
import torch

from oracle import tree as T
from tests import vc_harness as H
from tests.test_gpu_logprobs import check as check_logprobs
from tests.test_gpu_tree import attn, check_attn, q_bf16, random_parents, to_mask

pytestmark = pytest.mark.gpu

BAD_INDEX, TIMEOUT = 3, 6
LIMIT_NS = 20_000          # 20 us per wait


def vc():
    import lossless_compressed_kv_gb300 as m
    return m


def tree_case(seed, lens, n_q, hq, hkv, d):
    rng = np.random.default_rng(seed)
    full, hf = H.full_cache(rng, lens, hkv, d)
    qn, q = q_bf16(rng, (len(lens), n_q, hq, d))
    masks = [T.tree_plan(random_parents(rng, n_q), L)[0] for L in lens]
    return full, hf, qn, q, masks


@pytest.fixture
def fault():
    yield vc().debug_set_wait_fault
    vc().debug_set_wait_fault(0, False)


@pytest.mark.parametrize("n_q", [20, 40, 64])       # one, three (two launches) and four tiles of rows
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_waits_time_out_and_the_next_call_is_clean(fault, n_q, dtype):
    """No copy is issued: every wait on one can only reach its limit.  The call
    reports it, writes zeros and leaves nothing behind."""
    lens = [n_q, 3000, 900]
    full, hf, qn, q, masks = tree_case(n_q, lens, n_q, 14, 2, 64)
    fault(LIMIT_NS, True)
    out, st = attn(full, q, to_mask(masks), 0.125, max(lens), dtype)
    assert st == TIMEOUT and bool((out == 0).all())
    fault(0, False)
    out, st = attn(full, q, to_mask(masks), 0.125, max(lens), dtype)
    assert st == 0
    for b in range(3):
        check_attn(out, hf, qn, masks[b], 0.125, b)


@pytest.mark.parametrize("shapes", [((40, 8, 1, 128), (25, 8, 2, 128)), ((8, 4, 1, 64), (64, 8, 1, 128))])
def test_two_calls_at_once(shapes):
    """On two side streams, each with a workspace of its own, beside the other."""
    m = vc()
    cases = []
    for i, (n_q, hq, hkv, d) in enumerate(shapes):
        lens = [n_q + p for p in (2500, 0, 77)]
        full, hf, qn, q, masks = tree_case([i, n_q], lens, n_q, hq, hkv, d)
        ws = torch.empty(m.tree_workspace_bytes(full, n_q, hq, max(lens)), dtype=torch.uint8, device="cuda")
        cases.append((full, hf, qn, q, masks, to_mask(masks), max(lens), ws, [torch.empty_like(q) for _ in range(6)]))
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for k in range(6):
        for s, c in zip(streams, cases):
            m.tree_attn(c[3], c[0], c[5], 0.09, c[8][k], c[6], c[7], stream=s)
    torch.cuda.synchronize()
    for c in cases:
        for b in range(3):
            check_attn(c[8][0], c[1], c[2], c[4][b], 0.09, b)
        for o in c[8][1:]:
            assert torch.equal(o, c[8][0])


def test_graphs_that_share_a_workspace():
    """Two captured rounds of different sizes, replayed in turn on one workspace."""
    m = vc()
    cases = []
    for i, (n_q, hq, hkv, d, L) in enumerate([(40, 8, 1, 128, 1500), (9, 4, 2, 64, 5000)]):
        lens = [n_q + p for p in (L, 3)]
        full, hf, qn, q, masks = tree_case([7, i], lens, n_q, hq, hkv, d)
        cases.append((full, hf, qn, q, masks, to_mask(masks), max(lens), torch.empty_like(q)))
    ws = torch.empty(max(m.tree_workspace_bytes(c[0], c[3].shape[1], c[3].shape[2], c[6]) for c in cases),
                     dtype=torch.uint8, device="cuda")
    graphs = []
    for c in cases:
        m.tree_attn(c[3], c[0], c[5], 0.1, c[7], c[6], ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            m.tree_attn(c[3], c[0], c[5], 0.1, c[7], c[6], ws)
        graphs.append(g)
    for _ in range(3):
        for c in cases:
            c[7].fill_(7.0)
        ws.fill_(0xFF)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for c in cases:
            for b in range(2):
                check_attn(c[7], c[1], c[2], c[4][b], 0.1, b)


def test_lengths_beyond_the_table():
    """A length of more pages than the table has columns: zeros, reported; the
    other requests are served.  max_seq_len may be any upper bound."""
    n_q, lens = 12, [12, 300, 100]
    full, hf, qn, q, masks = tree_case(5, lens, n_q, 4, 2, 128)
    full.seq_lens[1] = full.block_table.shape[1] * 16 + 1
    out, st = attn(full, q, to_mask(masks), 0.1, 2 ** 31 - 1)
    assert st == BAD_INDEX and bool((out[1] == 0).all())
    for b in (0, 2):
        check_attn(out, hf, qn, masks[b], 0.1, b)


def test_an_accept_of_two_rounds_on_two_streams():
    """The bookkeeping calls take no workspace: any number at once."""
    m = vc()
    rng = np.random.default_rng(9)
    n_q, jobs = 33, []
    for _ in range(4):
        parents = [random_parents(rng, n_q) for _ in range(200)]
        tok, ver = rng.integers(0, 3, (2, 200, n_q))
        p, t, v = (H.to_dev(np.asarray(x, np.int32)) for x in (parents, tok, ver))
        jobs.append((parents, tok, ver, p, t, v, torch.empty(200, dtype=torch.int32, device="cuda"), torch.empty_like(p),
                     torch.empty_like(p), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for j in jobs:
        m.tree_accept(*j[3:9], stream=j[9])
    torch.cuda.synchronize()
    for j in jobs:
        for b in range(200):
            a, path, emitted = T.tree_accept(j[0][b], j[1][b], j[2][b])
            assert int(j[6][b]) == a
            pad = [-1] * (n_q - 1 - a)
            assert j[7][b].tolist() == list(path) + pad and j[8][b].tolist() == list(emitted) + pad


@pytest.mark.parametrize("v", [1000, 20000, 70000])
@pytest.mark.parametrize("scale", [1.0, -1.0])
def test_logits_of_great_size(v, scale):
    """From 2^30 on, a logit's neighbours in fp32 are 64 and more apart: all of
    the probability lies on the largest ones, however many bits the products
    with 1 / (tau log 2) lose."""
    rng = np.random.default_rng(v)
    top = np.float32(scale) * np.exp2(rng.uniform(29, 45, (40, 1))).astype(np.float32)
    steps = rng.integers(0, 6, (40, v))
    x = top.copy().repeat(v, 1)
    for _ in range(5):
        x = np.where(steps > 0, np.nextafter(x, np.float32(-np.inf)), x)
        steps = steps - 1
    x = H.to_dev(np.ascontiguousarray(x, np.float32))
    ids = H.to_dev(rng.integers(0, v, (40, 3)).astype(np.int32))
    _, ent, *_ = check_logprobs(x, ids, 4)
    assert np.isfinite(ent).all()


@pytest.mark.parametrize("v", [1000, 20000, 70000])
def test_calls_of_logprobs_at_once(v):
    """On four streams, a workspace each: the same bits as alone."""
    m = vc()
    g = torch.Generator(device="cuda")
    g.manual_seed(v)
    x = torch.randn((300, v), generator=g, device="cuda").to(torch.bfloat16)
    ids = torch.zeros((300, 1), dtype=torch.int32, device="cuda")
    jobs = [[torch.empty((300, 1), device="cuda"), torch.empty(300, device="cuda"),
             torch.empty((300, 5), dtype=torch.int32, device="cuda"), torch.empty((300, 5), device="cuda"),
             torch.empty(m.token_logprobs_workspace_bytes(300, v, 5), dtype=torch.uint8, device="cuda")] for _ in range(5)]
    streams = [torch.cuda.Stream() for _ in range(4)]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, j in zip(streams, jobs):
            m.token_logprobs(x, ids, j[0], j[4], entropy=j[1], top_ids=j[2], top_logprobs=j[3], stream=s)
    torch.cuda.synchronize()
    j = jobs[4]
    m.token_logprobs(x, ids, j[0], j[4], entropy=j[1], top_ids=j[2], top_logprobs=j[3])
    torch.cuda.synchronize()
    for o in jobs[:4]:
        assert all(torch.equal(a, b) for a, b in zip(o[:4], j[:4]))


TILES = [(16, 16, 2), (32, 16, 2), (40, 16, 2), (64, 16, 2)]      # n_q, hq, hkv: 1 to 4 tiles of 128 rows


@pytest.mark.parametrize("n_q,hq,hkv", TILES)
@pytest.mark.parametrize("d", [64, 128])
def test_maxima_that_grow_block_by_block(n_q, hq, hkv, d):
    """Keys that get longer for 16 blocks of 64, then start again: within a range
    of a dozen blocks the running maximum rises by more than 2^8 most times, and
    what is summed so far is scaled down each time."""
    rng = np.random.default_rng([n_q, d])
    lens = [int(x) for x in rng.integers(7000, 9000, 16)]
    full, hf = H.full_cache(rng, lens, hkv, d)
    kp = full.k_pages.view(torch.bfloat16).view(-1, hkv, 16, d)
    for b, L in enumerate(lens):
        pages = torch.as_tensor(hf["table"][b, :(L + 15) // 16].astype(np.int64), device="cuda")
        f = 1 + 3 * ((torch.arange(len(pages), device="cuda") // 4) % 16)
        kp[pages] = (kp[pages].float() * f.view(-1, 1, 1, 1)).to(torch.bfloat16)
    hf["k"] = full.k_pages.cpu().numpy().view(hf["k"].dtype).reshape(hf["k"].shape)
    qn, q = q_bf16(rng, (len(lens), n_q, hq, d))
    masks = [T.tree_plan(random_parents(rng, n_q), L)[0] for L in lens]
    scale = float(np.float32(d ** -0.5))
    out, st = attn(full, q, to_mask(masks), scale, max(lens), torch.float32)
    assert st == 0
    for b in (0, 7, 15):
        check_attn(out, hf, qn, masks[b], scale, b)


@pytest.mark.parametrize("n_q,hq,hkv", TILES)
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("junk", [float("nan"), -float("inf")])
def test_absent_nodes_may_hold_anything(n_q, hq, hkv, d, junk):
    """Absent nodes and slots behind the request, whatever the tiles: the same bits."""
    rng = np.random.default_rng([n_q, d, 1])
    lens = [n_q, 700, 6000, 64 * 33, 128 * 21 + 1]
    full, hf = H.full_cache(rng, lens, hkv, d)
    qn, q = q_bf16(rng, (len(lens), n_q, hq, d))
    parents = [random_parents(rng, n_q, absent=3) for _ in lens]
    masks = [T.tree_plan(p, L)[0] for p, L in zip(parents, lens)]
    clean, _ = attn(full, q, to_mask(masks), 0.1, max(lens))
    for pool in (full.k_pages, full.v_pages):
        p = pool.view(torch.bfloat16).view(-1, hkv, 16, d)
        for b, L in enumerate(lens):
            for pos in range(L - 3, (L + 15) // 16 * 16):
                p[int(hf["table"][b, pos // 16]), :, pos % 16] = junk
    out, st = attn(full, q, to_mask(masks), 0.1, max(lens))
    assert st == 0 and torch.equal(out, clean) and bool((out[:, -3:] == 0).all())
    for b in (0, 2):
        check_attn(clean, hf, qn, masks[b], 0.1, b)


def test_a_node_that_sees_an_infinite_value():
    """... ends as NaN, and no other does, in any tile."""
    n_q, hq, hkv, d, lens = 40, 8, 1, 128, [3000, 40]
    full, hf, qn, q, _ = tree_case(3, lens, n_q, hq, hkv, d)
    masks = [T.tree_plan([-1] + [i // 2 for i in range(n_q - 1)], L)[0] for L in lens]
    clean, _ = attn(full, q, to_mask(masks), 0.1, max(lens))
    vp = full.v_pages.view(torch.bfloat16).view(-1, hkv, 16, d)
    pos = lens[0] - n_q + 5
    vp[int(hf["table"][0, pos // 16]), :, pos % 16, 3] = float("inf")
    out, st = attn(full, q, to_mask(masks), 0.1, max(lens))
    sees = torch.tensor([bool(m >> 5 & 1) for m in masks[0]], device="cuda")
    assert st == 0 and torch.equal(out[1], clean[1]) and 1 < int(sees.sum()) < n_q
    assert out[0][sees].isnan().all() and torch.equal(out[0][~sees], clean[0][~sees])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("v,k", [(900, 3), (2100, 1), (2603, 30), (6001, 5), (8008, 0), (12001, 2), (20000, 1), (32000, 20),
                                 (40001, 7)])
def test_many_rows(dtype, v, k):
    """Every row of a batch that keeps each block busy for a dozen of them: all
    lengths of rows, all of whose results are checked (tolerances of
    test_gpu_logprobs; the entropy's is 640 2^-24 (2 + 2 entropy))."""
    m, rows, e = vc(), 2003, 2.0 ** -24
    g = torch.Generator(device="cuda")
    g.manual_seed(v)
    x = (torch.randn((rows, v), generator=g, device="cuda") * 3).to(dtype)
    ids = torch.randint(0, v, (rows, 2), generator=g, device="cuda", dtype=torch.int32)
    lp, ent = torch.empty((rows, 2), device="cuda"), torch.empty(rows, device="cuda")
    top, tlp = torch.empty((rows, k), dtype=torch.int32, device="cuda"), torch.empty((rows, k), device="cuda")
    ws = torch.full((m.token_logprobs_workspace_bytes(rows, v, k),), 0xFF, dtype=torch.uint8, device="cuda")
    m.token_logprobs(x, ids, lp, ws, entropy=ent, top_ids=top if k else None, top_logprobs=tlp if k else None)
    torch.cuda.synchronize()
    for r0 in range(0, rows, 500):
        want = x[r0:r0 + 500].double().log_softmax(1)
        w = want.gather(1, ids[r0:r0 + 500].long())
        assert bool(((lp[r0:r0 + 500] - w).abs() <= 640 * e + 4 * e * w.abs()).all())
        h = -(want.exp() * want).sum(1)
        assert bool(((ent[r0:r0 + 500] - h).abs() <= 640 * e * (2 + 2 * h)).all())
        if k:
            order = x[r0:r0 + 500].float().sort(dim=1, descending=True, stable=True)[1][:, :k]    # equal logits by id
            assert torch.equal(top[r0:r0 + 500].long(), order)
            w = want.gather(1, order)
            assert bool(((tlp[r0:r0 + 500] - w).abs() <= 640 * e + 4 * e * w.abs()).all())
