"""GPU tree operations (vc_tree_plan, vc_tree_attn, vc_tree_accept,
vc_tree_commit) against their 64-bit definitions, and a whole round of them.

Attention tolerance per channel: the probabilities enter the second product
in bf16 (half a step: 2^-8 of each, so 2^-8 sum_t p_t |v_tc|); a score is a
sum of head_dim exact products in fp32, off by at most D 2^-23 of sum |q k|
scale, which shifts p by as much relatively, in numerator and denominator
(factor 2, and 2 more for the shared reference maximum's rounding); exp2 and
the sums add below 2^-13 (n < 2^10 keys a chain of fp32 additions).  A bf16
output adds half a step, 2^-8 of the value."""
import math

import numpy as np
import pytest
import torch

import synth
from oracle import tree as T
from tests import vc_harness as H

pytestmark = pytest.mark.gpu


def vc():
    import lossless_compressed_kv_gb300 as m
    return m


def random_parents(rng, n_q, wide=8, absent=0):
    p = [-1] + [int(rng.integers(max(0, i - wide), i)) for i in range(1, n_q)]
    for i in range(n_q - absent, n_q):
        p[i] = -2
    return p


def to_mask(masks):
    return H.to_dev(np.array(masks, dtype=np.uint64).view(np.int64))


def attn(full, q, mask, scale, max_len, dtype=torch.bfloat16, ws=None):
    m = vc()
    out = torch.full(q.shape, 3.0, dtype=dtype, device="cuda")
    if ws is None:
        ws = torch.full((m.tree_workspace_bytes(full, q.shape[1], q.shape[2], max_len),), 0xFF, dtype=torch.uint8,
                        device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    m.tree_attn(q, full, mask, scale, out, max_len, ws, status=st)
    torch.cuda.synchronize()
    return out, int(st.item())


def q_bf16(rng, shape):
    qn = synth.normal_bf16(rng, shape)
    return synth.bf16_to_f32(qn).astype(np.float64), H.to_dev(qn.view(np.int16)).view(torch.bfloat16)


def check_attn(out, hf, qn, masks, scale, b, n=None):
    kb, vb = H.logical_full(hf, b, n)
    k, v = (synth.bf16_to_f32(t).astype(np.float64) for t in (kb, vb))
    ref, spread, serr = T.tree_attn(qn[b], k, v, masks, scale)
    e = 2.0 ** -8 + 2.0 ** -13 + 4 * qn.shape[-1] * 2.0 ** -23 * serr[..., None]
    tol = e * spread + (2.0 ** -8 * np.abs(ref) if out.dtype == torch.bfloat16 else 0.0)
    got = out[b].double().cpu().numpy()
    assert np.isfinite(got).all()
    bad = np.abs(got - ref) > tol
    assert not bad.any(), (b, np.argwhere(bad)[:4], got[bad][:4], ref[bad][:4], tol[bad][:4])


SHAPES = [  # hq, hkv, d, n_q, prefix lengths
    (4, 1, 64, 8, [512]),
    (4, 2, 128, 1, [0, 1, 15, 16, 17, 63, 64, 65]),
    (8, 1, 128, 17, [0, 5, 47, 48, 300]),
    (8, 8, 64, 5, [130, 0]),
    (5, 1, 128, 13, [100, 7]),
    (14, 2, 64, 40, [90, 640]),
    (32, 8, 128, 32, [200, 33]),
    (8, 1, 128, 64, [70, 0, 129]),
    (3, 1, 64, 64, [1000]),
]


@pytest.mark.parametrize("hq,hkv,d,n_q,pre", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_tree_attention(hq, hkv, d, n_q, pre, dtype):
    rng = np.random.default_rng([hq, d, n_q, len(pre)])
    lens = [p + n_q for p in pre]
    full, hf = H.full_cache(rng, lens, hkv, d, spare_pages=2)
    qn, q = q_bf16(rng, (len(pre), n_q, hq, d))
    masks = [T.tree_plan(random_parents(rng, n_q, absent=int(rng.integers(0, n_q))), L)[0] for L in lens]
    scale = float(np.float32(1.0 / math.sqrt(d)))
    out, st = attn(full, q, to_mask(masks), scale, max(lens), dtype)
    assert st == 0
    for b in range(len(pre)):
        check_attn(out, hf, qn, masks[b], scale, b)


@pytest.mark.parametrize("n_q,hq,hkv", [(25, 8, 2), (40, 8, 1), (64, 8, 1), (60, 10, 2)])
def test_long_ragged_batch(n_q, hq, hkv):
    """Contexts of many splits beside short ones; every row checked."""
    rng = np.random.default_rng([n_q, hq])
    lens = [n_q + p for p in (0, 3000, 17, 9001, 640, 1, 4096)]
    full, hf = H.full_cache(rng, lens, hkv, 64)
    qn, q = q_bf16(rng, (len(lens), n_q, hq, 64))
    masks = [T.tree_plan(random_parents(rng, n_q), L)[0] for L in lens]
    out, st = attn(full, q, to_mask(masks), 0.125, max(lens))
    assert st == 0
    for b in range(len(lens)):
        check_attn(out, hf, qn, masks[b], 0.125, b)


def test_many_short_requests():
    """More requests than the GPU has room for: several per block."""
    rng = np.random.default_rng(77)
    lens = [int(x) for x in rng.integers(3, 90, 500)]
    full, hf = H.full_cache(rng, lens, 2, 64)
    qn, q = q_bf16(rng, (500, 3, 4, 64))
    masks = [T.tree_plan(random_parents(rng, 3), L)[0] for L in lens]
    out, st = attn(full, q, to_mask(masks), 0.125, max(lens))
    assert st == 0
    for b in range(0, 500, 7):
        check_attn(out, hf, qn, masks[b], 0.125, b)


def test_any_mask_and_bits_past_the_tree():
    """Masks need not come from a tree; bits from n_q on are not read."""
    rng = np.random.default_rng(3)
    n_q, lens = 20, [20, 77, 300]
    full, hf = H.full_cache(rng, lens, 2, 128)
    qn, q = q_bf16(rng, (3, n_q, 8, 128))
    masks = [[int(x) for x in rng.integers(0, 1 << n_q, n_q)] for _ in lens]
    masks[0][3] = masks[1][4] = 0
    high = [[m | (0xFFFFFFFFFFF << n_q) if m else 0 for m in r] for r in masks]
    out, st = attn(full, q, to_mask(masks), 0.1, 300)
    out2, _ = attn(full, q, to_mask(high), 0.1, 300)
    assert st == 0 and torch.equal(out, out2)
    for b in range(3):
        check_attn(out, hf, qn, masks[b], 0.1, b)
    assert (out[0, 3] == 0).all() and (out[1, 4] == 0).all()
    # only bits past the tree set: as no bit at all
    only = [[1 << n_q] * n_q] * 3
    out3, _ = attn(full, q, to_mask(only), 0.1, 300)
    assert (out3 == 0).all()


def test_chain_agrees_with_verify_attn():
    rng = np.random.default_rng(4)
    n_q, lens = 9, [50, 4000]
    full, _ = H.full_cache(rng, lens, 2, 128)
    _, q = q_bf16(rng, (2, n_q, 8, 128))
    masks = [T.tree_plan([-1] + list(range(n_q - 1)), L)[0] for L in lens]
    out, _ = attn(full, q, to_mask(masks), 0.09, 4000, torch.float32)
    ref = torch.empty(q.shape, dtype=torch.float32, device="cuda")
    ws = torch.empty(vc().verify_workspace_bytes(full, n_q, 8, 4000), dtype=torch.uint8, device="cuda")
    vc().verify_attn(q, full, 0.09, ref, 4000, ws)
    torch.cuda.synchronize()
    assert H.row_err(out.cpu().numpy(), ref.cpu().numpy()) <= 2 * H.TOL


@pytest.mark.parametrize("junk", [float("nan"), float("inf"), -float("inf"), 3.0e38])
def test_masked_entries_may_hold_anything(junk):
    """Absent nodes, siblings and slots behind the request."""
    rng = np.random.default_rng(6)
    hkv, d, n_q = 2, 64, 12
    lens = [60, 150]
    full, hf = H.full_cache(rng, lens, hkv, d, capacity=[80, 170])
    parent = [-1, 0, 0, 1, 2, 3, 3, 4, 4, 2, -2, -2]
    masks = [T.tree_plan(parent, L)[0] for L in lens]
    qn, q = q_bf16(rng, (2, n_q, 8, d))
    clean, _ = attn(full, q, to_mask(masks), 0.125, 150)
    kp = full.k_pages.view(torch.bfloat16).view(-1, hkv, 16, d)
    vp = full.v_pages.view(torch.bfloat16).view(-1, hkv, 16, d)
    for b, L in enumerate(lens):
        # node 9 (nobody's ancestor), the absent nodes and everything behind the request
        for pos in [L - n_q + 9, L - 2, L - 1] + list(range(L, 80 if b == 0 else 160)):
            pg = int(hf["table"][b, pos // 16])
            kp[pg, :, pos % 16] = junk
            vp[pg, :, pos % 16] = junk
    out, st = attn(full, q, to_mask(masks), 0.125, 150)
    assert st == 0
    keep = [i for i in range(n_q) if i != 9]
    assert torch.equal(out[:, keep], clean[:, keep])
    if not math.isfinite(junk):
        assert out[:, 9].isnan().all()


def test_bad_lengths_and_pages_are_reported():
    rng = np.random.default_rng(7)
    lens = [30, 4, 90, 200]
    full, hf = H.full_cache(rng, lens, 1, 64)
    qn, q = q_bf16(rng, (4, 8, 4, 64))
    masks = [T.tree_plan(random_parents(rng, 8), max(L, 8))[0] for L in lens]
    out, st = attn(full, q, to_mask(masks), 0.125, 100)     # request 1 is shorter than its tree, 3 too long
    assert st == 3 and (out[1] == 0).all() and (out[3] == 0).all()
    check_attn(out, hf, qn, masks[0], 0.125, 0)
    check_attn(out, hf, qn, masks[2], 0.125, 2)
    for page in (-1, full.num_pages, 1 << 30):
        full.block_table.copy_(H.to_dev(hf["table"]))
        full.block_table[2, 2] = page
        out, st = attn(full, q, to_mask(masks), 0.125, 100)
        assert st == 3 and out[2].isfinite().all()
        check_attn(out, hf, qn, masks[0], 0.125, 0)


def test_same_bits_from_call_to_call_and_from_a_graph():
    rng = np.random.default_rng(8)
    lens = [700, 5000, 64]
    full, _ = H.full_cache(rng, lens, 2, 128)
    _, q = q_bf16(rng, (3, 33, 8, 128))
    mask = to_mask([T.tree_plan(random_parents(rng, 33), L)[0] for L in lens])
    a, _ = attn(full, q, mask, 0.09, 5000)
    b, _ = attn(full, q, mask, 0.09, 5000)
    assert torch.equal(a, b)
    ws = torch.empty(vc().tree_workspace_bytes(full, 33, 8, 5000), dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(a)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        vc().tree_attn(q, full, mask, 0.09, out, 5000, ws)
    for _ in range(3):
        out.zero_()
        ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, a)
    s = torch.cuda.Stream()
    out.zero_()
    torch.cuda.synchronize()
    vc().tree_attn(q, full, mask, 0.09, out, 5000, ws, stream=s)
    s.synchronize()
    assert torch.equal(out, a)


# ---------------------------------------------------------------------------
# plan, accept, commit
# ---------------------------------------------------------------------------

def bad_trees(rng, n_q):
    p = random_parents(rng, n_q)
    for _ in range(n_q // 4 + 1):
        i = int(rng.integers(0, n_q))
        p[i] = int(rng.choice([-3, -2, -1, i, n_q, 1 << 30]))
    return p


@pytest.mark.parametrize("n_q", [1, 2, 7, 32, 33, 63, 64])
@pytest.mark.parametrize("kind", ["tree", "chain", "bad"])
def test_plan_and_accept(n_q, kind):
    rng = np.random.default_rng([n_q, len(kind)])
    B = 40
    mk = dict(tree=lambda: random_parents(rng, n_q, absent=int(rng.integers(0, n_q))),
              chain=lambda: [-1] + list(range(n_q - 1)), bad=lambda: bad_trees(rng, n_q))[kind]
    parents = [mk() for _ in range(B)]
    lens = [int(x) for x in rng.integers(n_q, 3000, B)]
    if kind == "bad":
        lens[3] = n_q - 1
    tok = rng.integers(0, 3, (B, n_q)).astype(np.int32)
    ver = rng.integers(0, 3, (B, n_q)).astype(np.int32)
    for b in range(0, B, 2):                          # every other request: a long walk
        for i in range(n_q):
            kids = [j for j in range(n_q) if parents[b][j] == i and j > i]
            if kids:
                ver[b, i] = tok[b, kids[-1]]
    pd = H.to_dev(np.array(parents, np.int32))
    mask = torch.zeros((B, n_q), dtype=torch.int64, device="cuda")
    pos = torch.zeros((B, n_q), dtype=torch.int32, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    vc().tree_plan(pd, H.to_dev(np.array(lens, np.int32)), mask, pos, status=st)
    al = torch.zeros(B, dtype=torch.int32, device="cuda")
    path, em = torch.zeros_like(pos), torch.zeros_like(pos)
    vc().tree_accept(pd, H.to_dev(tok), H.to_dev(ver), al, path, em)
    mask, pos, al, path, em = (t.cpu().numpy() for t in (mask, pos, al, path, em))
    any_bad = False
    for b in range(B):
        m, p, bad = T.tree_plan(parents[b], lens[b])
        any_bad |= bad
        assert [int(x) & (2 ** 64 - 1) for x in mask[b]] == m and list(pos[b]) == p
        a, w, e = T.tree_accept(parents[b], tok[b], ver[b])
        assert int(al[b]) == a
        assert list(path[b]) == w + [-1] * (n_q - len(w)) and list(em[b]) == e + [-1] * (n_q - len(e))
    assert int(st.item()) == (3 if any_bad else 0)


@pytest.mark.parametrize("hkv,d,n_q,layers", [(1, 32, 5, 1), (2, 64, 64, 3), (8, 128, 33, 2), (3, 96, 20, 70)])
def test_commit(hkv, d, n_q, layers):
    rng = np.random.default_rng([hkv, d, n_q])
    lens = np.array([n_q, n_q + 3, n_q + 30, 2 * n_q + 17], np.int32)
    table, total = synth.block_tables(rng, lens)
    td, ld = H.to_dev(table), H.to_dev(lens)
    kvs = []
    for _ in range(layers):
        p = [torch.randint(0, 256, (total, hkv * 16 * d * 2), dtype=torch.uint8, device="cuda") for _ in range(2)]
        kvs.append(vc().PagedKV(*p, td, ld, hkv, d, 16))
    paths = [[0] + sorted(rng.choice(np.arange(1, n_q), size=int(rng.integers(0, n_q)), replace=False).tolist())
             for _ in lens]
    paths[1], paths[2] = list(range(n_q)), [0]
    al = np.array([len(p) - 1 for p in paths], np.int32)
    pa = np.array([p + [-1] * (n_q - len(p)) for p in paths], np.int32)
    before = [(kv.k_pages.clone(), kv.v_pages.clone()) for kv in kvs]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    vc().tree_commit(vc().KVLayers(kvs), H.to_dev(al), H.to_dev(pa), status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    for kv, old in zip(kvs, before):
        for new, was in zip((kv.k_pages, kv.v_pages), old):
            want = was.clone().view(total, hkv, 16, 2 * d)
            src = was.view(total, hkv, 16, 2 * d)
            for b, p in enumerate(paths):
                base = int(lens[b]) - n_q
                for j, i in enumerate(p):
                    want[table[b, (base + j) // 16], :, (base + j) % 16] = \
                        src[table[b, (base + i) // 16], :, (base + i) % 16]
            assert torch.equal(new.view(total, hkv, 16, 2 * d), want)


def test_commit_leaves_bad_requests_alone():
    rng = np.random.default_rng(1)
    n_q = 6
    lens = np.array([20, 20, 20, 5, 20, 20, 20], np.int32)
    full, _ = H.full_cache(rng, np.maximum(lens, 20), 2, 64)
    full.seq_lens.copy_(H.to_dev(lens))
    good = [0, 2, 5, -1, -1, -1]
    pa = np.array([good, [0, 3, 2, -1, -1, -1], [0, 2, 6, -1, -1, -1], good, [1, 2, 5, -1, -1, -1], good, good],
                  np.int32)
    al = np.array([2, 2, 2, 2, 2, 6, -2], np.int32)
    before = full.k_pages.clone()
    layers = vc().KVLayers([full])
    for only in range(1, 7):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        a = np.full(7, -1, np.int32)
        a[only] = al[only]
        vc().tree_commit(layers, H.to_dev(a), H.to_dev(pa), status=st)
        torch.cuda.synchronize()
        assert st.item() == 3 and torch.equal(full.k_pages, before), only
    full.block_table[0, 0] = 1 << 20                         # positions 14, 15 of the tree: 16 moves, 15 cannot
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    vc().tree_commit(layers, H.to_dev(np.array([2] + [-1] * 6, np.int32)), H.to_dev(pa), status=st)
    torch.cuda.synchronize()
    assert st.item() == 3


# ---------------------------------------------------------------------------
# a round of them together
# ---------------------------------------------------------------------------

def test_a_round_and_its_commit_continue_like_a_chain():
    """Rotary write of a tree's nodes, plan, attention, predictions with
    alternatives, walk, commit; then the committed cache gives the attention
    that the same tokens written as a chain give."""
    m = vc()
    torch.manual_seed(3)
    rng = np.random.default_rng(3)
    B, hq, hkv, d, n_q, pre, vocab, dm = 3, 8, 2, 128, 20, 75, 500, 256
    dev = "cuda"
    rot = m.Rotary(500000.0, d, factor=4.0, original_len=64, low_turns=1.0, high_turns=8.0, amplitude=1.05)
    wqkv = (torch.randn((dm, (hq + 2 * hkv) * d), device=dev) * dm ** -0.5).to(torch.bfloat16)
    head = (torch.randn((hq * d, vocab), device=dev) * 0.2).to(torch.bfloat16)
    emb = torch.randn((vocab, dm), device=dev)
    npg = (pre + n_q + 15) // 16
    table = H.to_dev(rng.permutation(B * npg).reshape(B, npg).astype(np.int32))
    lens = torch.full((B,), pre + n_q, dtype=torch.int32, device=dev)
    full = m.PagedKV.allocate(B * npg, hkv, d, 16, table, lens, zero=True)
    st = torch.zeros(1, dtype=torch.int32, device=dev)

    def write(cache, ids, pos, slot):
        n = ids.shape[1]
        x = torch.empty((B * n, dm), device=dev)
        m.embed(ids.reshape(-1).contiguous(), emb, x, status=st)
        qkv = torch.empty((B * n, (hq + 2 * hkv) * d), device=dev)
        m.linear(x, wqkv, qkv)
        q = torch.empty((B * n, hq, d), dtype=torch.bfloat16, device=dev)
        req = torch.arange(B, dtype=torch.int32, device=dev).repeat_interleave(n)
        req = torch.where(pos.reshape(-1) >= 0, req, -1)             # absent nodes are padding rows
        m.rotary_kv_write(qkv, req, pos.reshape(-1).contiguous(), hq, rot, q.view(B * n, hq, d), cache,
                          row_slot=slot.reshape(-1).contiguous(), status=st)
        return torch.where((pos >= 0)[..., None, None], q.view(B, n, hq, d), 0).contiguous()

    prompt = torch.randint(0, vocab, (B, pre), dtype=torch.int32, device=dev)
    pp = torch.arange(pre, dtype=torch.int32, device=dev).expand(B, pre)
    write(full, prompt, pp, pp)
    parent = H.to_dev(np.array([random_parents(rng, n_q, absent=a) for a in (0, 3, 19)], np.int32))
    tokens = torch.randint(0, vocab, (B, n_q), dtype=torch.int32, device=dev)
    mask = torch.empty((B, n_q), dtype=torch.int64, device=dev)
    pos = torch.empty((B, n_q), dtype=torch.int32, device=dev)
    m.tree_plan(parent, lens, mask, pos, status=st)
    slot = (pre + torch.arange(n_q, dtype=torch.int32, device=dev)).expand(B, n_q)
    q = write(full, tokens, pos, slot)
    out = torch.empty((B, n_q, hq, d), dtype=torch.float32, device=dev)
    ws = torch.empty(m.tree_workspace_bytes(full, n_q, hq, pre + n_q), dtype=torch.uint8, device=dev)
    m.tree_attn(q, full, mask, d ** -0.5, out, pre + n_q, ws, status=st)
    logits = torch.empty((B * n_q, vocab), device=dev)
    m.linear(out.view(B * n_q, hq * d), head, logits)
    ids = tokens.view(-1, 1).contiguous()
    lp = torch.empty((B * n_q, 1), device=dev)
    ent = torch.empty(B * n_q, device=dev)
    top = torch.empty((B * n_q, 2), dtype=torch.int32, device=dev)
    tlp = torch.empty((B * n_q, 2), device=dev)
    lws = torch.empty(m.token_logprobs_workspace_bytes(B * n_q, vocab, 2), dtype=torch.uint8, device=dev)
    m.token_logprobs(logits, ids, lp, lws, entropy=ent, top_ids=top, top_logprobs=tlp, status=st)
    ref = torch.log_softmax(logits.double(), -1)
    assert (lp[:, 0].double() - ref.gather(1, ids.long())[:, 0]).abs().max() < 1e-5
    assert torch.equal(top[:, 0].long(), logits.argmax(-1))
    # the verifier agrees with a path of the first two requests: their last child each time
    verified = top[:, 0].view(B, n_q).clone()
    ph, th, vh = parent.cpu().numpy(), tokens.cpu().numpy(), verified.cpu().numpy()
    for b in (0, 1):
        cur = 0
        while True:
            kids = [j for j in range(cur + 1, n_q) if ph[b, j] == cur]
            if not kids:
                break
            vh[b, cur] = th[b, kids[-1]]
            cur = kids[-1]
    verified.copy_(torch.from_numpy(vh))
    al = torch.empty(B, dtype=torch.int32, device=dev)
    path, em = (torch.empty((B, n_q), dtype=torch.int32, device=dev) for _ in range(2))
    m.tree_accept(parent, tokens, verified, al, path, em)
    m.tree_commit(m.KVLayers([full]), al, path, status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    ah = al.cpu().numpy()
    for b in range(B):
        a, w, e = T.tree_accept(ph[b], th[b], vh[b])
        assert ah[b] == a and list(path[b].cpu().numpy()[:a + 1]) == w and list(em[b].cpu().numpy()[:a + 1]) == e
    assert ah[0] > 1 and ah[1] > 1 and ah[2] == 0
    # the same tokens as a chain, in a cache of its own
    chain = m.PagedKV.allocate(B * npg, hkv, d, 16, table, lens, zero=True)
    write(chain, prompt, pp, pp)
    n = int(ah.max()) + 1
    ctok = torch.gather(tokens, 1, path[:, :n].clamp(min=0).long()).to(torch.int32)
    cpos = (pre + torch.arange(n, dtype=torch.int32, device=dev)).expand(B, n).contiguous()
    cpos = torch.where(path[:, :n] >= 0, cpos, -1)
    write(chain, ctok, cpos, cpos.clamp(min=0))
    kf, kc = (t.k_pages.view(torch.bfloat16).view(-1, hkv, 16, d) for t in (full, chain))
    vf, vcn = (t.v_pages.view(torch.bfloat16).view(-1, hkv, 16, d) for t in (full, chain))
    tb = table.cpu().numpy()
    for b in range(B):
        for p in range(pre + int(ah[b]) + 1):
            pg = int(tb[b, p // 16])
            assert torch.equal(kf[pg, :, p % 16], kc[pg, :, p % 16]), (b, p)
            assert torch.equal(vf[pg, :, p % 16], vcn[pg, :, p % 16]), (b, p)
