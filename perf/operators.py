"""The operators of a tree-drafted verification round, as measured cases.

A round that drafts a tree of tokens instead of a chain needs, next to the
chain operators of this library:

  rotary       rotary positions in general form, rotated K and V written into
               the paged cache at a slot of their own (``vc.rotary_kv_write``);
  tree_attn    attention of the tree's nodes over KV_full: every node sees the
               prefix and its own ancestors (``vc.tree_attn``);
  tree_round   the round's bookkeeping: masks and positions of the tree, the
               greedy walk, and the accepted path's cache entries moved to
               where a chain would have put them, for all layers
               (``vc.tree_plan``, ``vc.tree_accept``, ``vc.tree_commit``);
  logprobs     log probabilities of given tokens with entropy and the top
               alternatives, from which the next tree is drawn
               (``vc.token_logprobs``).

``own`` false: the plain form, elementary torch operations in 32 bits (64
where the comment says so).  ``own`` true: the library's calls.
"""
import math

import torch

own = False

PAGE = 16
TWO_PI = 2.0 * math.pi
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}

# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------


def listed():
    return [
        # one decode step of eight requests, 8B-shaped layer, frequencies stretched for a long context
        dict(name="rotary_decode", op="rotary", rows_each=1, batch=8, hq=32, hkv=8, d=128, rot=128, interleaved=False,
             scaling="parts", dtype="f32", start=32768),
        # a verification block of 40 tree nodes in four requests, 70B-shaped layer, half of each head rotated
        dict(name="rotary_block", op="rotary", rows_each=40, batch=4, hq=64, hkv=8, d=128, rot=64, interleaved=True,
             scaling="none", dtype="bf16", start=131072),
        # the prompt of the toy decoder: four requests of 16384 tokens
        dict(name="rotary_prompt", op="rotary", rows_each=16384, batch=4, hq=8, hkv=2, d=128, rot=128,
             interleaved=False, scaling="none", dtype="f32", start=0),
        # the tiny configuration: one request, one KV head, eight nodes
        dict(name="tree_tiny", op="tree_attn", batch=1, hq=4, hkv=1, d=64, ctx_lo=512, ctx_hi=512, n_q=8, ragged=False),
        # 8B-shaped layer at 32k, 32 nodes
        dict(name="tree_8b_32k", op="tree_attn", batch=8, hq=32, hkv=8, d=128, ctx_lo=32768, ctx_hi=32768, n_q=32,
             ragged=False),
        # 70B-shaped layer at 128k, 40 nodes
        dict(name="tree_70b_128k", op="tree_attn", batch=4, hq=64, hkv=8, d=128, ctx_lo=131072, ctx_hi=131072, n_q=40,
             ragged=False),
        # a served batch: 32 requests of unequal context, trees of up to 25 nodes
        dict(name="tree_batch_ragged", op="tree_attn", batch=32, hq=32, hkv=8, d=128, ctx_lo=8192, ctx_hi=65536, n_q=25,
             ragged=True),
        # the toy decoder's round: four requests, a comb of 33 nodes, two layers
        dict(name="round_toy", op="tree_round", batch=4, n_q=33, layers=2, hkv=2, d=128, ctx=256),
        # a served batch: 32 requests, 64 nodes, 32 layers
        dict(name="round_batch", op="tree_round", batch=32, n_q=64, layers=32, hkv=8, d=128, ctx=64),
        # a draft step of four requests: the alternatives from which a tree grows
        dict(name="logprobs_draft", op="logprobs", rows=4, vocab=32000, n_ids=1, top_k=8, dtype="f32",
             temperature=1.0),
        # a verification block of eight requests, 33 predictions each
        dict(name="logprobs_block", op="logprobs", rows=264, vocab=32000, n_ids=1, top_k=20, dtype="f32",
             temperature=0.8),
        # a prompt scored: 16384 positions of 16-bit logits
        dict(name="logprobs_prompt", op="logprobs", rows=16384, vocab=32000, n_ids=1, top_k=1, dtype="bf16",
             temperature=1.0),
    ]


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 6.8e12, w["flops"] / 1.9e15)


def draw(rng):
    op = rng.choice(["rotary", "tree_attn", "tree_round", "logprobs"])
    limit = max(_cost(c) for c in listed() if c["op"] == op)
    while True:
        if op == "rotary":
            d = rng.choice([64, 128, 256])
            hkv = rng.choice([1, 2, 4, 8])
            case = dict(op=op, rows_each=_log_int(rng, 1, 16384), batch=_log_int(rng, 1, 32),
                        hq=hkv * rng.choice([1, 2, 3, 4, 7, 8]), hkv=hkv, d=d,
                        rot=rng.choice([d, d // 2, 2 * rng.randint(1, d // 2)]), interleaved=rng.random() < 0.5,
                        scaling=rng.choice(["none", "linear", "parts"]), dtype=rng.choice(["f32", "bf16"]),
                        start=rng.choice([0, _log_int(rng, 1, 1 << 20)]))
        elif op == "tree_attn":
            hkv = rng.choice([1, 2, 4, 8])
            lo = _log_int(rng, 1, 131072)
            case = dict(op=op, batch=_log_int(rng, 1, 32), hq=hkv * rng.choice([1, 2, 3, 4, 5, 8]), hkv=hkv,
                        d=rng.choice([64, 128]), ctx_lo=lo, ctx_hi=rng.choice([lo, min(131072, 4 * lo)]),
                        n_q=rng.choice([1, rng.randint(2, 64), 64]), ragged=rng.random() < 0.5)
        elif op == "tree_round":
            case = dict(op=op, batch=_log_int(rng, 1, 64), n_q=rng.choice([1, rng.randint(2, 64), 64]),
                        layers=_log_int(rng, 1, 32), hkv=rng.choice([1, 2, 4, 8]), d=rng.choice([64, 128]),
                        ctx=rng.randint(1, 300))
        else:
            vocab = _log_int(rng, 1000, 131072)
            case = dict(op=op, rows=_log_int(rng, 1, 16384), vocab=vocab, n_ids=rng.choice([1, 1, 4]),
                        top_k=rng.choice([0, 1, 5, rng.randint(2, 32)]), dtype=rng.choice(["f32", "bf16", "f16"]),
                        temperature=rng.choice([1.0, 0.7, 1.3]))
        if _cost(case) <= limit:
            return case


def work(case):
    """Each input read once, each output written once; products counted where there are any."""
    op = case["op"]
    if op == "rotary":
        rows, hq, hkv, d = case["rows_each"] * case["batch"], case["hq"], case["hkv"], case["d"]
        size = 4 if case["dtype"] == "f32" else 2
        return {"bytes": rows * ((hq + 2 * hkv) * d * (size + 2) + 12), "flops": rows * (hq + hkv) * case["rot"] * 3}
    if op == "tree_attn":
        b, n_q, hq, hkv, d = case["batch"], case["n_q"], case["hq"], case["hkv"], case["d"]
        keys = sum(_contexts(case)) + b * n_q
        return {"bytes": keys * hkv * d * 4 + b * n_q * (hq * d * 4 + 8) + keys // 4, "flops": 4 * keys * n_q * hq * d}
    if op == "tree_round":
        b, n_q = case["batch"], case["n_q"]
        moved = b * min(n_q / 8, 3) * case["layers"] * case["hkv"] * case["d"] * 4   # a few accepted drafts each
        return {"bytes": 2 * moved + b * n_q * 40, "flops": 0}
    size = 4 if case["dtype"] == "f32" else 2
    rows, v = case["rows"], case["vocab"]
    return {"bytes": rows * (v * size + 8 * case["top_k"] + 8 * case["n_ids"] + 4), "flops": rows * v * 6}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _contexts(case):
    """Tokens before the tree of each request: spread evenly over the logarithm of [ctx_lo, ctx_hi]."""
    b, lo, hi = case["batch"], case["ctx_lo"], case["ctx_hi"]
    return [int(round(lo * (hi / lo) ** (i / max(1, b - 1)))) for i in range(b)]


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, dtype, std=1.0):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=g)


def _pages(g, caps):
    """A block table over shuffled pages that covers caps[b] tokens of request b, and the page count."""
    need = [(c + PAGE - 1) // PAGE for c in caps]
    total, width = sum(need), max(need)
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    n = torch.tensor(need, device="cuda")
    col = torch.arange(width, device="cuda")
    first = torch.cumsum(n, 0) - n
    table = torch.where(col[None] < n[:, None], perm[(first[:, None] + col[None]).clamp(max=total - 1)], 0)
    return table.to(torch.int32).contiguous(), total


def _tree(g, batch, n_q, ragged):
    """Random trees: node 0 is the root, every other node hangs on one of the eight nodes before it.  A ragged
    batch leaves the last nodes of some requests out (parent -2)."""
    i = torch.arange(n_q, device="cuda")
    u = torch.rand((batch, n_q), generator=g, device="cuda")
    lo = (i - 8).clamp(min=0)
    parent = lo + (u * (i - lo)).long().clamp(max=(i - lo - 1).clamp(min=0))
    parent[:, 0] = -1
    if ragged:
        n = torch.randint(1, n_q + 1, (batch, 1), generator=g, device="cuda")
        parent = torch.where(i[None] < n, parent, -2)
    return parent.to(torch.int32).contiguous()


def _closure(parent):
    """[b][i][j]: node j is i or one of its ancestors; no row and column for a node that is left out."""
    n = parent.shape[1]
    step = torch.nn.functional.one_hot(parent.long().clamp(min=0), n).double() * (parent >= 0)[..., None]
    anc = torch.matrix_power(step + torch.eye(n, dtype=torch.float64, device="cuda"), n) > 0
    return anc & (parent >= -1)[:, :, None]


def _bits(anc):
    """Truth values [..][n] as one 64-bit word each, value j at bit j."""
    n = anc.shape[-1]
    return (anc.long() << torch.arange(n, device="cuda")).sum(-1)


def _pool(g, layers, pages, hkv, d):
    return _normal(g, (layers, pages, hkv, PAGE, d), torch.bfloat16)


def _own_cache(vc, s, layer=None):
    k, v = (s["k"], s["v"]) if layer is None else (s["k"][layer], s["v"][layer])
    n, hkv, _, d = k.shape
    return vc.PagedKV(k.view(torch.uint8).view(n, -1), v.view(torch.uint8).view(n, -1), s["table"], s["lens"], hkv, d,
                      16)


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = dict(case)
    if op == "rotary":
        b, n = case["batch"], case["rows_each"]
        hq, hkv, d = case["hq"], case["hkv"], case["d"]
        m = b * n
        s["table"], pages = _pages(g, [n + 5] * b)
        s["k"], s["v"] = _pool(g, 1, pages, hkv, d)[0], _pool(g, 1, pages, hkv, d)[0]
        s["qkv"] = _normal(g, (m, (hq + 2 * hkv) * d), DTYPES[case["dtype"]])
        s["req"] = torch.arange(b, dtype=torch.int32, device="cuda").repeat_interleave(n)
        # the cache is written from slot 5 on, at slots of its own: positions lie further on
        s["slot"] = (torch.arange(n, dtype=torch.int32, device="cuda") + 5).repeat(b)
        s["pos"] = s["slot"] - 5 + case["start"]
        s["lens"] = torch.full((b,), n + 5, dtype=torch.int32, device="cuda")
        s["q"] = torch.zeros((m, hq, d), dtype=torch.bfloat16, device="cuda")
        s["params"] = dict(theta=500000.0, rot_dim=case["rot"], interleaved=case["interleaved"])
        if case["scaling"] == "linear":
            s["params"].update(factor=4.0)
        elif case["scaling"] == "parts":
            s["params"].update(factor=8.0, original_len=8192, low_turns=1.0, high_turns=4.0, amplitude=1.1)
        if own:
            import lossless_compressed_kv_gb300 as vc
            s["rotary"] = vc.Rotary(**s["params"])
            s["full"] = _own_cache(vc, s)
    elif op == "tree_attn":
        b, n_q, hq, hkv, d = case["batch"], case["n_q"], case["hq"], case["hkv"], case["d"]
        lens = [c + n_q for c in _contexts(case)]
        s["table"], pages = _pages(g, lens)
        s["k"], s["v"] = _pool(g, 1, pages, hkv, d)[0], _pool(g, 1, pages, hkv, d)[0]
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["max_len"] = max(lens)
        s["qs"] = _normal(g, (b, n_q, hq, d), torch.bfloat16)
        s["mask"] = _bits(_closure(_tree(g, b, n_q, case["ragged"]))).contiguous()
        s["scale"] = 1.0 / math.sqrt(d)
        s["out"] = torch.empty((b, n_q, hq, d), dtype=torch.bfloat16, device="cuda")
        if own:
            import lossless_compressed_kv_gb300 as vc
            s["full"] = _own_cache(vc, s)
            s["ws"] = torch.empty(vc.tree_workspace_bytes(s["full"], n_q, hq, s["max_len"]), dtype=torch.uint8,
                                  device="cuda")
    elif op == "tree_round":
        b, n_q, layers, hkv, d = case["batch"], case["n_q"], case["layers"], case["hkv"], case["d"]
        cap = case["ctx"] + n_q
        s["table"], pages = _pages(g, [cap] * b)
        s["k"], s["v"] = _pool(g, layers, pages, hkv, d), _pool(g, layers, pages, hkv, d)
        s["lens"] = torch.full((b,), cap, dtype=torch.int32, device="cuda")
        s["parent"] = _tree(g, b, n_q, True)
        # few distinct tokens, so that siblings may hold the same one; the verifier mostly agrees with a child
        s["tokens"] = torch.randint(0, 50, (b, n_q), generator=g, device="cuda", dtype=torch.int32)
        i = torch.arange(n_q, device="cuda").expand(b, n_q)
        child = torch.zeros((b, n_q), dtype=torch.long, device="cuda").scatter_reduce_(
            1, s["parent"].long().clamp(min=0), torch.where(s["parent"] >= 0, i, 0), "amax")
        agree = (torch.rand((b, n_q), generator=g, device="cuda") < 0.85) & (child > 0)
        other = torch.randint(0, 50, (b, n_q), generator=g, device="cuda", dtype=torch.int32)
        s["verified"] = torch.where(agree, s["tokens"].gather(1, child), other)
        for name, shape, dt in (("mask", (b, n_q), torch.int64), ("position", (b, n_q), torch.int32),
                                ("accept_len", (b,), torch.int32), ("path", (b, n_q), torch.int32),
                                ("emitted", (b, n_q), torch.int32)):
            s[name] = torch.zeros(shape, dtype=dt, device="cuda")
        if own:
            import lossless_compressed_kv_gb300 as vc
            s["layers_kv"] = vc.KVLayers([_own_cache(vc, s, i) for i in range(layers)])
    else:
        rows, v, n_ids, k = case["rows"], case["vocab"], case["n_ids"], case["top_k"]
        x = _normal(g, (rows, v), torch.float32, 2.5)
        # what a trained model gives: one token far above the rest in most rows
        at = torch.randint(0, v, (rows, 1), generator=g, device="cuda")
        x.scatter_add_(1, at, 10.0 + 4.0 * torch.randn((rows, 1), generator=g, device="cuda"))
        s["logits"] = x.to(DTYPES[case["dtype"]])
        del x
        ids = torch.randint(0, v, (rows, n_ids), generator=g, device="cuda")
        likely = torch.rand((rows, n_ids), generator=g, device="cuda") < 0.6
        s["ids"] = torch.where(likely, at, ids).to(torch.int32).contiguous()
        s["logprobs"] = torch.zeros((rows, n_ids), device="cuda")
        s["entropy"] = torch.zeros((rows,), device="cuda")
        s["top_ids"] = torch.zeros((rows, k), dtype=torch.int32, device="cuda")
        s["top_logprobs"] = torch.zeros((rows, k), device="cuda")
        if own:
            import lossless_compressed_kv_gb300 as vc
            s["ws"] = torch.empty(vc.token_logprobs_workspace_bytes(rows, v, k), dtype=torch.uint8, device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------


def _frequencies(p):
    """Radians per position of each rotated pair, in 64 bits (far positions need them)."""
    i = torch.arange(p["rot_dim"] // 2, dtype=torch.float64, device="cuda")
    f = torch.exp(i * (-2.0 * math.log(p["theta"]) / p["rot_dim"]))
    if p.get("factor", 1.0) == 1.0:
        return f
    if not p.get("original_len"):
        return f / p["factor"]
    turns = p["original_len"] * f / TWO_PI
    keep = ((turns - p["low_turns"]) / (p["high_turns"] - p["low_turns"])).clamp(0.0, 1.0)
    return f * ((1.0 - keep) / p["factor"] + keep)


def _plain_rotary(s):
    m, hq, hkv, d, rot = s["qkv"].shape[0], s["hq"], s["hkv"], s["d"], s["rot"]
    x = s["qkv"].float().view(m, hq + 2 * hkv, d)
    angle = s["pos"].double()[:, None] * _frequencies(s["params"])[None]
    amp = s["params"].get("amplitude", 1.0)
    cos, sin = (torch.cos(angle) * amp).float()[:, None], (torch.sin(angle) * amp).float()[:, None]
    qk = x[:, :hq + hkv]
    if s["interleaved"]:
        a, b = qk[..., 0:rot:2], qk[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = qk[..., :rot // 2], qk[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    qk = torch.cat([turned, qk[..., rot:]], -1).to(torch.bfloat16)
    page, at = s["table"][s["req"].long(), (s["slot"] // PAGE).long()].long(), (s["slot"] % PAGE).long()
    s["q"].copy_(qk[:, :hq])
    s["k"][page, :, at] = qk[:, hq:]
    s["v"][page, :, at] = x[:, hq + hkv:].to(torch.bfloat16)
    return s["q"], s["k"], s["v"]


def _rows_of(pool, table):
    """[B][kv head][token][channel] in 32 bits, gathered through the block table."""
    b, w = table.shape
    x = pool[table.long()]                         # [B][w][hkv][16][d]
    return x.transpose(1, 2).reshape(b, pool.shape[1], w * PAGE, pool.shape[3]).float()


def _plain_tree_attn(s):
    b, n_q, hq, hkv, d = s["batch"], s["n_q"], s["hq"], s["hkv"], s["d"]
    grp = hq // hkv
    q = s["qs"].float().view(b, n_q, hkv, grp, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, n_q * grp, d)
    scores = (q @ _rows_of(s["k"], s["table"]).transpose(-1, -2)).mul_(s["scale"])
    n = scores.shape[-1]
    at = torch.arange(n, device="cuda")[None] - (s["lens"].long() - n_q)[:, None]     # place in the tree
    bit = (s["mask"][:, :, None] >> at.clamp(0, 63)[:, None]) & 1
    seen = torch.where(at[:, None] < 0, s["mask"][:, :, None] != 0, (at[:, None] < n_q) & (bit != 0))
    seen = seen[:, None, :, None].expand(b, hkv, n_q, grp, n).reshape(b, hkv, n_q * grp, n)
    scores.masked_fill_(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = scores.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p @ _rows_of(s["v"], s["table"])) / torch.where(total == 0.0, 1.0, total)
    o = o.view(b, hkv, n_q, grp, d).permute(0, 2, 1, 3, 4).reshape(b, n_q, hq, d)
    return s["out"].copy_(o)


def _plain_tree_round(s):
    parent, n = s["parent"].long(), s["n_q"]
    anc = _closure(s["parent"])
    base = (s["lens"].long() - n)[:, None]
    here = parent >= -1
    s["mask"].copy_(_bits(anc))
    s["position"].copy_(torch.where(here, base + anc.sum(-1) - 1, -1))
    up = parent.clamp(min=0)
    hit = (parent >= 0) & (s["tokens"] == s["verified"].gather(1, up))
    i = torch.arange(n, device="cuda")
    twin = (up[:, :, None] == up[:, None, :]) & hit[:, None, :] & (i[None, :] < i[:, None])[None]
    ok = hit & ~twin.any(-1)                       # the first sibling that holds the verifier's token
    ok[:, 0] = parent[:, 0] == -1
    kept = ~(anc & ~ok[:, None, :]).any(-1) & here
    a = kept.sum(-1) - 1
    path = torch.where(kept, i, n).sort(-1).values
    last = path.gather(1, a.clamp(min=0)[:, None])
    nxt = torch.cat([path[:, 1:], torch.full_like(path[:, :1], n)], 1)     # path from its first accepted draft on
    tokens = s["tokens"].gather(1, nxt.clamp(max=n - 1)).long()
    end = s["verified"].gather(1, last.clamp(max=n - 1)).long()
    s["accept_len"].copy_(a)
    s["path"].copy_(torch.where(path < n, path, -1))
    s["emitted"].copy_(torch.where(i[None] < a[:, None], tokens, torch.where(i[None] == a[:, None], end, -1)))
    to = base + i[None]
    src = torch.where(path < n, base + path, to)
    b = torch.arange(parent.shape[0], device="cuda")[:, None]
    pg, at = s["table"][b, src // PAGE].long(), src % PAGE
    pt, att = s["table"][b, to // PAGE].long(), to % PAGE
    s["k"][:, pt, :, att] = s["k"][:, pg, :, at]
    s["v"][:, pt, :, att] = s["v"][:, pg, :, at]
    return {x: s[x] for x in ("mask", "position", "accept_len", "path", "emitted", "k", "v")}


def _order(x):
    """Whole numbers in the order of the values of a 32-bit tensor (equal values alike)."""
    bits = (x + 0.0).view(torch.int32).long()
    return torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)


def _plain_logprobs(s):
    x = s["logits"].float()
    top = x.amax(-1, keepdim=True)
    y = (x - top) / s["temperature"]
    p = y.exp()
    total = p.sum(-1, keepdim=True)
    log_total = total.log()
    s["entropy"].copy_((log_total - (p * y).sum(-1, keepdim=True) / total)[:, 0])
    s["logprobs"].copy_(y.gather(1, s["ids"].long()) - log_total)
    if s["top_k"]:
        v = x.shape[1]
        place = torch.arange(v - 1, -1, -1, device="cuda")
        key = (_order(x) * (1 << 20) + place).topk(s["top_k"], -1).values  # equal logits: the lowest id first
        ids = v - 1 - (key & ((1 << 20) - 1))
        s["top_ids"].copy_(ids)
        s["top_logprobs"].copy_(y.gather(1, ids) - log_total)
    return {n: s[n] for n in ("logprobs", "entropy", "top_ids", "top_logprobs")}


def _own_rotary(s):
    import lossless_compressed_kv_gb300 as vc
    vc.rotary_kv_write(s["qkv"], s["req"], s["pos"], s["hq"], s["rotary"], s["q"], s["full"], row_slot=s["slot"])
    return s["q"], s["k"], s["v"]


def _own_tree_attn(s):
    import lossless_compressed_kv_gb300 as vc
    vc.tree_attn(s["qs"], s["full"], s["mask"], s["scale"], s["out"], s["max_len"], s["ws"])
    return s["out"]


def _own_tree_round(s):
    import lossless_compressed_kv_gb300 as vc
    vc.tree_plan(s["parent"], s["lens"], s["mask"], s["position"])
    vc.tree_accept(s["parent"], s["tokens"], s["verified"], s["accept_len"], s["path"], s["emitted"])
    vc.tree_commit(s["layers_kv"], s["accept_len"], s["path"])
    return {x: s[x] for x in ("mask", "position", "accept_len", "path", "emitted", "k", "v")}


def _own_logprobs(s):
    import lossless_compressed_kv_gb300 as vc
    vc.token_logprobs(s["logits"], s["ids"], s["logprobs"], s["ws"], temperature=s["temperature"],
                      entropy=s["entropy"], top_ids=s["top_ids"], top_logprobs=s["top_logprobs"])
    return {n: s[n] for n in ("logprobs", "entropy", "top_ids", "top_logprobs")}


def run(state):
    if own:
        return {"rotary": _own_rotary, "tree_attn": _own_tree_attn, "tree_round": _own_tree_round,
                "logprobs": _own_logprobs}[state["op"]](state)
    return {"rotary": _plain_rotary, "tree_attn": _plain_tree_attn, "tree_round": _plain_tree_round,
            "logprobs": _plain_logprobs}[state["op"]](state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------


def _exact_rotary(s):
    hq, hkv, d, half, p = s["hq"], s["hkv"], s["d"], s["rot"] // 2, s["params"]
    f = []
    for i in range(half):
        w = p["theta"] ** (-i / half)
        if p.get("original_len"):
            r = p["original_len"] * w / TWO_PI
            k = min(1.0, max(0.0, (r - p["low_turns"]) / (p["high_turns"] - p["low_turns"])))
            w = k * w + (1 - k) * w / p["factor"]
        else:
            w = w / p.get("factor", 1.0)
        f.append(w)
    m = s["qkv"].shape[0]
    x = s["qkv"].double().view(m, hq + 2 * hkv, d)
    z = torch.polar(torch.full((m, half), float(p.get("amplitude", 1.0)), dtype=torch.float64, device="cuda"),
                    s["pos"].double()[:, None] * torch.tensor(f, dtype=torch.float64, device="cuda"))
    first = torch.arange(half, device="cuda") * (2 if s["interleaved"] else 1)
    second = first + (1 if s["interleaved"] else half)
    y = x.clone()
    c = torch.complex(x[:, :hq + hkv, first], x[:, :hq + hkv, second]) * z[:, None]
    y[:, :hq + hkv, first], y[:, :hq + hkv, second] = c.real, c.imag
    k, v = s["k"].double(), s["v"].double()
    page, at = s["table"][s["req"].long(), (s["slot"] // PAGE).long()].long(), (s["slot"] % PAGE).long()
    k[page, :, at], v[page, :, at] = y[:, hq:hq + hkv], y[:, hq + hkv:]
    return y[:, :hq], k, v


def _exact_tree_attn(s):
    b, n_q, hq, hkv, d = s["batch"], s["n_q"], s["hq"], s["hkv"], s["d"]
    grp = hq // hkv
    out = torch.zeros((b, n_q, hq, d), dtype=torch.float64, device="cuda")
    lens = s["lens"].tolist()
    for i in range(b):
        n = lens[i]
        pages = s["table"][i, :(n + PAGE - 1) // PAGE].long()
        bits = (s["mask"][i][:, None] >> torch.arange(n_q, device="cuda")) & 1
        bias = torch.zeros((n_q, n), dtype=torch.float64, device="cuda")
        bias[:, n - n_q:] = torch.where(bits != 0, 0.0, -math.inf)
        for h in range(hkv):
            k = s["k"][pages, h].reshape(-1, d)[:n].double()
            v = s["v"][pages, h].reshape(-1, d)[:n].double()
            for j in range(grp):
                e = s["qs"][i, :, h * grp + j].double() @ k.T * s["scale"] + bias
                out[i, :, h * grp + j] = torch.softmax(e, -1) @ v
    return torch.where((s["mask"] != 0)[..., None, None], out, 0.0)


def _exact_tree_round(s):
    parents, tokens, verified = s["parent"].tolist(), s["tokens"].tolist(), s["verified"].tolist()
    lens, table, n = s["lens"].tolist(), s["table"].tolist(), s["n_q"]
    k, v = s["k"].double(), s["v"].double()
    src_p, src_s, dst_p, dst_s = [], [], [], []
    for b, parent in enumerate(parents):
        base, cur, to = lens[b] - n, 0, 0
        while parent[0] == -1:
            child = next((j for j in range(cur + 1, n) if parent[j] == cur and tokens[b][j] == verified[b][cur]), None)
            if child is None:
                break
            cur, to = child, to + 1
            src, dst = base + cur, base + to
            src_p.append(table[b][src // PAGE])
            src_s.append(src % PAGE)
            dst_p.append(table[b][dst // PAGE])
            dst_s.append(dst % PAGE)
    k[:, dst_p, :, dst_s] = k[:, src_p, :, src_s]
    v[:, dst_p, :, dst_s] = v[:, src_p, :, src_s]
    return {"mask": None, "position": None, "accept_len": None, "path": None, "emitted": None, "k": k, "v": v}


def _exact_logprobs(s):
    out = {"logprobs": [], "entropy": [], "top_logprobs": []}
    for x in s["logits"].split(512):
        at = sum(t.shape[0] for t in out["entropy"])
        lp = torch.log_softmax(x.double() / s["temperature"], -1)
        out["logprobs"].append(lp.gather(1, s["ids"][at:at + x.shape[0]].long()))
        out["entropy"].append(-(lp.exp() * lp).sum(-1))
        out["top_logprobs"].append(lp.sort(-1, descending=True).values[:, :s["top_k"]])
    return {"top_ids": None, **{n: torch.cat(v) for n, v in out.items()}}


def exact(case, seed):
    s = prepare(case, seed)
    return {"rotary": _exact_rotary, "tree_attn": _exact_tree_attn, "tree_round": _exact_tree_round,
            "logprobs": _exact_logprobs}[case["op"]](s)
