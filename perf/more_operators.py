"""An 8-bit cache, the attention that reads it, and the pages that caches are made of, as measured cases.

  kv8_write    pages of KV_full held in 8 bits, e4m3 or int8, with one fp32 scale for each page (16 tokens) and KV
               head (``vc.kv8_write``);
  kv8_attn     attention over such a cache: one new token of each request, a block of them (causal), or a tree of
               drafts (``vc.kv8_attn``);
  pages        requests forked from a shared prompt: their pages shared, the page that a fork writes to copied
               first, pages given back (``vc.pages_free``, ``vc.pages_fork``, ``vc.pages_reserve``,
               ``vc.pages_copy``);
  compact      a pool's live pages moved to its lowest ids (``vc.pages_compact``, ``vc.pages_copy``).

``own`` false: the plain form, elementary torch operations in 32 bits.  ``own`` true: the library's calls.
"""
import math

import torch

own = False

PAGE = 16
E4M3 = torch.float8_e4m3fn
TINY = 2.0 ** -126
# the largest code's value, and the factor that makes a scale of a block's largest magnitude
TOP = {"e4m3": 448.0, "int8": 127.0}

# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------


def listed():
    return [
        # one decode step: the page of each of eight requests' new token is made anew, 8B-shaped layer
        dict(name="write_step", op="kv8_write", batch=8, hkv=8, d=128, code="e4m3", lo=4090, hi=4110, new=1),
        # the prompt of four requests, odd lengths
        dict(name="write_prompt", op="kv8_write", batch=4, hkv=8, d=128, code="int8", lo=16000, hi=16384, new=0),
        # the tiny configuration: one request, one KV head, one token
        dict(name="attn_tiny", op="kv8_attn", batch=1, hq=4, hkv=1, d=64, lo=512, hi=512, n_q=1, tree=False,
             code="e4m3"),
        # a decode step, 8B-shaped layer at 32k
        dict(name="attn_8b_32k", op="kv8_attn", batch=8, hq=32, hkv=8, d=128, lo=32768, hi=32768, n_q=1, tree=False,
             code="e4m3"),
        # a decode step, 70B-shaped layer at 128k
        dict(name="attn_70b_128k", op="kv8_attn", batch=4, hq=64, hkv=8, d=128, lo=131072, hi=131072, n_q=1,
             tree=False, code="int8"),
        # a served batch of unequal contexts, a block of five tokens each
        dict(name="attn_batch_block", op="kv8_attn", batch=32, hq=32, hkv=8, d=128, lo=4096, hi=32768, n_q=5,
             tree=False, code="e4m3"),
        # a tree of 32 nodes, 8B-shaped layer at 32k
        dict(name="attn_8b_tree", op="kv8_attn", batch=8, hq=32, hkv=8, d=128, lo=32768, hi=32768, n_q=32, tree=True,
             code="e4m3"),
        # a block of 40 tokens, 70B-shaped layer at 128k
        dict(name="attn_70b_block", op="kv8_attn", batch=4, hq=64, hkv=8, d=128, lo=131072, hi=131072, n_q=40,
             tree=False, code="int8"),
        # four samples of one short prompt, the toy decoder's two layers
        dict(name="fork_few", op="pages", prompts=1, forks=3, lo=250, hi=250, new=1, layers=2, hkv=2, d=128,
             pages=256),
        # eight prompts of odd lengths, seven more samples each, room for a round of 33 tokens
        dict(name="fork_batch", op="pages", prompts=8, forks=7, lo=3000, hi=4096, new=33, layers=4, hkv=8, d=128,
             pages=4096),
        # a small pool, half of it in use
        dict(name="compact_small", op="compact", batch=4, layers=2, hkv=2, d=128, pages=1024, live=0.5),
        # a pool of 8192 pages after a third of its requests left
        dict(name="compact_pool", op="compact", batch=24, layers=2, hkv=8, d=128, pages=8192, live=0.66),
    ]


def _log_int(rng, lo, hi):
    """An integer of [lo, hi], even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _cost(case):
    w = work(case)
    return max(w["bytes"] / 6.8e12, w["flops"] / 1.9e15)


def draw(rng):
    op = rng.choice(["kv8_write", "kv8_attn", "kv8_attn", "pages", "compact"])
    limit = max(_cost(c) for c in listed() if c["op"] == op)
    while True:
        if op == "kv8_write":
            lo = _log_int(rng, 1, 16384)
            case = dict(op=op, batch=_log_int(rng, 1, 32), hkv=rng.choice([1, 2, 4, 8]), d=rng.choice([64, 128]),
                        code=rng.choice(["e4m3", "int8"]), lo=lo, hi=rng.choice([lo, min(16384, 4 * lo)]),
                        new=rng.choice([0, 1, _log_int(rng, 1, 64)]))
        elif op == "kv8_attn":
            hkv = rng.choice([1, 2, 4, 8])
            lo = _log_int(rng, 1, 131072)
            case = dict(op=op, batch=_log_int(rng, 1, 32), hq=hkv * rng.choice([1, 2, 3, 4, 5, 8]), hkv=hkv,
                        d=rng.choice([64, 128]), lo=lo, hi=rng.choice([lo, min(131072, 4 * lo)]),
                        n_q=rng.choice([1, 1, rng.randint(2, 8), rng.randint(2, 64), 64]), tree=rng.random() < 0.5,
                        code=rng.choice(["e4m3", "int8"]))
        elif op == "pages":
            lo = _log_int(rng, 1, 4096)
            case = dict(op=op, prompts=_log_int(rng, 1, 8), forks=_log_int(rng, 1, 16), lo=lo,
                        hi=rng.choice([lo, min(4096, 4 * lo)]), new=rng.choice([1, _log_int(rng, 1, 64)]),
                        layers=_log_int(rng, 1, 8), hkv=rng.choice([1, 2, 4, 8]), d=rng.choice([64, 128]), pages=4096)
            rows = case["prompts"] * case["forks"]
            if case["prompts"] * (case["hi"] // PAGE + 1) + rows * (case["new"] // PAGE + 2) > 4096:
                continue
        else:
            case = dict(op=op, batch=_log_int(rng, 1, 64), layers=_log_int(rng, 1, 4), hkv=rng.choice([1, 2, 4, 8]),
                        d=rng.choice([64, 128]), pages=_log_int(rng, 100, 8192), live=rng.uniform(0.1, 0.9))
        if _cost(case) <= limit:
            return case


def _spread(n, lo, hi):
    """n lengths spread evenly over the logarithm of [lo, hi]."""
    return [int(round(lo * (hi / lo) ** (i / max(1, n - 1)))) for i in range(n)]


def work(case):
    """Each input read once, each output written once; products counted where there are any."""
    op = case["op"]
    if op == "kv8_write":
        rows = sum(n - _first(case, n) // PAGE * PAGE for n in _spread(case["batch"], case["lo"], case["hi"]))
        return {"bytes": 2 * rows * case["hkv"] * (3 * case["d"] + 0.25) + rows / 2, "flops": 0}
    if op == "kv8_attn":
        b, n_q, hq, hkv, d = case["batch"], case["n_q"], case["hq"], case["hkv"], case["d"]
        keys = sum(_spread(b, case["lo"], case["hi"])) + b * n_q
        return {"bytes": keys * hkv * (2 * d + 0.5) + b * n_q * (hq * d * 4 + 8) + keys // 4,
                "flops": 4 * keys * n_q * hq * d}
    if op == "pages":
        lens, f = _spread(case["prompts"], case["lo"], case["hi"]), case["forks"]
        copied = sum(f for n in lens if n % PAGE) * case["layers"] * case["hkv"] * case["d"] * PAGE * 4
        return {"bytes": 2 * copied + sum(n // PAGE + 1 for n in lens) * (1 + 2 * f) * 4 + 64, "flops": 0}
    moved = int(case["pages"] * case["live"] * (1 - case["live"]))
    return {"bytes": moved * case["layers"] * case["hkv"] * case["d"] * PAGE * 8 + case["pages"] * 16, "flops": 0}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _normal(g, shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, 1.0, generator=g)


def _pages_of(n):
    return (n + PAGE - 1) // PAGE


def _table(g, need, total=None):
    """A block table over shuffled pages, need[b] of them in row b (0 behind), and the pages in all."""
    total = total or sum(need)
    width = max(need)
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    n = torch.tensor(need, device="cuda")
    col = torch.arange(width, device="cuda")
    first = torch.cumsum(n, 0) - n
    table = torch.where(col[None] < n[:, None], perm[(first[:, None] + col[None]).clamp(max=total - 1)], 0)
    return table.to(torch.int32).contiguous(), total


def _keys_values(g, pages, hkv, d):
    """K with a few channels of larger values, V with pages of unequal ones; bf16 [page][head][token][channel]."""
    k, v = _normal(g, (pages, hkv, PAGE, d)), _normal(g, (pages, hkv, PAGE, d))
    k[..., ::37] *= 6.0
    v *= torch.exp(0.5 * _normal(g, (pages, hkv, 1, 1), torch.float32)).to(torch.bfloat16)
    return k, v


def _encode(x, code):
    """Codes and scales of blocks [..][16][d] (the last two axes are the block)."""
    x = x.float()
    scale = (x.abs().amax((-1, -2)) * (1.0 / TOP[code])).clamp(min=TINY)
    y = (x * scale.reciprocal()[..., None, None]).clamp(-TOP[code], TOP[code])
    return (y.to(E4M3) if code == "e4m3" else y.round().to(torch.int8)), scale


def _ancestors(g, batch, n_q):
    """Random trees as truth values [b][i][j]: node j is i or an ancestor; every node hangs on one of the eight before
    it, and the last nodes of some requests are left out."""
    i = torch.arange(n_q, device="cuda")
    lo = (i - 8).clamp(min=0)
    u = torch.rand((batch, n_q), generator=g, device="cuda")
    up = (lo + (u * (i - lo)).long()).clamp(max=(i - 1).clamp(min=0))
    anc = torch.eye(n_q, dtype=torch.bool, device="cuda").expand(batch, n_q, n_q).clone()
    for j in range(1, n_q):
        anc[:, j] |= anc[torch.arange(batch, device="cuda"), up[:, j]]
    n = torch.randint(1, n_q + 1, (batch, 1), generator=g, device="cuda")
    return anc & (i[None] < n)[:, :, None]


def _first(case, n):
    """The first position that is new to the 8-bit cache of a request of n tokens (0: all are)."""
    return max(0, n - case["new"]) if case["new"] else 0


def prepare(case, seed):
    g, op, s = _gen(seed), case["op"], dict(case)
    if op in ("kv8_write", "kv8_attn"):
        b, hkv, d = case["batch"], case["hkv"], case["d"]
        lens = _spread(b, case["lo"], case["hi"])
        if op == "kv8_attn":
            lens = [n + case["n_q"] for n in lens]
        s["table"], pages = _table(g, [_pages_of(n) for n in lens])
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["max_len"] = max(lens)
        s["k"], s["v"] = _keys_values(g, pages, hkv, d)
        (s["kc"], s["ks"]), (s["vc"], s["vs"]) = _encode(s["k"], case["code"]), _encode(s["v"], case["code"])
    if op == "kv8_write":
        # the 8-bit cache holds the pages before the new tokens, in an order of its own
        s["table8"], _ = _table(g, [_pages_of(n) for n in lens])
        s["first"] = torch.tensor([_first(case, n) for n in lens], dtype=torch.int32, device="cuda")
    elif op == "kv8_attn":
        n_q, hq = case["n_q"], case["hq"]
        del s["k"], s["v"]
        s["q"] = _normal(g, (b, n_q, hq, d))
        s["mask"] = None
        if case["tree"]:
            s["mask"] = (_ancestors(g, b, n_q).long() << torch.arange(n_q, device="cuda")).sum(-1).contiguous()
        s["scale"] = 1.0 / math.sqrt(d)
        s["out"] = torch.empty((b, n_q, hq, d), dtype=torch.bfloat16, device="cuda")
    elif op == "pages":
        # prompts in the first rows, their samples in the rows behind, empty so far
        p, f, n = case["prompts"], case["forks"], case["pages"]
        lens, rows = _spread(p, case["lo"], case["hi"]), p * (1 + f)
        need = [_pages_of(x) for x in lens]
        width = max(need) + case["new"] // PAGE + 2
        t, _ = _table(g, need, n)
        held = torch.tensor(need + [0] * (p * f), dtype=torch.int32, device="cuda")
        s["table"] = torch.full((rows, width), -1, dtype=torch.int32, device="cuda")
        s["table"][:p, :t.shape[1]] = torch.where(torch.arange(t.shape[1], device="cuda") < held[:p, None], t, -1)
        s["blocks"] = held
        s["refs"] = torch.zeros(n, dtype=torch.int32, device="cuda")
        s["refs"][s["table"][s["table"] >= 0].long()] = 1
        s["lens"] = torch.tensor(lens + [0] * (p * f), dtype=torch.int32, device="cuda")
        s["src"] = torch.arange(p, dtype=torch.int32, device="cuda").repeat_interleave(f)
        s["dst"] = torch.arange(p, rows, dtype=torch.int32, device="cuda")
        s["keep"] = torch.tensor([-1] * p + [0] * (p * f), dtype=torch.int32, device="cuda")
        # the samples go on by `new` tokens, the prompts stay
        s["want"] = torch.tensor([0] * p + [lens[i // f] + case["new"] for i in range(p * f)], dtype=torch.int32,
                                 device="cuda")
        for name in ("copy_src", "copy_dst", "granted"):
            s[name] = torch.zeros(rows, dtype=torch.int32, device="cuda")
        s["k"], s["v"] = (_normal(g, (case["layers"], n, case["hkv"], PAGE, case["d"])) for _ in range(2))
    elif op == "compact":
        b, n = case["batch"], case["pages"]
        live = max(b, int(n * case["live"]))
        need = [live // b + (i < live % b) for i in range(b)]
        t, _ = _table(g, need, n)
        s["blocks"] = torch.tensor(need, dtype=torch.int32, device="cuda")
        s["table0"] = torch.where(torch.arange(t.shape[1], device="cuda") < s["blocks"][:, None], t, -1).contiguous()
        s["refs0"] = torch.zeros(n, dtype=torch.int32, device="cuda")
        s["refs0"][s["table0"][s["table0"] >= 0].long()] = 1
        s["table"], s["refs"] = s["table0"].clone(), s["refs0"].clone()
        s["src"], s["dst"] = (torch.zeros(n // 2, dtype=torch.int32, device="cuda") for _ in range(2))
        s["remap"] = torch.zeros(n, dtype=torch.int32, device="cuda")
        s["moves"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        s["k"], s["v"] = (_normal(g, (case["layers"], n, case["hkv"], PAGE, case["d"])) for _ in range(2))
    if own:
        _plan(s)
    return s


def _plan(s):
    """What a program that uses the library keeps: its caches' handles and workspaces."""
    import lossless_compressed_kv_gb300 as vc
    op = s["op"]
    if op == "kv8_write":
        n, hkv, _, d = s["k"].shape
        s["full"] = vc.PagedKV(s["k"].view(torch.uint8).view(n, -1), s["v"].view(torch.uint8).view(n, -1), s["table"],
                               s["lens"], hkv, d, 16)
    if op in ("kv8_write", "kv8_attn"):
        s["cache"] = vc.PagedKV8(s["kc"], s["vc"], s["ks"], s["vs"], s["table8" if op == "kv8_write" else "table"],
                                 s["lens"])
    if op == "kv8_attn":
        s["ws"] = torch.empty(vc.kv8_workspace_bytes(s["cache"], s["n_q"], s["hq"], s["max_len"]), dtype=torch.uint8,
                              device="cuda")
    if op in ("pages", "compact"):
        s["map"] = vc.PageMap(s["table"], s["blocks"], s["refs"])
        s["arrays"] = vc.PageArrays([x[i] for i in range(s["layers"]) for x in (s["k"], s["v"])])
        s["ws"] = torch.empty(vc.pages_workspace_bytes(s["map"]), dtype=torch.uint8, device="cuda")


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------


def _plain_write(s):
    lens, first, code = s["lens"].long(), s["first"].long() // PAGE, s["code"]
    j = torch.arange(s["table"].shape[1], device="cuda")
    b, j = torch.nonzero((j[None] >= first[:, None]) & (j[None] * PAGE < lens[:, None]), as_tuple=True)
    src, dst = s["table"][b, j].long(), s["table8"][b, j].long()
    there = (j[:, None] * PAGE + torch.arange(PAGE, device="cuda") < lens[b][:, None])[:, None, :, None]
    for x, codes, scales in ((s["k"], s["kc"], s["ks"]), (s["v"], s["vc"], s["vs"])):
        c, scales[dst] = _encode(torch.where(there, x[src].float(), 0.0), code)
        codes.view(torch.uint8)[dst] = c.view(torch.uint8)
    return {n: s[n] for n in ("kc", "ks", "vc", "vs")}


def _decoded(codes, scales, table):
    """[B][kv head][token][channel] in 32 bits, gathered through the block table."""
    b, w = table.shape
    n, hkv, _, d = codes.shape
    x = codes.view(torch.uint8)[table.long()].view(codes.dtype).float() * scales[table.long()][..., None, None]
    return x.transpose(1, 2).reshape(b, hkv, w * PAGE, d)


def _plain_attn(s):
    b, n_q, hq, hkv, d = s["batch"], s["n_q"], s["hq"], s["hkv"], s["d"]
    grp = hq // hkv
    q = s["q"].float().view(b, n_q, hkv, grp, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, n_q * grp, d)
    scores = (q @ _decoded(s["kc"], s["ks"], s["table"]).transpose(-1, -2)).mul_(s["scale"])
    n = scores.shape[-1]
    mask = s["mask"]
    if mask is None:  # a block: token i sees those up to itself
        i = torch.arange(n_q, device="cuda")
        mask = (torch.where(i < 63, (2 << i.clamp(max=62)) - 1, -1)).expand(b, n_q)
    at = torch.arange(n, device="cuda")[None] - (s["lens"].long() - n_q)[:, None]     # place in the block
    bit = (mask[:, :, None] >> at.clamp(0, 63)[:, None]) & 1
    seen = torch.where(at[:, None] < 0, mask[:, :, None] != 0, (at[:, None] < n_q) & (bit != 0))
    seen = seen[:, None, :, None].expand(b, hkv, n_q, grp, n).reshape(b, hkv, n_q * grp, n)
    scores.masked_fill_(~seen, -math.inf)
    top = scores.amax(-1, keepdim=True)
    p = scores.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p @ _decoded(s["vc"], s["vs"], s["table"])) / torch.where(total == 0.0, 1.0, total)
    return s["out"].copy_(o.view(b, hkv, n_q, grp, d).permute(0, 2, 1, 3, 4).reshape(b, n_q, hq, d))


def _give(refs, pages, by):
    """refs of these pages (any shape, -1: none) changed by `by` for each time they are named."""
    refs.scatter_add_(0, pages.clamp(min=0).long().reshape(-1), torch.where(pages >= 0, by, 0).int().reshape(-1))


def _plain_pages(s):
    table, blocks, refs, lens = s["table"], s["blocks"], s["refs"], s["lens"]
    rows, width = table.shape
    col = torch.arange(width, device="cuda")[None]
    # free: pages behind those that keep[b] tokens need
    left = torch.where(s["keep"] < 0, blocks, torch.minimum(blocks, (s["keep"] + PAGE - 1) // PAGE))
    gone = (col >= left[:, None]) & (col < blocks[:, None])
    _give(refs, torch.where(gone, table, -1), -1)
    table.masked_fill_(gone, -1)
    blocks.copy_(left)
    # fork: the pages that hold the prompt's tokens, shared
    src, dst = s["src"].long(), s["dst"].long()
    n = (lens[src] + PAGE - 1) // PAGE
    shared = torch.where(col < n[:, None], table[src], -1)
    table[dst] = shared
    _give(refs, shared, 1)
    blocks[dst], lens[dst] = n, lens[src]
    # reserve: room for `want` tokens, and a page of its own to write to
    want, row = s["want"], torch.arange(rows, device="cuda")
    goal = (want + PAGE - 1) // PAGE
    write = (want > lens)[:, None] & (col >= lens[:, None] // PAGE) & (col < torch.minimum(blocks, goal)[:, None])
    write &= refs[table.clamp(min=0).long()] > 1
    p = torch.where(write, table, refs.numel()).long()
    count = torch.zeros(refs.numel() + 1, dtype=torch.int32, device="cuda")
    last = torch.full((refs.numel() + 1,), -1, dtype=torch.long, device="cuda")
    count.scatter_add_(0, p.reshape(-1), torch.ones_like(p, dtype=torch.int32).reshape(-1))
    last.scatter_reduce_(0, p.reshape(-1), row[:, None].expand(rows, width).reshape(-1), "amax")
    at = p.clamp(max=refs.numel() - 1)
    anew = write & ~((count[p] == refs[at]) & (last[p] == row[:, None]))   # the last of all its writers keeps a page
    need = torch.where(want > lens, anew.sum(1) + (goal - blocks).clamp(min=0), 0)
    upto = need.cumsum(0)
    free = torch.nonzero(refs == 0)[:, 0].int()
    ok = (upto <= free.numel()) | (want <= lens)
    new = (col >= blocks[:, None]) & (col < goal[:, None]) & (want > lens)[:, None]
    take = (anew | new) & ok[:, None]
    begin = (upto - need)[:, None] + torch.where(anew, anew.cumsum(1) - 1, anew.sum(1, keepdim=True) + col - blocks[:, None])
    got = free[begin.clamp(0, max(0, free.numel() - 1)).long()]
    part = (anew & ok[:, None] & (col == lens[:, None] // PAGE)) & (lens % PAGE != 0)[:, None]
    s["copy_src"].copy_(torch.where(part, table, -1).amax(1))
    s["copy_dst"].copy_(torch.where(part, got, -1).amax(1))
    s["granted"].copy_(ok)
    _give(refs, torch.where(anew & take, table, -1), -1)
    _give(refs, torch.where(take, got, -1), 1)
    table.copy_(torch.where(take, got, table))
    blocks.copy_(torch.where(ok & (want > lens), torch.maximum(blocks, goal), blocks))
    # copy: the pages that were written to in part
    here = s["copy_src"] >= 0
    a, z = s["copy_src"][here].long(), s["copy_dst"][here].long()
    s["k"][:, z], s["v"][:, z] = s["k"][:, a], s["v"][:, a]
    return {x: s[x] for x in ("table", "blocks", "refs", "lens", "copy_src", "copy_dst", "granted", "k", "v")}


def _plain_compact(s):
    table, refs = s["table"].copy_(s["table0"]), s["refs"].copy_(s["refs0"])
    live = refs > 0
    n = live.sum()
    i = torch.arange(refs.numel(), device="cuda")
    holes, high = torch.nonzero(~live & (i < n))[:, 0], torch.nonzero(live & (i >= n))[:, 0]
    s["remap"].copy_(torch.where(live, i, -1))
    s["remap"][high] = holes.int()
    s["src"].fill_(-1)[:high.numel()] = high.int()
    s["dst"].fill_(-1)[:high.numel()] = holes.int()
    s["moves"].fill_(high.numel())
    refs[holes] = refs[high]
    refs[high] = 0
    table.copy_(torch.where(table >= 0, s["remap"][table.clamp(min=0).long()], table))
    s["k"][:, holes], s["v"][:, holes] = s["k"][:, high], s["v"][:, high]
    return {x: s[x] for x in ("table", "refs", "remap", "src", "dst", "moves", "k", "v")}


def _own_write(s):
    import lossless_compressed_kv_gb300 as vc
    vc.kv8_write(s["full"], s["first"], s["cache"], s["max_len"])
    return {n: s[n] for n in ("kc", "ks", "vc", "vs")}


def _own_attn(s):
    import lossless_compressed_kv_gb300 as vc
    vc.kv8_attn(s["q"], s["cache"], s["scale"], s["out"], s["max_len"], s["ws"], mask=s["mask"])
    return s["out"]


def _own_pages(s):
    import lossless_compressed_kv_gb300 as vc
    vc.pages_free(s["map"], s["keep"])
    vc.pages_fork(s["map"], s["lens"], s["src"], s["dst"])
    vc.pages_reserve(s["map"], s["lens"], s["want"], s["granted"], s["copy_src"], s["copy_dst"], s["ws"])
    vc.pages_copy(s["arrays"], s["copy_src"], s["copy_dst"])
    return {x: s[x] for x in ("table", "blocks", "refs", "lens", "copy_src", "copy_dst", "granted", "k", "v")}


def _own_compact(s):
    import lossless_compressed_kv_gb300 as vc
    s["table"].copy_(s["table0"])
    s["refs"].copy_(s["refs0"])
    vc.pages_compact(s["map"], s["src"], s["dst"], s["moves"], s["remap"], s["ws"])
    vc.pages_copy(s["arrays"], s["src"], s["dst"], count=s["moves"])
    return {x: s[x] for x in ("table", "refs", "remap", "src", "dst", "moves", "k", "v")}


def run(state):
    if own:
        return {"kv8_write": _own_write, "kv8_attn": _own_attn, "pages": _own_pages,
                "compact": _own_compact}[state["op"]](state)
    return {"kv8_write": _plain_write, "kv8_attn": _plain_attn, "pages": _plain_pages,
            "compact": _plain_compact}[state["op"]](state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------


def _exact_write(s):
    """Scales, and codes before their rounding (those of int8, whole numbers, have no such value)."""
    top, lens, first = TOP[s["code"]], s["lens"].tolist(), s["first"].tolist()
    out = {"kc": s["kc"].to(torch.float32).double(), "vc": s["vc"].to(torch.float32).double(),
           "ks": s["ks"].double(), "vs": s["vs"].double()}
    for b, n in enumerate(lens):
        j0 = first[b] // PAGE
        src, dst = (s[t][b, j0:_pages_of(n)].long() for t in ("table", "table8"))
        for x, c, sc in (("k", "kc", "ks"), ("v", "vc", "vs")):
            y = s[x][src].double()
            if n % PAGE and src.numel():
                y[-1, :, n % PAGE:] = 0.0
            out[sc][dst] = y.abs().flatten(2).max(-1).values / top
            out[c][dst] = y / out[sc][dst].clamp(min=TINY)[..., None, None]
    if s["code"] == "int8":
        out["kc"] = out["vc"] = None
    return out


def _exact_attn(s):
    b, n_q, hq, hkv, d = s["batch"], s["n_q"], s["hq"], s["hkv"], s["d"]
    grp = hq // hkv
    out = torch.zeros((b, n_q, hq, d), dtype=torch.float64, device="cuda")
    for i, n in enumerate(s["lens"].tolist()):
        pages = s["table"][i, :_pages_of(n)].long()
        bias = torch.zeros((n_q, n), dtype=torch.float64, device="cuda")
        if s["mask"] is None:
            see = torch.ones((n_q, n_q), dtype=torch.bool, device="cuda").tril()
        else:
            see = ((s["mask"][i][:, None] >> torch.arange(n_q, device="cuda")) & 1) != 0
        bias[:, n - n_q:][~see] = -math.inf
        for h in range(hkv):
            k, v = ((s[c].view(torch.uint8)[pages, h].view(s[c].dtype).to(torch.float32).double()
                     * s[x][pages, h].double()[:, None, None]).reshape(-1, d)[:n] for c, x in (("kc", "ks"), ("vc", "vs")))
            for j in range(h * grp, (h + 1) * grp):
                out[i, :, j] = torch.softmax(s["q"][i, :, j].double() @ k.T * s["scale"] + bias, -1) @ v
        out[i, ~see.any(-1)] = 0.0
    return out


def _exact_pages(s):
    """The pools' values (everything else is whole numbers)."""
    lens, f, used = s["lens"].tolist(), s["forks"], set(s["table"][s["table"] >= 0].tolist())
    free = iter([p for p in range(s["pages"]) if p not in used])
    k, v = s["k"].double(), s["v"].double()
    table = s["table"].tolist()
    for p in range(s["prompts"]):
        for _ in range(f):
            n, goal = lens[p], _pages_of(lens[p] + s["new"])
            fresh = [next(free) for _ in range(n // PAGE, goal)]
            if n % PAGE:
                k[:, fresh[0]], v[:, fresh[0]] = k[:, table[p][n // PAGE]], v[:, table[p][n // PAGE]]
    return {**dict.fromkeys(("table", "blocks", "refs", "lens", "copy_src", "copy_dst", "granted")), "k": k, "v": v}


def _exact_compact(s):
    refs = s["refs0"].tolist()
    n = sum(r > 0 for r in refs)
    holes, high = [p for p in range(n) if refs[p] == 0], [p for p in range(n, len(refs)) if refs[p] > 0]
    k, v = s["k"].double(), s["v"].double()
    k[:, holes], v[:, holes] = k[:, high], v[:, high]
    return {**dict.fromkeys(("table", "refs", "remap", "src", "dst", "moves")), "k": k, "v": v}


def exact(case, seed):
    s = prepare(case, seed)
    return {"kv8_write": _exact_write, "kv8_attn": _exact_attn, "pages": _exact_pages,
            "compact": _exact_compact}[case["op"]](s)
