"""GPU 8-bit cache (vc_kv8_write, vc_kv8_attn) against its plain definitions.

What is written is equal bit for bit.  Attention's tolerance per channel is
derived in oracle/kv8.py (fp16 probabilities, fp32 scores); a bf16 output
adds half a step, 2^-8 of the value."""
import math

import numpy as np
import pytest
import torch

import synth
from oracle import kv8 as K
from tests import vc_harness as H

pytestmark = pytest.mark.gpu
CODES = {"e4m3": torch.float8_e4m3fn, "int8": torch.int8}


def vc():
    import lossless_compressed_kv_gb300 as m
    return m


def i32(x):
    return H.to_dev(np.array(x, dtype=np.int32))


def status():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------------------
# write
# ---------------------------------------------------------------------------


@pytest.mark.parametrize("d,code,hkv", [(64, "e4m3", 1), (128, "e4m3", 3), (64, "int8", 5), (128, "int8", 2)])
@pytest.mark.parametrize("first", [None, "last", "some"])
def test_write(d, code, hkv, first):
    m, rng = vc(), np.random.default_rng(d + hkv)
    lens = [1, 15, 16, 17, 0, 100, 33, 250] + [5] * 40
    full, hf = H.full_cache(rng, lens, hkv, d, [3, 9], 8.0, spare_pages=2)
    hf["k"][hf["table"][6, 0], 0] = 0                                  # a block of zeros
    for b, n in enumerate(lens):                                       # NaN behind the last token takes no part
        if n % 16:
            hf["v"][hf["table"][b, n // 16], :, n % 16:] = 0x7fc0
            hf["k"][hf["table"][b, n // 16], :, n % 16:] = 0xff80
    full.k_pages.copy_(H.to_dev(hf["k"].view(np.uint8).reshape(full.k_pages.shape)))
    full.v_pages.copy_(H.to_dev(hf["v"].view(np.uint8).reshape(full.v_pages.shape)))
    table, total = synth.block_tables(rng, lens, [n + 20 for n in lens])
    c8 = m.PagedKV8.allocate(total, hkv, d, CODES[code], H.to_dev(table), i32([0] * len(lens)))
    for t in (c8.k_codes, c8.v_codes):
        t.view(torch.uint8).fill_(0x55)
    for t in (c8.k_scales, c8.v_scales):
        t.fill_(-3.0)
    start = [0] * len(lens) if first is None else [max(0, n - 1) for n in lens] if first == "last" else \
        [int(rng.integers(0, n + 20)) for n in lens]
    st = status()
    m.kv8_write(full, None if first is None else i32(start), c8, max(lens), status=st)
    torch.cuda.synchronize()
    assert st.item() == 0
    for codes, scales, pool in ((c8.k_codes, c8.k_scales, hf["k"]), (c8.v_codes, c8.v_scales, hf["v"])):
        ref = np.full((total, hkv, 16, d), 0x55, np.uint8)
        rs = np.full((total, hkv), -3.0, np.float32)
        for b, n in enumerate(lens):
            for j in range(start[b] // 16, -(-n // 16) if start[b] < n else 0):
                x = synth.bf16_to_f32(pool[hf["table"][b, j]]).copy()
                x[:, max(0, n - 16 * j):] = 0.0
                for h in range(hkv):
                    ref[table[b, j], h], rs[table[b, j], h], _ = K.block(x[h], code)
        got = codes.view(torch.uint8).cpu().numpy()
        assert np.array_equal(scales.cpu().numpy(), rs)
        # (a zero has either sign in e4m3)
        assert np.array_equal(np.where(got == 0x80, 0, got), np.where(ref == 0x80, 0, ref)) if code == "e4m3" else np.array_equal(got, ref)


@pytest.mark.parametrize("code", ["e4m3", "int8"])
def test_write_infinities_nan_and_extremes(code):
    m, rng = vc(), np.random.default_rng(5)
    full, hf = H.full_cache(rng, [48], 1, 64)
    x = hf["k"][hf["table"][0]]
    x[0, 0, 2, 3], x[0, 0, 4, 5], x[0, 0, 6, 7] = 0x7fc1, 0x7f80, 0xff80
    x[1, 0] = synth.bf16_bits(synth.bf16_to_f32(x[1, 0]) * np.float32(2.0 ** 125))
    x[2, 0] = synth.bf16_bits(synth.bf16_to_f32(x[2, 0]) * np.float32(2.0 ** -124))
    hf["k"][hf["table"][0]] = x
    full.k_pages.copy_(H.to_dev(hf["k"].view(np.uint8).reshape(full.k_pages.shape)))
    c8 = m.PagedKV8.allocate(3, 1, 64, CODES[code], i32([[0, 1, 2]]), i32([48]))
    st = status()
    m.kv8_write(full, None, c8, 48, status=st)
    torch.cuda.synchronize()
    assert st.item() == 1
    for j in range(3):
        ref, s, _ = K.block(synth.bf16_to_f32(x[j, 0]), code)
        got = c8.k_codes[j, 0].view(torch.uint8).cpu().numpy()
        assert c8.k_scales[j, 0].item() == s
        assert np.array_equal(K.decode(got, code), K.decode(ref, code))


def test_write_reports_what_is_out_of_range():
    m, rng = vc(), np.random.default_rng(6)
    lens = [20, 20, 20, 20, 20]
    full, hf = H.full_cache(rng, lens, 2, 64)
    full.block_table[1, 1] = 99
    full.seq_lens[4] = 500
    c8 = m.PagedKV8.allocate(10, 2, 64, torch.int8, i32(np.arange(10).reshape(5, 2)), i32(lens))
    c8.block_table[2, 0] = -1
    st = status()
    m.kv8_write(full, i32([0, 0, 0, -1, 0]), c8, 32, status=st)
    torch.cuda.synchronize()
    assert st.item() == 3
    wrote = (c8.k_scales != 0).any(1).tolist()
    assert wrote == [True, True, True, False, False, True, False, False, False, False]


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------


def cache(rng, lens, hkv, d, code, k_scale=None, v_scale=None, junk=0xff):
    """An 8-bit cache of random codes and scales; junk behind the last token."""
    table, total = synth.block_tables(rng, lens)
    total += 1
    out = []
    for _ in range(2):
        x = rng.integers(0, 256, (total, hkv, 16, d), dtype=np.uint8)
        if code == "e4m3":
            x[(x & 0x7f) == 0x7f] = 0x3a
            x = np.where(rng.random(x.shape) < 0.9, (x & 0x87) | (rng.integers(2, 11, x.shape, dtype=np.uint8) << 3), x).astype(np.uint8)
        out.append(x)
    ks = (rng.uniform(0.5, 2.0, (total, hkv)) / (4.0 if code == "e4m3" else 60.0)).astype(np.float32)
    vs = (np.exp2(rng.uniform(-6, 3, (total, hkv)))).astype(np.float32)
    ks, vs = ks if k_scale is None else k_scale(ks), vs if v_scale is None else v_scale(vs)
    for b, n in enumerate(lens):
        if n % 16:
            for x in out:
                x[table[b, n // 16], :, n % 16:] = junk
    dt = CODES[code]
    c8 = vc().PagedKV8(*[H.to_dev(x).view(dt) for x in out], H.to_dev(ks), H.to_dev(vs), H.to_dev(table),
                       i32(lens))
    return c8, dict(k=out[0], v=out[1], ks=ks, vs=vs, table=table, lens=lens, code=code)


def run(q, c8, scale, max_len, mask=None, dtype=torch.float32, ws=None):
    m = vc()
    out = torch.full(q.shape, 3.0, dtype=dtype, device="cuda")
    n_q = q.shape[1] if q.dim() == 4 else 1
    if ws is None:
        ws = torch.full((m.kv8_workspace_bytes(c8, n_q, q.shape[-2], max_len),), 0xFF, dtype=torch.uint8, device="cuda")
    st = status()
    m.kv8_attn(q, c8, scale, out, max_len, ws, mask=mask, status=st)
    torch.cuda.synchronize()
    return out, int(st.item())


def q_of(rng, shape):
    x = synth.normal_bf16(rng, shape)
    return synth.bf16_to_f32(x).astype(np.float64), H.to_dev(x.view(np.int16)).view(torch.bfloat16)


def values(h, b, head):
    n = h["lens"][b]
    pg = h["table"][b, :-(-n // 16)]
    fix = lambda s: np.clip(np.where(np.isnan(s), 0, s), 2.0 ** -126, 2.0 ** 122).astype(np.float64)  # noqa: E731
    k, v = ((K.decode(h[c][pg, head], h["code"]) * fix(h[s][pg, head])[:, None, None]).reshape(-1, h[c].shape[3])[:n]
            for c, s in (("k", "ks"), ("v", "vs")))
    return k, v, float(fix(h["vs"][pg, head]).max() * K.TOP[h["code"]])


def check(out, h, qn, scale, mask=None, half=2.0 ** -24, only=None):
    out = out.double().cpu().numpy()
    B, n_q, hq, d = qn.shape
    hkv = h["k"].shape[1]
    for b in range(B):
        n = h["lens"][b]
        if n < n_q or (only is not None and b not in only):
            assert n >= n_q or not out[b].any()
            continue
        seen = np.zeros((n_q, n), bool)
        for i in range(n_q):
            bits = (1 << (i + 1)) - 1 if mask is None else int(mask[b][i]) & ((1 << n_q) - 1)
            if bits:
                seen[i, :n - n_q] = True
                seen[i, n - n_q:] = [(bits >> j) & 1 for j in range(n_q)]
        for g in range(hkv):
            k, v, top = values(h, b, g)
            for head in range(g * hq // hkv, (g + 1) * hq // hkv):
                ref, tol = K.attn(qn[b, :, head], k, v, seen, scale, top)
                err = np.abs(out[b, :, head] - ref)
                assert (err <= tol + half * np.abs(ref) + 1e-30).all(), (b, head, float((err - tol).max()), n)


LENS = {"one": [1, 2, 15, 16, 17], "mixed": [64, 0, 65, 79, 300, 1037, 16, 80, 96], "long": [5000]}


@pytest.mark.parametrize("code", ["e4m3", "int8"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("hq,hkv,n_q,lens", [(1, 1, 1, "one"), (8, 1, 1, "mixed"), (12, 4, 1, "long"), (7, 1, 2, "mixed"),
                                             (6, 2, 3, "mixed"), (8, 1, 4, "long"), (10, 2, 5, "one"), (8, 2, 13, "mixed"),
                                             (5, 5, 33, "mixed"), (8, 2, 32, "mixed"), (8, 1, 64, "mixed"),
                                             (4, 1, 40, "long"), (6, 1, 64, "long"), (8, 8, 1, "one"), (3, 1, 64, "mixed")])
def test_attention_of_a_block(code, d, hq, hkv, n_q, lens):
    rng = np.random.default_rng(hq * 100 + n_q)
    lens = [max(n, n_q) if n else 0 for n in LENS[lens]]
    c8, h = cache(rng, lens, hkv, d, code)
    qn, q = q_of(rng, (len(lens), n_q, hq, d))
    out, st = run(q, c8, 1 / math.sqrt(d), max(lens))
    assert st == 0
    check(out, h, qn, 1 / math.sqrt(d))
    again, _ = run(q, c8, 1 / math.sqrt(d), max(lens))
    assert torch.equal(out, again)
    half, _ = run(q, c8, 1 / math.sqrt(d), max(lens), dtype=torch.bfloat16)
    check(half, h, qn, 1 / math.sqrt(d), half=2.0 ** -8)
    if n_q == 1:
        flat, _ = run(q[:, 0], c8, 1 / math.sqrt(d), max(lens))
        assert torch.equal(flat, out[:, 0])


@pytest.mark.parametrize("code,d,hq,n_q", [("e4m3", 128, 2, 4), ("int8", 64, 4, 7), ("e4m3", 64, 8, 8), ("int8", 128, 8, 33),
                                           ("e4m3", 128, 5, 64), ("int8", 64, 2, 64), ("e4m3", 64, 8, 50)])
def test_attention_of_a_tree(code, d, hq, n_q):
    """Masks of trees, of nothing, of all, with bits behind n_q; rows whose only keys are the block's."""
    rng = np.random.default_rng(n_q)
    lens = [n_q, n_q + 1, 16 * 9, 700, n_q + 15]
    lens = [max(n, n_q) for n in lens]
    c8, h = cache(rng, lens, 2, d, code)
    mask = [[int(rng.integers(0, 1 << 62)) | 1 << i for i in range(n_q)] for _ in lens]
    mask[0][0], mask[1], mask[2][n_q - 1], mask[3][0] = 0, [0] * n_q, (1 << 64) - 1, 1 << (n_q - 1)
    t = H.to_dev(np.array(mask, dtype=np.uint64).view(np.int64))
    qn, q = q_of(rng, (len(lens), n_q, 2 * hq, d))
    out, st = run(q, c8, 0.1, max(lens), mask=t)
    assert st == 0
    check(out, h, qn, 0.1, mask)


def test_many_requests_and_long_ranges():
    """Ranges of many pages (ids are read 32 at a time), requests beyond a warp's lanes."""
    rng = np.random.default_rng(9)
    lens = [45000, 44987, 30001, 52000, 45008, 44000] + [3] * 70
    c8, h = cache(rng, lens, 8, 64, "int8")
    qn, q = q_of(rng, (len(lens), 1, 8, 64))
    out, st = run(q, c8, 0.125, max(lens))
    assert st == 0
    check(out, h, qn, 0.125)


@pytest.mark.parametrize("hq,n_q,d,code", [(32, 3, 64, "e4m3"), (64, 2, 128, "int8"), (8, 33, 128, "e4m3"), (8, 48, 64, "int8"),
                                           (16, 64, 128, "int8"), (32, 40, 64, "e4m3"), (40, 64, 128, "e4m3"),
                                           (64, 64, 64, "int8")])
def test_long_ranges_of_many_rows(hq, n_q, d, code):
    """Ranges of several units, and of more blocks than any ring holds."""
    rng = np.random.default_rng(16)
    lens = [12000, 6001, n_q, 70, 300, 9999, 4096, 150, 64, 2500]
    c8, h = cache(rng, lens, 8, d, code)
    qn, q = q_of(rng, (len(lens), n_q, hq, d))
    out, st = run(q, c8, 1 / math.sqrt(d), max(lens))
    assert st == 0
    keep = [0, 2, 3, 7, 8] if n_q < 64 else [1, 2, 4]
    check(out[keep], {**h, "lens": [lens[b] for b in keep], "table": h["table"][keep]}, qn[keep], 1 / math.sqrt(d))


def odd_scales(s):
    s[::3] = 0.0
    s[1::7] = np.nan
    s[2::5] *= -1
    return s


@pytest.mark.parametrize("n_q", [1, 40])
@pytest.mark.parametrize("v_scale", [lambda s: np.exp2(np.random.default_rng(1).uniform(-40, 40, s.shape)).astype(np.float32),
                                     lambda s: np.full_like(s, 2.0 ** -126), odd_scales])
def test_scales_of_all_sizes(v_scale, n_q):
    rng = np.random.default_rng(10)
    c8, h = cache(rng, [400, 130], 2, 128, "e4m3", v_scale=v_scale)
    qn, q = q_of(rng, (2, n_q, 8, 128))
    out, st = run(q, c8, 0.05, 400)
    assert st == 0 and torch.isfinite(out).all()
    check(out, h, qn, 0.05)


@pytest.mark.parametrize("n_q", [1, 40])
def test_large_and_small_queries(n_q):
    """Rows of Q from 2^-100 to 2^60, with K's scales to match one of them."""
    rng = np.random.default_rng(11)
    c8, h = cache(rng, [200], 1, 64, "int8", k_scale=lambda s: (s * 2.0 ** -60).astype(np.float32))
    qn, q = q_of(rng, (1, n_q, 4, 64))
    f = torch.tensor([2.0 ** 60, 2.0 ** 61, 2.0 ** -100, 0.0], device="cuda")
    q2 = (q.float() * f[:, None]).to(torch.bfloat16)
    out, st = run(q2, c8, 0.125, 200)
    assert st == 0
    check(out, h, qn * f.cpu().numpy()[:, None].astype(np.float64), 0.125)


@pytest.mark.parametrize("n_q", [1, 3, 40])
def test_refused_and_idle_requests(n_q):
    """Too short, too long for the call or the table, idle, a bad page: zeros and a report; the others as ever."""
    rng = np.random.default_rng(12)
    lens = [100, 0, 300, 90]
    c8, h = cache(rng, lens, 2, 64, "e4m3")
    qn, q = q_of(rng, (4, n_q, 4, 64))
    out, st = run(q, c8, 0.125, 200)
    assert st == 3 and not out[1].any() and not out[2].any()
    check(out, h, qn, 0.125, only=[0, 3])
    out, st = run(q, c8, 0.125, 300)
    assert st == 0
    if n_q > 1:
        c8.seq_lens[0] = n_q - 1
        out, st = run(q, c8, 0.125, 300)
        assert st == 3 and not out[0].any()
        check(out, h, qn, 0.125, only=[2, 3])
        c8.seq_lens[0] = 100
    c8.block_table[3, 2] = c8.num_pages
    out, st = run(q, c8, 0.125, 300)
    assert st == 3
    check(out, h, qn, 0.125, only=[0, 2])


@pytest.mark.parametrize("n_q", [12, 40])
def test_waits_that_run_out(n_q):
    """(Few rows are served without waits on other warps.)"""
    m, rng = vc(), np.random.default_rng(13)
    c8, h = cache(rng, [3000, 40], 2, 128, "int8")
    qn, q = q_of(rng, (2, n_q, 8, 128))
    try:
        m.debug_set_wait_fault(1000000, 1)
        out, st = run(q, c8, 0.1, 3000)
        assert st == 6 and not out.any()
        m.debug_set_wait_fault(1000000, 2)
        out, st = run(q, c8, 0.1, 3000)
        assert st == 6 and not out[0].any()
    finally:
        m.debug_set_wait_fault(0, 0)
    out, st = run(q, c8, 0.1, 3000)
    assert st == 0
    check(out, h, qn, 0.1)


@pytest.mark.parametrize("n_q", [1, 12, 64])
def test_streams_graphs_and_calls_at_once(n_q):
    """Two streams with a workspace each; a graph replayed with other lengths and contents."""
    m, rng = vc(), np.random.default_rng(14)
    a, ha = cache(rng, [900, 77], 2, 64, "e4m3")
    b, hb = cache(rng, [333, 1200, 64], 1, 128, "int8")
    qa, ta = q_of(rng, (2, n_q, 8, 64))
    qb, tb = q_of(rng, (3, n_q, 8, 128))
    oa, ob = torch.zeros(ta.shape, device="cuda"), torch.zeros(tb.shape, device="cuda")
    wa = torch.empty(m.kv8_workspace_bytes(a, n_q, 8, 1000), dtype=torch.uint8, device="cuda")
    wb = torch.empty(m.kv8_workspace_bytes(b, n_q, 8, 1200), dtype=torch.uint8, device="cuda")
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        m.kv8_attn(ta, a, 0.125, oa, 1000, wa, stream=s1)
        m.kv8_attn(tb, b, 0.1, ob, 1200, wb, stream=s2)
    torch.cuda.synchronize()
    check(oa, ha, qa, 0.125)
    check(ob, hb, qb, 0.1)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.kv8_attn(ta, a, 0.125, oa, 1000, wa)
    lens = [max(n_q, 450), 70]
    a.seq_lens.copy_(i32(lens))
    ha["lens"] = lens
    oa.zero_()
    # (the last page now ends inside: what lies behind is junk like any other)
    g.replay()
    torch.cuda.synchronize()
    check(oa, ha, qa, 0.125)


def test_quantised_attention_is_near_the_full_one():
    """Written from KV_full and read back, against the bf16 cache's attention.

    A code is off by half a step: scale / 2 (int8), 2^-4 of the value or 2^-10
    scale (e4m3); the scale follows the block.  A score is then off by at most
    e = scale sum |q_c| dk_c, so every p by a factor within exp(+-2e) (numerator
    and denominator), and the result by (exp(2e) - 1) sum p (|v| + dv) + sum p dv,
    beside the kernel's own error."""
    m, rng = vc(), np.random.default_rng(15)
    lens, sm = [777, 130], 1 / math.sqrt(128)
    full, hf = H.full_cache(rng, lens, 2, 128, [5], 6.0)
    qn, q = q_of(rng, (2, 1, 8, 128))
    for code in CODES:
        c8 = m.PagedKV8.allocate(full.num_pages, 2, 128, CODES[code], full.block_table, full.seq_lens)
        m.kv8_write(full, None, c8, 777)
        out, st = run(q, c8, sm, 777)
        assert st == 0
        for b in range(2):
            pages = hf["table"][b, :-(-lens[b] // 16)]
            kv = [synth.bf16_to_f32(x).astype(np.float64) for x in H.logical_full(hf, b)]
            off = []
            for x, s in zip(kv, (c8.k_scales, c8.v_scales)):
                s = np.repeat(s.double().cpu().numpy()[pages], 16, 0)[:lens[b], :, None]
                off.append(s * 0.5 * (1 + 2.0 ** -20) if code == "int8" else np.maximum(np.abs(x) * 2.0 ** -4, s * 2.0 ** -10) * (1 + 2.0 ** -20))
            for head in range(8):
                g = head // 4
                (k, v), (dk, dv) = (x[:, g] for x in kv), (x[:, g] * np.ones((1, 128)) for x in off)
                seen = np.ones((1, lens[b]), bool)
                qh = qn[b, :, head]
                ref, own = K.attn(qh, k, v, seen, sm, 1.0)
                e = sm * float((np.abs(qh) @ dk.T).max())
                p = np.exp(sm * (k @ qh[0]))
                p /= p.sum()
                most = math.expm1(2 * e) * (p @ (np.abs(v) + dv)) + p @ dv
                err = np.abs(out[b, :, head].double().cpu().numpy() - ref)
                assert (err <= most + 2 * own).all()
                assert err.max() < np.abs(v).max()
