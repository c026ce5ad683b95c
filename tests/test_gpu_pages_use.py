"""The 8-bit cache and the pages together, as a server uses them: prompts
written to KV_full and quantised, samples forked from them, new tokens drafted
over the 8-bit cache and verified in a block, requests that end, and the pool
compacted under those that go on."""
import math

import numpy as np
import pytest
import torch

from oracle import kv8 as K
from tests import vc_harness as H

pytestmark = pytest.mark.gpu
HQ, HKV, D, LAYERS, POOL = 8, 2, 64, 2, 96
SCALE = 1 / math.sqrt(D)


def vc():
    import lossless_compressed_kv_gb300 as m
    return m


def i32(x):
    return H.to_dev(np.array(x, dtype=np.int32))


class Server:
    """Rows of a batch over one page map; the tokens' K and V also kept as plain lists."""

    def __init__(self, rows, code):
        m = vc()
        self.rng, self.st = np.random.default_rng(21), torch.zeros(1, dtype=torch.int32, device="cuda")
        self.map = m.PageMap.allocate(POOL, rows, 24)
        self.lens = i32([0] * rows)
        self.full = [m.PagedKV.allocate(POOL, HKV, D, 16, self.map.table, self.lens, zero=True) for _ in range(LAYERS)]
        self.kv8 = [m.PagedKV8.allocate(POOL, HKV, D, code, self.map.table, self.lens) for _ in range(LAYERS)]
        self.arrays = m.PageArrays([t for f, c in zip(self.full, self.kv8) for t in
                                    (f.k_pages, f.v_pages, c.k_codes, c.v_codes, c.k_scales, c.v_scales)])
        self.ws = torch.empty(m.pages_workspace_bytes(self.map), dtype=torch.uint8, device="cuda")
        self.granted, self.src, self.dst = (i32([0] * rows) for _ in range(3))
        self.rotary = m.Rotary(theta=10000.0, rot_dim=0)     # (nothing is turned: K stays as it was given)
        self.code = "int8" if code is torch.int8 else "e4m3"
        self.kept = [[] for _ in range(rows)]                # per row: tokens' (k, v) of every layer, bf16 values

    def append(self, counts):
        """counts[b] new tokens for each row, in one pass: pages first, then K and V, then the 8-bit pages."""
        m = vc()
        first = self.lens.clone()
        want = self.lens + i32(counts)
        m.pages_reserve(self.map, self.lens, want, self.granted, self.src, self.dst, self.ws, status=self.st)
        m.pages_copy(self.arrays, self.src, self.dst, status=self.st)
        assert self.granted.all()
        n, before = sum(counts), first.tolist()
        req = i32([b for b, c in enumerate(counts) for _ in range(c)])
        pos = i32([before[b] + i for b, c in enumerate(counts) for i in range(c)])
        qkv = torch.from_numpy(self.rng.standard_normal((LAYERS, n, (HQ + 2 * HKV) * D), dtype=np.float32)).to(torch.bfloat16).cuda()
        q = torch.empty((n, HQ, D), dtype=torch.bfloat16, device="cuda")
        self.lens.copy_(want)
        for x, f, c in zip(qkv, self.full, self.kv8):
            m.rotary_kv_write(x, req, pos, HQ, self.rotary, q, f, status=self.st)
            m.kv8_write(f, first, c, 24 * 16, status=self.st)
        kv = qkv.float().view(LAYERS, n, HQ + 2 * HKV, D)[:, :, HQ:].cpu().numpy()
        at = 0
        for b, c in enumerate(counts):
            self.kept[b] = self.kept[b] + [kv[:, at + i] for i in range(c)]
            at += c

    def attend(self, n_q):
        """Queries of the last n_q tokens of every row, each layer: (values, results)."""
        m, rows = vc(), len(self.kept)
        out = []
        for c in self.kv8:
            q = torch.from_numpy(self.rng.standard_normal((rows, n_q, HQ, D), dtype=np.float32)).to(torch.bfloat16).cuda()
            o = torch.empty(q.shape, dtype=torch.float32, device="cuda")
            ws = torch.empty(m.kv8_workspace_bytes(c, n_q, HQ, 24 * 16), dtype=torch.uint8, device="cuda")
            m.kv8_attn(q, c, SCALE, o, 24 * 16, ws, status=self.st)
            out.append((q, o))
        return out

    def check(self, n_q, res):
        torch.cuda.synchronize()
        assert self.st.item() == 0
        for layer, (q, o) in enumerate(res):
            q, o = q.double().cpu().numpy(), o.double().cpu().numpy()
            for b, kept in enumerate(self.kept):
                n = len(kept)
                if n == 0:
                    assert not o[b].any()
                    continue
                kv = np.stack([t[layer] for t in kept])       # [n][2 HKV][D]
                pad = np.zeros((-(-n // 16) * 16, 2 * HKV, D), np.float32)
                pad[:n] = kv
                seen = np.tril(np.ones((n, n), bool))[n - n_q:]
                for h in range(HKV):
                    vals, top = [], 0.0
                    for x in (h, HKV + h):
                        blocks = [K.block(pad[i:i + 16, x], self.code) for i in range(0, len(pad), 16)]
                        vals.append(np.concatenate([K.decode(c, self.code) * np.float64(s) for c, s, _ in blocks])[:n])
                        top = max(float(s) for _, s, _ in blocks) * float(K.TOP[self.code])
                    for head in range(h * HQ // HKV, (h + 1) * HQ // HKV):
                        ref, tol = K.attn(q[b, :, head], *vals, seen, SCALE, top)
                        assert (np.abs(o[b, :, head] - ref) <= tol + 1e-6 * np.abs(ref)).all(), (layer, b, head)


@pytest.mark.parametrize("code", [torch.float8_e4m3fn, torch.int8])
def test_a_server(code):
    m = vc()
    s = Server(7, code)
    s.append([70, 33, 0, 0, 0, 0, 0])                        # two prompts
    m.pages_fork(s.map, s.lens, i32([0, 0, 1]), i32([2, 3, 4]), status=s.st)
    for b, p in ((2, 0), (3, 0), (4, 1)):
        s.kept[b] = list(s.kept[p])
    assert s.map.refs.max().item() == 3
    for step in range(3):                                    # drafting: the forks part from their prompts
        s.append([1, 1, 1, 1, 1, 0, 0])
        s.check(1, s.attend(1))
    s.append([17, 5, 6, 20, 9, 0, 0])                        # a block of five at the end of each
    s.lens[5:] = 0
    s.check(5, s.attend(5))
    used = int((s.map.refs > 0).sum())
    m.pages_free(s.map, i32([0, -1, 0, -1, -1, -1, -1]), status=s.st)   # two requests end
    s.lens[0], s.lens[2] = 0, 0
    s.kept[0], s.kept[2] = [], []
    rng_state = s.rng.bit_generator.state
    before = s.attend(5)
    s.check(5, before)
    moves, remap = i32([0]), i32([0] * POOL)
    src, dst = i32([0] * (POOL // 2)), i32([0] * (POOL // 2))
    m.pages_compact(s.map, src, dst, moves, remap, s.ws, status=s.st)
    m.pages_copy(s.arrays, src, dst, count=moves, status=s.st)
    live = int((s.map.refs > 0).sum())
    assert 0 < live < used and (s.map.refs[:live] > 0).all() and not (s.map.refs[live:] > 0).any()
    s.rng.bit_generator.state = rng_state
    after = s.attend(5)
    s.check(5, after)
    for (_, a), (_, b) in zip(before, after):                # the same bits: results follow from lengths and contents
        assert torch.equal(a, b)
    s.append([0, 40, 0, 1, 12, 30, 0])                       # those that go on, and a new one
    s.check(1, s.attend(1))
