"""GPU vc_rotary_kv_write against the 64-bit definition.

Tolerance per value of a rotated pair (a, b): the result is rounded once to
bf16 (half a step: 2^-8 of the value); before that the angle is off by at most
2 roundings of a number up to pi (2 * 2^-24 * pi), the fast sine and cosine by
2^-21 in [-pi, pi], and the two products and their sum by 3 * 2^-24: together
below 2^-19 (|a| + |b|) amplitude."""
import math

import numpy as np
import pytest
import torch

from oracle import tree as T
from tests import vc_harness as H

pytestmark = pytest.mark.gpu


def vc():
    import lossless_compressed_kv_gb300 as m
    return m


def run(rng, dtype, hq, hkv, d, params, reqs, pos, slot, batch, max_blocks, strided=0, misalign=0):
    m, nh = len(reqs), hq + 2 * hkv
    pages = batch * max_blocks + 3
    table = rng.permutation(pages)[:batch * max_blocks].reshape(batch, max_blocks).astype(np.int32)
    wide = torch.from_numpy(rng.standard_normal((m, nh * d + strided + misalign)).astype(np.float32)).to(dtype).cuda()
    qkv = wide[:, misalign:misalign + nh * d]
    before = torch.full((pages, hkv * 16 * d), 7.0, dtype=torch.bfloat16, device="cuda")
    k, v = before.clone(), before.clone()
    kv = vc().PagedKV(k.view(torch.uint8), v.view(torch.uint8), H.to_dev(table),
                      torch.zeros(batch, dtype=torch.int32, device="cuda"), hkv, d, 16)
    q = torch.full((m, hq, d), 5.0, dtype=torch.bfloat16, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    vc().rotary_kv_write(qkv, H.to_dev(np.array(reqs, np.int32)), H.to_dev(np.array(pos, np.int32)), hq,
                         vc().Rotary(**params), q, kv,
                         row_slot=None if slot is None else H.to_dev(np.array(slot, np.int32)), status=st)
    torch.cuda.synchronize()
    x = qkv.double().cpu().numpy().reshape(m, nh, d)
    kp, vp = (t.double().cpu().numpy().reshape(pages, hkv, 16, d) for t in (k, v))
    return x, q.double().cpu().numpy(), kp, vp, table, int(st.item())


def check(x, q, kp, vp, table, hq, hkv, params, reqs, pos, slot, skipped=()):
    fr = {k: params[k] for k in ("theta", "rot_dim", "factor", "original_len", "low_turns", "high_turns") if k in params}
    f = T.rotary_frequencies(**fr) if params["rot_dim"] else np.zeros(0)
    inter, amp = params.get("interleaved", False), params.get("amplitude", 1.0)
    n = len(f)
    want = T.rotary(x[:, :hq + hkv], pos, f, inter, amp)
    pair = np.zeros_like(want)
    i0 = np.arange(n) * 2 if inter else np.arange(n)
    i1 = i0 + 1 if inter else i0 + n
    both = np.abs(x[:, :hq + hkv][..., i0]) + np.abs(x[:, :hq + hkv][..., i1])
    pair[..., i0] = pair[..., i1] = both * abs(amp)
    tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -19 * pair
    wrote_k, wrote_v = np.full_like(kp, 7.0), np.full_like(vp, 7.0)
    for r, b in enumerate(reqs):
        if b == -1 or r in skipped:
            assert (q[r] == 5.0).all()
            continue
        s = (pos if slot is None else slot)[r]
        pg, at = table[b, s // 16], s % 16
        assert (np.abs(q[r] - want[r, :hq]) <= tol[r, :hq]).all(), r
        assert (np.abs(kp[pg, :, at] - want[r, hq:]) <= tol[r, hq:]).all(), r
        # V is rounded to bf16 and nothing else
        assert (np.abs(vp[pg, :, at] - x[r, hq + hkv:]) <= 2.0 ** -8 * np.abs(x[r, hq + hkv:])).all(), r
        wrote_k[pg, :, at], wrote_v[pg, :, at] = kp[pg, :, at], vp[pg, :, at]
    assert (wrote_k == kp).all() and (wrote_v == vp).all()      # nothing else was written


SCALED = dict(theta=500000.0, factor=8.0, original_len=8192, low_turns=1.0, high_turns=4.0, amplitude=1.25)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("hq,hkv,d", [(4, 1, 64), (32, 8, 128), (7, 1, 32), (3, 3, 96), (8, 2, 256)])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot", ["all", "half", "two", "odd", "none"])
def test_layouts_and_parts(dtype, hq, hkv, d, inter, rot):
    rng = np.random.default_rng([hq, d, inter, len(rot)])
    r = dict(all=d, half=d // 2, two=2, odd=d // 2 + 6, none=0)[rot]
    params = dict(theta=10000.0, rot_dim=r, interleaved=inter)
    reqs, slot = [0, 0, 1, -1, 2, 1], [0, 1, 15, 0, 33, 16]
    pos = [0, 1, 7, -5, 4000, 7]
    got = run(rng, dtype, hq, hkv, d, params, reqs, pos, slot, 3, 3)
    assert got[-1] == 0
    check(*got[:-1], hq, hkv, params, reqs, pos, slot)


@pytest.mark.parametrize("scaling", [{}, dict(factor=4.0), {k: v for k, v in SCALED.items() if k != "theta"}])
@pytest.mark.parametrize("theta", [1.0, 10000.0, 500000.0])
def test_far_positions(scaling, theta):
    """Angles stay exact at positions where a 32-bit product would be off."""
    rng = np.random.default_rng(5)
    params = dict(theta=theta, rot_dim=128, **scaling)
    pos = [0, 1, 4095, 32768, 131071, 1 << 20, (1 << 22) - 1]
    slot = list(range(len(pos)))
    got = run(rng, torch.float32, 2, 1, 128, params, [0] * len(pos), pos, slot, 1, 1)
    check(*got[:-1], 2, 1, params, [0] * len(pos), pos, slot)


@pytest.mark.parametrize("dtype,strided,misalign", [(torch.float32, 5, 0), (torch.float32, 0, 1), (torch.float32, 4, 4),
                                                    (torch.bfloat16, 3, 0), (torch.bfloat16, 0, 1),
                                                    (torch.bfloat16, 8, 8)])
def test_strided_and_misaligned_rows(dtype, strided, misalign):
    rng = np.random.default_rng(6)
    params = dict(theta=10000.0, rot_dim=64, **{k: v for k, v in SCALED.items() if k != "theta"})
    reqs, pos = [0] * 9, list(range(9))
    got = run(rng, dtype, 4, 2, 64, params, reqs, pos, None, 1, 1, strided, misalign)
    check(*got[:-1], 4, 2, params, reqs, pos, None)


@pytest.mark.parametrize("m", [1, 3, 129, 1000])
def test_many_rows_slot_is_position(m):
    rng = np.random.default_rng(m)
    params = dict(theta=500000.0, rot_dim=128)
    reqs = [i % 3 for i in range(m)]
    pos = [i // 3 for i in range(m)]
    got = run(rng, torch.float32, 8, 2, 128, params, reqs, pos, None, 3, 64)
    assert got[-1] == 0
    check(*got[:-1], 8, 2, params, reqs, pos, None)


def test_bad_rows_are_skipped_and_reported():
    rng = np.random.default_rng(8)
    params = dict(theta=10000.0, rot_dim=64)
    reqs, pos, slot = [0, 3, -2, 0, 0, 0, 1], [3, 0, 0, -1, 2, 2, 2], [0, 0, 0, 1, 48, -1, 2]
    got = run(rng, torch.float32, 2, 1, 64, params, reqs, pos, slot, 3, 3)
    assert got[-1] == 3
    check(*got[:-1], 2, 1, params, reqs, [max(p, 0) for p in pos], slot, skipped=(1, 2, 3, 4, 5))


def test_non_finite_values_stay_in_their_row():
    rng = np.random.default_rng(9)
    qkv = torch.randn((3, 3 * 64), device="cuda")
    qkv[1] = float("nan")
    kv = vc().PagedKV.allocate(1, 1, 64, 16, torch.zeros((1, 1), dtype=torch.int32, device="cuda"),
                               torch.zeros(1, dtype=torch.int32, device="cuda"), zero=True)
    q = torch.zeros((3, 1, 64), dtype=torch.bfloat16, device="cuda")
    i = torch.arange(3, dtype=torch.int32, device="cuda")
    vc().rotary_kv_write(qkv, torch.zeros_like(i), i, 1, vc().Rotary(1e4, 64), q, kv)
    k = kv.k_pages.view(torch.bfloat16).view(16, 64)
    assert q[1].isnan().all() and k[1].isnan().all()
    assert q[[0, 2]].isfinite().all() and k[[0, 2]].isfinite().all() and (k[3:] == 0).all()


def test_captured_and_replayed():
    """The call in a graph follows its position and slot buffers."""
    torch.manual_seed(0)
    qkv = torch.randn((4, 6 * 128), device="cuda")
    kv = vc().PagedKV.allocate(8, 2, 128, 16, torch.arange(8, dtype=torch.int32, device="cuda").view(4, 2),
                               torch.zeros(4, dtype=torch.int32, device="cuda"), zero=True)
    req = torch.arange(4, dtype=torch.int32, device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    q, q2 = (torch.zeros((4, 2, 128), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    r = vc().Rotary(1e4, 128, interleaved=True)
    vc().rotary_kv_write(qkv, req, pos, 2, r, q, kv)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        vc().rotary_kv_write(qkv, req, pos, 2, r, q, kv)
    pos.copy_(torch.tensor([3, 17, 5, 30]))
    g.replay()
    kv2 = vc().PagedKV.allocate(8, 2, 128, 16, kv.block_table, kv.seq_lens, zero=True)
    vc().rotary_kv_write(qkv, req, pos, 2, r, q2, kv2)
    torch.cuda.synchronize()
    assert torch.equal(q, q2)
    a, b = (t.k_pages.view(torch.bfloat16).view(8, 2, 16, 128) for t in (kv, kv2))
    for i, p in enumerate([3, 17, 5, 30]):
        assert torch.equal(a[2 * i + p // 16, :, p % 16], b[2 * i + p // 16, :, p % 16])


def test_agrees_with_rope_kv_write_near_the_start():
    """Where vc_rope_kv_write's fp32 angles are good (small positions) both agree to a bf16 step."""
    torch.manual_seed(1)
    m, hq, hkv, d = 64, 8, 2, 128
    qkv = torch.randn((m, (hq + 2 * hkv) * d), device="cuda")
    req, pos = torch.zeros(m, dtype=torch.int32, device="cuda"), torch.arange(m, dtype=torch.int32, device="cuda")
    out = []
    for f in ("rope", "rotary"):
        kv = vc().PagedKV.allocate(4, hkv, d, 16, torch.arange(4, dtype=torch.int32, device="cuda")[None],
                                   torch.zeros(1, dtype=torch.int32, device="cuda"), zero=True)
        q = torch.zeros((m, hq, d), dtype=torch.bfloat16, device="cuda")
        if f == "rope":
            vc().rope_kv_write(qkv, req, pos, hq, 500000.0, q, kv)
        else:
            vc().rotary_kv_write(qkv, req, pos, hq, vc().Rotary(500000.0, d), q, kv)
        out.append((q.float(), kv.k_pages.view(torch.bfloat16).float(), kv.v_pages.clone()))
    # one bf16 step (2^-7) of the value, and the angle's fp32 error (64 * 2^-23 radians) times |a| + |b| < 12
    for a, b in zip(out[0][:2], out[1][:2]):
        assert ((a - b).abs() <= 2.0 ** -7 * b.abs() + 12 * 64 * 2.0 ** -23).all()
    assert torch.equal(out[0][2], out[1][2])


@pytest.mark.parametrize("factor", [1.0, 1.5, 8.0])
def test_the_angle_is_as_exact_as_stated(factor):
    """Where a sine or cosine is next to zero bf16 has digits to spare.  Off by
    at most 2^-21 (angle) + 2^-21 (sine, cosine) + half a bf16 step; the far
    positions' share (2^22 2^-55 turns) and the product with 1 add below 2^-28."""
    pos = np.arange(1 << 22)
    t = pos / factor
    near = np.concatenate([np.argsort(np.abs(f(t)))[:400] for f in (np.sin, np.cos)] + [pos[-100:]])
    p = H.to_dev(near.astype(np.int32))
    n = len(near)
    qkv = torch.zeros((n, 3 * 32), device="cuda")
    qkv[:, 0] = 1.0
    kv = vc().PagedKV.allocate(n // 16 + 1, 1, 32, 16, torch.arange(n // 16 + 1, dtype=torch.int32, device="cuda")[None],
                               torch.zeros(1, dtype=torch.int32, device="cuda"), zero=True)
    q = torch.zeros((n, 1, 32), dtype=torch.bfloat16, device="cuda")
    vc().rotary_kv_write(qkv, torch.zeros_like(p), p, 1, vc().Rotary(1e4, 2, factor=factor), q, kv,
                         row_slot=torch.arange(n, dtype=torch.int32, device="cuda"))
    got = q[:, 0, :2].double().cpu().numpy()
    want = np.stack([np.cos(t[near]), np.sin(t[near])], 1)
    assert (np.abs(got - want) <= 2.0 ** -20 + 2.0 ** -28 + 2.0 ** -8 * np.abs(want)).all()
