"""Refusals of the tree-drafting entry points: on the host, before any CUDA
work (these paths return before touching a device)."""
import ctypes as C

import pytest
import torch

FAKE = C.c_void_p(1 << 20)   # never dereferenced


@pytest.fixture(scope="module")
def vc():
    import __graft_entry__
    __graft_entry__._builder().build()
    import lossless_compressed_kv_gb300 as m
    return m


def cache(vc, d=128, bits=16, batch=1, hkv=2, k=1 << 20, v=1 << 21):
    return vc.PagedKVStruct(k, v, 4, FAKE.value, FAKE.value, batch, 1, vc.KVFormat(hkv, d, bits))


def rot(vc, **kw):
    return vc.Rotary(**{**dict(theta=10000.0, rot_dim=128), **kw}).struct()


def rotary_call(vc, r, c, dtype=0, m=1, stride=6 * 128, hq=2, qkv=FAKE):
    return vc.STATUS[vc.library().vc_rotary_kv_write(qkv, dtype, stride, m, FAKE, FAKE, None, hq, C.byref(r),
                                                     FAKE, C.byref(c), None, None)]


@pytest.mark.parametrize("bad", [dict(theta=0.5), dict(theta=float("nan")), dict(theta=float("inf")), dict(rot_dim=3),
                                 dict(rot_dim=-2), dict(rot_dim=130), dict(factor=0.5), dict(factor=float("nan")),
                                 dict(original_len=-1), dict(amplitude=float("inf")),
                                 dict(factor=2.0, original_len=10, low_turns=4.0, high_turns=4.0),
                                 dict(factor=2.0, original_len=10, low_turns=float("nan"), high_turns=4.0)])
def test_rotary_refuses_parameters(vc, bad):
    assert rotary_call(vc, rot(vc, **bad), cache(vc)) == "VC_ERR_INVALID_ARG"


def test_rotary_refuses_arguments(vc):
    r = rot(vc)
    assert rotary_call(vc, r, cache(vc), stride=6 * 128 - 1) == "VC_ERR_INVALID_ARG"
    assert rotary_call(vc, r, cache(vc), m=-1) == "VC_ERR_INVALID_ARG"
    assert rotary_call(vc, r, cache(vc), hq=0) == "VC_ERR_INVALID_ARG"
    assert rotary_call(vc, r, cache(vc), qkv=None) == "VC_ERR_INVALID_ARG"
    assert rotary_call(vc, r, cache(vc, bits=4)) == "VC_ERR_UNSUPPORTED"
    assert rotary_call(vc, r, cache(vc), dtype=2) == "VC_ERR_UNSUPPORTED"
    assert rotary_call(vc, r, cache(vc), m=0) == "VC_OK"
    assert rotary_call(vc, r, cache(vc, batch=0)) == "VC_OK"


def test_tree_calls_refuse_arguments(vc):
    L, S = vc.library(), vc.STATUS
    assert S[L.vc_tree_plan(FAKE, 1, 0, FAKE, FAKE, FAKE, None, None)] == "VC_ERR_INVALID_ARG"
    assert S[L.vc_tree_plan(FAKE, 1, 65, FAKE, FAKE, FAKE, None, None)] == "VC_ERR_UNSUPPORTED"
    assert S[L.vc_tree_plan(None, 1, 4, FAKE, FAKE, FAKE, None, None)] == "VC_ERR_INVALID_ARG"
    assert S[L.vc_tree_plan(None, 0, 4, None, None, None, None, None)] == "VC_OK"
    assert S[L.vc_tree_accept(FAKE, FAKE, FAKE, -1, 4, FAKE, FAKE, FAKE, None)] == "VC_ERR_INVALID_ARG"
    assert S[L.vc_tree_accept(FAKE, FAKE, FAKE, 1, 65, FAKE, FAKE, FAKE, None)] == "VC_ERR_UNSUPPORTED"
    assert S[L.vc_tree_accept(FAKE, FAKE, None, 1, 4, FAKE, FAKE, FAKE, None)] == "VC_ERR_INVALID_ARG"
    assert S[L.vc_tree_accept(None, None, None, 0, 4, None, None, None, None)] == "VC_OK"

    def attn(c, n_q=4, hq=4, scale=1.0, dtype=1, q=FAKE, ws=FAKE, nbytes=1 << 40):
        return S[L.vc_tree_attn(q, n_q, hq, C.byref(c), FAKE, scale, FAKE, dtype, 64, ws, nbytes, None, None)]

    assert attn(cache(vc), n_q=65) == "VC_ERR_UNSUPPORTED"
    assert attn(cache(vc), hq=5) == "VC_ERR_UNSUPPORTED"
    assert attn(cache(vc), hq=18) == "VC_ERR_UNSUPPORTED"
    assert attn(cache(vc, d=96)) == "VC_ERR_UNSUPPORTED"
    assert attn(cache(vc, bits=4)) == "VC_ERR_UNSUPPORTED"
    assert attn(cache(vc), dtype=2) == "VC_ERR_UNSUPPORTED"
    assert attn(cache(vc), n_q=0) == "VC_ERR_INVALID_ARG"
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert attn(cache(vc), scale=scale) == "VC_ERR_INVALID_ARG"
    assert attn(cache(vc), q=None) == "VC_ERR_INVALID_ARG"
    assert attn(cache(vc), q=C.c_void_p((1 << 20) + 8)) == "VC_ERR_INVALID_ARG"
    assert attn(cache(vc, k=(1 << 20) + 8)) == "VC_ERR_INVALID_ARG"
    assert attn(cache(vc), ws=None) == "VC_ERR_WORKSPACE"
    assert attn(cache(vc), nbytes=0) == "VC_ERR_WORKSPACE"
    assert attn(cache(vc, batch=0), q=None) == "VC_OK"
    c = cache(vc)
    assert L.vc_tree_workspace_bytes(C.byref(c), 4, 4, 64) > 0
    assert L.vc_tree_workspace_bytes(C.byref(c), 65, 4, 64) == 0
    assert L.vc_tree_workspace_bytes(C.byref(c), 4, 4, -1) == 0


def test_commit_refuses_arguments(vc):
    L, S = vc.library(), vc.STATUS

    def commit(*caches, n_q=4, lens=FAKE):
        arr = (vc.PagedKVStruct * max(1, len(caches)))(*caches)
        return S[L.vc_tree_commit(arr, len(caches), n_q, lens, FAKE, None, None)]

    a, b = cache(vc), cache(vc, k=1 << 22, v=1 << 23)
    assert commit() == "VC_OK"
    assert commit(cache(vc, batch=0), lens=None) == "VC_OK"
    assert commit(a, n_q=0) == "VC_ERR_INVALID_ARG"
    assert commit(a, n_q=65) == "VC_ERR_UNSUPPORTED"
    assert commit(cache(vc, bits=4)) == "VC_ERR_UNSUPPORTED"
    assert commit(a, lens=None) == "VC_ERR_INVALID_ARG"
    assert commit(a, a) == "VC_ERR_INVALID_ARG"                                       # the same pools twice
    assert commit(a, cache(vc, k=1 << 22, v=1 << 20)) == "VC_ERR_INVALID_ARG"         # a pool of the other kind
    assert commit(cache(vc, k=1 << 20, v=1 << 20)) == "VC_ERR_INVALID_ARG"
    assert commit(a, cache(vc, d=64, k=1 << 22, v=1 << 23)) == "VC_ERR_INVALID_ARG"
    assert commit(a, cache(vc, batch=2, k=1 << 22, v=1 << 23)) == "VC_ERR_INVALID_ARG"
    b.block_table = FAKE.value + 64
    assert commit(a, b) == "VC_ERR_INVALID_ARG"
    assert commit(cache(vc, k=(1 << 20) + 2)) == "VC_ERR_INVALID_ARG"


def test_logprobs_refuse_arguments(vc):
    L, S = vc.library(), vc.STATUS

    def call(x=FAKE, dtype=0, rows=2, vocab=10, stride=10, ids=FAKE, n_ids=1, tau=1.0, k=2, lp=FAKE, ti=FAKE, tl=FAKE,
             ws=FAKE, nbytes=1 << 40):
        return S[L.vc_token_logprobs(x, dtype, rows, vocab, stride, ids, n_ids, tau, k, lp, None, ti, tl, ws, nbytes,
                                     None, None)]

    for bad in (dict(rows=-1), dict(vocab=0), dict(stride=9), dict(n_ids=-1), dict(tau=0.0), dict(tau=-1.0),
                dict(tau=float("nan")), dict(tau=float("inf")), dict(k=-1), dict(x=None), dict(ids=None),
                dict(lp=None), dict(ti=None), dict(tl=None)):
        assert call(**bad) == "VC_ERR_INVALID_ARG", bad
    assert call(vocab=(1 << 22) + 1, stride=1 << 23) == "VC_ERR_UNSUPPORTED"
    assert call(dtype=3) == "VC_ERR_UNSUPPORTED" and call(k=65) == "VC_ERR_UNSUPPORTED"
    assert call(ws=None) == "VC_ERR_WORKSPACE" and call(nbytes=0) == "VC_ERR_WORKSPACE"
    assert call(rows=0, x=None, ids=None, lp=None, ws=None) == "VC_OK"
    assert L.vc_token_logprobs_workspace_bytes(2, 10, 65) == 0
    assert L.vc_token_logprobs_workspace_bytes(-1, 10, 1) == 0


def test_wrappers_refuse_tensors(vc):
    """Types, shapes, strides and devices (here: none but the CPU)."""
    i = torch.zeros((2, 4), dtype=torch.int32)
    m = torch.zeros((2, 4), dtype=torch.int64)
    one = torch.zeros(2, dtype=torch.int32)
    for args in ((i, one, m, i), (i.float(), one, m, i), (i, one[:1], m, i), (i, one, i, i), (i.T, one, m, i)):
        with pytest.raises(ValueError):
            vc.tree_plan(*args)
    with pytest.raises(ValueError):
        vc.tree_accept(i, i, i, one, i, i[:1])
    with pytest.raises(ValueError, match="CUDA device"):
        vc.token_logprobs(torch.zeros((2, 8)), i, torch.zeros((2, 4)), torch.zeros(8, dtype=torch.uint8))
    with pytest.raises(ValueError, match="contiguous"):
        vc.token_logprobs(torch.zeros((8, 2)).T, i, torch.zeros((2, 4)), torch.zeros(8, dtype=torch.uint8))
    kv = vc.PagedKV(torch.zeros((2, 4096), dtype=torch.uint8), torch.zeros((2, 4096), dtype=torch.uint8),
                    torch.zeros((2, 1), dtype=torch.int32), one, 1, 128, 16)
    with pytest.raises(ValueError):
        vc.KVLayers([kv])
    with pytest.raises(ValueError):
        vc.rotary_kv_write(torch.zeros((2, 384)), one, one, 2, vc.Rotary(1e4, 128), torch.zeros((2, 2, 128)), kv)
    with pytest.raises(ValueError):
        vc.tree_attn(torch.zeros((2, 4, 1, 128), dtype=torch.bfloat16), kv, m, 1.0, torch.zeros((2, 4, 1, 128)), 16,
                     torch.zeros(8, dtype=torch.uint8))


def test_refusals_at_the_ends_of_the_ranges(vc):
    """Addresses off their type's boundary, blocks that 32 bits do not count,
    scales and temperatures whose base-2 form is not finite."""
    L, S = vc.library(), vc.STATUS
    odd = C.c_void_p((1 << 20) + 1)
    assert rotary_call(vc, rot(vc), cache(vc), qkv=odd) == "VC_ERR_INVALID_ARG"
    assert rotary_call(vc, rot(vc), cache(vc), dtype=1, qkv=odd) == "VC_ERR_INVALID_ARG"
    assert rotary_call(vc, rot(vc), cache(vc, k=(1 << 20) + 1)) == "VC_ERR_INVALID_ARG"
    assert rotary_call(vc, rot(vc), cache(vc), hq=1 << 22, stride=1 << 40) == "VC_ERR_UNSUPPORTED"

    def attn(scale, batch=1, blocks=1, longest=64):
        c = cache(vc, batch=batch)
        c.max_blocks = blocks
        return S[L.vc_tree_attn(FAKE, 4, 4, C.byref(c), FAKE, scale, FAKE, 1, longest, FAKE, 0, None, None)]

    assert attn(3e38) == "VC_ERR_UNSUPPORTED"
    assert attn(1.0, 1 << 20, 1 << 20, 2 ** 31 - 1) == "VC_ERR_UNSUPPORTED"
    assert attn(1.0, 1 << 20, 1 << 20, 64) == "VC_ERR_WORKSPACE"         # counted by what can be reached
    assert attn(1.0, 1, 1, 2 ** 31 - 1) == "VC_ERR_WORKSPACE"

    def lp(dtype, tau, logits=FAKE):
        return S[L.vc_token_logprobs(logits, dtype, 1, 8, 8, None, 0, tau, 0, None, None, None, None, FAKE, 0, None,
                                     None)]

    assert lp(0, 1e-39) == "VC_ERR_UNSUPPORTED"
    assert lp(0, 1.0) == "VC_ERR_WORKSPACE"
    for dtype in (0, 1, 2):
        assert lp(dtype, 1.0, odd) == "VC_ERR_INVALID_ARG"
    assert lp(0, 1.0, C.c_void_p((1 << 20) + 2)) == "VC_ERR_INVALID_ARG"


def test_wrappers_refuse_halves(vc):
    x, i = torch.zeros((2, 8)), torch.zeros((2, 1), dtype=torch.int32)
    with pytest.raises(ValueError, match="come together"):
        vc.token_logprobs(x, i, x[:, :1], x, top_ids=i)
    with pytest.raises(ValueError, match="come together"):
        vc.token_logprobs(x, i, x[:, :1], x, top_logprobs=x[:, :1])


def test_wrappers_refuse_workspaces_of_fewer_bytes_than_they_count(vc, monkeypatch):
    """A broadcast workspace has one element's memory, whatever its shape says."""
    monkeypatch.setattr(vc, "_device", lambda: -1)          # where CPU tensors are
    monkeypatch.setattr(vc, "_on", lambda stream, dev: None)
    class NotReached:
        def __getattr__(self, name):
            return lambda *a: pytest.fail(name)

    monkeypatch.setattr(vc, "_lib", NotReached())
    wide = torch.zeros(1, dtype=torch.uint8).expand(1 << 40)
    one, m = torch.zeros(2, dtype=torch.int32), torch.zeros((2, 4), dtype=torch.int64)
    kv = vc.PagedKV(torch.zeros((2, 4096), dtype=torch.uint8), torch.zeros((2, 4096), dtype=torch.uint8),
                    torch.zeros((2, 1), dtype=torch.int32), one, 1, 128, 16)
    q = torch.zeros((2, 4, 1, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="workspace"):
        vc.tree_attn(q, kv, m, 1.0, torch.zeros_like(q), 16, wide)
    with pytest.raises(ValueError, match="workspace"):
        vc.token_logprobs(torch.zeros((2, 8)), one.view(2, 1), torch.zeros((2, 1)), wide)
