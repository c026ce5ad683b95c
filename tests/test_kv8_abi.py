"""Refusals of the 8-bit cache's and the pages' entry points: on the host,
before any CUDA work (these paths return before touching a device)."""
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


def kv8(vc, **kw):
    f = dict(k_codes=1 << 20, v_codes=1 << 21, k_scales=1 << 22, v_scales=1 << 23, num_pages=4, block_table=1 << 20,
             seq_lens=1 << 20, batch=1, max_blocks=1, num_kv_heads=2, head_dim=128, code=0)
    return vc.PagedKV8Struct(**{**f, **kw})


def full(vc, d=128, bits=16, batch=1, hkv=2, k=1 << 20):
    return vc.PagedKVStruct(k, 1 << 21, 4, FAKE.value, FAKE.value, batch, 1, vc.KVFormat(hkv, d, bits))


def test_write_refuses(vc):
    def call(f, c, n=16):
        return vc.STATUS[vc.library().vc_kv8_write(C.byref(f), None, C.byref(c), n, None, None)]

    assert call(full(vc, hkv=3), kv8(vc)) == "VC_ERR_INVALID_ARG"
    assert call(full(vc, d=64), kv8(vc)) == "VC_ERR_INVALID_ARG"
    assert call(full(vc, batch=2), kv8(vc)) == "VC_ERR_INVALID_ARG"
    assert call(full(vc), kv8(vc), -1) == "VC_ERR_INVALID_ARG"
    assert call(full(vc, bits=4), kv8(vc)) == "VC_ERR_UNSUPPORTED"
    assert call(full(vc, d=96), kv8(vc, head_dim=96)) == "VC_ERR_UNSUPPORTED"
    assert call(full(vc), kv8(vc, code=2)) == "VC_ERR_UNSUPPORTED"
    assert call(full(vc, k=(1 << 20) + 8), kv8(vc)) == "VC_ERR_INVALID_ARG"
    assert call(full(vc), kv8(vc, v_codes=(1 << 20) + 8)) == "VC_ERR_INVALID_ARG"
    assert call(full(vc), kv8(vc, k_scales=None)) == "VC_ERR_INVALID_ARG"
    assert call(full(vc, batch=0), kv8(vc, batch=0, k_codes=None)) == "VC_OK"


def test_attention_refuses(vc):
    def call(c, n_q=4, hq=4, scale=1.0, dtype=1, q=FAKE, ws=FAKE, nbytes=1 << 40, n=16):
        return vc.STATUS[vc.library().vc_kv8_attn(q, n_q, hq, C.byref(c), None, scale, FAKE, dtype, n, ws, nbytes, None,
                                                  None)]

    assert call(kv8(vc), n_q=65) == "VC_ERR_UNSUPPORTED"
    assert call(kv8(vc), n_q=0) == "VC_ERR_INVALID_ARG"
    assert call(kv8(vc), hq=5) == "VC_ERR_UNSUPPORTED"
    assert call(kv8(vc), hq=18) == "VC_ERR_UNSUPPORTED"
    assert call(kv8(vc, head_dim=96)) == "VC_ERR_UNSUPPORTED"
    assert call(kv8(vc, code=3)) == "VC_ERR_UNSUPPORTED"
    assert call(kv8(vc), dtype=2) == "VC_ERR_UNSUPPORTED"
    assert call(kv8(vc, num_pages=1 << 40)) == "VC_ERR_UNSUPPORTED"
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert call(kv8(vc), scale=scale) == "VC_ERR_INVALID_ARG"
    assert call(kv8(vc), n=-1) == "VC_ERR_INVALID_ARG"
    assert call(kv8(vc), q=None) == "VC_ERR_INVALID_ARG"
    assert call(kv8(vc), q=C.c_void_p((1 << 20) + 8)) == "VC_ERR_INVALID_ARG"
    assert call(kv8(vc, k_codes=(1 << 20) + 4)) == "VC_ERR_INVALID_ARG"
    assert call(kv8(vc, seq_lens=None)) == "VC_ERR_INVALID_ARG"
    assert call(kv8(vc), ws=C.c_void_p((1 << 20) + 16)) == "VC_ERR_INVALID_ARG"
    assert call(kv8(vc), ws=None) == "VC_ERR_WORKSPACE"
    assert call(kv8(vc), nbytes=100) == "VC_ERR_WORKSPACE"
    assert call(kv8(vc, batch=0), q=None, ws=None) == "VC_OK"
    L = vc.library()
    size = lambda c, n_q=1, hq=4, n=1000: L.vc_kv8_workspace_bytes(C.byref(c), n_q, hq, n)  # noqa: E731
    assert size(kv8(vc)) > 0 and size(kv8(vc), n_q=65) == 0 and size(kv8(vc, code=9)) == 0 and size(kv8(vc), n=-1) == 0
    assert L.vc_kv8_workspace_bytes(None, 1, 4, 16) == 0


def page_map(vc, **kw):
    f = dict(table=1 << 20, blocks=1 << 21, refs=1 << 22, num_pages=10, batch=2, max_blocks=3)
    return vc.PageMapStruct(**{**f, **kw})


def test_pages_refuse(vc):
    L, S, F = vc.library(), vc.STATUS, FAKE
    ref = C.byref

    def each(m, ok):
        got = [S[x] for x in (L.vc_pages_free(ref(m), F, None, None), L.vc_pages_fork(ref(m), F, F, F, 1, None, None),
                              L.vc_pages_reserve(ref(m), F, F, F, F, F, F, 1 << 40, None, None),
                              L.vc_pages_compact(ref(m), F, F, 5, F, F, F, 1 << 40, None, None))]
        assert got == [ok] * 4, got

    for kw in (dict(batch=-1), dict(max_blocks=-1), dict(num_pages=-1), dict(num_pages=1 << 31), dict(table=None),
               dict(blocks=None), dict(refs=None), dict(max_blocks=0)):
        each(page_map(vc, **kw), "VC_ERR_INVALID_ARG")
    m = page_map(vc)
    assert S[L.vc_pages_free(ref(m), None, None, None)] == "VC_ERR_INVALID_ARG"
    assert S[L.vc_pages_fork(ref(m), F, F, F, -1, None, None)] == "VC_ERR_INVALID_ARG"
    assert S[L.vc_pages_fork(ref(m), F, F, None, 1, None, None)] == "VC_ERR_INVALID_ARG"
    assert S[L.vc_pages_fork(ref(m), F, None, None, 0, None, None)] == "VC_OK"
    assert S[L.vc_pages_reserve(ref(m), F, F, F, F, F, None, 0, None, None)] == "VC_ERR_WORKSPACE"
    assert S[L.vc_pages_reserve(ref(m), F, F, F, F, F, F, 100, None, None)] == "VC_ERR_WORKSPACE"
    assert S[L.vc_pages_reserve(ref(m), F, F, F, F, None, F, 1 << 40, None, None)] == "VC_ERR_INVALID_ARG"
    assert S[L.vc_pages_compact(ref(m), F, F, 4, F, F, F, 1 << 40, None, None)] == "VC_ERR_INVALID_ARG"
    assert S[L.vc_pages_compact(ref(m), F, F, 5, F, F, None, 0, None, None)] == "VC_ERR_WORKSPACE"
    assert L.vc_pages_workspace_bytes(ref(page_map(vc, num_pages=-1))) == 0

    def copy(arrays, pages=4, src=F, n=1):
        x = (vc.PageArrayStruct * len(arrays))(*[vc.PageArrayStruct(*a) for a in arrays])
        return S[L.vc_pages_copy(x, len(arrays), pages, src, F, n, None, None, None)]

    for bad in ((None, 16), (1 << 20, 0), (1 << 20, 6), ((1 << 20) + 2, 16)):
        assert copy([bad]) == "VC_ERR_INVALID_ARG"
    assert copy([(1 << 20, 1 << 33)]) == "VC_ERR_UNSUPPORTED"
    assert copy([(1 << 20, 16)], src=None) == "VC_ERR_INVALID_ARG"
    assert copy([(1 << 20, 16)], n=-1) == "VC_ERR_INVALID_ARG"
    assert copy([(1 << 20, 16)], n=0) == "VC_OK" and copy([]) == "VC_OK"


def test_python_checks_tensors(vc):
    z = lambda *s, dt=torch.int32: torch.zeros(s, dtype=dt)  # noqa: E731
    c = vc.PagedKV8(z(4, 2, 16, 64, dt=torch.int8), z(4, 2, 16, 64, dt=torch.int8), z(4, 2, dt=torch.float32),
                    z(4, 2, dt=torch.float32), z(1, 2), z(1))
    q = z(1, 1, 4, 64, dt=torch.bfloat16)
    with pytest.raises(ValueError, match="current CUDA device"):
        vc.kv8_attn(q, c, 1.0, q, 32, z(8, dt=torch.uint8))
    with pytest.raises(ValueError, match="of the cache"):
        vc.kv8_attn(q[..., :32], c, 1.0, q, 32, z(8, dt=torch.uint8))
    assert vc.kv8_workspace_bytes(c, 1, 4, 32) > 0
    m = vc.PageMap.allocate(4, 2, 3, device="cpu")
    with pytest.raises(ValueError, match="current CUDA device"):
        vc.pages_free(m, z(2))
    with pytest.raises(ValueError, match="same pages"):
        vc.PageArrays([z(4, 4), z(5, 4)])
