"""GPU vc_token_logprobs against the 64-bit definition.

Tolerances: y = (x - max) / tau takes three roundings (3 * 2^-24 |y|).  log S:
each e^y is off by 2^-22 and by its argument's error, at most 4 * 2^-24 |y|
e^y <= 2 * 2^-24; a sum of fewer than 600 fp32 additions in a chain adds 600 *
2^-24 of S, in all below 640 * 2^-24; the same for the sum of y e^y (terms at
most 0.37 off by as much).  Ids are exact."""
import math

import numpy as np
import pytest
import torch

from oracle import tree as T

pytestmark = pytest.mark.gpu
E = 2.0 ** -24


def vc():
    import lossless_compressed_kv_gb300 as m
    return m


def call(x, ids, k, tau=1.0, entropy=True):
    rows, v = x.shape
    n = ids.shape[1]
    lp = torch.full((rows, n), 9.0, device="cuda")
    ent = torch.full((rows,), 9.0, device="cuda") if entropy else None
    top = torch.full((rows, k), 9, dtype=torch.int32, device="cuda") if k else None
    tlp = torch.full((rows, k), 9.0, device="cuda") if k else None
    ws = torch.full((vc().token_logprobs_workspace_bytes(rows, v, k),), 0xFF, dtype=torch.uint8, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    vc().token_logprobs(x, ids, lp, ws, temperature=tau, entropy=ent, top_ids=top, top_logprobs=tlp, status=st)
    torch.cuda.synchronize()
    z = lambda t: None if t is None else t.cpu().numpy()  # noqa: E731
    return z(lp), z(ent), z(top), z(tlp), int(st.item())


def check(x, ids, k, tau=1.0, rows=None):
    lp, ent, top, tlp, st = call(x, ids, k, tau)
    xh, ih = x.double().cpu().numpy(), ids.cpu().numpy()
    for r in range(x.shape[0]) if rows is None else rows:
        a, e, t, tl = T.token_logprobs(xh[r], ih[r], tau, k)
        close(lp[r], a, r)
        if k:
            assert list(top[r]) == t, (r, top[r], t)
            close(tlp[r], tl, r)
        if math.isnan(e):
            assert math.isnan(ent[r])
        else:
            assert abs(ent[r] - e) <= 640 * E * (2 + 2 * e), (r, ent[r], e)
    return lp, ent, top, tlp, st


def close(got, want, r):
    got, want = np.asarray(got, np.float64), np.asarray(want, np.float64)
    assert (np.isnan(got) == np.isnan(want)).all(), r
    f = np.isfinite(want)
    assert (got[~f & ~np.isnan(want)] == want[~f & ~np.isnan(want)]).all(), (r, got, want)
    assert (np.abs(got[f] - want[f]) <= 640 * E + 4 * E * np.abs(want[f])).all(), (r, got[f], want[f])


def logits(seed, rows, v, dtype, std=3.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn((rows, v), generator=g, device="cuda") * std).to(dtype)


def some_ids(seed, rows, v, n):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randint(0, v, (rows, n), generator=g, device="cuda", dtype=torch.int32)


DT = [torch.float32, torch.bfloat16, torch.float16]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("v", [1, 2, 3, 31, 32, 33, 127, 1000, 1001, 4099, 32000, 50257, 131072, 131075])
@pytest.mark.parametrize("k", [0, 1, 20, 64])
def test_sizes(dtype, v, k):
    check(logits(v, 3, v, dtype), some_ids(v, 3, v, 2), k)


@pytest.mark.parametrize("rows", [1, 5, 300])
@pytest.mark.parametrize("v", [257, 9000])
def test_rows(rows, v):
    check(logits(rows, rows, v, torch.float32), some_ids(rows, rows, v, 1), 8, 0.7, range(0, rows, 13))


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("off,pad", [(1, 0), (0, 3), (3, 5), (7, 9), (8, 8)])
def test_strided_and_misaligned_rows(dtype, off, pad):
    wide = logits(off, 4, 5003 + off + pad, dtype)
    check(wide[:, off:off + 5003], some_ids(1, 4, 5003, 3), 9)
    check(wide[:, off:off + 17], some_ids(1, 4, 17, 3), 20)


@pytest.mark.parametrize("dtype", DT)
def test_ties_go_to_the_lowest_id(dtype):
    v = 20000
    x = torch.zeros((6, v), dtype=dtype, device="cuda")
    x[1] = torch.arange(v, device="cuda").remainder(7).to(dtype)
    x[2, 5000:] = 1.0
    x[3, ::100] = 2.0
    x[3, 1::100] = -0.0
    x[4] = -torch.arange(v, device="cuda").float().div(1000).floor().to(dtype)
    x[5, :3000] = 4.0                                 # a long run of equal maxima
    check(x, some_ids(2, 6, v, 2), 64)


@pytest.mark.parametrize("dtype", DT)
def test_sorted_rows(dtype):
    """Rising and falling rows: one thread's or one part's elements hold all the largest."""
    v = 40000
    up = torch.linspace(-10, 10, v, device="cuda").to(dtype)
    x = torch.stack([up, up.flip(0), up.view(-1, 200).T.reshape(-1), up.view(200, -1).T.reshape(-1)])
    check(x, some_ids(3, 4, v, 2), 64)


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("v", [9, 1000, 40000])
def test_rows_with_nothing_left_and_without_distribution(dtype, v):
    x = logits(4, 9, v, dtype)
    inf = float("inf")
    x[1] = -inf                                        # every token ruled out
    x[2] = -inf
    x[2, v - 2] = -5.0                                 # all but one
    x[3, ::2] = -inf
    x[4, v // 2] = float("nan")
    x[5, v - 1] = inf
    x[6] = torch.finfo(dtype).min                      # the type's lowest value everywhere
    x[7, 1:] = torch.finfo(dtype).min
    x[8, 0] = -float("nan")
    lp, ent, top, tlp, _ = check(x, some_ids(5, 9, v, 2), 5)
    assert (lp[1] == -inf).all() and ent[1] == 0 and (top[1] == -1).all() and (tlp[1] == -inf).all()
    assert ent[2] == 0 and top[2, 0] == v - 2 and tlp[2, 0] == 0 and (top[2, 1:] == -1).all()
    for r in (4, 5, 8):
        assert np.isnan(lp[r]).all() and np.isnan(ent[r]) and (top[r] == -1).all() and np.isnan(tlp[r]).all()
    assert abs(ent[6] - math.log(v)) < 1e-3


def test_ids_outside_the_vocabulary():
    x = logits(6, 2, 100, torch.float32)
    ids = torch.tensor([[-1, 5, 99], [0, -1, -1]], dtype=torch.int32, device="cuda")
    lp, _, _, _, st = check(x, ids, 2)
    assert st == 0 and lp[0, 0] == 0 and lp[1, 1] == 0
    for bad in (100, -2, 1 << 30):
        ids[1, 0] = bad
        lp, _, _, _, st = check(x, ids, 0)
        assert st == 3 and lp[1, 0] == 0


def test_all_but_certain_rows_keep_their_digits():
    """log p of the likeliest token and the entropy, where S = 1 + 1e-9."""
    x = torch.full((2, 3000), -40.0, device="cuda")
    x[:, 7], x[:, 8] = 0.0, -21.0
    x[1] *= 0.5
    ids = torch.tensor([[7], [7]], dtype=torch.int32, device="cuda")
    lp, ent, top, _, _ = call(x, ids, 1, 0.5 if False else 1.0)
    for r in range(2):
        a, e, _, _ = T.token_logprobs(x[r].double().cpu().numpy(), [7], 1.0, 1)
        assert abs(lp[r, 0] - a[0]) <= 1e-4 * abs(a[0]) and abs(ent[r] - e) <= 1e-4 * e


@pytest.mark.parametrize("tau", [1e-30, 1e-3, 0.5, 3.0, 1e6, 3e38])
def test_temperatures(tau):
    x = logits(7, 3, 2000, torch.float32)
    lp, ent, top, tlp, _ = call(x, some_ids(7, 3, 2000, 2), 4, tau)
    t32 = float(np.float32(tau))
    for r in range(3):
        a, e, t, tl = T.token_logprobs(x[r].double().cpu().numpy(), some_ids(7, 3, 2000, 2)[r].cpu().numpy(), t32, 4)
        assert list(top[r]) == t and abs(ent[r] - e) <= 640 * E * (2 + 2 * e)
        for got, want in list(zip(lp[r], a)) + list(zip(tlp[r], tl)):
            assert abs(got - want) <= 640 * E + 4 * E * abs(want) or (want < -3.4e38 and got == -np.inf)


def test_same_bits_and_a_graph():
    x = logits(8, 40, 32000, torch.bfloat16)
    ids = some_ids(8, 40, 32000, 1)
    a, b = call(x, ids, 20), call(x, ids, 20)
    for p, q in zip(a[:4], b[:4]):
        assert (p == q).all()
    ws = torch.full((vc().token_logprobs_workspace_bytes(40, 32000, 20),), 0xFF, dtype=torch.uint8, device="cuda")
    lp = torch.zeros((40, 1), device="cuda")
    top = torch.zeros((40, 20), dtype=torch.int32, device="cuda")
    tlp = torch.zeros((40, 20), device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        vc().token_logprobs(x, ids, lp, ws, top_ids=top, top_logprobs=tlp)
    x.copy_(x.flip(0))
    ids.copy_(ids.flip(0))
    g.replay()
    torch.cuda.synchronize()
    assert (lp.cpu().numpy()[::-1] == a[0]).all() and (top.cpu().numpy()[::-1] == a[2]).all()
    assert (tlp.cpu().numpy()[::-1] == a[3]).all()


def test_nothing_asked():
    """Entropy alone; no ids, no alternatives."""
    x = logits(9, 2, 500, torch.float32)
    ids = torch.zeros((2, 0), dtype=torch.int32, device="cuda")
    _, ent, _, _, st = call(x, ids, 0)
    p = torch.softmax(x.double(), -1)
    assert st == 0 and np.allclose(ent, -(p * p.log()).sum(-1).cpu().numpy(), rtol=1e-5)
    assert call(x, some_ids(1, 2, 500, 1), 1, entropy=False)[4] == 0
