"""Arrays of pages whose tensors were resized in place: read anew, or refused."""
import pytest
import torch

from tests.test_gpu_pages import i32, status, vc

pytestmark = pytest.mark.gpu


def counted(*shape):
    n = 1
    for x in shape:
        n *= x
    return torch.arange(n, device="cuda", dtype=torch.int32).view(shape)


def test_a_pool_that_grew():
    m, st = vc(), status()
    t, scales = counted(4, 8), counted(4, 2)
    a = m.PageArrays([t, scales])
    t.set_(counted(8, 8))
    scales.set_(counted(8, 2))
    m.pages_copy(a, i32([7]), i32([0]), status=st)
    torch.cuda.synchronize()
    assert st.item() == 0 and t[0].tolist() == list(range(56, 64)) and scales[0].tolist() == [14, 15]
    assert torch.equal(t[1:], counted(8, 8)[1:])


def test_a_pool_of_other_pages_where_it_was():
    m = vc()
    t = counted(4, 16)
    a = m.PageArrays([t])
    t.resize_(8, 8)
    assert t.shape == (8, 8)
    m.pages_copy(a, i32([7]), i32([2]))
    torch.cuda.synchronize()
    ref = counted(8, 8)
    ref[2] = ref[7]
    assert torch.equal(t, ref)


def test_pools_that_no_longer_agree():
    m = vc()
    t, u = counted(4, 8), counted(4, 8)
    a = m.PageArrays([t, u])
    t.set_(counted(2, 8))
    with pytest.raises(ValueError, match="same pages"):
        m.pages_copy(a, i32([1]), i32([0]))
    t.set_(counted(4, 16)[:, :8])
    with pytest.raises(ValueError, match="contiguous"):
        m.pages_copy(a, i32([1]), i32([0]))
    t.set_(counted(4, 8))
    m.pages_copy(a, i32([1]), i32([0]))
    torch.cuda.synchronize()
    assert t[0].tolist() == u[0].tolist() == list(range(8, 16))
