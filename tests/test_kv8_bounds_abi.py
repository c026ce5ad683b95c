"""vc_kv8_attn's workspace where max_seq_len is as large as it can be (on the
host): the largest bound asks for no fewer ranges than a smaller one."""
import ctypes as C

import pytest

from tests.test_kv8_abi import kv8, vc  # noqa: F401 (vc: the fixture)


@pytest.mark.parametrize("n_q,hq,d", [(1, 8, 128), (1, 2, 64), (4, 16, 64), (4, 8, 128), (16, 8, 128), (64, 8, 64), (64, 16, 128)])
@pytest.mark.parametrize("batch", [1, 3, 200])
def test_the_largest_bound(vc, n_q, hq, d, batch):  # noqa: F811
    size = lambda n: vc.library().vc_kv8_workspace_bytes(C.byref(kv8(vc, head_dim=d, batch=batch)), n_q, hq, n)  # noqa: E731
    assert size(1) <= size(1000) <= size(1 << 24) == size((1 << 31) - 100) == size((1 << 31) - 10) == size((1 << 31) - 1)
