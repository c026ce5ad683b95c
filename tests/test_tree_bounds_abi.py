"""vc_tree_attn's workspace where max_seq_len is as large as it can be (on the
host): the largest bound asks for no fewer ranges than a smaller one."""
import ctypes as C

import pytest

from tests.test_tree_abi import cache, vc  # noqa: F401 (vc: the fixture)


@pytest.mark.parametrize("n_q,hq,d", [(4, 4, 128), (33, 16, 64), (40, 16, 128), (64, 16, 128)])
@pytest.mark.parametrize("batch", [1, 3, 200])
def test_the_largest_bound(vc, n_q, hq, d, batch):  # noqa: F811
    size = lambda n: vc.library().vc_tree_workspace_bytes(C.byref(cache(vc, d=d, batch=batch)), n_q, hq, n)  # noqa: E731
    assert size(1) <= size(1000) <= size(1 << 24) == size((1 << 31) - 100) == size((1 << 31) - 10) == size((1 << 31) - 1)
