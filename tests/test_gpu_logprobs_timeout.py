"""The bounded waits of vc_token_logprobs' ring, made to run out (host-side
fault injection, no GPU fault): a row whose logits did not arrive is NaN and
-1, never what the outputs or the workspace held before; the others are what
they always are, and the next call is clean."""
import pytest
import torch

pytestmark = pytest.mark.gpu

TIMEOUT, SMS = 6, 152
# rows of each ring (2, 4, 8 and 16 warps to a part), and of two, three and nine parts
CASES = [(torch.bfloat16, 2603, 5), (torch.bfloat16, 6001, 1), (torch.float32, 6001, 20), (torch.float16, 32000, 0),
         (torch.bfloat16, 32001, 20), (torch.float32, 16000, 1), (torch.float32, 20000, 3), (torch.bfloat16, 70000, 1),
         (torch.float32, 131075, 5)]


def vc():
    import lossless_compressed_kv_gb300 as m
    return m


@pytest.fixture
def fault():
    yield vc().debug_set_wait_fault
    vc().debug_set_wait_fault(0, 0)


class Call:
    """A call whose outputs and workspace stay from one time to the next."""

    def __init__(self, dtype, v, k, rows):
        g = torch.Generator(device="cuda")
        g.manual_seed(v + k)
        self.x = (torch.randn((rows, v), generator=g, device="cuda") * 3).to(dtype)
        self.ids = torch.randint(0, v, (rows, 40), generator=g, device="cuda", dtype=torch.int32)
        self.ids[:, 1] = self.ids[:, 35] = -1
        self.lp, self.ent = torch.empty((rows, 40), device="cuda"), torch.empty(rows, device="cuda")
        self.top = torch.empty((rows, k), dtype=torch.int32, device="cuda")
        self.tlp = torch.empty((rows, k), device="cuda")
        self.k = k
        self.ws = torch.full((vc().token_logprobs_workspace_bytes(rows, v, k),), 0xFF, dtype=torch.uint8, device="cuda")

    def run(self):
        st = torch.zeros(1, dtype=torch.int32, device="cuda")
        vc().token_logprobs(self.x, self.ids, self.lp, self.ws, entropy=self.ent, top_ids=self.top if self.k else None,
                            top_logprobs=self.tlp if self.k else None, status=st)
        torch.cuda.synchronize()
        return int(st.item()), [t.clone() for t in (self.lp, self.ent, self.top, self.tlp)]


def is_void(out, ids):
    """Per row: whether it is given as one that did not arrive."""
    lp, ent, top, tlp = out
    return (torch.where(ids >= 0, lp.isnan(), lp == 0).all(1) & ent.isnan() & (top == -1).all(1) & tlp.isnan().all(1))


def is_same(out, clean):
    """Per row: whether all outputs have the clean call's bits."""
    return torch.stack([(a.view(torch.int32).flatten(1) == b.view(torch.int32).flatten(1)).all(1)
                        for a, b in zip((out[0], out[1][:, None], out[2], out[3]),
                                        (clean[0], clean[1][:, None], clean[2], clean[3]))]).all(0)


@pytest.mark.parametrize("dtype,v,k", CASES)
@pytest.mark.parametrize("rows", [3, 700])
def test_no_copy_at_all(fault, dtype, v, k, rows):
    c = Call(dtype, v, k, rows)
    st, clean = c.run()
    assert st == 0 and not is_void(clean, c.ids).any()
    fault(20_000, 1)
    st, out = c.run()
    assert st == TIMEOUT and bool(is_void(out, c.ids).all())
    fault(0, 0)
    st, out = c.run()
    assert st == 0 and bool(is_same(out, clean).all())


@pytest.mark.parametrize("dtype,v,k", CASES)
def test_every_other_block_without_copies(fault, dtype, v, k):
    """Void where a row, or one of its parts, fell to such a block; elsewhere the
    same bits.  Parts are dealt out to the blocks in turn."""
    rows = 700
    c = Call(dtype, v, k, rows)
    _, clean = c.run()
    fault(2_000_000, 2)
    st, out = c.run()
    lost = torch.arange(rows, device="cuda") % SMS % 2 == 1
    if v > (16376 if dtype == torch.float32 else 32760):                # several parts: one is in an odd block
        lost[:] = True
    assert st == TIMEOUT
    assert torch.equal(is_void(out, c.ids), lost) and torch.equal(is_same(out, clean), ~lost)


@pytest.mark.parametrize("dtype,v,k", CASES)
def test_a_limit_that_runs_out_while_copies_are_under_way(fault, dtype, v, k):
    """Each row is whole or void, and the blocks end after their copies."""
    c = Call(dtype, v, k, 700)
    _, clean = c.run()
    fault(1, 0)
    st, out = c.run()
    void, same = is_void(out, c.ids), is_same(out, clean)
    assert bool((void ^ same).all()) and st == (TIMEOUT if bool(void.any()) else 0)
    fault(0, 0)
    st, out = c.run()
    assert st == 0 and bool(is_same(out, clean).all())


def test_rows_in_registers_wait_for_nothing(fault):
    c = Call(torch.float32, 900, 5, 50)
    _, clean = c.run()
    fault(1, 1)
    st, out = c.run()
    assert st == 0 and bool(is_same(out, clean).all())
