"""A step with drafted tokens at its smallest: nobody drafts anything."""

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def cc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    import compression_coupled_collectives_gb300 as m

    torch.cuda.set_device(0)
    return m


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("parents", [False, True])
@pytest.mark.parametrize("words", [None, 2])
def test_a_plan_without_rows(cc, words, parents):
    """Packed tensors of no rows, with masks too: lengths and tables are what they were, no page is given."""
    tables = cc.StepTables.empty(3, 4, 9, 16)
    held, count = ints([2, 0, 1]), ints([6])
    tables.held.copy_(held), tables.free_count.copy_(count)
    got = cc.step_plan(tables, ints([17, 0, 3]), ints([0, 0, 0]), 0, mask_words=words, parents=ints([]) if parents else None)
    assert got["cu_tokens"].tolist() == [0, 0, 0, 0] and got["kv_lens"].tolist() == [17, 0, 3]
    assert torch.equal(tables.held, held) and torch.equal(tables.free_count, count)
    assert got["slots"].numel() == got["positions"].numel() == 0
    assert words is None or got["mask"].shape == (0, 2)
    with pytest.raises(cc.CcclError):  # a row more than there is room for
        cc.step_plan(tables, ints([17, 0, 3]), ints([0, 1, 0]), 0, mask_words=words)


def test_a_step_without_rows(cc):
    """The other calls on the same batch."""
    tables = cc.StepTables.empty(2, 4, 9, 16)
    plan = cc.step_plan(tables, ints([0, 0]), ints([0, 0]), 0, mask_words=1)
    cache = cc.KvCache.empty(9, 16, 2, 64)
    batch = cc.KvBatch(tables.page_table, plan["cu_tokens"], plan["kv_lens"], n_tokens=0, max_new=1, max_len=1)
    q, kv = (torch.empty(0, h, 64, dtype=torch.bfloat16, device="cuda") for h in (4, 2))
    assert cc.step_write(cache, batch, cc.StepRotary(64), q, kv, kv, positions=plan["positions"]).shape == q.shape
    out, lse = cc.step_attention(cache, batch, q, plan["mask"])
    assert out.shape == q.shape and lse.shape == (0, 4)
    p = torch.empty(0, 100, device="cuda")
    path, kept, following = cc.step_verify(p, None, ints([]), None, p[:, 0].contiguous(), plan["cu_tokens"])
    assert path.numel() == 0 and kept.tolist() == [0, 0] and following.tolist() == [-1, -1]
    assert cc.step_keep(cache, batch, path, kept).tolist() == [0, 0]
