"""Keeping drafted tokens: what the outputs may lie over, and batches without rows."""

import pytest
import torch

from kv_reference import Case

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


def test_lengths_over_what_the_call_reads_are_refused(cc):
    """Wherever an input and the lengths have a number in common; side by side they may lie."""
    c = Case([60, 60, 60], [20, 20, 20], heads=2, dim=64, page=16, seed=4)
    cache, _ = c.objects(cc)
    pool = ints([0] * 200)
    kv_lens, cu, kept, path, table = pool[10:13], pool[20:24], pool[30:33], pool[40:100], pool[110:122].view(3, 4)
    kv_lens.copy_(c.len_dev), cu.copy_(c.cu), kept.copy_(ints([1, 1, 1])), table.copy_(c.table)
    before = pool.clone()
    batch = cc.KvBatch(table, cu, kv_lens, n_tokens=60, max_new=20, max_len=60)
    ws = cc.empty_step_workspace()
    for lo, hi in ((10, 13), (20, 24), (30, 33), (40, 100), (110, 122)):
        for at in (lo - 2, lo, hi - 1):
            with pytest.raises(cc.CcclError):
                cc.cccl_step_keep(cache, batch, path, kept, pool[at:at + 3], ws)
        assert torch.equal(pool, before)
        for at in (lo - 3, hi):
            cc.cccl_step_keep(cache, batch, path, kept, pool[at:at + 3], ws)
            assert pool[at:at + 3].tolist() == [41, 41, 41]
            pool.copy_(before)
    assert cc.cccl_get_result(ws)[1] == cc.CCCL_OK


def test_a_batch_without_rows_has_lengths_all_the_same(cc):
    """n_tokens 0: nothing moves, every length is written; counts that do not fit are reported; batch 0 is a no-op."""
    c = Case([60, 0, 9], [0, 0, 0], heads=2, dim=64, page=16, seed=4)
    cache, batch = c.objects(cc)
    start = [c.k.clone(), c.v.clone()]
    path = ints([])
    assert cc.step_keep(cache, batch, path, ints([0, 0, 0])).tolist() == [60, 0, 9]
    ws, lens = cc.empty_step_workspace(), ints([-1, -1, -1])
    cc.cccl_step_keep(cache, batch, path, ints([0, 1, 0]), lens, ws)
    assert cc.cccl_get_result(ws)[1] == cc.CCCL_ERR_INVALID_ARG and lens.tolist() == [60, 0, 9]
    none = cc.KvBatch(c.table[:0], ints([0]), ints([]), n_tokens=0, max_new=1, max_len=1)
    ws = cc.empty_step_workspace()
    cc.cccl_step_keep(cache, none, path, ints([]), ints([]), ws)
    assert cc.cccl_get_result(ws)[1] == cc.CCCL_OK
    assert torch.equal(c.k, start[0]) and torch.equal(c.v, start[1])


def test_lengths_beside_the_tables_rows_are_taken(cc):
    """In the gap between two rows of a table that is a slice, up to their very ends, and no further."""
    c = Case([60, 40], [20, 20], heads=2, dim=64, page=16, seed=4)
    cache, _ = c.objects(cc)
    pool = torch.zeros(2, 8, dtype=torch.int32, device="cuda")
    table = pool[:, 1:5]
    table.copy_(c.table)
    batch = cc.KvBatch(table, c.cu, c.len_dev, n_tokens=40, max_new=20, max_len=60)
    path, kept, ws, flat = ints([0] * 40), ints([1, 1]), cc.empty_step_workspace(), pool.view(-1)
    for at in (5, 6, 7, 13):
        cc.cccl_step_keep(cache, batch, path, kept, flat[at:at + 2], ws)
        assert flat[at:at + 2].tolist() == [41, 21]
    for at in (0, 1, 4, 8, 9, 12):
        with pytest.raises(cc.CcclError):
            cc.cccl_step_keep(cache, batch, path, kept, flat[at:at + 2], ws)
    assert torch.equal(table, c.table) and cc.cccl_get_result(ws)[1] == cc.CCCL_OK
