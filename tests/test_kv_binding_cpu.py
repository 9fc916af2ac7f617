"""The paged cache's binding: what a tensor's strides say is what the call gets."""

import pytest
import torch


@pytest.fixture(scope="module")
def cc():
    import __graft_entry__

    __graft_entry__.build()
    import compression_coupled_collectives_gb300 as m

    return m


def batch(cc, table):
    n = table.shape[0]
    return cc.KvBatch(table, torch.zeros(n + 1, dtype=torch.int32), torch.zeros(n, dtype=torch.int32), n_tokens=1,
                      max_new=1, max_len=1)


def test_tables_whose_rows_overlap_are_refused(cc):
    one = torch.arange(5, dtype=torch.int32)[None]
    with pytest.raises(ValueError):
        batch(cc, one.expand(4, -1))
    with pytest.raises(ValueError):
        batch(cc, torch.arange(20, dtype=torch.int32).as_strided((4, 5), (3, 1)))
    assert batch(cc, one.expand(4, -1).contiguous())._c.table_stride == 5


def test_row_strides_reach_the_call(cc):
    wide = torch.arange(40, dtype=torch.int32).view(4, 10)
    for table, stride, pages in ((wide, 10, 10), (wide[:, :3], 10, 3), (wide[:, 2:3], 10, 1), (wide[::2], 20, 10),
                                 (wide[:1], 10, 10), (wide[:1].expand(1, -1), 10, 10),
                                 (torch.arange(7, dtype=torch.int32).expand(1, 7), 7, 7), (wide[:0], 10, 10)):
        b = batch(cc, table)
        assert (b._c.table_stride, b._c.table_pages) == (stride, pages)
        assert (b._c.page_table or 0) == table.data_ptr()
