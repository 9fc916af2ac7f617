"""The binding of a step with drafted tokens on a machine without a GPU: what is
refused before the library is called."""

import pytest
import torch


@pytest.fixture(scope="module")
def cc():
    import __graft_entry__

    __graft_entry__.build()
    import compression_coupled_collectives_gb300 as m

    return m


def ints(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


class Elsewhere(torch.Tensor):
    """A tensor that says it lies on another device."""

    def get_device(self):
        return 1


def test_a_workspace_on_another_device_is_refused(cc):
    """In every call: a report into it would go through another device's address."""
    ws = torch.zeros(64, dtype=torch.uint8).as_subclass(Elsewhere)
    tables = cc.StepTables(ints(2, 5), ints(2), ints(9), ints(1), page_tokens=16)
    cache = cc.KvCache.empty(4, 16, 2, 64, device="cpu")
    batch = cc.KvBatch(ints(2, 5), ints(3), ints(2), n_tokens=4, max_new=2, max_len=9)
    rotary = cc.StepRotary(64, device="cpu")
    q, kv = torch.zeros(4, 4, 64, dtype=torch.bfloat16), torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    p = torch.zeros(4, 9)
    for call in (lambda: cc.cccl_step_plan(tables, ints(2), ints(2), ws, cu_tokens=ints(3), kv_lens=ints(2), rows=4),
                 lambda: cc.cccl_step_write(cache, batch, rotary, q, kv, kv, q, ws),
                 lambda: cc.cccl_step_attention(cache, batch, q, ints(4, 1), q, ws),
                 lambda: cc.cccl_step_verify(p, None, ints(4), None, torch.zeros(4), ints(3), ints(4), ints(2), ints(2), ws),
                 lambda: cc.cccl_step_keep(cache, batch, ints(4), ints(2), None, ws)):
        with pytest.raises(ValueError, match="ws is on another device|on the cache's device"):
            call()
