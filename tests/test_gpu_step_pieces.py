"""Attention over trees where a block gets many pieces of different kinds: shared
by two warpgroups, of a single tile of tokens, of more than one tile of rows,
whole and cut, in runs longer than the ring that hands them on."""

import pytest
import torch

import step_schedule as sched
from step_reference import TreeCase

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


@pytest.mark.parametrize("fmt", ["16bit", "int8"])
@pytest.mark.parametrize("case", sorted(sched.CASES))
def test_runs_of_pieces(cc, case, fmt):
    lens, new, heads, group, window = sched.CASES[case]
    c = TreeCase(lens, new, heads=heads, group=group, dim=64, fmt=fmt, seed=len(case), layout="htd")
    ref, ref_lse, tol, ltol = c.attention(window=window)
    for over in ({}, dict(max_len=1 << 20)):  # items whole; cut at shares' ends
        cache, batch = c.objects(cc, **over)
        ws = cc.empty_kv_workspace(cache, batch, heads * group)
        outs = []
        for _ in range(3):
            out = torch.full_like(c.q, float("nan"))
            lse = torch.full(c.q.shape[:2], float("nan"), device="cuda")
            cc.cccl_step_attention(cache, batch, c.q, c.mask, out, ws, window=window, lse=lse)
            assert cc.cccl_get_result(ws)[1] == cc.CCCL_OK
            outs.append((out, lse))
        out, lse = outs[0]
        assert ((out.double() - ref).abs() <= tol).all()
        assert ((lse.double() - ref_lse).abs() <= ltol).all()
        for again in outs[1:]:
            assert torch.equal(again[0], out) and torch.equal(again[1], lse)


@pytest.mark.parametrize("fmt", ["16bit", "e4m3"])
@pytest.mark.parametrize("heads,tiles", [(2, 7), (1, 13), (1, 17), (5, 4)])
def test_one_tree_of_many_row_tiles(cc, heads, tiles, fmt):
    """As many shares for each of its items, or (17: too many SMs would be idle; 20: too few for each) an even cut."""
    new = 32 * tiles - 5  # groups of 8: rows of 256
    c = TreeCase([9001], [new], heads=heads, group=8, dim=64, fmt=fmt, seed=tiles)
    ref, ref_lse, tol, ltol = c.attention()
    cache, batch = c.objects(cc)
    out, lse = cc.step_attention(cache, batch, c.q, c.mask)
    assert ((out.double() - ref).abs() <= tol).all() and ((lse.double() - ref_lse).abs() <= ltol).all()
