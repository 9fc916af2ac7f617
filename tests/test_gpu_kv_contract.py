"""Corners of what include/cccl_kv.h says, on the GPU against binary64."""

import math

import pytest
import torch

from kv_reference import Case

pytestmark = pytest.mark.gpu

CUT = dict(max_len=1 << 20)


@pytest.fixture(scope="module")
def cc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    import compression_coupled_collectives_gb300 as m

    torch.cuda.set_device(0)
    return m


def check(c, out, lse, **kw):
    ref, ref_lse, tol, ltol = c.attention(**kw)
    assert torch.isfinite(out).all() and ((out.double() - ref).abs() <= tol).all()
    none = ref_lse == -math.inf
    assert (lse[none] == -math.inf).all() and not out[none].any()
    assert ((lse.double() - ref_lse).abs() <= ltol)[~none].all()


@pytest.mark.parametrize("over", [{}, CUT])
@pytest.mark.parametrize("window", [0, 1, 20])
@pytest.mark.parametrize("fmt", ["16bit", "int8"])
@pytest.mark.parametrize("new", [3, 70])
def test_rows_before_position_zero(cc, new, fmt, window, over):
    """More new rows than tokens: causal rows at negative positions see nothing, others every key."""
    c = Case([2, new - 1, 0, new + 40], [new] * 4, heads=2, group=3, dim=64, page=16, fmt=fmt, seed=90, fill=math.nan)
    cache, batch = c.objects(cc, **over)
    for causal in (True, False):
        out, lse = cc.kv_attention(cache, batch, c.q, causal=causal, window=window)
        check(c, out, lse, causal=causal, window=window)
        if window == 0:
            assert (lse[:new - 2] == -math.inf).all() == causal
