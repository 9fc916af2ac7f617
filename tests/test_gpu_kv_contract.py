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


@pytest.mark.parametrize("fmt", ["16bit", "int8", "e4m3"])
@pytest.mark.parametrize("new", [1, 40])
def test_a_scale_of_zero_keeps_what_is_not_finite(cc, new, fmt):
    """0 times a score is 0 where the score is finite (the result is a mean) and NaN elsewhere."""
    c = Case([300, 60], [new, new], heads=2, group=4, dim=128, page=16, fmt=fmt, seed=91)
    ref, ref_lse, tol, ltol = c.attention(scale=0.0)
    for over in ({}, CUT):
        q = c.q.clone()
        q[0, 1, 5], q[-1, 6, 127], q[-1, 2, 0] = math.nan, math.inf, -math.inf
        cache, batch = c.objects(cc, **over)
        out, lse = cc.kv_attention(cache, batch, q, scale=0.0)
        odd = ~torch.isfinite(q).all(-1)
        assert out[odd].isnan().all() and lse[odd].isnan().all()
        assert ((out.double() - ref).abs() <= tol)[~odd].all()
        assert ((lse.double() - ref_lse).abs() <= ltol)[~odd].all()


@pytest.mark.parametrize("fmt", ["16bit", "int8", "e4m3"])
def test_a_slot_named_twice_affects_no_other(cc, fmt):
    """Two sequences end in the same page: their rows for its slots clash, all others are stored and read back."""
    c = Case([40, 40], [40, 40], heads=2, group=1, dim=64, page=16, fmt=fmt, seed=92)
    c.table[1, 2] = c.table[0, 2]  # positions 32 .. 39 of both
    cache, batch = c.objects(cc)
    before = c.k.clone()
    cc.kv_write(cache, batch, c.k_new, c.v_new)
    k, v = cc.kv_read(cache, batch)
    clash = (torch.arange(80, device="cuda") % 40) >= 32
    for got, new in ((k, c.k_new), (v, c.v_new)):
        if fmt == "16bit":
            assert torch.equal(got[~clash], new[~clash])
        else:
            # half a step of a code (E4M3: 2^-4 of a value), and the rounding to bf16
            largest = new.double().abs().amax(-1, keepdim=True)
            bound = largest / 254 if fmt == "int8" else new.double().abs() * 2.0 ** -4 + largest * 2.0 ** -18
            err = (got.double() - new.double()).abs()
            assert (err <= (bound + (new.double().abs() + bound) * 2.0 ** -8) * (1 + 2.0 ** -16))[~clash].all()
        assert torch.equal(got[:40][32:], got[40:][32:])  # whatever it is, both read the same
    used = torch.zeros(c.pages, 16, dtype=torch.bool, device="cuda")
    for b in range(2):
        for p in range(40):
            used[int(c.table[b, p // 16]), p % 16] = True
    assert torch.equal(c.k[~used].view(torch.uint8), before[~used].view(torch.uint8))


@pytest.mark.parametrize("new", [2, 40])
def test_rows_of_no_sequence_keep_their_log_sums(cc, new):
    """Rows before the first sequence's and after the last one's: neither result nor log-sum-exp is written."""
    c = Case([100, 50], [new, new], heads=2, group=2, dim=64, page=16, seed=93)
    ref, ref_lse, tol, ltol = c.attention()
    q = torch.cat([c.q[:3], c.q, c.q[:4]])
    out, lse = torch.full_like(q, 5.0), torch.full((q.shape[0], 4), 5.0, device="cuda")
    cache, _ = c.objects(cc)
    for over in (100, 1 << 20):
        batch = cc.KvBatch(c.table, c.cu + 3, c.len_dev, n_tokens=q.shape[0], max_new=new, max_len=over)
        ws = cc.empty_kv_workspace(cache, batch, 4)
        cc.cccl_kv_attention(cache, batch, q, out, ws, lse=lse)
        assert cc.cccl_get_result(ws)[1] == cc.CCCL_OK
        assert ((out[3:-4].double() - ref).abs() <= tol).all()
        assert ((lse[3:-4].double() - ref_lse).abs() <= ltol).all()
        for t in (out, lse):
            assert (t[:3] == 5.0).all() and (t[-4:] == 5.0).all()


@pytest.mark.parametrize("new", [1, 64])
def test_rows_worked_out_again_apply_scales_in_order(cc, new):
    """Key scales near binary32's limit and scores of zero: an infinite value leaves the other channels' mean alone."""
    c = Case([300], [new], heads=1, group=2, dim=64, page=16, fmt="e4m3", seed=94)
    c.q[:] = 0
    c.ks[:] = 2.0 ** 127
    ref, ref_lse, tol, ltol = c.attention(scale=4.0)
    at = (int(c.table[0, 3]), 2)
    c.v[at][0, 7] = 0x7F  # E4M3's NaN in one channel
    for over in ({}, CUT):
        cache, batch = c.objects(cc, **over)
        out, lse = cc.kv_attention(cache, batch, c.q, scale=4.0)
        assert out[..., 7].isnan().all()
        keep = torch.arange(64, device="cuda") != 7
        assert ((out.double() - ref).abs() <= tol)[..., keep].all()
        assert ((lse.double() - ref_lse).abs() <= ltol).all()


@pytest.mark.parametrize("fmt", ["16bit", "int8"])
@pytest.mark.parametrize("spoil", ["length", "negative length", "past the rows", "order"])
def test_writes_and_reads_report_every_sequence(cc, fmt, spoil):
    """Also one that no row leads to: the others' tokens are stored and read as ever."""
    lens, new = [40, 50, 30, 20], [40, 0, 30, 20]
    c = Case(lens, new, heads=2, group=1, dim=64, page=16, fmt=fmt, seed=95)
    cache, batch = c.objects(cc)
    cc.kv_write(cache, batch, c.k_new, c.v_new)
    good = cc.kv_read(cache, batch)
    cu, kv_lens = c.cu.clone(), c.len_dev.clone()
    if spoil == "length":
        kv_lens[1] = 100000
    elif spoil == "negative length":
        kv_lens[1] = -1
    elif spoil == "past the rows":
        cu[-1] += 7
    else:
        cu[1] = 45  # sequence 0 ends past sequence 1's end
        cu[2] = 40
    bad = cc.KvBatch(c.table, cu, kv_lens, n_tokens=c.T, max_new=40, max_len=50)
    for write in (True, False):
        ws = cc.empty_kv_workspace(cache, bad)
        k, v = torch.zeros_like(c.k_new), torch.zeros_like(c.v_new)
        if write:
            cc.cccl_kv_write(cache, bad, c.k_new, c.v_new, ws)
        else:
            cc.cccl_kv_read(cache, bad, k, v, ws)
        assert cc.cccl_get_result(ws)[1] == cc.CCCL_ERR_INVALID_ARG
    if "length" in spoil:
        for a, b in zip((k, v), good):
            assert torch.equal(a, b)


@pytest.mark.parametrize("new", [1, 64])
@pytest.mark.parametrize("fmt", ["16bit", "int8"])
@pytest.mark.parametrize("scale", [1e-38, -1e-38, 1e-44, 1e30])
def test_scales_of_any_size(cc, scale, fmt, new):
    """Scales next to binary32's limits, with queries (and for the largest keys) of a size that suits."""
    c = Case([300, 129], [new, new], heads=2, group=2, dim=64, page=16, fmt=fmt, seed=96)
    if scale == 1e30:
        c.q = (c.q.float() * 1e-30).to(c.dtype)
    elif scale != 1e-44:
        c.q = (c.q.float() * 1e36).to(c.dtype)
    for over in ({}, CUT):
        cache, batch = c.objects(cc, **over)
        out, lse = cc.kv_attention(cache, batch, c.q, scale=scale)
        check(c, out, lse, scale=scale)
