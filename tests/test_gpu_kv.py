"""The paged cache calls on the GPU against their definitions in binary64."""

import math

import pytest
import torch

from kv_reference import LIMIT, UNIT, Case, codes64, quantise

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def cc():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    import compression_coupled_collectives_gb300 as m

    torch.cuda.set_device(0)
    return m


def same_bits(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


# ------------------------------------------------------------------ write and read
SHAPES = [
    # lens, new, heads, dim, page
    ([1], [1], 1, 16, 1),
    ([5, 0, 33, 16], [5, 0, 3, 16], 2, 64, 16),
    ([40, 7], [40, 7], 3, 128, 24),
    ([100, 1, 257], [1, 1, 1], 8, 128, 16),
    ([61], [60], 5, 80, 7),
    ([300] * 40, [50] * 40, 2, 112, 32),
    ([3, 9], [7, 9], 2, 96, 4),  # more new rows than cached tokens: four of them lie before position 0
]


@pytest.mark.parametrize("layout", ["thd", "htd", "kv"])
@pytest.mark.parametrize("fmt", ["16bit", "int8", "e4m3"])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_write_then_read(cc, shape, dtype, fmt, layout):
    lens, new, heads, dim, page = SHAPES[shape]
    c = Case(lens, new, heads=heads, group=1, dim=dim, page=page, dtype=dtype, fmt=fmt, layout=layout, seed=shape)
    if c.T > 3:  # a vector of zeros, one of the type's extremes, one of its smallest numbers
        c.k_new[0] = 0
        c.k_new[1] = torch.finfo(dtype).max * torch.sign(c.k_new[1].float()).to(dtype)
        c.v_new[2] = (torch.finfo(dtype).tiny * torch.randint(-3, 4, c.v_new[2].shape, device="cuda")).to(dtype) / 2
    # slices of one fused tensor
    fused = torch.cat([c.k_new, c.k_new, c.v_new], 1)
    k_new, v_new = fused[:, heads:2 * heads], fused[:, 2 * heads:]
    before = [None if t is None else t.clone() for t in (c.k, c.v, c.ks, c.vs)]
    cache, batch = c.objects(cc)
    cc.kv_write(cache, batch, k_new, v_new)

    want = [None if t is None else t.clone() for t in before]
    row = 0
    inside = torch.zeros(c.T, dtype=torch.bool, device="cuda")
    for b, n in enumerate(c.new):
        for i in range(n):
            p = c.lens[b] - n + i
            if p >= 0:
                at = (int(c.table[b, p // page]), p % page)
                inside[row + i] = True
                for x, data, scales in ((k_new, 0, 2), (v_new, 1, 3)):
                    if fmt == "16bit":
                        want[data][at] = x[row + i]
                    else:
                        codes, scale = quantise(x[row + i], fmt)
                        want[data][at], want[scales][at] = codes, scale
        row += n
    for got, ref in zip((c.k, c.v, c.ks, c.vs), want):
        assert ref is None or same_bits(got, ref)  # what was not written keeps its bytes

    k_back, v_back = cc.kv_read(cache, batch)
    for back, x in ((k_back, k_new), (v_back, v_new)):
        assert not back[~inside].any()
        if fmt == "16bit":
            assert same_bits(back[inside], x[inside])
            continue
        codes, scale = quantise(x, fmt)
        code_val = codes64(codes, fmt).float() * scale[..., None]
        assert same_bits(back[inside], code_val.to(dtype)[inside])
        # and no further from the value than the format allows: half a code step
        # (a few ulps of binary32 in scale and inverse), then one rounding
        v = x.double()[inside]
        s = scale.double()[inside][..., None]
        half = s / 2 if fmt == "int8" else torch.maximum(v.abs() * 2.0 ** -4, s * 2.0 ** -10)
        bound = half * (1 + 2.0 ** -16) + v.abs() * 2.0 ** -21 + (v.abs() + half) * UNIT[dtype] + s * 2.0 ** -16
        normal = s.expand_as(v) > 2.0 ** -100  # below, binary32 itself has few bits left
        floor = torch.finfo(dtype).smallest_normal * UNIT[dtype] * 2
        assert ((back[inside].double() - v).abs() <= bound + floor)[normal].all()


def test_write_marks_vectors_that_are_not_finite(cc):
    for fmt in ("int8", "e4m3"):
        c = Case([8], [8], heads=2, dim=64, fmt=fmt)
        c.k_new[2, 0, 5] = float("nan")
        c.k_new[3, 1, 63] = float("-inf")
        c.v_new[4, 0, 0] = float("inf")
        cache, batch = c.objects(cc)
        cc.kv_write(cache, batch, c.k_new, c.v_new)
        k, v = cc.kv_read(cache, batch)
        bad_k = torch.zeros(8, 2, dtype=torch.bool, device="cuda")
        bad_k[2, 0] = bad_k[3, 1] = True
        bad_v = torch.zeros(8, 2, dtype=torch.bool, device="cuda")
        bad_v[4, 0] = True
        for x, bad in ((k, bad_k), (v, bad_v)):
            assert x.isnan()[bad].all() and x.isfinite()[~bad].all()


# ------------------------------------------------------------------ attention
def check(c, out, lse, **kw):
    ref, ref_lse, tol, ltol = c.attention(**kw)
    err = (out.double() - ref).abs()
    assert torch.isfinite(out).all()
    assert (err <= tol).all(), "worst %g of its bound" % (err / tol.clamp(min=1e-300)).max()
    none = ref_lse == -math.inf
    assert (lse[none] == -math.inf).all() and not out[none].any()
    assert ((lse.double() - ref_lse).abs() <= ltol)[~none].all()


ATTEND = [
    # lens, new, heads, group, dim, page
    ([1], [1], 1, 1, 16, 1),
    ([0], [1], 2, 2, 64, 16),
    ([2, 0, 17], [1, 2, 1], 2, 4, 64, 16),
    ([517], [1], 8, 4, 128, 16),
    ([1999, 3, 640, 128, 127, 129], [1] * 6, 3, 1, 64, 24),
    ([1000, 31, 64], [1, 1, 1], 2, 16, 128, 64),
    ([900, 77], [1, 1], 1, 17, 96, 5),
    ([300, 5, 64], [4, 5, 3], 2, 4, 128, 16),
    ([130, 257, 64], [130, 33, 64], 2, 4, 128, 16),
    ([100, 2, 0, 300], [60, 9, 4, 0], 2, 3, 80, 24),  # rows before position 0: nothing visible
    ([700], [700], 1, 1, 128, 16),
    ([513], [257], 2, 5, 112, 32),
    ([2050], [190], 3, 8, 64, 16),
]


# what makes a call cut items among blocks and join their parts: an expectation of long sequences
CUT = dict(max_len=1 << 20)


@pytest.mark.parametrize("fmt", ["16bit", "int8", "e4m3"])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("shape", range(len(ATTEND)))
def test_attention(cc, shape, dtype, fmt):
    lens, new, heads, group, dim, page = ATTEND[shape]
    c = Case(lens, new, heads=heads, group=group, dim=dim, page=page, dtype=dtype, fmt=fmt, seed=shape,
             layout=["thd", "htd", "kv"][shape % 3], fill=float("nan"))
    for over in ({}, CUT):
        cache, batch = c.objects(cc, **over)
        out, lse = cc.kv_attention(cache, batch, c.q)
        check(c, out, lse)


LONGER = [
    # lens, new, heads, group, dim, page: tiles that whole pages cover, at every page size that divides or is
    # divided by a tile, and at others; rows below, at and above one tile of rows
    ([3000, 1025], [70, 64], 2, 4, 128, 8),
    ([2700], [129], 1, 2, 64, 64),
    ([1500, 4000], [33, 300], 2, 1, 128, 128),
    ([2900, 128], [40, 128], 1, 8, 96, 256),
    ([2600, 513, 1024], [20, 100, 3], 2, 6, 16, 48),
    ([1300], [90], 2, 3, 48, 16),
    ([5000], [12], 2, 4, 128, 16),
    ([5000, 700], [1, 1], 2, 8, 128, 128),
    ([2048], [2], 1, 16, 64, 12),
    ([900], [60], 1, 2, 64, 200),
]


@pytest.mark.parametrize("window", [0, 700])
@pytest.mark.parametrize("dtype,fmt", [(BF, "16bit"), (HF, "16bit"), (BF, "int8"), (HF, "int8"), (BF, "e4m3")])
@pytest.mark.parametrize("shape", range(len(LONGER)))
def test_attention_over_many_tiles(cc, shape, dtype, fmt, window):
    lens, new, heads, group, dim, page = LONGER[shape]
    c = Case(lens, new, heads=heads, group=group, dim=dim, page=page, dtype=dtype, fmt=fmt, seed=20 + shape,
             layout=["htd", "kv", "thd"][shape % 3], fill=float("nan"))
    for over in ({}, CUT):
        cache, batch = c.objects(cc, **over)
        out, lse = cc.kv_attention(cache, batch, c.q, window=window)
        check(c, out, lse, window=window)


def test_many_sequences(cc):
    """As many as a call takes, some of them without tokens."""
    lens = [(7 * b) % 41 for b in range(1024)]
    new = [min(n, 1 + b % 3) if b % 5 else 0 for b, n in enumerate(lens)]
    c = Case(lens, new, heads=1, group=2, dim=64, page=16, fmt="int8", seed=40)
    for over in ({}, CUT):
        cache, batch = c.objects(cc, **over)
        out, lse = cc.kv_attention(cache, batch, c.q)
        check(c, out, lse)
        cache, batch = c.objects(cc, max_new=500, **over)  # the other kernel
        out, lse = cc.kv_attention(cache, batch, c.q)
        check(c, out, lse)


def test_queries_of_very_different_sizes(cc):
    """One row's size has no effect on another's, and a row of infinities none on its neighbours."""
    for fmt in ("int8", "e4m3", "16bit"):
        for new in (1, 40):
            c = Case([400], [new], heads=1, group=8, dim=64, page=16, fmt=fmt, seed=41)
            c.q[:, 1] *= 1e30
            c.q[:, 2] *= 1e-30
            c.q[:, 3] = float("inf")
            c.q[:, 4] = 0
            cache, batch = c.objects(cc)
            out, lse = cc.kv_attention(cache, batch, c.q)
            ref, ref_lse, tol, ltol = c.attention()
            rows = [0, 2, 4, 5, 6, 7]
            assert ((out.double() - ref).abs() <= tol)[:, rows].all()
            assert ((lse.double() - ref_lse).abs() <= ltol)[:, rows].all()
            # one key holds all of the weight
            assert ((out.double() - ref).abs() <= tol)[:, 1].all()
            assert out[:, 3].isnan().all()


@pytest.mark.parametrize("new", [1, 70])
@pytest.mark.parametrize("fmt", ["16bit", "int8"])
@pytest.mark.parametrize("causal,window", [(True, 1), (True, 37), (True, 128), (False, 0), (False, 50), (True, 1 << 40)])
def test_attention_masks(cc, causal, window, fmt, new):
    c = Case([300, 129, 1, 40], [new, new, new, new], heads=2, group=3, dim=64, page=16, fmt=fmt, seed=window % 1000,
             fill=float("inf"))
    for over in ({}, CUT):
        cache, batch = c.objects(cc, **over)
        out, lse = cc.kv_attention(cache, batch, c.q, causal=causal, window=window)
        check(c, out, lse, causal=causal, window=window if window < 1 << 31 else 0)


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
def test_attention_scales(cc, scale, new):
    c = Case([211, 90], [new, new], heads=2, group=2, dim=128, k_gain=2.0, seed=3)
    cache, batch = c.objects(cc)
    out, lse = cc.kv_attention(cache, batch, c.q, scale=scale)
    check(c, out, lse, scale=scale)


@pytest.mark.parametrize("new", [1, 5, 200])
@pytest.mark.parametrize("fmt", ["16bit", "e4m3"])
def test_hints_do_not_change_what_is_computed(cc, fmt, new):
    """max_new and max_len may be wrong: the result keeps to its bounds."""
    c = Case([700, 300, 210], [new] * 3, heads=2, group=4, dim=128, fmt=fmt, seed=9)
    for max_new, max_len in ((1, 1), (1, 100000), (4096, 1), (4096, 100000)):
        cache, batch = c.objects(cc, max_new=max_new, max_len=max_len)
        out, lse = cc.kv_attention(cache, batch, c.q)
        check(c, out, lse)


@pytest.mark.parametrize("over", [{}, CUT])
@pytest.mark.parametrize("new", [1, 64])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_hidden_values_have_no_effect(cc, value, new, over):
    """K and V of hidden positions inside the cache hold what must not be read."""
    c = Case([260], [new], heads=2, group=2, dim=128, page=16, seed=5)
    window = 100
    first_seen = c.lens[0] - new - window + 1
    for p in range(first_seen):
        at = (int(c.table[0, p // 16]), p % 16)
        c.k[at], c.v[at] = value, value
    if new > 1:  # the last new token is seen by the last row alone
        p = c.lens[0] - 1
        c.v[int(c.table[0, p // 16]), p % 16] = value
        c.k[int(c.table[0, p // 16]), p % 16] = value
    cache, batch = c.objects(cc, **over)
    out, lse = cc.kv_attention(cache, batch, c.q, window=window)
    rows = slice(0, c.T - 1) if new > 1 else slice(0, c.T)
    ref, ref_lse, tol, ltol = c.attention(window=window)
    assert torch.isfinite(out[rows]).all()
    assert ((out.double() - ref).abs() <= tol)[rows].all()
    assert ((lse.double() - ref_lse).abs() <= ltol)[rows].all()
    if new > 1:
        assert not torch.isfinite(out[-1]).all()  # where it is visible, it shows


@pytest.mark.parametrize("over", [{}, CUT])
@pytest.mark.parametrize("new", [1, 64])
def test_visible_values_go_where_the_formula_takes_them(cc, new, over):
    c = Case([200], [new], heads=2, group=2, dim=64, page=16, seed=6)
    at = (int(c.table[0, 3]), 2)
    c.v[at][0, 7] = float("inf")  # head 0, one channel
    cache, batch = c.objects(cc, **over)
    out, _ = cc.kv_attention(cache, batch, c.q)
    assert (out[:, :2, 7] == math.inf).all()
    keep = torch.ones(64, dtype=torch.bool, device="cuda")
    keep[7] = False
    ref, _, tol, _ = c.attention()
    assert ((out.double() - ref).abs() <= tol)[:, 2:].all()
    assert ((out.double() - ref).abs() <= tol)[:, :2][..., keep].all()


@pytest.mark.parametrize("over", [{}, CUT])
@pytest.mark.parametrize("new", [1, 64])
def test_large_values_do_not_overflow_on_the_way(cc, new, over):
    """Values near binary32's limit: the mean of equal values is that value."""
    c = Case([500], [new], heads=1, group=2, dim=64, seed=7)
    big = torch.tensor(3e38, device="cuda").to(BF)
    c.v[:] = big
    c.q[:] = 0
    cache, batch = c.objects(cc, **over)
    out, _ = cc.kv_attention(cache, batch, c.q)
    assert (out.float() / big.float() - 1).abs().max() <= 2.0 ** -8


@pytest.mark.parametrize("over", [{}, dict(max_new=32, max_len=600), dict(max_len=4000), dict(max_len=8000)])
@pytest.mark.parametrize("window", [0, 300])
@pytest.mark.parametrize("fmt", ["16bit", "int8", "e4m3"])
def test_few_items_shared_by_blocks(cc, fmt, window, over):
    """Sequences without new tokens, of fewer tiles than an item has blocks, and more rows than the program said."""
    c = Case([900, 40, 0, 513, 130], [200, 33, 0, 64, 1], heads=2, group=4, dim=112, page=16, fmt=fmt, seed=60,
             fill=float("nan"))
    cache, batch = c.objects(cc, **over)
    out, lse = cc.kv_attention(cache, batch, c.q, window=window)
    check(c, out, lse, window=window)


@pytest.mark.parametrize("new", [1, 9, 64, 300])
def test_values_that_are_not_finite_in_shared_items(cc, new):
    c = Case([700], [new], heads=2, group=2, dim=64, page=16, seed=61)
    for p, head, value in ((5, 0, math.inf), (390, 0, math.inf), (390, 1, math.nan)):
        c.v[(int(c.table[0, p // 16]), p % 16)][head, 7] = value
    cache, batch = c.objects(cc)
    out, _ = cc.kv_attention(cache, batch, c.q)
    assert (out[:, :2, 7] == math.inf).all() and torch.isnan(out[:, 2:, 7]).all()
    keep = torch.arange(64, device="cuda") != 7
    c.v.nan_to_num_(0.0, 0.0, 0.0)
    ref, _, tol, _ = c.attention()
    assert ((out.double() - ref).abs() <= tol)[..., keep].all()


def test_strided_queries_outputs_and_guards(cc):
    """q and out as slices of wider tensors; nothing around the output changes."""
    for new in (1, 50):
        c = Case([400, 60], [new, new], heads=2, group=4, dim=128, seed=8)
        wide = torch.full((c.T, 3, 8, 128), 7.0, dtype=BF, device="cuda")
        wide[:, 1] = c.q
        frame = torch.full((c.T + 2, 10, 144), 3.0, dtype=BF, device="cuda")
        out = frame[1:-1, 1:-1, 8:136]
        lse = torch.empty(c.T, 8, device="cuda")
        cache, batch = c.objects(cc)
        ws = cc.empty_kv_workspace(cache, batch, 8)
        cc.cccl_kv_attention(cache, batch, wide[:, 1], out, ws, lse=lse)
        assert cc.cccl_get_result(ws)[1] == 0
        check(c, out, lse)
        mask = torch.ones_like(frame, dtype=torch.bool)
        mask[1:-1, 1:-1, 8:136] = False
        assert (frame[mask] == 3.0).all()


def test_rows_of_no_sequence_are_left_alone(cc):
    c = Case([100, 50], [2, 3], heads=2, group=2, dim=64, seed=11)
    extra = 4
    q = torch.cat([c.q, c.q[:extra]])
    out = torch.full_like(q, 5.0)
    fmt_cache, _ = c.objects(cc)
    batch = cc.KvBatch(c.table, c.cu, c.len_dev, n_tokens=c.T + extra, max_new=3, max_len=100)
    ws = cc.empty_kv_workspace(fmt_cache, batch, 4)
    cc.cccl_kv_attention(fmt_cache, batch, q, out, ws)
    lse = torch.empty(c.T, 4, device="cuda")
    ref, _, tol, _ = c.attention()
    assert ((out[:c.T].double() - ref).abs() <= tol).all()
    assert (out[c.T:] == 5.0).all()
    k, v = cc.kv_read(fmt_cache, cc.KvBatch(c.table, c.cu, c.len_dev, n_tokens=c.T, max_new=3, max_len=100))
    assert k.shape == (c.T, 2, 64) and lse.shape == (c.T, 4)


def test_device_errors_are_reported_and_clamped(cc):
    """Table entries outside the pool, lengths past the table, cu_tokens past the rows."""
    for new in (1, 40):
        c = Case([200, 90], [new, new], heads=2, group=2, dim=64, seed=12)
        cache, batch = c.objects(cc)
        good, _ = cc.kv_attention(cache, batch, c.q)
        for spoil in ("page", "negative page", "length", "negative length", "cu", "cu order"):
            table, cu, lens = c.table.clone(), c.cu.clone(), c.len_dev.clone()
            if spoil == "page":
                table[1, 2] = c.pages
            elif spoil == "negative page":
                table[1, 0] = -1
            elif spoil == "length":
                lens[1] = 100000
            elif spoil == "negative length":
                lens[1] = -5
            elif spoil == "cu":
                cu[2] = 2 * new + 1000
            else:
                cu[2] = 0
            bad = cc.KvBatch(table, cu, lens, n_tokens=c.T, max_new=new, max_len=200)
            ws = cc.empty_kv_workspace(cache, bad, 4)
            out = torch.zeros_like(c.q)
            cc.cccl_kv_attention(cache, bad, c.q, out, ws)
            assert cc.cccl_get_result(ws)[1] == cc.CCCL_ERR_INVALID_ARG, spoil
            assert torch.equal(out[:new], good[:new]), spoil  # sequence 0 is whole
            # the status stays until it is cleared
            cc.cccl_kv_attention(cache, batch, c.q, out, ws)
            assert cc.cccl_get_result(ws)[1] == cc.CCCL_ERR_INVALID_ARG
            assert torch.equal(out, good)
            cc.cccl_kv_clear_status(ws)
            assert cc.cccl_get_result(ws)[1] == 0
            with pytest.raises(cc.CcclError):
                cc.kv_attention(cache, bad, c.q)
            if spoil != "cu order":
                ws = cc.empty_kv_workspace(cache, bad)
                ko, vo = (torch.empty(c.T, 2, 64, dtype=BF, device="cuda") for _ in range(2))
                cc.cccl_kv_read(cache, bad, ko, vo, ws)
                # a read meets a bad page only where its rows lie
                if spoil not in ("page", "negative page") or new == 40 and spoil == "page":
                    assert cc.cccl_get_result(ws)[1] == (0 if spoil == "page" and 90 - 40 > 47 else
                                                        cc.CCCL_ERR_INVALID_ARG), spoil


def test_refusals_on_the_gpu(cc):
    """Buffers that are too small, not aligned, or not in one allocation: refused, and nothing runs."""
    c = Case([100], [4], heads=2, group=2, dim=64, seed=16)
    cache, batch = c.objects(cc)
    ws = cc.empty_kv_workspace(cache, batch, 4)
    out = torch.full_like(c.q, 2.0)

    def refused(f, *a, **kw):
        with pytest.raises(cc.CcclError) as e:
            f(*a, **kw)
        assert e.value.status == cc.CCCL_ERR_INVALID_ARG

    refused(cc.cccl_kv_attention, cache, batch, c.q, out, ws[:-16])
    refused(cc.cccl_kv_attention, cache, batch, c.q, out, ws[4:])
    refused(cc.cccl_kv_attention, cache, batch, c.q, out, ws, window=-1)
    refused(cc.cccl_kv_attention, cache, batch, c.q, out, ws, scale=float("nan"))
    odd = torch.zeros(c.q.numel() + 8, dtype=BF, device="cuda")[1:1 + c.q.numel()].view(c.q.shape)  # 2-byte aligned
    refused(cc.cccl_kv_attention, cache, batch, odd, out, ws)
    refused(cc.cccl_kv_attention, cache, batch, c.q, odd, ws)
    refused(cc.cccl_kv_attention, cache, batch, torch.zeros(c.T, 3, 64, dtype=BF, device="cuda"),
            torch.zeros(c.T, 3, 64, dtype=BF, device="cuda"), ws)  # 3 query heads for 2 kv heads
    host = torch.zeros(c.T, 2, 64, dtype=BF)
    refused(cc.cccl_kv_write, cache, batch, host, host, ws)
    refused(cc.cccl_kv_write, cache, batch, c.k_new, c.v_new, ws[:8])
    assert (out == 2.0).all()
    assert cc.cccl_get_result(ws)[1] == 0


def test_empty_calls_do_nothing(cc):
    c = Case([20], [0], heads=2, dim=64)
    cache, batch = c.objects(cc)
    out, lse = cc.kv_attention(cache, batch, c.q)
    assert out.numel() == 0 and lse.numel() == 0
    cc.kv_write(cache, batch, c.k_new, c.v_new)
    none = cc.KvBatch(c.table[:0], torch.zeros(1, dtype=torch.int32, device="cuda"), c.len_dev[:0], n_tokens=0,
                      max_new=1, max_len=1)
    cc.kv_read(cache, none)


def test_offsets_past_32_bits(cc):
    """A pool of more than 2^32 bytes a side, its last pages in use."""
    page, heads, dim = 64, 8, 128
    pages = (1 << 32) // (page * heads * dim) + 64  # int8: one byte a value
    free, _ = torch.cuda.mem_get_info()
    if free < 3 * pages * page * heads * dim:
        pytest.skip("not enough device memory")
    small = Case([200, 330], [1, 40], heads=heads, group=2, dim=dim, page=page, fmt="int8", seed=13)
    k, v = (torch.empty(pages, page, heads, dim, dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.empty(pages, heads, page, device="cuda").transpose(1, 2) for _ in range(2))
    shift = pages - small.pages
    for far, near in ((k, small.k), (v, small.v), (ks, small.ks), (vs, small.vs)):
        far[shift:] = near
    table = torch.where(small.table < small.pages, small.table + shift, small.table)
    cache, _ = small.objects(cc)
    batch = cc.KvBatch(table, small.cu, small.len_dev, n_tokens=small.T, max_new=40, max_len=330)
    far = cc.KvCache(k, v, ks, vs, dtype=BF, fmt=cc.CCCL_KV_INT8)
    out, lse = cc.kv_attention(far, batch, small.q)
    check(small, out, lse)
    near_k, near_v = cc.kv_read(cache, small.objects(cc)[1])
    far_k, far_v = cc.kv_read(far, batch)
    assert same_bits(near_k, far_k) and same_bits(near_v, far_v)
    cc.kv_write(far, batch, small.k_new, small.v_new)
    cc.kv_write(cache, small.objects(cc)[1], small.k_new, small.v_new)
    assert same_bits(k[shift:], small.k) and same_bits(vs[shift:], small.vs)


@pytest.mark.parametrize("new", [1, 130])
def test_repeated_calls_streams_and_graphs_agree(cc, new):
    """The same bits on every call, on another stream, and from a graph's replays."""
    c = Case([3000, 700, 64 + new], [new] * 3, heads=2, group=4, dim=128, fmt="int8", seed=14)
    cache, batch = c.objects(cc)
    first, _ = cc.kv_attention(cache, batch, c.q)
    for _ in range(3):
        assert torch.equal(cc.kv_attention(cache, batch, c.q)[0], first)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out, _ = cc.kv_attention(cache, batch, c.q, stream=side)
    assert torch.equal(out, first)
    ws = cc.empty_kv_workspace(cache, batch, 8)
    out = torch.zeros_like(c.q)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cc.cccl_kv_write(cache, batch, c.k_new, c.v_new, ws)
        cc.cccl_kv_attention(cache, batch, c.q, out, ws)
    graph.replay()
    torch.cuda.synchronize()
    after = out.clone()
    check_new = cc.kv_attention(cache, batch, c.q)
    assert torch.equal(after, check_new[0])
    check(c, *check_new)
    c.q.copy_(torch.randn_like(c.q.float()).to(BF))  # new inputs, the same graph
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, cc.kv_attention(cache, batch, c.q)[0])


def test_limits_of_e4m3_codes(cc):
    """Every code, with scales that are and are not powers of two."""
    codes = torch.arange(256, device="cuda").to(torch.uint8).view(torch.int8)
    codes = torch.where(codes.view(torch.uint8) & 0x7F == 0x7F, torch.zeros_like(codes), codes)  # NaN codes out
    c = Case([4], [4], heads=1, group=1, dim=64, page=4, fmt="e4m3", seed=15)
    for rows in (c.k, c.v):
        for p in range(4):
            rows[int(c.table[0, 0]), p, 0] = codes[64 * p:64 * p + 64]
    cache, batch = c.objects(cc)
    k, v = cc.kv_read(cache, batch)
    ref_k, ref_v = c.stored(0)
    for got, ref in ((k, ref_k), (v, ref_v)):
        assert ((got.double() - ref).abs() <= ref.abs() * UNIT[BF]).all()
    out, lse = cc.kv_attention(cache, batch, c.q)
    check(c, out, lse)
    assert LIMIT["e4m3"] == 448.0
