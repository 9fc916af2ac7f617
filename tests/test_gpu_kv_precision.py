"""What the paged cache's attention may be off by, from the number formats alone:
rows in which one key outweighs the rest, values whose sizes differ from token to
token, and the precision of calls with few rows."""

import math

import pytest
import torch

from kv_reference import TINY, UNIT, Case, quantise

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
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


def put(c, which, b, pos, x, head=slice(None)):
    """Store x[..., dim] as the keys ("k") or values ("v") of one position."""
    at = (int(c.table[b, pos // c.page]), pos % c.page)
    x = x.to(c.dtype)
    if c.fmt == "16bit":
        getattr(c, which)[at][head] = x
    else:
        codes, scale = quantise(x, c.fmt)
        getattr(c, which)[at][head] = codes
        getattr(c, which + "s")[at][head] = scale


def few_rows(c):
    """Whether the call takes the kernel for few rows a kv head."""
    return c.group * max(c.new) <= (24 if c.fmt == "16bit" else 32)


def bounds(c, window=0):
    """Result in binary64, and what a kernel may be off by:

    - a score by d = (dim + 8) 2^-23 scale sum |q k| (any order of binary32 sums,
      the scale's and the key scale's products); a probability by 2 d (its score,
      the maximum's) + 2^-20 (the exponential and its argument), relatively, and
      again through the sum of all;
    - binary32 sums over L keys (any order): (L + 16) 2^-24 of the sum of sizes,
      for numerator and denominator;
    - a probability's rounding for the second product: calls with few rows hold it
      as the sum of two 16-bit values (bf16 2^-16, fp16 2^-22), others as one
      (2^-8, 2^-11); 8-bit caches and fp16 ones take fp16, whose smallest step adds
      2^-25 of a largest probability (times its value's scale) of 2^14 (few rows)
      or 2^9 (others; over 8-bit caches 2^5);
    - the result's one rounding."""
    half = c.dtype == HF or c.fmt != "16bit"
    few = few_rows(c)
    p_unit = (2.0 ** -22 if half else 2.0 ** -16) if few else (2.0 ** -11 if half else 2.0 ** -8)
    p_floor = (2.0 ** -39 if few else 2.0 ** -34 if c.fmt == "16bit" else 2.0 ** -30) if half else 0.0
    u, scale, G = UNIT[c.dtype], 1.0 / math.sqrt(c.dim), c.group
    out = torch.zeros(c.T, c.heads * G, c.dim, dtype=torch.float64, device=c.device)
    tol = torch.zeros_like(out)
    row = 0
    for b, n in enumerate(c.new):
        k, v = c.stored(b)
        seen = c.visible(b, True, window)
        vs = torch.ones(c.lens[b], c.heads, dtype=torch.float64, device=c.device)
        if c.fmt != "16bit":
            rows = c.table[b, :-(-c.lens[b] // c.page)].long()
            vs = c.vs[rows].flatten(0, 1)[:c.lens[b]].double().abs()
        for h in range(c.heads * G):
            q = c.q[row:row + n, h].double()
            kk, vv, sc = k[:, h // G], v[:, h // G], vs[:, h // G]
            hidden = ~seen.any(0)  # what no row sees may hold anything
            kk = torch.where(hidden[:, None], 0.0, kk)
            s = torch.where(seen, q @ kk.T * scale, -math.inf)
            p = torch.softmax(s, -1)
            clean = torch.nan_to_num(torch.where(hidden[:, None], 0.0, vv), 0.0, 0.0, 0.0)
            o, av = p @ clean, p @ clean.abs()
            largest = torch.where(seen, p, 0.0).amax(1, keepdim=True) * torch.where(seen, sc, 0.0).amax(1, keepdim=True)
            codes = clean.abs() / torch.where(sc > 0, sc, 1.0)[:, None]
            floor = p_floor * largest * (seen.double() @ codes)
            mag = torch.where(seen, q.abs() @ kk.abs().T, 0.0).amax(1, keepdim=True) * scale
            d = (c.dim + 8) * 2.0 ** -23 * mag
            rel = 2 * (2 * d + 2.0 ** -20) + 2 * (c.lens[b] + 16) * 2.0 ** -24 + p_unit
            e = rel * av + floor
            out[row:row + n, h], tol[row:row + n, h] = o, e + u * (o.abs() + e) + TINY[c.dtype]
        row += n
    return out, tol


def check(c, out, window=0, rows=slice(None)):
    ref, tol = bounds(c, window)
    err = (out.double() - ref).abs()[rows]
    assert torch.isfinite(out[rows]).all()
    assert (err <= tol[rows]).all(), "worst %g of its bound" % (err / tol[rows]).max()


TYPES = [(HF, "16bit"), (BF, "16bit"), (BF, "int8"), (HF, "int8"), (BF, "e4m3")]


def axis_case(length, new, dtype, fmt, **kw):
    """Every query is 8 along channel 0 (and small elsewhere), every key 0 there: a key's score is chosen by that
    channel; values are positive."""
    c = Case([length], [new], heads=2, group=4, dim=128, page=16, dtype=dtype, fmt=fmt, fill=0.0 if fmt == "16bit" else None,
             **kw)
    g = torch.Generator(device="cuda").manual_seed(kw.get("seed", 0) + 1)
    c.q = (0.3 * torch.randn(c.q.shape, generator=g, device="cuda")).to(dtype)
    c.q[..., 0] = 8
    for p in range(length):
        k = 0.5 * torch.randn(2, 128, generator=g, device="cuda")
        k[:, 0] = 0
        put(c, "k", 0, p, k)
        put(c, "v", 0, p, 0.5 + torch.rand(2, 128, generator=g, device="cuda"))
    return c


def axis_key(nats):
    """A key whose score with those queries is `nats`."""
    k = torch.zeros(2, 128, device="cuda")
    k[:, 0] = nats * 128 ** 0.5 / 8
    return k


@pytest.mark.parametrize("length,new", [(700, 1), (700, 64), (3000, 1), (1500, 2), (3000, 64)])
@pytest.mark.parametrize("dtype,fmt", TYPES)
def test_one_key_outweighs_the_rest(cc, dtype, fmt, length, new):
    """The first key has nearly all of the weight and a value of zero: the result is what the others leave."""
    c = axis_case(length, new, dtype, fmt, seed=80)
    for nats in (12, 15, 18):
        put(c, "k", 0, 0, axis_key(nats))
        put(c, "v", 0, 0, torch.zeros(2, 128, device="cuda"))
        for over in ({}, CUT, dict(max_len=2000)):
            cache, batch = c.objects(cc, **over)
            check(c, cc.kv_attention(cache, batch, c.q)[0])


@pytest.mark.parametrize("new", [1, 2, 64])
@pytest.mark.parametrize("dtype,fmt", [(BF, "int8"), (HF, "int8"), (BF, "e4m3"), (HF, "e4m3"), (HF, "16bit")])
def test_one_value_far_larger_than_the_rest(cc, dtype, fmt, new):
    """It has next to no weight, or only the last row sees it: the other values keep their bits."""
    length = 700
    small, large = (1.0, 2.0 ** 20) if dtype == BF else (2.0 ** -12, 2.0 ** 8)
    for where in ("faint", "last"):
        c = axis_case(length, new, dtype, fmt, seed=81)
        for p in range(length):
            put(c, "v", 0, p, small * (0.5 + torch.rand(2, 128, device="cuda")))
        big = large * (0.5 + torch.rand(2, 128, device="cuda"))
        if where == "faint":
            put(c, "k", 0, 600, axis_key(-40))
            put(c, "v", 0, 600, big)
        elif new > 1:
            put(c, "v", 0, length - 1, big)
        for over in ({}, CUT):
            cache, batch = c.objects(cc, **over)
            out, _ = cc.kv_attention(cache, batch, c.q)
            check(c, out)
            if where == "last" and fmt != "16bit" and dtype == BF and new > 1:
                # of any size: nothing of it reaches the other rows
                scales = c.vs.clone()
                for junk in (1e30, 3e38, math.inf, math.nan, -1e30):
                    c.vs[int(c.table[0, (length - 1) // 16]), (length - 1) % 16] = junk
                    got, _ = cc.kv_attention(cache, batch, c.q)
                    c.vs.copy_(scales)
                    check(c, got, rows=slice(0, new - 1))


@pytest.mark.parametrize("new", [1, 64])
@pytest.mark.parametrize("dtype,fmt", [(BF, "int8"), (HF, "int8"), (BF, "e4m3"), (BF, "16bit"), (HF, "16bit")])
def test_values_of_many_sizes(cc, dtype, fmt, new):
    """Every token's values have a size of their own, and (8-bit caches) a scale of either sign."""
    c = axis_case(600, new, dtype, fmt, seed=82)
    g = torch.Generator(device="cuda").manual_seed(83)
    span = 12 if dtype == BF else 6
    for p in range(600):
        size = 2.0 ** float(torch.randint(-span, span + 1, (1,), generator=g, device="cuda"))
        put(c, "v", 0, p, size * torch.randn(2, 128, generator=g, device="cuda"))
        put(c, "k", 0, p, axis_key(0) + 2 * torch.randn(2, 128, generator=g, device="cuda"))
    if fmt != "16bit":
        c.vs[:, ::2] *= -1
    for over in ({}, CUT):
        cache, batch = c.objects(cc, **over)
        check(c, cc.kv_attention(cache, batch, c.q)[0])


@pytest.mark.parametrize("new", [1, 64])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("power", [-85, 95])
def test_value_scales_of_any_size(cc, fmt, power, new):
    c = axis_case(500, new, BF, fmt, seed=84)
    c.vs *= 2.0 ** power
    for over in ({}, CUT):
        cache, batch = c.objects(cc, **over)
        check(c, cc.kv_attention(cache, batch, c.q)[0])


def opposed(dtype, fmt, new, device="cuda"):
    """Few keys of like weight whose values nearly cancel: what a probability is rounded by shows in the result."""
    lens = [2, 3, 4, 5, 6, 9, 12, 16] * 4
    c = Case(lens, [min(new, n) for n in lens], heads=4, group=4, dim=16, page=16, dtype=dtype, fmt=fmt, seed=85, device=device)
    g = torch.Generator(device=device).manual_seed(86)
    for b, n in enumerate(lens):
        # K and V of one size: 8-bit codes are the same for all but their signs
        sign = torch.where(torch.arange(n) % 2 == 0, 1.0, -1.0)
        for p in range(n):
            k = torch.randint(0, 2, (4, 16), generator=g, device=device) * 1.0 - 0.5
            put(c, "k", b, p, k)
            put(c, "v", b, p, torch.full((4, 16), 1.0, device=device) * float(sign[p]))
    c.q = (0.5 * torch.randn(c.q.shape, generator=g, device=device)).to(dtype)
    return c


@pytest.mark.parametrize("dtype,fmt", TYPES)
def test_few_rows_keep_their_probabilities(cc, dtype, fmt):
    c = opposed(dtype, fmt, 1)
    assert few_rows(c)
    for over in ({}, CUT):
        cache, batch = c.objects(cc, **over)
        check(c, cc.kv_attention(cache, batch, c.q)[0])


@pytest.mark.parametrize("length,new", [(131077, 1), (70001, 150)])
@pytest.mark.parametrize("dtype,fmt", TYPES)
def test_long_contexts(cc, dtype, fmt, length, new):
    c = Case([length], [new], heads=1, group=4, dim=64, page=16, dtype=dtype, fmt=fmt, seed=87)
    cache, batch = c.objects(cc)
    check(c, cc.kv_attention(cache, batch, c.q)[0])
