"""Attention of drafted tokens on the GPU against its definition in binary64
(the bounds are kv_reference's: the kernels are those of causal attention)."""

import random

import pytest
import torch

from step_reference import TreeCase, ancestors, trees

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16
CUT = dict(max_len=1 << 20)  # what makes a call cut items among blocks and join their parts


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
    assert torch.isfinite(out[torch.isfinite(ref).all(-1)]).all()
    assert ((out.double() - ref).abs() <= tol).all(), ((out.double() - ref).abs() - tol).max()
    empty = ref_lse == -float("inf")
    assert torch.equal(lse == -float("inf"), empty)
    assert ((lse.double() - ref_lse).abs() <= ltol)[~empty].all()
    assert not out[empty].any()


def attend(cc, c, over=None, **kw):
    cache, batch = c.objects(cc, **(over or {}))
    out, lse = cc.step_attention(cache, batch, c.q, c.mask, **kw)
    return out, lse


SHAPES = [
    # lens, new, heads, group, dim, page
    ([1], [1], 1, 1, 16, 1),
    ([517], [5], 2, 4, 128, 16),
    ([33, 7, 200], [16, 7, 1], 2, 2, 64, 16),
    ([700, 70, 0, 5], [33, 64, 0, 5], 1, 4, 128, 24),
    ([1100, 129], [61, 2], 2, 8, 96, 64),
    ([300, 128], [40, 100], 2, 3, 80, 7),
    ([90, 260], [90, 130], 1, 1, 112, 128),
    ([5, 40], [9, 60], 2, 2, 64, 16),  # more drafted tokens than cached ones: some lie before position 0
    ([2100], [17], 1, 16, 128, 32),
]


@pytest.mark.parametrize("fmt", ["16bit", "int8", "e4m3"])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("shape", range(len(SHAPES)))
def test_trees(cc, shape, dtype, fmt):
    lens, new, heads, group, dim, page = SHAPES[shape]
    c = TreeCase(lens, new, heads=heads, group=group, dim=dim, page=page, dtype=dtype, fmt=fmt, seed=shape,
                 layout=["thd", "htd", "kv"][shape % 3], fill=float("nan"), mask_pad=shape % 2)
    # (the last two: the kernel for many rows, whatever their number, and the one for few)
    for over in ({}, CUT, dict(max_new=500), dict(max_new=1, max_len=1)):
        check(c, *attend(cc, c, over))


@pytest.mark.parametrize("fmt", ["16bit", "int8"])
@pytest.mark.parametrize("new", [3, 40])
def test_any_masks(cc, new, fmt):
    """Masks that are no tree's: random bits, nobody, everybody, not itself; sequences without cached tokens."""
    r = random.Random(new)
    lens = [new, new + 1, 4 * new, 200, new]
    bits = [[r.getrandbits(new) for _ in range(new)] for _ in lens]
    bits[0][0] = bits[1][1] = bits[0][new - 1] = bits[3][0] = 0
    bits[2][1] = (1 << new) - 1
    bits[4] = [1 << (new - 1 - i) for i in range(new)]
    c = TreeCase(lens, [new] * len(lens), bits, heads=2, group=3, dim=64, fmt=fmt, seed=new, fill=float("inf"))
    for over in ({}, CUT, dict(max_new=500)):
        out, lse = attend(cc, c, over)
        check(c, out, lse)
        assert not out[0].any() and (lse[0] == -float("inf")).all()  # nothing cached, no bit set


@pytest.mark.parametrize("new,words", [(70, 1), (70, 2), (33, 1), (40, 5), (200, 7)])
def test_words_of_masks(cc, new, words):
    """Tokens behind the last word are seen by none; words behind the last token take no part."""
    bits = [[(1 << 32 * words) - 1 if i % 3 == 0 else m for i, m in enumerate(ancestors(trees([new], 3)[0]))],
            [(1 << 32 * words) - 1] * 5]
    c = TreeCase([new + 30, 9], [new, 5], bits, words=words, heads=1, group=2, dim=64, seed=words, fill=float("nan"))
    for over in ({}, CUT):
        check(c, *attend(cc, c, over))


@pytest.mark.parametrize("window", [1, 2, 5, 17, 64, 130, 1 << 40])
@pytest.mark.parametrize("new", [4, 45])
def test_windows(cc, new, window):
    """The last tokens of a row's own path, whether the window ends before the draft or in it."""
    c = TreeCase([new, new + 3, 300, 1000], [new] * 4, heads=1, group=4, dim=64, seed=window % 97, fill=float("nan"))
    c.bits[2][0] = 0  # sees cached tokens alone
    c.mask[2 * new] = 0
    for over in ({}, CUT, dict(max_new=500)):
        out, lse = attend(cc, c, over, window=window)
        check(c, out, lse, window=window if window < 1 << 31 else 0)


@pytest.mark.parametrize("new", [6, 50])
@pytest.mark.parametrize("fmt", ["16bit", "e4m3"])
def test_what_hidden_tokens_hold_has_no_effect(cc, fmt, new):
    """A drafted token's NaN or infinity reaches the rows that see it and no others."""
    c = TreeCase([new + 100], [new], heads=2, group=2, dim=64, fmt=fmt, seed=new, page=16)
    bad, t = new // 2, new + 100
    at = (int(c.table[0, (t - new + bad) // 16]), (t - new + bad) % 16)
    if fmt == "16bit":
        c.k[at], c.v[at] = float("nan"), float("inf")
    else:
        c.ks[at], c.vs[at] = float("nan"), float("nan")
    sees = torch.tensor([m >> bad & 1 for m in c.bits[0]], dtype=torch.bool)
    assert sees.any() and not sees.all()
    ref, _, tol, _ = c.attention()
    for over in ({}, CUT, dict(max_new=500)):
        out, _ = attend(cc, c, over)
        assert out[sees].isnan().all()
        assert ((out.double() - ref).abs() <= tol)[~sees].all()


@pytest.mark.parametrize("fmt", ["16bit", "int8"])
def test_a_chain_is_causal_attention(cc, fmt):
    """Masks of a chain give what the causal call gives (the kernels may divide the work otherwise: both keep to
    the definition's bounds)."""
    for new in (1, 4, 60):
        c = TreeCase([400, 60], [new, new], [[(2 << i) - 1 for i in range(new)]] * 2, heads=2, group=4, dim=128, fmt=fmt,
                     seed=5)
        out, lse = attend(cc, c)
        check(c, out, lse)
        cache, batch = c.objects(cc)
        other, other_lse = cc.kv_attention(cache, batch, c.q)
        _, _, tol, ltol = c.attention()
        assert ((out.double() - other.double()).abs() <= 2 * tol).all()
        assert ((lse.double() - other_lse.double()).abs() <= 2 * ltol).all()


@pytest.mark.parametrize("scale", [0.0, -0.4, 3.0])
def test_scales(cc, scale):
    for new in (3, 40):
        c = TreeCase([150, 90], [new, new], heads=2, group=2, dim=64, k_gain=2.0, seed=3)
        out, lse = attend(cc, c, scale=scale)
        check(c, out, lse, scale=scale)


def test_many_sequences(cc):
    lens = [(7 * b) % 61 for b in range(1024)]
    new = [min(n, 1 + b % 9) if b % 5 else 0 for b, n in enumerate(lens)]
    c = TreeCase(lens, new, heads=1, group=2, dim=64, fmt="int8", seed=40)
    for over in ({}, CUT, dict(max_new=500)):
        check(c, *attend(cc, c, over))


def test_strides_and_rows_of_no_sequence(cc):
    """Slices of fused tensors; rows before the first and behind the last sequence stay as they are."""
    c = TreeCase([200, 40], [12, 12], heads=2, group=2, dim=64, seed=9)
    cache, _ = c.objects(cc)
    rows = c.T + 7
    fused = torch.zeros(rows, 6, 64, dtype=BF, device="cuda")
    fused[3:3 + c.T, 1:5] = c.q
    out = torch.full((rows, 9, 64), 7.0, dtype=BF, device="cuda")
    mask = torch.zeros(rows, 3, dtype=torch.int32, device="cuda")
    mask[3:3 + c.T, 1:2] = c.mask
    lse = torch.full((rows, 4), 5.0, device="cuda")
    batch = cc.KvBatch(c.table, c.cu + 3, c.len_dev, n_tokens=rows, max_new=12, max_len=200)
    ws = cc.empty_kv_workspace(cache, batch, 4)
    cc.cccl_step_attention(cache, batch, fused[:, 1:5], mask[:, 1:2], out[:, 2:6], ws, lse=lse)
    assert cc.cccl_get_result(ws)[1] == 0
    check(c, out[3:3 + c.T, 2:6], lse[3:3 + c.T])
    keep = torch.ones(rows, 9, dtype=torch.bool, device="cuda")
    keep[3:3 + c.T, 2:6] = False
    assert (out[keep] == 7).all() and (lse[:3] == 5).all() and (lse[3 + c.T:] == 5).all()


def test_same_bits_again_and_in_a_graph(cc):
    for lens, new in (([900, 333], [5, 5]), ([900, 333, 80], [40, 33, 64])):
        c = TreeCase(lens, new, heads=2, group=4, dim=128, seed=2)
        for over in ({}, CUT):
            cache, batch = c.objects(cc, **over)
            ws = cc.empty_kv_workspace(cache, batch, 8)
            out = torch.empty_like(c.q)
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                cc.cccl_step_attention(cache, batch, c.q, c.mask, out, ws)
                side.synchronize()
                first = out.clone()
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph, stream=side):
                    cc.cccl_step_attention(cache, batch, c.q, c.mask, out, ws)
            for _ in range(3):
                out.zero_()
                graph.replay()
                torch.cuda.synchronize()
                assert torch.equal(out, first)
            # the masks and lengths are read when the graph runs
            kept = c.mask.clone()
            c.mask.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert not torch.equal(out, first)
            c.mask.copy_(kept)


def test_reported_errors(cc):
    c = TreeCase([100, 50], [8, 8], heads=1, group=2, dim=64, seed=1)
    for entry in (-1, 1 << 30):
        kept = c.table.clone()
        c.table[0, 1] = entry
        with pytest.raises(cc.CcclError):
            attend(cc, c)
        c.table.copy_(kept)
    for at, bad in ((0, -5), (1, 1 << 30)):
        kept = c.len_dev.clone()
        c.len_dev[at] = bad
        with pytest.raises(cc.CcclError):
            attend(cc, c)
        c.len_dev.copy_(kept)
    check(c, *attend(cc, c))


@pytest.mark.parametrize("fmt", ["16bit", "int8"])
def test_long_contexts(cc, fmt):
    """One tree of several row tiles a head, with as many blocks for each; few rows over many tiles."""
    for lens, new, heads, group in (([20011], [61], 2, 8), ([9000], [3], 1, 4), ([12345, 700], [33, 33], 2, 4)):
        c = TreeCase(lens, new, heads=heads, group=group, dim=128, page=64, fmt=fmt, seed=len(lens))
        check(c, *attend(cc, c))
