"""A step with drafted tokens on the GPU against the definitions of
step_reference: plan, write with rotary positions, verify, keep, and a run of
all of them."""

import random

import pytest
import torch

import step_reference as ref
from kv_reference import LIMIT, TINY, UNIT, Case, codes64

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


def ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def same_bits(a, b):
    return torch.equal(a.contiguous().flatten().view(torch.uint8), b.contiguous().flatten().view(torch.uint8))


# ------------------------------------------------------------------ plan
class Plan:
    """Sequences that hold pages, and what joins them."""

    def __init__(self, cc, lens, new, page, *, tree=True, words=None, spare=5, width=None, extra_rows=0, seed=0, over=0.3):
        r = random.Random(seed)
        B = len(lens)
        self.lens, self.new, self.page = list(lens), list(new), page
        self.held = [-(-n // page) + (1 if r.random() < over else 0) for n in lens]
        need = [max(0, -(-(n + m) // page) - h) for n, m, h in zip(lens, new, self.held)]
        self.width = width or max([h + n for h, n in zip(self.held, need)] + [1])
        pages = list(range(sum(self.held) + sum(need) + spare))
        r.shuffle(pages)
        self.table = [[pages.pop() for _ in range(h)] + [-9] * (self.width - h) for h in self.held]
        self.free, self.count = pages + [-7, -7], len(pages)
        self.rows = sum(new) + extra_rows
        self.parents = [p for ps in ref.trees(new, seed) for p in ps] + [-5] * extra_rows if tree else None
        self.words = words
        self.dev()
        self.cc = cc

    def dev(self):
        self.d = {"lens": ints(self.lens), "new": ints(self.new), "held": ints(self.held), "free": ints(self.free),
                  "count": ints([self.count]), "table": ints(self.table)}
        if self.parents is not None:
            self.d["parents"] = ints(self.parents)

    def run(self, in_place=True):
        """The plan's outputs as lists (those behind the last row included) and the status."""
        cc, d = self.cc, self.d
        tables = cc.StepTables(d["table"], d["held"], d["free"], d["count"], page_tokens=self.page)
        ws = cc.empty_step_workspace()
        o = {"cu_tokens": torch.full((len(self.lens) + 1,), -3, dtype=torch.int32, device="cuda"),
             "slots": torch.full((self.rows,), -3, dtype=torch.int64, device="cuda"),
             "positions": torch.full((self.rows,), -3, dtype=torch.int32, device="cuda")}
        o["kv_lens"] = d["lens"] if in_place else torch.empty_like(d["lens"])
        if not in_place:
            o["held"], o["free_count"] = torch.empty_like(d["held"]), torch.empty_like(d["count"])
        if self.words:
            o["mask"] = torch.full((self.rows, self.words + 2), -3, dtype=torch.int32, device="cuda")[:, 1:-1]
        cc.cccl_step_plan(tables, d["lens"], d["new"], ws, parents=d.get("parents"), rows=self.rows, **o)
        status = cc.cccl_get_result(ws)[1]
        o.setdefault("held", d["held"])
        o.setdefault("free_count", d["count"])
        got = {k: v.tolist() for k, v in o.items()}
        got["table"] = d["table"].tolist()
        return got, status

    def want(self):
        return ref.plan(self.lens, self.new, self.held, self.table, self.free, self.count, self.page, self.parents,
                        self.rows, self.width, self.words or 0)


PLANS = [
    # lens, new, page
    ([0], [1], 16),
    ([15, 16, 17, 0], [1, 1, 1, 0], 16),
    ([100, 3, 0, 77, 64], [33, 5, 64, 0, 32], 24),
    ([9, 9, 9], [0, 0, 0], 8),
    ([50] * 40, [b % 7 for b in range(40)], 1),
    ([1000, 5], [700, 3000], 128),
    ([b % 50 for b in range(1024)], [b % 11 for b in range(1024)], 7),
]


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("kind", ["tree", "chain", "prompt"])
@pytest.mark.parametrize("shape", range(len(PLANS)))
def test_plan(cc, shape, kind, in_place):
    lens, new, page = PLANS[shape]
    if kind != "prompt":
        new = [min(n, 1024) for n in new]
    words = None if kind == "prompt" else max(1, -(-max(new) // 32)) + shape % 2
    p = Plan(cc, lens, new, page, tree=kind == "tree", words=words and min(words, 32), extra_rows=shape, seed=shape)
    want = p.want()
    got, status = p.run(in_place)
    assert status == 0
    T = sum(new)
    for k in ("table", "cu_tokens", "kv_lens", "held", "free_count"):
        assert got[k] == want[k], k
    for k in ("slots", "positions") + (("mask",) if p.words else ()):
        assert got[k][:T] == want[k], k
        behind = [-3] * p.words if k == "mask" else -3
        assert got[k][T:] == [behind] * (p.rows - T), k


def test_plan_without_masks_has_the_trees_positions(cc):
    p = Plan(cc, [30, 4], [9, 50], 16, words=None, seed=4)
    got, status = p.run()
    want = p.want()
    assert status == 0 and got["positions"] == want["positions"] and got["slots"] == want["slots"]


def test_plan_twice_in_place_goes_on_from_there(cc):
    p = Plan(cc, [10, 0, 31], [5, 40, 1], 16, words=2, spare=30, width=12, seed=1)
    first = p.want()
    got, _ = p.run()
    assert got["held"] == first["held"] and got["free_count"] == first["free_count"]
    p.lens, p.held, p.table, p.count = first["kv_lens"], first["held"], first["table"], first["free_count"][0]
    second = p.want()
    got, status = p.run()
    assert status == 0
    for k in ("table", "cu_tokens", "kv_lens", "held", "free_count", "slots", "positions", "mask"):
        assert got[k] == second[k], k


@pytest.mark.parametrize("what", ["lens", "new", "held", "held_high", "count", "count_high", "table", "rows", "words", "free", "tree"])
def test_plan_gives_nothing_where_something_does_not_fit(cc, what):
    p = Plan(cc, [10, 20, 30], [5, 40, 1] if what != "tree" else [5, 1025, 1], 16, words=2 if what != "tree" else None,
             spare=0 if what == "free" else 4, seed=3, over=0.0)
    status = cc.CCCL_ERR_INVALID_ARG
    if what == "lens":
        p.lens[1] = -1
    elif what == "new":
        p.new[2] = -1
    elif what == "held":
        p.held[0] = -1
    elif what == "held_high":
        p.held[0] = p.width + 1
    elif what == "count":
        p.count = -1
    elif what == "count_high":
        p.count = len(p.free) + 1
    elif what == "table":
        p.lens[0] = p.width * 16 - 4
    elif what == "rows":
        p.rows -= 1
        p.parents.pop()
    elif what == "words":
        p.words = 1
    elif what == "free":
        p.count -= 1
        status = cc.CCCL_ERR_CAPACITY
    p.dev()
    assert p.want() == ("capacity" if what == "free" else "invalid")
    got, seen = p.run()
    assert seen == status
    assert got["cu_tokens"] == [0, 0, 0, 0] and got["kv_lens"] == p.lens and got["held"] == p.held
    assert got["free_count"] == [p.count] and got["table"] == p.table
    assert set(got["slots"]) == set(got["positions"]) == {-3}


def test_plan_takes_parents_that_are_not_earlier_as_none(cc):
    p = Plan(cc, [8, 8], [4, 4], 16, words=1, seed=2)
    p.parents = [-1, 1, 0, 9, -1, -4, 1, 2]
    p.dev()
    got, status = p.run()
    assert status == cc.CCCL_ERR_INVALID_ARG
    assert [m[0] for m in got["mask"]] == [1, 2, 5, 8, 1, 2, 6, 14]
    assert got["positions"] == [8, 8, 9, 8, 8, 8, 9, 10]


def test_a_plan_in_a_graph_reads_lengths_when_it_runs(cc):
    tables = cc.StepTables.empty(2, 10, 20, 16)
    lens, new = ints([0, 0]), ints([20, 3])
    out = {"cu_tokens": ints([0] * 3), "kv_lens": lens, "slots": ints([0] * 40, torch.int64), "positions": ints([0] * 40)}
    ws = cc.empty_step_workspace()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        cc.cccl_step_plan(tables, lens, new, ws, **out)
    for step, n in enumerate(((20, 3), (5, 30), (17, 0))):
        new.copy_(ints(n))
        graph.replay()
        torch.cuda.synchronize()
    assert lens.tolist() == [42, 33] and tables.held.tolist() == [3, 3] and tables.free_count.tolist() == [14]
    assert tables.page_table[:, :3].tolist() == [[0, 1, 5], [2, 3, 4]]
    assert out["slots"][:17].tolist() == [16 + i for i in range(9, 16)] + [80 + i for i in range(10)]
    assert cc.cccl_get_result(ws)[1] == 0


# ------------------------------------------------------------------ write
ROTARY = [
    # lens, new, heads, group, dim, rot, page
    ([1], [1], 1, 1, 16, 16, 1),
    ([5, 0, 33, 16], [5, 0, 3, 16], 2, 3, 64, 32, 16),
    ([40, 7], [40, 7], 3, 1, 128, 128, 24),
    ([100, 1, 257], [1, 1, 1], 8, 4, 128, 64, 16),
    ([61], [60], 5, 2, 80, 16, 7),
    ([300] * 40, [50] * 40, 2, 2, 112, 112, 32),
    ([3, 9], [7, 9], 2, 2, 96, 48, 4),  # four rows lie before position 0
]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("fmt", ["16bit", "int8", "e4m3"])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("shape", range(len(ROTARY)))
def test_write(cc, shape, dtype, fmt, interleaved):
    lens, new, heads, group, dim, rot, page = ROTARY[shape]
    c = Case(lens, new, heads=heads, group=group, dim=dim, page=page, dtype=dtype, fmt=fmt, seed=shape,
             layout=["thd", "htd", "kv"][shape % 3])
    rotary = cc.StepRotary(rot, base=[1e4, 5e5][shape % 2], interleaved=interleaved, factor=4.0,
                           original_length=[0, 4096][shape // 2 % 2], magnitude=1.25)
    turns = [t & (1 << 64) - 1 for t in rotary.turns.tolist()]
    own = [t - n + i for t, n in zip(lens, new) for i in range(n)]
    given = None
    if shape % 2:  # far and near, twice the same, before 0
        r = random.Random(shape)
        given = [r.choice([0, 1, 131072 + r.randrange(9), 2 ** 31 - 1, r.randrange(5000), -3]) for _ in own]
    at = given or own
    fused = torch.cat([c.q, c.k_new, c.v_new], 1)
    parts = fused.split([heads * group, heads, heads], 1)
    before = [None if t is None else t.clone() for t in (c.k, c.v, c.ks, c.vs)]
    v_codes = Case(lens, new, heads=heads, group=group, dim=dim, page=page, dtype=dtype, fmt=fmt, seed=shape,
                   layout=["thd", "htd", "kv"][shape % 3])
    cc.kv_write(*v_codes.objects(cc), c.k_new, c.v_new)
    cache, batch = c.objects(cc)
    positions = None if given is None else ints(given)
    q_out = cc.step_write(cache, batch, rotary, *parts, positions=positions)

    def off(size):  # angles and their cosines, three roundings, all relative to |a| + |b|
        return 2.0 ** -21 * 1.25 * size

    y, size = ref.rotated(c.q, at, turns, 1.25, interleaved)
    assert ((q_out.double() - y).abs() <= off(size) + UNIT[dtype] * (y.abs() + off(size)) + TINY[dtype]).all()
    assert same_bits(q_out[..., rot:], c.q[..., rot:])
    y, size = ref.rotated(c.k_new, at, turns, 1.25, interleaved)
    # v goes where and as kv_write puts it
    assert same_bits(c.v, v_codes.v) and (c.vs is None or same_bits(c.vs, v_codes.vs))
    rows = [(i, int(c.table[b, p // page]), p % page) for b, (t, n) in enumerate(zip(lens, new))
            for i, p in zip(range(sum(new[:b]), sum(new)), range(t - n, t)) if p >= 0]
    idx, pages, slots = (ints([r[k] for r in rows], torch.int64) for k in range(3))
    y, e = y[idx], off(size[idx])
    if fmt == "16bit":
        got = c.k[pages, slots].double()
        assert ((got - y).abs() <= e + UNIT[dtype] * (y.abs() + e) + TINY[dtype]).all()
        assert same_bits(c.k[pages, slots][..., rot:], c.k_new[idx][..., rot:])
    else:
        s = c.ks[pages, slots].double()
        top = y.abs().amax(-1)
        assert ((s * LIMIT[fmt] - top).abs() <= e.amax(-1) + top * 2.0 ** -22).all()
        got = codes64(c.k[pages, slots], fmt) * s[..., None]
        big = y.abs() + e
        half = s[..., None] / 2 if fmt == "int8" else torch.maximum(big * 2.0 ** -4, s[..., None] * 2.0 ** -10)
        assert ((got - y).abs() <= e + half * (1 + 2.0 ** -16) + big * 2.0 ** -20).all()
    # what was not written keeps its bytes
    for t, kept in ((c.k, before[0]), (c.ks, before[2])):
        if t is not None:
            t[pages, slots] = kept[pages, slots]
            assert same_bits(t, kept)


def test_write_in_place_and_without_queries(cc):
    c = Case([50, 9], [20, 9], heads=2, group=2, dim=64, seed=5)
    rotary = cc.StepRotary(64)
    cache, batch = c.objects(cc)
    want = cc.step_write(cache, batch, rotary, c.q, c.k_new, c.v_new)
    k = c.k.clone()
    rows = c.T + 5  # rows of no sequence stay as they are
    q = torch.full((rows, 4, 64), 3.0, dtype=BF, device="cuda")
    q[2:2 + c.T] = c.q
    pad = torch.zeros(rows, 2, 64, dtype=BF, device="cuda")
    kk, vv = pad.clone(), pad.clone()
    kk[2:2 + c.T], vv[2:2 + c.T] = c.k_new, c.v_new
    batch = cc.KvBatch(c.table, c.cu + 2, c.len_dev, n_tokens=rows, max_new=20, max_len=50)
    ws = cc.empty_step_workspace()
    c.k.zero_()
    cc.cccl_step_write(cache, batch, rotary, q, kk, vv, q, ws)
    assert cc.cccl_get_result(ws)[1] == 0
    assert same_bits(q[2:2 + c.T], want) and (q[:2] == 3).all() and (q[2 + c.T:] == 3).all()
    used = c.k.abs().sum((2, 3)) > 0
    assert used.sum() == c.T and same_bits(c.k[used], k[used])
    c.k.zero_()
    cc.cccl_step_write(cache, batch, rotary, None, kk, vv, None, ws)
    assert same_bits(c.k[used], k[used])
    with pytest.raises(ValueError):
        cc.cccl_step_write(cache, batch, rotary, q, kk, vv, None, ws)


def test_write_marks_vectors_that_are_not_finite(cc):
    for fmt in ("int8", "e4m3"):
        c = Case([8], [8], heads=2, dim=64, fmt=fmt)
        c.k_new[2, 0, 5] = float("nan")
        c.k_new[3, 1, 63] = float("-inf")
        c.v_new[4, 0, 0] = float("inf")
        cache, batch = c.objects(cc)
        cc.step_write(cache, batch, cc.StepRotary(32), None, c.k_new, c.v_new)
        k, v = cc.kv_read(cache, batch)
        bad_k = torch.zeros(8, 2, dtype=torch.bool, device="cuda")
        bad_k[2, 0] = bad_k[3, 1] = True
        bad_v = torch.zeros(8, 2, dtype=torch.bool, device="cuda")
        bad_v[4, 0] = True
        for x, bad in ((k, bad_k), (v, bad_v)):
            assert x.isnan()[bad].all() and x.isfinite()[~bad].all()


# ------------------------------------------------------------------ verify
class Draft:
    def __init__(self, sizes, vocab, *, draft=True, chain=False, seed=0, sharp=2.0, near=0.7, few=None, pad=0, lead=0,
                 wide=3):
        g = torch.Generator().manual_seed(seed)
        self.sizes, T = sizes, sum(sizes) + lead
        self.cu = [lead]
        for n in sizes:
            self.cu.append(self.cu[-1] + n)
        z = torch.randn(T, vocab, generator=g) * sharp
        p = torch.softmax(z, -1)
        q = torch.softmax(z + near * torch.randn(T, vocab, generator=g), -1)
        tree = ref.trees(sizes, seed, wide)
        self.parents = None if chain else [-1] * lead + [x for ps in tree for x in ps]
        self.tokens = [0] * lead
        for n, lo, ps in zip(sizes, self.cu, tree):
            for i in range(n):
                up = max(0, i - 1 if chain else ps[i])
                if draft:
                    x = int(torch.multinomial(q[lo + up], 1, generator=g))
                else:
                    x = int(torch.randint(few or min(vocab, 4), (1,), generator=g))
                    x = int(q[lo + up].topk(min(vocab, few or 4)).indices[x])
                self.tokens.append(x)
        self.u = torch.rand(T, generator=g)
        self.p = torch.zeros(T, vocab + pad)[:, :vocab]
        self.q = torch.zeros(T, vocab + pad)[:, :vocab] if draft else None
        self.p.copy_(p)
        if draft:
            self.q.copy_(q)
        self.cuda()

    def cuda(self):
        def move(x):  # strides and all
            base = x._base if x._base is not None else x
            return base.cuda()[:, :x.shape[1]]

        self.dp, self.dq = move(self.p), None if self.q is None else move(self.q)

    def run(self, cc):
        parents = None if self.parents is None else ints(self.parents)
        return cc.step_verify(self.dp, self.dq, ints(self.tokens), parents, self.u.cuda(), ints(self.cu))

    def check(self, cc):
        path, n_kept, following = self.run(cc)
        w_path, w_kept, w_next = ref.verify(self.p.tolist(), None if self.q is None else self.q.tolist(), self.tokens,
                                            self.parents, self.u.tolist(), self.cu)
        lo = self.cu[0]
        assert n_kept.tolist() == w_kept and path.tolist()[lo:] == w_path[lo:]
        assert following.tolist() == w_next
        return w_kept


@pytest.mark.parametrize("draft", [True, False])
@pytest.mark.parametrize("chain", [True, False])
@pytest.mark.parametrize("vocab,pad", [(1, 0), (2, 1), (31, 0), (128, 0), (501, 0), (1000, 8), (4097, 0), (9000, 0)])
def test_verify(cc, vocab, pad, chain, draft):
    """Against whole numbers; rows at any alignment; trees of no token, one, and more than a warp's."""
    sizes = [1, 0, 5, 2, 40, 9] if vocab < 4000 else [6, 0, 33]
    kept = set()
    for seed in range(3):
        d = Draft(sizes, vocab, draft=draft, chain=chain, seed=100 * seed + vocab, pad=pad, lead=seed)
        kept |= set(d.check(cc))
    assert not draft or vocab < 3 or len(kept) > 2  # (tokens that no draft drew are seldom kept)


def test_verify_refuses_many_children(cc):
    """Children that are refused one after another, alike ones among them: the sums that are needed for the later ones."""
    for seed in range(4):
        for draft in (True, False):
            d = Draft([24, 12, 30], 300, draft=draft, seed=seed, sharp=1.0, near=3.0, few=6, wide=12)
            d.parents = [-1] + [0] * 23 + [-1] + [0] * 11 + [-1] + [0] * 15 + [3] * 14
            d.u = torch.rand(66, generator=torch.Generator().manual_seed(seed)) * 0.5 + 0.5
            d.check(cc)


def test_verify_refuses_hundreds(cc):
    """A draft that insists on what the target never says: A grows by one with every child."""
    n, vocab = 600, 40
    d = Draft([n], vocab, seed=2)
    d.parents = [-1] + [0] * (n - 1)
    d.tokens = [5] * n
    d.p[0] = 1.0 / (vocab - 1)
    d.p[0, 5] = 0
    d.q[0] = 0
    d.q[0, 5] = 1.0
    d.cuda()
    assert d.check(cc) == [1]
    d.q[0] = 1e-6  # and now and then something else
    d.q[0, 5] = 0.5
    d.cuda()
    d.check(cc)


def test_verify_of_rows_that_are_no_probabilities(cc):
    """Sums that leave 64 bits: some token of the vocabulary, and the call after it is right."""
    for vocab in (1 << 20, 5000):
        p = torch.ones(4, vocab, device="cuda")
        cu = ints([0, 1, 4])
        for q in (None, torch.zeros_like(p)):
            path, kept, following = (torch.full((n,), -3, dtype=torch.int32, device="cuda") for n in (4, 2, 2))
            cc.cccl_step_verify(p, q, ints([0, 1, 2, 3]), None, torch.full((4,), 0.9, device="cuda"), cu, path, kept,
                                following, cc.empty_step_workspace())
            assert kept.tolist() == [1, 3]
            assert all(0 <= y < vocab for y in following.tolist())
    Draft([5, 3], 700, seed=1).check(cc)


def test_verify_at_the_ends_of_the_random_numbers(cc):
    d = Draft([4, 4, 4], 700, seed=8)
    for u in (0.0, 1.0 - 2.0 ** -24, 1.0, 2.0, -1.0, float("nan")):
        d.u = torch.full((12,), u)
        if u != u:  # nothing is kept; the next token is the first with a weight
            _, kept, following = d.run(cc)
            assert kept.tolist() == [1, 1, 1]
            assert all(0 <= y < 700 for y in following.tolist())
        else:
            d.check(cc)


def test_verify_takes_odd_probabilities_as_documented(cc):
    """NaN and negative values count as 0, larger ones as 1, tiny ones are cut off."""
    d = Draft([6, 6, 3], 600, seed=3, near=2.0)
    d.p[:, ::7] = float("nan")
    d.p[:, 1::7] = -0.5
    d.p[1, 5] = float("inf")
    d.p[2] = 1e-38
    d.p[3, 3::7] *= 1e-30
    d.q[:, 2::5] = float("nan")
    d.q[4, 3] = float("-inf")
    d.cuda()
    d.check(cc)


def test_verify_when_nothing_is_left(cc):
    """A draft that the target equals, refused all the same, leaves the target itself; a row of zeros is reported."""
    d = Draft([3, 3], 400, seed=5)
    d.p[0] = d.q[0] = 0.0
    d.p[0, 17] = d.q[0, 17] = 0.25
    d.tokens[1] = 3  # the draft never draws it
    d.cuda()
    d.check(cc)
    d.dp[3:6] = 0
    parents = ints(d.parents)
    ws = cc.empty_step_workspace()
    path, kept, following = (torch.full((n,), -3, dtype=torch.int32, device="cuda") for n in (6, 2, 2))
    cc.cccl_step_verify(d.dp, d.dq, ints(d.tokens), parents, d.u.cuda(), ints(d.cu), path, kept, following, ws)
    assert cc.cccl_get_result(ws)[1] == cc.CCCL_ERR_INVALID_ARG
    assert following[1] == 0 and kept[1] == 1


def test_verify_passes_over_what_is_no_token(cc):
    d = Draft([10, 10], 300, seed=6)
    for i, x in ((2, -1), (3, 300), (4, 1 << 30), (13, -5)):
        d.tokens[i] = x
    d.parents[5], d.parents[6], d.parents[17] = -1, 9, 7
    d.check(cc)


def test_verify_of_long_trees(cc):
    sizes = [1024, 700]
    for draft in (True, False):
        d = Draft(sizes, 20, draft=draft, seed=7, near=0.2)
        d.check(cc)
        d = Draft(sizes, 20, draft=draft, chain=True, seed=7, near=0.0)
        d.u = torch.zeros(1724)  # all are kept
        assert d.check(cc) == sizes
    # one more than are gone through: reported
    d = Draft([1025], 20, chain=True, seed=9, near=0.0)
    d.u = torch.zeros(1025)
    ws = cc.empty_step_workspace()
    path, kept, following = (torch.full((n,), -3, dtype=torch.int32, device="cuda") for n in (1025, 1, 1))
    cc.cccl_step_verify(d.dp, d.dq, ints(d.tokens), None, d.u.cuda(), ints(d.cu), path, kept, following, ws)
    assert cc.cccl_get_result(ws)[1] == cc.CCCL_ERR_INVALID_ARG
    assert kept.tolist() == [1024] and path.tolist() == list(range(1024)) + [-1]


def test_verify_of_a_large_vocabulary(cc):
    """As many values as a row can have, and ones where blocks or warps have no part; the sum is looked up in 64 bits."""
    for vocab in (1 << 20, 128001, 70000):
        g = torch.Generator(device="cuda").manual_seed(vocab)
        p = torch.softmax(torch.randn(12, vocab, generator=g, device="cuda"), -1)
        u = torch.rand(12, generator=g, device="cuda")
        u[0], u[1], u[2] = 0.0, 1 - 2.0 ** -24, 0.5
        cu = torch.arange(13, dtype=torch.int32, device="cuda")
        _, kept, following = cc.step_verify(p, None, cu[:12].contiguous(), None, u, cu)
        assert kept.tolist() == [1] * 12
        upto = p.double().cumsum(1)
        goal = u.double() * upto[:, -1]
        y = following.long()[:, None]
        # 2^20 values cut off at 2^-56 each, and the reference's own sums
        slack = vocab * 2.0 ** -53
        low = torch.where(y > 0, upto.gather(1, (y - 1).clamp(min=0)), 0.0)[:, 0]
        assert (low <= goal + slack).all() and (upto.gather(1, y)[:, 0] >= goal - slack).all()


def test_verified_tokens_are_distributed_as_the_targets(cc):
    """The first token after the root, over 60000 trees of three children: with and without the draft's probabilities,
    each token's share is the target's within five standard deviations."""
    vocab, B, rounds = 6, 1000, 60
    g = torch.Generator(device="cuda").manual_seed(11)
    p1, q1 = (torch.softmax(1.5 * torch.randn(vocab, generator=g, device="cuda"), -1) for _ in range(2))
    cu = torch.arange(0, 4 * B + 1, 4, dtype=torch.int32, device="cuda")
    parents = ints([-1, 0, 0, 0] * B)
    p = p1.expand(4 * B, vocab).contiguous()
    q = q1.expand(4 * B, vocab).contiguous()
    for draft in (True, False):
        count = torch.zeros(vocab, dtype=torch.float64, device="cuda")
        for _ in range(rounds):
            if draft:
                tokens = torch.multinomial(q1, 4 * B, replacement=True, generator=g).to(torch.int32)
            else:
                tokens = ints([0, 2, 5, 1] * B)
            u = torch.rand(4 * B, generator=g, device="cuda")
            path, kept, following = cc.step_verify(p, q if draft else None, tokens, parents, u, cu)
            first = torch.where(kept > 1, tokens.view(B, 4).gather(1, path.view(B, 4)[:, 1:2].clamp(min=0).long())[:, 0],
                                following)
            count += torch.bincount(first.long(), minlength=vocab).double()
        share, n = count / count.sum(), B * rounds
        assert ((share - p1.double()).abs() <= 5 * (p1.double() * (1 - p1.double()) / n).sqrt()).all()


# ------------------------------------------------------------------ keep
def paths_of(new, seed, most=None):
    r = random.Random(seed)
    return [[0] + sorted(r.sample(range(1, n), r.randint(0, min(n - 1, most or n)))) if n else [] for n in new]


@pytest.mark.parametrize("layout", ["thd", "htd", "kv"])
@pytest.mark.parametrize("fmt", ["16bit", "int8", "e4m3"])
@pytest.mark.parametrize("shape", range(5))
def test_keep(cc, shape, fmt, layout):
    lens, new, heads, dim, page = [([1], [1], 1, 16, 1), ([40, 0, 7], [33, 0, 7], 2, 64, 16), ([100, 70], [64, 70], 3, 80, 24),
                                   ([300, 200, 5], [200, 150, 9], 8, 128, 7), ([2000], [1500], 1, 112, 64)][shape]
    c = Case(lens, new, heads=heads, dim=dim, page=page, fmt=fmt, layout=layout, seed=shape)
    paths = paths_of([min(a, b) for a, b in zip(lens, new)], shape)
    want = [None if t is None else t.clone() for t in (c.k, c.v, c.ks, c.vs)]
    for b, path in enumerate(paths):
        for k, i in enumerate(path):
            f, t = lens[b] - new[b] + i, lens[b] - new[b] + k
            if f >= 0 and t >= 0:
                f, t = (int(c.table[b, f // page]), f % page), (int(c.table[b, t // page]), t % page)
                for x in want:
                    if x is not None:
                        x[t] = x[f].clone()
    cache, batch = c.objects(cc)
    path = ints([i for p, n in zip(paths, new) for i in p + [-1] * (n - len(p))])
    got = cc.step_keep(cache, batch, path, ints([len(p) for p in paths]))
    assert got.tolist() == [max(0, t - n + len(p)) for t, n, p in zip(lens, new, paths)]
    for x, w in zip((c.k, c.v, c.ks, c.vs), want):
        assert w is None or same_bits(x, w)


def test_keep_reports_what_is_no_path(cc):
    c = Case([60, 60], [20, 20], heads=2, dim=64, page=16, seed=4)
    cache, batch = c.objects(cc)
    start = [c.k.clone(), c.v.clone()]

    def run(path, kept):
        for x, y in zip((c.k, c.v), start):
            x.copy_(y)
        ws, lens = cc.empty_step_workspace(), ints([0, 0])
        cc.cccl_step_keep(cache, batch, ints(path), ints(kept), lens, ws)
        return cc.cccl_get_result(ws)[1], lens.tolist()

    own = list(range(20))
    assert run(own + own, [20, 5]) == (0, [60, 45])
    assert same_bits(c.k, start[0])
    bad = cc.CCCL_ERR_INVALID_ARG
    for path in ([0, 0] + own[2:], [0, 20] + own[2:], [0, -1] + own[2:], [0, 1 << 30] + own[2:]):
        assert run(path + own, [2, 1]) == (bad, [42, 41])
        assert same_bits(c.k, start[0]) and same_bits(c.v, start[1])
    assert run(own + own, [-1, 21]) == (bad, [40, 60])
    assert run([0, 5] + own[2:] + own, [2, 1]) == (0, [42, 41])
    assert not same_bits(c.k, start[0])
    entry = c.table[0, 2].item()
    c.table[0, 2] = -1  # where token 1 lies
    assert run([0, 5] + own[2:] + own, [2, 1]) == (bad, [42, 41])
    assert same_bits(c.k, start[0])
    c.table[0, 2] = entry


# ------------------------------------------------------------------ a run of them together
@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("fmt", ["16bit", "int8"])
def test_steps_together(cc, fmt, captured):
    """Several steps of three sequences, eager or as one captured graph whose inputs change: after each, the cache
    holds what writing the kept tokens one after the other at their positions holds, and the kept tokens' attention
    is causal attention over that."""
    B, N, H, G, D, page, vocab, steps = 3, 13, 2, 3, 64, 16, 500, 5
    g = torch.Generator(device="cuda").manual_seed(3)
    code = {"16bit": cc.CCCL_KV_16BIT, "int8": cc.CCCL_KV_INT8}[fmt]
    cache, plain = (cc.KvCache.empty(80, page, H, D, fmt=code) for _ in range(2))
    for x in (cache.k, cache.v, plain.k, plain.v):
        x.zero_()
    tables = cc.StepTables.empty(B, 20, 80, page)
    rotary = cc.StepRotary(D, interleaved=True)
    lens = ints([0] * B)
    new, parents = ints([0] * B), ints([0] * (B * N))
    q, k, v = (torch.zeros(B * N, h, D, dtype=BF, device="cuda") for h in (H * G, H, H))
    p, qd = torch.zeros(B * N, vocab, device="cuda"), torch.zeros(B * N, vocab, device="cuda")
    tokens, u = ints([0] * (B * N)), torch.zeros(B * N, device="cuda")
    out, q_rot = torch.empty_like(q), torch.empty_like(q)
    plan = {"cu_tokens": ints([0] * (B + 1)), "kv_lens": ints([0] * B), "slots": ints([0] * (B * N), torch.int64),
            "positions": ints([0] * (B * N)), "mask": torch.zeros(B * N, 1, dtype=torch.int32, device="cuda")}
    batch = cc.KvBatch(tables.page_table, plan["cu_tokens"], plan["kv_lens"], n_tokens=B * N, max_new=N, max_len=300)
    path, n_kept, following = ints([0] * (B * N)), ints([0] * B), ints([0] * B)
    ws = cc.empty_kv_workspace(cache, batch, H * G)

    def step():
        cc.cccl_step_plan(tables, lens, new, ws, parents=parents, **plan)
        cc.cccl_step_write(cache, batch, rotary, q, k, v, q_rot, ws, positions=plan["positions"])
        cc.cccl_step_attention(cache, batch, q_rot, plan["mask"], out, ws)
        cc.cccl_step_verify(p, qd, tokens, parents, u, plan["cu_tokens"], path, n_kept, following, ws)
        cc.cccl_step_keep(cache, batch, path, n_kept, lens, ws)

    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    if captured:
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
            step()
    plain_table = torch.arange(60, dtype=torch.int32, device="cuda").view(B, 20)
    done = [0] * B
    for s in range(steps):
        sizes = [[1, 13, 6], [13, 1, 2], [7, 0, 13], [5, 5, 5], [1, 1, 1]][s]
        T = sum(sizes)
        new.copy_(ints(sizes))
        tree = ref.trees(sizes, s)
        parents[:T] = ints([x for ps in tree for x in ps])
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape, generator=g, device="cuda"))
        z = torch.randn(B * N, vocab, generator=g, device="cuda")
        p.copy_(torch.softmax(z, -1))
        qd.copy_(torch.softmax(z + 0.3 * torch.randn(z.shape, generator=g, device="cuda"), -1))
        up = [max(x, 0) + lo for ps, lo in zip(tree, [0] + torch.tensor(sizes).cumsum(0).tolist()) for x in ps]
        tokens[:T] = torch.multinomial(qd[ints(up, torch.int64)], 1, generator=g)[:, 0].int()
        u.copy_(torch.rand(B * N, generator=g, device="cuda"))
        graph.replay() if captured else step()
        assert cc.cccl_get_result(ws)[1] == 0
        w_path, w_kept, w_next = ref.verify(p.tolist(), qd.tolist(), tokens.tolist(), parents.tolist(), u.tolist(),
                                            plan["cu_tokens"].tolist())
        assert (path.tolist()[:T], n_kept.tolist(), following.tolist()) == (w_path[:T], w_kept, w_next)
        done = [a + b for a, b in zip(done, w_kept)]
        assert lens.tolist() == done
        # the kept tokens, one after the other, in another cache
        rows = [lo + i for lo, n in zip(plan["cu_tokens"].tolist(), w_kept) for i in w_path[lo:lo + n]]
        cu = ints([0] + torch.tensor(w_kept).cumsum(0).tolist())
        if not rows:
            continue
        idx = ints(rows, torch.int64)
        seq = cc.KvBatch(plain_table, cu, lens.clone(), n_tokens=len(rows), max_new=max(w_kept), max_len=max(done))
        q_seq = cc.step_write(plain, seq, rotary, q[idx], k[idx], v[idx])
        assert same_bits(q_seq, q_rot[idx])
        want, _ = cc.kv_attention(plain, seq, q_seq)
        # the same keys and weights summed in another order, rounded to bf16 on both sides (and probabilities, in
        # the kernel for many rows): a few units of 2^-8 of values of size 1
        assert ((out[idx].float() - want.float()).abs() <= 4 * 2.0 ** -8 * (1 + want.float().abs())).all()
        every = cc.KvBatch(plain_table, ints([0] + torch.tensor(done).cumsum(0).tolist()), lens.clone(),
                           n_tokens=sum(done), max_new=max(done), max_len=max(done))
        mine = cc.KvBatch(tables.page_table, every.cu_tokens, lens.clone(), n_tokens=sum(done), max_new=max(done),
                          max_len=max(done))
        for a, b in zip(cc.kv_read(plain, every), cc.kv_read(cache, mine)):
            assert same_bits(a, b)
    assert sum(done) > steps * B


def test_calls_on_another_stream(cc):
    side = torch.cuda.Stream()
    c = ref.TreeCase([100, 60], [9, 9], heads=2, group=2, dim=64, seed=1)
    cache, batch = c.objects(cc)
    rotary = cc.StepRotary(64)
    d = Draft([9, 9], 300, seed=2)
    torch.cuda.synchronize()
    want = (cc.step_write(cache, batch, rotary, c.q, c.k_new, c.v_new), *cc.step_attention(cache, batch, c.q, c.mask))
    args = (d.dp, d.dq, ints(d.tokens), ints(d.parents), d.u.cuda(), ints(d.cu))
    verdict = cc.step_verify(*args)
    torch.cuda.synchronize()
    got = (cc.step_write(cache, batch, rotary, c.q, c.k_new, c.v_new, stream=side),
           *cc.step_attention(cache, batch, c.q, c.mask, stream=side))
    for a, b in zip(want + verdict, got + cc.step_verify(*args, stream=side)):
        assert same_bits(a, b)
    assert cc.step_keep(cache, batch, verdict[0], verdict[1], stream=side).tolist() == \
        [91 + int(verdict[1][0]), 51 + int(verdict[1][1])]


def test_places_past_32_bits(cc):
    """Rows of probabilities and pages of a cache whose offsets do not fit 32 bits."""
    rows, vocab = 2052, 1 << 20
    p = torch.zeros(rows, vocab, device="cuda")
    p[2049, 77], p[2050, 900000], p[2051, vocab - 1] = 1.0, 1.0, 1.0
    tokens = ints([0] * 2050 + [77, 900000])
    cu = ints([2049, 2052])
    path, kept, following = cc.step_verify(p, None, tokens, None, torch.full((rows,), 0.5, device="cuda"), cu)
    assert kept.tolist() == [3] and following.tolist() == [vocab - 1] and path.tolist()[2049:] == [0, 1, 2]
    del p

    def pool(dtype):  # three pages, 2^31 values from one to the next
        whole = torch.empty(2 * (1 << 31) + 16 * 2 * 64, dtype=dtype, device="cuda")
        return whole.as_strided((3, 16, 2, 64), (1 << 31, 128, 64, 1))

    small = ref.TreeCase([40], [9], heads=2, group=2, dim=64, seed=3, spare=0)
    k, v = pool(BF), pool(BF)
    for far, near in ((k, small.k), (v, small.v)):
        far.copy_(near)
    rotary = cc.StepRotary(64)
    cache, batch = small.objects(cc)
    far = cc.KvCache(k, v)
    path, kept = ints([0, 4, 7, 8] + [-1] * 5), ints([4])
    for c in (cache, far):
        small.got = (cc.step_write(c, batch, rotary, small.q, small.k_new, small.v_new),
                     *cc.step_attention(c, batch, small.q, small.mask), cc.step_keep(c, batch, path, kept))
        if c is cache:
            want = small.got
    for a, b in zip(want, small.got):
        assert same_bits(a, b)
    assert same_bits(k, small.k) and same_bits(v, small.v)


def test_calls_at_the_same_time(cc):
    """Two streams, each with its own workspace and outputs, over one cache."""
    c = ref.TreeCase([500, 60, 900], [40, 9, 40], heads=2, group=4, dim=128, seed=6)
    cache, batch = c.objects(cc)
    d = Draft([40, 9, 40], 5000, seed=2)
    args = (d.dp, d.dq, ints(d.tokens), ints(d.parents), d.u.cuda(), ints(d.cu))
    want, _ = cc.step_attention(cache, batch, c.q, c.mask)
    verdict = cc.step_verify(*args)
    torch.cuda.synchronize()
    runs = []
    for _ in range(2):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            runs.append((s, torch.empty_like(c.q), cc.empty_kv_workspace(cache, batch, 8),
                         [torch.empty_like(x) for x in verdict], cc.empty_step_workspace()))
    torch.cuda.synchronize()
    for _ in range(20):
        for s, out, ws, outs, ws2 in runs:
            cc.cccl_step_attention(cache, batch, c.q, c.mask, out, ws, stream=s)
            cc.cccl_step_verify(*args, *outs, ws2, stream=s)
    torch.cuda.synchronize()
    for _, out, ws, outs, ws2 in runs:
        assert same_bits(out, want) and all(same_bits(a, b) for a, b in zip(outs, verdict))
        assert cc.cccl_get_result(ws)[1] == 0 and cc.cccl_get_result(ws2)[1] == 0


def test_guard_bands(cc):
    """Nothing is written past the outputs: each lies in a larger allocation that keeps its pattern."""
    def band(n, dtype):
        whole = torch.full((n + 64,), 77, dtype=dtype, device="cuda")
        return whole, whole[32:32 + n]

    p = Plan(cc, [30, 4, 0], [9, 50, 3], 16, words=2, seed=4)
    tables = cc.StepTables(p.d["table"], p.d["held"], p.d["free"], p.d["count"], page_tokens=16)
    names = {"cu_tokens": 4, "kv_lens": 3, "held": 3, "free_count": 1, "slots": 62, "positions": 62}
    made = {k: band(n, torch.int64 if k == "slots" else torch.int32) for k, n in names.items()}
    mask, view = band(62 * 2, torch.int32)
    cc.cccl_step_plan(tables, p.d["lens"], p.d["new"], cc.empty_step_workspace(), parents=p.d["parents"],
                      mask=view.view(62, 2), **{k: v[1] for k, v in made.items()})
    d = Draft([9, 50, 3], 123, seed=4)
    outs = [band(n, torch.int32) for n in (62, 3, 3)]
    cc.cccl_step_verify(d.dp, d.dq, ints(d.tokens), ints(d.parents), d.u.cuda(), ints(d.cu), *(o[1] for o in outs),
                        cc.empty_step_workspace())
    torch.cuda.synchronize()
    for whole, view in [*made.values(), (mask, view), *outs]:
        assert (whole[:32] == 77).all() and (whole[-32:] == 77).all()
        assert not (view == 77).all()
