"""What the operators of a decoding step with drafted tokens are timed on, and their plain forms.

Five operators around one paged key/value cache, as a serving program calls them
in a step that drafts a tree of tokens a sequence (a chain is a tree too):
`plan` builds block tables, slot maps, positions and ancestor masks from the
requests' lengths, `rotate` gives queries and keys their rotary positions and
stores keys and values, `tree` is the attention of the drafted tokens over the
cached ones and their own ancestors, `verify` accepts or rejects them against
the target's probabilities, `keep` moves the accepted ones' keys and values
together.  run() computes them with elementary torch operations when `own` is
false and through the package's entry points when it is true.
"""

import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
_LIMIT = {"int8": 127.0, "e4m3": 448.0}


def _plan(name, batch, new, ctx, page=16, words=2, ragged=True, shape=1):
    return {"name": name, "op": "plan", "batch": batch, "new": new, "ctx": ctx, "page": page, "words": words,
            "ragged": ragged, "shape": shape}


def _cached(name, op, dtype, fmt, heads, group, dim, page, batch, new, ctx, ragged=True, layout="thd", shape=1, **more):
    return {"name": name, "op": op, "dtype": dtype, "fmt": fmt, "heads": heads, "group": group, "dim": dim,
            "page": page, "batch": batch, "new": new, "ctx": ctx, "ragged": ragged, "layout": layout, "shape": shape,
            **more}


def _verify(name, batch, new, vocab, draft, wide, ragged=True, shape=1):
    return {"name": name, "op": "verify", "batch": batch, "new": new, "vocab": vocab, "draft": draft, "wide": wide,
            "ragged": ragged, "shape": shape}


def listed():
    return [
        # 64 users' trees of up to 33 tokens: tables, slots, positions and masks of one step, all latency
        _plan("plan_trees", 64, 33, 4096),
        # 32 prompts of up to 4096 tokens admitted at once: slots and positions, no tree
        _plan("plan_prompts", 32, 4096, 4096, words=0),
        # 32 users' chains of up to 5 tokens into an 8-bit cache, interleaved pairs in half of each head
        _cached("rotate_chains_int8", "rotate", "bf16", "int8", 8, 4, 128, 16, 32, 5, 4096, rot=64, interleaved=True,
                base=10000.0, factor=1.0, original=0, tree=False),
        # four prompts' queries and keys, frequencies stretched for long contexts
        _cached("rotate_prompts_bf16", "rotate", "bf16", "16bit", 8, 4, 128, 16, 4, 4096, 32768, rot=128,
                interleaved=False, base=500000.0, factor=8.0, original=8192, tree=False),
        # one user's tree of 5 tokens over a short context: the smallest attention call
        _cached("tree_short_bf16", "tree", "bf16", "16bit", 8, 4, 128, 16, 1, 5, 517, window=0),
        # 32 users' trees of up to 16 tokens over contexts up to the framework's 4096 tokens
        _cached("tree_users_bf16", "tree", "bf16", "16bit", 8, 4, 128, 16, 32, 16, 4096, window=0),
        # 16 users' trees of up to 33 tokens over long contexts held in 8 bits, heads outermost in a page
        _cached("tree_long_int8", "tree", "bf16", "int8", 8, 4, 128, 64, 16, 33, 32768, layout="htd", window=0),
        # one user's wide tree over a whole book, eight query heads a key head
        _cached("tree_book_fp16", "tree", "fp16", "16bit", 8, 8, 128, 64, 1, 61, 131072 + 5, window=0),
        # 64 users' chains of 4 drafted tokens with the draft model's probabilities
        _verify("verify_chains", 64, 5, 128000, True, 1),
        # 16 users' trees of up to 33 tokens that a draft proposed without probabilities, an odd vocabulary
        _verify("verify_trees", 16, 33, 50257, False, 4),
        # 64 users' accepted tokens moved together in one layer
        _cached("keep_users_bf16", "keep", "bf16", "16bit", 8, 4, 128, 16, 64, 33, 4096, kept=7),
        # many users' long accepted paths in an 8-bit cache, pages that end inside them
        _cached("keep_many_e4m3", "keep", "bf16", "e4m3", 8, 4, 128, 24, 512, 64, 1000, kept=16),
    ]


def draw(rng):
    def log_int(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    for _ in range(10000):
        op = rng.choice(["plan", "rotate", "tree", "tree", "tree", "verify", "keep"])
        shape, ragged = rng.randrange(1 << 30), rng.random() < 0.8
        if op == "plan":
            tree = rng.random() < 0.6
            batch, new, ctx = log_int(1, 512), log_int(1, 128 if tree else 4096), log_int(16, 131072)
            if batch * new > (1 << 17) or batch * ctx > (1 << 24):
                continue
            return {"op": op, "batch": batch, "new": new, "ctx": ctx, "page": rng.choice([16, 24, 32, 64, 128]),
                    "words": -(-new // 32) + rng.randrange(2) if tree else 0, "ragged": ragged, "shape": shape}
        if op == "verify":
            batch, draft = log_int(1, 64), rng.random() < 0.5
            wide = rng.choice([1, 2, 4])
            new, vocab = log_int(1, 9 if wide == 1 else 64), log_int(1000, 152000)
            if batch * new * vocab * (2 if draft else 1) > 9e7:
                continue
            return {"op": op, "batch": batch, "new": new, "vocab": vocab, "draft": draft, "wide": wide,
                    "ragged": ragged, "shape": shape}
        c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "fp16"]), "fmt": rng.choice(["16bit", "int8", "e4m3"]),
             "heads": rng.choice([1, 2, 3, 8, 12]), "group": rng.choice([1, 2, 4, 6, 8]),
             "dim": rng.choice([64, 80, 96, 128, 128]), "page": rng.choice([16, 16, 24, 32, 64]),
             "batch": log_int(1, 64), "ragged": ragged, "layout": rng.choice(["thd", "htd"]), "shape": shape}
        c["ctx"] = log_int(64, 131072)
        if op == "rotate":
            c["tree"] = rng.random() < 0.5
            c["new"] = log_int(1, 64) if c["tree"] else log_int(1, min(4096, c["ctx"]))
            c["rot"] = rng.choice([c["dim"], c["dim"], c["dim"] // 32 * 16])
            c["interleaved"] = rng.random() < 0.5
            c["base"] = rng.choice([10000.0, 500000.0, 1000000.0])
            c["factor"] = rng.choice([1.0, 4.0, 8.0])
            c["original"] = rng.choice([0, 4096, 8192])
        else:
            c["new"] = log_int(1, 64)
        c["new"] = min(c["new"], c["ctx"])
        if op == "tree":
            c["window"] = log_int(c["new"], c["ctx"]) if rng.random() < 0.25 else 0
        elif op == "keep":
            c["kept"] = rng.randint(1, max(1, (c["new"] + 1) // 2))
        w = work(c)
        pool = sum(_lengths(c)[0]) * c["heads"] * c["dim"] * 2 * _elem(c)
        # what the plain form lays out at once
        padded = c["batch"] * c["ctx"] * c["heads"] * max(c["dim"], c["group"] * c["new"]) if op == "tree" else 0
        if w["bytes"] <= 0.5e9 and pool <= 1.2e9 and padded <= 8e8 and w["flops"] <= 3e11:
            return c
    raise RuntimeError("no case of the ranges drawn")


def _elem(c):
    return 2 if c["fmt"] == "16bit" else 1


def _lengths(c):
    """(tokens cached, new tokens) of every sequence; the new ones are the last of the cached ones."""
    r = random.Random(c["shape"])
    total, new = [], []
    ctx = c.get("ctx", c["new"])
    for b in range(c["batch"]):
        t = ctx if b == 0 or not c["ragged"] else r.randint(max(1, ctx // 4), ctx)
        n = c["new"] if b == 0 or not c["ragged"] else r.randint(max(1, c["new"] // 4), c["new"])
        total.append(t if "ctx" in c else n)
        new.append(min(n, total[-1]))
    return total, new


def _parents(c, new):
    """A tree a sequence: the root is token 0, every other token hangs from an earlier one, most from a near one."""
    r = random.Random(c["shape"] + 1)
    return [[-1] + [r.randint(max(0, (i - 1) // 2 - 2), i - 1) for i in range(1, n)] for n in new]


def _kept(c, new):
    """Accepted paths: the root, then tokens that lie past the places they move to (or stay), so that a second pass
    over the same cache finds what the first one found."""
    r = random.Random(c["shape"] + 2)
    paths = []
    for b, n in enumerate(new):
        k = min(c["kept"] if b == 0 or not c["ragged"] else r.randint(1, c["kept"]), (n + 1) // 2)
        paths.append([0] + sorted(r.sample(range(k, n), k - 1)))
    return paths


def work(case):
    c = case
    total, new = _lengths(c)
    T, B = sum(new), c["batch"]
    if c["op"] == "plan":  # lengths in and out, tables' new entries, a row's slot, position, parent and mask
        pages = T // c["page"] + B
        return {"bytes": 36 * B + 8 * pages + T * (12 + (4 + 4 * c["words"] if c["words"] else 0)), "flops": 0}
    if c["op"] == "verify":  # the row that the last token is drawn from, and a few numbers of every drafted token
        return {"bytes": 4 * B * c["vocab"] * (2 if c["draft"] else 1) + 28 * T + 8 * B, "flops": 0}
    H, D = c["heads"], c["dim"]
    stored = H * (2 * D * _elem(c) + (8 if c["fmt"] != "16bit" else 0))  # K and V of one token, with scales
    if c["op"] == "rotate":
        return {"bytes": T * (2 * H * D * 2 + 2 * H * c["group"] * D * 2 + stored), "flops": 0}
    if c["op"] == "keep":
        moved = sum(sum(i != k for k, i in enumerate(p)) for p in _kept(c, new))
        return {"bytes": 2 * moved * stored + 4 * sum(map(len, _kept(c, new))) + 12 * B, "flops": 0}
    pairs = keys = 0
    for t, n in zip(total, new):
        seen = min(t - n, c["window"]) if c["window"] else t - n
        keys += seen + n
        pairs += n * (seen + 1)
    heads = H * c["group"]
    return {"bytes": 2 * T * heads * D * 2 + keys * stored + 8 * T, "flops": 4 * D * heads * pairs}


# ------------------------------------------------------------------ inputs
def _values(gen, shape, scale, dtype):
    """N(0, 1) times one scale per head (the second last axis)."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return (x * scale[:, None]).to(dtype)


def _quantise(x, fmt):
    """Codes (as bytes) and scales of vectors x[..., D]: a = max|x|, scale = a / L, code = x * (L / a)."""
    x = x.float()
    a = x.abs().amax(-1)
    limit = torch.full_like(a, _LIMIT[fmt])
    scale = a / limit
    inv = torch.where(a > 0, (limit / a).clamp(max=torch.finfo(torch.float32).max), torch.zeros_like(a))
    y = torch.clamp(x * inv[..., None], -_LIMIT[fmt], _LIMIT[fmt])
    if fmt == "int8":
        return torch.round(y).nan_to_num(0.0).to(torch.int8), scale
    return y.to(torch.float8_e4m3fn).view(torch.int8), scale


def _ints(x, dtype=torch.int32):
    return torch.tensor(x, dtype=dtype, device="cuda")


def _depths(parents):
    d = []
    for p in parents:
        d.append(0 if p < 0 else d[p] + 1)
    return d


def _mask_words(parents, words):
    """Each token's ancestors and itself as bits, 32 a word."""
    bits = []
    for i, p in enumerate(parents):
        bits.append((bits[p] if p >= 0 else 0) | 1 << i)
    as_int = lambda w: w - (1 << 32) if w >> 31 else w  # noqa: E731
    return [[as_int(m >> 32 * w & 0xFFFFFFFF) for w in range(words)] for m in bits]


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    total, new = _lengths(c)
    B, T = c["batch"], sum(new)
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    s = {"case": c, "total": total, "new": new, "cu": cu, "rows": T, "new_dev": _ints(new)}
    if c["op"] == "plan":
        return _prepare_plan(s, gen)
    if c["op"] == "verify":
        return _prepare_verify(s, gen)
    dtype = _DTYPES[c["dtype"]]
    H, D, P = c["heads"], c["dim"], c["page"]
    need = [-(-t // P) for t in total]
    pages = sum(need) + 3
    # the pages of all sequences lie mixed in the pool
    perm = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros(B, max(need), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    k_head = torch.exp(torch.empty(H, device="cuda").uniform_(math.log(0.1), math.log(10.0), generator=gen))
    v_head = torch.exp(torch.empty(H, device="cuda").uniform_(math.log(0.1), math.log(10.0), generator=gen))
    # K and V of a layer: [pages, page, heads, dim], tokens or heads outermost within a page
    shape = (pages, P, H, D) if c["layout"] == "thd" else (pages, H, P, D)
    store = dtype if c["fmt"] == "16bit" else torch.int8
    k, v = (torch.empty(shape, dtype=store, device="cuda") for _ in range(2))
    if c["layout"] == "htd":
        k, v = k.transpose(1, 2), v.transpose(1, 2)
    ks = vs = None
    if c["fmt"] != "16bit":
        ks, vs = (torch.empty(pages, H, P, device="cuda").transpose(1, 2) for _ in range(2))
    step = max(1, (1 << 26) // (P * H * D))
    for a in range(0, pages, step):
        n = min(step, pages - a)
        for data, scales, head in ((k, ks, k_head), (v, vs, v_head)):
            x = _values(gen, (n, P, H, D), head, dtype)
            if scales is None:
                data[a:a + n] = x
            else:
                codes, scale = _quantise(x, c["fmt"])
                data[a:a + n] = codes
                scales[a:a + n] = scale
    s |= {"k": k, "v": v, "ks": ks, "vs": vs, "table": table, "dtype": dtype, "cu_dev": _ints(cu),
          "len_dev": _ints(total)}
    heads = H * c["group"]
    if c["op"] == "rotate":
        # queries, keys and values as one fused projection's output
        q_head = torch.ones(heads, device="cuda")
        qkv = torch.cat([_values(gen, (T, len(h), D), h, dtype) for h in (q_head, k_head, v_head)], 1)
        s |= {"qkv": qkv, "q": qkv[:, :heads], "k_new": qkv[:, heads:heads + H], "v_new": qkv[:, heads + H:]}
        depth = [_depths(p) for p in _parents(c, new)] if c["tree"] else [range(n) for n in new]
        s["positions"] = _ints([t - n + d for t, n, ds in zip(total, new, depth) for d in ds])
        s["inv_freq"] = torch.tensor(_inv_freq(c), dtype=torch.float64, device="cuda")
    elif c["op"] == "tree":
        s["q"] = torch.randn(T, heads, D, generator=gen, device="cuda").to(dtype)
        words = -(-max(new) // 32)
        s["mask"] = _ints([m for p in _parents(c, new) for m in _mask_words(p, words)])
    else:
        paths = _kept(c, new)
        s["path"] = _ints([i for p, n in zip(paths, new) for i in p + [-1] * (n - len(p))])
        s["n_kept"] = _ints([len(p) for p in paths])
    if own:
        import compression_coupled_collectives_gb300 as cc

        fmt = {"16bit": cc.CCCL_KV_16BIT, "int8": cc.CCCL_KV_INT8, "e4m3": cc.CCCL_KV_E4M3}[c["fmt"]]
        s["cc"] = cc
        s["cache"] = cc.KvCache(k, v, ks, vs, dtype=dtype, fmt=fmt)
        s["batch"] = cc.KvBatch(table, s["cu_dev"], s["len_dev"], n_tokens=T, max_new=max(new), max_len=max(total))
        s["ws"] = cc.empty_kv_workspace(s["cache"], s["batch"], heads if c["op"] == "tree" else 0)
        if c["op"] == "rotate":
            s["rotary"] = cc.StepRotary(c["rot"], base=c["base"], interleaved=c["interleaved"], factor=c["factor"],
                                        original_length=c["original"], magnitude=_magnitude(c), device="cuda")
            s["q_out"] = torch.empty(T, heads, D, dtype=dtype, device="cuda")
            if c["fmt"] != "16bit":
                s["k_out"], s["v_out"] = (torch.empty(T, H, D, dtype=dtype, device="cuda") for _ in range(2))
        elif c["op"] == "tree":
            s["out"] = torch.empty_like(s["q"])
        else:
            s["lens_out"] = torch.empty(B, dtype=torch.int32, device="cuda")
    return s


def _prepare_plan(s, gen):
    c, P = s["case"], s["case"]["page"]
    # cached so far; a sequence may hold a page more than its tokens need, from a step that drafted more than it kept
    lens = [t - n for t, n in zip(s["total"], s["new"])]
    r = random.Random(c["shape"] + 3)
    held = [-(-n // P) + (r.random() < 0.3) for n in lens]
    width = max(max(-(-t // P) for t in s["total"]), max(held)) + 1
    need = [max(0, -(-t // P) - h) for t, h in zip(s["total"], held)]
    pages = sum(held) + sum(need) + 7
    perm = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros(len(held), width, dtype=torch.int32, device="cuda")
    held_dev = _ints(held)
    inside = torch.arange(width, device="cuda")[None] < held_dev[:, None]
    table[inside] = perm[:sum(held)]
    s |= {"table": table, "lens": _ints(lens), "held": held_dev, "free": perm[sum(held):].clone(),
          "free_count": _ints([pages - sum(held)])}
    if c["words"]:
        s["parents"] = _ints([p for ps in _parents(c, s["new"]) for p in ps])
    if own:
        import compression_coupled_collectives_gb300 as cc

        s["cc"] = cc
        s["ws"] = cc.empty_step_workspace()
        s["tables"] = cc.StepTables(table, held_dev, s["free"], s["free_count"], page_tokens=P)
        s["outs"] = {"cu_tokens": torch.empty(c["batch"] + 1, dtype=torch.int32, device="cuda"),
                     "kv_lens": torch.empty_like(s["lens"]), "held": torch.empty_like(held_dev),
                     "free_count": torch.empty_like(s["free_count"]),
                     "slots": torch.empty(s["rows"], dtype=torch.int64, device="cuda"),
                     "positions": torch.empty(s["rows"], dtype=torch.int32, device="cuda")}
        if c["words"]:
            s["outs"]["mask"] = torch.empty(s["rows"], c["words"], dtype=torch.int32, device="cuda")
    return s


def _prepare_verify(s, gen):
    c, V, T = s["case"], s["case"]["vocab"], s["rows"]
    r = random.Random(c["shape"] + 4)
    parents = []
    for n in s["new"]:  # at most `wide` children a token
        ps, children = [-1], [0]
        for i in range(1, n):
            open_ = [k for k in range(max(0, (i - 1) // c["wide"] - 1), i) if children[k] < c["wide"]]
            p = open_[0] if r.random() < 0.7 else r.choice(open_)
            children[p] += 1
            ps.append(p)
            children.append(0)
        parents.append(ps)
    rank = [[sum(q == p for q in ps[:i]) for i, p in enumerate(ps)] for ps in parents]
    first_row = [a for a, ps in zip(s["cu"], parents) for _ in ps]
    parent_row = _ints([max(p, 0) for ps in parents for p in ps], torch.int64) + _ints(first_row, torch.int64)
    s["parents"] = _ints([p for ps in parents for p in ps])
    s["p"] = torch.empty(T, V, device="cuda")
    draft = torch.empty(T, V, device="cuda")
    step = max(1, (1 << 26) // V)
    for a in range(0, T, step):  # the target's logits, and a draft model's that are near them
        z = torch.randn(min(step, T - a), V, generator=gen, device="cuda") * 2.5
        s["p"][a:a + step] = torch.softmax(z, -1)
        z += 0.5 * torch.randn(z.shape, generator=gen, device="cuda")
        draft[a:a + step] = torch.softmax(z, -1)
    if c["draft"]:  # tokens drawn from the draft's probabilities
        x = torch.cat([torch.multinomial(draft[parent_row[a:a + step]], 1, generator=gen) for a in range(0, T, step)])
        s["q"] = draft
    else:  # its likeliest ones, a different one for each child
        x = torch.topk(draft, c["wide"], dim=-1).indices[parent_row].gather(
            1, _ints([r % c["wide"] for rs in rank for r in rs], torch.int64)[:, None])
        s["q"] = None
    s["tokens"] = x[:, 0].to(torch.int32)
    s["uniform"] = torch.rand(T, generator=gen, device="cuda")
    s["cu_dev"] = _ints(s["cu"])
    del draft
    if own:
        import compression_coupled_collectives_gb300 as cc

        s["cc"] = cc
        s["ws"] = cc.empty_step_workspace()
        s["path"] = torch.empty(T, dtype=torch.int32, device="cuda")
        s["n_kept"], s["next"] = (torch.empty(c["batch"], dtype=torch.int32, device="cuda") for _ in range(2))
    return s


def _inv_freq(c):
    """Radians a position of every pair.  Stretched by parts: a pair that turns fewer than once over the original
    length is slowed by the factor, one that turns more than 32 times stays, the ones between are mixed."""
    out = []
    for i in range(c["rot"] // 2):
        f = c["base"] ** (-2.0 * i / c["rot"])
        stay = 0.0
        if c["original"]:
            stay = min(1.0, max(0.0, (c["original"] * f / (2 * math.pi) - 1.0) / 31.0))
        out.append(f * stay + f / c["factor"] * (1.0 - stay))
    return out


def _magnitude(c):
    return 0.1 * math.log(c["factor"]) + 1.0 if c["original"] else 1.0


# ------------------------------------------------------------------ one pass
def _rows_of(s):
    """Of every packed row: its sequence and its number within it."""
    rows = torch.arange(s["rows"], device="cuda")
    end = s["new_dev"].long().cumsum(0)
    seq = torch.repeat_interleave(torch.arange(len(end), device="cuda"), s["new_dev"].long(), output_size=s["rows"])
    return seq, rows - (end - s["new_dev"])[seq]


def _plain_plan(s):
    c, P = s["case"], s["case"]["page"]
    lens, new, held = s["lens"], s["new_dev"], s["held"]
    after = lens + new
    need = ((after + P - 1) // P - held).clamp(min=0)
    upto = need.cumsum(0)
    free_left = s["free_count"] - upto[-1:]
    column = torch.arange(s["table"].shape[1], device="cuda")[None]
    which = column - held[:, None]
    fresh = (which >= 0) & (which < need[:, None])
    taken = s["free_count"] - 1 - ((upto - need)[:, None] + which)
    s["table"].copy_(torch.where(fresh, s["free"][taken.clamp(0, len(s["free"]) - 1).long()], s["table"]))
    cu = torch.cat([torch.zeros_like(new[:1]), new.cumsum(0).to(torch.int32)])
    seq, i = _rows_of(s)
    place = lens[seq].long() + i
    outs = {"table": s["table"], "cu": cu, "lens": after, "held": held + need.to(torch.int32),
            "free_count": free_left.to(torch.int32),
            "slots": s["table"][seq, place // P].long() * P + place % P}
    if not c["words"]:
        return {**outs, "positions": place.to(torch.int32)}
    # ancestors by pointer doubling
    rows = torch.arange(s["rows"], device="cuda")
    parent = torch.where(s["parents"] >= 0, rows - i + s["parents"], rows)
    depth = (s["parents"] >= 0).to(torch.int32)
    word = torch.arange(c["words"], device="cuda")[None]
    mask = torch.where(word == (i // 32)[:, None], (1 << (i % 32))[:, None], 0)
    for _ in range(max(1, (c["new"] - 1).bit_length())):
        mask = mask | mask[parent]
        depth = depth + depth[parent]
        parent = parent[parent]
    return {**outs, "positions": lens[seq] + depth, "mask": mask.to(torch.int32)}


def _rotated(s, x):
    """x [rows, heads, dim] in binary32 with its rotary positions; angles in binary64."""
    c, R = s["case"], s["case"]["rot"]
    angle = s["positions"].double()[:, None] * s["inv_freq"][None]
    cos, sin = ((f(angle).float() * _magnitude(c))[:, None] for f in (torch.cos, torch.sin))
    x = x.float()
    if c["interleaved"]:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., R:]], -1)


def _slots(s):
    """Page and slot of every packed row."""
    P = s["case"]["page"]
    seq, i = _rows_of(s)
    place = (s["len_dev"] - s["new_dev"]).long()[seq] + i
    return s["table"][seq, place // P].long(), place % P


def _plain_rotate(s):
    c = s["case"]
    q = _rotated(s, s["q"]).to(s["dtype"])
    pages, slots = _slots(s)
    k, v = _rotated(s, s["k_new"]), s["v_new"]
    if c["fmt"] == "16bit":
        s["k"][pages, slots], s["v"][pages, slots] = k.to(s["dtype"]), v
        return q, s["k"], s["v"]
    outs = []
    for x, data, scales in ((k, s["k"], s["ks"]), (v, s["v"], s["vs"])):
        codes, scale = _quantise(x, c["fmt"])
        data[pages, slots] = codes
        scales[pages, slots] = scale
        back = codes.view(torch.float8_e4m3fn).float() if c["fmt"] == "e4m3" else codes.float()
        outs.append((back * scale[..., None]).to(s["dtype"]))
    return q, outs[0], outs[1], s["ks"], s["vs"]


def _padded(s):
    """K and V of all sequences, [batch, kv heads, longest, dim] in binary32 (places past a sequence's end: any)."""
    got = []
    for data, scales in ((s["k"], s["ks"]), (s["v"], s["vs"])):
        x = data[s["table"].long()]
        if scales is not None:
            x = x.view(torch.float8_e4m3fn) if s["case"]["fmt"] == "e4m3" else x
            x = x.float() * scales[s["table"].long()][..., None]
        got.append(x.float().flatten(1, 2)[:, :max(s["total"])].transpose(1, 2))
    return got


def _plain_tree(s):
    c, G = s["case"], s["case"]["group"]
    B, N, H, D = c["batch"], max(s["new"]), c["heads"], c["dim"]
    k, v = _padded(s)
    seq, i = _rows_of(s)
    q = torch.zeros(B, N, H * G, D, device="cuda")
    q[seq, i] = s["q"].float()
    q = q.view(B, N, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * N, D)
    # what a drafted token sees: all that was cached before, and the drafted ones in its mask
    before = (s["len_dev"] - s["new_dev"]).long()
    at = torch.arange(k.shape[2], device="cuda")[None, :] - before[seq][:, None]
    bits = s["mask"][torch.arange(s["rows"], device="cuda")[:, None], (at // 32).clamp(0, s["mask"].shape[1] - 1)]
    drafted = (at >= 0) & (at < s["new_dev"].long()[seq][:, None]) & ((bits >> (at % 32)) & 1 != 0)
    seen = (at < 0) | drafted
    if c["window"]:  # the last `window` tokens of its path
        seen &= at + c["window"] >= drafted.sum(1, keepdim=True)
    hidden = torch.ones(B, N, k.shape[2], dtype=torch.bool, device="cuda")
    hidden[seq, i] = ~seen
    x = torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(D))
    x = x.view(B, H, G, N, -1).masked_fill_(hidden[:, None, None], float("-inf"))
    x -= x.amax(-1, keepdim=True)
    x.exp_()
    o = torch.matmul(x.view(B, H, G * N, -1), v).view(B, H, G, N, D) / x.sum(-1, keepdim=True)
    return o.permute(0, 3, 1, 2, 4)[seq, i].reshape(s["q"].shape).to(s["dtype"])


def _plain_verify(s):
    """Tokens in order, all sequences at once; probabilities and their sums in binary64."""
    B, V = s["case"]["batch"], s["case"]["vocab"]
    new, start = s["new_dev"].long(), s["cu_dev"].long()[:-1]
    each = torch.arange(B, device="cuda")
    at, n_kept = torch.zeros_like(start), (new > 0).long()
    path = torch.full((s["rows"] + 1,), -1, dtype=torch.int32, device="cuda")
    path[torch.where(new > 0, start, s["rows"])] = 0
    taken = torch.zeros(B, dtype=torch.float64, device="cuda")  # how many times q is taken off p, or p's part that is
    out = torch.zeros(B, V, dtype=torch.bool, device="cuda") if s["q"] is None else None  # tokens rejected here
    for i in range(1, max(s["new"])):
        row = torch.where(i < new, start + i, start)
        token = s["tokens"][row].long()
        tried = (i < new) & (s["parents"][row] == at)
        u = s["uniform"][row].double()
        here = start + at
        p = s["p"][here, token].double()
        if s["q"] is None:
            p = torch.where(out[each, token], 0.0, p)
            left, chance = 1.0 - taken, p
            take = tried & (u * left < p)
        else:
            q = s["q"][here, token].double()
            left = (s["p"][here].double() - taken[:, None] * s["q"][here].double()).clamp(min=0).sum(1)
            left = torch.where(taken > 0, left, 1.0)
            take = tried & (u * left * q < (p - taken * q).clamp(min=0))
            chance = left
        missed = tried & ~take
        at = torch.where(take, i, at)
        path[torch.where(take, start + n_kept, s["rows"])] = i
        n_kept = n_kept + take
        taken = torch.where(take, 0.0, torch.where(missed, taken + chance, taken))
        if out is not None:
            out &= ~take[:, None]
            out[each, token] |= missed
    here = (start + at).clamp(max=s["rows"] - 1)
    p = s["p"][here].double()
    if s["q"] is None:
        rest = p.masked_fill(out, 0.0)
    else:
        rest = (p - taken[:, None] * s["q"][here].double()).clamp(min=0)
    rest = torch.where(rest.sum(1, keepdim=True) > 0, rest, p)
    upto = rest.cumsum(1)
    goal = s["uniform"][start.clamp(max=s["rows"] - 1)].double()[:, None] * upto[:, -1:]
    token = (upto > goal).to(torch.int8).argmax(1)
    return (path[:s["rows"]], n_kept.to(torch.int32), torch.where(new > 0, token, -1).to(torch.int32))


def _plain_keep(s):
    P = s["case"]["page"]
    seq, i = _rows_of(s)
    moved = i < s["n_kept"].long()[seq]
    before = (s["len_dev"] - s["new_dev"]).long()[seq]
    at = (before + torch.where(moved, s["path"].long(), i))
    place = before + i
    from_page, from_slot = s["table"][seq, at // P].long(), at % P
    to_page, to_slot = s["table"][seq, place // P].long(), place % P
    outs = []
    for x in (s["k"], s["v"], s["ks"], s["vs"]):
        if x is not None:  # (rows past the kept ones move to where they are)
            x[to_page, to_slot] = torch.where(moved.view(-1, *[1] * (x.dim() - 2)), x[from_page, from_slot],
                                              x[to_page, to_slot])
            outs.append(x.view(torch.float8_e4m3fn) if s["case"]["fmt"] == "e4m3" and x.dim() == 4 else x)
    return (*outs, (s["len_dev"] - s["new_dev"] + s["n_kept"]).to(torch.int32))


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return {"plan": _plain_plan, "rotate": _plain_rotate, "tree": _plain_tree, "verify": _plain_verify,
                "keep": _plain_keep}[op](s)
    cc = s["cc"]
    if op == "plan":
        o = s["outs"]
        cc.cccl_step_plan(s["tables"], s["lens"], s["new_dev"], s["ws"], parents=s.get("parents"), **o)
        outs = {"table": s["table"], "cu": o["cu_tokens"], "lens": o["kv_lens"], "held": o["held"],
                "free_count": o["free_count"], "slots": o["slots"], "positions": o["positions"]}
        return {**outs, "mask": o["mask"]} if "mask" in o else outs
    if op == "verify":
        cc.cccl_step_verify(s["p"], s["q"], s["tokens"], s["parents"], s["uniform"], s["cu_dev"], s["path"],
                            s["n_kept"], s["next"], s["ws"])
        return s["path"], s["n_kept"], s["next"]
    if op == "tree":
        cc.cccl_step_attention(s["cache"], s["batch"], s["q"], s["mask"], s["out"], s["ws"],
                               window=s["case"]["window"])
        return s["out"]
    if op == "rotate":
        cc.cccl_step_write(s["cache"], s["batch"], s["rotary"], s["q"], s["k_new"], s["v_new"], s["q_out"], s["ws"],
                           positions=s["positions"])
        if s["case"]["fmt"] == "16bit":
            return s["q_out"], s["k"], s["v"]
        # what was written, as the values that the codes stand for
        cc.cccl_kv_read(s["cache"], s["batch"], s["k_out"], s["v_out"], s["ws"])
        return s["q_out"], s["k_out"], s["v_out"], s["ks"], s["vs"]
    cc.cccl_step_keep(s["cache"], s["batch"], s["path"], s["n_kept"], s["lens_out"], s["ws"])
    outs = [s["k"], s["v"]] + ([] if s["ks"] is None else [s["ks"], s["vs"]])
    if s["case"]["fmt"] == "e4m3":
        outs[:2] = [x.view(torch.float8_e4m3fn) for x in outs[:2]]
    return (*outs, s["lens_out"])


# ------------------------------------------------------------------ in 64 bits
def _place64(s, b, position):
    page = position // s["case"]["page"]
    return s["rows_of_table"][b][page], position % s["case"]["page"]


def _exact_rotate(s):
    c, R = s["case"], s["case"]["rot"]
    half = torch.arange(R // 2, dtype=torch.float64, device="cuda")
    freq = torch.pow(torch.tensor(c["base"], dtype=torch.float64, device="cuda"), -half / (R / 2))
    if c["original"]:
        turns = c["original"] * freq / (2 * math.pi)
        mix = ((turns - 1) / 31).clamp(0, 1)
        freq = mix * freq + (1 - mix) * freq / c["factor"]
    else:
        freq = freq / c["factor"]
    turn = torch.polar(torch.full_like(freq, _magnitude(c)).expand(s["rows"], -1).contiguous(),
                       s["positions"].double()[:, None] * freq)[:, None]

    def turned(x):
        x = x.double()
        pairs = x[..., :R].unflatten(-1, (-1, 2)) if c["interleaved"] else x[..., :R].unflatten(-1, (2, -1)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
        z = z if c["interleaved"] else z.transpose(-1, -2)
        return torch.cat([z.flatten(-2), x[..., R:]], -1)

    places = [_place64(s, b, p) for b, (t, n) in enumerate(zip(s["total"], s["new"])) for p in range(t - n, t)]
    pages, slots = (_ints([p[i] for p in places], torch.int64) for i in (0, 1))
    outs, tables = [turned(s["q"])], []
    for x, which in ((turned(s["k_new"]), "k"), (s["v_new"].double(), "v")):
        if c["fmt"] == "16bit":
            whole = s[which].double()
            whole[pages, slots] = x
            outs.append(whole)
            continue
        unit = x.abs().max(dim=-1, keepdim=True).values / _LIMIT[c["fmt"]]
        ratio = torch.where(unit > 0, x / unit, torch.zeros_like(x))
        if c["fmt"] == "int8":
            code = torch.round(ratio)
        else:  # to 4 significant bits, steps of 2^-9 below 2^-6
            power = torch.floor(torch.log2(ratio.abs().clamp(min=2.0 ** -6)))
            grain = torch.exp2(power - 3)
            code = torch.round(ratio / grain) * grain
        outs.append(code * unit)
        table = s[which + "s"].double()
        table[pages, slots] = unit.squeeze(-1)
        tables.append(table)
    return tuple(outs + tables)


def _exact_tree(s):
    c = s["case"]
    G, scale = c["group"], 1.0 / math.sqrt(c["dim"])
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    row = 0
    for b, (t, n) in enumerate(zip(s["total"], s["new"])):
        pages = s["table"][b].long()
        pos = torch.arange(t, device="cuda")
        page = torch.div(pos, c["page"], rounding_mode="floor")
        kv = []
        for which in ("k", "v"):
            x = s[which][pages[page], pos - page * c["page"]]
            if c["fmt"] != "16bit":
                x = x.contiguous().view(torch.float8_e4m3fn).float() if c["fmt"] == "e4m3" else x
                x = x.double() * s[which + "s"][pages[page], pos - page * c["page"]].double().unsqueeze(-1)
            kv.append(x.double())
        seen = torch.zeros(n, t, dtype=torch.bool)
        for i, parent in enumerate(s["parents_of"][b]):
            if i:
                seen[i] = seen[parent]
            seen[i, t - n + i] = True
        width = seen.sum(1)
        for i in range(n):
            seen[i, max(0, t - n + int(width[i]) - c["window"]) if c["window"] else 0:t - n] = True
        seen = seen.cuda()
        for h in range(c["heads"] * G):
            score = (s["q"][row:row + n, h].double() @ kv[0][:, h // G].T * scale).masked_fill(~seen, -math.inf)
            out[row:row + n, h] = torch.softmax(score, -1) @ kv[1][:, h // G]
        row += n
    return out


def exact(case, seed):
    c = case
    if c["op"] in ("plan", "verify"):  # whole numbers
        return None
    s = prepare(case, seed)
    s["rows_of_table"] = s["table"].tolist()
    if c["op"] == "rotate":
        return _exact_rotate(s)
    if c["op"] == "tree":
        s["parents_of"] = _parents(c, s["new"])
        return _exact_tree(s)
    outs = []
    for x in (s["k"], s["v"], s["ks"], s["vs"]):
        if x is None:
            continue
        x = x.view(torch.float8_e4m3fn) if c["fmt"] == "e4m3" and x.dim() == 4 else x
        if "float" not in str(x.dtype):
            outs.append(None)
            continue
        y = x.float().double()
        to, source = [], []
        for b, path in enumerate(_kept(c, s["new"])):
            base = s["total"][b] - s["new"][b]
            for k, i in enumerate(path):
                to.append(_place64(s, b, base + k))
                source.append(_place64(s, b, base + i))
        pick = lambda places: tuple(_ints([p[i] for p in places], torch.int64) for i in (0, 1))  # noqa: E731
        y[pick(to)] = y[pick(source)]
        outs.append(y)
    return (*outs, None)
