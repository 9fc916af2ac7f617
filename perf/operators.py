"""What the paged key/value cache operators are timed on, and their plain forms.

Three operators around one paged cache: `write` stores new tokens' keys and
values (as 8-bit codes with a binary32 scale per token and head, or as they
are), `read` takes tokens out again, `attend` is the attention of the new
tokens of every sequence over its cached ones (a chunk of a prompt, or one
token each).  run() computes them with elementary torch operations in binary32
when `own` is false and through the package's entry points when it is true.
"""

import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
_LIMIT = {"int8": 127.0, "e4m3": 448.0}


def _case(name, op, dtype, fmt, heads, group, dim, page, batch, new, ctx, ragged=True, window=0, layout="thd", shape=1):
    return {"name": name, "op": op, "dtype": dtype, "fmt": fmt, "heads": heads, "group": group, "dim": dim,
            "page": page, "batch": batch, "new": new, "ctx": ctx, "ragged": ragged, "window": window,
            "layout": layout, "shape": shape}


def listed():
    return [
        # one decoding step's append for 32 users: the smallest write, all latency
        _case("write_tokens_int8", "write", "bf16", "int8", 8, 4, 128, 16, 32, 1, 4096),
        # four prompts' keys and values into the cache, cut from a fused projection
        _case("write_prompts_e4m3", "write", "bf16", "e4m3", 8, 4, 128, 16, 4, 4096, 4096),
        # one short conversation taken out again, pages that end inside a tile
        _case("read_short_e4m3", "read", "fp16", "e4m3", 8, 4, 64, 24, 1, 333, 333),
        # 32 users' caches of the framework's 4096 tokens, read back as 16-bit values to be sent on
        _case("read_users_int8", "read", "bf16", "int8", 8, 4, 128, 16, 32, 4096, 4096, ragged=False),
        # one user's token over a short context: the smallest attention call
        _case("token_short_bf16", "attend", "bf16", "16bit", 8, 4, 128, 16, 1, 1, 517),
        # 64 users' tokens over contexts up to the framework's 4096 tokens
        _case("tokens_batch_bf16", "attend", "bf16", "16bit", 8, 4, 128, 16, 64, 1, 4096),
        # 32 users' tokens over long contexts held in 8 bits: the largest read of a cache
        _case("tokens_long_int8", "attend", "bf16", "int8", 8, 4, 128, 64, 32, 1, 32768, layout="htd"),
        # one user's token over a whole book: few rows, one long axis
        _case("token_book_e4m3", "attend", "bf16", "e4m3", 8, 8, 128, 64, 1, 1, 131072 + 5),
        # heads that share nothing, small head size, odd lengths
        _case("tokens_unshared_fp16", "attend", "fp16", "16bit", 12, 1, 64, 24, 17, 1, 1999),
        # short questions onto earlier turns
        _case("turns_fp16", "attend", "fp16", "16bit", 8, 4, 128, 16, 6, 97, 1500),
        # a chunk of a long prompt
        _case("chunk_long_bf16", "attend", "bf16", "16bit", 8, 4, 128, 16, 1, 4096, 32768),
        # ragged chunks of several prompts over an 8-bit cache, sliding window
        _case("chunks_window_int8", "attend", "bf16", "int8", 8, 4, 128, 64, 5, 2048, 12000, window=4096),
    ]


def draw(rng):
    def log_int(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    for _ in range(10000):
        op = rng.choice(["write", "read", "attend", "attend", "attend"])
        c = {"op": op, "dtype": rng.choice(["bf16", "bf16", "fp16"]), "fmt": rng.choice(["16bit", "int8", "e4m3"]),
             "heads": rng.choice([1, 2, 3, 8, 12]), "group": rng.choice([1, 2, 4, 6, 8]),
             "dim": rng.choice([64, 80, 96, 128, 128]), "page": rng.choice([16, 16, 24, 32, 64]),
             "batch": log_int(1, 64), "ragged": rng.random() < 0.8, "window": 0,
             "layout": rng.choice(["thd", "htd"]), "shape": rng.randrange(1 << 30)}
        c["ctx"] = log_int(64, 131072)
        if op == "read":
            c["new"] = c["ctx"]
        elif rng.random() < 0.5:
            c["new"] = 1
        else:
            c["new"] = log_int(2, min(4096, c["ctx"]))
        if op == "attend" and rng.random() < 0.25:
            c["window"] = log_int(16, c["ctx"])
        w = work(c)
        pool = sum(_lengths(c)[0]) * c["heads"] * c["dim"] * 2 * _elem(c)
        if w["bytes"] <= 0.8e9 and pool <= 2.2e9 and w["flops"] <= 1.5e12 and (op != "read" or w["bytes"] >= 1e4):
            return c
    raise RuntimeError("no case of the ranges drawn")


def _elem(c):
    return 2 if c["fmt"] == "16bit" else 1


def _lengths(c):
    """(tokens cached, new tokens) of every sequence; the new ones are the last of the cached ones."""
    r = random.Random(c["shape"])
    total, new = [], []
    for b in range(c["batch"]):
        t = c["ctx"] if b == 0 or not c["ragged"] else r.randint(max(1, c["ctx"] // 4), c["ctx"])
        n = c["new"] if b == 0 or not c["ragged"] else r.randint(max(1, c["new"] // 4), c["new"])
        total.append(t)
        new.append(t if c["op"] == "read" else min(n, t))
    return total, new


def _first(c, pos):
    """The first position that a token at `pos` attends to."""
    return max(0, pos - c["window"] + 1) if c["window"] else 0


def work(case):
    c = case
    total, new = _lengths(c)
    T, H, D = sum(new), c["heads"], c["dim"]
    stored = H * (2 * D * _elem(c) + (8 if c["fmt"] != "16bit" else 0))  # K and V of one token, with scales
    if c["op"] in ("write", "read"):
        return {"bytes": T * (2 * H * D * 2 + stored), "flops": 0}
    pairs = 0
    keys = 0
    for t, n in zip(total, new):
        keys += t - _first(c, t - n)
        if c["window"]:
            pairs += sum(p + 1 - _first(c, p) for p in range(t - n, t))
        else:
            pairs += n * (t - n) + n * (n + 1) // 2
    heads = H * c["group"]
    return {"bytes": 2 * T * heads * D * 2 + keys * stored, "flops": 4 * D * heads * pairs}


# ------------------------------------------------------------------ inputs
def _values(gen, shape, scale, dtype):
    """N(0, 1) times one scale per head (the second last axis)."""
    x = torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
    return (x * scale[:, None]).to(dtype)


def _quantise(x, fmt):
    """Codes (as bytes) and scales of 16-bit vectors x[..., D]: a = max|x|, scale = a / L, code = x * (L / a)."""
    x = x.float()
    a = x.abs().amax(-1)
    limit = torch.full_like(a, _LIMIT[fmt])
    scale = a / limit
    inv = torch.where(a > 0, (limit / a).clamp(max=torch.finfo(torch.float32).max), torch.zeros_like(a))
    y = torch.clamp(x * inv[..., None], -_LIMIT[fmt], _LIMIT[fmt])
    if fmt == "int8":
        return torch.round(y).nan_to_num(0.0).to(torch.int8), scale
    return y.to(torch.float8_e4m3fn).view(torch.int8), scale


def prepare(case, seed):
    c = case
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    dtype = _DTYPES[c["dtype"]]
    total, new = _lengths(c)
    H, D, P, B = c["heads"], c["dim"], c["page"], c["batch"]
    need = [-(-t // P) for t in total]
    pages = sum(need) + 3
    # the pages of all sequences lie mixed in the pool
    perm = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    table = torch.zeros(B, max(need), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    cu = [0]
    for n in new:
        cu.append(cu[-1] + n)
    T = cu[-1]
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
    s = {"case": c, "k": k, "v": v, "ks": ks, "vs": vs, "table": table, "total": total, "new": new, "cu": cu,
         "dtype": dtype, "scale": 1.0 / math.sqrt(D)}
    if c["op"] == "attend":
        s["q"] = torch.randn(T, H * c["group"], D, generator=gen, device="cuda").to(dtype)
    elif c["op"] == "write":
        # K and V as the last two thirds of a fused projection's output
        qkv = torch.cat([_values(gen, (T, H, D), h, dtype) for h in (k_head, k_head, v_head)], 1)
        s["qkv"], s["k_new"], s["v_new"] = qkv, qkv[:, H:2 * H], qkv[:, 2 * H:]
    s["cu_dev"] = torch.tensor(cu, dtype=torch.int32, device="cuda")
    s["len_dev"] = torch.tensor(total, dtype=torch.int32, device="cuda")
    if own:
        import compression_coupled_collectives_gb300 as cc

        fmt = {"16bit": cc.CCCL_KV_16BIT, "int8": cc.CCCL_KV_INT8, "e4m3": cc.CCCL_KV_E4M3}[c["fmt"]]
        s["cc"] = cc
        s["cache"] = cc.KvCache(k, v, ks, vs, dtype=dtype, fmt=fmt)
        s["batch"] = cc.KvBatch(table, s["cu_dev"], s["len_dev"], n_tokens=T, max_new=max(new), max_len=max(total))
        s["ws"] = cc.empty_kv_workspace(s["cache"], s["batch"], H * c["group"])
        if c["op"] == "attend":
            s["out"] = torch.empty_like(s["q"])
        else:
            s["k_out"], s["v_out"] = (torch.empty(T, H, D, dtype=dtype, device="cuda") for _ in range(2))
    return s


# ------------------------------------------------------------------ one pass
def _gather(s, b, lo, hi):
    """K and V of positions lo..hi-1 of sequence b, [tokens, heads, dim] in binary32."""
    P = s["case"]["page"]
    rows = s["table"][b, lo // P:-(-hi // P)].long()
    off = lo - lo // P * P
    got = []
    for data, scales in ((s["k"], s["ks"]), (s["v"], s["vs"])):
        x = data[rows].flatten(0, 1)[off:off + hi - lo]
        if scales is not None:
            if s["case"]["fmt"] == "e4m3":
                x = x.view(torch.float8_e4m3fn)
            x = x.float() * scales[rows].flatten(0, 1)[off:off + hi - lo][..., None]
        got.append(x.float())
    return got


def _plain_write(s):
    c, P = s["case"], s["case"]["page"]
    pages, slots = [], []
    for b, (t, n) in enumerate(zip(s["total"], s["new"])):
        pos = torch.arange(t - n, t, device="cuda")
        pages.append(s["table"][b].long()[pos // P])
        slots.append(pos % P)
    pages, slots = torch.cat(pages), torch.cat(slots)
    if c["fmt"] == "16bit":
        s["k"][pages, slots], s["v"][pages, slots] = s["k_new"], s["v_new"]
        return s["k"], s["v"]
    outs = []
    for x, data, scales in ((s["k_new"], s["k"], s["ks"]), (s["v_new"], s["v"], s["vs"])):
        codes, scale = _quantise(x, c["fmt"])
        data[pages, slots] = codes
        scales[pages, slots] = scale
        back = data[pages, slots]
        back = back.view(torch.float8_e4m3fn).float() if c["fmt"] == "e4m3" else back.float()
        outs.append((back * scales[pages, slots][..., None]).to(s["dtype"]))
    return outs[0], outs[1], s["ks"], s["vs"]


def _plain_read(s):
    ks, vs = zip(*[_gather(s, b, 0, t) for b, t in enumerate(s["total"])])
    return torch.cat([x.to(s["dtype"]) for x in ks]), torch.cat([x.to(s["dtype"]) for x in vs])


def _plain_attend(s):
    c, G = s["case"], s["case"]["group"]
    out = torch.empty_like(s["q"])
    for b, (t, n) in enumerate(zip(s["total"], s["new"])):
        lo = _first(c, t - n)
        k, v = _gather(s, b, lo, t)
        pos = torch.arange(t - n, t, device="cuda")[:, None]
        at = torch.arange(lo, t, device="cuda")[None, :]
        hidden = at > pos
        if c["window"]:
            hidden |= at <= pos - c["window"]
        q = s["q"][s["cu"][b]:s["cu"][b + 1]].float()
        for h in range(c["heads"]):
            qh = q[:, h * G:(h + 1) * G].transpose(0, 1)  # [group, new, dim]
            x = torch.matmul(qh, k[:, h].t()) * s["scale"]
            x.masked_fill_(hidden, float("-inf"))
            x -= x.amax(-1, keepdim=True)
            x.exp_()
            o = torch.matmul(x, v[:, h]) / x.sum(-1, keepdim=True)
            out[s["cu"][b]:s["cu"][b + 1], h * G:(h + 1) * G] = o.transpose(0, 1).to(s["dtype"])
    return out


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return {"write": _plain_write, "read": _plain_read, "attend": _plain_attend}[op](s)
    cc = s["cc"]
    if op == "attend":
        cc.cccl_kv_attention(s["cache"], s["batch"], s["q"], s["out"], s["ws"], scale=s["scale"],
                             window=s["case"]["window"])
        return s["out"]
    if op == "write":
        cc.cccl_kv_write(s["cache"], s["batch"], s["k_new"], s["v_new"], s["ws"])
        if s["case"]["fmt"] == "16bit":
            return s["k"], s["v"]
    # what was written, as the values that the codes stand for
    cc.cccl_kv_read(s["cache"], s["batch"], s["k_out"], s["v_out"], s["ws"])
    if op == "write":
        return s["k_out"], s["v_out"], s["ks"], s["vs"]
    return s["k_out"], s["v_out"]


# ------------------------------------------------------------------ in 64 bits
def _stored64(s, which, b, positions):
    """The stored K ("k") or V ("v") of the given positions of sequence b, [tokens, heads, dim] in binary64."""
    page = torch.div(positions, s["case"]["page"], rounding_mode="floor")
    pages, slots = s["table"][b].long()[page], positions - page * s["case"]["page"]
    x = s[which][pages, slots]
    if s["case"]["fmt"] == "16bit":
        return x.double()
    x = x.contiguous().view(torch.float8_e4m3fn).float().double() if s["case"]["fmt"] == "e4m3" else x.double()
    return x * s[which + "s"][pages, slots].double().unsqueeze(-1)


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "write":
        outs, tables = [], []
        pages, slots = [], []
        for b, (t, n) in enumerate(zip(s["total"], s["new"])):
            for p in range(t - n, t):
                pages.append((b, p // c["page"]))
                slots.append(p % c["page"])
        rows = s["table"].cpu()
        pages = torch.tensor([int(rows[b, i]) for b, i in pages], device="cuda")
        slots = torch.tensor(slots, device="cuda")
        for x, which in ((s["k_new"], "k"), (s["v_new"], "v")):
            x = x.double()
            if c["fmt"] == "16bit":
                whole = s[which].double()
                whole[pages, slots] = x
                outs.append(whole)
                continue
            limit = _LIMIT[c["fmt"]]
            biggest = x.abs().max(dim=-1, keepdim=True).values
            unit = biggest / limit
            ratio = torch.where(biggest > 0, x / unit, torch.zeros_like(x))
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
    if c["op"] == "read":
        return tuple(torch.cat([_stored64(s, w, b, torch.arange(t, device="cuda")) for b, t in enumerate(s["total"])])
                     for w in ("k", "v"))
    if work(c)["flops"] > 6e12:
        return None
    G, scale = c["group"], 1.0 / math.sqrt(c["dim"])
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    row = 0
    for b, (t, n) in enumerate(zip(s["total"], s["new"])):
        pos = torch.arange(t, device="cuda")
        k, v = _stored64(s, "k", b, pos), _stored64(s, "v", b, pos)
        for i in range(0, n, 512):  # some tokens at a time
            m = min(512, n - i)
            here = t - n + i + torch.arange(m, device="cuda")
            seen = pos[None] <= here[:, None]
            if c["window"]:
                seen &= pos[None] > here[:, None] - c["window"]
            last = int(here[-1]) + 1
            for h in range(c["heads"] * G):
                q = s["q"][row + i:row + i + m, h].double()
                score = (q @ k[:last, h // G].T * scale).masked_fill(~seen[:, :last], -math.inf)
                out[row + i:row + i + m, h] = torch.softmax(score, -1) @ v[:last, h // G]
        row += n
    return out
