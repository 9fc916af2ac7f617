"""The definitions of a step with drafted tokens (include/cccl_step.h) for tests:
plans, rotary positions, verification and kept tokens, in whole numbers or
binary64, and trees for the paged caches of kv_reference (none of the package's
code)."""

import math
import random

import torch

from kv_reference import Case


def trees(sizes, seed, wide=3):
    """Parents of random trees: the root first, every token hangs from an earlier one."""
    r = random.Random(seed)
    return [[-1] + [r.randint(max(0, (i - 1) // wide - 1), i - 1) for i in range(1, n)] if n else [] for n in sizes]


def ancestors(parents):
    """Every token's ancestors and itself, as bits of one number."""
    bits = []
    for i, p in enumerate(parents):
        bits.append((bits[p] if 0 <= p < i else 0) | 1 << i)
    return bits


def depths(parents):
    d = []
    for i, p in enumerate(parents):
        d.append(d[p] + 1 if 0 <= p < i else 0)
    return d


def words_of(bits, words):
    """int32 words of masks given as whole numbers."""
    out = []
    for m in bits:
        row = [m >> 32 * w & 0xFFFFFFFF for w in range(words)]
        out.append([w - (1 << 32) if w >> 31 else w for w in row])
    return out


class TreeCase(Case):
    """A cache whose new tokens see each other by masks: bits[b][i], a whole number a token."""

    def __init__(self, lens, new, bits=None, *, words=None, mask_pad=0, **kw):
        super().__init__(lens, new, **kw)
        self.bits = bits or [ancestors(p) for p in trees(new, kw.get("seed", 0) + 7)]
        self.words = words or max(1, -(-max(list(new) + [1]) // 32))
        rows = [w for b in self.bits for w in words_of(b, self.words)]
        self.mask = torch.full((self.T, self.words + mask_pad), -1, dtype=torch.int32, device=self.device)
        self.mask = self.mask[:, :self.words]
        if rows:
            self.mask.copy_(torch.tensor(rows, dtype=torch.int32))

    def visible(self, b, causal, window):
        n, t = self.new[b], self.lens[b]
        seen = torch.zeros(n, t, dtype=torch.bool)
        for i in range(n):
            on_path = list(range(max(t - n, 0)))
            on_path += [t - n + k for k in range(min(n, 32 * self.words)) if self.bits[b][i] >> k & 1 and t - n + k >= 0]
            if window:
                on_path = on_path[-window:]
            seen[i, on_path] = True
        return seen.to(self.device)


def plan(lens, new, held, table, free, count, page, parents, rows, width, words):
    """The plan as lists, or the name of what is reported when nothing is given to anyone."""
    B = len(lens)
    for b in range(B):
        if lens[b] < 0 or new[b] < 0 or not 0 <= held[b] <= width or lens[b] + new[b] > width * page:
            return "invalid"
        if (words and new[b] > 32 * words) or (parents is not None and new[b] > 1024):
            return "invalid"
    if sum(new) > rows or not 0 <= count <= len(free):
        return "invalid"
    table, cu, after, holds, slots, positions, masks = [list(r) for r in table], [0], [], [], [], [], []
    for b in range(B):
        cu.append(cu[-1] + new[b])
        after.append(lens[b] + new[b])
        need = max(0, -(-after[b] // page) - held[b])
        for j in range(need):
            if count == 0:
                return "capacity"
            count -= 1
            table[b][held[b] + j] = free[count]
        holds.append(held[b] + need)
        tree = list(range(-1, new[b] - 1)) if parents is None else parents[cu[b]:cu[b + 1]]
        positions += [lens[b] + d for d in depths(tree)]
        masks += ancestors(tree)
        for i in range(new[b]):
            p = lens[b] + i
            slots.append(table[b][p // page] * page + p % page)
    return {"table": table, "cu_tokens": cu, "kv_lens": after, "held": holds, "free_count": [count], "slots": slots,
            "positions": positions, "mask": words_of(masks, words) if words else None}


def rotated(x, positions, turns, magnitude, interleaved):
    """x [rows, heads, dim] with its rotary positions in binary64, and |a| + |b| of every value's pair."""
    R = 2 * len(turns)
    angle = torch.tensor([[(int(p) * int(t) & (1 << 64) - 1) / 2.0 ** 64 * 2 * math.pi for t in turns]
                          for p in positions], dtype=torch.float64, device=x.device)
    cos, sin = torch.cos(angle)[:, None] * magnitude, torch.sin(angle)[:, None] * magnitude
    y, size = x.double().clone(), torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    at = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    a, b = x[..., at[0]].double(), x[..., at[1]].double()
    y[..., at[0]], y[..., at[1]] = a * cos - b * sin, b * cos + a * sin
    size[..., at[0]] = size[..., at[1]] = a.abs() + b.abs()
    return y, size


def _limited(x):
    return min(x, 1.0) if x > 0 else 0.0  # (what is not a number is not above 0)


def verify(p, q, tokens, parents, uniform, cu, most=1024):
    """p, q: lists of rows of numbers.  Returns path, n_kept, next_token, in whole numbers as documented."""
    scale = 1 << 56

    def fixed(x):
        return int(_limited(x) * scale)

    path, n_kept, following = [None] * len(tokens), [], []
    for lo, hi in zip(cu, cu[1:]):
        n = min(hi - lo, most)
        if hi == lo:
            n_kept.append(0)
            following.append(-1)
            continue
        at, A, refused, left, kept = 0, 0, [], scale, [0]

        def weights(row, A, refused):
            out = [fixed(x) for x in p[row]]
            if q is not None and A:
                out = [max(0, x - (A * fixed(y) >> 53)) for x, y in zip(out, q[row])]
            for t in refused:
                out[t] = 0
            return out

        for i in range(1, n):
            x, up = tokens[lo + i], i - 1 if parents is None else parents[lo + i]
            if up != at or up >= i or not 0 <= x < len(p[0]):
                continue
            u = uniform[lo + i]
            px = _limited(p[lo + at][x])
            if q is None:
                keep = x not in refused and fixed(u) * left < fixed(px) * scale
            elif A == 0:
                keep = u * _limited(q[lo + at][x]) < px
            else:
                w = weights(lo + at, A, [])
                S = sum(w)
                keep = u * (S / scale) * _limited(q[lo + at][x]) < w[x] / scale
            if keep:
                at, A, refused, left = i, 0, [], scale
                kept.append(i)
            elif q is None:
                if x not in refused:
                    refused.append(x)
                    left = max(0, left - fixed(px))
            else:
                A += 1 << 53 if A == 0 else S >> 3
        w = weights(lo + at, A, refused)
        if sum(w) == 0:
            w = weights(lo + at, 0, [])
        goal, run, y = min(fixed(uniform[lo]) * sum(w) // scale, sum(w) - 1), 0, 0
        if sum(w):
            for y, x in enumerate(w):
                run += x
                if run > goal:
                    break
        for k in range(hi - lo):
            path[lo + k] = kept[k] if k < len(kept) else -1
        n_kept.append(len(kept))
        following.append(y if sum(w) else 0)
    return path, n_kept, following
