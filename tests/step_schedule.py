"""How attention over trees with many rows is divided among blocks, and how a
block's roles wait for one another, for tests without a GPU.

pieces() gives every block's pieces as (tiles of tokens, tiles of rows, rows):
the division of a call's items (one sequence, kv head and 256 rows each, in
tiles of 128 tokens) among equal shares of their line.  Block runs the roles of
one block over them: a walking role that hands pieces on through a ring of four,
loads, products and two warpgroups of softmax.  Barriers keep a phase's parity
and no more, as the device's do.  Nothing here computes attention."""

import random

RING, TOKENS, ROWS, TILE_ROWS, SHARES = 4, 128, 256, 128, 152


def _ragged(seed, batch, lo, hi, most):
    r = random.Random(seed)
    lens = [r.randint(lo, hi) for _ in range(batch)]
    return lens, [min(t, r.randint(max(1, most // 4), most)) for t in lens]


# lens, new, heads, group, window: calls that give some blocks a shared piece and, behind it, more pieces in a row of
# a single tile each than the ring holds
CASES = {
    "ragged": (*_ragged(1, 256, 50, 300, 16), 4, 4, 0),
    "ragged_heads": (*_ragged(2, 64, 50, 200, 16), 12, 4, 0),
    "one_of_two_tiles": (([200] + [100] * 15) * 48, [12] * 768, 2, 4, 0),
    "one_of_many_tiles": (([520] + [60] * 31) * 24, ([9] + [11] * 31) * 24, 2, 4, 0),
    "wide_among_them": (*_ragged(3, 300, 40, 260, 40), 4, 4, 0),
    "window": (*_ragged(4, 200, 300, 1500, 20), 4, 3, 64),
    "sorted": (sorted(_ragged(5, 400, 30, 400, 16)[0], reverse=True), [16] * 400, 2, 6, 0),
}


def items(lens, new, heads, group, window=0):
    """(tiles of tokens, rows) of every item, along the line."""
    out = []
    for t, n in zip(lens, new):
        first, last = max(t - n - window, 0) if window else 0, t
        tiles = 1 if first >= last else -(-last // TOKENS) - first // TOKENS
        for _ in range(heads):
            out += [(tiles, min(ROWS, n * group - r)) for r in range(0, n * group, ROWS)]
    return out


def pieces(lens, new, heads, group, window=0, whole=True, shares=SHARES):
    """The pieces of each block: (tiles of tokens of the piece, rows)."""
    line = items(lens, new, heads, group, window)
    total = sum(n for n, _ in line)
    shares = max(min(shares, total), 1)
    each, rest = divmod(total, shares)
    start = [each * c + rest * c // shares for c in range(shares + 1)]
    blocks, at, c = [[] for _ in range(shares)], 0, 0
    for tiles, rows in line:
        end = at + tiles
        while start[c + 1] <= at:
            c += 1
        if whole:  # the block that an item begins in does all of it
            blocks[c].append((tiles, rows))
        else:
            k, x = c, at
            while x < end:
                upto = min(end, start[k + 1])
                blocks[k].append((upto - x, rows))
                x, k = upto, k + 1
        at = end
    return blocks


def own_tiles(piece, i):
    """Tiles of tokens that warpgroup i takes of a piece: of a narrow one every second."""
    count, rows = piece
    if rows <= TILE_ROWS:
        return (count - i + 1) // 2
    return count


def shared(piece):
    return piece[1] <= TILE_ROWS and piece[0] > 1


def run_of_single_tiles(block):
    """The longest run of pieces of one tile and no more than 128 rows behind a shared one."""
    longest = run = 0
    behind = False
    for p in block:
        if shared(p):
            behind, run = True, 0
        elif own_tiles(p, 1) == 0:
            run += behind
            longest = max(longest, run)
        else:
            behind, run = False, 0
    return longest


class Barrier:
    def __init__(self, arrivals):
        self.need, self.left, self.phase = arrivals, arrivals, 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left, self.phase = self.need, self.phase + 1

    def after(self, turn):
        """A wait for the phase of `turn`'s parity: over when that one is, and not when the next of it has begun."""
        return lambda: self.phase & 1 != turn & 1


def soon():
    """A step that waits for nothing (others may come between)."""
    return True


class Block:
    """The roles over one block's pieces.  `search_first`: a warpgroup looks for its next piece, however many it has
    no tiles of lie between, before it ends the one at hand; else it ends that one as soon as it meets such a piece."""

    WARPS = 2  # of a warpgroup

    def __init__(self, pieces, slots, search_first=False):
        self.pieces, self.slots, self.search_first = list(pieces) + [None], slots, search_first
        W = self.WARPS

        def pair(n):
            return [Barrier(n), Barrier(n)]

        self.q_full, self.s_full, self.p_full, self.o_full = pair(W), pair(1), pair(W), pair(1)
        self.half_full, self.half_read = pair(W), pair(W)
        self.kv_full, self.kv_free = ([Barrier(1) for _ in range(slots)] for _ in range(2))
        self.piece_full, self.piece_free = [Barrier(1) for _ in range(RING)], [Barrier(2 + 2 * W) for _ in range(RING)]
        self.reading = {(i, w): set() for i in range(2) for w in range(W)}  # accumulators that a warp is reading

    def walk(self):
        for n in range(len(self.pieces)):
            if n >= RING:
                yield self.piece_free[n % RING].after(n // RING - 1)
            self.piece_full[n % RING].arrive()

    def take(self, n):
        yield self.piece_full[n % RING].after(n // RING)
        self.piece_free[n % RING].arrive()

    def load(self):
        entry = 0
        for n, piece in enumerate(self.pieces):
            yield from self.take(n)
            for _ in range(2 * piece[0] if piece else 0):
                s, use = entry % self.slots, entry // self.slots
                if use:
                    yield self.kv_free[s].after(use - 1)
                self.kv_full[s].arrive()
                entry += 1

    def anew(self, i):
        """A product into accumulator i that keeps nothing of what is there."""
        assert not any(i in r for r in self.reading.values()), "an accumulator is overwritten while it is read"

    def multiply(self):
        S, entry, q, p = self.slots, 0, [0, 0], [0, 0]
        full = lambda e: self.kv_full[e % S].after(e // S)  # noqa: E731
        for n, piece in enumerate(self.pieces):
            yield from self.take(n)
            if piece is None:
                return
            count, rows = piece
            if rows <= TILE_ROWS:
                qk = pv = 0

                def scores():
                    return qk < count and qk < pv + 2 and full(entry + 2 * qk)() and \
                        (qk > 1 or self.q_full[qk].after(q[qk])())

                def values():
                    return pv < qk and full(entry + 2 * pv + 1)() and self.p_full[pv & 1].after(p[pv & 1])()

                while pv < count:
                    yield lambda: scores() or values()
                    if scores():
                        if qk < 2:
                            q[qk] += 1
                        self.s_full[qk & 1].arrive()
                        self.kv_free[(entry + 2 * qk) % S].arrive()
                        qk += 1
                    else:
                        p[pv & 1] += 1
                        if pv < 2:
                            self.anew(pv)
                        self.kv_free[(entry + 2 * pv + 1) % S].arrive()
                        if pv + 2 >= count:
                            self.o_full[pv & 1].arrive()
                        pv += 1
                entry += 2 * count
                continue
            yield full(entry)
            for i in range(2):
                yield self.q_full[i].after(q[i])
                q[i] += 1
                self.s_full[i].arrive()
            self.kv_free[entry % S].arrive()
            entry += 1
            for j in range(count):
                more = j + 1 < count
                yield full(entry)
                for i in range(2):
                    yield self.p_full[i].after(p[i])
                    p[i] += 1
                    if j == 0:
                        self.anew(i)
                    if more:
                        if i == 0:
                            yield full(entry + 1)
                        self.s_full[i].arrive()
                    else:
                        self.o_full[i].arrive()
                self.kv_free[entry % S].arrive()
                if more:
                    self.kv_free[(entry + 1) % S].arrive()
                entry += 2 if more else 1

    def soften(self, i, warp):
        s = o = halves = taken = 0
        at, reading = None, self.reading[i, warp]  # at: the piece at hand
        while True:
            while True:
                piece = self.pieces[taken]
                yield from self.take(taken)
                taken += 1
                skipped = piece is not None and own_tiles(piece, i) == 0
                if not skipped or (at is not None and not self.search_first):
                    break
            if at is not None:  # its end
                yield self.o_full[i].after(o)
                o += 1
                reading.add(i)
                if shared(at):
                    self.half_full[i].arrive()
                    yield self.half_full[i ^ 1].after(halves)
                    halves += 1
                    reading.add(i ^ 1)
                yield soon
                reading.clear()
                if shared(at):
                    self.half_read[i].arrive()
                at = None
            if skipped:
                continue
            if piece is None:
                return
            self.q_full[i].arrive()
            at = piece
            for j in range(own_tiles(piece, i)):
                yield self.s_full[i].after(s)
                s += 1
                if j == 0 and halves > 0:
                    yield self.half_read[i ^ 1].after(halves - 1)
                self.p_full[i].arrive()

    def run(self, rng):
        """The names of the roles that wait for ever: none when all end."""
        roles = {"walk": self.walk(), "load": self.load(), "multiply": self.multiply()}
        roles |= {"softmax %d.%d" % at: self.soften(*at) for at in self.reading}
        waits = dict.fromkeys(roles, soon)
        while roles:
            ready = [name for name in roles if waits[name]()]
            if not ready:
                return sorted(roles)
            name = rng.choice(ready)
            try:
                waits[name] = next(roles[name])
            except StopIteration:
                del roles[name]
        return []
