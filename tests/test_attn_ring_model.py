"""A model of the tcgen05 attention kernel's load ring, its roles in any order (CPU only).

A block's producer loads K and V tiles into a ring of slots; per stream one issuer multiplies them
and hands the slots back, and a softmax group works between the two products. They meet at mbarriers,
of which a waiter sees only the parity: "the phase of this parity is complete" is also true two
phases later, and before the phase begins. The model takes one step of a random role at a time, lets
copies land in any order, and looks at every use: is the slot filled with the tile meant, is the
item's entry still that item, are the tile's bad-page marks still its own, does anyone arrive too
often or wait for ever.

``skips=True`` is an issuer that passes over the other stream's tiles of a split item without
waiting for them (the slots' hand-back counted by the stream that uses them): it must fail.
"""
import random

import pytest

ITEMS, GONE = 8, 8


class Barrier:
    def __init__(self, count):
        self.count = self.left = count
        self.phase = 0

    def arrive(self):
        assert self.left > 0
        self.left -= 1
        if self.left == 0:
            self.left, self.phase = self.count, self.phase + 1

    def done(self, parity):
        return (self.phase & 1) != parity


class Stream:
    """An issuer and its softmax group."""

    def __init__(self, own):
        self.own = own                       # its tiles, (item, tile), in order
        self.item, self.tile, self.end, self.split = -1, 0, 0, False
        self.scores, self.products = [], 0   # S issued: position of K; P V issued
        self.softmaxed, self.softmax_item = 0, 0


def _run(rng, streams, slots, skips):
    """'ok', or what went wrong."""
    items = [(streams == 2 and rng.random() < .6, rng.randint(1, 5)) for _ in range(rng.randint(4, 24))]
    first, seq = [], 0                       # number of an item's first tile
    for _, tiles in items:
        first.append(seq)
        seq += tiles
    full = [Barrier(1) for _ in range(slots)]
    empty = [Barrier(streams) for _ in range(slots)]
    content, flight = [None] * slots, []     # position loaded; copies on their way
    board, marks, published = {}, {}, 0
    load = [0, 0, 0]                         # the producer's item, tile, K or V
    st = [Stream([(i, t) for i, (split, tiles) in enumerate(items) for t in range(tiles)
                  if not split or t % 2 == s]) for s in range(streams)]
    upto = [[sum(j <= i for j, _ in q.own) for i in range(len(items))] for q in st]
    roles = ["load", "load", "land", "land"] + [("issue", q) for q in st] * 2 + [("softmax", q) for q in st]

    def hand_back(slot, twice):
        empty[slot].arrive()
        if twice:
            empty[slot].arrive()

    for _ in range(60000):
        if all(q.item == len(items) and q.products == len(q.scores) for q in st):
            return "ok"
        role = rng.choice(roles)
        if role == "load":
            i, t, kv = load
            if i > len(items):
                continue
            if t == kv == 0 and published == i:
                if i >= 2 and min(q.softmax_item for q in st) < i - 1:
                    continue                 # the query buffer of item i - 2 is in use
                board[i % ITEMS], published = i, i + 1
                if i == len(items):          # the last entry: no more items
                    load[0] += 1
                continue
            if i == len(items):
                continue
            pos = (first[i] + t) * 2 + kv
            slot = pos % slots
            if kv == 0:
                marks[(pos // 2) % GONE] = pos // 2
            if not empty[slot].done(((pos // slots) & 1) ^ 1):
                continue
            if any(f[0] == slot for f in flight):
                return "loaded over a copy in flight"
            flight.append((slot, pos))
            load[2] = 1 - kv
            load[1] += kv
            if load[1] == items[i][1]:
                load[0], load[1] = i + 1, 0
        elif role == "land":
            if flight:
                slot, pos = flight.pop(rng.randrange(len(flight)))
                content[slot] = pos
                full[slot].arrive()
        elif role[0] == "softmax":
            q = role[1]
            n = q.softmaxed
            if n < len(q.scores) and q.softmax_item == q.own[n][0]:
                i, t = q.own[n]
                if t == items[i][1] - 1:     # tokens past the end: V's rows are cleared first
                    pos = (first[i] + t) * 2 + 1
                    slot = pos % slots
                    if n > 0 and q.products < n or not full[slot].done((pos // slots) & 1):
                        continue
                    if content[slot] != pos or any(f[0] == slot for f in flight):
                        return "softmax: V of another tile"
                if marks[(first[i] + t) % GONE] != first[i] + t:
                    return "softmax: marks of another tile"
                if board[i % ITEMS] != i:
                    return "softmax: entry of another item"
                q.softmaxed += 1
            elif (q.softmax_item < min(published, len(items))
                  and q.products >= upto[st.index(q)][q.softmax_item]):
                q.softmax_item += 1
        else:
            q = role[1]
            s = st.index(q)
            k = q.products
            if k < len(q.scores) and k < q.softmaxed:
                pos = q.scores[k] + 1
                slot = pos % slots
                if full[slot].done((pos // slots) & 1):
                    if content[slot] != pos:
                        return "P V: V of another tile"
                    hand_back(slot, skips and items[q.own[k][0]][0])
                    q.products += 1
            if q.item < len(items) and q.tile >= q.end:
                i = q.item + 1
                arrivals = len(range(i % ITEMS, published, ITEMS))
                if (arrivals & 1) != ((i // ITEMS) & 1):
                    if board[i % ITEMS] != i:
                        return "issuer: entry of another item"
                    q.item = i
                    if i < len(items):
                        q.split, q.end = items[i]
                        q.tile = s if skips and q.split else 0
            elif q.item < len(items):
                pos = (first[q.item] + q.tile) * 2
                slot, v = pos % slots, (pos + 1) % slots
                if q.split and q.tile % 2 != s:
                    # (a V tile that this stream has still to multiply: the slot's next fill
                    # cannot be told yet)
                    if q.products < len(q.scores) and q.scores[q.products] + 1 + slots <= pos + 1:
                        continue
                    if full[slot].done((pos // slots) & 1) and full[v].done(((pos + 1) // slots) & 1):
                        if content[slot] != pos or content[v] != pos + 1:
                            return "passed: another tile"
                        empty[slot].arrive()
                        empty[v].arrive()
                        q.tile += 1
                elif len(q.scores) - q.products < 2 and full[slot].done((pos // slots) & 1):
                    if content[slot] != pos:
                        return "S: K of another tile"
                    hand_back(slot, skips and q.split)
                    q.scores.append(pos)
                    q.tile += 2 if skips and q.split else 1
    return "stuck"


def _outcomes(streams, slots, skips, runs, seed):
    rng, seen = random.Random(seed), {}
    for _ in range(runs):
        try:
            r = _run(rng, streams, slots, skips)
        except AssertionError:
            r = "arrived too often"
        seen[r] = seen.get(r, 0) + 1
    return seen


# head_dim to 64: two streams, 8 slots; to 128: two, 6; to 256: one, 3
@pytest.mark.parametrize("streams,slots", [(2, 8), (2, 6), (1, 3)])
def test_every_use_finds_its_tile(streams, slots):
    assert _outcomes(streams, slots, False, 400, 3) == {"ok": 400}


@pytest.mark.parametrize("slots", [6, 8])
def test_an_issuer_that_skips_fills_uses_wrong_tiles(slots):
    seen = _outcomes(2, slots, True, 100, 3)
    assert seen.get("ok", 0) < 100, seen
