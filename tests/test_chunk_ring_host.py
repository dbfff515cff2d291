"""The ring through which chunk_attn_kernel's softmax warps hand a piece's maxima
and sums to the epilogue warps (csrc/chunk_attn.cu): no entry may be written for a
later piece before it has been read.

Tiles alternate between the two softmax warpgroups, so in a piece of one tile one
of them has nothing to wait for and writes its entry at once.  The tests take the
kernel's waits as they stand: as a graph of what happens before what, over every
short run of piece lengths, and as a run of all the roles on mbarriers with their
arrival counts and phase parities, in random order."""
import itertools
import os
import random
import re

import pytest

SOURCE = os.path.join(os.path.dirname(__file__), "..", "tree_speculative_decoding_jt_gb300", "csrc", "chunk_attn.cu")
with open(SOURCE) as f:
    RING = int(re.search(r"constexpr int kRing = (\d+);", f.read()).group(1))
BUFFERS = 3  # score buffers: S(t) waits for PV(t - 3)


def exposed(lengths, ring):
    """Pieces whose entry some warpgroup may write before the epilogue has read
    the entry of the piece `ring` before it."""
    first = [sum(lengths[:n]) for n in range(len(lengths))]
    tiles = sum(lengths)
    piece = [n for n, c in enumerate(lengths) for _ in range(c)]
    # read[event]: the epilogue has surely read the entries of the pieces up to
    # this one when the event has happened
    s, p, pv, word = ([-1] * tiles for _ in range(4))
    done = [[-1] * tiles, [-1] * tiles]      # what warpgroup w knows past its tile t
    know = [-1, -1]
    for t in range(tiles):
        w = t & 1
        s[t] = pv[t - BUFFERS] if t >= BUFFERS else -1
        know[w] = max(know[w], s[t], word[t - 1] if t else -1)
        word[t] = p[t] = done[w][t] = know[w]
        n = piece[t]
        # the epilogue gives O up past its read of the piece's entry
        pv[t] = max(p[t], pv[t - 1] if t else -1, n - 1 if t == first[n] else -1)
    bad = []
    for n in range(ring, len(lengths)):
        last = first[n] + lengths[n] - 1
        for w in (0, 1):
            t = last if last & 1 == w else last - 1
            if (done[w][t] if t >= 0 else -1) < n - ring:
                bad.append((n, w))
    return bad


def test_a_shorter_ring_is_exposed():
    """What the graph says of rings that are too short, so that it is seen to tell."""
    assert not exposed([2, 2, 2, 2, 2, 2, 2], 4)
    assert exposed([2, 2, 1, 1, 1, 1, 1], 4) and exposed([5, 4, 3, 2, 1, 1, 1, 1], 4)
    assert exposed([2, 1, 1, 1, 1], 3)


def test_no_entry_is_written_before_it_has_been_read():
    for n in (6, 7, 8):
        for lengths in itertools.product((1, 2, 3), repeat=n):
            assert not exposed(lengths, RING), lengths
    rng = random.Random(1)
    for _ in range(3000):
        lengths = [rng.choice([1, 1, 1, 2, 2, 3, 4, 5, 9]) for _ in range(rng.randint(6, 40))]
        assert not exposed(lengths, RING), lengths


class Barrier:
    def __init__(self, count):
        self.count = self.pending = count
        self.phase = 0

    def arrive(self):
        self.pending -= 1
        if self.pending == 0:
            self.pending = self.count
            self.phase += 1

    def passed(self, parity):  # the phase of this parity has completed
        return (self.phase & 1) != parity


def simulate(lengths, ring, rng, slow):
    """All roles of a CTA pair in random order (the epilogue `slow` times as
    seldom); the entries that the epilogue read for each (CTA, rows, piece)."""
    ranks, quarters = (0, 1), range(4)
    s_full = [[Barrier(1) for _ in range(BUFFERS)] for _ in ranks]
    o_done = [[Barrier(1) for _ in range(BUFFERS)] for _ in ranks]
    p_full = [Barrier(8) for _ in range(BUFFERS)]
    o_free = Barrier(8)
    x_bar = {(x, i, q): Barrier(2) for x in ranks for i in range(ring) for q in quarters}
    words, xch, got = {}, {}, {}

    def score_issuer():
        for t in range(sum(lengths)):
            if t >= BUFFERS:
                while not o_done[0][t % BUFFERS].passed((t // BUFFERS - 1) & 1):
                    yield
            for x in ranks:
                s_full[x][t % BUFFERS].arrive()
            yield

    def output_issuer():
        t = 0
        for n, count in enumerate(lengths):
            if n:
                while not o_free.passed((n - 1) & 1):
                    yield
            for _ in range(count):
                while not p_full[t % BUFFERS].passed((t // BUFFERS) & 1):
                    yield
                for x in ranks:
                    o_done[x][t % BUFFERS].arrive()
                t += 1
                yield

    def softmax(x, wg, q):
        at = 0
        for n, count in enumerate(lengths):
            mine = 0
            for t in range(at, at + count):
                if t & 1 != wg:
                    continue
                while not s_full[x][t % BUFFERS].passed((t // BUFFERS) & 1):
                    yield
                while t and words.get((x, q, (t - 1) % 4)) != t:  # the partner's word of the tile before
                    yield
                words[x, q, t % 4] = t + 1
                mine += 1
                yield
                p_full[t % BUFFERS].arrive()
            at += count
            xch[x, n % ring, wg, q] = (n, mine)
            yield
            x_bar[x, n % ring, q].arrive()

    def epilogue(x, q):
        last = -1
        for n, count in enumerate(lengths):
            last += count
            while not x_bar[x, n % ring, q].passed((n // ring) & 1):
                yield
            got[x, q, n] = [xch.get((x, n % ring, wg, q)) for wg in (0, 1)]
            while not o_done[x][last % BUFFERS].passed((last // BUFFERS) & 1):
                yield
            o_free.arrive()
            yield

    roles = [(score_issuer(), 1.0), (output_issuer(), 1.0)]
    roles += [(softmax(x, wg, q), rng.uniform(0.2, 1.0)) for x in ranks for wg in (0, 1) for q in quarters]
    roles += [(epilogue(x, q), rng.uniform(0.2, 1.0) / slow) for x in ranks for q in quarters]
    steps = 0
    while roles:
        steps += 1
        assert steps < 400000, "the roles wait for one another"
        i = rng.choices(range(len(roles)), [w for _, w in roles])[0]
        if next(roles[i][0], roles) is roles:
            roles.pop(i)
    return got


@pytest.mark.parametrize("slow", [1, 30])
def test_the_roles_in_random_order_read_their_own_pieces(slow):
    for seed in range(25):
        rng = random.Random(seed)
        lengths = [2, 2, 1, 1, 1, 1, 1] if seed == 0 else [rng.choice([1, 1, 1, 2, 3, 4]) for _ in range(rng.randint(6, 14))]
        got = simulate(lengths, RING, rng, slow)
        starts = [sum(lengths[:n]) for n in range(len(lengths))]
        for (x, q, n), entries in got.items():
            own = [(n, sum(t & 1 == wg for t in range(starts[n], starts[n] + lengths[n]))) for wg in (0, 1)]
            assert entries == own, (seed, lengths, x, q, n, entries)
