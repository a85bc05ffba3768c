"""The hand-offs of the K8/V8 attention kernel (attention_k8v8.cuh) on the CPU,
under random schedules: every role, every barrier and ring, with what stands in a
buffer in place of its numbers.  A barrier tells odd phases from even only, as the
hardware's do, so a wait that is lapped goes on too early or never.  The rings'
sizes are read from the kernel's source; the roles restate its loops.

Wrong schedules show as a buffer that holds something else than its reader
expects, or as a state in which nothing can go on."""
import os
import random
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.abspath(__file__)), "..", "fp8_paged_kv_append_gb300", "csrc")
SRC = open(os.path.join(CSRC, "attention_k8v8.cuh")).read()


def constant(name, value=r"(\d+)"):
    found = re.findall(rf"constexpr (?:int|uint32_t) {name} = {value}", SRC)
    assert len(found) == 1, name
    return found[0]


STAGES = [int(x) for x in constant("kStages", r"kWide \? (\d+) : (\d+)")]  # wide, narrow
K_TILES, V_HALVES, PIECES = (int(constant(n)) for n in ("kKTiles", "kVHalves", "kPieceRing"))
WIDEN = int(constant("kWidenWarps"))
INFO = 8      # tiles whose rejected pages are kept for the softmax
SOFTMAX = 2   # warps of a slot here (four in the kernel, all alike)


def test_the_source_still_has_what_is_restated_here():
    assert re.search(r"info\[\(tiles \+ tile\) & 7\]", SRC) and "info[tiles & 7] = bad" in SRC
    assert "nan_rows[(p_idx & 3) * 2" in SRC and PIECES == 4
    counts = {"kBarQEmpty": 2, "kBarKEmpty": 2, "kBarVEmpty": 2, "kBarPFull": 4, "kBarJoin": 8, "kBarTurn": 4,
              "kBarOEmpty": 8, "kBarTaken": 16}
    assert int(constant("kPieceReaders")) == counts["kBarTaken"]
    assert "kBarQEmpty && i < kBarKstFull) || (i >= kBarKEmpty && i < kBarSFull)) count = 2" in SRC
    assert "if (i == kBarJoin) count = 8" in SRC and "if (i >= kBarOEmpty) count = 8" in SRC


class Wrong(Exception):
    pass


def expect(holds, *what):
    if not holds:
        raise Wrong(what)


class Barrier:
    def __init__(self, count):
        self.count = self.left = count
        self.phase = 0

    def arrive(self):
        self.left -= 1
        if self.left == 0:
            self.left = self.count
            self.phase += 1

    def test(self, parity):
        """The phase of this parity is complete (or one before or behind it that looks
        the same)."""
        return self.phase & 1 != parity & 1


class Ring:
    def __init__(self, n):
        self.n, self.at, self.phase, self.wrapped = n, 0, 0, False

    def next(self):
        self.at += 1
        if self.at == self.n:
            self.at, self.phase, self.wrapped = 0, self.phase ^ 1, True


class Piece:
    """Tiles [0, tiles) of a segment, halves of 64 positions; turn: the slot of the first
    one, where there is one row tile."""
    def __init__(self, index, two, tiles, odd, turn, first_tile):
        self.index, self.two, self.tiles, self.turn = index, two, tiles, turn
        self.halves_all = 2 * tiles - odd
        self.first_tile = first_tile  # of all tiles of the CTA

    def halves(self, t):
        return 2 if 2 * t + 1 < self.halves_all else 1

    def own(self, w, count_only=False):
        tiles = range(self.tiles) if self.two else range(w ^ self.turn, self.tiles, 2)
        return sum(self.halves(t) for t in tiles) if count_only else list(tiles)


class Kernel:
    """One CTA.  variant: None, or a mistake that has to be found."""

    def __init__(self, shapes, wide, rng, variant=None):
        self.wide, self.rng, self.variant = wide, rng, variant
        self.stages = STAGES[0 if wide else 1]
        self.pieces, turn, tiles = [], 0, 0
        for i, (two, n, odd) in enumerate(shapes):
            self.pieces.append(Piece(i, two, n, odd, turn, tiles))
            tiles += n
            if not two and variant not in ("no turns", "no turns, no waits"):
                turn ^= n & 1
        warps = 2 + 2 * WIDEN + 2 + 2 * SOFTMAX
        self.bars = {}
        for name, n, count in (
                ("QFull", 2, 1), ("QEmpty", 2, 2), ("KstFull", self.stages, 1), ("KstEmpty", self.stages, WIDEN),
                ("VstFull", self.stages, 1), ("VstEmpty", self.stages, WIDEN), ("KFull", K_TILES, WIDEN),
                ("KEmpty", K_TILES, 2), ("VFull", V_HALVES, WIDEN), ("VEmpty", V_HALVES, 2), ("SFull", 2, 1),
                ("PFull", 4, SOFTMAX), ("ODone", 2, 1), ("OEmpty", 2, 2 * SOFTMAX), ("Join", 1, 2 * SOFTMAX),
                ("Turn", 2, SOFTMAX), ("Piece", PIECES, 1), ("Taken", PIECES, warps)):
            for i in range(n):
                self.bars[name, i] = Barrier(count)
        self.ring = [None] * PIECES
        self.nan_rows = [None] * PIECES
        self.staged = {"K": [None] * self.stages, "V": [None] * self.stages}
        self.tile = {"K": [[None] * WIDEN for _ in range(K_TILES)], "V": [[None] * WIDEN for _ in range(V_HALVES)]}
        self.info = [None] * INFO
        self.q, self.s = [None, None], [None, None]
        self.p = [[None] * SOFTMAX for _ in range(4)]
        self.o = [None, None]  # [piece, products added, warps that have still to read it]
        self.issued = [[], []]  # to the tensor cores, by slot

    # ---- waits: a role yields what has to hold before it goes on -----------------------------

    def wait(self, name, i, parity):
        bar = self.bars[name, i]
        return lambda: bar.test(parity)

    def arrive(self, name, i):
        self.bars[name, i].arrive()

    def get_piece(self, ring):
        yield self.wait("Piece", ring.at, ring.phase)
        piece = self.ring[ring.at]
        self.arrive("Taken", ring.at)
        ring.next()
        return piece

    # ---- the roles ----------------------------------------------------------------------------

    def load(self, side):
        """Codes; V's warp describes the pieces, K's loads the queries."""
        ring, dst, described = Ring(PIECES), Ring(self.stages), Ring(PIECES)
        full, empty = side + "stFull", side + "stEmpty"
        todo, uses, count = list(self.pieces) + [None], [0, 0], 0
        due = True
        while True:
            if due and side == "V" and todo:
                if described.wrapped:
                    yield self.wait("Taken", described.at, described.phase ^ 1)
                self.ring[described.at] = todo.pop(0)
                self.nan_rows[described.at] = set()
                self.arrive("Piece", described.at)
                described.next()
            due = False
            if not count:
                piece = yield from self.get_piece(ring)
                if piece is None:
                    return
                h, count = 0, piece.halves_all
            if dst.wrapped:
                yield self.wait(empty, dst.at, dst.phase ^ 1)
            if side == "K" and h % 2 == 0:
                self.info[(piece.first_tile + h // 2) % INFO] = (piece.index, h // 2)
            yield None
            self.staged[side][dst.at] = (piece.index, h)
            self.arrive(full, dst.at)
            dst.next()
            first = h == (0 if side == "V" else min(1, piece.halves_all - 1))
            h, count = h + 1, count - 1
            if first:
                due = True
                if side == "K":
                    for i in range(2 if piece.two else 1):
                        at = i if piece.two else (piece.index & 1 if self.wide else 0)
                        if uses[at]:
                            yield self.wait("QEmpty", at, (uses[at] - 1) & 1)
                        uses[at] += 1
                        yield None
                        self.q[at] = (piece.index, i)
                        self.arrive("QFull", at)

    def widen(self, side, rank):
        ring, src = Ring(PIECES), Ring(self.stages)
        dst = Ring(K_TILES if side == "K" else V_HALVES)
        while True:
            at = ring.at
            piece = yield from self.get_piece(ring)
            if piece is None:
                return
            for h in range(piece.halves_all):
                yield self.wait(side + "stFull", src.at, src.phase)
                if (side == "V" or h % 2 == 0) and dst.wrapped:
                    yield self.wait(side + "Empty", dst.at, dst.phase ^ 1)
                expect(self.staged[side][src.at] == (piece.index, h), "stage", side, piece.index, h)
                if side == "V":
                    self.nan_rows[at].add((piece.index, h))
                yield None
                self.tile[side][dst.at][rank] = (piece.index, h)
                self.arrive(side + "stEmpty", src.at)
                src.next()
                if side == "V" or h % 2 or h + 1 == piece.halves_all:
                    self.arrive(side + "Full", dst.at)
                    dst.next()

    def mma(self, w):
        """Barriers by lane: what each waits for next; `ready` as of the last look."""
        lanes = {"K": ["KFull", 0, 0], "V": ["VFull", 0, 0], "P0": ["PFull", w, 0], "P1": ["PFull", w + 2, 0],
                 "Q0": ["QFull", 0, 0], "Q1": ["QFull", 1, 0], "O": ["OEmpty", w, 1]}
        ready = set()

        def poll(need):
            def look():
                if not need <= ready:
                    ready.clear()
                    ready.update(n for n, (name, i, parity) in lanes.items() if self.bars[name, i].test(parity))
                return need <= ready
            return look

        def used(names):
            for n in names:
                lanes[n][2] ^= 1
            ready.difference_update(names)

        def step(n, size):
            lane = lanes[n]
            lane[1] += 1
            if lane[1] == size:
                lane[1] = 0
                lane[2] ^= 1
            ready.discard(n)

        ring, queue = Ring(PIECES), self.issued[w]
        piece, t, tiles, t_first, more, passes = None, 0, 0, 0, True, False
        v_skip = o_skip = o_parts = pieces = q = 0
        q_need, o_on, o_first, o_last, o_two, o_id = set(), False, False, False, False, None
        while True:
            s_on = t < tiles
            if not s_on and more and not passes:
                piece = yield from self.get_piece(ring)
                more = piece is not None
                if more:
                    tiles, t_first = piece.tiles, 0 if piece.two else w ^ piece.turn
                    t = t_first
                    q = w if piece.two else (pieces & 1 if self.wide else 0)
                    q_need = {"Q0", "Q1"} if piece.two else {f"Q{q}"}
                    pieces += 1
                    if t_first:
                        step("K", K_TILES)
                        v_skip += piece.halves(0)
                    s_on = t < tiles
                    passes = not s_on
            if not s_on and not o_on and not passes:
                break
            for _ in range(o_skip):
                step("V", V_HALVES)
            o_skip = 0
            for op in range(o_parts + 1):
                if op < o_parts:
                    need = {"V", f"P{op}"} | ({"O"} if o_first and op == 0 else set())
                    yield poll(need)
                    at = lanes["V"][1]
                    queue.append(("PV", op, at, o_id, o_first and op == 0))
                    queue.append(("arrive", "VEmpty", at))
                    if not o_two:
                        self.arrive("VEmpty", at)
                    if o_last and op + 1 == o_parts:
                        queue.append(("arrive", "ODone", w))
                    used(need - {"V"})
                    step("V", V_HALVES)
                elif s_on:
                    yield poll({"K"} | (q_need if t == t_first else set()))
                    at = lanes["K"][1]
                    queue.append(("S", at, (piece.index, t), q, w if piece.two else 0, piece.halves(t)))
                    queue.append(("arrive", "SFull", w))
                    queue.append(("arrive", "KEmpty", at))
                    if not piece.two:
                        self.arrive("KEmpty", at)
                    step("K", K_TILES)
            o_on, o_parts = s_on, 0
            if s_on:
                o_two, o_first, o_id, o_parts = piece.two, t == t_first, (piece.index, t), piece.halves(t)
                o_skip, v_skip = v_skip, 0
                t += 1 if piece.two else 2
                o_last = t >= tiles
                if not piece.two and t <= tiles:
                    step("K", K_TILES)
                    v_skip = piece.halves(t - 1)
                if o_last:
                    for i in ((0, 1) if piece.two else (q,)):
                        queue.append(("arrive", "QEmpty", i))
                    used(q_need)
            elif passes:
                passes, tiles = False, 0
                if self.variant in ("no waits", "no turns, no waits"):
                    self.arrive("QEmpty", q)
                else:
                    yield poll(q_need)
                    self.arrive("QEmpty", q)
                    yield poll({"O"})
                used(q_need | {"O"})
                self.arrive("ODone", w)
        yield lambda: not queue

    def execute(self, w):
        """What the tensor cores take next of slot w's."""
        op = self.issued[w].pop(0)
        if op[0] == "arrive":
            self.arrive(op[1], op[2])
        elif op[0] == "S":
            _, at, tile, q, row_tile, halves = op
            expect(self.tile["K"][at] == [(tile[0], 2 * tile[1] + halves - 1)] * WIDEN, "keys", op)
            expect(self.q[q] == (tile[0], row_tile), "queries", op)
            expect(self.s[w] is None, "scores not read", op)
            self.s[w] = [tile, SOFTMAX]
            self.p[w], self.p[w + 2] = [None] * SOFTMAX, [None] * SOFTMAX
        else:
            _, part, at, tile, first = op
            expect(self.tile["V"][at] == [(tile[0], 2 * tile[1] + part)] * WIDEN, "values", op)
            expect(self.p[w + 2 * part] == [tile] * SOFTMAX, "weights", op)
            if first:
                expect(self.o[w] is None, "output not read", op)
                self.o[w] = [tile[0], 0, None]
            expect(self.o[w] and self.o[w][0] == tile[0], "output", op)
            self.o[w][1] += 1

    def read_output(self, w, piece, readers):
        expected = piece.own(w, True)
        if not expected:
            return  # the slot had no tile: nothing to read
        expect(self.o[w] and self.o[w][:2] == [piece.index, expected], "output", w, piece.index, self.o[w])
        if self.o[w][2] is None:
            self.o[w][2] = readers
        self.o[w][2] -= 1
        if not self.o[w][2]:
            self.o[w] = None

    def softmax(self, w, rank):
        ring, units, turns, joins, p_idx = Ring(PIECES), 0, 0, 0, 0
        while True:
            yield self.wait("Piece", ring.at, ring.phase)
            piece = self.ring[ring.at]
            if piece is None:
                return
            added = 0
            for t in piece.own(w):
                yield self.wait("SFull", w, units & 1)
                units += 1
                expect(self.s[w] and self.s[w][0] == (piece.index, t), "scores", w, piece.index, t, self.s[w])
                expect(self.info[(piece.first_tile + t) % INFO] == (piece.index, t), "rejected pages")
                if added:  # O may be rescaled: every product so far is in it
                    expect(self.o[w] and self.o[w][:2] == [piece.index, added], "rescale", w, piece.index, t)
                if piece.two:
                    yield self.wait("Turn", w, (turns + 1 - w) & 1)
                    turns += 1
                for part in range(piece.halves(t)):
                    yield None
                    expect(self.info[(piece.first_tile + t) % INFO] == (piece.index, t), "rejected pages")
                    self.p[w + 2 * part][rank] = (piece.index, t)
                    added += 1
                    if part + 1 == piece.halves(t):  # its last look at the scores
                        self.s[w][1] -= 1
                        if not self.s[w][1]:
                            self.s[w] = None
                    self.arrive("PFull", w + 2 * part)
                if piece.two:
                    self.arrive("Turn", w ^ 1)
            yield self.wait("ODone", w, p_idx & 1)
            if not piece.two:
                self.arrive("Join", 0)
                yield self.wait("Join", 0, joins & 1)
                joins += 1
                yield self.wait("ODone", w ^ 1, p_idx & 1)
            expect(self.nan_rows[ring.at] == {(piece.index, h) for h in range(piece.halves_all)}, "NaN rows")
            yield None
            self.read_output(w, piece, SOFTMAX if piece.two else 2 * SOFTMAX)
            if not piece.two:
                self.read_output(w ^ 1, piece, 2 * SOFTMAX)
            self.arrive("OEmpty", w)
            self.arrive("OEmpty", w if piece.two else w ^ 1)
            self.arrive("Taken", ring.at)
            ring.next()
            p_idx += 1

    # ---- a schedule ---------------------------------------------------------------------------

    def run(self):
        roles = [self.load("K"), self.load("V"), self.mma(0), self.mma(1)]
        roles += [self.widen(side, r) for side in "KV" for r in range(WIDEN)]
        roles += [self.softmax(w, r) for w in (0, 1) for r in range(SOFTMAX)]
        rng = self.rng
        due = [[role, None, rng.choice([1, 1, 3, 10])] for role in roles]  # role, condition, speed
        tensor = rng.choice([1, 3, 10])
        while due:
            able = [d for d in due if d[1] is None or d[1]()]
            busy = [w for w in (0, 1) if self.issued[w]]
            if not able and not busy:
                raise Wrong("nothing can go on")
            weights = [d[2] for d in able] + ([tensor] if busy else [])
            i = rng.choices(range(len(weights)), weights)[0]
            if i == len(able):
                self.execute(rng.choice(busy))
                continue
            try:
                able[i][1] = next(able[i][0])
            except StopIteration:
                due.remove(able[i])


def schedule(seed, variant=None):
    rng = random.Random(seed)
    wide = rng.random() < 0.7
    shapes = [(wide and rng.random() < 0.5, rng.choice([1, 1, 1, 2, 3, 4, 5, 12]), rng.choice([0, 1]))
              for _ in range(rng.randint(1, 14))]
    Kernel(shapes, wide, rng, variant).run()


@pytest.mark.parametrize("block", range(8))
def test_random_schedules(block):
    for seed in range(40 * block, 40 * block + 40):
        schedule(seed)


@pytest.mark.parametrize("shape", [[(False, 1, 1)] * 24, [(False, 1, 0)] * 24, [(True, 1, 1)] * 16,
                                   [(False, 1, 1), (True, 1, 1)] * 10, [(False, 2, 1)] * 12,
                                   [(False, 12, 0)] + [(False, 1, 1)] * 12, [(True, 12, 1), (False, 1, 1)] * 4])
def test_many_short_pieces(shape):
    for wide in (True, False):
        if wide or not any(two for two, _, _ in shape):
            for seed in range(12):
                Kernel(shape, wide, random.Random(seed)).run()


# Mistakes that have to be found: slots that do not take turns over all tiles of pieces
# with one row tile, but begin each piece anew, so that one of them may be lapped; a slot
# that does not wait for a piece without a tile for it; both.
@pytest.mark.parametrize("variant", ["no turns", "no waits", "no turns, no waits"])
def test_mistakes_are_found(variant):
    found = 0
    for seed in range(200):
        try:
            schedule(seed, variant)
        except Wrong:
            found += 1
    assert found > 0


@pytest.mark.parametrize("tiles", [4, 6])
def test_too_few_entries_of_rejected_pages_are_found(tiles, monkeypatch):
    monkeypatch.setitem(globals(), "INFO", tiles)
    with pytest.raises(Wrong):
        for seed in range(200):
            schedule(seed)
