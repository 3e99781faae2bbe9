"""A CPU model of the mbarrier protocol of the 4-bit decode on tcgen05
(`relattn_decode_fp4_tc_kernel`): softmax warps (with and without live rows),
two groups of conversion warps, the product issuer and the tensor core, written
step for step after the kernel's waits, arrives, issues and commits.  A CTA
walks pieces of any number of tiles.  Interleavings of the agents are run to
completion, at random and with one agent held back as long as another can move
(every order of "the product completes before the first poll" is among those),
and checked for

* deadlock (every agent finishes),
* parity aliasing (a wait sees a barrier in the phase it asks for or in the next
  one; the kernel's parity waits cannot tell others from these: two phases
  ahead the waiter would spin until its bound, one behind it would pass early),
* buffer hazards: a K or V tile rewritten under a pending product; S overwritten
  before every softmax warp has read it; P overwritten under a pending P V; Q
  overwritten under a pending Q K^T; O rescaled or read out before its products
  have landed; a NaN list overwritten before it is read.

Waits can be dropped or taken as an earlier form of the kernel had them: those
protocols must fail, which pins the model itself.
"""
import random

import pytest

KST = VST = 2        # stages of K and V tiles
WARPS = 4            # softmax warps
GROUPS = 2           # conversion groups, one agent each


class Bar:
    def __init__(self, count):
        self.count, self.pending, self.phase = count, 0, 0

    def arrive(self):
        self.pending += 1
        assert self.pending <= self.count
        if self.pending == self.count:
            self.pending, self.phase = 0, self.phase + 1

    def passed(self, want):
        """test_wait.parity of phase `want`: true while the phase under way has the
        other parity.  That means `want` has just completed, provided the barrier
        is in that phase or the one after it."""
        assert want <= self.phase <= want + 1, "parity aliasing"
        return (self.phase ^ want) & 1 == 1


class Model:
    def __init__(self, pieces, live, rng, drop=(), slow=None):
        """pieces: tiles of each piece; live: softmax warps with query rows (the
        others only take part in the barriers); drop: waits left out, or "two
        waits" at a piece's end; slow: the agent that moves only when no other
        can (an index into agents, or "tc")."""
        self.pieces, self.live_warps, self.rng, self.drop, self.slow = pieces, live, rng, set(drop), slow
        self.B = {"qf": Bar(WARPS), "od": Bar(1)}
        for s in range(KST):
            self.B[f"kf{s}"], self.B[f"ke{s}"] = Bar(1), Bar(1)
        for s in range(VST):
            self.B[f"vf{s}"], self.B[f"ve{s}"] = Bar(1), Bar(1)
        for s in range(2):
            self.B[f"sf{s}"], self.B[f"pf{s}"] = Bar(1), Bar(WARPS)
        self.k_tile, self.v_tile = [None] * KST, [None] * VST
        self.s_tile, self.s_read = [None] * 2, [set(range(WARPS)) for _ in range(2)]
        self.p_tile, self.q_piece = {}, {}
        self.nan_list, self.nan_read = [None] * 4, [set(range(WARPS)) for _ in range(4)]
        self.tc = []                          # issued, not yet executed: products and commits
        self.done_s, self.done_pv = set(), set()
        self.agents = [self.softmax(w) for w in range(WARPS)] + [self.converter(t) for t in range(GROUPS)] + [self.issuer()]

    def wait(self, name, want):
        if want < 0:
            return
        while not self.B[name].passed(want):
            yield

    def pending(self, kind, tile=None):
        return any(op[0] == kind and (tile is None or op[1] == tile) for op in self.tc)

    # ---------------------------------------------------------------- agents
    def softmax(self, w):
        g = 0
        for piece, n in enumerate(self.pieces):
            assert not self.pending("S"), "Q overwritten under a pending product"
            self.q_piece[w] = piece
            self.B["qf"].arrive()
            yield
            first = g
            for i in range(n):
                yield from self.wait(f"sf{g & 1}", g >> 1)
                assert self.s_tile[g & 1] == g, "a wrong S"
                assert self.nan_list[g & 3] == g, "a wrong NaN list"
                follows = w in self.live_warps or "every warp" not in self.drop
                if i > 0 and follows and "od" not in self.drop:
                    yield from self.wait("od", g - 1)
                if w in self.live_warps:
                    assert not self.pending("PV"), "P overwritten, or O rescaled, under a pending product"
                    assert set(range(first, g)) <= self.done_pv
                    self.p_tile[w] = g
                self.s_read[g & 1].add(w)
                self.nan_read[g & 3].add(w)
                yield
                self.B[f"pf{g & 1}"].arrive()
                g += 1
                yield
            if "two waits" in self.drop:
                yield from self.wait("od", g - 2)
            if "last" not in self.drop:
                yield from self.wait("od", g - 1)
            if w in self.live_warps:
                assert set(range(first, g)) <= self.done_pv, "O read before its last product"
            yield

    def converter(self, turn):
        g = 0
        for n in self.pieces:
            for i in range(n):
                if (g + i) % GROUPS != turn:
                    continue
                t = g + i
                assert self.nan_read[t & 3] == set(range(WARPS)), "a NaN list overwritten before it was read"
                self.nan_list[t & 3], self.nan_read[t & 3] = t, set()
                if "ke" not in self.drop:
                    yield from self.wait(f"ke{t % KST}", t // KST - 1)
                assert t < KST or t - KST in self.done_s, "K rewritten under a pending product"
                self.k_tile[t % KST] = t
                yield
                self.B[f"kf{t % KST}"].arrive()
                if "ve" not in self.drop:
                    yield from self.wait(f"ve{t % VST}", t // VST - 1)
                assert t < VST or t - VST in self.done_pv, "V rewritten under a pending product"
                self.v_tile[t % VST] = t
                yield
                self.B[f"vf{t % VST}"].arrive()
            g += n

    def issuer(self):
        g = 0

        def pv(t):
            if "pf" not in self.drop:
                yield from self.wait(f"pf{t & 1}", t >> 1)
            yield from self.wait(f"vf{t % VST}", t // VST)
            self.tc += [("PV", t), ("commit", f"ve{t % VST}"), ("commit", "od")]

        for piece, n in enumerate(self.pieces):
            yield from self.wait("qf", piece)
            for i in range(n):
                yield from self.wait(f"kf{g % KST}", g // KST)
                self.tc += [("S", g), ("commit", f"ke{g % KST}"), ("commit", f"sf{g & 1}")]
                yield
                if i > 0:
                    yield from pv(g - 1)
                g += 1
            yield from pv(g - 1)

    # ------------------------------------------------------ the tensor core
    def tensor_step(self):
        kind, x = self.tc.pop(0)
        if kind == "commit":
            self.B[x].arrive()
        elif kind == "S":
            assert self.k_tile[x % KST] == x
            assert self.s_read[x & 1] == set(range(WARPS)), "S overwritten before it was read"
            self.s_tile[x & 1], self.s_read[x & 1] = x, set()
            self.done_s.add(x)
        else:
            assert self.v_tile[x % VST] == x
            assert all(self.p_tile[w] == x for w in self.live_warps), "a wrong P"
            self.done_pv.add(x)

    def snapshot(self):
        return (len(self.tc), tuple((b.phase, b.pending) for b in self.B.values()))

    def run(self):
        """An agent that waits yields without changing anything, so a pass over
        all of them that changes nothing is a deadlock."""
        alive = dict(enumerate(self.agents))
        idle = 0
        while alive or self.tc:
            names = list(alive) + (["tc"] if self.tc else [])
            self.rng.shuffle(names)
            if self.slow in names:               # last, and only when the others stand still
                names.remove(self.slow)
                names.append(self.slow)
            before = self.snapshot()
            moved = False
            for x in names:
                if x == self.slow and moved:
                    break
                at, count = self.snapshot(), len(alive)
                if x == "tc":
                    self.tensor_step()
                else:
                    try:
                        next(alive[x])
                    except StopIteration:
                        del alive[x]
                moved = moved or self.snapshot() != at or len(alive) != count
                if moved and self.slow is None and self.rng.random() < 0.5:
                    break
            idle = 0 if moved or self.snapshot() != before else idle + 1
            assert idle < 20, "deadlock"         # (an agent takes at most a few steps that change no barrier)


PIECES = [(1,), (2,), (3,), (7,), (1, 1, 1), (1, 2, 1, 3), (2, 1, 4), (5, 1, 1, 2)]
AGENTS = list(range(WARPS + GROUPS + 1)) + ["tc", None]


@pytest.mark.parametrize("pieces", PIECES)
@pytest.mark.parametrize("live", [(0,), (0, 1, 2), (0, 1, 2, 3)])
def test_decode_protocol(pieces, live):
    for slow in AGENTS:
        for seed in range(8):
            Model(pieces, live, random.Random(seed), slow=slow).run()


def fails(drop, live=(0, 1)):
    for pieces in PIECES:
        for slow in AGENTS:
            for seed in range(8):
                try:
                    Model(pieces, live, random.Random(seed), drop=drop, slow=slow).run()
                except AssertionError as e:
                    return str(e) or "hazard"
    return ""


def test_two_waits_at_a_pieces_end_cannot_tell_phases_apart():
    """A warp that asks for the product before the last, and polls only after the
    last one too has completed, never sees that phase: with live rows at once,
    and without following the products tile by tile either way."""
    assert "aliasing" in fails(("two waits",))
    assert "aliasing" in fails(("two waits", "every warp"))
    assert "aliasing" in fails(("every warp",))


@pytest.mark.parametrize("drop", ["od", "last", "ke", "ve", "pf"])
def test_protocol_model_catches_a_dropped_wait(drop):
    assert fails((drop,))
