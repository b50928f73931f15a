"""The barriers of the launch over shared prefixes, followed on the CPU over random
interleavings of its roles: producer, converters (e4m3 pages), issuer, softmax, copies in
flight and the tensor cores' queue. A wait passes by parity, as the hardware's does; each
has to pass on the turn that it is meant for, and what is read has to be what was meant.
"""
import os
import random

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                      "linear_attention_state_rssm_gb300", "csrc", "attn_shared_tc.cuh")


class Barrier:
    def __init__(self, name, count):
        self.name, self.count, self.pending, self.bytes, self.phase = name, count, count, 0, 0

    def arrive(self):
        assert self.pending >= 1, ("one arrival too many", self.name, self.phase)
        self.pending -= 1
        self._turn()

    def expect(self, n):
        self.bytes += n
        self.arrive()

    def landed(self, n):
        self.bytes -= n
        self._turn()

    def _turn(self):
        if self.pending == 0 and self.bytes == 0:
            self.phase += 1
            self.pending = self.count

    def passes(self, parity):
        return (self.phase & 1) != parity


def wait(bar, turn):
    while not bar.passes(turn & 1):
        yield
    assert bar.phase == turn + 1, ("passed on another turn", bar.name, turn, bar.phase)


def sizes(D, codes):
    """Places of the operands' ring and of the codes' ring, steps whose powers are kept."""
    units = 2 if D == 256 else (4 if codes else 6) if D == 128 else 8
    return units, (1 if D == 256 else 3 if D == 128 else 4) if codes else 0, units // 2 + 1


def follow(D, codes, steps, seed, kept=None, teams=False):
    """One run of a CTA. kept: steps whose powers are kept, if not what the kernel has;
    teams: two groups of converters that take units by turns."""
    rnd = random.Random(seed)
    NU, NR, NE = sizes(D, codes)
    NE = NE if kept is None else kept
    halves = 1 if teams else 2     # converters that arrive for a unit

    def bars(name, n, count=1):
        return [Barrier(f"{name}[{i}]", count) for i in range(n)]
    full, empty = bars("full", NU, halves if codes else 1), bars("empty", NU)
    rfull, rempty = bars("rfull", NR), bars("rempty", NR, halves)
    sfull, pfull, odone, efull = bars("sfull", 2), bars("pfull", 2), bars("odone", 2), bars("efull", NE)
    copies, queue = [], []         # in flight; issued, in order
    raw, ring, powers = [None] * NR, [None] * NU, [None] * NE
    done = [0] * (2 * steps)       # converters that are through with a unit

    def producer():
        for i in range(2 * steps):
            to, bar = (raw, rfull) if codes else (ring, full)
            n = len(to)
            if i >= n:
                yield from wait((rempty if codes else empty)[i % n], i // n - 1)
            bar[i % n].expect(1)
            copies.append((bar[i % n], to, i % n, i))
            yield
        for i in range(max(0, 2 * steps - n), 2 * steps):
            while not bar[i % n].passes(i // n & 1):
                yield

    def converter(half):
        for i in range(half if teams else 0, 2 * steps, 2 if teams else 1):
            yield from wait(rfull[i % NR], i // NR)
            if i >= NU:
                yield from wait(empty[i % NU], i // NU - 1)
            assert raw[i % NR] == i, ("codes of another unit", i, raw[i % NR])
            yield
            if i % 2 == 0 and half == 0:
                powers[i // 2 % NE] = i // 2
                efull[i // 2 % NE].arrive()
            yield
            done[i] += 1
            if done[i] == halves:
                ring[i % NU] = i
            rempty[i % NR].arrive()
            yield
            full[i % NU].arrive()
            yield

    def issuer():
        def scores(j):
            yield from wait(full[2 * j % NU], 2 * j // NU)
            assert ring[2 * j % NU] == 2 * j, ("keys of another step", j)
            queue.extend((sfull[j & 1], empty[2 * j % NU]))
        yield from scores(0)
        for j in range(steps):
            if j + 1 < steps:
                yield from scores(j + 1)
            u = 2 * j + 1
            yield from wait(full[u % NU], u // NU)
            assert ring[u % NU] == u, ("values of another step", j)
            yield from wait(pfull[j & 1], j >> 1)
            queue.extend((odone[j & 1], empty[u % NU]))

    def softmax():
        for j in range(steps):
            if codes:
                yield from wait(efull[j % NE], j // NE)
                assert powers[j % NE] == j, ("powers of another step", j)
            yield from wait(sfull[j & 1], j >> 1)
            yield
            if j > 0 and rnd.random() < 0.3:    # the reference moves
                yield from wait(odone[(j - 1) & 1], (j - 1) >> 1)
            yield
            assert not codes or powers[j % NE] == j, ("powers written over", j)
            pfull[j & 1].arrive()
        yield from wait(odone[(steps - 1) & 1], (steps - 1) >> 1)

    roles = [producer(), issuer(), softmax()] + ([converter(0), converter(1)] if codes else [])
    pace = [rnd.choice((1, 1, 5, 30)) for _ in roles] + [rnd.choice((1, 10)) for _ in range(2)]
    live, COPY, TENSOR = list(range(len(roles))), -2, -1
    for _ in range(100000):
        if not live:
            return
        who = rnd.choices(live + [COPY, TENSOR], [pace[i] for i in live] + pace[-2:])[0]
        if who == COPY and copies:
            bar, to, at, i = copies.pop(rnd.randrange(len(copies)))
            to[at] = i
            bar.landed(1)
        elif who == TENSOR and queue:
            queue.pop(0).arrive()
        elif who >= 0:
            try:
                next(roles[who])
            except StopIteration:
                live.remove(who)
    raise AssertionError("stuck")


def test_sizes_are_the_kernels():
    text = open(SOURCE).read()
    for line in ("int NU = D == 256 ? 2 : D == 128 ? (Q8 ? 4 : 6) : 8;",
                 "int NR = !Q8 ? 0 : D == 256 ? 1 : D == 128 ? 3 : 4;",
                 "int NE = Q8 ? NU / 2 + 1 : 0;"):
        assert line in text


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("codes", [False, True])
def test_every_wait_ends_on_its_turn(D, codes):
    for steps in (1, 2, 3, 5, 8, 13):
        for seed in range(40):
            follow(D, codes, steps, 7919 * seed + steps)


def fails(**kw):
    for seed in range(200):
        try:
            follow(128, True, 9, seed, **kw)
        except AssertionError:
            return True
    return False


def test_mistakes_are_seen():
    """Powers kept for fewer steps; two groups of converters at one ring of codes."""
    assert not fails()
    assert fails(kept=2)
    assert fails(teams=True)
