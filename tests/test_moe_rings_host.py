"""The pipelines of the experts' products as a model on the CPU: agents (the warps of
csrc/moe_experts.cu) step in random order through their waits and arrivals on
barriers that, as mbarriers do, know of a round only its parity. Every wait that
passes must have passed on the round it meant, and every run must end: no schedule
may let a wait pass a round early or find the barrier a round further."""
import random

import pytest


class Barrier:
    def __init__(self, count):
        self.count, self.pending, self.rounds = count, count, 0    # rounds: completed ones

    def arrive(self):
        assert self.pending > 0
        self.pending -= 1
        if self.pending == 0:
            self.rounds, self.pending = self.rounds + 1, self.count


class EarlyWait(AssertionError):
    pass


def wait(bar, rnd):
    """Yields until the parity test for round `rnd` passes, then checks that it meant that round."""
    while bar.rounds % 2 == rnd % 2:       # the phase of that parity has not completed
        if bar.rounds > rnd:
            raise EarlyWait("a round further: this wait never ends")
        yield
    if bar.rounds != rnd + 1:
        raise EarlyWait(f"passed on round {bar.rounds - 1} instead of {rnd}")


def run(agents, rng):
    live = list(agents)
    idle = 0
    # some agents are slow for long stretches: only a few are stepped at a time
    favoured = live[:]
    while live:
        if rng.random() < 0.02 or not favoured:
            favoured = rng.sample(live, rng.randint(1, len(live)))
        a = rng.choice(favoured)
        try:
            next(a)
            idle += 1
        except StopIteration:
            live.remove(a)
            favoured = [f for f in favoured if f is not a]
            idle = 0
        assert idle < 400000, "no progress"


def memory(rng, flying, loads):
    """Loads in flight land in any order."""
    for _ in range(loads):
        while not flying:
            yield
        yield
        flying.pop(rng.randrange(len(flying))).arrive()


def small(rng, units, stages, groups=2, packed=4, wide=3, token=5):
    """moe_product_small_kernel: one block, `units` tiles of `stages` stages."""
    total = units * stages
    mk = lambda n, c: [Barrier(c) for _ in range(n)]  # noqa: E731
    p_full, p_empty = mk(packed, 1), mk(packed, 4)
    t_full, ready, done = mk(token, 2), mk(token, 5), mk(token, 1)
    accf, acc_empty = mk(2, 2), mk(2, 4)
    flying = []

    def tma():
        for g in range(total):
            if g >= packed:
                yield from wait(p_empty[g % packed], g // packed - 1)
            yield
            flying.append(p_full[g % packed])

    def tokens():
        for g in range(total):
            if g >= token:
                yield from wait(done[g % token], g // token - 1)
            yield
            t_full[g % token].arrive()
        for g in range(max(0, total - token), total):
            yield from wait(done[g % token], g // token)

    def widen(group):
        for g in range(group, total, groups):
            yield from wait(p_full[g % packed], g // packed)
            if g >= wide:
                yield from wait(done[(g - wide) % token], (g - wide) // token)
            yield
            ready[g % token].arrive()
            yield
            p_empty[g % packed].arrive()

    def scales(me):
        for g in range(me, total, 2):
            yield from wait(t_full[g % token], g // token)
            yield
            ready[g % token].arrive()

    def mma(me):
        for u in range(units):
            if u >= 2:
                yield from wait(acc_empty[u & 1], (u >> 1) - 1)
            for k in range(me, stages, 2):
                g = u * stages + k
                yield from wait(ready[g % token], g // token)
                yield
                done[g % token].arrive()
            accf[u & 1].arrive()
            yield

    def epilogue():
        for u in range(units):
            yield from wait(accf[u & 1], u >> 1)
            yield
            acc_empty[u & 1].arrive()

    agents = [memory(rng, flying, total), tma(), tokens(), tokens(), scales(0), scales(1), mma(0), mma(1)] + [epilogue() for _ in range(4)]
    agents += [widen(g) for g in range(groups) for _ in range(4)]
    run(agents, rng)


def large(rng, units, kc, groups=3, packed=3, oper=5, scale_threads=1):
    """moe_product_large_kernel: a pair of blocks, tiles of kc stages, packed stages of two."""
    total, kp = units * kc, (kc + 1) // 2
    mk = lambda n, c: [Barrier(c) for _ in range(n)]  # noqa: E731
    ready, s_full, acc_empty = mk(oper, 8), mk(oper, 1), mk(2, 8)
    cta = [dict(flying=[], p_full=mk(packed, 1), p_empty=mk(packed, 4), t_full=mk(oper, 1), done=mk(oper, 1), accf=mk(2, 1))
           for _ in range(2)]

    def tma(c):
        for pk in range(units * kp):
            if pk >= packed:
                yield from wait(c["p_empty"][pk % packed], pk // packed - 1)
            yield
            c["flying"].append(c["p_full"][pk % packed])

    def tokens(c):
        for g in range(total):
            if g >= oper:
                yield from wait(c["done"][g % oper], g // oper - 1)
            yield
            c["flying"].append(c["t_full"][g % oper])
        for g in range(max(0, total - oper), total):
            yield from wait(c["done"][g % oper], g // oper)

    def widen(c, group):
        pk = 0
        for u in range(units):
            for q in range(kp):
                if pk % groups == group:
                    yield from wait(c["p_full"][pk % packed], pk // packed)
                    halves = min(2, kc - 2 * q)
                    for h in range(halves):
                        g = u * kc + 2 * q + h
                        if g >= oper:
                            yield from wait(c["done"][g % oper], g // oper - 1)
                        yield
                        if h + 1 == halves:
                            c["p_empty"][pk % packed].arrive()
                        yield from wait(c["t_full"][g % oper], g // oper)
                        yield
                        ready[g % oper].arrive()
                pk += 1

    def scales(me):
        for g in range(me, total, scale_threads):
            yield from wait(ready[g % oper], g // oper)
            yield
            s_full[g % oper].arrive()

    def mma():
        for u in range(units):
            if u >= 2:
                yield from wait(acc_empty[u & 1], (u >> 1) - 1)
            for k in range(kc):
                g = u * kc + k
                yield from wait(s_full[g % oper], g // oper)
                for c in rng.sample(cta, 2):       # the commit reaches the blocks at different times
                    yield
                    c["done"][g % oper].arrive()
            for c in cta:
                c["accf"][u & 1].arrive()

    def epilogue(c):
        for u in range(units):
            yield from wait(c["accf"][u & 1], u >> 1)
            yield
            acc_empty[u & 1].arrive()

    agents = [mma()] + [scales(i) for i in range(scale_threads)]
    for c in cta:
        agents += [memory(rng, c["flying"], units * kp + total), tma(c), tokens(c)] + [epilogue(c) for _ in range(4)]
        agents += [widen(c, g) for g in range(groups) for _ in range(4)]
    run(agents, rng)


@pytest.mark.parametrize("units,stages", [(1, 1), (7, 1), (5, 2), (5, 3), (3, 4), (3, 5), (2, 8), (2, 11)])
def test_small_tiles(units, stages):
    for seed in range(25):
        small(random.Random(seed), units, stages)


@pytest.mark.parametrize("units,kc", [(1, 1), (7, 1), (5, 2), (5, 3), (3, 5), (2, 8), (2, 11)])
def test_large_tiles(units, kc):
    for seed in range(20):
        large(random.Random(seed), units, kc)


def breaks(f, *args, **kw):
    for seed in range(300):
        try:
            f(random.Random(seed), *args, **kw)
        except AssertionError:
            return True
    return False


def test_the_model_sees_what_breaks():
    # a third widening group of small tiles; two scale threads that take turns on large ones; packed slots that
    # change between groups
    assert breaks(small, 5, 3, groups=3)
    assert breaks(large, 4, 4, scale_threads=2)
    assert breaks(large, 4, 8, groups=2)
