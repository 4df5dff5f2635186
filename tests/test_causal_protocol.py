"""Barrier protocol of the causal tensor-core kernel (ssd_causal_tc.cu), checked
on the CPU.

One CTA, a run of tiles. The producer loads C, B (two slots each; three for B
alone in the state pass) and x (three slots). Two warps write the facts of the
even and the odd tiles into four slots. Group C builds diag(w) X in halves, the
MMAs of which add up S; it takes S into the state and writes the state's copy
that C H reads. Groups A and B build M over G for the even and the odd tiles and
read Y for the output. The issuing thread takes whatever is ready: S, then Y,
then G.

Each schedule (random heavy-tailed delays on loads and MMAs, random stepping) is
checked for phase overruns, deadlock and stale reads. Planted variants that the
model must catch: C released with G although C H reads it later, x released by
group C although Y and the output read it later, diag(w) X written without waiting
for the MMAs of the half before, the state's copy written without waiting for C H
of the tile before, and M written before G is complete.
"""
import random

from protocol_sim import Bug, Sched, run_roles

VEC = 4


class AnyOf:
    """A barrier that is complete as soon as one of several phases is."""

    def __init__(self, S):
        self.S, self.phases = S, []

    @property
    def c(self):
        return 1 if any(ready(self.S, b, k) for b, k in self.phases) else 0


def ready(S, name, k):
    """The parity test of phase k."""
    b = S.bar(name, S.counts.get(name, 1))
    if b.c >= k + 2:
        raise Bug(f"overrun on {name}: testing phase {k}, completed {b.c}")
    return (b.c & 1) != (k & 1)


class Run(Sched):
    def __init__(self, seed, n, state=False, heavy=0.1, **planted):
        super().__init__(seed, heavy)
        self.n, self.state = n, state
        self.planted = planted
        self.ring = 3 if state else 2
        self.counts = {}
        if not state:
            for i in range(VEC):
                self.counts['VF', i] = 2
            for i in range(3):
                self.counts['XE', i] = 2
        self.any = AnyOf(self)
        self.bars['any'] = self.any


def producer(S):
    for n in range(S.n):
        if n >= 3:
            yield ('wait', ('XE', n % 3), n // 3 - 1)
        yield ('tma', ('XF', n % 3), [(('x', n % 3), n)])
        for k in ('B',) if S.state else ('C', 'B'):
            if n >= S.ring:
                yield ('wait', (k + 'E', n % S.ring), n // S.ring - 1)
            yield ('tma', (k + 'F', n % S.ring), [((k, n % S.ring), n)])


def facts(S, w):
    for n in range(w, S.n, 2):
        if n >= VEC:
            yield ('wait', ('VF', n % VEC), n // VEC - 1)
        yield ('write', ('info', n % VEC), n)
        yield ('arrive', ('VR', n % VEC))


def issuer(S):
    s = g = y = 0                       # halves of S, tiles of G and Y issued
    while s < 2 * S.n or (not S.state and y < S.n):
        t, hf = s >> 1, s & 1
        want = []
        if t < S.n:
            want.append([(('XW', hf), t)] + ([] if hf else [(('BF', t % S.ring), t // S.ring)]))
        else:
            want.append(None)
        if S.state:
            want += [None, None]
        else:
            want.append([(('M', y % 2), y // 2), ('H', y)] if y < g else None)
            if g < S.n:
                want.append([(('CF', g % 2), g // 2), (('BF', g % 2), g // 2)] + ([(('GF', g % 2), g // 2 - 1)] if g >= 2 else []))
            else:
                want.append(None)
        pick = next((i for i, w in enumerate(want) if w and all(ready(S, b, k) for b, k in w)), None)
        if pick is None:
            # blocked: until a phase that was missing completes
            S.any.phases = [(b, k) for w in want if w for b, k in w if not ready(S, b, k)]
            yield ('wait', 'any', 0)
            continue
        if pick == 0:
            buf = hf if S.state else 0
            acc = ('S', t % 2 if S.state else 0)
            yield ('mma', [(('xw', buf), (t, hf)), (('B', t % S.ring), t)] + ([(acc, (t, 0))] if hf else []), [(acc, (t, hf))])
            yield ('commit', ('SR', hf))
            if hf and (S.state or g > t):
                yield ('commit', ('BE', t % S.ring))
            s += 1
        elif pick == 1:
            yield ('mma', [(('GM', y % 2), ('M', y)), (('x', y % 3), y), (('C', y % 2), y), ('h', y)], [(('Y', y % 2), y)])
            yield ('commit', ('Y', y % 2))
            if not S.planted.get('c_with_g'):
                yield ('commit', ('CE', y % 2))
            y += 1
        else:
            yield ('mma', [(('C', g % 2), g), (('B', g % 2), g)], [(('GM', g % 2), ('G', g))])
            yield ('commit', ('G', g % 2))
            if s > 2 * g + 1:
                yield ('commit', ('BE', g % 2))
            if S.planted.get('c_with_g'):
                yield ('commit', ('CE', g % 2))
            g += 1


def group_c(S):
    for n in range(S.n + 1):
        tile = n < S.n
        if tile:
            yield ('wait', ('VR', n % VEC), n // VEC)
            yield ('wait', ('XF', n % 3), n // 3)
        for hf in (0, 1):
            if n >= 1 and (S.state or hf == 0) and not S.planted.get('no_s_wait'):
                yield ('wait', ('SR', hf if S.state else 1), n - 1)
            if not S.state and hf == 0 and n >= 1:
                yield ('read', ('S', 0), (n - 1, 1))
            if not S.state and hf == 1:
                if not tile:
                    return
                yield ('wait', ('SR', 0), n)
            if tile:
                yield ('read', ('info', n % VEC), n)
                yield ('read', ('x', n % 3), n)
                yield ('write', ('xw', hf if S.state else 0), (n, hf))
                yield ('arrive', ('XW', hf))
        if S.state:
            if n >= 1:
                yield ('read', ('S', (n - 1) % 2), (n - 1, 1))
        if not tile:
            return
        if not S.state:
            if n >= 1 and not S.planted.get('no_y_wait'):
                yield ('wait', ('Y', (n - 1) % 2), (n - 1) // 2)
            yield ('write', 'h', n)
            yield ('arrive', 'H')
        yield ('arrive', ('VF', n % VEC))
        yield ('arrive', ('XE', n % 3))
        if S.planted.get('x_by_c'):
            yield ('arrive', ('XE', n % 3))


def group(S, w):
    for n in range(w, S.n, 2):
        yield ('wait', ('VR', n % VEC), n // VEC)
        if not S.planted.get('no_g_wait'):
            yield ('wait', ('G', n % 2), n // 2)
        yield ('read', ('info', n % VEC), n)
        yield ('read', ('GM', n % 2), ('G', n))
        yield ('write', ('GM', n % 2), ('M', n))
        yield ('arrive', ('M', n % 2))
        yield ('wait', ('Y', n % 2), n // 2)
        yield ('read', ('Y', n % 2), n)
        yield ('read', ('x', n % 3), n)
        yield ('read', ('info', n % VEC), n)
        yield ('arrive', ('VF', n % VEC))
        yield ('arrive', ('GF', n % 2))
        if not S.planted.get('x_by_c'):
            yield ('arrive', ('XE', n % 3))


def run(S):
    roles = {'producer': producer(S), 'facts0': facts(S, 0), 'facts1': facts(S, 1), 'issuer': issuer(S), 'c': group_c(S)}
    if not S.state:
        roles |= {'a': group(S, 0), 'b': group(S, 1)}
    run_roles(S, roles, S.counts)


def schedules(count, state=False, **planted):
    fails = []
    for seed in range(count):
        r = random.Random(seed)
        S = Run(seed, r.choice([1, 2, 3, 5, 9, 14]), state, r.choice([0.0, 0.05, 0.2, 0.5]), **planted)
        try:
            run(S)
        except Bug as e:
            fails.append(f"seed {seed}: {e}")
    return fails


def test_causal_protocol_has_no_overrun_deadlock_or_race():
    fails = schedules(600)
    assert not fails, "\n".join(fails[:5])


def test_state_pass_has_no_overrun_deadlock_or_race():
    fails = schedules(600, state=True)
    assert not fails, "\n".join(fails[:5])


def test_model_catches_c_released_before_c_h_has_read_it():
    assert schedules(300, c_with_g=True)


def test_model_catches_x_released_by_group_c_alone():
    assert schedules(300, x_by_c=True)


def test_model_catches_terms_written_under_the_mma():
    assert schedules(300, no_s_wait=True)
    assert schedules(300, state=True, no_s_wait=True)


def test_model_catches_the_state_written_under_c_h():
    assert schedules(300, no_y_wait=True)


def test_model_catches_the_mask_before_g():
    assert schedules(300, no_g_wait=True)
