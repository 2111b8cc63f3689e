"""The barriers of the tensor-core attention kernel as a model on the CPU: its producers, issuing
warps, keeper of V and softmax groups as coroutines that run in any order, with barriers that tell
a wait only the parity of their phase, as the hardware's do. A run fails where a warp reads a tile
that is not the one it means, or where nothing can go on.

A segment is (two, n): n key tiles, for two row tiles (each slot takes every key tile) or one (the
slots take the key tiles in turn; with n = 1 slot 1 has none)."""
import random

import pytest


class Stuck(Exception):
    pass


def run(segs, stages, rng, q_per_slot=True, slow=()):
    """One run of a CTA. slow: names of warps that go on only when nothing else can. q_per_slot:
    the query barrier of a slot of its own; False: one for both slots, which every segment uses."""
    kfull, kempty, vfull, vempty, vready = ([0] * stages for _ in range(5))
    kc, vc, ka, va = [None] * stages, [None] * stages, [0] * stages, [0] * stages
    sf, pf, pv, sbuf = ([[0, 0], [0, 0]] for _ in range(4))
    pipes, q_full, q_arrived, bars = [[], []], [0, 0], [0, 0], [0, 0]
    q_tile = [None, None]  # the segment whose rows a slot's products would read

    def passed(ctr, i, parity):  # a wait for the phase of that parity
        return lambda: (ctr[i] & 1) != parity

    def arrive(count, ctr, i):  # of two
        count[i] += 1
        if count[i] == 2:
            count[i] = 0
            ctr[i] += 1

    def has_tile(slot, two, n):
        return two or n > slot

    def producer(full, empty, content):
        pos = 0
        for s, (two, n) in enumerate(segs):
            for t in range(n):
                st, par = pos % stages, (pos // stages) & 1
                yield passed(empty, st, par ^ 1)
                content[st] = (s, t)
                full[st] += 1
                pos += 1

    def keeper():
        pos = 0
        for s, (two, n) in enumerate(segs):
            for t in range(n):
                st = pos % stages
                yield passed(vfull, st, (pos // stages) & 1)
                assert vc[st] == (s, t)
                vready[st] += 1
                pos += 1

    def tensor(slot):  # a slot's products and commits, in the order of their issue
        while True:
            yield lambda: pipes[slot]
            pipes[slot].pop(0)()

    def issuer(slot):
        kp = vp = u0 = q_phase = 0
        pipe = pipes[slot]
        for s, (two, n) in enumerate(segs):
            ahead, sh = (2, 0) if two else (4, 1)

            def mine(t):
                return two or (t & 1) == slot

            def score(u, t):
                def f(pos=kp % stages):
                    assert kc[pos] == (s, t) and q_tile[slot] == s
                    sbuf[slot][u & 1] = (s, t)
                    sf[slot][u & 1] += 1
                pipe.append(f)

            def free(pos, is_mine, count, ctr):
                if is_mine:
                    pipe.append(lambda: arrive(count, ctr, pos))
                else:
                    arrive(count, ctr, pos)
            if not q_per_slot or has_tile(slot, two, n):
                yield passed(q_full, slot if q_per_slot else 0, q_phase & 1)
                q_phase += 1
            for t in range(min(n, ahead)):
                yield passed(kfull, kp % stages, (kp // stages) & 1)
                if mine(t):
                    score(u0 + (t >> sh), t)
                free(kp % stages, mine(t), ka, kempty)
                kp += 1
            for t in range(n):
                yield passed(vready, vp % stages, (vp // stages) & 1)
                if mine(t):
                    u = u0 + (t >> sh)
                    yield passed(pf[slot], u & 1, (u >> 1) & 1)

                    def f(pos=vp % stages, u=u, t=t, s=s):
                        assert vc[pos] == (s, t) and sbuf[slot][u & 1] == ("p", s, t)
                        pv[slot][u & 1] += 1
                    pipe.append(f)
                free(vp % stages, mine(t), va, vempty)
                vp += 1
                if t + ahead < n:
                    yield passed(kfull, kp % stages, (kp // stages) & 1)
                    if mine(t):
                        score(u0 + (t >> sh) + 2, t + ahead)
                    free(kp % stages, mine(t), ka, kempty)
                    kp += 1
            u0 += n if two else (n + 1 - slot) // 2

    def softmax(slot):
        u = met = 0

        def meet():
            nonlocal met
            met += 1
            bars[slot] = met
            return lambda m=met: bars[1 - slot] >= m
        for s, (two, n) in enumerate(segs):
            yield meet()
            # both groups load the query rows of both slots
            for x in range(2):
                if q_per_slot and not has_tile(x, two, n):
                    continue
                q_tile[x] = s
                if q_per_slot or x == 0:
                    arrive(q_arrived, q_full, x)
            tiles = 0
            for t in range(0 if two else slot, n, 1 if two else 2):
                yield passed(sf[slot], u & 1, (u >> 1) & 1)
                assert sbuf[slot][u & 1] == (s, t)
                if tiles and rng.random() < 0.3:  # the running maximum rises: O is rescaled
                    yield passed(pv[slot], (u - 1) & 1, ((u - 1) >> 1) & 1)
                    assert sum(pv[slot]) == u
                sbuf[slot][u & 1] = ("p", s, t)
                pf[slot][u & 1] += 1
                tiles += 1
                u += 1
            if tiles:
                yield passed(pv[slot], (u - 1) & 1, ((u - 1) >> 1) & 1)
                assert sum(pv[slot]) == u
            if not two and n > 1:
                yield meet()
                yield meet()

    warps = {"k": producer(kfull, kempty, kc), "v": producer(vfull, vempty, vc), "keep": keeper(),
             "mma0": issuer(0), "mma1": issuer(1), "soft0": softmax(0), "soft1": softmax(1),
             "tensor0": tensor(0), "tensor1": tensor(1)}
    weight = {w: rng.random() + 0.01 for w in warps}
    waits = {w: next(p, None) for w, p in warps.items()}
    while any(c is not None for w, c in waits.items() if w[:6] != "tensor") or any(pipes):
        ready = [w for w, c in waits.items() if c is not None and c()]
        if not ready:
            raise Stuck([w for w, c in waits.items() if c is not None])
        ready = [w for w in ready if w not in slow] or ready
        w = rng.choices(ready, [weight[x] for x in ready])[0]
        waits[w] = next(warps[w], None)


def _segments(rng):
    """Runs of short segments among long ones; one key tile and one row tile most often."""
    return [(rng.random() < 0.3, rng.choice([1, 1, 1, 2, 3, 4, 5, 9, 20]))
            for _ in range(rng.randint(1, 9))]


@pytest.mark.parametrize("slow", [(), ("mma0",), ("mma1",), ("soft0", "soft1"), ("keep",), ("k",),
                                  ("v", "mma1"), ("tensor0", "mma1")], ids="-".join)
@pytest.mark.parametrize("stages", [5, 8])
def test_every_warp_meets_its_own_tiles(stages, slow):
    rng = random.Random(stages * 100 + len(slow))
    for _ in range(150):
        run(_segments(rng), stages, rng, slow=slow)


@pytest.mark.parametrize("stages", [5, 8])
def test_a_late_issuer_of_a_slot_without_tiles(stages):
    """One key tile for one row tile, many times in a row: slot 1 has nothing to compute, and its
    issuing warp may be as late as the stages of K and V allow. With one query barrier for both
    slots the barrier is then two phases on, which a parity cannot tell from none."""
    for n in range(2, 12):
        segs = [(False, 1)] * n + [(False, 2)]
        run(segs, stages, random.Random(n), slow=("mma1",))
    with pytest.raises(Stuck):
        run([(False, 1)] * 4 + [(False, 2)], stages, random.Random(0), q_per_slot=False,
            slow=("mma1",))
