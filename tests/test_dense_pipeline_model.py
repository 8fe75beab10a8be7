"""Model check of the dense products' pipeline (csrc/k_dense.cu, gemm16_kernel), on CPU, with waits that run out.

The roles of a pair of CTAs are restated as the sequence of waits, arrivals and copies that the kernel performs, with
the same ring indices, phases and barrier counts:

* TMA, one warp in each CTA: per slab, waits its own `empty`, then copies its A and B parts; the bytes of both
  CTAs are counted on the leader's `full`, where the leader expects both.  Afterwards each sends the leader the
  number of its copies and arrives on the leader's `stopped`.
* MMA, in the leader: per accumulation, waits `acc_empty`; per slab, waits `full`, issues, commits to both CTAs'
  `empty` and, at the end, to both `acc_full`; at last, or when a wait ran out, to both `drain`.  In the second case
  it waits for `drain`, `stopped` and then the last phase of every stage, supplying what one of the two CTAs never
  asked for.
* epilogue, in each CTA: waits `acc_full`, reads, arrives on the leader's `acc_empty`; after a wait that ran out it
  waits no more and writes NaN for this and every further accumulation.

Copies land in any order, MMAs and commits complete in issue order, and a random scheduler interleaves the roles.  In
half of the runs some waits run out: the role stops, its CTA's abort flag is set, and the CTA's other roles stop at
their next wait that is not met.  The checks: without that, nothing deadlocks and every slab is multiplied
once, from the stage that holds it; with it, every role ends, no wait of the last part runs out, no copy
is in flight when the CTAs leave, and every result is written: NaN, or made of all its slabs.
"""
import random

import pytest


class Bar:
    """An mbarrier: `count` arrivals and a transaction count of zero (it may pass below zero: bytes that land before
    they are expected) complete a phase."""

    def __init__(self, count):
        self.count = self.pending = count
        self.tx = self.done = 0

    def arrive(self, expect_tx=0):
        self.tx += expect_tx
        self.pending -= 1
        assert self.pending >= 0
        self.check()

    def complete_tx(self, n):
        self.tx -= n
        self.check()

    def check(self):
        if self.pending == 0 and self.tx == 0:
            self.done += 1
            self.pending = self.count

    def ready(self, phase):
        # a parity tells neighbouring phases apart only
        assert self.done <= phase + 2, "waiter fell behind"
        return self.done > phase


def run_pair(units, nk, stages, seed, expire, drained=True, epi=2):
    """units: accumulations of nk slabs.  Returns (copies in flight at the end, slabs multiplied, aborted, results:
    whether the accumulation was complete, by (CTA, warp, accumulation))."""
    rnd = random.Random(seed)
    full = [Bar(1) for _ in range(stages)]            # the leader's
    empty = [[Bar(1) for _ in range(stages)] for _ in range(2)]
    acc_full = [[Bar(1) for _ in range(2)] for _ in range(2)]
    acc_empty = [Bar(2 * epi) for _ in range(2)]      # the leader's
    drain, stopped = [Bar(1), Bar(1)], Bar(2)
    abort, held = [False, False], [[None] * stages for _ in range(2)]
    copies, tensor, multiplied = [], [], []
    sent, results = {}, {}

    def tma(rank):
        n = 0
        for _ in range(units * nk):
            if not (yield rank, empty[rank][n % stages], n // stages - 1):
                break
            if rank == 0:
                full[n % stages].arrive(expect_tx=2)
            copies.append((rank, n))
            n += 1
        sent[rank] = n
        stopped.arrive()

    def mma():
        n = 0
        for t in range(units):
            if not (yield 0, acc_empty[t % 2], t // 2 - 1):
                break
            k = 0
            while k < nk:
                if not (yield 0, full[n % stages], n // stages):
                    break
                tensor.append(("mma", n))
                tensor.append(("empty", n % stages))
                n, k = n + 1, k + 1
            if k < nk:
                break
            tensor.append(("acc", t % 2))
        tensor.append(("drain", 0))
        if n == units * nk or not drained:
            return
        assert (yield None, drain[0], 0)
        assert (yield None, stopped, 0)
        most = max(sent.values())
        assert most - min(sent.values()) <= stages
        for k in range(max(0, most - stages), most):
            if k >= sent[1]:
                full[k % stages].complete_tx(1)
            if k >= sent[0]:
                full[k % stages].arrive(expect_tx=1)
            assert (yield None, full[k % stages], k // stages)

    def epilogue(rank, w):
        ok = True
        for t in range(units):
            if ok:
                ok = yield rank, acc_full[rank][t % 2], t // 2
            if ok:
                assert set(range(t * nk, (t + 1) * nk)) <= set(multiplied)
                acc_empty[t % 2].arrive()
            results[rank, w, t] = ok

    def leave(rank):                                  # one lane of the MMA warp, after its role
        assert (yield None, drain[rank], 0)

    roles = [tma(0), tma(1), mma(), *(epilogue(r, w) for r in (0, 1) for w in range(epi)), leave(0), leave(1)]
    waits = {i: next(r, None) for i, r in enumerate(roles)}
    waits = {i: w for i, w in waits.items() if w is not None}

    def resume(i, met):
        try:
            waits[i] = roles[i].send(met)
        except StopIteration:
            del waits[i]

    quiet = 0
    while waits:
        moves = [("role", i) for i, (_, bar, ph) in waits.items() if bar.ready(ph)]
        stuck = [i for i, (rank, bar, ph) in waits.items() if rank is not None and not bar.ready(ph)]
        moves += [("stop", i) for i in stuck if abort[waits[i][0]]]
        moves += [("copy", i) for i in range(len(copies))] + [("tensor", 0)] * bool(tensor)
        if expire and stuck and rnd.random() < expire:
            i = rnd.choice(stuck)                     # this wait runs out
            abort[waits[i][0]] = True
            resume(i, False)
            continue
        if not moves:
            quiet += 1
            # (a wait that nothing will meet: it runs out; without injected faults that is a deadlock)
            assert expire and stuck and quiet < 100, ("deadlock", list(waits))
            i = rnd.choice(stuck)
            abort[waits[i][0]] = True
            resume(i, False)
            continue
        kind, i = rnd.choice(moves)
        if kind == "role":
            resume(i, True)
        elif kind == "stop":
            resume(i, False)
        elif kind == "copy":
            rank, n = copies.pop(i)
            held[rank][n % stages] = n
            full[n % stages].complete_tx(1)
        else:
            what, v = tensor.pop(0)
            if what == "mma":
                assert held[0][v % stages] == held[1][v % stages] == v
                multiplied.append(v)
            else:
                for r in (0, 1):
                    {"empty": empty[r], "acc": acc_full[r], "drain": [drain[r]]}[what][v].arrive()
    return len(copies), multiplied, any(abort), results


SHAPES = [(1, 1, 6), (1, 20, 6), (3, 7, 6), (5, 2, 12), (2, 40, 7), (9, 1, 6)]


@pytest.mark.parametrize("units,nk,stages", SHAPES)
def test_every_slab_is_multiplied_once(units, nk, stages):
    for seed in range(30):
        flying, done, aborted, results = run_pair(units, nk, stages, seed, 0.0)
        assert flying == 0 and not aborted and done == list(range(units * nk))
        assert len(results) == 4 * units and all(results.values())


@pytest.mark.parametrize("units,nk,stages", SHAPES)
def test_waits_that_run_out(units, nk, stages):
    for seed in range(200):
        flying, done, _, results = run_pair(units, nk, stages, 1000 + seed, (0.002, 0.02, 0.2)[seed % 3])
        assert flying == 0 and done == list(range(len(done)))
        assert len(results) == 4 * units             # nothing is left as it was


def test_the_model_sees_copies_that_nobody_waits_for():
    left = [run_pair(3, 7, 6, 1000 + seed, 0.02, drained=False)[0] for seed in range(200)]
    assert any(left)
