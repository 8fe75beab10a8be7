"""Model check of the pipeline of the products that dequantise on the way (csrc/k_skinny.cu, skinny_kernel), on CPU,
with waits that run out.

The roles of one CTA are restated with the ring indices, phases and barriers of the kernel: three groups of
dequantising warps that take the stages in turn (wait `empty`, write A, arrive `a_full`), the warp that copies token tiles
(wait `empty`, expect and copy on `b_full`; at the end waits for its last copies), the MMA warp (wait `acc_empty` for a
new segment, `b_full`, `a_full`; commits `empty`, at a segment's end `acc_full`, at last `drain`) and the warps of the
results (wait `acc_full`, write, arrive `acc_empty`).  Where no tile is shared, the sets of dequantising warps wait for
`drain` and write their share of the last segment's results.  A role whose wait runs out raises the abort flag; who
writes results writes NaN from there on.

Checks: nothing deadlocks, every stage is multiplied once and holds its own unit, no copy is in flight at the end, and
every result is written: NaN, or made of all its units."""
import random

import pytest

from test_dense_pipeline_model import Bar

GROUPS = 3


def run_cta(u0, u1, ks, stages, whole, seed, expire):
    rnd = random.Random(seed)
    N = u1 - u0
    a_full, b_full, empty = ([Bar(1) for _ in range(stages)] for _ in range(3))
    acc_full, acc_empty, drain = [Bar(1), Bar(1)], [Bar(1), Bar(1)], Bar(1)
    abort, held_a, held_b = [False], [None] * stages, [None] * stages
    copies, tensor, multiplied, results = [], [], [], {}
    # segments: the units of one tile in this CTA's range
    segs, u = [], u0
    while u < u1:
        end = min(u // ks * ks + ks, u1)
        segs.append(range(u - u0, end - u0))
        u = end

    def dequant(g):
        ok = True
        for n in range(g, N, GROUPS):
            ok = yield True, empty[n % stages], n // stages - 1
            if not ok:
                break
            held_a[n % stages] = n
            a_full[n % stages].arrive()
        if whole:
            if ok:
                ok = yield True, drain, 0
            ok = ok and not abort[0]
            if ok:
                assert set(segs[-1]) <= set(multiplied)
            results[len(segs) - 1, g] = ok

    def tma():
        issued = 0
        for n in range(N):
            if not (yield True, empty[n % stages], n // stages - 1):
                break
            b_full[n % stages].arrive(expect_tx=1)
            copies.append(n)
            issued += 1
        for s in range(stages):
            if issued > s:
                n = issued - 1 - s
                assert (yield False, b_full[n % stages], n // stages)

    def mma():
        for i, seg in enumerate(segs):
            if not (yield True, acc_empty[i % 2], i // 2 - 1):
                break
            ok = True
            for n in seg:
                ok = yield True, b_full[n % stages], n // stages
                if ok:
                    ok = yield True, a_full[n % stages], n // stages
                if not ok:
                    break
                tensor.append(("mma", n))
                tensor.append(("empty", n % stages))
            if not ok:
                break
            tensor.append(("acc", i % 2))
        tensor.append(("drain", 0))
        assert (yield False, drain, 0)

    def epilogue():
        ok = True
        for i, seg in enumerate(segs):
            if ok:
                ok = yield True, acc_full[i % 2], i // 2
            if ok:
                assert set(seg) <= set(multiplied)
                acc_empty[i % 2].arrive()
            results[i, "own"] = ok

    roles = [dequant(g) for g in range(GROUPS)] + [tma(), mma(), epilogue()]
    waits = {i: next(r, None) for i, r in enumerate(roles)}
    waits = {i: w for i, w in waits.items() if w is not None}

    def resume(i, met):
        try:
            waits[i] = roles[i].send(met)
        except StopIteration:
            del waits[i]

    while waits:
        moves = [("role", i) for i, (_, bar, ph) in waits.items() if bar.ready(ph)]
        stuck = [i for i, (bounded, bar, ph) in waits.items() if bounded and not bar.ready(ph)]
        moves += [("stop", i) for i in stuck if abort[0]]
        moves += [("copy", i) for i in range(len(copies))] + [("tensor", 0)] * bool(tensor)
        if stuck and ((expire and rnd.random() < expire) or (expire and not moves)):
            abort[0] = True
            resume(rnd.choice(stuck), False)
            continue
        assert moves, ("deadlock", list(waits))
        kind, i = rnd.choice(moves)
        if kind == "role":
            resume(i, True)
        elif kind == "stop":
            resume(i, False)
        elif kind == "copy":
            n = copies.pop(i)
            held_b[n % stages] = n
            b_full[n % stages].complete_tx(1)
        else:
            what, v = tensor.pop(0)
            if what == "mma":
                assert held_a[v % stages] == held_b[v % stages] == v
                multiplied.append(v)
            else:
                {"empty": empty, "acc": acc_full, "drain": [drain]}[what][v].arrive()
    return len(copies), multiplied, results, len(segs) + (GROUPS if whole else 0)


RANGES = [(0, 1, 1, False), (0, 7, 7, True), (5, 25, 8, False), (3, 41, 4, False), (0, 12, 1, True), (9, 60, 17, False),
          (0, 2, 2, True)]


@pytest.mark.parametrize("stages", [3, 4, 5])
@pytest.mark.parametrize("u0,u1,ks,whole", RANGES)
def test_every_unit_is_multiplied_once(u0, u1, ks, whole, stages):
    for seed in range(30):
        flying, done, results, n = run_cta(u0, u1, ks, stages, whole, seed, 0.0)
        assert flying == 0 and done == list(range(u1 - u0)) and len(results) == n and all(results.values())


@pytest.mark.parametrize("stages", [3, 4, 5])
@pytest.mark.parametrize("u0,u1,ks,whole", RANGES)
def test_waits_that_run_out(u0, u1, ks, whole, stages):
    for seed in range(150):
        flying, done, results, n = run_cta(u0, u1, ks, stages, whole, 500 + seed, (0.002, 0.02, 0.2)[seed % 3])
        assert flying == 0 and done == list(range(len(done))) and len(results) == n
