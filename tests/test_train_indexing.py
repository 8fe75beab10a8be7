"""Host-side checks of the index arithmetic behind the gated, gradient and cross-entropy kernels,
restated in Python: work ranges, ring stages and phases, tile walks, shared-memory plans and lane maps.
No GPU needed."""
import itertools

import pytest

SMS = 148


# ------------------------------------------------------------------ products dequantised on the way
MAX_N, MAX_STAGES, GROUPS, A_BYTES = 144, 5, 3, 32768
TAIL = 2 * 16 * 128 * 4 + 2 * 256 * 4 + (4 * MAX_STAGES + 5) * 8 + 32


def skinny_plan(M, tiles, k):
    tt = -(-M // MAX_N)
    n = -(-(-(-M // tt)) // 16) * 16
    tt = -(-M // n)
    ks = -(-k // 128)
    T = tiles * tt
    units = T * ks
    cost = {SMS: -(-units // SMS) * 600 + 3000 + -(-SMS // T) * 60}
    for c in range(1, min(ks, 64, SMS // T) + 1):
        cost.setdefault(T * c, 10 ** 9)
        cost[T * c] = min(cost[T * c], -(-ks // c) * 600 + (c * 60 + 1000 if c > 1 else 0) + (600 if ks % c else 0))
    return n, tt, ks, min(min(cost, key=cost.get), units), units


def first(units, grid, c):
    return units * c // grid


@pytest.mark.parametrize("M,tiles,k", [
    (1, 1, 64), (17, 22, 512), (50, 4, 2742), (77, 172, 4096), (19, 86, 4096), (144, 3, 22016), (145, 7, 4096),
    (256, 40, 27648), (352, 172, 4096), (300, 1, 128), (64, 500, 100), (50, 22, 512), (50, 44, 1024), (288, 3, 49152)])
def test_skinny_ranges_cover_every_stage_once(M, tiles, k):
    n, tt, ks, grid, units = skinny_plan(M, tiles, k)
    assert n % 16 == 0 and n <= MAX_N and n * tt >= M and n * (tt - 1) < M
    stages = min((232448 - 1024 - TAIL) // (A_BYTES + n * 256), MAX_STAGES)
    assert stages >= GROUPS and 6 * (2 * 16 * 128 * 4 + 2 * 256 * 4) <= stages * (A_BYTES + n * 256)
    assert 1024 + stages * (A_BYTES + n * 256) + TAIL <= 232448
    seen, slots = [], {}
    for c in range(grid):
        u0, u1 = first(units, grid, c), first(units, grid, c + 1)
        assert u0 < u1
        seen += range(u0, u1)
        u = u0
        while u < u1:                                # segments: whole tiles, or partial sums in a slot of their own
            T = u // ks
            b0, b1 = T * ks, T * ks + ks
            end = min(b1, u1)
            if not (u == b0 and end == b1):
                slot = 2 * c + (0 if u0 > b0 else 1)
                assert slot not in slots.values() and slot < 2 * grid
                slots[(T, c)] = slot
            u = end
    assert seen == list(range(units)) and units * (grid + 1) < 2 ** 31
    # the second kernel finds exactly the CTAs that left partial sums
    for T in range(tiles * tt):
        b0, b1 = T * ks, (T + 1) * ks
        c0, c1 = (((u + 1) * grid - 1) // units for u in (b0, b1 - 1))
        assert first(units, grid, c0) <= b0 < first(units, grid, c0 + 1)
        assert first(units, grid, c1) <= b1 - 1 < first(units, grid, c1 + 1)
        own = [c for t, c in slots if t == T]
        assert own == ([] if c0 == c1 else list(range(c0, c1 + 1)))
        for c in own:
            assert slots[(T, c)] == 2 * c + (1 if c == c0 else 0)


@pytest.mark.parametrize("stages", [3, 4, 5])
@pytest.mark.parametrize("grp", range(GROUPS))
def test_skinny_ring_stage_and_phase(stages, grp):
    st, ph = grp, 1
    for n in range(grp, 300, GROUPS):
        assert st == n % stages and ph == (n // stages & 1) ^ 1
        # the group's last unit waited for unit n - GROUPS - stages; a parity wait for unit n - stages
        # is unambiguous once unit n - 2 stages is consumed
        assert n - 2 * stages < 0 or n - GROUPS - stages >= n - 2 * stages
        st += GROUPS
        if st >= stages:
            st -= stages
            ph ^= 1


def test_skinny_stage_bytes_written_once_without_bank_conflicts():
    """256 threads x (2 rows, 4 words): every 16-byte column of the 32 KB stage once, in the 128-byte
    swizzle, and the eight lanes of a store phase in eight 16-byte columns of the banks."""
    written = {}
    for b, i in itertools.product(range(2), range(4)):
        phase = []
        for tid in range(256):
            r, q4 = tid >> 2, tid & 3
            rot = 2 if q4 >= 2 else 0
            sx0 = ((q4 & 1) * 4) ^ (r & 7) ^ rot
            addr = (q4 >> 1) * 16384 + r * 128 + b * 64 * 128 + ((sx0 ^ i) << 4)
            word = (i + rot) & 3                      # the word of the quarter that this store holds
            row, col = r + 64 * b, q4 * 32 + word * 8
            blk, ch = col // 64, col % 64 // 8
            assert addr == blk * 16384 + row * 128 + ((ch ^ (row & 7)) << 4)
            assert addr not in written
            written[addr] = 1
            phase.append(addr % 128 // 16)
            if len(phase) == 8:
                assert sorted(phase) == list(range(8))
                phase = []
    assert len(written) == 2048


# ------------------------------------------------------------------ dense products
def tile_cols(M, N):
    best, cost = 256, None
    for bn in range(256, 63, -32):
        slab = 350 + bn if bn <= 192 else 272 * bn // 100
        tiles = -(-M // 256) * -(-N // bn)
        c = -(-tiles // (SMS // 2)) * slab
        if cost is None or c < cost:
            best, cost = bn, c
    return best


@pytest.mark.parametrize("mt,nt", [(1, 1), (8, 16), (9, 3), (17, 5), (63, 16), (1, 125), (16, 2)])
def test_dense_tile_walk_visits_every_tile_once(mt, nt):
    seen = set()
    for t in range(mt * nt):
        band = t // (8 * nt)
        r = t - band * 8 * nt
        h = min(mt - band * 8, 8)
        n = r // h
        m = band * 8 + (r - n * h)
        assert 0 <= m < mt and 0 <= n < nt
        seen.add((m, n))
    assert len(seen) == mt * nt


@pytest.mark.parametrize("M,N", [(1, 64), (2048, 22016), (2048, 4096), (2048, 5120), (129, 512), (32000, 4096), (513, 64)])
def test_dense_tiles_and_ring(M, N):
    bn = tile_cols(M, N)
    assert bn % 32 == 0 and 64 <= bn <= 256
    for mn_major in (False, True):
        bh = bn // 2
        stage = 16384 + ((bh + 63) // 64 * 8192 if mn_major else (bh * 128 + 1023) // 1024 * 1024)
        stages = min(192 * 1024 // stage, 12)
        assert stages >= 6 and stage % 1024 == 0


@pytest.mark.parametrize("nk,splits", [(156, 9), (8, 1), (35, 4), (17, 2)])
def test_dense_k_splits_cover_k(nk, splits):
    at = [nk * i // splits for i in range(splits + 1)]
    assert at[0] == 0 and at[-1] == nk and all(a < b for a, b in zip(at, at[1:]))


def test_ce_vocabulary_pieces():
    for M, V in itertools.product((1, 129, 2048, 5000, 100000), (1, 100, 4096, 9973, 32000, 250000)):
        vc = max((64 << 20) // (2 * M), 4096)
        pieces = -(-V // vc)
        vc = -(-(-(-V // pieces)) // 256) * 256
        ldd = min(vc, -(-V // 64) * 64)
        covered = 0
        for v0 in range(0, V, vc):
            n = min(V - v0, vc)
            assert n <= ldd and -(-n // 16) * 16 <= ldd  # a 16-column store stays inside the row
            covered += n
        assert covered == V


# ------------------------------------------------------------------ gated decode
def gd_plan(M, I, gs, nt, pt):
    chunks = -(-I // 128)
    groups = chunks * (128 // gs)
    rs = groups | 1
    parts = [(chunks * 16 * M + 1) * 16, groups * nt * 8 * 16, -(-pt * 32 * rs * 8 // 16) * 16, (pt + 16) * 32 * nt * 32]
    return chunks, groups, rs, sum(parts) + 17 * 4


@pytest.mark.parametrize("F,I,gs", [(1, 64, 64), (11008, 4096, 128), (13824, 5120, 128), (1371, 512, 32), (300, 8128, 32),
                                    (14000, 4096, 64)])
def test_gated_decode_steps_and_slots(F, I, gs):
    tiles = -(-F // 16)
    grid = min(tiles, SMS)
    starts = [tiles * b // grid for b in range(grid + 1)]
    assert starts[0] == 0 and starts[-1] == tiles and all(a < b for a, b in zip(starts, starts[1:]))
    chunks = -(-I // 128)
    for nt in {b - a for a, b in zip(starts, starts[1:])}:
        steps = nt * chunks
        bounds = [steps * w // 16 for w in range(17)]
        slots = {}
        for w in range(16):
            for s in range(bounds[w], bounds[w + 1]):
                slots.setdefault((s // chunks, w), 0)
                slots[(s // chunks, w)] += 1
        used = [t + w for t, w in slots]
        assert len(set(used)) == len(used) and max(used) < nt + 16
        for t in range(nt):                           # the summing warp finds the same segments
            found = [w for w in range(16) if bounds[w] < (t + 1) * chunks and bounds[w + 1] > t * chunks
                     and bounds[w + 1] > bounds[w]]
            assert found == [w for tt, w in slots if tt == t]
            assert sum(slots[(t, w)] for w in found) == chunks


@pytest.mark.parametrize("gs", [128, 64, 32])
def test_gated_decode_words_of_one_mma_lie_in_one_group(gs):
    def place(r):
        if gs == 128:
            return r >> 2, r & 3
        if gs == 64:
            return (r & 7) >> 1, (r >> 3) * 2 + (r & 1)
        return r & 3, r >> 2
    at = [place(r) for r in range(16)]
    assert sorted(at) == [(t, j) for t in range(4) for j in range(4)]
    per = 4 // (128 // gs)                            # word slots of a group
    for r, (t, j) in enumerate(at):
        assert r * 8 // gs == j // per
    # what a lane loads is what it holds: contiguous words
    for t in range(4):
        words = [at.index((t, j)) for j in range(4)]
        if gs == 128:
            assert words == list(range(4 * t, 4 * t + 4))
        elif gs == 64:
            assert words == [2 * t, 2 * t + 1, 8 + 2 * t, 9 + 2 * t]
        else:
            assert words == [t, 4 + t, 8 + t, 12 + t]


def test_gated_decode_shared_memory_fits():
    for M, I, gs in itertools.product(range(1, 17), (64, 512, 4096, 5120, 11008, 49152), (32, 64, 128)):
        if I % gs:
            continue
        nt = 1 if M <= 8 else 2
        fit = [n for n in range(1, 33) if gd_plan(M, I, gs, nt, n)[3] <= 224 * 1024]
        assert fit == list(range(1, len(fit) + 1))
        if M == 1 and I <= 11008 and gs == 128:
            assert len(fit) >= 2
