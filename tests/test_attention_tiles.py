"""How attention's workgroups find their tiles (csrc/attention_device.h), gone
through on the CPU for offsets of every kind: with valid ones every tile has
its workgroups, with others every row and slot stays inside the buffers."""
import random

import pytest

SLOTS, SPLIT_TOKENS, SORTED, MOST_PARTS, KEYS = 512, 1024, 256, 8, 128


def segments(cu, T):
    """(start, length, is a sequence): before, between and after the offsets."""
    edges = [0] + [min(max(c, 0), T) for c in cu] + [T]
    return [(a, b - a if b > a else 0, 0 < i < len(cu)) for i, (a, b) in enumerate(zip(edges[:-1], edges[1:]))], edges


def find_tile(cu, T, shift, tile):
    segs, edges = segments(cu, T)
    seg = sum((edges[i] >> shift) + i <= tile for i in range(len(segs))) - 1
    start, length, sequence = segs[seg]
    at = tile - ((edges[seg] >> shift) + seg)
    return start, length if at >= 0 else 0, max(at, 0), sequence, 0, 1, 0


def launch(T, S, H, Hk, units=256):
    """The dk, dv launch: workgroups a key head, extra ones, least, fair."""
    extra = SLOTS // 2 // Hk if T >= SPLIT_TOKENS else 0
    return T // KEYS + S + 2 + extra, extra, max(1, 8 // (H // Hk)), Hk / units


def find_tile_by_size(cu, T, extra, least, fair, rank):
    segs, _ = segments(cu, T)
    n = [-(-length // KEYS) for _, length, _ in segs]
    work = sum(0.5 * m * (m + 1) for m, s in zip(n, segs) if s[2])
    larger = lambda m: sum(max(x - m, 0) for x in n)
    most = max(n)
    whole, cut, parts = most, 0, 1
    if extra > 0:
        share = max(least, -int(-min(work * fair, 1e9) // 1))
        if most > share:
            cut = max(larger(share), 1)
            parts = min(max((most + share // 2) // share, 2), MOST_PARTS, 1 + extra // cut)
            whole = share
    above = lambda m: larger(m) + (parts - 1) * (cut if m < whole else larger(m))
    if rank >= above(0):
        return 0, 0, 0, False, 0, 1, 0
    lo, hi = 1, most
    while lo < hi:
        m = (lo + hi) // 2
        lo, hi = (lo, m) if above(m) <= rank else (m + 1, hi)
    r = rank - above(lo)
    part, of, slot = 0, 1, 0
    assert r >= 0
    if lo > whole and rank < 2 * extra:
        part, of, slot, r = r % parts, parts, rank, r // parts
    having = [i for i, x in enumerate(n) if x >= lo]
    if r >= len(having):
        return 0, 0, 0, False, part, of, slot
    start, length, sequence = segs[having[r]]
    return start, length, n[having[r]] - lo, sequence, part, of, slot


def key_workgroups(cu, T, H, Hk):
    tiles, extra, least, fair = launch(T, len(cu) - 1, H, Hk)
    for rank in range(tiles):
        if len(cu) + 1 <= SORTED:
            yield extra, find_tile_by_size(cu, T, extra, least, fair, rank)
        else:
            yield extra, find_tile(cu, T, 7, rank)


def check(cu, T, H, Hk, valid):
    segs, _ = segments(cu, T)
    done = {}
    for extra, (start, length, tile, sequence, part, parts, slot) in key_workgroups(cu, T, H, Hk):
        assert 0 <= start and length >= 0 and start + length <= T
        if tile * KEYS >= length:
            continue                                            # the workgroup ends there
        assert tile >= 0
        if parts > 1:
            first = slot - part
            assert 0 <= part < parts <= MOST_PARTS and 0 <= first and first + part < 2 * extra
            assert 2 * extra * Hk <= SLOTS
            done.setdefault((start, length, tile), []).append((first, part, parts))
        else:
            done.setdefault((start, length, tile), []).append(None)
    if valid:
        want = {(start, length, t) for start, length, _ in segs for t in range(-(-length // KEYS))}
        assert set(done) == want
        slots = []
        for got in done.values():
            if got == [None]:
                continue
            first, _, parts = got[0]
            assert sorted(got) == [(first, i, parts) for i in range(parts)]
            slots += range(first, first + parts)
        assert len(slots) == len(set(slots))
    # the query tiles: 32, 64 or 128 rows
    shared = H // Hk
    hb = 2 if shared % 4 == 0 else 1 if shared % 2 == 0 else 0
    rows = 128 >> hb
    seen = {}
    for tile in range(T // rows + len(cu) + 1):
        start, length, at, *_ = find_tile(cu, T, 7 - hb, tile)
        assert 0 <= start and start + length <= T
        if 0 <= at and at * rows < length:
            seen[(start, length, at)] = seen.get((start, length, at), 0) + 1
        else:
            assert at * rows >= length
    if valid:
        assert seen == {(start, length, t): 1 for start, length, _ in segs for t in range(-(-length // rows))}


@pytest.mark.parametrize("seed", range(60))
def test_valid_offsets(seed):
    rng = random.Random(seed)
    T = rng.choice([1, 33, 1000, 1024, 3000, 20000])
    S = rng.choice([0, 1, 2, 7, 60, 61, 62, 63, 253, 254, 255, 300])
    points = sorted(rng.choice([rng.randrange(T + 1), rng.randrange(T + 1), 0, T]) for _ in range(S + 1))
    Hk = rng.choice([1, 2, 3, 8, 32])
    check(points, T, Hk * rng.choice([1, 2, 4, 8]), Hk, True)


@pytest.mark.parametrize("seed", range(120))
def test_any_offsets(seed):
    rng = random.Random(1000 + seed)
    T = rng.choice([1, 1000, 1024, 1100, 3000, 20000])
    S = rng.choice([1, 2, 5, 61, 62, 253, 254, 255, 300])
    kind = rng.randrange(3)
    points = [[rng.randrange(-50, T + 50), rng.choice([0, T, T + 5, -2 ** 31, 2 ** 31 - 1]), (i % 2) * T][kind]
              for i in range(S + 1)]
    Hk = rng.choice([1, 2, 8, 300])
    check(points, T, Hk * rng.choice([1, 4]), Hk, False)
