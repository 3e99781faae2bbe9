"""A CPU model of how the 4-bit decode cuts its work: the plan (slots of a row,
ranges of a CTA) and the walk of the CTAs over units whose band tiles count
several times, after `plan_decode_fp4`, `Ranges` and `next_piece`.

For random batches, exact and generous bounds, right and wrong totals, every
number of splits and CTA counts down to one it checks that every tile of every
unit is in exactly one piece, that every slot below `splits` is filled by exactly
one piece or marked empty exactly once (the merge reads them all), that no slot
lies past them, and that with exact bounds no piece is longer than its limit.
"""
import random

import pytest

MOST = {False: 2048, True: 512}          # tiles of a piece: warp-level and tcgen05 kernel
BATCH = 384                              # sequences that are laid end to end


def cdiv(a, b):
    return -(-a // b)


def plan(tc, batch, unit, weight, total_k, tile, heads, ctas, want, max_tiles):
    """unit: most weighted tiles of a unit; weight: what the band adds to one."""
    most, least, small = MOST[tc], 4 if tc else 2, 0 if tc else 8
    total = (min(total_k, batch * max_tiles * tile) // tile + batch * (1 + weight)) * heads
    share = max(cdiv(total, ctas), least)
    waves = cdiv(share, most)
    length, ranges = cdiv(share, waves), ctas * waves
    pieces = cdiv(min(unit, total_k // tile + 1 + weight), most)
    least = 1 if want > 0 else least
    splits = max(pieces, 1)
    whole = batch > BATCH or want == 1 or (want <= 0 and unit <= max(length, small))
    if not whole:
        splits = max(want, pieces + 1 if pieces > 1 else 2) if want > 0 else cdiv(unit, length) + 1
        splits = min(splits, unit + 1, ranges)
        whole = splits == 1
    c_min = 0 if whole else least if splits == ranges else max(cdiv(unit, splits - 1), least)
    return splits, whole, waves, c_min


def walk(p, tc, tiles, plain, extra, heads, ctas):
    """Yields (unit, slot, first tile, tiles, slots used) of every piece."""
    splits, whole, waves, c_min = p
    most = MOST[tc]
    if whole:
        for hr in range(heads):
            for b, n in enumerate(tiles):
                C, x = max(most, n // splits + 1), 0
                while x < n:
                    left = min(n - x, C - x % C)
                    yield (hr, b), x // C, x, left, (n - 1) // C + 1
                    x += left
        return
    weighted = [n + extra * (n - s) for n, s in zip(tiles, plain)]
    prefix = [sum(weighted[:b]) for b in range(len(tiles) + 1)]
    per = prefix[-1]
    total = per * heads
    share = max(cdiv(total, ctas), 1)
    k = min(cdiv(share, most), waves)
    C = max(cdiv(share, k), c_min)

    def tile(b, v):
        return v if v <= plain[b] else plain[b] + (v - plain[b] + extra) // (extra + 1)

    for c in range(ctas):
        x = min(c * k * C, total)
        end = x + min(k * C, total - x)
        while x < end:
            hr, xb = divmod(x, per)
            b = max(i for i in range(len(tiles)) if prefix[i] <= xb)
            v0 = xb - prefix[b]
            n = min(weighted[b] - v0, end - x, C - x % C)
            start = hr * per + prefix[b]
            t0 = tile(b, v0)
            yield (hr, b), x // C - start // C, t0, tile(b, v0 + n) - t0, (start + weighted[b] - 1) // C - start // C + 1
            x += n


@pytest.mark.parametrize("tc", [False, True])
@pytest.mark.parametrize("want", [0, 1, 2, 3, 50, 100000])
def test_every_tile_and_every_slot_once(tc, want):
    for seed in range(50):
        rng = random.Random(1000 * want + seed)
        batch, heads = rng.choice([1, 1, 2, 5, 40]), rng.choice([1, 2, 3])
        extra = rng.choice([0, 6 if tc else 1])
        ctas, tile = rng.choice([1, 2, 7, 152 if tc else 608]), 128 if tc else 64
        tiles = [rng.choice([0, 1, 3, 10, 100, 3000, 30000]) * rng.randint(0, 2) + rng.randint(0, 3) for _ in range(batch)]
        longest = max(max(tiles), 1)
        bound = rng.choice([longest, longest, 3 * longest, 1 << 24])
        band = min(bound, rng.choice([0, 2, 9, 17])) if extra else 0
        plain = [max(n - band, 0) for n in tiles]
        keys = sum(tiles) * tile
        total_k = rng.choice([keys, keys, keys // 100, 3 * keys])
        p = plan(tc, batch, bound + extra * band, extra * band, total_k, tile, heads, ctas, want, bound)
        splits = p[0]
        filled, covered = {}, {(h, b): [] for h in range(heads) for b in range(batch)}
        for unit, slot, t0, n, used in walk(p, tc, tiles, plain, extra, heads, ctas):
            marked = [slot] if n == 0 else list(range(used, splits)) if t0 == 0 else []
            for s in marked + ([slot] if n else []):
                assert 0 <= s < splits and (unit, s) not in filled, (seed, unit, s)
                filled[unit, s] = True
            if n:
                covered[unit].append((t0, n))
            if bound == longest and total_k >= keys:
                assert n <= MOST[tc], (seed, n)
        for (h, b), pieces in covered.items():
            at = 0
            for t0, n in sorted(pieces):
                assert t0 == at, (seed, h, b)
                at += n
            assert at == tiles[b]
            if tiles[b] and splits > 1:
                assert sum(u == (h, b) for u, _ in filled) == splits, (seed, h, b)
