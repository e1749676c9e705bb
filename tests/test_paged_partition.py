"""How the paged attention divides its work, restated on the host: the closed forms of the plan, the
walk of every CTA over its units, which partials it leaves and which of them are joined."""
import random

import pytest

TILE = 128


def pair_tiles(ctx, n_q, s, pairs):
    """KV tiles of a KV head's first `pairs` pairs of Q tiles (s tokens each), closed form."""
    if pairs <= 0:
        return 0
    cut = 0
    if pairs * s > n_q:
        cut = (ctx + n_q - 1) // TILE + 1
        pairs -= 1
    a = ctx + s - 1
    if s >= TILE:
        return cut + pairs * (a // TILE + 1) + (s // TILE) * pairs * (pairs - 1) // 2
    r = TILE // s

    def F(n):
        m = n // r
        return r * (m * (m - 1) // 2) + m * (n - m * r)

    return cut + pairs + F(a // s + pairs) - F(a // s)


def sequence(n_q, ctx, G):
    tiles = (n_q * G + 127) // 128
    pairs, odd = tiles >> 1, tiles & 1
    units = 2 * pair_tiles(ctx, n_q, 256 // G, pairs) + ((ctx + n_q - 1) // TILE + 1 if odd else 0)
    return pairs, odd, units


def cta_of(t, U, n):
    return ((t + 1) * n - 1) // U


@pytest.mark.parametrize("G", [1, 2, 4, 8, 16])
def test_closed_form_of_the_pairs(G):
    rng = random.Random(G)
    s = 256 // G
    for _ in range(400):
        n_q, ctx = rng.randint(1, 3000), rng.choice((0, 1, 127, 128, rng.randint(0, 5000)))
        pairs = sequence(n_q, ctx, G)[0]
        for P in {0, 1, pairs // 2, pairs}:
            if P <= pairs:
                want = sum((ctx + min((p + 1) * s, n_q) - 1) // TILE + 1 for p in range(P))
                assert pair_tiles(ctx, n_q, s, P) == want


def chunk_division(G, hkv, seqs, n):
    """Every CTA's walk; asserts that each (item, Q tile, KV tile) is done once, that a CTA leaves at
    most one partial per slot, and that the CTAs joined for a Q tile are those that hold it."""
    plan = [0]
    for n_q, ctx in seqs:
        plan.append(plan[-1] + (hkv * sequence(n_q, ctx, G)[2] if n_q else 0))
    U, TQ = plan[-1], 128 // G
    if U == 0:
        return
    done, partial, joins, whole = {}, {}, {}, set()
    for c in range(n):
        lo, hi = U * c // n, U * (c + 1) // n
        left = hi - lo
        if left <= 0:
            continue
        b = max(i for i in range(len(seqs)) if plan[i] <= lo and plan[i + 1] > plan[i])
        n_q, ctx = seqs[b]
        pairs, odd, head = sequence(n_q, ctx, G)
        g, r = divmod(lo - plan[b], head)
        p = max(q for q in range(pairs + odd) if 2 * pair_tiles(ctx, n_q, 2 * TQ, q) <= r)
        before = r - 2 * pair_tiles(ctx, n_q, 2 * TQ, p)
        units = left
        while left > 0:
            pair = p < pairs
            w, t0 = (2 if pair else 1), p * 2 * TQ
            tiles = (ctx + min(t0 + w * TQ, n_q) - 1) // TILE + 1
            tiles0 = (ctx + t0 + TQ - 1) // TILE + 1 if pair else tiles
            k0, k1 = -(-before // w), min(tiles, -(-(before + left) // w))
            for X in ((0, 1) if pair else (0,)):
                mine = tiles0 if pair and X == 0 else tiles
                end, item = min(k1, mine), (b, g, p, X)
                for k in range(k0, end):
                    assert (item, k) not in done
                    done[item, k] = c
                if k0 < end:
                    if k0 == 0 and k1 >= mine:
                        whole.add(item)
                    else:
                        slot = 0 if k0 else 1
                        assert (c, slot, X) not in partial
                        partial[c, slot, X] = item
                        if k0 == 0:
                            us = lo + units - left
                            joins[c, X] = cta_of(us + w * (mine - 1), U, n), item
            left -= w * tiles - before
            if left <= 0:
                break
            before = 0
            p += 1
            if p == pairs + odd:
                p, g = 0, g + 1
                if g == hkv:
                    g, b = 0, b + 1
                    while plan[b + 1] == plan[b]:
                        b += 1
                    n_q, ctx = seqs[b]
                    pairs, odd, head = sequence(n_q, ctx, G)
    want = set()
    for b, (n_q, ctx) in enumerate(seqs):
        tiles = (n_q * G + 127) // 128 if n_q else 0
        for g in range(hkv):
            for q in range(tiles):
                X = q & 1 if q >> 1 < tiles >> 1 else 0
                for k in range((ctx + min((q + 1) * TQ, n_q) - 1) // TILE + 1):
                    want.add(((b, g, q >> 1, X), k))
    assert want == set(done)
    joined = set()
    for (c, X), (last, item) in joins.items():
        parts = [c] + [i for i in range(c + 1, last + 1) if (i, 0, X) in partial]
        assert all(partial[i, 0, X] == item for i in parts[1:])
        assert set(parts) == {done[x] for x in done if x[0] == item}
        joined.add(item)
    assert joined == set(partial.values()) and not joined & whole


@pytest.mark.parametrize("n_cta", [1, 2, 7, 37, 148])
def test_chunk_work_is_divided_and_joined_exactly(n_cta):
    rng = random.Random(n_cta)
    for _ in range(150):
        G = rng.choice((1, 2, 4, 8, 16))
        seqs = [(rng.choice((0, 1, 2, rng.randint(1, 40), rng.randint(1, 700))),
                 rng.choice((0, 1, 127, 128, rng.randint(0, 3000)))) for _ in range(rng.randint(1, 5))]
        chunk_division(G, rng.choice((1, 2, 3)), seqs, n_cta)


@pytest.mark.parametrize("n_cta", [1, 5, 148, 256])
def test_decode_partials_have_slots_of_their_own(n_cta):
    """A row's CTAs are those between the first and the last tile's; with fewer tiles than CTAs
    (some CTAs empty) there are as many pieces as tiles; slot row + CTA is never shared."""
    rng = random.Random(n_cta)
    for _ in range(200):
        hkv = rng.choice((1, 2, 8))
        rows = []  # (row index, tiles); sequences without a token keep their row numbers
        for b in range(rng.randint(1, 6)):
            tiles = rng.choice((0, 1, rng.randint(1, 40)))
            rows += [(b * hkv + g, tiles) for g in range(hkv) if tiles]
        U = sum(t for _, t in rows)
        if not U:
            continue
        slots, at = set(), 0
        owner = [c for c in range(n_cta) for _ in range(U * c // n_cta, U * (c + 1) // n_cta)]
        for row, tiles in rows:
            first, last = cta_of(at, U, n_cta), cta_of(at + tiles - 1, U, n_cta)
            have = sorted(set(owner[at:at + tiles]))
            assert have[0] == first and have[-1] == last
            assert len(have) == (tiles if U < n_cta else last - first + 1)
            if len(have) > 1:
                for c in have:
                    assert row + c not in slots and row + c < len(range(6 * hkv)) + 256
                    slots.add(row + c)
            at += tiles
