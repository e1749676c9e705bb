"""Consecutive items of the paged attention's chunk form, restated on the host: which batches make
a CTA finish a pair of Q tiles and load the q of another item behind it, and which bytes of a Q
tile's shared memory each warp touches then."""
import pytest

from test_paged_partition import TILE, pair_tiles, sequence

SMS = 148
ROW_BYTES, HALF = 128, 128 * 128

# (new tokens, cached tokens, page, query heads, KV heads): far more pairs than SMs. The lengths
# leave 20, 52 and 84 rows in the second Q tile of the last pair (16 heads in 8 groups), so that
# three, two and one of its four warps have no rows; a whole tile; other group sizes; a context.
STEADY = [([330] * 24, [0] * 24, 64, 16, 8), ([346] * 24, [0] * 24, 16, 16, 8), ([362] * 24, [5] * 24, 32, 16, 8),
          ([200] * 32, [0] * 32, 64, 16, 8), ([1100] * 4, [30] * 4, 128, 16, 8), ([470, 128] * 8, [100, 0] * 8, 256, 16, 8),
          ([90] * 40, [17] * 40, 64, 32, 4), ([333] * 12, [0] * 12, 64, 16, 16), ([50] * 200, [3] * 200, 16, 16, 1)]


def successions(seqs, G, hkv, n_cta=SMS):
    """Pairs whose Q tile 0 or 1 a CTA finishes whole (its rows are staged over the tile) and
    follows by another item that loads q into the same tile: (all of them, those with rows missing)."""
    TQ, plan = 128 // G, [0]
    for n_q, ctx in seqs:
        plan.append(plan[-1] + (hkv * sequence(n_q, ctx, G)[2] if n_q else 0))
    items = []  # (units, tiles of Q tile 0, tiles, pair, rows of Q tile 1)
    for n_q, ctx in seqs:
        pairs, odd, _ = sequence(n_q, ctx, G) if n_q else (0, 0, 0)
        head = []
        for p in range(pairs + odd):
            w, t0 = (2 if p < pairs else 1), p * 2 * TQ
            tiles = (ctx + min(t0 + w * TQ, n_q) - 1) // TILE + 1
            head.append((w * tiles, (ctx + t0 + TQ - 1) // TILE + 1, tiles, p < pairs, min(TQ, n_q - t0 - TQ) * G))
        items += head * hkv
    U, n, short = plan[-1], 0, 0
    for c in range(n_cta):
        lo, hi = U * c // n_cta, U * (c + 1) // n_cta
        at, staged = 0, (False, False, 0)
        for units, tiles0, tiles, pair, rows in items:
            w = 2 if pair else 1
            k0, k1 = max(0, -(-(lo - at) // w)), min(tiles, -(-(hi - at) // w))
            at += units
            if at - units >= hi or k0 >= k1:
                continue
            loads = (k0 < min(k1, tiles0), True) if pair else (True, False)
            for X in (0, 1):
                if staged[X] and loads[X]:
                    n += 1
                    short += X == 1 and staged[2] <= 96
            staged = (pair and k0 == 0 and k1 >= tiles0, pair and k0 == 0 and k1 >= tiles, rows)
    return n, short


def test_units_agree_with_the_plan():
    for n_q, ctx, G in ((700, 33, 2), (90, 17, 8), (5, 500, 16)):
        pairs, odd, units = sequence(n_q, ctx, G)
        assert units == 2 * pair_tiles(ctx, n_q, 256 // G, pairs) + odd * ((ctx + n_q - 1) // TILE + 1)


@pytest.mark.parametrize("qlens,ctx,page,hq,hkv", STEADY)
def test_steady_batches_follow_pairs_by_pairs(qlens, ctx, page, hq, hkv):
    n, short = successions(list(zip(qlens, ctx)), hq // hkv, hkv)
    assert n >= 50
    rows = [(t * hq // hkv - 1) % 256 + 1 - 128 for t in qlens]
    assert short > 0 or not any(0 < r <= 96 for r in rows)


def pieces(row):
    """The 16-byte pieces of a Q tile that hold a row's q (bf16: two halves of 64 dims; e4m3: two
    terms of 128 dims); the row's finished values are staged in the same ones."""
    return {half * HALF + row * ROW_BYTES + (((c ^ row) & 7) << 4) for half in (0, 1) for c in range(8)}


def test_a_warp_touches_its_own_rows_of_a_q_tile():
    """No barrier stands between the staging of finished rows and the next item's q: a warp may
    only touch what no other warp does."""
    owner = {}
    for row in range(128):
        assert len(pieces(row)) == 16
        for at in pieces(row):
            assert owner.setdefault(at, row // 32) == row // 32
    assert len(owner) == 2 * HALF // 16


def test_rows_staged_end_to_end_would_meet_another_warps_q():
    """256 bytes a row in order, the layout that looks natural: of every warp, staged rows lie where
    another warp's q goes."""
    q = {at: row // 32 for row in range(128) for at in pieces(row)}
    met = {row // 32 for row in range(128) for c in range(16) if q[row * 256 + 16 * c] != row // 32}
    assert met == {0, 1, 2, 3}
