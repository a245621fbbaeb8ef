"""How the packed attention shares out an item's tiles (CPU, with the sources' own constants): every CTA between
the first and the last one of an item begins a tile of it, so the merge finds a part of each."""

import os
import random
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "streaming_kv_cache_duo_gb300",
                    "csrc")


def _text(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def _constants():
    """Places of a share at least, and per head dim (two, one, stream_two, stream_one, item_two, item_one)."""
    text = _text("ragged_internal.h")
    places = [tuple(map(int, m.split(", "))) for m in re.findall(r"kRaggedPlaces\d+ = \{(\d+(?:, \d+){5})\}", text)]
    return int(re.search(r"kRaggedLeast = (\d+)", text).group(1)), places


def test_a_tile_takes_no_more_places_than_a_share_has():
    least, places = _constants()
    assert len(places) == 2 and max(max(p[:4]) for p in places) <= least
    # and the compiler sees to it, of the only ones there are
    assert "static_assert(tiles_fit_a_share(kRaggedPlaces128) && tiles_fit_a_share(kRaggedPlaces64)" in _text("ragged_internal.h")
    assert "RaggedPlaces{" not in _text("duo_api.cu") and "RaggedPlaces{" not in _text("attn_ragged.cu")


def _holders(W, ctas, first, place, tiles):
    """CTAs in whose share a tile begins."""
    out = []
    for c in range(ctas):
        lo, hi = c * W // ctas, (c + 1) * W // ctas
        j = max(0, -((first - lo) // place))  # the first tile from lo on
        if j < tiles and first + j * place < hi:
            out.append(c)
    return out


def test_every_cta_of_a_shared_item_has_a_tile():
    """The kernel's shares and owner of a place, on random lines of items."""
    least, sets = _constants()
    rng = random.Random(3)
    for _ in range(600):
        p = rng.choice(sets)
        items, W = [], 0
        for _ in range(rng.randint(1, 40)):
            kind = rng.randrange(4)
            items.append((W + p[4 + kind % 2], p[kind], max(1, int(2 ** rng.uniform(0, 9)))))
            W = items[-1][0] + items[-1][1] * items[-1][2]
        ctas = min(152, max(1, W // least))
        for first, place, tiles in items:
            got = _holders(W, ctas, first, place, tiles)
            end = ((first + (tiles - 1) * place + 1) * ctas + W - 1) // W - 1
            assert got == list(range(got[0], end + 1))
