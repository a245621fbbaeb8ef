"""The 8-bit block rounding and the block tables' oracle against hand-worked values, brute force
and properties of their definitions."""

import numpy as np
import pytest

from oracle.kv8 import BLOCK, Kv8Rows, block_tables_update, quantize_block, round_e4m3


def _e4m3_grid():
    vals = [m * 2.0 ** -9 for m in range(8)]
    vals += [(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8)]
    return np.array([v for v in vals if v <= 448])


def test_e4m3_rounding_is_the_nearest_grid_value():
    grid = _e4m3_grid()
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.uniform(0, 470, 4000), np.exp2(rng.uniform(-14, 8.8, 4000)), grid])
    got = round_e4m3(x)
    best = np.abs(grid[None] - np.minimum(x, 448)[:, None]).min(1)
    assert np.all(np.isin(got, grid)) and np.all(np.abs(got - np.minimum(x, 448)) <= best)
    assert np.array_equal(round_e4m3(-x), -got)
    # ties go to the even mantissa: 17 lies between 16 (even) and 18, 19 between 18 and 20 (even)
    assert list(round_e4m3([17.0, 19.0, 2.0 ** -10, 3 * 2.0 ** -10])) == [16.0, 20.0, 0.0, 2.0 ** -8]


def test_e4m3_rounding_matches_torch():
    torch = pytest.importorskip("torch")
    x = np.random.default_rng(1).standard_normal(20000).astype(np.float32) * 100
    x = np.clip(x, -448, 448)
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(round_e4m3(x), want)


def test_int8_block_by_hand():
    x = np.zeros((BLOCK, 2))
    x[0] = [127.0, -63.5]  # scale 1: halves go to even
    x[1] = [0.5, 1.5]
    c, s = quantize_block(x, "int8")
    assert s == 1.0 and list(c[0]) == [127.0, -64.0] and list(c[1]) == [0.0, 2.0] and not c[2:].any()


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_block_edge_values(code):
    c, s = quantize_block(np.zeros((BLOCK, 4)), code)
    assert s == 0 and not c.any()
    for bad in (np.inf, -np.inf, np.nan):
        x = np.ones((BLOCK, 4))
        x[5, 2] = bad
        c, s = quantize_block(x, code)
        assert np.isnan(s) and not c.any()
    # the largest value maps to the end of the grid, whatever its size
    for top in (3e38, 1.0, 1e-40):
        x = np.zeros((BLOCK, 4), np.float32)
        x[3, 1] = -top
        c, s = quantize_block(x, code)
        assert c[3, 1] == -{"int8": 127, "e4m3": 448}[code] and np.isfinite(s)


@pytest.mark.parametrize("code", ["int8", "e4m3"])
def test_error_is_at_most_half_a_step(code):
    x = np.random.default_rng(2).standard_normal((BLOCK, 128)).astype(np.float32)
    c, s = quantize_block(x, code)
    err = np.abs(c * np.float64(s) - x)
    if code == "int8":
        assert err.max() <= 0.5 * s * (1 + 2 ** -16)
    else:  # half a step of the value's binade, or of the smallest
        assert np.all(err <= np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * s) * (1 + 2 ** -16))
    # a scale from another maximum fails the same bound
    assert np.abs(np.rint(x / (s * 0.9)).clip(-127, 127) * s * 0.9 - x).max() > 0.5 * s


def test_rows_do_not_depend_on_the_split():
    x = np.random.default_rng(3).standard_normal((200, 8)).astype(np.float32)
    one = Kv8Rows(8, "int8")
    one.append(x)
    many = Kv8Rows(8, "int8")
    for t in range(200):
        many.append(x[t:t + 1])
    assert np.array_equal(one.rows(), many.rows()) and len(one.codes) == 3 and len(one.tail) == 8
    assert np.array_equal(one.tail, x[192:])


def test_block_tables_by_hand():
    table = np.full((2, 1, 4), -1)
    table[0, 0, 0] = 7
    free = np.array([0, 1, 2, 3, 4, 5, 6, -1])
    # sequence 0 has 3 tokens in block 7 and takes 6 (block size 4): positions 3 ... 8, blocks 6, 5
    r = block_tables_update(table, free, 7, [3, 0], [6, 2], 4, 10)
    assert list(r["block_table"][0, 0]) == [7, 6, 5, -1] and list(r["block_table"][1, 0]) == [4, -1, -1, -1]
    assert r["free_count"] == 4 and list(r["seq_lens"]) == [9, 2] and not r["turned_down"]
    assert list(r["slots"][:, 0]) == [31, 24, 25, 26, 27, 20, 16, 17, -1, -1]
    assert list(r["token_pos"]) == [3, 4, 5, 6, 7, 8, 0, 1, -1, -1]
    assert list(r["token_seq"]) == [0] * 6 + [1] * 2 + [-1] * 2 and list(r["cu_new"]) == [0, 6, 8]


def test_block_tables_conserve_blocks():
    rng = np.random.default_rng(4)
    B, planes, bs, mb = 6, 2, 4, 5
    nb = 40
    table, free, count, lens = np.full((B, planes, mb), -1), np.arange(nb), nb, np.zeros(B, int)
    turned = 0
    for _ in range(300):
        new = rng.integers(0, 6, B)
        new[rng.random(B) < 0.15] = -1
        r = block_tables_update(table, free, count, lens, new, bs, 20)
        table, free, count, lens = r["block_table"], r["free_list"], r["free_count"], r["seq_lens"]
        turned += r["turned_down"]
        used = [table[b, p, j] for b in range(B) for p in range(planes) for j in range(-(-lens[b] // bs))]
        assert sorted(used + list(free[:count])) == list(range(nb))
        stored = r["slots"][r["token_pos"] >= 0].ravel()
        assert len(set(stored)) == stored.size  # no two tokens share a row
    assert 0 < turned < 300
