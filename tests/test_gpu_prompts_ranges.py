"""The calls for prompts at the ends of their ranges: sequences without rows, small and large value scales."""
import numpy as np
import pytest

from paged_cases import Cache
from test_gpu_prompts import Prompt, Rope, Shared, _fork, _room

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------------------------------------ sequences without rows
def test_first_rows_of_sequences_without_rows_are_not_looked_at():
    lens, live = [40, 50, 20, 60, 0], [4, 0, 3, 0, 0]
    c = Cache(101, [36, 50, 17, 60, 0], 2, "e4m3", spare=20)
    _room(c, lens)
    r = Rope(c, live, 2, 128, False, gap=1)
    for b, x in ((1, -1), (3, r.tokens + 1), (4, 2 ** 31 - 1)):
        r.args[0][b] = x
    assert r.call() == 0
    r.check()
    p = Prompt(c, live, 2, gap=1)
    for b, x in ((1, -2 ** 31), (3, p.tokens + 1), (4, 2 ** 31 - 1)):
        p.ints[0][b] = x
    p.call()
    p.check()


# ------------------------------------------------------------------------------------------------ value scales
def _far(c, powers, seed=7):
    """Value scales times powers of two; then what the kernels of prompts and shared pages take them for."""
    rng = np.random.default_rng(seed)
    c.scale["v"] = c.scale["v"] * 2.0 ** rng.integers(*powers, c.scale["v"].shape).astype(np.float32)
    return np.where(c.scale["v"] == 0, np.float32(0), np.maximum(c.scale["v"], np.float32(2.0 ** -60)))


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("powers,status", [((-80, -79), 4096), ((-70, -50), 4096), ((-90, 0), 4096), ((-50, 40), 0), ((-52, -51), 0)])
def test_value_scales_below_the_range_are_told_of(fmt, powers, status):
    c = Cache(102, [700, 90, 333], 2, fmt)
    taken = _far(c, powers)
    p = Prompt(c, [300, 90, 1], 3)
    p.call()
    c.scale["v"] = taken
    p.check(status=status)


@pytest.mark.parametrize("kind,status", [("large", 4096), ("nan", 4096), ("zero", 0), ("behind", 0), ("no page", 128)])
def test_value_scales_that_are_told_of(kind, status):
    """A scale above the range or none at all, of a page that is read; zeros and what is not read are not told of."""
    c = Cache(103, [300, 200], 1, "int8")
    page = c.table[0][1]
    if kind == "zero":
        c.codes["v"][0, page], c.scale["v"][0, page] = 0, 0.0
    elif kind == "behind":
        c.scale["v"][0, c.table[1][3], :, 1:] = 2.0 ** 90        # positions from 208 on
    elif kind == "no page":
        c.scale["v"][0, page] = 2.0 ** 90
        c.table[0][1] = -1
    else:
        c.scale["v"][0, page] = 2.0 ** 61 if kind == "large" else np.nan
    p = Prompt(c, [300, 200], 2)
    p.call()
    if kind == "behind":
        c.scale["v"][0, c.table[1][3], :, 1:] = np.nan           # (no part of the error bounds)
    if status != 4096:
        p.check(status=status)
    assert int(p.status.item()) == status


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("where", ["shared", "own", "all"])
def test_value_scales_of_shared_calls_below_the_range_are_told_of(fmt, where):
    c = Cache(104, [700 + 9 * b for b in range(16)], 2, fmt)
    _fork(c, 2, 8, 640)
    pages = {"shared": [c.table[9][4]], "own": [c.table[3][10]], "all": range(c.pages)}[where]
    for page in pages:
        c.scale["v"][0, page] *= np.float32(2.0 ** -70)
    taken = np.maximum(c.scale["v"], np.float32(2.0 ** -60))
    s = Shared(c, [8, 2, 1, 5] * 4, 8, 8, 8)
    s.call()
    exact, c.scale["v"] = c.scale["v"], taken
    s.check(status=4096)
    c.scale["v"] = exact                                         # slot by slot all scales are what they are
    s = Shared(c, [8, 2, 1, 5] * 4, 8, 8, 8, width=0)
    s.ints[2] = s.ints[2][:, :16].contiguous()
    s.call()
    s.check()


@pytest.mark.parametrize("blocks", [(0, 3, 5, 6, 12), tuple(range(17)), tuple(range(8, 30))])
@pytest.mark.parametrize("power", [-50, 0, 40])
def test_zero_values_next_to_small_and_large_ones(power, blocks):
    """Blocks of zeros, whole tiles of them at the beginning and behind others."""
    c = Cache(103, [600], 1, "int8")
    c.scale["v"] = c.scale["v"] * np.float32(2.0 ** power)
    for blk in blocks:
        page, part = c.table[0][blk // 4], blk % 4
        c.codes["v"][0, page, 0, 16 * part:16 * part + 16] = 0
        c.scale["v"][0, page, 0, part] = 0.0
    for sink in (True, False):
        p = Prompt(c, [600], 2, sink=sink)
        p.call()
        p.check()
