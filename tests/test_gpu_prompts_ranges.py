"""The calls for prompts at the ends of their ranges: sequences without rows, small and large value scales, tables so wide that
costs of the deal are counted coarsely, rows of tiny numbers."""
import numpy as np
import pytest
import torch

from paged_cases import Cache, ints
from test_gpu_prompts import Prompt, Rope, Shared, _fork, _room
from test_gpu_shared_split import Split, slot_by_slot

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
    s = Split(c, [8, 2, 1, 5] * 4, 8, 8, 8)
    s.call()
    exact, c.scale["v"] = c.scale["v"], taken
    s.check(status=4096)
    c.scale["v"] = exact                                         # slot by slot all scales are what they are
    s = Shared(c, [8, 2, 1, 5] * 4, 8, 8, 8, width=0)
    s.ints[2] = s.ints[2][:, :16].contiguous()
    assert slot_by_slot(16, 8, 2, 8, 8, 16, 0)
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


# ------------------------------------------------------------------------------------------------ the deal's costs
def cost_shift(units, max_pages):
    """By which power of two the library counts the costs of `units` units of up to max_pages pages more coarsely."""
    most, shift = 21 + 5 * (max_pages // 2 + 1), 0
    while units * ((most >> shift) + 1) >= 1 << 30:
        shift += 1
    return shift


def _wide(rows, width):
    table = torch.full((len(rows), width), -1, dtype=torch.int32, device="cuda")
    table[:, :len(rows[0])] = ints(rows)
    return table


# At 5 and more a unit of one tile would cost nothing by the count; it is given a cost of 1.
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("kv,width,shift", [(4, 2 ** 23, 1), (8, 2 ** 23, 2), (8, 2 ** 25 - 1, 4), (32, 2 ** 25 - 1, 6)])
@pytest.mark.parametrize("window", [0, 300])
def test_prompts_behind_wide_tables(fmt, kv, width, shift, window):
    lens, live = [5000 if kv < 32 else 1500, 700, 64, 129, 0, 900, 1], [40, 300, 64, 129, 0, 3, 1]
    c = Cache(105, lens, kv, fmt)
    p = Prompt(c, live, 3, window=window)
    assert cost_shift(kv * (len(lens) + p.tokens * 3 // 256), width) == shift
    p.ints[3] = _wide(c.table, width)
    p.call()
    p.check()


@pytest.mark.parametrize("kv,width,shift", [(2, 2 ** 23, 1), (4, 2 ** 25 - 1, 4), (16, 2 ** 25 - 1, 6)])
def test_shared_pages_behind_wide_tables(kv, width, shift):
    n = 16
    c = Cache(106, [700 + 190 * b for b in range(n)], kv, "int8")
    _fork(c, 2, 8, 640)
    s = Split(c, [8, 1, 0, 5] * 4, 8, 8, 8)
    assert cost_shift(kv * (2 * n + n * 8 * 8 // 256), width) == shift
    s.ints[2] = _wide(c.table, width)
    s.call()
    s.check()


def test_far_windows_of_many_heads():
    """The same windows at the beginning and at the end of the longest sequences there can be: the deal, and with it the order
    of sums, differs."""
    width, by, kv = 2 ** 25 - 1, 2 ** 25 - 50, 16
    c = Cache(107, [900, 840, 1000], kv, "int8")
    p = Prompt(c, [200, 1, 33], 3, window=100)
    near = p.ints[3]
    p.ints[2] += 64 * by
    p.ints[3] = torch.full((3, width), -1, dtype=torch.int32, device="cuda")
    p.ints[3][:, by:by + near.shape[1]] = near
    assert cost_shift(kv * (3 + p.tokens * 3 // 256), width) == 3
    p.call()
    p.check()


# ------------------------------------------------------------------------------------------------ tiny rows
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("rot,interleaved", [(128, False), (64, True)])
@pytest.mark.parametrize("old,new", [(1e-25, 1e-24), (1e-24, 1e-26), (1e-30, 1e-28), (1e-36, 1e-35), (1.0, 1e-30), (1e-30, 1.0)])
def test_rotated_append_of_tiny_rows(fmt, rot, interleaved, old, new):
    """Scales of which quotients are divided, in blocks that begin with older rows; pages without new rows stay."""
    lens, live, kv = [40, 25, 64, 7, 100], [9, 20, 1, 7, 80], 2
    c = Cache(108, [n - r for n, r in zip(lens, live)], kv, fmt, spare=20, spread=old)
    _room(c, lens)
    others = [p for p in range(c.pages) if not any(p in row[(n - r) // 64:-(-n // 64)] for row, n, r in zip(c.table, lens, live))]
    r = Rope(c, live, 2, rot, interleaved, spread=new)
    before = [t.clone() for t in r.dev]
    assert r.call() == 0
    r.check()
    for t, was in zip(r.dev, before):
        assert len(others) > 15 and torch.equal(t[others].view(torch.uint8), was[others].view(torch.uint8))


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("older", [0.0, 1.0, 1e-30])
def test_rotated_append_of_zeros(fmt, older):
    """Blocks whose new rows are all zero, behind older rows (of zeros too) and without any."""
    lens, live = [40, 25, 18, 64], [9, 20, 2, 64]
    c = Cache(109, [n - r for n, r in zip(lens, live)], 2, fmt, spare=20, spread=older)
    _room(c, lens)
    r = Rope(c, live, 2, 64, False, spread=0.0)
    assert r.call() == 0
    r.check()
    for n, row in zip(lens, c.table):                            # and rows behind them
        assert np.isfinite(c.scale["k"][0, row[(n - 1) // 64], :, (n - 1) % 64 // 16]).all()
    again = Rope(c, live, 2, 64, False, spread=1.0, seed=5)
    again.dev = r.dev
    assert again.call() == 0
    again.check()
