"""Pins of the paged cache's oracle (CPU): closed forms and invariants."""
import math

import numpy as np
import pytest

import oracle.paged as P
from paged_cases import Cache


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_codes_stand_for_rows_within_half_a_step(fmt):
    c = Cache(3, [150], 2, fmt)
    rng = np.random.default_rng(3)
    rng.permutation(c.pages)
    x = rng.standard_normal((150, 2, 128)).astype(np.float32)       # the K rows that Cache drew first
    pg = np.array(c.table[0])[np.arange(150) // 64]
    of = np.arange(150) % 64
    s = c.scale["k"][0][pg, :, of // 16][..., None]
    back = P.decode(c.codes["k"][0][pg, :, of], fmt) * s
    # E4M3: 2^-4 of the value, or half the subnormal step; INT8: half a step of the block's scale
    half = np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10 * s) if fmt == "e4m3" else 0.5 * s
    assert np.all(np.abs(back - x) <= half * (1 + 1e-5))


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_appending_in_two_parts_keeps_or_raises_scales(fmt):
    rng = np.random.default_rng(5)
    x = rng.standard_normal((40, 1, 128)).astype(np.float32)
    x[20] *= 50.0                                                    # the second part raises its block's scale
    once = [np.zeros((1, 1, 64, 128), np.uint8), np.zeros((1, 1, 4), np.float32)]
    twice = [a.copy() for a in once]
    P.append(x, 0, 40, [0], *once, fmt)
    P.append(x[:19], 0, 19, [0], *twice, fmt)
    P.append(x[19:], 19, 40, [0], *twice, fmt)
    np.testing.assert_array_equal(once[1], twice[1])
    a, b = (P.decode(p[0][0, 0], fmt) * p[1][0, 0].repeat(16)[:, None] for p in (once, twice))
    step = once[1][0, 0].repeat(16)[:, None]
    assert np.all(np.abs(a - b) <= (step if fmt == "int8" else 2.0 ** -3 * np.abs(a) + 2.0 ** -9 * step) + 1e-12)
    np.testing.assert_array_equal(a[19:40], b[19:40])


def test_nonfinite_rows_do_not_touch_the_scale():
    for fmt in ("e4m3", "int8"):
        codes, scale = np.zeros((1, 1, 64, 128), np.uint8), np.zeros((1, 1, 4), np.float32)
        x = np.ones((2, 1, 128), np.float32)
        x[1, 0, :3] = [np.inf, -np.inf, np.nan]
        P.append(x, 0, 2, [0], codes, scale, fmt)
        assert scale[0, 0, 0] == np.float32(1) / P.TOP[fmt]
        top = float(P.TOP[fmt])
        np.testing.assert_array_equal(P.decode(codes[0, 0, 1, :4], fmt), [top, -top, 0, top])


def test_attention_of_equal_keys_is_the_mean():
    c = Cache(7, [70, 5], 1, "e4m3")
    c.codes["k"][:] = 0
    c.scale["k"][:] = 1.0
    q = np.ones((2, 2, 3, 128))
    out, lse, *_ = P.attention(q, [2, 0], c.lens, c.table, c.codes["k"][0], c.codes["v"][0], c.scale["k"][0],
                               c.scale["v"][0], "e4m3", 0.1, sink=[-np.inf, 0.0, 1.0])
    pg, of = np.array(c.table[0])[np.arange(70) // 64], np.arange(70) % 64
    v = P.decode(c.codes["v"][0][pg, 0, of], "e4m3").astype(np.float64) * c.scale["v"][0][pg, 0, of // 16][:, None]
    for r, n in ((0, 69), (1, 70)):
        for m, e in enumerate((0.0, 1.0, math.e)):
            # 70 terms below 4, each rounded to 2^-53
            np.testing.assert_allclose(out[0, r, m], v[:n].sum(0) / (n + e), rtol=1e-12, atol=70 * 4 * 2.0 ** -53)
            assert abs(lse[0, r, m] - math.log(n + e)) < 1e-12
    assert np.all(out[1] == 0) and np.all(lse[1] == -np.inf)
    w, *_ = P.attention(q, [1, 0], c.lens, c.table, c.codes["k"][0], c.codes["v"][0], c.scale["k"][0], c.scale["v"][0],
                        "e4m3", 0.1, window=3)
    np.testing.assert_allclose(w[0, 0, 0], v[67:70].mean(0), rtol=1e-12, atol=1e-14)


def _counted(table, n):
    c = [0] * n
    for row in table:
        for p in row:
            if p >= 0:
                c[p] += 1
    return c


def test_page_operations_keep_the_counts():
    rng = np.random.default_rng(11)
    table, lens, refs = [[-1] * 8 for _ in range(6)], [0] * 6, [0] * 40
    for step in range(200):
        new = [int(rng.integers(0, 40)) if lens[b] < 400 else 0 for b in range(6)]
        before = [list(r) for r in table]
        copies = P.extend(table, lens, refs, new)
        if copies is None:
            assert table == before
        assert refs == _counted(table, 40)
        for b in range(6):                        # what a sequence is about to write is its own
            if copies is not None and new[b]:
                assert all(refs[table[b][x]] == 1 for x in range((lens[b] - new[b]) // 64, -(-lens[b] // 64)))
        src = [int(s) for s in rng.integers(-1, 3, 6)]
        P.reorder(table, lens, refs, src, group=3)
        assert refs == _counted(table, 40)
        if step % 10 == 0:
            to, n, moves = P.compact(table, refs)
            assert refs == _counted(table, 40) and all(r > 0 for r in refs[:n]) and not any(refs[n:])
            assert not {a for a, _ in moves} & {b for _, b in moves}
        lens = [max(0, n - int(rng.integers(0, 8))) if rng.random() < 0.3 else n for n in lens]   # rejected drafts


def test_beam_selection_small():
    l = np.log(np.array([[0.5, 0.25, 0.25], [0.1, 0.8, 0.1]]))
    p, t, s, _ = P.beam_select(l, [0.0, -1.0], 2, 4)
    assert p.tolist() == [[0, 1, 0, 0]] and t.tolist() == [[0, 1, 1, 2]]
    np.testing.assert_allclose(s[0], np.log([0.5, 0.8 * math.exp(-1), 0.25, 0.25]), rtol=1e-12)
    p, t, s, _ = P.beam_select(l, [0.0, -1.0], 2, 3, finished=[1, 1], end_token=2)
    assert p.tolist() == [[0, 1, -1]] and t.tolist() == [[2, 2, -1]] and s[0, 2] == -np.inf
    p, t, s, _ = P.beam_select(np.array([[np.inf, 0.0, np.inf, np.nan]]), [0.0], 1, 3)
    assert t.tolist() == [[0, 2, -1]] and abs(s[0, 0] + math.log(2)) < 1e-12
