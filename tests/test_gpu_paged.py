"""Coding into pages and verify attention over them, against the oracle (oracle/paged.py)."""
import numpy as np
import pytest
import torch

import oracle.paged as P
import speculative_decode_verify_gb300 as va
from paged_cases import Cache, attention_bounds, bf16, ints
from test_paged_host import _calls

pytestmark = pytest.mark.gpu
D = 128
SCALE = D ** -0.5


def _same_codes(got, want, fmt):
    """The same values (a zero's sign is free); NaN codes are compared as bytes."""
    got, want = got.view(np.uint8), want.view(np.uint8)
    nan = (want & 0x7F) == 0x7F if fmt == "e4m3" else np.zeros(want.shape, bool)
    np.testing.assert_array_equal(got[nan], want[nan])
    np.testing.assert_array_equal(P.decode(got, fmt)[~nan], P.decode(want, fmt)[~nan])


def _append(c, live, rows, dev, seed=1, spread=1.0, special=False):
    """Append rows on the GPU pools ``dev`` and in the cache's own arrays; returns the status word."""
    rng = np.random.default_rng(seed)
    new, status = {}, torch.zeros(1, dtype=torch.int32, device="cuda")
    for w in "kv":
        x = rng.standard_normal((len(c.lens), rows, c.kv, D)).astype(np.float32) * spread
        if special:
            x[:, 0, 0, :5] = [np.inf, -np.inf, np.nan, 1e-30, 0.0]
            x[:, -1, -1] = 0.0
        new[w] = bf16(x)
    va.kv_page_append_b8(new["k"][0].cuda(), new["v"][0].cuda(), ints(live), ints(c.lens), ints(c.table), *dev,
                         dev_status=status)
    for w in "kv":
        for b, n in enumerate(c.lens):
            if live[b] > 0:
                P.append(new[w][1][b].astype(np.float32), n - live[b], n, c.table[b], c.codes[w][0], c.scale[w][0], c.fmt)
    return int(status.item())


def _check_pool(c, dev):
    for i, w in enumerate("kv"):
        _same_codes(dev[i].view(torch.uint8).cpu().numpy(), c.codes[w][0], c.fmt)
        np.testing.assert_array_equal(dev[2 + i].cpu().numpy(), c.scale[w][0])   # NaN where none was written


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("lens,live,rows,kv", [
    ([1, 16, 17, 64, 65, 130], [1, 1, 1, 1, 1, 1], 1, 1),
    ([5, 23, 64, 70, 128, 3], [5, 6, 0, 6, 3, 3], 6, 2),          # a sequence without rows, blocks begun and new
    ([200, 333], [200, 150], 200, 3),                              # prompts: whole, and behind a history
    ([8], [8], 8, 8),
])
@pytest.mark.parametrize("spread", [1.0, 30.0])                    # 30: the older rows of a block are coded again
def test_append_is_the_oracles_bit_for_bit(fmt, lens, live, rows, kv, spread):
    c = Cache(21, [n - r for n, r in zip(lens, live)], kv, fmt, spare=20)
    free = [p for p in range(c.pages) if c.refs[p] == 0]
    c.table = [r + [-1] * 8 for r in c.table]
    c.lens = list(lens)
    for b, n in enumerate(lens):
        for x in range(-(-n // 64)):
            if c.table[b][x] < 0:
                c.table[b][x] = free.pop()
    dev = c.dev(0)
    assert _append(c, live, rows, dev, spread=spread) == 0
    _check_pool(c, dev)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("exponent", [0, 100, -70, -79, -81, -100, -120])      # of the blocks' largest value
def test_append_rounds_every_quotient_of_bfloat16_values_correctly(fmt, exponent):
    """A block for each of the 128 significands of the largest value; in it, each significand of an element under 15
    exponents (and their negatives).  Then a larger row: the 15 before it are coded again from their codes."""
    top = (1 + np.arange(128) / 128) * 2.0 ** exponent
    x = np.zeros((128, 16, 1, D), np.float32)
    for r in range(15):
        x[:, r, 0] = (-1) ** r * (1 + np.arange(128) / 128) * 2.0 ** (exponent - 1 - r)
    x[:, 14, 0, 0] = top
    x[:, 15, 0] = x[:, 3, 0] * 1.5
    x[:, 15, 0, 5] = 2 * top[::-1]
    c = Cache(29, [0] * 128, 1, fmt, spare=128)
    c.table = [[b] for b in range(128)]
    dev = c.dev(0)
    for start, end in ((0, 15), (15, 16)):
        t, rows = bf16(x[:, start:end])
        va.kv_page_append_b8(t.cuda(), t.cuda(), ints([end - start] * 128), ints([end] * 128), ints(c.table), *dev)
        for w in "kv":
            for b in range(128):
                P.append(rows[b].astype(np.float32), start, end, c.table[b], c.codes[w][0], c.scale[w][0], fmt)
        _check_pool(c, dev)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("grows", [(0, 1), (2, 5)])             # K's and V's new row, in powers of two
def test_append_codes_every_older_code_again_correctly_for_every_pair_of_scales(fmt, grows):
    """A block for each pair of significands of the older rows' largest value and of the new row's; in its older row every
    code (K: positive, V: negative)."""
    kv, top = 64, P.TOP[fmt]
    every = np.minimum(np.arange(128), 126 if fmt == "e4m3" else 127).astype(np.uint8)
    row = {"k": every, "v": every | 0x80 if fmt == "e4m3" else (-every.astype(np.int8)).view(np.uint8)}
    for part in range(4):
        n = 4096 * part + np.arange(4096).reshape(64, kv)
        older, newer = n // 128, n % 128
        c = Cache(30, [0] * 64, kv, fmt, spare=64)
        c.table, c.lens, new = [[b] for b in range(64)], [2] * 64, {}
        for w, g in zip("kv", grows):
            c.codes[w][0, :, :, 0] = row[w]
            c.scale[w][0, :, :, 0] = ((128 + older) / 128).astype(np.float32) / top
            x = np.zeros((64, 1, kv, D), np.float32)
            x[:, 0, :, 0] = (128 + newer) / 128 * 2.0 ** g
            new[w] = bf16(x)
        dev = c.dev(0)
        va.kv_page_append_b8(new["k"][0].cuda(), new["v"][0].cuda(), ints([1] * 64), ints(c.lens), ints(c.table), *dev)
        for w in "kv":
            for b in range(64):
                P.append(new[w][1][b].astype(np.float32), 1, 2, c.table[b], c.codes[w][0], c.scale[w][0], fmt)
        _check_pool(c, dev)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_append_codes_infinities_and_nan_and_says_so(fmt):
    c = Cache(22, [37, 64], 2, fmt)
    dev = c.dev(0)
    assert _append(c, [4, 2], 4, dev, special=True) == 512
    _check_pool(c, dev)


@pytest.mark.parametrize("bad,bit", [("count", 1024), ("length", 4), ("page", 128), ("above", 1024)])
def test_append_leaves_a_wrong_sequence_alone(bad, bit):
    c = Cache(23, [40, 80, 70], 1, "e4m3")
    dev = c.dev(0)
    before = [t.clone() for t in dev]
    lens, live, table = list(c.lens), [2, 2, 2], [list(r) for r in c.table]
    if bad == "count":
        live[1] = 3
    elif bad == "length":
        lens[1] = 64 * len(table[1]) + 1
    elif bad == "above":
        lens[1] = 1
    else:
        table[1][1] = c.pages
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    new = torch.ones(3, 2, 1, D, dtype=torch.bfloat16, device="cuda")
    va.kv_page_append_b8(new, new, ints(live), ints(lens), ints(table), *dev, dev_status=status)
    assert int(status.item()) == bit
    mine = [p for p in c.table[1] if p >= 0]
    for a, b in zip(dev, before):
        a, b = a.cpu().numpy(), b.cpu().numpy()
        np.testing.assert_array_equal(a[mine].view(np.uint8), b[mine].view(np.uint8))
        if a.shape[-1] == D:                                      # codes of another sequence have changed
            assert any(not np.array_equal(a[p].view(np.uint8), b[p].view(np.uint8)) for p in c.table[0] if p >= 0)


@pytest.mark.parametrize("live", [1, 5, 40])
def test_append_to_the_last_positions_that_a_table_can_hold(live):
    """A table of 2^25 - 1 pages, full: blocks behind the last would begin past 2^31, and their table entries lie in the
    next sequence's row, which has no page there."""
    width, rows, fmt = 2 ** 25 - 1, 100, "int8"
    lens = [64 * width, 5]
    table = torch.full((2, width), -1, dtype=torch.int32, device="cuda")
    table[0, width - 1], table[1, 0] = 3, 1
    rng = np.random.default_rng(28)
    codes = [rng.integers(-127, 128, (4, 2, 64, D)).astype(np.int8).view(np.uint8) for _ in "kv"]
    scale = [rng.random((4, 2, 4)).astype(np.float32) for _ in "kv"]
    dev = [torch.as_tensor(c.copy()).view(torch.int8).cuda() for c in codes] + [torch.as_tensor(s.copy()).cuda() for s in scale]
    new = [bf16(rng.standard_normal((2, rows, 2, D))) for _ in "kv"]
    status = ints([0])
    va.kv_page_append_b8(new[0][0].cuda(), new[1][0].cuda(), ints([live, 2]), ints(lens), table, *dev, dev_status=status)
    assert int(status.item()) == 0
    for i in range(2):
        for b, (n, page) in enumerate(((live, {width - 1: 3}), (2, {0: 1}))):
            P.append(new[i][1][b].astype(np.float32), lens[b] - n, lens[b], page, codes[i], scale[i], fmt)
        _same_codes(dev[i].view(torch.uint8).cpu().numpy(), codes[i], fmt)
        np.testing.assert_array_equal(dev[2 + i].cpu().numpy(), scale[i])


@pytest.mark.parametrize("name", sorted(_calls()))
def test_the_binding_refuses_a_host_tensor_among_the_others(name):
    call, args = _calls()[name]
    for key, t in args.items():
        if torch.is_tensor(t):
            mixed = {k: x.cuda() if torch.is_tensor(x) and k != key else x for k, x in args.items()}
            with pytest.raises(ValueError):
                call(**mixed)


# ------------------------------------------------------------------------------------------------ attention
def _attend(c, dev, live, rows, group, window=0, sink=None, scale=SCALE, seed=9, spread=1.0, table=None, lens=None,
            ws=None, qs=None):
    heads = c.kv * group
    rng = np.random.default_rng(seed)
    qt, qn = bf16(rng.standard_normal((len(c.lens), rows, heads, D)) * spread) if qs is None else qs
    n = len(c.lens)
    if ws is None:
        ws = torch.zeros(va.va_paged_workspace_bytes(n, rows, c.kv, group), dtype=torch.uint8, device="cuda")
    out = torch.full((n, rows, heads, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((n, rows, heads), float("nan"), device="cuda")
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    sk = None if sink is None else torch.tensor(sink, dtype=torch.float32, device="cuda")
    va.verify_attn_paged_b8(qt.cuda(), ints(live), ints(lens or c.lens), ints(table or c.table), *dev, scale, sk, ws, out,
                            lse, window=window, dev_status=status)
    return qn, out.double().cpu().numpy(), lse.double().cpu().numpy(), int(status.item())


def _check(c, got, live, window=0, sink=None, scale=SCALE, table=None, status=0):
    qn, out, lse, st = got
    want = P.attention(qn, live, c.lens, table or c.table, c.codes["k"][0], c.codes["v"][0], c.scale["k"][0],
                       c.scale["v"][0], c.fmt, scale, sink, window)
    assert st == status
    tol_out, tol_lse = attention_bounds(*want)
    assert np.array_equal(np.isfinite(lse), np.isfinite(want[1]))
    some = np.isfinite(want[1])
    assert np.all(np.abs(lse[some] - want[1][some]) <= tol_lse[some])
    assert np.all(np.isfinite(out)) and np.all(np.abs(out - want[0]) <= tol_out), np.max(np.abs(out - want[0]) / tol_out)
    for b, n in enumerate(live):
        assert np.all(out[b, n:] == 0) and np.all(lse[b, n:] == -np.inf)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("lens,live,rows,kv,group", [
    ([1], [1], 1, 1, 1),
    ([1, 15, 16, 17, 63, 64, 65, 129], [1] * 8, 1, 1, 6),
    ([300, 0, 77, 8], [8, 0, 3, 8], 8, 2, 6),                       # 48 matrix rows; an empty sequence
    ([64, 640, 33], [5, 2, 0], 5, 3, 3),
    ([900, 200], [7, 8], 8, 1, 8),                                  # 64 matrix rows
    ([1000, 31, 450], [2, 1, 2], 2, 4, 5),
    ([128, 70], [3, 4], 4, 1, 8),                                   # 32
    ([190, 66], [3, 3], 3, 2, 8),                                   # 24
    ([222, 99, 512], [5, 5, 1], 5, 2, 7),                           # 35
    ([222, 99], [8, 6], 8, 1, 5),                                   # 40
    ([222, 99], [8, 1], 8, 1, 7),                                   # 56
])
def test_attention_matches_the_oracle(fmt, lens, live, rows, kv, group):
    c = Cache(31, lens, kv, fmt)
    sink = list(np.linspace(-2, 3, kv * group))
    _check(c, _attend(c, c.dev(0), live, rows, group, sink=sink), live, sink=sink)
    _check(c, _attend(c, c.dev(0), live, rows, group), live)


@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 65, 200, 10 ** 6])
def test_windows(window):
    """Entries below every window are -1: those pages have been freed."""
    c = Cache(32, [500, 64, 3, 129], 2, "int8")
    live = [6, 6, 3, 1]
    table = [list(r) for r in c.table]
    for b, n in enumerate(c.lens):
        for x in range(max(0, n - live[b] - window + 1) // 64):
            table[b][x] = -1
    _check(c, _attend(c, c.dev(0), live, 6, 2, window=window, table=table), live, window=window)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("rows,group", [(1, 6), (6, 2), (8, 3), (8, 6), (8, 8)])
@pytest.mark.parametrize("window", [20, 40, 90])
def test_values_before_the_window_do_not_matter(fmt, rows, group, window):
    """Blocks before every row's window, in pages whose end is seen, get scales of 2^60 and more: output and bounds are
    those of the cache without them."""
    c = Cache(44, [500, 442, 1343, 190], 2, fmt)
    live, dev, hidden = [rows] * 4, c.dev(0), 0
    for b, n in enumerate(c.lens):
        first = n - rows - window + 1                        # the first position that a row sees
        for block in range(first // 64 * 4, first // 16):
            dev[3][c.table[b][block // 4], :, block % 4] = 2.0 ** (60 + 20 * (block % 4))
            hidden += 1
    assert hidden
    _check(c, _attend(c, dev, live, rows, group, window=window), live, window=window)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("spread,scale", [(40.0, SCALE), (1.0, -0.3), (1.0, 0.0), (1e-4, 5.0), (1.0, 3.0)])
def test_peaky_flat_and_negative_scores(fmt, spread, scale):
    c = Cache(33, [700, 90], 1, fmt)
    _check(c, _attend(c, c.dev(0), [3, 4], 4, 6, scale=scale, spread=spread), [3, 4], scale=scale)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_scales_that_differ_by_orders_of_magnitude(fmt):
    c = Cache(34, [400, 400], 2, fmt)
    rng = np.random.default_rng(2)
    for w, low, high in (("k", -3, 0), ("v", -12, 12)):
        s = c.scale[w]
        f = 10.0 ** rng.uniform(low, high, s.shape)
        c.scale[w] = (s * np.sort(f, axis=1 if w == "k" else 3)).astype(np.float32)
    c.scale["v"][:, c.table[0][2]] = 0.0                             # rows of zeros
    _check(c, _attend(c, c.dev(0), [2, 2], 2, 6), [2, 2])


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("rows,group", [(4, 7), (8, 6), (8, 8)])
def test_scales_that_differ_by_orders_of_magnitude_with_many_pairs(fmt, rows, group):
    c = Cache(43, [1300, 400], 1, fmt)
    rng = np.random.default_rng(3)
    for w, low, high in (("k", -3, 0), ("v", -12, 12)):
        f = np.sort(10.0 ** rng.uniform(low, high, c.scale[w].shape), axis=1 if w == "k" else 3)
        c.scale[w] = (c.scale[w] * f).astype(np.float32)
    c.scale["v"][:, c.table[0][2]] = 0.0
    _check(c, _attend(c, c.dev(0), [rows, rows], rows, group), [rows, rows])


def _far_apart(seed, lens, kv, fmt, rows, group, down, small=(1,)):
    """A cache whose blocks `small` of every sequence have V scales 2^-down of the others', and queries whose weight is on a
    key of the first of them."""
    c = Cache(seed, lens, kv, fmt)
    for b, n in enumerate(c.lens):
        for block in small:
            if 16 * block < n:
                c.scale["v"][0, c.table[b][block // 4], :, block % 4] *= np.float32(2.0 ** -down)
    rng = np.random.default_rng(seed)
    q = rng.standard_normal((len(lens), rows, kv, group, D)) * 0.1
    for b, n in enumerate(c.lens):
        at = 16 * small[0] + 3
        if at < n - rows:
            page = c.table[b][at // 64]
            k = P.decode(c.codes["k"][0, page, :, at % 64], fmt) * c.scale["k"][0, page, :, at % 64 // 16, None]
            q[b] += k[None, :, None] * np.array([2.0, 0.5, 1.0, 1.5, 0.0, 2.0, 1.0, 0.7])[None, None, :group, None]
    return c, bf16(q.reshape(len(lens), rows, kv * group, D))


def _check_far(c, got, live, small, sink=None, window=0, table=None, status=0):
    """As _check, but a page with a block of `small` next to others is computed in fp32 (an exponential and sums over at most
    8 x 256 keys: 2^-16), so that the bound's term for weights below f16's range (2^-30 of n keys of the largest
    code and scale, at the segment's largest weight) is left for the keys of the other pages alone."""
    qn, out, lse, st = got
    table = table or c.table
    want = P.attention(qn, live, c.lens, table, c.codes["k"][0], c.codes["v"][0], c.scale["k"][0], c.scale["v"][0], c.fmt,
                       SCALE, sink, window)
    assert st == status
    rest = np.zeros(want[1].shape)              # the largest weight of a key in another page
    for b, n in enumerate(live):
        pages = [x for x in range(-(-c.lens[b] // 64)) if 0 <= table[b][x] < c.pages and x not in [i // 4 for i in small]]
        for h in range(qn.shape[2]):
            for x in pages:
                kv = h // (qn.shape[2] // c.kv)
                k = P.decode(c.codes["k"][0, table[b][x], kv], c.fmt) * np.repeat(c.scale["k"][0, table[b][x], kv], 16)[:, None]
                for r in range(n):
                    p = c.lens[b] - n + r - 64 * x              # the row's position in the page
                    lo = max(0, p - window + 1) if window else 0
                    if p >= lo and lo < 64:
                        z = SCALE * (k[lo:p + 1].astype(np.float64) @ qn[b, r, h])
                        rest[b, r, h] = max(rest[b, r, h], np.exp(z.max() - want[1][b, r, h]))
    tol_out, tol_lse = attention_bounds(*want[:4], want[4] * rest)
    assert np.all(np.abs(out - want[0]) <= tol_out), np.max(np.abs(out - want[0]) / np.maximum(tol_out, 1e-300))
    some = np.isfinite(want[1])
    assert np.array_equal(some, np.isfinite(lse)) and np.all(np.abs(lse[some] - want[1][some]) <= tol_lse[some])
    for b, n in enumerate(live):
        assert np.all(out[b, n:] == 0) and np.all(lse[b, n:] == -np.inf)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("rows,group", [(1, 6), (3, 4), (8, 3), (8, 6), (8, 8)])
@pytest.mark.parametrize("down", [8, 11, 20, 24, 28, 31, 45, 70])
def test_a_block_of_small_values_that_carries_the_weight(fmt, rows, group, down):
    c, q = _far_apart(45, [700, 0, 130, 40], 2, fmt, rows, group, down)
    live = [rows, 0, rows, min(rows, 2)]
    for sink in (None, list(np.linspace(-2, 30, 2 * group))):
        got = _attend(c, c.dev(0), live, rows, group, qs=q, sink=sink)
        if down < 11:
            _check(c, got, live, sink=sink)
        else:
            _check_far(c, got, live, (1,), sink=sink)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("rows,group", [(2, 5), (8, 6)])
@pytest.mark.parametrize("window,none", [(0, True), (150, False), (150, True), (70, False)])
def test_scales_far_apart_in_windows_and_with_pages_that_are_none(fmt, rows, group, window, none):
    small = (41, 42, 43, 14, 17, 1, 2, 80)
    c, q = _far_apart(46, [700, 300, 64, 1300], 2, fmt, rows, group, 40, small)
    live = [rows, 1, rows, rows]
    table = [list(r) for r in c.table]
    if none:
        table[0][9] = -1
        table[3][19] = c.pages
    _check_far(c, _attend(c, c.dev(0), live, rows, group, qs=q, window=window, table=table), live, small, window=window,
               table=table, status=128 if none else 0)


@pytest.mark.parametrize("rows,group", [(1, 6), (8, 6)])
def test_scales_far_apart_leave_the_other_heads_bits_alone(rows, group):
    """Calls in which one sequence's one head has such scales, and calls without them, on one workspace."""
    c, q = _far_apart(47, [900, 300, 500], 2, "e4m3", rows, group, 0)
    dev, live = c.dev(0), [rows, rows, 1]
    ws = torch.full((va.va_paged_workspace_bytes(3, rows, 2, group),), 0xFF, dtype=torch.uint8, device="cuda")
    plain = _attend(c, dev, live, rows, group, qs=q, ws=ws)
    c.scale["v"][0, c.table[1][0], 1, 1] *= np.float32(2.0 ** -30)
    far = [_attend(c, c.dev(0), live, rows, group, qs=q, ws=ws) for _ in range(2)]
    for i in (1, 2):
        np.testing.assert_array_equal(far[0][i], far[1][i])
        same = np.ones(far[0][i].shape, bool)
        same[1, :, group:] = False
        np.testing.assert_array_equal(far[0][i][same], plain[i][same])
    _check(c, far[0], live)
    again = _attend(c, dev, live, rows, group, qs=q, ws=ws)
    for i in (1, 2):
        np.testing.assert_array_equal(again[i], plain[i])


@pytest.mark.parametrize("rows,group", [(2, 6), (8, 6)])
def test_scales_far_apart_and_a_query_without_a_number(rows, group):
    c, clean = _far_apart(48, [700, 130], 2, "e4m3", rows, group, 30)
    q = clean[0].clone()
    q[0, 1, 2, 7] = float("nan")
    got = [_attend(c, c.dev(0), [rows, rows], rows, group, qs=(t, None)) for t in (clean[0], q)]
    hit = np.zeros(got[0][2].shape, bool)
    hit[0, 1, 2] = True
    assert np.all(np.isnan(got[1][1][hit])) and np.all(np.isnan(got[1][2][hit]))
    for i in (1, 2):
        np.testing.assert_array_equal(got[0][i][~hit], got[1][i][~hit])


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("rows,group", [(1, 6), (3, 4), (8, 6)])
@pytest.mark.parametrize("up", [-130, -60, 85, 97, 110, 118])
def test_values_near_the_ends_of_the_range(fmt, rows, group, up):
    """All values times 2^up: the weighted sums stay in fp32's range as long as the output does (values of 2^-130 lose digits
    of their scales, which the oracle takes as they are; an output below 2^-126 is a multiple of 2^-133 in bf16)."""
    c = Cache(49, [700, 64, 130], 2, fmt)
    with np.errstate(all="ignore"):
        c.scale["v"] = (c.scale["v"] * 2.0 ** up).astype(np.float32)
    live = [rows] * 3
    qn, out, lse, st = _attend(c, c.dev(0), live, rows, group)
    want = P.attention(qn, live, c.lens, c.table, c.codes["k"][0], c.codes["v"][0], c.scale["k"][0], c.scale["v"][0], fmt, SCALE)
    tol, _ = attention_bounds(*want)
    assert st == 0 and np.all(np.isfinite(out)) and np.all(np.abs(out - want[0]) <= tol + 2.0 ** -133)


def test_pages_that_are_none_are_masked_and_told():
    c = Cache(35, [300, 200, 64], 1, "e4m3")
    for bad in (-1, c.pages, 2 ** 31 - 1, -7):
        table = [list(r) for r in c.table]
        table[0][1] = table[2][0] = bad
        table[1][3] = table[1][0]
        for sink in (None, [0.5, 1.5]):
            _check(c, _attend(c, c.dev(0), [2, 1, 2], 2, 2, table=table, sink=sink), [2, 1, 2], table=table, sink=sink,
                   status=128)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("rows,group,window", [(8, 3, 0), (8, 6, 0), (8, 8, 0), (5, 5, 200), (7, 8, 65)])
def test_many_pairs_with_pages_that_are_none_windows_and_empty_sequences(fmt, rows, group, window):
    c = Cache(42, [700, 0, 129, 64, 1500, 3], 2, fmt)
    live = [rows, 0, 1, rows, 2, 3]
    table = [list(r) for r in c.table]
    table[0][9] = table[4][22] = -1
    table[2][2] = c.pages
    table[4][20] = table[4][21]
    _check(c, _attend(c, c.dev(0), live, rows, group, window=window, table=table, spread=2.0), live, window=window, table=table,
           status=128)


def test_wrong_counts_make_an_empty_sequence():
    c = Cache(36, [300, 200, 64], 1, "e4m3")
    for live, lens, bit in (([2, 3, 2], None, 1024), ([2, -1, 2], None, 1024), ([2, 2, 2], [300, 64 * 6 + 1, 64], 4),
                            ([2, 2, 2], [300, 1, 64], 1024)):
        qn, out, lse, st = _attend(c, c.dev(0), live, 2, 2, lens=lens)
        assert st == bit and np.all(out[1] == 0) and np.all(lse[1] == -np.inf)
        ok = [2, 0, 2]
        want = P.attention(qn, ok, c.lens, c.table, c.codes["k"][0], c.codes["v"][0], c.scale["k"][0], c.scale["v"][0],
                           "e4m3", SCALE)
        tol, _ = attention_bounds(*want)
        assert np.all(np.abs(out - want[0]) <= tol)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_many_short_and_one_long(fmt):
    """Work split over a long axis next to sequences that share one CTA; shared pages."""
    lens = [3000] + [int(n) for n in np.random.default_rng(4).integers(0, 150, 70)]
    c = Cache(37, lens, 2, fmt)
    live = [min(n, 1 + i % 2) for i, n in enumerate(lens)]
    _check(c, _attend(c, c.dev(0), live, 2, 3), live)


def test_one_workspace_serves_calls_of_every_shape_and_replays():
    c = Cache(38, [200, 333, 64], 2, "e4m3")
    dev = c.dev(0)
    ws = torch.zeros(va.va_paged_workspace_bytes(3, 8, 2, 8), dtype=torch.uint8, device="cuda")
    for rows, group in ((8, 8), (1, 1), (3, 6), (8, 6)):
        live = [min(rows, 2), rows, rows]
        _check(c, _attend(c, dev, live, rows, group, ws=ws), live)
    # a captured call, replayed over changed lengths and interleaved with an eager call on the same workspace
    rows, group = 2, 6
    qt, qn = bf16(np.random.default_rng(1).standard_normal((3, rows, 12, D)))
    q, live, lens, table = qt.cuda(), ints([1, 1, 1]), ints([1, 1, 1]), ints(c.table)
    out, lse = torch.zeros(3, rows, 12, D, dtype=torch.bfloat16, device="cuda"), torch.zeros(3, rows, 12, device="cuda")
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        va.verify_attn_paged_b8(q, live, lens, table, *dev, SCALE, None, ws, out, lse)
    for now, n in (([200, 333, 64], [2, 1, 0]), ([70, 64, 2], [2, 2, 2]), ([200, 333, 64], [2, 1, 0])):
        lens.copy_(ints(now))
        live.copy_(ints(n))
        graph.replay()
        c2 = c
        want = P.attention(qn, n, now, c2.table, c2.codes["k"][0], c2.codes["v"][0], c2.scale["k"][0], c2.scale["v"][0],
                           "e4m3", SCALE)
        tol, _ = attention_bounds(*want)
        got = out.double().cpu().numpy()
        assert np.all(np.abs(got - want[0]) <= tol)
        first = out.clone()
        _check(c, _attend(c, dev, [1, 2, 2], 2, 3, ws=ws), [1, 2, 2])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(first, out)             # the same inputs give the same bits


def test_another_stream():
    c = Cache(39, [500, 77], 2, "int8")
    dev = c.dev(0)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = _attend(c, dev, [4, 3], 4, 6)
    _check(c, got, [4, 3])


@pytest.mark.parametrize("rows,group", [(2, 3), (4, 8)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_query_without_a_number_keeps_to_its_own_rows(rows, group, bad):
    c = Cache(40, [900, 130], 2, "e4m3")
    dev, live = c.dev(0), [rows, rows]
    clean, _ = bf16(np.random.default_rng(2).standard_normal((2, rows, 2 * group, D)))
    q = clean.clone()
    q[0, 1, 2, 7] = bad
    got = [_attend(c, dev, live, rows, group, qs=(t, None)) for t in (clean, q)]
    hit = np.zeros(got[0][2].shape, bool)
    hit[0, 1, 2] = True
    assert np.all(np.isnan(got[1][1][hit])) and np.all(np.isnan(got[1][2][hit]))
    for i in (1, 2):
        np.testing.assert_array_equal(got[0][i][~hit], got[1][i][~hit])


def test_two_calls_at_once():
    """On two streams, with workspaces of their own and one pool, again and again."""
    c = Cache(41, [2500, 64, 700], 2, "int8")
    dev = c.dev(0)
    calls = []
    for rows, group in ((1, 6), (8, 6)):
        q, _ = bf16(np.random.default_rng(rows).standard_normal((3, rows, 2 * group, D)))
        calls.append([q.cuda(), ints([rows] * 3), torch.zeros(3, rows, 2 * group, D, dtype=torch.bfloat16, device="cuda"),
                      torch.zeros(va.va_paged_workspace_bytes(3, rows, 2, group), dtype=torch.uint8, device="cuda"),
                      torch.cuda.Stream()])
    lens, table = ints(c.lens), ints(c.table)
    want = []
    for q, live, out, ws, _ in calls:
        va.verify_attn_paged_b8(q, live, lens, table, *dev, SCALE, None, ws, out)
        want.append(out.clone())
        out.zero_()
    torch.cuda.synchronize()
    for _ in range(20):
        for q, live, out, ws, stream in calls:
            va.verify_attn_paged_b8(q, live, lens, table, *dev, SCALE, None, ws, out, stream=stream)
    torch.cuda.synchronize()
    for (_, _, out, _, _), w in zip(calls, want):
        assert torch.equal(out, w)


def test_positions_and_pool_offsets_past_32_bits_of_bytes():
    """A pool of over 4 GB (page numbers whose byte offsets pass 2^32) and a history of 131,080 positions."""
    kv, fmt, n = 8, "int8", 131080
    need = -(-n // 64)
    pages = 4 * 2 ** 30 // (kv * 64 * D) + need + 8
    codes = [torch.zeros(pages, kv, 64, D, dtype=torch.int8, device="cuda") for _ in range(2)]
    scale = [torch.zeros(pages, kv, 4, device="cuda") for _ in range(2)]
    first = pages - need
    g = torch.Generator(device="cuda").manual_seed(3)
    for c, s in zip(codes, scale):
        c[first:] = torch.randint(-127, 128, c[first:].shape, generator=g, device="cuda", dtype=torch.int8)
        s[first:] = torch.rand(s[first:].shape, generator=g, device="cuda") * 0.02
    table = torch.arange(first, pages, dtype=torch.int32, device="cuda")[None]
    q = torch.randn(1, 2, kv, D, generator=g, device="cuda").to(torch.bfloat16)
    out, lse = torch.zeros_like(q), torch.zeros(1, 2, kv, device="cuda")
    ws = torch.zeros(va.va_paged_workspace_bytes(1, 2, kv, 1), dtype=torch.uint8, device="cuda")
    va.verify_attn_paged_b8(q, ints([2]), ints([n]), table, *codes, *scale, SCALE, None, ws, out, lse)
    for h in range(kv):
        k, v = ((c[first:, h].double() * s[first:, h].double().repeat_interleave(16, 1)[..., None]).reshape(-1, D)[:n]
                for c, s in zip(codes, scale))
        for r in range(2):
            z = SCALE * (k[:n - 1 + r] @ q[0, r, h].double())
            w = torch.softmax(z, 0)
            want, size = w @ v[:n - 1 + r], w @ v[:n - 1 + r].abs()
            reach = SCALE * float((k.abs() @ q[0, r, h].double().abs()).max())
            tol, tol_lse = attention_bounds(want.cpu().numpy(), float(torch.logsumexp(z, 0)), size.cpu().numpy(),
                                            np.array(reach), np.array(n * 127 * 0.02))
            assert np.all(np.abs(out[0, r, h].double().cpu().numpy() - want.cpu().numpy()) <= tol)
            assert abs(float(lse[0, r, h]) - float(torch.logsumexp(z, 0))) <= tol_lse


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("n,kv,group,rows", [(64 * 152 * 9, 1, 1, 1), (70001, 8, 1, 2), (100000, 1, 6, 3), (64 * 152 * 16, 1, 8, 4),
                                             (196608, 1, 6, 8), (90000, 2, 7, 8), (64 * 152 * 8 + 1, 3, 4, 3)])
def test_long_histories_in_which_a_cta_reuses_its_stages(fmt, n, kv, group, rows):
    need = -(-n // 64)
    g = torch.Generator(device="cuda").manual_seed(n)
    if fmt == "int8":
        codes = [torch.randint(-127, 128, (need, kv, 64, D), generator=g, device="cuda", dtype=torch.int8) for _ in range(2)]
        value, top = [c.double() for c in codes], 127.0
    else:
        f8 = [torch.randn(need, kv, 64, D, generator=g, device="cuda").mul_(80).clamp_(-448, 448).to(torch.float8_e4m3fn)
              for _ in range(2)]
        codes, value, top = f8, [c.double() for c in f8], 448.0
    scale = [torch.rand(need, kv, 4, generator=g, device="cuda") * 2 / top for _ in range(2)]
    k, v = ((c * s.double().repeat_interleave(16, 2)[..., None]).transpose(0, 1).reshape(kv, -1, D)
            for c, s in zip(value, scale))
    table = torch.randperm(need, generator=g, device="cuda").to(torch.int32)
    codes = [torch.empty_like(c).view(torch.uint8).index_copy_(0, table.long(), c.view(torch.uint8)).view(c.dtype) for c in codes]
    pool_scale = [torch.empty_like(s).index_copy_(0, table.long(), s) for s in scale]
    q = torch.randn(1, rows, kv * group, D, generator=g, device="cuda").to(torch.bfloat16)
    out, lse, status = torch.zeros_like(q), torch.zeros(q.shape[:3], device="cuda"), ints([0])
    ws = torch.zeros(va.va_paged_workspace_bytes(1, rows, kv, group), dtype=torch.uint8, device="cuda")
    va.verify_attn_paged_b8(q, ints([rows]), ints([n]), table[None], *codes, *pool_scale, SCALE, None, ws, out, lse,
                            dev_status=status)
    assert int(status.item()) == 0
    for r in range(rows):
        p = n - rows + r + 1
        x = q[0, r].double().view(kv, group, D)
        z = SCALE * x @ k[:, :p].transpose(1, 2)
        total = torch.logsumexp(z, -1)
        w = torch.exp(z - total[..., None])
        want, size = w @ v[:, :p], w @ v[:, :p].abs()
        reach = SCALE * (x.abs() @ k[:, :p].abs().transpose(1, 2)).amax(-1)
        tol, tol_lse = attention_bounds(*(t.cpu().numpy() for t in (want, total, size, reach)),
                                        np.array(p * 2.0)[None, None])
        assert np.all(np.abs(out[0, r].double().view(kv, group, D).cpu().numpy() - want.cpu().numpy()) <= tol)
        assert np.all(np.abs(lse[0, r].double().view(kv, group).cpu().numpy() - total.cpu().numpy()) <= tol_lse)
