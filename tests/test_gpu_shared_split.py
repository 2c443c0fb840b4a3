"""Attention over shared pages in sizes that its own kernels take: pages that are none, short windows, groups with nothing in
common, calls at once, captured and replayed ones.  (Calls whose sizes say that little is read twice are handed to
verify_attn_paged_b8; here each call's sizes are looked at first.)"""
import pytest
import torch

import speculative_decode_verify_gb300 as va
from paged_cases import Cache
from test_gpu_prompts import SCALE, Shared, _fork

pytestmark = pytest.mark.gpu


def slot_by_slot(n_seqs, n_rows, kv, group, share, max_pages, window):
    """The library's rule on the sizes of a call: True where it is handed to verify_attn_paged_b8."""
    pages = min(max_pages, (window + n_rows) // 64 + 2) if window else max_pages
    pairs, whole = n_rows * group, n_rows * group * share
    rest = whole % 256
    tile = 9 * (whole // 256) + (9 if rest > 128 else 6 if rest else 0)
    return n_seqs * kv * pages * (1 + (pairs + 7) // 8) <= 6000 + 33 * n_seqs * kv + n_seqs // share * kv * pages * tile


class Split(Shared):
    """A call whose sizes go to the kernels of shared pages."""

    def call(self):
        n, rows, heads, _ = self.qd.shape
        assert not slot_by_slot(n, rows, self.c.kv, heads // self.c.kv, self.share or n, self.ints[2].shape[1], self.window)
        super().call()


def test_the_rule_on_sizes_is_the_librarys():
    """On both sides of the rule's border for a call: results are those of verify_attn_paged_b8 bit for bit where the rule
    hands it the call, and the groups' sums meet in another order, with other roundings, where not."""
    kv, group, share, n = 2, 8, 8, 16
    c = Cache(80, [700 + 9 * b for b in range(n)], kv, "e4m3")
    _fork(c, 2, share, 640)
    border = next(w for w in range(16, 4096) if not slot_by_slot(n, 8, kv, group, share, w, 0))
    same = []
    for width in (border - 1, border):
        s = Shared(c, [8] * n, 8, group, share, width=width)
        s.ints[2] = s.ints[2][:, :width].contiguous()
        s.call()
        ws = torch.empty(va.va_paged_workspace_bytes(n, 8, kv, group), dtype=torch.uint8, device="cuda")
        out, lse = torch.empty_like(s.out), torch.empty_like(s.lse)
        va.verify_attn_paged_b8(s.qd, *s.ints, *s.dev, SCALE, s.sd, ws, out, lse)
        same.append(torch.equal(out, s.out) and torch.equal(lse, s.lse))
        s.check()
    assert same == [True, False]


# (slots, share, rows, KV heads, group): few pairs a slot, and many
SIZES = [(8, 4, 2, 1, 3), (16, 8, 8, 1, 8), (6, 3, 4, 3, 6)]


def _live(n, rows):
    return [rows - (3 * b) % rows for b in range(n)]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("sink", [True, False])
@pytest.mark.parametrize("n,share,rows,kv,group", SIZES)
def test_pages_that_are_none(fmt, sink, n, share, rows, kv, group):
    c = Cache(81, [760 + 37 * b for b in range(n)], kv, fmt)
    _fork(c, n // share, share, 704)                             # eleven shared pages
    for b in range(share):
        c.table[b][2] = c.table[b][3] = -1                       # a whole tile of the shared ones
        c.table[b][5], c.table[b][10] = c.pages, 10 ** 8         # one page of a tile, the last one
    c.table[share][11] = -7                                      # of a slot's own
    c.table[share + 1][11] = c.table[share + 1][12] = c.pages + 3
    s = Split(c, _live(n, rows), rows, group, share, sink=sink)
    s.call()
    s.check(status=128)


@pytest.mark.parametrize("sink", [True, False])
def test_slots_that_see_no_page(sink):
    """Every visible page of a slot, or of a whole group, is none."""
    c = Cache(82, [330, 340, 350, 360, 330, 340, 350, 360], 2, "e4m3")
    _fork(c, 2, 4, 320)
    for b in range(4):
        c.table[b] = [-1] * len(c.table[b])
    c.table[5] = [c.pages + b for b in range(len(c.table[5]))]
    s = Split(c, [4, 1, 0, 3, 2, 4, 1, 1], 4, 6, 4, sink=sink)
    s.call()
    s.check(status=128)
    dark = [0, 1, 3, 5]
    assert (s.out[dark] == 0).all()


@pytest.mark.parametrize("share,fmt,own,window,sink", [
    (12, "int8", False, 400, True), (12, "int8", True, 520, False), (12, "int8", False, 700, False), (12, "e4m3", True, 400, True),
    (0, "int8", False, 400, False), (0, "int8", True, 520, True), (0, "int8", False, 700, True), (0, "e4m3", False, 520, False)])
def test_short_windows(share, fmt, own, window, sink):
    """Windows that begin inside what is shared for some slots and, shorter than their own pages, behind it for others.  Entries
    below every window of a group are no page, or those below a slot's own window (of which the group then shares less)."""
    n, kv = 48, 8
    lens, live = [650 + 23 * b for b in range(n)], [(8, 1, 0, 5)[b % 4] for b in range(n)]
    c = Cache(83, lens, kv, fmt)
    _fork(c, n // (share or n), share or n, 640)
    below = [max(0, length - r - window + 1) // 64 for length, r in zip(lens, live)]
    for b in range(n):
        first = b - b % (share or n)
        mine = [below[j] for j in range(first, first + (share or n)) if live[j]]
        for x in range(below[b] if own and b % 3 == 0 else min(mine)):
            c.table[b][x] = -1
    s = Split(c, live, 8, 8, share, window=window, sink=sink, width=0)
    s.call()
    s.check()


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("sink", [True, False])
@pytest.mark.parametrize("lens,live,rows,kv,group,share,prefix", [
    ([90, 200, 33, 0], [4, 4, 2, 0], 4, 2, 6, 0, 0),            # nothing in common
    ([3000, 2000, 700, 64], [8, 3, 8, 1], 8, 1, 8, 1, 0),        # groups of one
    ([130, 140], [8, 7], 8, 1, 8, 2, 128),
    ([64, 65, 66, 63], [1, 1, 1, 1], 1, 1, 6, 4, 64),            # the prefix's page ends with a row's own key
    ([300, 280, 350, 300, 70, 71, 333, 290], [2, 0, 3, 1, 3, 0, 0, 0], 3, 2, 4, 4, 256),
    ([500] * 12, [8] * 12, 8, 1, 8, 12, 448),                    # more than 256 pairs
    ([1, 1, 1, 1], [1, 1, 1, 1], 1, 1, 1, 4, 0),
    ([129] * 4, [1] * 4, 1, 3, 8, 4, 128),                       # one key behind what is shared
    ([192] * 4, [1] * 4, 1, 3, 8, 4, 192),                       # all is shared
])
def test_groups(fmt, sink, lens, live, rows, kv, group, share, prefix):
    c = Cache(84, lens, kv, fmt)
    _fork(c, len(lens) // (share or len(lens)), share or len(lens), prefix)
    s = Split(c, live, rows, group, share, sink=sink)
    s.call()
    s.check()


def test_a_page_more_than_once():
    """The same page twice in a slot's table, and the same slot twice in a group."""
    c = Cache(85, [500, 500, 480, 500], 2, "int8")
    _fork(c, 1, 4, 384)
    for b in range(4):
        c.table[b][2] = c.table[b][1]
    c.table[1] = list(c.table[0])
    c.table[3][6] = c.table[3][0]
    s = Split(c, [4, 4, 1, 2], 4, 8, 4)
    s.call()
    s.check()


def test_a_first_slot_of_a_group_without_rows():
    """Rows of the table of slots without live rows hold anything, the group's first among them."""
    c = Cache(86, [400, 420, 410, 430, 400, 390], 2, "e4m3")
    _fork(c, 2, 3, 384)
    for b in (0, 4):
        c.table[b] = [10 ** 9] * len(c.table[b])
    s = Split(c, [0, 8, 3, 8, 0, 1], 8, 8, 3)
    s.call()
    s.check()


def test_is_verify_attention():
    c = Cache(87, [900 + 50 * b for b in range(16)], 2, "e4m3")
    _fork(c, 4, 4, 832)
    s = Split(c, _live(16, 8), 8, 8, 4)
    s.call()
    ws = torch.empty(va.va_paged_workspace_bytes(16, 8, 2, 8), dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(s.out), torch.empty_like(s.lse)
    va.verify_attn_paged_b8(s.qd, *s.ints, *s.dev, SCALE, s.sd, ws, out, lse)
    torch.testing.assert_close(s.out.float(), out.float(), rtol=2.0 ** -7, atol=2.0 ** -9)
    torch.testing.assert_close(s.lse, lse, rtol=0, atol=1e-4)


def test_two_calls_at_once_on_two_streams():
    calls = []
    for i, (n, share, rows, kv, group) in enumerate(SIZES + SIZES[:1]):
        c = Cache(88 + i, [900 + 31 * b for b in range(n)], kv, ("e4m3", "int8")[i % 2])
        _fork(c, n // share, share, 832)
        calls.append(Split(c, _live(n, rows), rows, group, share, seed=i))
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(5):
        for x, s in zip(calls, streams):
            with torch.cuda.stream(s):
                x.call()
    torch.cuda.synchronize()
    for x in calls:
        x.check()


@pytest.mark.parametrize("n,share,rows,kv,group", SIZES)
def test_captured_and_replayed_with_other_groups(n, share, rows, kv, group):
    """One graph, replayed behind changes of lengths, live rows, tables and queries on the device."""
    width = 4096
    cases = []
    for i, prefix in enumerate((704, 0, 320, 704)):
        c = Cache(91, [760 + 37 * ((b + i) % n) for b in range(n)], kv, "e4m3")
        _fork(c, n // share, share, prefix)
        live = _live(n, rows) if i != 3 else [0] * n
        cases.append(Split(c, live, rows, group, share, seed=i, width=width))
    s = Split(cases[0].c, cases[0].live, rows, group, share, width=width)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.call()
        with torch.cuda.graph(graph, stream=side):
            s.call()
    torch.cuda.synchronize()
    for x in cases + cases[:2]:
        for to, new in zip([*s.ints, *s.dev, s.qd, s.sd], [*x.ints, *x.dev, x.qd, x.sd]):
            assert to.shape == new.shape
            to.copy_(new)
        s.out.fill_(7.0), s.lse.fill_(7.0)
        graph.replay()
        torch.cuda.synchronize()
        x.out, x.lse, x.status = s.out, s.lse, s.status
        x.check()
