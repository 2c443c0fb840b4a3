"""Operations on pages against the oracle's sequential programs, and whole runs of the paged cache's calls."""
import numpy as np
import pytest
import torch

import oracle.paged as P
import speculative_decode_verify_gb300 as va
from paged_cases import Cache, attention_bounds, bf16, ints

pytestmark = pytest.mark.gpu
D = 128


class Pool:
    """Device state with every page's bytes telling pages apart, and the oracle's copy of it."""

    def __init__(self, seed, table, lens, pages, layers=2, kv=2):
        self.table, self.lens, self.pages = [list(r) for r in table], list(lens), pages
        self.refs = [0] * pages
        for row in self.table:
            for p in row:
                if p >= 0:
                    self.refs[p] += 1
        rng = np.random.default_rng(seed)
        self.host = [rng.integers(0, 256, (layers, pages, kv, 64, D), dtype=np.uint8) for _ in "kv"]
        self.host += [rng.standard_normal((layers, pages, kv, 4)).astype(np.float32) for _ in "kv"]
        self.dev = [torch.as_tensor(a.copy()).cuda() for a in self.host]
        self.t, self.n, self.r = ints(self.table), ints(self.lens), ints(self.refs)
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")
        self.ws = torch.full((va.va_page_ops_workspace_bytes(len(lens), len(table[0]), pages),), 0xA5,
                             dtype=torch.uint8, device="cuda")

    def moved(self, pairs):
        pairs = list(pairs)
        for a in self.host:
            for s, d in pairs:
                a[:, d] = a[:, s]

    def extend(self, new):
        va.kv_page_extend(self.t, self.n, ints(new), self.r, *self.dev, self.ws, dev_status=self.status)
        copies = P.extend(self.table, self.lens, self.refs, new)
        if copies is not None:
            self.moved(copies)
        return copies

    def reorder(self, src, group=0):
        va.kv_page_reorder(self.t, self.n, ints(src), self.r, group=group, dev_status=self.status)
        P.reorder(self.table, self.lens, self.refs, src, group)

    def compact(self):
        to, n = torch.full((self.pages,), -9, dtype=torch.int32, device="cuda"), ints([-9])
        va.kv_page_compact(self.t, self.r, *self.dev, to, n, self.ws, dev_status=self.status)
        want, live, moves = P.compact(self.table, self.refs)
        self.moved(moves)
        assert to.tolist() == want and n.tolist() == [live]

    def check(self, status=0):
        assert int(self.status.item()) == status
        assert self.t.tolist() == self.table and self.n.tolist() == self.lens and self.r.tolist() == self.refs
        for a, b in zip(self.dev, self.host):
            np.testing.assert_array_equal(a.cpu().numpy().view(np.uint8), b.view(np.uint8))


@pytest.mark.parametrize("slots,group,width,pages,seed", [(1, 1, 3, 4, 1), (6, 3, 9, 60, 2), (40, 8, 5, 300, 3),
                                                          (300, 5, 4, 1500, 4), (1024, 1024, 2, 2100, 5)])
def test_random_runs(slots, group, width, pages, seed):
    rng = np.random.default_rng(seed)
    s = Pool(seed, [[-1] * width for _ in range(slots)], [0] * slots, pages, layers=1 if slots > 100 else 2)
    for step in range(12):
        room = [width * 64 - n for n in s.lens]
        s.extend([int(min(r, rng.integers(0, 90))) if rng.random() < 0.8 else 0 for r in room])
        s.check(int(s.status.item()) & 256)                     # short of pages: nothing has changed
        s.status.zero_()
        s.reorder([int(x) for x in rng.integers(-1, group, slots)], group)
        s.check()
        if step % 3 == 2:
            s.compact()
            s.check()
        back = [max(0, n - int(rng.integers(0, 70))) if rng.random() < 0.3 else n for n in s.lens]   # rejected drafts
        s.lens = back
        s.n.copy_(ints(back))


def test_copy_on_write_keeps_the_last_holder_in_place():
    # slots 0-2 share a page begun, slot 3 shares a full one, slot 4's page is its own
    s = Pool(7, [[5, -1], [5, -1], [5, -1], [2, -1], [3, 2]], [10, 10, 10, 64, 70], 9)
    s.extend([1, 0, 1, 1, 1])                                    # slot 1 holds page 5 outside the call
    assert s.table == [[0, -1], [5, -1], [1, -1], [2, 4], [3, 6]]
    s.check()
    s.reorder([0, 1, 0, 3, 1])
    s.extend([1, 1, 1, 0, 1])                                    # all holders of 0 and of 5 write: the lowest keep
    s.check()
    assert s.table[0][0] == 0 and s.table[1][0] == 5


def test_too_few_pages_changes_nothing():
    s = Pool(8, [[0, -1, -1], [1, -1, -1]], [64, 10], 4)
    assert s.extend([100, 60]) is None
    s.check(256)
    s.status.zero_()
    assert s.extend([128, 0]) == []
    s.check()


@pytest.mark.parametrize("slots,new,free", [(4, 150, [5, 16383, 16384, 16385, 20000, 32767, 32768, 39990, 39991, 39998, 39999, 12]),
                                            (3, 25000, list(range(100, 36000, 30))),
                                            (1024, 64, [0] + list(range(20000, 22000)))])
def test_free_pages_far_into_a_large_pool(slots, new, free):
    pages, width = 40000, 400
    refs = np.ones(pages, np.int32)
    refs[free] = 0
    table = np.full((slots, width), -1, np.int32)
    codes = torch.zeros(pages, 1, 64, D, dtype=torch.uint8, device="cuda")
    scale = torch.zeros(pages, 1, 4, device="cuda")
    t, r, n, status = ints(table.tolist()), ints(refs.tolist()), ints([0] * slots), ints([0])
    ws = torch.empty(va.va_page_ops_workspace_bytes(slots, width, pages), dtype=torch.uint8, device="cuda")
    va.kv_page_extend(t, n, ints([new] * slots), r, codes, codes, scale, scale, ws, dev_status=status)
    table, refs, lens = table.tolist(), refs.tolist(), [0] * slots
    assert P.extend(table, lens, refs, [new] * slots) == [] and int(status.item()) == 0
    assert t.tolist() == table and r.tolist() == refs and n.tolist() == lens


def test_every_slot_shares_one_page():
    s = Pool(12, [[7, -1]] * 900, [3] * 900, 1000)
    s.extend([1] * 900)
    s.check()
    s = Pool(13, [[7, -1]] * 900, [3] * 900, 1000)
    s.extend([0, 0] + [1] * 898)
    s.check()


@pytest.mark.parametrize("change,bit", [("negative", 1024), ("long", 4), ("page", 128), ("free", 128), ("length", 1024)])
def test_extend_refuses_and_changes_nothing(change, bit):
    s = Pool(9, [[0, 1], [2, -1]], [70, 20], 6)
    new = [3, 5]
    if change == "negative":
        new[1] = -1
    elif change == "long":
        new[1] = 109
    elif change == "length":
        s.lens[1] = -5
        s.n.copy_(ints(s.lens))
    else:
        s.table[1][0] = 6 if change == "page" else 4             # no page, and a page that is free
        s.t.copy_(ints(s.table))
    va.kv_page_extend(s.t, s.n, ints(new), s.r, *s.dev, s.ws, dev_status=s.status)
    s.check(bit)


def test_reorder_tells_of_wrong_sources_and_entries():
    s = Pool(10, [[0, 1], [2, -1], [3, -1], [4, -1]], [70, 20, 9, 9], 6)
    va.kv_page_reorder(s.t, s.n, ints([2, -2, 1, 1]), s.r, group=2, dev_status=s.status)
    P.reorder(s.table, s.lens, s.refs, [0, 1, 1, 1], 2)
    s.check(1024)
    s.status.zero_()
    s.table[0][0] = 77
    s.t.copy_(ints(s.table))
    va.kv_page_reorder(s.t, s.n, ints([0, 0, -1, 1]), s.r, group=2, dev_status=s.status)
    assert int(s.status.item()) == 128
    assert s.t.tolist() == [[77, 1], [77, 1], [-1, -1], [4, -1]] and s.r.tolist()[1:5] == [2, 0, 0, 1]


def test_copy():
    s = Pool(11, [[0]], [1], 70, layers=3)
    src, dst = list(range(0, 60, 3)), list(range(1, 61, 3))
    va.kv_page_copy(ints(src), ints(dst), *s.dev, dev_status=s.status)
    s.moved(zip(src, dst))
    s.check()
    va.kv_page_copy(ints([0, 70, -1, 3]), ints([2, 5, 8, 71]), *s.dev, dev_status=s.status)
    s.moved([(0, 2)])
    s.check(128)


@pytest.mark.parametrize("pages,live", [(1, 1), (33, 0), (33, 33), (1000, 17), (70000, 40), (40000, 39990)])
def test_compaction_of_any_filling(pages, live):
    rng = np.random.default_rng(pages)
    ids = [int(p) for p in rng.permutation(pages)[:live]]
    width = max(1, -(-live // 7))
    table = [(ids[i * width:(i + 1) * width] + [-1] * width)[:width] for i in range(8)]
    refs = ints([0] * pages)
    host = [0] * pages
    for row in table:
        for p in row:
            if p >= 0:
                host[p] += 1
    refs.copy_(ints(host))
    codes = torch.randint(0, 256, (pages, 1, 64, D), dtype=torch.uint8, device="cuda")
    codes2, sc, sc2 = codes.flip(0).contiguous(), torch.rand(pages, 1, 4, device="cuda"), torch.rand(pages, 1, 4, device="cuda")
    want_c, want_s = codes.clone(), sc2.clone()
    to, n = torch.zeros(pages, dtype=torch.int32, device="cuda"), ints([0])
    ws = torch.empty(va.va_page_ops_workspace_bytes(8, width, pages), dtype=torch.uint8, device="cuda")
    t, status = ints(table), ints([0])
    va.kv_page_compact(t, refs, codes, codes2, sc, sc2, to, n, ws, dev_status=status)
    moved_to, count, moves = P.compact(table, host)
    if moves:
        a, b = (torch.tensor(x, device="cuda") for x in zip(*moves))
        want_c[b], want_s[b] = want_c[a], want_s[a]
    assert int(status.item()) == 0 and n.tolist() == [count] and to.tolist() == moved_to
    assert t.tolist() == table and refs.tolist() == host
    assert torch.equal(codes, want_c) and torch.equal(sc2, want_s)


# ------------------------------------------------------------------------------------------------ runs
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_beam_search_over_the_paged_cache(fmt):
    """Prompts of two requests, then steps of three hypotheses each: extend, append, attention, selection, reorder.
    Every hypothesis keeps a cache of its own in the oracle (one pool each, nothing shared)."""
    requests, beams, kv, group, vocab, steps = 2, 3, 2, 3, 500, 70
    slots, rng = requests * beams, np.random.default_rng(5)
    pages, width = 40, 5
    t = {"uint8" if fmt == "e4m3" else "int8": torch.uint8 if fmt == "e4m3" else torch.int8}.popitem()[1]
    pool = [torch.zeros(pages, kv, 64, D, dtype=t, device="cuda") for _ in "kv"]
    pool += [torch.zeros(pages, kv, 4, device="cuda") for _ in "kv"]
    table, lens, refs = ints([[-1] * width] * slots), ints([0] * slots), ints([0] * pages)
    ws_p = torch.empty(va.va_page_ops_workspace_bytes(slots, width, pages), dtype=torch.uint8, device="cuda")
    ws_a = torch.zeros(va.va_paged_workspace_bytes(slots, 1, kv, group), dtype=torch.uint8, device="cuda")
    ws_b = torch.zeros(va.va_beam_workspace_bytes(requests, beams, vocab, beams), dtype=torch.uint8, device="cuda")
    status = ints([0])
    codes = lambda: {w: np.zeros((width, kv, 64, D), np.uint8) for w in "kv"}   # noqa: E731
    scales = lambda: {w: np.zeros((width, kv, 4), np.float32) for w in "kv"}    # noqa: E731
    own = [(codes(), scales(), 0) for _ in range(slots)]

    def put(new_k, new_v, live):
        va.kv_page_append_b8(new_k[0].cuda(), new_v[0].cuda(), ints(live), lens, table, *pool, dev_status=status)
        for b in range(slots):
            c, s, n = own[b]
            for w, x in (("k", new_k), ("v", new_v)):
                if live[b]:
                    P.append(x[1][b].astype(np.float32), n, n + live[b], list(range(width)), c[w], s[w], fmt)
            own[b] = (c, s, n + live[b])

    # the prompts go to the first slot of each request, which the others fork
    prompt = [75, 0, 0, 20, 0, 0]
    va.kv_page_extend(table, lens, ints(prompt), refs, *pool, ws_p, dev_status=status)
    put(bf16(rng.standard_normal((slots, 75, kv, D))), bf16(rng.standard_normal((slots, 75, kv, D))), prompt)
    src = [0] * slots
    scores, out_scores = torch.tensor([0.0, -np.inf, -np.inf] * requests, device="cuda"), torch.zeros(requests, beams, device="cuda")
    parents, tokens = (torch.zeros(requests, beams, dtype=torch.int32, device="cuda") for _ in range(2))
    for step in range(steps):
        va.kv_page_reorder(table, lens, ints(src) if step == 0 else parents.view(-1), refs, group=beams, dev_status=status)
        took = src if step == 0 else parents.view(-1).tolist()
        olds = own
        own = [({w: olds[b // beams * beams + took[b]][0][w].copy() for w in "kv"},
                {w: olds[b // beams * beams + took[b]][1][w].copy() for w in "kv"},
                olds[b // beams * beams + took[b]][2]) for b in range(slots)]
        va.kv_page_extend(table, lens, ints([1] * slots), refs, *pool, ws_p, dev_status=status)
        put(bf16(rng.standard_normal((slots, 1, kv, D))), bf16(rng.standard_normal((slots, 1, kv, D))), [1] * slots)
        if step % 23 == 0:
            qt, qn = bf16(rng.standard_normal((slots, 1, kv * group, D)))
            out, lse = torch.zeros(qt.shape, dtype=torch.bfloat16, device="cuda"), torch.zeros(qt.shape[:3], device="cuda")
            va.verify_attn_paged_b8(qt.cuda(), ints([1] * slots), lens, table, *pool, D ** -0.5, None, ws_a, out, lse,
                                    dev_status=status)
            for b in range(slots):
                c, s, n = own[b]
                assert n == int(lens[b])
                want = P.attention(qn[b:b + 1], [1], [n], [list(range(width))], c["k"], c["v"], s["k"], s["v"], fmt, D ** -0.5)
                tol, tol_lse = attention_bounds(*want)
                assert np.all(np.abs(out[b:b + 1].double().cpu().numpy() - want[0]) <= tol)
                assert np.all(np.abs(lse[b:b + 1].double().cpu().numpy() - want[1]) <= tol_lse)
        logits = torch.as_tensor(rng.standard_normal((slots, vocab)).astype(np.float32) * 2)
        want_p, want_t, want_s, gap = P.beam_select(logits.double().numpy(), scores.tolist(), beams, beams)
        va.va_beam_select(logits.cuda(), scores, beams, parents, tokens, out_scores, ws_b)
        if gap > 1e-5:
            assert parents.tolist() == want_p.tolist() and tokens.tolist() == want_t.tolist()
        scores.copy_(out_scores.view(-1))
    assert int(status.item()) == 0
    live = refs.tolist()
    counted = [0] * pages
    for row in table.tolist():
        for p in row:
            if p >= 0:
                counted[p] += 1
    assert live == counted
    # nothing is left behind once every slot is freed
    va.kv_page_reorder(table, lens, ints([-1] * slots), refs)
    assert refs.tolist() == [0] * pages and lens.tolist() == [0] * slots


def test_a_verify_step_with_rejected_drafts_as_one_graph():
    """extend + append + attention captured once; between replays the lengths go back to what was accepted."""
    kv, group, slots, rows, fmt = 1, 6, 3, 4, "e4m3"
    c = Cache(41, [60, 100, 5], kv, fmt, spare=12)
    pool = c.dev(0)
    table, lens, refs = ints([r + [-1] * 3 for r in c.table]), ints(c.lens), ints(c.refs)
    live, status = ints([rows, rows, 2]), ints([0])
    ws_p = torch.empty(va.va_page_ops_workspace_bytes(slots, table.shape[1], c.pages), dtype=torch.uint8, device="cuda")
    ws_a = torch.zeros(va.va_paged_workspace_bytes(slots, rows, kv, group), dtype=torch.uint8, device="cuda")
    kn, vn = (torch.zeros(slots, rows, kv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    q = torch.zeros(slots, rows, kv * group, D, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        va.kv_page_extend(table, lens, live, refs, *pool, ws_p, dev_status=status)
        va.kv_page_append_b8(kn, vn, live, lens, table, *pool, dev_status=status)
        va.verify_attn_paged_b8(q, live, lens, table, *pool, D ** -0.5, None, ws_a, out, None, dev_status=status)
    rng = np.random.default_rng(8)
    codes, scale, n = {w: c.codes[w][0] for w in "kv"}, {w: c.scale[w][0] for w in "kv"}, list(c.lens)
    for step in range(8):
        new = {w: bf16(rng.standard_normal(kn.shape)) for w in "kv"}
        kn.copy_(new["k"][0])
        vn.copy_(new["v"][0])
        qt, qn = bf16(rng.standard_normal(q.shape))
        q.copy_(qt)
        graph.replay()
        rowsof = table.tolist()
        for b, r in enumerate([rows, rows, 2]):
            for w in "kv":
                P.append(new[w][1][b].astype(np.float32), n[b], n[b] + r, rowsof[b], codes[w], scale[w], fmt)
            n[b] += r
        assert lens.tolist() == n and int(status.item()) == 0
        want = P.attention(qn, [rows, rows, 2], n, rowsof, codes["k"], codes["v"], scale["k"], scale["v"], fmt, D ** -0.5)
        tol, _ = attention_bounds(*want)
        assert np.all(np.abs(out.double().cpu().numpy() - want[0]) <= tol)
        n = [n[0] - step % 4, n[1] - 3, n[2] - 1]
        lens.copy_(ints(n))
