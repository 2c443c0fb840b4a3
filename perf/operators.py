"""Cases of the operators over a paged 8-bit K/V cache that many sequences share, and their plain forms.

  append  new K/V rows coded into the pages, one scale per 16 tokens and head
  attn    verify attention of every sequence's live rows over its pages
  step    the pages of one beam step: hypotheses take their parents' pages, then room for one token each
  compact live pages moved to the lowest page numbers
  beam    the best hypotheses over beams x vocabulary

``run`` computes the plain forms with elementary torch operations where ``own`` is false and calls the
library where it is true.  ``exact`` computes the definitions again, in 64 bits.
"""
import math

import numpy as np
import torch

own = False

PAGE, BLOCK, D = 64, 16, 128
TOP = {"e4m3": 448.0, "int8": 127.0}


# ------------------------------------------------------------------------------------------------ cases
def listed():
    return [
        # four short chats on one rank of a tensor-parallel model (one KV head, six query heads), one token each:
        # the smallest decode call, where latency counts
        dict(name="attn decode 4x1K", op="attn", fmt="e4m3", seqs=4, kv_heads=1, group=6, rows=1, min_len=900,
             max_len=1024, window=0, beams=1, sink=True),
        # a decode batch on one GPU with ragged histories from one token to 16K, eight KV heads
        dict(name="attn decode 64x16K", op="attn", fmt="e4m3", seqs=64, kv_heads=8, group=6, rows=1, min_len=1,
             max_len=16384, window=0, beams=1, sink=False),
        # verification of up to eight rows over one 192K history (48 matrix rows share every key)
        dict(name="attn verify 192K", op="attn", fmt="e4m3", seqs=1, kv_heads=1, group=6, rows=8, min_len=196608,
             max_len=196608, window=0, beams=1, sink=True),
        # sliding-window layers (window 4,096) of a batch that verifies five rows each, INT8 codes
        dict(name="attn window 32x40K int8", op="attn", fmt="int8", seqs=32, kv_heads=2, group=6, rows=5,
             min_len=700, max_len=40000, window=4096, beams=1, sink=True),
        # eight hypotheses of each of eight requests: the pages of a prefix are shared
        dict(name="attn beams 8x8x4K int8", op="attn", fmt="int8", seqs=64, kv_heads=4, group=4, rows=1,
             min_len=1500, max_len=4101, window=0, beams=8, sink=False),
        # a whole 16K prompt coded into empty pages
        dict(name="append prompt 16K", op="append", fmt="e4m3", seqs=1, kv_heads=8, rows=16384, min_len=16384,
             max_len=16384, layers=1),
        # a verify step's rows for a batch: they start in the middle of a block, whose older rows are there
        dict(name="append rows 64x6 int8", op="append", fmt="int8", seqs=64, kv_heads=8, rows=6, min_len=70,
             max_len=1000, layers=1),
        # one request, four hypotheses: the next step's pages
        dict(name="step 1x4", op="step", fmt="e4m3", groups=1, beams=4, kv_heads=2, layers=2, min_len=1000,
             max_len=1000),
        # 32 requests of eight hypotheses, four layers
        dict(name="step 32x8", op="step", fmt="int8", groups=32, beams=8, kv_heads=2, layers=4, min_len=300,
             max_len=4000),
        # a pool left with holes by requests that ended
        dict(name="compact 4096 pages", op="compact", fmt="e4m3", pages=4096, live=1500, seqs=24, kv_heads=2,
             layers=4),
        # one request with four beams over the 160,000-token vocabulary
        dict(name="beam 1x4x160000", op="beam", dtype="float32", groups=1, beams=4, vocab=160000, out=4),
        # 32 requests of eight beams, bf16 logits of an odd vocabulary in padded rows, twice as many candidates
        dict(name="beam 32x8x151669 bf16", op="beam", dtype="bfloat16", groups=32, beams=8, vocab=151669, out=16),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["attn", "attn", "attn", "append", "step", "compact", "beam"])
    fmt = rng.choice(["e4m3", "int8"])
    if op == "attn":
        beams = rng.choice([1, 1, 1, 2, 5])
        seqs = beams * _log(rng, 1, 64 // beams)
        kv = rng.choice([1, 2, 3, 8])
        most = min(200000, 64 * 8 * 16384 // (seqs * kv) // 4)
        top = _log(rng, 64, most)
        return dict(op=op, fmt=fmt, seqs=seqs, kv_heads=kv, group=rng.randint(1, 8), rows=rng.randint(1, 8),
                    min_len=_log(rng, 1, top), max_len=top, window=rng.choice([0, 0, _log(rng, 1, 8192)]),
                    beams=beams, sink=rng.random() < 0.5)
    if op == "append":
        seqs, kv = _log(rng, 1, 64), rng.choice([1, 2, 3, 8])
        rows = _log(rng, 1, 16384 * 8 // (seqs * kv))
        low = _log(rng, 1, 2000)
        return dict(op=op, fmt=fmt, seqs=seqs, kv_heads=kv, rows=rows, min_len=rows + low,
                    max_len=rows + low + rng.randint(0, 500), layers=1)
    if op == "step":
        beams = rng.randint(2, 8)
        top = _log(rng, 40, 4000)
        return dict(op=op, fmt=fmt, groups=_log(rng, 1, 32), beams=beams, kv_heads=rng.choice([1, 2]),
                    layers=rng.randint(1, 4), min_len=_log(rng, 1, top), max_len=top)
    if op == "compact":
        pages = _log(rng, 64, 4096)
        return dict(op=op, fmt=fmt, pages=pages, live=_log(rng, 8, pages // 2), seqs=_log(rng, 1, 40),
                    kv_heads=rng.choice([1, 2]), layers=rng.randint(1, 4))
    beams = rng.randint(1, 8)
    return dict(op=op, dtype=rng.choice(["float32", "bfloat16"]), groups=_log(rng, 1, 20), beams=beams,
                vocab=_log(rng, 100, 160000), out=rng.randint(beams, 2 * beams))


# ------------------------------------------------------------------------------------------------ sizes of a case
def _spread(n, lo, hi):
    """n lengths from lo to hi, spread over their logarithm; the first is hi."""
    return [hi if i == 0 else max(lo, min(hi, int(round(lo * (hi / lo) ** ((i * 0.6180339887) % 1.0)))))
            for i in range(n)]


def _lens(case):
    n = case["seqs"]
    lens = _spread(n, case["min_len"], case["max_len"])
    live = [min(lens[i], case["rows"] - (i * 3) % case["rows"]) for i in range(n)]
    if case["op"] == "attn" and case["beams"] > 1:   # the hypotheses of a request are equally long
        lens = [lens[i - i % case["beams"]] for i in range(n)]
        live = [live[i - i % case["beams"]] for i in range(n)]
    return lens, live


def _extent(case, n, live):
    lo = max(0, n - live - case["window"] + 1) if case["window"] else 0
    return n - lo if live else 0


def _step_sizes(case):
    lens = _spread(case["groups"], case["min_len"], case["max_len"])
    parents = [(j * 5) // 8 for j in range(case["beams"])]     # some parents have several children, some none
    return lens, parents


def work(case):
    op = case["op"]
    if op == "attn":
        lens, live = _lens(case)
        heads, m = case["kv_heads"], case["group"]
        seen = 0
        for i, n in enumerate(lens):
            if i % case["beams"] == 0:
                seen += _extent(case, n, live[i])
            else:     # the pages of its own
                seen += min(_extent(case, n, live[i]), PAGE + n % PAGE)
        rows = sum(live)
        pairs = sum(_extent(case, n, r) * r for n, r in zip(lens, live))
        return {"bytes": seen * heads * (2 * D + 8 / BLOCK) + rows * heads * m * (4 * D + 4),
                "flops": 4.0 * D * heads * m * pairs}
    if op == "append":
        lens, live = _lens(case)
        n = sum(live) * case["kv_heads"] * D * 2
        return {"bytes": 3.0 * n, "flops": 4.0 * n}
    if op == "step":
        lens, parents = _step_sizes(case)
        page = case["layers"] * case["kv_heads"] * 2 * (PAGE * D + 4 * PAGE // BLOCK)
        copies = sum((case["beams"] - len(set(parents))) for n in lens if n % PAGE)
        table = 4 * sum(-(-n // PAGE) for n in lens) * case["beams"]
        return {"bytes": 2.0 * copies * page + 4.0 * table, "flops": 0.0}
    if op == "compact":
        page = case["layers"] * case["kv_heads"] * 2 * (PAGE * D + 4 * PAGE // BLOCK)
        moved = case["live"] * (1 - case["live"] / case["pages"])   # live pages are spread evenly
        return {"bytes": 2.0 * moved * page + 8.0 * case["pages"], "flops": 0.0}
    n = case["groups"] * case["beams"] * case["vocab"]
    return {"bytes": n * (4.0 if case["dtype"] == "float32" else 2.0), "flops": 3.0 * n}


# ------------------------------------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _code(x, top, fmt):
    """Blocks [..., 16, 128] float32 to codes (bytes) and one scale each."""
    scale = x.abs().amax((-1, -2)) / torch.full((), top, device=x.device)
    return _round(x / torch.where(scale > 0, scale, 1.0)[..., None, None], fmt), scale


def _round(x, fmt):
    if fmt == "int8":
        return x.round().clamp(-127, 127).to(torch.int8).view(torch.uint8)
    return x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _value(codes, fmt):
    return (codes.view(torch.int8) if fmt == "int8" else codes.view(torch.float8_e4m3fn)).to(torch.float32)


def _view(codes, fmt):
    return codes.view(torch.int8) if fmt == "int8" else codes.view(torch.float8_e4m3fn)


def _pool(case, n_pages, g):
    """Pages full of coded N(0, 1) rows, some keys four times as large: codes [layers, pages, heads, 64, 128]."""
    layers, heads, fmt = case.get("layers", 1), case["kv_heads"], case["fmt"]
    out = []
    for which in range(2):
        codes = torch.empty(layers * n_pages, heads, PAGE, D, dtype=torch.uint8, device="cuda")
        scale = torch.empty(layers * n_pages, heads, PAGE // BLOCK, device="cuda")
        for a in range(0, codes.shape[0], 4096):
            n = min(4096, codes.shape[0] - a)
            x = torch.randn(n, heads, PAGE // BLOCK, BLOCK, D, generator=g, device="cuda")
            if which == 0:
                x *= 1 + 3 * (torch.rand(n, heads, PAGE // BLOCK, BLOCK, 1, generator=g, device="cuda") < 0.05)
            c, s = _code(x, TOP[fmt], fmt)
            codes[a:a + n] = c.reshape(n, heads, PAGE, D)
            scale[a:a + n] = s
        out += [codes.view(layers, n_pages, heads, PAGE, D), scale.view(layers, n_pages, heads, PAGE // BLOCK)]
    return {"k_codes": out[0], "k_scale": out[1], "v_codes": out[2], "v_scale": out[3]}


def _ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _tables(pages_of, width, n_pages, g):
    """Page numbers of each row's pages (lists of labels) as a table of shuffled page numbers."""
    where = torch.randperm(n_pages, generator=g, device="cuda").tolist()
    rows = [[where[p] for p in r] + [-1] * (width - len(r)) for r in pages_of]
    refs = [0] * n_pages
    for r in pages_of:
        for p in r:
            refs[where[p]] += 1
    return _ints(rows), _ints(refs)


def _prepare_attn(case, g):
    lens, live = _lens(case)
    pages_of, n_pages = [], 0
    for i, n in enumerate(lens):
        need, first = -(-n // PAGE), i - i % case["beams"]
        shared = pages_of[first][:max(0, need - 2)] if i != first else []
        own_pages = need - len(shared)
        pages_of.append(shared + list(range(n_pages, n_pages + own_pages)))
        n_pages += own_pages
    s = _pool(case, n_pages + 3, g)
    s = {k: v[0] for k, v in s.items()}
    s["table"], s["refs"] = _tables(pages_of, max(len(p) for p in pages_of) + 1, n_pages + 3, g)
    heads = case["kv_heads"] * case["group"]
    s["q"] = torch.randn(case["seqs"], case["rows"], heads, D, generator=g, device="cuda").to(torch.bfloat16)
    s["sink"] = torch.randn(heads, generator=g, device="cuda") if case["sink"] else None
    s["lens"], s["live"] = _ints(lens), _ints(live)
    s["out"] = torch.empty_like(s["q"])
    s["lse"] = torch.empty(case["seqs"], case["rows"], heads, device="cuda")
    s["max_len"] = max(lens)
    return s


def _prepare_append(case, g):
    lens, live = _lens(case)
    need = [-(-n // PAGE) for n in lens]
    first = [sum(need[:i]) for i in range(len(need))]
    n_pages = sum(need) + 2
    s = _pool(case, n_pages, g)
    s = {k: v[0] for k, v in s.items()}
    s["table"], s["refs"] = _tables([list(range(a, a + n)) for a, n in zip(first, need)], max(need), n_pages, g)
    shape = (case["seqs"], case["rows"], case["kv_heads"], D)
    s["k_new"] = torch.randn(shape, generator=g, device="cuda").mul_(1.5).to(torch.bfloat16)
    s["v_new"] = torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)
    s["lens"], s["live"] = _ints(lens), _ints(live)
    s["blocks"] = (case["rows"] + 2 * BLOCK - 2) // BLOCK
    return s


def _prepare_step(case, g):
    lens, kinds = _step_sizes(case)
    beams, pages_of, n_pages = case["beams"], [], 0
    for n in lens:
        need = -(-n // PAGE)
        shared = list(range(n_pages, n_pages + max(0, need - 3)))
        n_pages += len(shared)
        for _ in range(beams):
            mine = need - len(shared)
            pages_of.append(shared + list(range(n_pages, n_pages + mine)))
            n_pages += mine
    total = n_pages + 2 * len(pages_of)
    s = _pool(case, total, g)
    s["table0"], s["refs0"] = _tables(pages_of, max(len(p) for p in pages_of) + 2, total, g)
    s["lens0"] = _ints([n for n in lens for _ in range(beams)])
    order = torch.rand(case["groups"], beams, generator=g, device="cuda").argsort(1)
    s["parents"] = order[:, kinds].to(torch.int32).reshape(-1).contiguous()
    s["one"] = torch.ones_like(s["lens0"])
    for k in ("table", "refs", "lens"):
        s[k] = s[k + "0"].clone()
    s["status"] = _ints([0])
    return s


def _prepare_compact(case, g):
    total, live, seqs = case["pages"], case["live"], case["seqs"]
    s = _pool(case, total, g)
    ids = torch.randperm(total, generator=g, device="cuda")[:live].tolist()
    rows = [ids[i::seqs] for i in range(seqs)]
    for i in range(1, seqs):                       # a sequence shares the first pages of the one before
        rows[i] = rows[i - 1][:len(rows[i - 1]) // 3] + rows[i]
    refs = [0] * total
    for r in rows:
        for p in r:
            refs[p] += 1
    width = max(len(r) for r in rows)
    s["table0"], s["refs0"] = _ints([r + [-1] * (width - len(r)) for r in rows]), _ints(refs)
    s["table"], s["refs"] = s["table0"].clone(), s["refs0"].clone()
    s["moved_to"], s["n_live"] = torch.empty_like(s["refs"]), _ints([0])
    return s


def _prepare_beam(case, g):
    rows, vocab = case["groups"] * case["beams"], case["vocab"]
    wide = -(-vocab // 8) * 8
    dt = getattr(torch, case["dtype"])
    logits = torch.empty(rows, wide, dtype=dt, device="cuda")
    for a in range(0, rows, 64):
        logits[a:a + 64] = (torch.randn(min(64, rows - a), wide, generator=g, device="cuda") * 2.5).to(dt)
    s = {"logits": logits[:, :vocab]}
    s["scores"] = -torch.rand(rows, generator=g, device="cuda") * 6 - 10
    s["finished"] = (torch.rand(rows, generator=g, device="cuda") < 0.15).to(torch.int32)
    shape = (case["groups"], case["out"])
    s["parents"], s["tokens"] = (torch.empty(shape, dtype=torch.int32, device="cuda") for _ in range(2))
    s["out_scores"] = torch.empty(shape, device="cuda")
    return s


def prepare(case, seed):
    s = globals()["_prepare_" + case["op"]](case, _gen(seed))
    s["case"] = dict(case)
    return s


# ------------------------------------------------------------------------------------------------ plain forms
def _plain_attn(s):
    c = s["case"]
    b, r, h, m, dev = c["seqs"], c["rows"], c["kv_heads"], c["group"], s["q"].device
    n_pages = -(-s["max_len"] // PAGE)
    ids = s["table"][:, :n_pages].clamp(min=0).long()

    def dense(codes, scale):
        x = _value(codes[ids], c["fmt"]).view(b, n_pages, h, PAGE // BLOCK, BLOCK, D)
        return (x * scale[ids][..., None, None]).transpose(1, 2).reshape(b, h, n_pages * PAGE, D)

    q = s["q"].float().view(b, r, h, m, D).transpose(1, 2).reshape(b, h, r * m, D)
    score = (q @ dense(s["k_codes"], s["k_scale"]).transpose(-1, -2)) * D ** -0.5
    row = torch.arange(r, device=dev)
    at = (s["lens"] - s["live"])[:, None] + row                                        # positions [b, r]
    key = torch.arange(n_pages * PAGE, device=dev)
    seen = (key <= at[..., None]) & (row < s["live"][:, None])[..., None]              # [b, r, keys]
    if c["window"]:
        seen &= key > at[..., None] - c["window"]
    seen = seen[:, None, :, None].expand(b, 1, r, m, key.numel()).reshape(b, 1, r * m, key.numel())
    score = torch.where(seen, score, -math.inf)
    sink = torch.full((h, m), -math.inf, device=dev) if s["sink"] is None else s["sink"].view(h, m)
    sink = sink[:, None].expand(h, r, m).reshape(1, h, r * m)
    real = (row < s["live"][:, None])[:, None, :, None].expand(b, h, r, m).reshape(b, h, r * m)
    top = torch.where(real, torch.maximum(score.amax(-1), sink), 0.0)
    p = torch.exp(score - top[..., None])
    total = p.sum(-1) + torch.exp(sink - top)
    out = (p @ dense(s["v_codes"], s["v_scale"])) / torch.where(real, total, 1.0)[..., None]
    lse = torch.where(real, top + total.log(), -math.inf)

    def back(x):
        return x.view(b, h, r, m, *x.shape[3:]).transpose(1, 2).reshape(b, r, h * m, *x.shape[3:])

    return back(out).to(torch.bfloat16), back(lse)


def _plain_append(s):
    c = s["case"]
    b, h, dev, fmt = c["seqs"], c["kv_heads"], s["lens"].device, c["fmt"]
    start = s["lens"] - s["live"]
    block = start[:, None] // BLOCK + torch.arange(s["blocks"], device=dev)            # [b, blocks]
    at = block[..., None] * BLOCK + torch.arange(BLOCK, device=dev)                    # [b, blocks, 16]
    new = (at >= start[:, None, None]) & (at < s["lens"][:, None, None])
    old = at < start[:, None, None]
    page = torch.gather(s["table"], 1, (block // (PAGE // BLOCK)).clamp(max=s["table"].shape[1] - 1).long()).long()
    part = (block % (PAGE // BLOCK)).long()
    take = (at - start[:, None, None]).clamp(0, c["rows"] - 1).long()
    seq = torch.arange(b, device=dev)[:, None, None]
    some = new.any(-1)
    out = []
    for name in ("k", "v"):
        codes, scale = s[name + "_codes"], s[name + "_scale"]
        x = s[name + "_new"][seq, take].float().transpose(2, 3)                         # [b, blocks, h, 16, D]
        held = codes.view(*codes.shape[:2], PAGE // BLOCK, BLOCK, D)[page, :, part]     # [b, blocks, h, 16, D]
        was = scale[page, :, part]                                                      # [b, blocks, h]
        is_new, is_old = new[:, :, None, :, None], old[:, :, None, :, None]
        fresh = torch.where(is_new, x, 0.0).abs().amax((-1, -2)) / torch.full((), TOP[fmt], device=dev)
        now = torch.where(old.any(-1)[..., None], torch.maximum(fresh, was), fresh)
        by = torch.where(now > 0, now, 1.0)[..., None, None]
        again = _round(_value(held, fmt) * was[..., None, None] / by, fmt)
        held = torch.where(is_old & (now > was)[..., None, None], again, held)
        held = torch.where(is_new, _round(x / by, fmt), held)
        codes.view(*codes.shape[:2], PAGE // BLOCK, BLOCK, D)[page[some], :, part[some]] = held[some]
        scale[page[some], :, part[some]] = now[some]
        out += [_view(codes, fmt), scale]
    return out


def _plain_step(s):
    c = s["case"]
    table, refs, lens, n = s["table"], s["refs"], s["lens"], s["refs"].numel()
    table.copy_(s["table0"]), refs.copy_(s["refs0"]), lens.copy_(s["lens0"])
    slot = torch.arange(lens.numel(), device=lens.device)
    src = slot // c["beams"] * c["beams"] + s["parents"].long()
    taken = table[src]

    def count(t):
        return torch.bincount(t[t >= 0], minlength=n).to(torch.int32)

    refs += count(taken) - count(table)
    table.copy_(taken), lens.copy_(lens[src])
    # room for one more token: the pages that will be written are there and are nobody else's
    col = torch.arange(table.shape[1], device=lens.device)
    written = (col >= (lens // PAGE)[:, None]) & (col < (-(-(lens + s["one"]) // PAGE))[:, None])
    page = table.long().clamp(min=0)
    held = written & (table >= 0)
    holders = torch.bincount(page[held], minlength=n)
    order = torch.arange(table.numel(), device=lens.device).view_as(table)
    first = torch.full((n,), table.numel(), device=lens.device).scatter_reduce(0, page[held], order[held], "amin")
    shared = held & (refs[page] > 1) & ~((holders[page] == refs[page]) & (first[page] == order))
    fresh = written & (shared | (table < 0))
    ids = (refs == 0).nonzero().view(-1)
    ids = ids[torch.arange(fresh.sum(), device=lens.device)]
    begun = shared & (col * PAGE < lens[:, None])
    from_, to = page[begun], torch.empty_like(page).masked_scatter_(fresh, ids)[begun]
    refs -= torch.bincount(page[shared], minlength=n).to(torch.int32)
    refs[ids] = 1
    table[fresh] = ids.to(torch.int32)
    lens += s["one"]
    for name in ("k_codes", "k_scale", "v_codes", "v_scale"):
        s[name][:, to] = s[name][:, from_]
    return [table, refs, lens] + [_view(s["k_codes"], c["fmt"]), s["k_scale"], _view(s["v_codes"], c["fmt"]), s["v_scale"]]


def _plain_compact(s):
    c = s["case"]
    table, refs = s["table"], s["refs"]
    table.copy_(s["table0"]), refs.copy_(s["refs0"])
    number = torch.arange(refs.numel(), device=refs.device)
    live = refs > 0
    n = live.sum()
    movers, holes = number[live & (number >= n)], number[~live & (number < n)]
    to = torch.where(live, number, -1).to(torch.int32)
    to[movers] = holes.to(torch.int32)
    for name in ("k_codes", "k_scale", "v_codes", "v_scale"):
        s[name][:, holes] = s[name][:, movers]
    refs[holes] = refs[movers]
    refs[movers] = 0
    table.copy_(torch.where(table >= 0, to[table.clamp(min=0).long()], -1))
    s["moved_to"].copy_(to), s["n_live"].copy_(n)
    return [table, refs, s["moved_to"], s["n_live"], _view(s["k_codes"], c["fmt"]), s["k_scale"],
            _view(s["v_codes"], c["fmt"]), s["v_scale"]]


def _plain_beam(s):
    c = s["case"]
    g, beams, vocab = c["groups"], c["beams"], c["vocab"]
    x = s["logits"].double()        # candidates of different beams lie close together: 64 bits
    top = x.amax(-1, keepdim=True)
    score = s["scores"].double()[:, None] + (x - top - (x - top).exp().sum(-1, keepdim=True).log())
    token = torch.arange(vocab, device=x.device)
    ended = torch.where(token == 2, s["scores"].double()[:, None], -math.inf)
    score = torch.where(s["finished"][:, None] > 0, ended, score)
    best, at = score.view(g, beams * vocab).sort(dim=-1, descending=True, stable=True)
    best, at = best[:, :c["out"]], at[:, :c["out"]]
    none = best == -math.inf
    parents, tokens = torch.where(none, -1, at // vocab), torch.where(none, -1, at % vocab)
    return parents.to(torch.int32), tokens.to(torch.int32), best.to(torch.float32)


# ------------------------------------------------------------------------------------------------ the library's calls
def _own_attn(s):
    import speculative_decode_verify_gb300 as va
    c = s["case"]
    if "workspace" not in s:
        s["workspace"] = torch.zeros(va.va_paged_workspace_bytes(c["seqs"], c["rows"], c["kv_heads"], c["group"]),
                                     dtype=torch.uint8, device="cuda")
    va.verify_attn_paged_b8(s["q"], s["live"], s["lens"], s["table"], _view(s["k_codes"], c["fmt"]),
                            _view(s["v_codes"], c["fmt"]), s["k_scale"], s["v_scale"], D ** -0.5, s["sink"],
                            s["workspace"], s["out"], s["lse"], window=c["window"])
    return s["out"], s["lse"]


def _own_append(s):
    import speculative_decode_verify_gb300 as va
    k, v = _view(s["k_codes"], s["case"]["fmt"]), _view(s["v_codes"], s["case"]["fmt"])
    va.kv_page_append_b8(s["k_new"], s["v_new"], s["live"], s["lens"], s["table"], k, v, s["k_scale"], s["v_scale"])
    return [k, s["k_scale"], v, s["v_scale"]]


def _workspace(s, va):
    if "workspace" not in s:
        s["workspace"] = torch.zeros(va.va_page_ops_workspace_bytes(*s["table"].shape, s["refs"].numel()),
                                     dtype=torch.uint8, device="cuda")
    return s["workspace"]


def _own_step(s):
    import speculative_decode_verify_gb300 as va
    c = s["case"]
    k, v = _view(s["k_codes"], c["fmt"]), _view(s["v_codes"], c["fmt"])
    table, refs, lens = s["table"], s["refs"], s["lens"]
    table.copy_(s["table0"]), refs.copy_(s["refs0"]), lens.copy_(s["lens0"])
    va.kv_page_reorder(table, lens, s["parents"], refs, group=c["beams"])
    va.kv_page_extend(table, lens, s["one"], refs, k, v, s["k_scale"], s["v_scale"], _workspace(s, va))
    return [table, refs, lens, k, s["k_scale"], v, s["v_scale"]]


def _own_compact(s):
    import speculative_decode_verify_gb300 as va
    k, v = _view(s["k_codes"], s["case"]["fmt"]), _view(s["v_codes"], s["case"]["fmt"])
    table, refs = s["table"], s["refs"]
    table.copy_(s["table0"]), refs.copy_(s["refs0"])
    va.kv_page_compact(table, refs, k, v, s["k_scale"], s["v_scale"], s["moved_to"], s["n_live"], _workspace(s, va))
    return [table, refs, s["moved_to"], s["n_live"], k, s["k_scale"], v, s["v_scale"]]


def _own_beam(s):
    import speculative_decode_verify_gb300 as va
    c = s["case"]
    if "workspace" not in s:
        s["workspace"] = torch.zeros(va.va_beam_workspace_bytes(c["groups"], c["beams"], c["vocab"], c["out"]),
                                     dtype=torch.uint8, device="cuda")
    va.va_beam_select(s["logits"], s["scores"], c["beams"], s["parents"], s["tokens"], s["out_scores"], s["workspace"],
                      finished=s["finished"], end_token=2)
    return s["parents"], s["tokens"], s["out_scores"]


def run(state):
    return globals()[("_own_" if own else "_plain_") + state["case"]["op"]](state)


# ------------------------------------------------------------------------------------------------ definitions, 64 bits
def _exact_attn(case, s):
    h, m, r = case["kv_heads"], case["group"], case["rows"]
    lens, live = _lens(case)
    out = torch.zeros(case["seqs"], r, h * m, D, dtype=torch.float64, device="cuda")
    lse = torch.full((case["seqs"], r, h * m), -math.inf, dtype=torch.float64, device="cuda")
    table = s["table"].tolist()
    for b, n in enumerate(lens):
        ids = torch.tensor(table[b][:-(-n // PAGE)], device="cuda")
        kv = []
        for w in "kv":
            x = s[w + "_codes"][ids]
            x = x.view(torch.int8) if case["fmt"] == "int8" else x.view(torch.float8_e4m3fn)
            x = x.double() * s[w + "_scale"][ids].double().repeat_interleave(BLOCK, -1)[..., None]
            kv.append(x.permute(1, 0, 2, 3).reshape(h, -1, D)[:, :n])
        for i in range(live[b]):
            p = n - live[b] + i
            lo = max(0, p - case["window"] + 1) if case["window"] else 0
            q = s["q"][b, i].double().view(h, m, D)
            z = torch.einsum("hmd,hnd->hmn", q, kv[0][:, lo:p + 1]) / math.sqrt(D)
            if s["sink"] is not None:
                z = torch.cat([z, s["sink"].double().view(h, m, 1)], -1)
            total = torch.logsumexp(z, -1)
            w = torch.exp(z[..., :p + 1 - lo] - total[..., None])
            out[b, i] = torch.einsum("hmn,hnd->hmd", w, kv[1][:, lo:p + 1]).reshape(h * m, D)
            lse[b, i] = total.reshape(-1)
    return out, lse


def _grid(fmt):
    """The values that a code can stand for, ascending."""
    if fmt == "int8":
        return np.arange(-127, 128, dtype=np.float64)
    half = [m / 8 * 2.0 ** -6 for m in range(8)] + [(1 + m / 8) * 2.0 ** e for e in range(-6, 9) for m in range(8)]
    half = half[:-1]                                    # the last is no number
    return np.array([-v for v in half[:0:-1]] + half)


def _nearest(x, fmt):
    """The grid's value nearest to x; of two equally near ones, the one with the even code."""
    grid = _grid(fmt)
    zero = int(np.searchsorted(grid, 0.0))
    i = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    lo, hi = x - grid[i - 1], grid[i] - x
    up = (hi < lo) | ((hi == lo) & ((i - zero) % 2 == 0))
    return grid[np.where(up, i, i - 1)]


def _exact_append(case, s):
    if case["seqs"] * case["rows"] * case["kv_heads"] > 140000:
        return None
    lens, live = _lens(case)
    fmt, top, table = case["fmt"], TOP[case["fmt"]], s["table"].tolist()
    out = []
    for w in "kv":
        codes = s[w + "_codes"]
        value = (codes.view(torch.int8) if fmt == "int8" else codes.view(torch.float8_e4m3fn)).double().cpu().numpy()
        scale = s[w + "_scale"].double().cpu().numpy()
        rows = s[w + "_new"].double().cpu().numpy()
        for b, n in enumerate(lens):
            start = n - live[b]
            for a in range(start - start % BLOCK, n, BLOCK):
                page, part = table[b][a // PAGE], a % PAGE // BLOCK
                lo, hi = max(a, start), min(a + BLOCK, n)
                x = rows[b, lo - start:hi - start].transpose(1, 0, 2)
                now = (np.abs(x).max((1, 2)) / top).astype(np.float32).astype(np.float64)
                if lo > a:
                    was = scale[page, :, part].copy()
                    now = np.maximum(now, was)
                    held = value[page, :, a % PAGE:a % PAGE + lo - a]
                    back = (held * was[:, None, None]).astype(np.float32).astype(np.float64)
                    back = _nearest((back / np.where(now > 0, now, 1)[:, None, None]).astype(np.float32).astype(np.float64), fmt)
                    value[page, :, a % PAGE:a % PAGE + lo - a] = np.where((now > was)[:, None, None], back, held)
                quotient = (x / np.where(now > 0, now, 1)[:, None, None]).astype(np.float32).astype(np.float64)
                value[page, :, lo % PAGE:lo % PAGE + hi - lo] = _nearest(quotient, fmt)
                scale[page, :, part] = now
        out += [None if fmt == "int8" else value, scale]
    return out


def _exact_beam(case, s):
    scores, done = s["scores"].double().cpu().numpy(), s["finished"].cpu().numpy()
    best = []
    for row in range(case["groups"] * case["beams"]):
        if done[row]:
            best.append(np.array([scores[row]]))
            continue
        x = s["logits"][row].double().cpu().numpy()
        top = np.sort(x)[::-1][:case["out"]]
        best.append(scores[row] + top - (x.max() + math.log(math.fsum(np.exp(x - x.max())))))
    out = np.full((case["groups"], case["out"]), -np.inf)
    for g in range(case["groups"]):
        every = np.sort(np.concatenate(best[g * case["beams"]:(g + 1) * case["beams"]]))[::-1][:case["out"]]
        out[g, :len(every)] = every
    return None, None, out


def exact(case, seed):
    """The outputs that are computed numbers, in 64 bits; pages and whole numbers have no such value."""
    if case["op"] not in ("attn", "append", "beam"):
        return None
    return globals()["_exact_" + case["op"]](case, prepare(case, seed))
