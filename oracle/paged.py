"""CPU oracle of the paged 8-bit cache: its coding, verify attention over it, the operations on its pages, and beam
search's selection.  TEST INFRASTRUCTURE, NOT PRODUCT CODE (same rules as the rest of ``oracle/``).

Attention and selection are computed in float64 from the definitions.  Where float32 decides a code (the scale, the
product of an older code with its scale, the quotient) the oracle takes the same float32 operations, so codes and
scales must match bit for bit.  The page operations are plain sequential programs over Python integers.
"""
from __future__ import annotations

import math

import numpy as np

from .kv_codec import e4m3_decode, e4m3_encode_bits

__all__ = ["PAGE", "BLOCK", "TOP", "decode", "encode", "append", "attention", "reorder", "extend", "compact",
           "beam_select"]

PAGE, BLOCK, D = 64, 16, 128
TOP = {"e4m3": np.float32(448.0), "int8": np.float32(127.0)}


def decode(codes, fmt):
    """Codes (bytes) to the float32 values that they stand for, scale apart."""
    if fmt == "int8":
        return np.asarray(codes).view(np.int8).astype(np.float32)
    return e4m3_decode(np.asarray(codes).view(np.uint8)).astype(np.float32)


def encode(x, fmt):
    """float32 quotients to codes: nearest, ties to even, the largest code past the range."""
    if fmt == "int8":
        return np.clip(np.rint(x), -127, 127).astype(np.int8).view(np.uint8)
    return e4m3_encode_bits(np.asarray(x, np.float32)).astype(np.uint8)


def append(new, start, end, table_row, codes, scale, fmt):
    """One sequence's rows ``new`` [rows, heads, 128] (float32; infinities and NaN allowed) to positions start..end-1
    of ``codes`` [pages, heads, 64, 128] (bytes) and ``scale`` [pages, heads, 4], in place."""
    with np.errstate(all="ignore"):
        for a in range(start - start % BLOCK, end, BLOCK):
            page, part = int(table_row[a // PAGE]), a % PAGE // BLOCK
            lo, hi = max(a, start), min(a + BLOCK, end)
            for h in range(codes.shape[1]):
                x = np.asarray(new[lo - start:hi - start, h], np.float32)
                x = np.where(np.isnan(x), np.float32(0), x)
                finite = np.abs(x[np.isfinite(x)])
                s = np.float32(finite.max() if finite.size else 0) / TOP[fmt]
                row = codes[page, h]
                if lo > a:
                    was = scale[page, h, part]
                    if s > was:
                        at = slice(a % PAGE, a % PAGE + lo - a)
                        row[at] = encode((decode(row[at], fmt) * was).astype(np.float32) / s, fmt)
                    s = max(s, was)
                at = slice(lo % PAGE, lo % PAGE + hi - lo)
                row[at] = encode(x / s, fmt) if s > 0 else 0
                scale[page, h, part] = s


def attention(q, live, lens, table, k_codes, v_codes, k_scale, v_scale, fmt, scale, sink=None, window=0):
    """q [n_seqs, n_rows, heads, 128] float64 -> (out, lse, size, reach, top): the output, the log-sum-exp, per element
    sum_j w_j |v_j|, per row max_j scale sum_d |q_d k_jd| and the number of keys times the largest value that a
    code of the sequence's values could stand for (what a kernel's error bounds are made of)."""
    n, rows, heads, _ = q.shape
    kv = k_codes.shape[1]
    g = heads // kv
    out, size = np.zeros(q.shape), np.zeros(q.shape)
    lse, reach, top_v = np.full(q.shape[:3], -np.inf), np.zeros(q.shape[:3]), np.zeros(q.shape[:3])
    for b in range(n):
        for r in range(int(live[b])):
            p = int(lens[b]) - int(live[b]) + r
            lo = max(0, p - window + 1) if window else 0
            js = [j for j in range(lo, p + 1) if 0 <= table[b][j // PAGE] < k_codes.shape[0]]
            pg, of = np.array([int(table[b][j // PAGE]) for j in js], int), np.array([j % PAGE for j in js], int)
            for h in range(kv):
                k = decode(k_codes[pg, h, of], fmt).astype(np.float64) * k_scale[pg, h, of // BLOCK, None].astype(np.float64)
                v = decode(v_codes[pg, h, of], fmt).astype(np.float64) * v_scale[pg, h, of // BLOCK, None].astype(np.float64)
                every = {int(table[b][x]) for x in range(-(-int(lens[b]) // PAGE))} & set(range(k_codes.shape[0]))
                largest = max([float(np.nanmax(v_scale[list(every), h]))] if every else [0.0]) * float(TOP[fmt])
                for m in range(h * g, (h + 1) * g):
                    top_v[b, r, m] = len(js) * largest
                    s = scale * (k @ q[b, r, m])
                    z = s if sink is None else np.append(s, float(sink[m]))
                    if not z.size or z.max() == -np.inf:
                        continue
                    top = z.max()
                    total = top + math.log(np.exp(z - top).sum())
                    w = np.exp(s - total)
                    out[b, r, m], size[b, r, m], lse[b, r, m] = w @ v, w @ np.abs(v), total
                    reach[b, r, m] = abs(scale) * (np.abs(k) @ np.abs(q[b, r, m])).max() if js else 0.0
    return out, lse, size, reach, top_v


def reorder(table, lens, refs, src, group=0):
    n = len(lens)
    group = group or n
    old, old_lens = [list(r) for r in table], list(lens)
    for j in range(n):
        s = -1 if src[j] < 0 else j // group * group + int(src[j])
        new = [-1] * len(old[j]) if s < 0 else old[s]
        for p in old[j]:
            if p >= 0:
                refs[p] -= 1
        for p in new:
            if p >= 0:
                refs[p] += 1
        table[j], lens[j] = list(new), 0 if s < 0 else old_lens[s]


def extend(table, lens, refs, n_new):
    """Returns the copies [(from, to)], or None if there are not enough free pages (nothing is changed then)."""
    written = [(b, x) for b in range(len(lens)) if n_new[b] > 0
               for x in range(lens[b] // PAGE, -(-(lens[b] + n_new[b]) // PAGE))]
    holders = {}
    for b, x in written:
        if table[b][x] >= 0:
            holders.setdefault(table[b][x], []).append((b, x))
    keeps = {e[0] for p, e in holders.items() if len(e) == refs[p]}
    wanting = [(b, x) for b, x in written if table[b][x] < 0 or (b, x) not in keeps]
    free = [p for p in range(len(refs)) if refs[p] == 0][:len(wanting)]
    if len(free) < len(wanting):
        return None
    copies = []
    for (b, x), page in zip(wanting, free):
        p = table[b][x]
        if p >= 0:
            refs[p] -= 1
            if x * PAGE < lens[b]:
                copies.append((p, page))
        table[b][x] = page
        refs[page] = 1
    for b in range(len(lens)):
        lens[b] += n_new[b]
    return copies


def compact(table, refs):
    """Returns (moved_to, number of live pages, moves)."""
    live = [p for p in range(len(refs)) if refs[p] > 0]
    n = len(live)
    moves = list(zip([p for p in live if p >= n], [p for p in range(n) if refs[p] <= 0]))
    to = [p if refs[p] > 0 else -1 for p in range(len(refs))]
    for a, b in moves:
        to[a], refs[b], refs[a] = b, refs[a], 0
    for row in table:
        for x, p in enumerate(row):
            if p >= 0:
                row[x] = to[p]
    return to, n, moves


def beam_select(logits, scores, n_beams, n_out, finished=None, end_token=0):
    """logits [rows, vocab] float64 -> (parents, tokens, scores [groups, n_out] float64, gap): gap is the smallest
    distance between neighbouring scores of different hypotheses around the selection."""
    rows = logits.shape[0]
    parents = np.full((rows // n_beams, n_out), -1, np.int64)
    tokens, best = parents.copy(), np.full(parents.shape, -np.inf)
    gap = np.inf
    with np.errstate(all="ignore"):
        for g in range(rows // n_beams):
            cand = []
            for i in range(n_beams):
                row = g * n_beams + i
                if finished is not None and finished[row]:
                    cand.append((float(scores[row]), i, 0, end_token))
                    continue
                l = np.where(np.isnan(logits[row]), -np.inf, logits[row])
                top = l.max()
                if top == -np.inf:
                    continue
                above = np.where(l == top, 0.0, l - top)
                log_sum = math.log(np.exp(above).sum())
                order = np.argsort(-l, kind="stable")[:n_out]
                cand += [(float(scores[row]) + (above[t] - log_sum), i, j, int(t)) for j, t in enumerate(order)]
            cand = [c for c in cand if c[0] > -np.inf]
            cand.sort(key=lambda c: (-c[0], c[1], c[2]))
            for a, b in zip(cand[:n_out], cand[1:n_out + 1]):
                if a[1] != b[1] and a[0] != b[0]:
                    gap = min(gap, a[0] - b[0])
            for r, c in enumerate(cand[:n_out]):
                parents[g, r], tokens[g, r], best[g, r] = c[1], c[3], c[0]
    return parents, tokens, best, gap
