"""Paged caches for the tests: pools of coded rows, tables of shuffled pages, and the oracle's view of them."""
import numpy as np
import torch

import oracle.paged as P

D = P.D


def bf16(x):
    """float32 values rounded to bfloat16 (torch tensor) and the same values as float64 (numpy)."""
    t = torch.as_tensor(np.asarray(x, np.float32)).to(torch.bfloat16)
    return t, t.double().numpy()


class Cache:
    """Sequences of the given lengths in a pool whose unused places hold NaN codes (E4M3) or the largest code (INT8)
    and NaN scales; page numbers are shuffled and the table has a column more than the longest needs."""

    def __init__(self, seed, lens, kv, fmt, spare=3, layers=1, spread=1.0):
        self.rng = np.random.default_rng(seed)
        self.fmt, self.kv, self.lens = fmt, kv, [int(n) for n in lens]
        need = [-(-n // P.PAGE) for n in self.lens]
        self.pages = sum(need) + spare
        order = self.rng.permutation(self.pages)
        self.table = [[-1] * (max(need) + 1) for _ in need]
        at = 0
        for b, n in enumerate(need):
            self.table[b][:n] = [int(p) for p in order[at:at + n]]
            at += n
        self.refs = [0] * self.pages
        for row in self.table:
            for p in row:
                if p >= 0:
                    self.refs[p] += 1
        poison = 0x7F
        shape = (layers, self.pages, kv, P.PAGE, D)
        self.codes = {w: np.full(shape, poison, np.uint8) for w in "kv"}
        self.scale = {w: np.full(shape[:3] + (P.PAGE // P.BLOCK,), np.nan, np.float32) for w in "kv"}
        for w in "kv":
            for layer in range(layers):
                for b, n in enumerate(self.lens):
                    if n:
                        x = self.rng.standard_normal((n, kv, D)).astype(np.float32) * spread
                        P.append(x, 0, n, self.table[b], self.codes[w][layer], self.scale[w][layer], fmt)

    def dev(self, layer=None):
        """Pools on the GPU: (k_codes, v_codes, k_scale, v_scale), of one layer or of all."""
        pick = (lambda a: a) if layer is None else (lambda a: a[layer])
        t = torch.int8 if self.fmt == "int8" else torch.uint8
        codes = [torch.as_tensor(pick(self.codes[w]).copy()).view(t).cuda() for w in "kv"]
        return codes + [torch.as_tensor(pick(self.scale[w]).copy()).cuda() for w in "kv"]


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def attention_bounds(out, lse, size, reach, top):
    """Largest error of an output and of a log-sum-exp.  Scores are sums of 128 products in fp32 with a few more
    roundings (at most 140 of 2^-24, relative to sum |q k| scale) and enter an exponential that is 2^-21 exact, in a
    total of fp32 sums; weights are rounded to 11 bits (2^-11 each) before the product with V, which is again
    summed in fp32; the output is rounded once to bf16 (2^-8 relative).  A weight below f16's normal range is rounded to
    2^-25 of its unit; with the largest at 2^6 units or more and R at most twice the largest scale, n keys of codes up
    to the top one are off by n 2^-25 2 (scale x top) / 2^6 = 2^-30 n (scale x top) in all."""
    score = (140 * 2.0 ** -24 * reach + 2.0 ** -20)
    tol_out = 2.0 ** -8 * np.abs(out) + size * (2.0 ** -11 + 2 * score + 2.0 ** -16)[..., None] + 2.0 ** -30 * np.asarray(top)[..., None]
    tol_lse = score + 2.0 ** -22 * np.abs(np.where(np.isfinite(lse), lse, 0.0)) + 2.0 ** -18
    return tol_out, tol_lse
