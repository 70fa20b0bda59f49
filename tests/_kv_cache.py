"""Caches for the tests: values on the CPU, pools on any device in several
memory layouts, everything that is not a token of a sequence NaN."""

import numpy as np
import torch

from oracle import kv_cache as okv

TORCH = {"bf16": torch.bfloat16, "f16": torch.float16,
         "e4m3": torch.float8_e4m3fn}


def rounded(x, dtype):
    return torch.from_numpy(np.ascontiguousarray(x)).to(dtype)


def pool_memory(pages, page, n_kv, d, dtype, layout, device, count=2):
    """``count`` uninitialised pools [pages, page, n_kv, d] of equal strides.
    heads: a head's tokens are neighbours; tokens: a token's heads are; both:
    K and V take turns by pages of one tensor; wide: room behind vectors."""
    tail = () if d is None else (d,)
    kw = dict(dtype=dtype, device=device)
    if layout == "heads":
        return [torch.empty((pages, n_kv, page) + tail, **kw).transpose(1, 2)
                for _ in range(count)]
    if layout == "tokens":
        return [torch.empty((pages, page, n_kv) + tail, **kw)
                for _ in range(count)]
    if layout == "both":
        x = torch.empty((pages, count, page, n_kv) + tail, **kw)
        return [x[:, i] for i in range(count)]
    assert layout == "wide"
    if d is None:
        return [torch.empty((pages, page, 2 * n_kv), **kw)[..., ::2]
                for _ in range(count)]
    return [torch.empty((pages + 1, page, n_kv + 1, d + 16), **kw)
            [1:, :, 1:, :d] for _ in range(count)]


def page_table(lens, page, rng, spare=2):
    """(table [b, cols], pages in the pool): pages in any order, -1 behind a
    sequence's last."""
    need = [-(-max(int(n), 0) // page) for n in lens]
    cols, total = max(max(need), 1), sum(need) + spare
    order = rng.permutation(total)[:sum(need)]
    table = np.full((len(lens), cols), -1, np.int32)
    at = 0
    for i, n in enumerate(need):
        table[i, :n] = order[at:at + n]
        at += n
    return table, total


class Cache:
    """A cache with its lengths; k, v: what the pools stand for (fp64), NaN
    where no sequence has a token; .cache: the pools on the device."""

    def __init__(self, lens, page, n_kv, d, kind, seed, layout="heads",
                 device="cuda", stale="nan", std=1.0):
        rng = self.rng = np.random.default_rng(seed)
        self.lens, self.page, self.n_kv, self.d = list(lens), page, n_kv, d
        self.kind = kind
        self.table, self.pages = page_table(lens, page, rng)
        live = np.zeros((self.pages, page), bool)
        for i, n in enumerate(lens):
            t = np.arange(max(n, 0))
            live[self.table[i][t // page], t % page] = True
        shape = (self.pages, page, n_kv, d)
        pools = pool_memory(*shape, TORCH[kind], layout, device)
        scales = [None, None]
        if kind == "e4m3":
            scales = pool_memory(*shape[:3], None, torch.float32, layout,
                                 device)
        self.values = []
        for pool, scale in zip(pools, scales):
            x = rng.standard_normal(shape).astype(np.float32) * std
            x *= np.exp(0.5 * rng.standard_normal(shape[:3] + (1,)))
            bad = {"nan": np.nan, "inf": np.inf, "-inf": -np.inf,
                   "max": 3e38}[stale]
            if kind == "e4m3":
                codes, s = okv.quantize(x)
                codes[~live] = 0x7f if stale == "nan" else 0x7e
                s[~live] = np.float32(np.inf if stale != "max" else 3e38)
                pool.view(torch.uint8).copy_(torch.from_numpy(codes))
                scale.copy_(torch.from_numpy(s))
                with np.errstate(invalid="ignore", over="ignore"):
                    self.values.append(okv.dequantize(codes, s))
            else:
                x[~live] = bad
                if kind == "f16" and stale == "max":
                    x[~live] = 65504.0
                t = rounded(x, TORCH[kind])
                pool.copy_(t)
                self.values.append(t.double().numpy())
        self.cache = (*pools, *scales)
        self.dev_table = torch.from_numpy(self.table).to(device)
        self.dev_lens = torch.tensor(self.lens, dtype=torch.int32,
                                     device=device)

    @property
    def args(self):
        return self.cache, self.dev_table, self.dev_lens


HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def attend_bounds(c, q, scale, out_dtype):
    """(out, lse, bound of |out|'s error, bound of lse's) for queries q (fp64
    [rows, n_q, d]) over the Cache c.

    A score is a sum of d products in fp32, at worst d + 4 roundings of 2^-22
    each (tensor cores cut rather than round) of Σ|q·k| and three of the score
    itself: e_x.  A weight e^x is then off by the factor e_x and by 2^-21 of
    the exponential's own.  In front of the product with V it is rounded: to
    fp16 (2^-11, or 2^-25 of the largest weight where it is subnormal) over
    fp16 values, and with the value's scale multiplied in over E4M3 codes; to
    two bf16 parts (2^-16) over bf16 values.  Σ w|v| / l is what a relative
    error of the weights can do to the sum.  The sum and its quotient in fp32
    add n + 8 roundings of 2^-22 of the same at most, the output's rounding
    half a step."""
    rows, n_q, d = q.shape
    group = n_q // c.n_kv
    out, lse = np.zeros((rows, n_q, d)), np.full((rows, n_q), -np.inf)
    e_out, e_lse = np.zeros_like(out), np.zeros_like(lse)
    k, v = c.values
    sv = None if c.kind != "e4m3" else c.cache[3].cpu().double().numpy()
    u = 2.0 ** -22
    last, found = None, {}
    for row, i, p in okv.tokens(c.lens, rows):
        if i != last:
            last, n = i, c.lens[i]
            found = [okv.sequence(x, c.table, i, n).swapaxes(0, 1).copy()
                     for x in (k, v)]
            scales = np.ones((c.n_kv, n)) if sv is None else \
                okv.sequence(sv, c.table, i, n).T
        for g in range(c.n_kv):
            ks, vs, s = found[0][g, :p + 1], found[1][g, :p + 1], \
                scales[g, :p + 1]
            heads = slice(g * group, (g + 1) * group)
            qs = q[row, heads].T                       # [d, group]
            x = scale * (ks @ qs)
            top = x.max(axis=0)
            w = np.exp(x - top)
            total = w.sum(axis=0)
            o = w.T @ vs / total[:, None]
            out[row, heads], lse[row, heads] = o, top + np.log(total)
            e_x = (d + 4) * u * abs(scale) * \
                (np.abs(ks) @ np.abs(qs)).max(axis=0) + \
                3 * u * np.abs(x).max(axis=0)
            far = np.abs(vs)
            spread = w.T @ far / total[:, None]
            e_w = e_x + 2 * u + (2.0 ** -16 if c.kind == "bf16"
                                 else 2.0 ** -11)
            e = spread * (e_w + e_x + (p + 9) * u)[:, None]
            if c.kind != "bf16":
                heaviest = (w * s[:, None]).max(axis=0) / total
                e += 2.0 ** -25 * heaviest[:, None] * (far / s[:, None]).sum(0)
            e_out[row, heads] = e + HALF[out_dtype] * (np.abs(o) + e) + \
                (2.0 ** -25 if out_dtype == torch.float16 else 0.0)
            e_lse[row, heads] = e_x + (p + 9) * u + \
                2 * u * np.abs(lse[row, heads])
    return out, lse, e_out, e_lse
