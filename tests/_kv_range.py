"""Bounds for the attention over a cache whose weights or scales span far more
than a fp16 number does: as _kv_cache.attend_bounds, but for what is lost of
weights below fp16's normal numbers."""

import numpy as np
import torch

from _kv_cache import HALF
from oracle import kv_cache as okv

TINY = 2.0 ** -109    # value scales below it count as 0
NO_VALUE = 2.0 ** -80   # what counts as the scale of a vector of zeros


def bounds(c, q, scale, out_dtype):
    """(out, lse, bound of |out|'s error, bound of lse's), rows that see nothing
    aside, for queries q (fp64 [rows, n_q, d]) over the Cache c.

    Scores, exponentials, sums and the output's rounding as in attend_bounds.  A
    weight is rounded to fp16 where the largest is 2^11 or more, so that it loses
    2^-11 of itself, or 2^-25 · 2^-11 = 2^-36 of the largest where it is
    subnormal: over E4M3 codes with the values' scales multiplied in, of which
    those of zeros count as 2^-80."""
    rows, n_q, d = q.shape
    group = n_q // c.n_kv
    out, lse = np.zeros((rows, n_q, d)), np.full((rows, n_q), -np.inf)
    e_out, e_lse = np.zeros_like(out), np.zeros_like(lse)
    u = 2.0 ** -22
    for row, i, p in okv.tokens(c.lens, rows):
        for g in range(c.n_kv):
            ks, vs = (okv.sequence(x, c.table, i, p + 1)[:, g]
                      for x in c.values)
            s = np.ones(p + 1)
            if c.kind == "e4m3":
                s = okv.sequence(c.cache[3].cpu().double().numpy(), c.table, i,
                                 p + 1)[:, g]
            nothing = (s < TINY) | ((s == 1) & ~vs.any(axis=1)
                                    if c.kind == "e4m3" else False)
            s = np.where(nothing, NO_VALUE, s)
            vs = np.where(nothing[:, None], 0.0, vs)
            for h in range(g * group, (g + 1) * group):
                x = scale * (ks @ q[row, h])
                top = x.max()
                w = np.exp(x - top)
                total = w.sum()
                o = w @ vs / total
                out[row, h], lse[row, h] = o, top + np.log(total)
                t = x + np.log(s)
                e_x = (d + 4) * u * abs(scale) * \
                    (np.abs(ks) @ np.abs(q[row, h])).max() + \
                    3 * u * max(np.abs(x).max(), np.abs(t).max())
                spread = w @ np.abs(vs) / total
                e = spread * (2 * e_x + 2 * u + (p + 9) * u + (
                    2.0 ** -16 if c.kind == "bf16" else 2.0 ** -11))
                if c.kind != "bf16":
                    e += 2.0 ** -36 * (w * s).max() / total * \
                        (np.abs(vs) / s[:, None]).sum(axis=0)
                e_out[row, h] = e + HALF[out_dtype] * (np.abs(o) + e) + \
                    (2.0 ** -25 if out_dtype == torch.float16 else 0.0)
                e_lse[row, h] = e_x + (p + 9) * u + 2 * u * abs(lse[row, h])
    return out, lse, e_out, e_lse


def agree(got, gl, want, seen=slice(None)):
    """The device's out and lse within `want`'s bounds, in rows `seen`."""
    out, lse, e_out, e_lse = (x[seen] for x in want)
    got = got.double().cpu().numpy()[seen]
    gl = gl.double().cpu().numpy()[seen]
    worst = np.abs(got - out) / np.maximum(e_out, 1e-300)
    assert (worst <= 1).all(), f"out: {worst.max():.2f} of the bound"
    worst = np.abs(gl - lse) / e_lse
    assert (worst <= 1).all(), f"lse: {worst.max():.2f} of the bound"
