"""Oracle for the key-value cache and the attention over it (numpy).

Test infrastructure: see the package docstring.

Definition (include/tp.h, "key-value cache"): row j of the m new rows of
sequence i is the token at position p = lens[i] − m + j, none where p < 0; it
lies in page table[i][p // page] at p mod page.  A row of queries sees the
tokens t ≤ p of its sequence: out = Σ e^(x_t) v_t / Σ e^(x_t) with
x_t = scale·q·k_t, 0 where it sees nothing, and lse = ln Σ e^(x_t).

Pins: tests/test_kv_cache_host.py.
"""

import numpy as np

from . import fp8_block
from .fp8 import e4m3_decode


def tokens(lens, rows, start=None):
    """(row, sequence, position) of each row that is a token."""
    b = len(lens)
    if start is None:
        start = np.arange(b + 1) * (rows // b)
    for i in range(b):
        for row in range(start[i], start[i + 1]):
            p = int(lens[i]) - (int(start[i + 1]) - row)
            if p >= 0:
                yield row, i, p


def quantize(x):
    """(codes, scales) of vectors [..., d], a scale for each."""
    flat = np.ascontiguousarray(x, np.float32).reshape(-1, x.shape[-1])
    q, s = fp8_block.quantize(flat, "row")
    return q.reshape(x.shape), s[0].reshape(x.shape[:-1])


def dequantize(codes, scales):
    return e4m3_decode(codes) * np.asarray(scales, np.float64)[..., None]


def sequence(pool, table, i, n):
    """The first n tokens of sequence i, [n, n_kv, ...], of a pool
    [pages, page, n_kv, ...]."""
    page = pool.shape[1]
    t = np.arange(n)
    return pool[table[i][t // page], t % page]


def attend(q, k, v, table, lens, scale):
    """(out [rows, n_q, d], lse [rows, n_q]) of q over pools of values."""
    rows, n_q, d = q.shape
    group = n_q // k.shape[2]
    out = np.zeros((rows, n_q, d))
    lse = np.full((rows, n_q), -np.inf)
    for row, i, p in tokens(lens, rows):
        ks, vs = (sequence(x, table, i, p + 1) for x in (k, v))
        for h in range(n_q):
            x = scale * (ks[:, h // group] @ q[row, h])
            top = x.max()
            w = np.exp(x - top)
            out[row, h] = w @ vs[:, h // group] / w.sum()
            lse[row, h] = top + np.log(w.sum())
    return out, lse


def step(x, r, gamma, W, pools, table, lens, n_q, d, eps):
    """A generation step's attention block (residual + RMSNorm, block-scaled
    projections, cache and attention), each step's stored tensor rounded as the
    device stores it.  W: Wq, Wk, Wv, Wo; pools: k and v as values
    [pages, page, n_kv, d], written in place, and whether the cache holds E4M3
    codes."""
    from .fp8 import round_bf16
    from .norm import rmsnorm_forward
    k_pool, v_pool, quantized = pools

    def deq(v, group):
        return fp8_block.dequantize(*fp8_block.quantize(v, group))

    x1 = round_bf16(x if r is None else x + r)
    y = deq(rmsnorm_forward(x1, gamma, eps)["y"], "row")
    rows, n_kv = x.shape[0], k_pool.shape[2]
    q, k, v = (round_bf16(y @ deq(W[w], "block").T).reshape(rows, -1, d)
               for w in ("Wq", "Wk", "Wv"))
    assert k.shape[1] == n_kv and q.shape[1] == n_q
    page = k_pool.shape[1]
    for row, i, p in tokens(lens, rows):
        at = table[i][p // page], p % page
        for pool, new in ((k_pool, k), (v_pool, v)):
            pool[at] = dequantize(*quantize(new[row])) if quantized \
                else new[row]
    o, _ = attend(q, k_pool, v_pool, table, lens, d ** -0.5)
    Z = deq(round_bf16(o.reshape(rows, -1)), "row") @ deq(W["Wo"], "block").T
    return x1, Z
