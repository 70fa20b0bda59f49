"""The bounds of _kv_range without a GPU: they come with the definition's values,
the roundings that the kernels make stay within them, and mistakes do not."""

import numpy as np
import pytest
import torch

from _kv_cache import Cache
from _kv_range import NO_VALUE, bounds
from oracle import kv_cache as okv


def one_head(kind, k, v, s=None):
    """A Cache of one sequence and head whose vectors' first elements are k
    (keys, the others 0) and whose values are v·s."""
    n, d = v.shape
    c = Cache([n], 16, 1, d, kind, 5, device="cpu")
    t = np.arange(n)
    at = c.table[0][t // 16], t % 16
    c.values[0][at] = 0.0
    c.values[0][at + (0, 0)] = k
    if s is not None:
        c.cache[3][at + (0,)] = torch.from_numpy(s).float()
        v = v * s[:, None]
    c.values[1][at] = v[:, None]
    return c


def replay(k, v, s, below, skip=None, none=None):
    """Output and log-sum-exp with weights rounded to fp16 at 2^below of the
    largest; `skip`: tokens left out; `none`: what counts as the scale of those
    without a value."""
    live = np.ones(len(k), bool) if skip is None else ~skip
    sv = s if none is None else np.where(none, NO_VALUE, s)
    t = np.where(live, k + np.log(sv), -np.inf)
    w = np.exp(t - t.max()) * 2.0 ** below
    w16 = w.astype(np.float16).astype(np.float64)
    total = (w / sv).sum()
    return w16 @ v / total, np.log(total) + t.max() - below * np.log(2.0)


def holds(c, out, lse):
    want, wl, eo, el = (x[0, 0] for x in bounds(
        c, np.eye(1, c.d)[None], 1.0, torch.bfloat16))
    return bool((np.abs(out - want) <= eo).all() and np.abs(lse - wl) <= el)


def test_bounds_come_with_the_same_attention():
    for kind in ("bf16", "f16", "e4m3"):
        c = Cache([9, 0, 5], 4, 2, 64, kind, 3, device="cpu")
        q = np.random.default_rng(4).standard_normal((6, 6, 64))
        out, lse, eo, el = bounds(c, q, 0.2, torch.bfloat16)
        with np.errstate(invalid="ignore"):
            want, wl = okv.attend(q, *c.values, c.table, c.lens, 0.2)
        assert np.allclose(out, want, rtol=1e-12, atol=1e-14)
        assert np.allclose(lse, wl, rtol=1e-12)
        seen = np.isfinite(lse)
        assert (eo[seen] <= 2.0 ** -8 * np.abs(out[seen]) + 2.0 ** -7).all()
        assert (el[seen] <= 2.0 ** -9).all() and (eo[~seen] == 0).all()


@pytest.mark.parametrize("kind", ["f16", "e4m3"])
def test_a_heavy_token_without_a_value(kind):
    rng, n = np.random.default_rng(6), 400
    v = rng.integers(1, 8, (n, 64)).astype(float)
    s = np.full(n, 2.0 ** -8) if kind == "e4m3" else np.ones(n)
    k = np.where(np.arange(n) == 3, 20.0, 0.0)
    v[3] = 0.0
    c = one_head(kind, k, v, s if kind == "e4m3" else None)
    assert holds(c, *replay(k, v, s, 11))
    # the largest weight at 1: the others' are below fp16's smallest number
    assert not holds(c, *replay(k, v, s, 0))


def test_scales_of_zero_count():
    rng, n = np.random.default_rng(7), 60
    v = rng.integers(1, 8, (n, 64)).astype(float)
    k = rng.standard_normal(n)
    s = rng.uniform(0.01, 0.02, n).astype(np.float32).astype(float)
    zero = np.arange(n) % 3 == 1
    s[zero] = 0.0
    c = one_head("e4m3", k, v, s)
    v[zero] = 0.0
    assert holds(c, *replay(k, v, s, 11, none=zero))
    with np.errstate(divide="ignore", invalid="ignore"):   # left out
        t = np.where(zero, 1.0, s)
        assert not holds(c, *replay(k, v, t, 11, skip=zero))


def test_zeros_beside_small_values():
    rng, n = np.random.default_rng(8), 60
    v = rng.integers(1, 8, (n, 64)).astype(float)
    k = rng.standard_normal(n)
    s = rng.uniform(1, 2, n).astype(np.float32).astype(float) * 2.0 ** -40
    zeros = np.arange(n) % 7 == 2
    s[zeros], v[zeros] = 1.0, 0.0
    c = one_head("e4m3", k, v, s)
    assert holds(c, *replay(k, v, s, 11, none=zeros))
    assert not holds(c, *replay(k, v, s, 11))
