"""Attention of new tokens over a paged cache where weights, scales or values
are far apart, against the fp64 definition (_kv_range.bounds)."""

import numpy as np
import pytest
import torch

from _kv_cache import Cache
from _kv_range import agree, bounds
from oracle import kv_cache as okv
from test_gpu_attn_decode import attend, queries

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


def first_element_alone(c, x, k):
    """Keys whose product with the queries (1, 0, …) is k[t] for token t of the
    one sequence; returns the queries."""
    n, table = c.lens[0], c.table[0]
    t = np.arange(n)
    c.values[0][table[t // c.page], t % c.page] = 0.0
    c.values[0][table[t // c.page], t % c.page, :, 0] = k[:, None]
    at = torch.from_numpy(table[t // c.page]).long().cuda(), \
        torch.from_numpy(t % c.page).cuda()
    if c.kind == "e4m3":
        codes, s = okv.quantize(c.values[0][table[t // c.page], t % c.page])
        c.cache[0].view(torch.uint8)[at] = torch.from_numpy(codes).cuda()
        c.cache[2][at] = torch.from_numpy(s).cuda()
    else:
        c.cache[0][at] = torch.from_numpy(
            c.values[0][table[t // c.page], t % c.page]).to(
                c.cache[0].dtype).cuda()
    x[:] = 0.0
    x[..., 0] = 1.0
    return torch.from_numpy(x).to(BF16).cuda()


def set_values(c, t, codes=None, scale=None):
    """Codes (or 16-bit values, all of a vector the same) and scales of tokens t
    of the one sequence."""
    page, off = c.table[0][t // c.page], t % c.page
    at = torch.from_numpy(page).long().cuda(), torch.from_numpy(off).cuda()
    if c.kind != "e4m3":
        c.cache[1][at] = codes
        c.values[1][page, off] = codes
        return
    v, s = c.cache[1].view(torch.uint8), c.cache[3]
    if codes is not None:
        v[at] = codes
    if scale is not None:
        s[at] = scale
    with np.errstate(invalid="ignore"):
        c.values[1] = okv.dequantize(v.cpu().numpy(), s.cpu().numpy())


# ------------------------------------------------------------- weights far apart
@pytest.mark.parametrize("nats", [10.0, 17.5, 20.0])
@pytest.mark.parametrize("n", [192, 5000])
@pytest.mark.parametrize("kind", ["bf16", "f16", "e4m3"])
def test_heavy_tokens_without_a_value(tp, kind, n, nats):
    # in each step of a warp one token has nearly all the weight and no value:
    # what is left is the others' part
    c = Cache([n], 16, 1, 128, kind, 101)
    x, _ = queries(c, 1, 8, BF16, 9)
    t = np.arange(n)
    if kind == "e4m3":
        set_values(c, t, scale=2.0 ** -8)
    set_values(c, t[t % 16 == 0], codes=0)
    q = first_element_alone(c, x, np.where(t % 16 == 0, nats, 0.0))
    out, lse = attend(tp, c, q, scale=1.0)
    tp.device_status()
    agree(out, lse, bounds(c, x, 1.0, BF16))


# --------------------------------------------------------------- scales of values
@pytest.mark.parametrize("scale", ["nan", "inf", "1e-45", "0", "-1", "-inf"])
@pytest.mark.parametrize("n", [50, 700])
def test_scales_of_a_token_that_a_row_does_not_see(tp, n, scale):
    # the third of four new tokens; the first two rows do not see it
    c = Cache([n, 6], 16, 1, 128, "e4m3", 102)
    x, q = queries(c, 8, 8, BF16, 9)
    for i, m in enumerate(c.lens):
        at = int(c.table[i][(m - 2) // 16]), (m - 2) % 16
        c.cache[2][at] = c.cache[3][at] = float(scale)
        for k in c.values:
            k[at] = np.nan
    out, lse = attend(tp, c, q)
    tp.device_status()
    with np.errstate(invalid="ignore"):
        want = bounds(c, x, c.d ** -0.5, BF16)
    agree(out, lse, want, [0, 1, 4, 5])
    if scale in ("nan", "inf", "-inf"):   # of its key too: rows that see it
        assert torch.isnan(out[[2, 3, 6, 7]]).all()


@pytest.mark.parametrize("scale", ["nan", "-1"])
def test_a_values_scale_that_is_none(tp, scale):
    # where it is seen the output is NaN; its weight is known
    c = Cache([90], 16, 1, 128, "e4m3", 111)
    x, q = queries(c, 1, 8, BF16, 9)
    _, want, _, bound = bounds(c, x, c.d ** -0.5, BF16)
    set_values(c, np.array([50]), scale=float(scale))
    out, lse = attend(tp, c, q)
    tp.device_status()
    assert torch.isnan(out).all()
    assert (np.abs(lse.double().cpu().numpy() - want) <= bound).all()


@pytest.mark.parametrize("size", [-108, -60, 0, 60, 110, 119])
@pytest.mark.parametrize("n", [300, 20000])
def test_values_of_any_size(tp, n, size):
    # scales of 2^size: from the smallest that kv_cache_write makes to bf16's end
    c = Cache([n, 40], 64, 1, 128, "e4m3", 103)
    codes, vs = c.cache[1].view(torch.uint8), c.cache[3]
    vs.copy_(torch.where(torch.isfinite(vs), 2.0 ** size, vs))
    with np.errstate(invalid="ignore"):
        c.values[1] = okv.dequantize(codes.cpu().numpy(), vs.cpu().numpy())
    x, q = queries(c, 2, 8, BF16, 9, std=0.1)
    out, lse = attend(tp, c, q)
    tp.device_status()
    agree(out, lse, bounds(c, x, c.d ** -0.5, BF16))


@pytest.mark.parametrize("n", [3, 300, 20000])
def test_scales_of_zero(tp, n):
    # whatever the codes are, the value is 0, and its weight counts
    c = Cache([n], 64, 1, 128, "e4m3", 104)
    x, q = queries(c, 2, 8, BF16, 9)
    t = np.arange(n)
    set_values(c, t[t % 3 == 1], scale=0.0)
    set_values(c, t[t % 12 == 5], scale=2.0 ** -130)
    agree(*attend(tp, c, q), bounds(c, x, c.d ** -0.5, BF16))
    # no token has a value
    set_values(c, t, scale=0.0)
    c.values[1][:] = 0.0
    out, lse = attend(tp, c, q)
    tp.device_status()
    assert not out.any()
    agree(out, lse, bounds(c, x, c.d ** -0.5, BF16))


@pytest.mark.parametrize("size", [2.0 ** -26, 1.0])
@pytest.mark.parametrize("n", [60, 5000])
def test_values_of_zeros_among_others(tp, n, size):
    # as kv_cache_write stores them: the scale of zeros is 1, far above others'
    c = Cache([n], 16, 1, 128, "e4m3", 105, std=size)
    x, _ = queries(c, 1, 8, BF16, 9)
    t = np.arange(n)
    zeros = t % 16 == 0
    set_values(c, t[zeros], codes=0, scale=1.0)
    # with as much weight as the others, and with nearly all of it
    for nats in (0.0, 20.0):
        q = first_element_alone(c, x, np.where(zeros, nats, 0.0))
        out, lse = attend(tp, c, q, scale=1.0)
        agree(out, lse, bounds(c, x, 1.0, BF16))
    # codes of −0, and nothing but zeros
    set_values(c, t, codes=0x80, scale=1.0)
    out, lse = attend(tp, c, q, scale=1.0)
    tp.device_status()
    assert not out.any()
    agree(out, lse, bounds(c, x, 1.0, BF16))


def test_a_nan_beside_zeros(tp):
    c = Cache([40], 16, 1, 128, "e4m3", 106)
    x, q = queries(c, 1, 8, BF16, 9)
    set_values(c, np.arange(40), codes=0, scale=1.0)
    c.cache[1].view(torch.uint8)[int(c.table[0][1]), 3, 0, 77] = 0xff
    out, lse = attend(tp, c, q)
    tp.device_status()
    assert torch.isnan(out[0, :, 77]).all() and torch.isfinite(lse).all()
    out[0, :, 77] = 0.0
    assert not out.any()


# ------------------------------------------------------------------- fp16's end
@pytest.mark.parametrize("n", [40, 3000])
def test_outputs_that_fp16_does_not_hold(tp, n):
    c = Cache([n], 16, 2, 64, "e4m3", 107)
    set_values(c, np.arange(n), codes=0x70, scale=1024.0)   # 128 · 1024
    c.cache[1].view(torch.uint8)[:, :, 1] = 0x60            # 32 · 1024
    c.values[1][:, :, 1] = 32.0 * 1024
    x, q = queries(c, 1, 4, F16, 9)
    out, lse = attend(tp, c, q)
    with pytest.raises(tp.TPError, match="TP_ERR_RANGE"):
        tp.device_status()
    assert torch.isinf(out[0, :2]).all()
    assert (out[0, 2:] == 32768.0).all() and torch.isfinite(lse).all()
    out, _ = attend(tp, c, q.bfloat16())     # which holds them
    tp.device_status()
    assert (out[0, :2] == 131072.0).all() and (out[0, 2:] == 32768.0).all()


@pytest.mark.parametrize("kind", ["f16", "e4m3"])
def test_means_of_fp16s_largest_value(tp, kind):
    # one token's weight is 1, the others' are just above 1/2, where each is
    # rounded up by 0.4 of fp16's step: a mean that is 2^-11.5 too large
    c = Cache([16], 16, 1, 128, kind, 108)
    t = np.arange(16)
    if kind == "e4m3":
        set_values(c, t, codes=0x7e, scale=65504.0 / 448.0)
    else:
        set_values(c, t, codes=65504.0)
    x, _ = queries(c, 1, 8, BF16, 9)
    q = first_element_alone(c, x, np.where(t == 0, 0.0, 1.0)).half()
    out, _ = attend(tp, c, q, scale=float(np.log(0.5 * (1 + 0.6 * 2.0 ** -10))))
    tp.device_status()
    assert (out == 65504.0).all()


def test_an_infinite_value_is_no_output_beyond_fp16(tp):
    c = Cache([40], 16, 1, 128, "f16", 109)
    x, q = queries(c, 1, 8, F16, 9)
    c.cache[1][int(c.table[0][0]), 3, 0, 5] = float("inf")
    out, lse = attend(tp, c, q)
    tp.device_status()
    assert not torch.isfinite(out[0, :, 5]).any() and torch.isfinite(lse).all()
    out[0, :, 5] = 0.0
    assert torch.isfinite(out).all()


# ------------------------------------------------------------ many new tokens
@pytest.mark.parametrize("kind,d", [("bf16", 128), ("f16", 64), ("e4m3", 128),
                                    ("e4m3", 64)])
def test_many_new_tokens_of_which_late_ones_are_nan(tp, kind, d):
    # 64 new tokens of 8 heads: 16 tiles of rows, each with another end
    c = Cache([150, 70, 20], 16, 1, d, kind, 110)
    x, q = queries(c, 3 * 64, 8, BF16, 9)
    first_bad = 40           # of each sequence's rows
    for i, n in enumerate(c.lens):
        for t in range(max(0, n - 64 + first_bad), n):
            at = int(c.table[i][t // 16]), t % 16
            for pool, k in zip(c.cache[:2], c.values):
                if kind == "e4m3":
                    pool.view(torch.uint8)[at] = 0x7f
                else:
                    pool[at] = float("nan")
                k[at] = np.nan
    out, lse = attend(tp, c, q)
    tp.device_status()
    with np.errstate(invalid="ignore"):
        want = bounds(c, x, c.d ** -0.5, BF16)
    rows = np.array([64 * i + j for i in range(3) for j in range(first_bad)])
    seen = np.isfinite(want[1][rows]).all(axis=1)
    assert np.isneginf(lse[torch.from_numpy(rows[~seen])].cpu().numpy()).all()
    assert not out[torch.from_numpy(rows[~seen]).cuda()].any()
    agree(out, lse, want, rows[seen])
    for i, n in enumerate(c.lens):   # and those that see one
        late = out[64 * i + max(first_bad, 64 - n):64 * (i + 1)]
        assert torch.isnan(late).all()
