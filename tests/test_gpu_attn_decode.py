"""Attention of new tokens over a paged cache, against the fp64 oracle with
bounds derived from the roundings that it makes (_kv_cache.attend_bounds).
Whatever is not a token of a sequence is NaN in the pools."""

import numpy as np
import pytest
import torch

from _kv_cache import Cache, TORCH, attend_bounds, rounded

pytestmark = pytest.mark.gpu

BF16, F16 = torch.bfloat16, torch.float16


def queries(c, rows, n_q, dtype, seed, std=1.0, strided=True):
    x = np.random.default_rng(seed).standard_normal((rows, n_q, c.d)) * std
    t = rounded(x, dtype)
    dev = torch.full((rows, n_q + 2, c.d), float("nan"), dtype=dtype,
                     device="cuda")
    q = dev[:, 1:1 + n_q] if strided else dev[:, :n_q].contiguous()
    q.copy_(t)
    return t.double().numpy(), q


def attend(tp, c, q, lse=True, scale=None, **kw):
    out = torch.full((q.shape[0], q.shape[1] + 1, c.d), 7.0, dtype=q.dtype,
                     device="cuda")
    ls = torch.full(q.shape[:2], 7.0, device="cuda") if lse else None
    tp.attn_decode(q, *c.args, out[:, 1:], lse=ls, scale=scale, **kw)
    assert (out[:, 0] == 7.0).all()
    return out[:, 1:], ls


def check(tp, c, n_q, new, dtype, std=1.0, scale=None, strided=True, seed=9):
    rows = len(c.lens) * new
    x, q = queries(c, rows, n_q, dtype, seed, std, strided)
    out, lse = attend(tp, c, q, scale=scale)
    tp.device_status()
    want, wl, eo, el = attend_bounds(c, x, c.d ** -0.5 if scale is None
                                     else scale, dtype)
    got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
    empty = np.isinf(wl)
    assert (np.isneginf(gl) == empty).all()
    assert (got[empty] == 0).all()
    worst = (np.abs(got - want) / np.maximum(eo, 1e-300))[~empty]
    assert (worst <= 1).all(), f"out: {worst.max():.2f} of the bound"
    worst = np.abs(gl[~empty] - wl[~empty]) / el[~empty]
    assert (worst <= 1).all(), f"lse: {worst.max():.2f} of the bound"


TYPES = [("bf16", BF16), ("f16", BF16), ("f16", F16), ("e4m3", BF16),
         ("e4m3", F16)]
CASES = [   # lens, new, n_q, n_kv, d, page, layout
    ([1], 1, 1, 1, 64, 16, "heads"),
    ([2], 1, 8, 8, 128, 1, "tokens"),
    ([15, 16, 17, 0, 1], 1, 8, 2, 128, 16, "heads"),
    ([31, 33, 64, 65, 100], 1, 5, 1, 64, 32, "wide"),
    ([130, 1, 0, 77], 4, 16, 2, 128, 24, "both"),
    ([3, 2, 1, 0], 3, 6, 3, 128, 2, "heads"),
    ([260], 5, 8, 1, 128, 7, "tokens"),
    ([700, 13], 8, 32, 4, 64, 100, "heads"),
    ([9] * 40 + [130] + [0] * 3, 1, 4, 4, 64, 8, "heads"),
    ([1500], 1, 64, 8, 128, 64, "heads"),
    ([2049, 511], 2, 24, 8, 128, 1, "wide")]


@pytest.mark.parametrize("kind,dtype", TYPES)
@pytest.mark.parametrize("case", CASES)
def test_against_the_oracle(tp, case, kind, dtype):
    lens, new, n_q, n_kv, d, page, layout = case
    c = Cache(lens, page, n_kv, d, kind, sum(lens) + d, layout)
    check(tp, c, n_q, new, dtype)


@pytest.mark.parametrize("kind,dtype", TYPES)
def test_more_sequences_than_ctas(tp, kind, dtype):
    lens = [(37 * i) % 90 for i in range(400)]
    c = Cache(lens, 16, 2, 64, kind, 77)
    check(tp, c, 4, 1, dtype)


@pytest.mark.parametrize("kind,dtype", TYPES)
def test_a_long_sequence_among_short_ones(tp, kind, dtype):
    c = Cache([3, 20000, 0, 130, 1], 64, 1, 128, kind, 78)
    check(tp, c, 8, 1, dtype)


@pytest.mark.parametrize("stale", ["nan", "inf", "-inf", "max"])
@pytest.mark.parametrize("kind", ["bf16", "f16", "e4m3"])
def test_unused_places_have_no_influence(tp, kind, stale):
    c = Cache([17, 31, 129], 32, 2, 128, kind, 79, stale=stale)
    check(tp, c, 4, 1, BF16)
    check(tp, c, 4, 3, BF16)


@pytest.mark.parametrize("kind,dtype", TYPES)
def test_scores_far_apart(tp, kind, dtype):
    # one key outweighs all, elsewhere the maximum moves again and again
    c = Cache([400, 90], 16, 2, 128, kind, 80, std=3.0)
    check(tp, c, 8, 1, dtype, std=8.0)
    check(tp, c, 8, 1, dtype, scale=-0.25)
    check(tp, c, 8, 1, dtype, scale=0.0)


def test_scales_of_values_far_apart(tp):
    # the heaviest token's value scale is 2^-60 of another's: its weight in
    # the sum is that of its value, not that of its probability
    c = Cache([200], 16, 1, 128, "e4m3", 81)
    vs = c.cache[3]
    f = torch.exp2(torch.randint(-60, 40, vs.shape, device="cuda").float())
    live = torch.isfinite(vs)
    vs.copy_(torch.where(live, vs * f, vs))
    codes = c.cache[1].view(torch.uint8).cpu().numpy()
    from oracle import kv_cache as okv
    with np.errstate(invalid="ignore"):
        c.values[1] = okv.dequantize(codes, vs.cpu().numpy())
    check(tp, c, 8, 1, BF16, std=4.0)


@pytest.mark.parametrize("std", [2.0 ** -30, 2.0 ** 20])
@pytest.mark.parametrize("kind", ["bf16", "f16", "e4m3"])
def test_queries_of_any_size(tp, kind, std):
    # far outside of what fp16 holds
    c = Cache([100], 16, 1, 128, kind, 82)
    check(tp, c, 4, 1, BF16, std=std, scale=0.1 / std)


def test_dense_queries_and_no_lse(tp):
    c = Cache([100, 5], 16, 2, 128, "bf16", 83)
    check(tp, c, 4, 1, BF16, strided=False)
    _, q = queries(c, 2, 4, BF16, 9)
    a, _ = attend(tp, c, q)
    b, _ = attend(tp, c, q, lse=False)
    assert torch.equal(a, b)


def test_a_nan_among_the_tokens_stays_in_its_heads(tp):
    c = Cache([40, 40], 16, 2, 64, "bf16", 84)
    c.cache[0][int(c.table[1][0]), 3, 1, 5] = float("nan")
    _, q = queries(c, 2, 4, BF16, 9)
    out, lse = attend(tp, c, q)
    tp.device_status()
    bad = torch.isnan(out).any(dim=2).cpu()
    assert bad.tolist() == [[False] * 4, [False, False, True, True]]
    assert torch.equal(torch.isnan(lse).cpu(), bad)


@pytest.mark.parametrize("lens", [[40, 0], [900, 3]])
@pytest.mark.parametrize("kind", ["bf16", "f16", "e4m3"])
def test_queries_that_are_nan(tp, kind, lens):
    c = Cache(lens, 16, 2, 64, kind, 92)
    _, q = queries(c, 2, 4, BF16, 9)
    q[:, 1] = float("nan")
    out, lse = attend(tp, c, q)
    tp.device_status()
    out, lse = out.cpu(), lse.cpu()
    assert torch.isnan(out[0, 1]).all() and torch.isnan(lse[0, 1])
    assert not torch.isnan(out[:, [0, 2, 3]]).any()
    assert not torch.isnan(lse[:, [0, 2, 3]]).any()
    if lens[1] == 0:
        assert not out[1].any() and torch.isneginf(lse[1]).all()


@pytest.mark.parametrize("kind", ["bf16", "f16", "e4m3"])
def test_a_nan_in_a_token_that_a_row_does_not_see(tp, kind):
    # the third of four new tokens has NaN keys and values
    c = Cache([50, 6], 16, 1, 128, kind, 93)
    x, q = queries(c, 8, 8, BF16, 9)
    clean, _ = attend(tp, c, q)
    for i, n in enumerate(c.lens):
        at = int(c.table[i][(n - 2) // 16]), (n - 2) % 16
        for t in c.cache[:2]:
            if kind == "e4m3":
                t.view(torch.uint8)[at] = 0x7f
            else:
                t[at] = float("nan")
    out, lse = attend(tp, c, q)
    tp.device_status()
    for i in range(2):
        rows = slice(4 * i, 4 * i + 2)
        assert torch.equal(out[rows], clean[rows])
        assert torch.isfinite(lse[rows]).all()
        rows = slice(4 * i + 2, 4 * i + 4)
        assert torch.isnan(out[rows]).all() and torch.isnan(lse[rows]).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_pages_outside_the_pool(tp, kind):
    # their tokens are left out, everything else is as if they were not there
    c = Cache([40, 33, 70], 16, 2, 64, kind, 85)
    x, q = queries(c, 3, 4, BF16, 9)
    for bad in (-1, c.pages, 2 ** 31 - 1, -2 ** 31):
        c.dev_table[0, 2] = bad
        out, lse = attend(tp, c, q)
        with pytest.raises(tp.TPError, match="TP_ERR_PAGE"):
            tp.device_status()
        assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    # the same pools with a length that ends in front of the bad page
    c.dev_lens[0] = 32
    short, slse = attend(tp, c, q)
    tp.device_status()
    lim = 2.0 ** -6 * out.float().abs().max()
    assert ((short.float() - out.float()).abs() <= lim).all()
    assert ((lse - slse).abs() <= 1e-4).all()
    # a length beyond what the table can list
    c.dev_lens[0] = 10 ** 9
    out, _ = attend(tp, c, q)
    with pytest.raises(tp.TPError, match="TP_ERR_PAGE"):
        tp.device_status()
    assert torch.isfinite(out).all()


def test_shared_pages(tp):
    # two sequences with a common prefix read the same pages
    c = Cache([64, 64], 16, 1, 128, "bf16", 86)
    c.table[1, :2] = c.table[0, :2]
    c.dev_table.copy_(torch.from_numpy(c.table))
    check(tp, c, 4, 1, BF16)


def test_repeated_calls_agree_to_the_bit(tp):
    c = Cache([5000, 3, 777], 64, 2, 128, "e4m3", 87)
    _, q = queries(c, 3, 16, BF16, 9)
    a = attend(tp, c, q)
    for _ in range(5):
        b = attend(tp, c, q)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_two_streams_at_once(tp):
    cs = [Cache([3000, 50], 32, 2, 128, k, 88) for k in ("bf16", "e4m3")]
    qs = [queries(c, 2, 8, BF16, 9)[1] for c in cs]
    alone = [attend(tp, c, q) for c, q in zip(cs, qs)]
    outs = [[torch.empty_like(q) for _ in range(20)] for q in qs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for i in range(20):
        for c, q, o, s in zip(cs, qs, outs, streams):
            tp.attn_decode(q, *c.args, o[i], stream=s)
    torch.cuda.synchronize()
    tp.device_status()
    for (a, _), o in zip(alone, outs):
        assert all(torch.equal(a, x) for x in o)


def test_captured_while_the_sequences_grow(tp):
    # one graph of write and attention, replayed as lens moves on the device;
    # its workspace is the caller's
    c = Cache([60, 0, 17], 8, 2, 128, "bf16", 89)
    cols = 16
    table = torch.arange(3 * cols, dtype=torch.int32,
                         device="cuda").view(3, cols)
    cache = tp.kv_cache_empty(3 * cols, 8, 2, 128, tp.BF16)
    for t in cache[:2]:
        t.fill_(float("nan"))
    lens = torch.zeros(3, dtype=torch.int32, device="cuda")
    qkv = torch.zeros(3, 8, 128, dtype=BF16, device="cuda")
    q, k, v = qkv[:, :4], qkv[:, 4:6], qkv[:, 6:]
    out = torch.empty(3, 4, 128, dtype=BF16, device="cuda")
    ws = torch.empty(max(16, tp.attn_decode_workspace_bytes(
        cache, table, lens, 3, 4)), dtype=torch.uint8, device="cuda")

    def step():
        tp.kv_cache_write(k, v, cache, table, lens)
        tp.attn_decode(q, cache, table, lens, out, ws=ws)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    rng = np.random.default_rng(5)
    past = []
    for n in range(20):
        lens += 1
        qkv.copy_(rounded(rng.standard_normal((3, 8, 128)), BF16))
        past.append(qkv.double().cpu())
        g.replay()
        x = torch.stack(past, 1)                      # [3, n, 8, 128]
        kk = x[:, :, 4:6].repeat_interleave(2, 2)
        vv = x[:, :, 6:].repeat_interleave(2, 2)
        s = torch.einsum("bhd,bthd->bht", x[:, -1, :4], kk) / 128 ** 0.5
        w = torch.einsum("bht,bthd->bhd", s.softmax(-1), vv)
        # half a step of the output and what the weights' rounding can add
        assert (out.double().cpu() - w).abs().max() <= \
            w.abs().max() * 2.0 ** -8 + vv.abs().max() * 2.0 ** -12
    tp.device_status()


def test_long_offsets(tp):
    # a page whose elements lie behind 2^32 of the pool's
    n_kv, d, page = 8, 128, 1024
    pages = (1 << 32) // (n_kv * d * page) + 2
    mem = torch.zeros((pages, n_kv, page, d), dtype=torch.uint8,
                      device="cuda").transpose(1, 2)
    s = torch.ones((pages, n_kv, page), device="cuda").transpose(1, 2)
    c = Cache([900], page, n_kv, d, "e4m3", 90)
    at = int(c.table[0, 0])
    mem[pages - 1].copy_(c.cache[0][at].view(torch.uint8))
    s[pages - 1].copy_(c.cache[2][at])
    x, q = queries(c, 1, 16, BF16, 9)
    near = torch.empty_like(q)
    far = torch.empty_like(q)
    k, ks = c.cache[0], c.cache[2]
    tp.attn_decode(q, (k, k, ks, ks), c.dev_table, c.dev_lens, near)
    table = torch.full_like(c.dev_table, pages - 1)
    tp.attn_decode(q, (mem, mem, s, s), table, c.dev_lens, far)
    tp.device_status()
    assert torch.equal(near, far)


def test_a_workspace_too_small_is_refused(tp):
    c = Cache([4000], 16, 1, 128, "bf16", 91)
    _, q = queries(c, 1, 4, BF16, 9)
    need = tp.attn_decode_workspace_bytes(*c.args, 1, 4)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    a, _ = attend(tp, c, q, ws=ws)
    b, _ = attend(tp, c, q)
    assert torch.equal(a, b)
    if need > 16:
        with pytest.raises(tp.TPError, match="TP_ERR_WORKSPACE"):
            attend(tp, c, q, ws=ws[:need - 16])


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_thousands_of_places_in_the_batch(tp, kind):
    lens = [(i * 7) % 5 for i in range(3000)]
    lens[1700] = 700
    c = Cache(lens, 4, 1, 64, kind, 94)
    check(tp, c, 2, 1, BF16)


def test_two_captured_graphs(tp):
    # with a workspace each, replayed at once; with one of theirs, in turn
    cs = [Cache([3000, 50, 0], 32, 2, 128, k, 95) for k in ("bf16", "e4m3")]
    qs = [queries(c, 3, 8, BF16, 9)[1] for c in cs]
    alone = [attend(tp, c, q) for c, q in zip(cs, qs)]
    need = max(tp.attn_decode_workspace_bytes(*c.args, 3, 8) for c in cs)
    for shared in (False, True):
        ws = [torch.empty(need, dtype=torch.uint8, device="cuda")
              for _ in range(2)]
        outs, graphs = [], []
        for i, (c, q) in enumerate(zip(cs, qs)):
            out = torch.zeros_like(q)
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g):
                for _ in range(5):
                    tp.attn_decode(q, *c.args, out,
                                   ws=ws[0 if shared else i])
            graphs.append(g)
            outs.append(out)
        side = torch.cuda.Stream()
        for _ in range(5):
            graphs[0].replay()
            if shared:
                graphs[1].replay()
            else:
                with torch.cuda.stream(side):
                    graphs[1].replay()
        torch.cuda.synchronize()
        for (a, _), o in zip(alone, outs):
            assert torch.equal(a, o)
    tp.device_status()


def test_a_call_between_others_is_ordered_after_them(tp):
    # the second kernel may be launched early, but reads after the first; what
    # follows on the stream reads after both
    c = Cache([9000], 32, 1, 128, "bf16", 96)
    _, q = queries(c, 1, 8, BF16, 9, strided=False)
    q2 = q.clone().neg_()
    want = [attend(tp, c, x)[0].clone() for x in (q, q2)]
    out = torch.empty_like(q)
    got = torch.empty(40, *q.shape, dtype=BF16, device="cuda")
    x = q.clone()
    for i in range(40):
        x.copy_(q2 if i % 2 else q)
        tp.attn_decode(x, *c.args, out)
        got[i].copy_(out)
    for i in range(40):
        assert torch.equal(got[i], want[i % 2])
    tp.device_status()


def test_idle_places_queries_have_no_influence(tp):
    c = Cache([0, 40, 0], 16, 2, 128, "f16", 97)
    _, q = queries(c, 3, 4, BF16, 9)
    a = attend(tp, c, q)
    q[0] = float("nan")
    q[2] = float("inf")
    b = attend(tp, c, q)
    tp.device_status()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert not b[0][0].any() and not b[0][2].any()


@pytest.mark.parametrize("sign", [-1, 1])
def test_scores_of_1e34(tp, sign):
    # every score is the same far value: the values' mean
    c = Cache([300, 17], 16, 1, 128, "bf16", 98)
    c.cache[0].fill_(2.0 ** 53 * sign)
    q = torch.full((2, 8, 128), 2.0 ** 53, dtype=BF16, device="cuda")
    out, lse = attend(tp, c, q, scale=1.0)
    tp.device_status()
    for i, n in enumerate(c.lens):
        t = np.arange(n)
        x = c.values[1][c.table[i][t // 16], t % 16][:, 0]
        # one weight of 1 each, the sum's n + 9 roundings, the output's
        e = (n + 9) * 2.0 ** -22 * np.abs(x).mean(0) + \
            2.0 ** -8 * np.abs(x.mean(0))
        assert (np.abs(out[i].double().cpu().numpy() - x.mean(0)) <=
                e * 1.01).all()
        far = lse[i].double().cpu().numpy() / (sign * 2.0 ** 113)
        assert (np.abs(far - 1) <= 2.0 ** -20).all()


@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_the_same_sequences_under_a_wider_table(tp, kind):
    # a narrow table leaves every sequence to one CTA and needs no join
    c = Cache([100, 0, 64, 7], 16, 2, 128, kind, 99)
    x, q = queries(c, 4, 8, BF16, 9)
    n = tp.launch_count()
    narrow = attend(tp, c, q)
    assert tp.launch_count() - n == 1
    c.dev_table = torch.nn.functional.pad(c.dev_table, (0, 500), value=-1)
    n = tp.launch_count()
    wide = attend(tp, c, q)
    assert tp.launch_count() - n == 2
    tp.device_status()
    want, wl, eo, el = attend_bounds(c, x, c.d ** -0.5, BF16)
    for out, lse in (narrow, wide):
        got, gl = out.double().cpu().numpy(), lse.double().cpu().numpy()
        seen = np.isfinite(wl)
        assert (np.isfinite(gl) == seen).all() and not got[~seen].any()
        assert (np.abs(got - want) <= eo).all()
        assert (np.abs(gl[seen] - wl[seen]) <= el[seen]).all()
