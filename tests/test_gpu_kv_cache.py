"""Key-value cache written and read on the GPU, against the oracle bit for bit:
a 16-bit value is rounded once, a code and its scale are fp32 arithmetic that
numpy repeats."""

import numpy as np
import pytest
import torch

from oracle import kv_cache as okv
from oracle import fp8_block as ob
from _kv_cache import Cache, TORCH, page_table, pool_memory, rounded

pytestmark = pytest.mark.gpu

FILL = 0x5b     # bytes of what nothing writes


def pools(pages, page, n_kv, d, kind, layout):
    p = pool_memory(pages, page, n_kv, d, TORCH[kind], layout, "cuda")
    s = [None, None]
    if kind == "e4m3":
        s = pool_memory(pages, page, n_kv, None, torch.float32, layout, "cuda")
    for t in p:
        t.view(torch.uint8).fill_(FILL)
    for t in s:
        if t is not None:
            t.fill_(-7.0)
    return (*p, *s)


def bits(t):
    return torch.empty(t.shape, dtype=t.dtype).copy_(t).view(
        torch.uint8).numpy()


def source(rng, rows, n_kv, d, dtype, strided):
    x = rng.standard_normal((rows, 2 * n_kv + 3, d)).astype(np.float32)
    x *= np.exp(rng.standard_normal((rows, 2 * n_kv + 3, 1)))
    t = rounded(x, dtype)
    dev = t.cuda()
    k, v = dev[:, 3:3 + n_kv], dev[:, 3 + n_kv:]
    if not strided:
        k, v = k.contiguous(), v.contiguous()
    return t[:, 3:3 + n_kv], t[:, 3 + n_kv:], k, v


def want_write(cache, table, lens, start, k, v, kind):
    """The pools' and scales' bytes after the write, by the oracle."""
    out = [None if t is None else t.contiguous().cpu() for t in cache]
    for row, i, p in okv.tokens(lens, k.shape[0], start):
        page = out[0].shape[1]
        at = int(table[i][p // page]), p % page
        for j, x in ((0, k[row]), (1, v[row])):
            if kind == "e4m3":
                codes, s = okv.quantize(x.float().numpy())
                out[j].view(torch.uint8)[at] = torch.from_numpy(codes)
                out[j + 2][at] = torch.from_numpy(s)
            else:
                out[j][at] = x.to(TORCH[kind])
    return [None if t is None else bits(t) for t in out]


CASES = [   # lens, new (None: start), n_kv, d, page, layout, strided
    ([1], 1, 1, 64, 16, "heads", False),
    ([37], 1, 8, 128, 16, "heads", True),
    ([5, 0, 9, 1], 1, 2, 128, 4, "tokens", True),
    ([5, 0, 9, 1], 3, 3, 64, 1, "both", True),
    ([33, 64, 0, 65, 7], None, 2, 128, 32, "heads", True),
    ([33, 64, 0, 65, 7], None, 1, 64, 100, "wide", False),
    ([300], None, 5, 128, 7, "tokens", True),
    ([17] * 70 + [0, 3], 2, 1, 128, 8, "both", False)]


@pytest.mark.parametrize("kind", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("src", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("case", CASES)
def test_write_and_read(tp, case, src, kind):
    lens, new, n_kv, d, page, layout, strided = case
    rng = np.random.default_rng(len(lens) * 100 + d + page)
    table, pages = page_table(lens, page, rng)
    start = None
    rows = len(lens) * (new or 0)
    if new is None:     # two rows in front, three behind
        start = 2 + np.concatenate(([0], np.cumsum(lens)))
        rows = start[-1] + 3
    k, v, dk, dv = source(rng, rows, n_kv, d, src, strided)
    cache = pools(pages, page, n_kv, d, kind, layout)
    want = want_write(cache, table, lens, start, k, v, kind)
    dt = torch.from_numpy(table).cuda()
    dl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ds = None if start is None else torch.tensor(start, dtype=torch.int32,
                                                 device="cuda")
    tp.kv_cache_write(dk, dv, cache, dt, dl, start=ds)
    tp.device_status()
    for name, t, w in zip(("k", "v", "ks", "vs"), cache, want):
        if t is not None:
            assert (bits(t) == w).all(), name

    # read back: the same rows, the others as they were
    for out in (torch.bfloat16, torch.float16):
        got = [torch.full((rows, n_kv + 1, d), 3.0, dtype=out,
                          device="cuda")[:, 1:] for _ in range(2)]
        tp.kv_cache_read(cache, dt, dl, *got, start=ds)
        tp.device_status()
        for x, g in ((k, got[0]), (v, got[1])):
            w = torch.full((rows, n_kv, d), 3.0, dtype=out)
            for row, i, p in okv.tokens(lens, rows, start):
                if kind == "e4m3":
                    c, s = okv.quantize(x[row].float().numpy())
                    val = okv.dequantize(c, s).astype(np.float32)
                    w[row] = torch.from_numpy(val).to(out)
                else:
                    w[row] = x[row].to(TORCH[kind]).to(out)
            assert (bits(g) == bits(w)).all()


def test_special_values_quantized(tp):
    # zeros, one far value, NaN, infinities, a largest magnitude below 2^-100
    x = torch.zeros(5, 1, 128, dtype=torch.bfloat16)
    x[1, 0, 5], x[1, 0, 6] = -3.0, 448.0
    x[2, 0, :] = 1.0
    x[2, 0, 9] = float("nan")
    x[3, 0, 0], x[3, 0, 1] = float("-inf"), 2.0
    x[4, 0, 3] = 2.0 ** -120
    cache = tp.kv_cache_empty(1, 8, 1, 128, tp.FP8)
    t = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    n = torch.tensor([5], dtype=torch.int32, device="cuda")
    tp.kv_cache_write(x.cuda(), x.cuda(), cache, t, n)
    k, v = (torch.empty(5, 1, 128, dtype=torch.bfloat16, device="cuda")
            for _ in range(2))
    tp.kv_cache_read(cache, t, n, k, v)
    tp.device_status()
    x32 = x.float().numpy()[:, 0]
    lost = ~np.isfinite(x32)    # NaN, and an infinity times the factor 0
    with np.errstate(invalid="ignore"):
        q, s = ob.quantize(np.where(np.isnan(x32), 0, x32), "row")
    assert (cache[2][0, :5, 0].cpu().numpy() == s[0]).all()
    codes = cache[0][0, :5, 0].view(torch.uint8).cpu().numpy()
    assert (((codes & 0x7f) == 0x7f) == lost).all()
    assert (codes == q)[~lost].all()
    k = k.cpu().float()
    assert torch.equal(k[:2, 0], x[:2, 0].float()) and not k[0].any()
    assert torch.isnan(k[2, 0, 9]) and (k[2, 0, :9] == 1.0).all()
    assert torch.isnan(k[3]).all()          # an infinite scale
    assert (k[4].abs() <= 2.0 ** -110).all()


def test_an_fp16_overflow_is_reported(tp):
    x = torch.full((1, 1, 64), 7e4, dtype=torch.bfloat16, device="cuda")
    cache = tp.kv_cache_empty(1, 1, 1, 64, tp.F16)
    one = torch.ones(1, dtype=torch.int32, device="cuda")
    zero = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    tp.kv_cache_write(x, x, cache, zero, one)
    with pytest.raises(tp.TPError, match="TP_ERR_RANGE"):
        tp.device_status()
    x.fill_(float("inf"))       # fp16 has infinities
    tp.kv_cache_write(x, x, cache, zero, one)
    tp.device_status()


def test_bad_tables_and_lengths_are_reported_and_not_followed(tp):
    page, d, n_kv = 4, 64, 2
    cache = pools(6, page, n_kv, d, "bf16", "heads")
    before = [bits(t) for t in cache[:2]]
    table = torch.tensor([[1, -1], [6, 2], [2 ** 31 - 1, -2 ** 31]],
                         dtype=torch.int32, device="cuda")
    lens = torch.tensor([7, 3, 2], dtype=torch.int32, device="cuda")
    rows = torch.ones(3, n_kv, d, dtype=torch.bfloat16, device="cuda")
    tp.kv_cache_write(rows, rows, cache, table, lens)
    with pytest.raises(tp.TPError, match="TP_ERR_PAGE"):
        tp.device_status()
    out = torch.full_like(rows, 3.0), torch.full_like(rows, 3.0)
    tp.kv_cache_read(cache, table, lens, *out)
    with pytest.raises(tp.TPError, match="TP_ERR_PAGE"):
        tp.device_status()
    assert (out[0] == 3.0).all() and (out[1] == 3.0).all()
    # a length beyond the table's columns
    lens.fill_(9)
    tp.kv_cache_write(rows, rows, cache, table, lens)
    with pytest.raises(tp.TPError, match="TP_ERR_PAGE"):
        tp.device_status()
    for t, w in zip(cache, before):
        assert (bits(t) == w).all()
    tp.device_status()          # cleared


def test_offsets_beyond_32_bits(tp):
    # pages whose elements lie behind 2^32 of the pool's
    n_kv, d, page = 8, 128, 1024
    pages = (1 << 32) // (n_kv * d * page) + 3
    k = torch.empty((pages, n_kv, page, d), dtype=torch.float8_e4m3fn,
                    device="cuda").transpose(1, 2)
    s = torch.ones((pages, n_kv, page), device="cuda").transpose(1, 2)
    cache = (k, k, s, s)
    rng = np.random.default_rng(3)
    x, _, dx, _ = source(rng, 1500, n_kv, d, torch.bfloat16, True)
    table = torch.tensor([[pages - 1, pages - 2]], dtype=torch.int32,
                         device="cuda")
    lens = torch.tensor([1500], dtype=torch.int32, device="cuda")
    tp.kv_cache_write(dx, dx, cache, table, lens)
    out = torch.empty(1500, n_kv, d, dtype=torch.bfloat16, device="cuda")
    tp.kv_cache_read(cache, table, lens, out, out.clone())
    tp.device_status()
    c, sc = okv.quantize(x.float().numpy())
    got = k[pages - 1].view(torch.uint8).cpu().numpy()
    assert (got == c[:1024]).all()
    w = torch.from_numpy(okv.dequantize(c, sc).astype(np.float32))
    assert torch.equal(out.cpu(), w.bfloat16())


def test_captured_with_lengths_that_grow(tp):
    # one capture of write and read; the lengths move between replays
    rng = np.random.default_rng(4)
    cache = pools(8, 4, 2, 64, "bf16", "heads")
    table = torch.tensor([[5, 1, 7], [0, 2, 3]], dtype=torch.int32,
                         device="cuda")
    lens = torch.tensor([3, 0], dtype=torch.int32, device="cuda")
    k = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    got = torch.empty_like(k), torch.empty_like(k)

    def step():
        tp.kv_cache_write(k, k, cache, table, lens)
        tp.kv_cache_read(cache, table, lens, *got)

    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for n in range(5):
        lens += 1
        x = rounded(rng.standard_normal((2, 2, 64)), torch.bfloat16)
        k.copy_(x)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0].cpu(), x) and torch.equal(got[1].cpu(), x)
        at = lens.cpu() - 1
        for i in range(2):
            p = int(at[i])
            assert torch.equal(cache[0][int(table[i, p // 4]), p % 4].cpu(),
                               x[i])
    tp.device_status()


def test_round_trip_through_another_stream(tp):
    c = Cache([50, 20], 16, 2, 128, "bf16", 5)
    side = torch.cuda.Stream()
    rows = 70
    start = torch.tensor([0, 50, 70], dtype=torch.int32, device="cuda")
    k, v = (torch.empty(rows, 2, 128, dtype=torch.bfloat16, device="cuda")
            for _ in range(2))
    torch.cuda.synchronize()
    tp.kv_cache_read(*c.args, k, v, start=start, stream=side)
    copy = [torch.empty_like(t) for t in c.cache[:2]]
    tp.kv_cache_write(k, v, copy, *c.args[1:], start=start, stream=side)
    side.synchronize()
    for i, n in enumerate(c.lens):
        t = np.arange(n)
        at = torch.from_numpy(c.table[i][t // 16]).long(), \
            torch.from_numpy(t % 16)
        for a, b in zip(copy, c.cache):
            assert torch.equal(a.cpu()[at], b.cpu()[at])


@pytest.mark.parametrize("kind", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("src,d,n_kv,page,ragged", [
    (torch.bfloat16, 128, 8, 16, True), (torch.float16, 128, 3, 33, False),
    (torch.bfloat16, 64, 1, 100, True), (torch.float16, 64, 5, 8, False)])
def test_many_rows(tp, kind, src, d, n_kv, page, ragged):
    # enough vectors for four a thread, on a device of any number of SMs
    vecs = 9 * 256 * 16 // d * 160
    b = 7
    m = vecs // n_kv // b + 3
    rng = np.random.default_rng(d + n_kv)
    lens = [m + 5 * i if i % 3 else m - 11 * i for i in range(b)]
    table, pages = page_table(lens, page, rng)
    start, rows = None, b * m
    if ragged:
        start = 1 + np.concatenate(([0], np.cumsum(lens)))
        start[3:] -= 40        # the third one's newest but for the first 40
        rows = start[-1] + 2
    k, v, dk, dv = source(rng, rows, n_kv, d, src, True)
    cache = pools(pages, page, n_kv, d, kind, "heads")
    dt = torch.from_numpy(table).cuda()
    dl = torch.tensor(lens, dtype=torch.int32, device="cuda")
    ds = None if start is None else torch.tensor(start, dtype=torch.int32,
                                                 device="cuda")
    want = [None if t is None else t.contiguous().cpu() for t in cache]
    at = np.array(list(okv.tokens(lens, rows, start)))
    row, place = torch.from_numpy(at[:, 0]), \
        (torch.from_numpy(table[at[:, 1], at[:, 2] // page]).long(),
         torch.from_numpy(at[:, 2] % page))
    values = []
    for j, x in ((0, k), (1, v)):
        if kind == "e4m3":
            codes, s = okv.quantize(x.float().numpy())
            want[j].view(torch.uint8)[place] = torch.from_numpy(codes)[row]
            want[j + 2][place] = torch.from_numpy(s)[row]
            values.append(torch.from_numpy(okv.dequantize(codes, s)
                                           .astype(np.float32)))
        else:
            want[j][place] = x[row].to(TORCH[kind])
            values.append(x.to(TORCH[kind]))
    tp.kv_cache_write(dk, dv, cache, dt, dl, start=ds)
    tp.device_status()
    for t, w in zip(cache, want):
        if t is not None:
            assert (bits(t) == bits(w)).all()
    got = [torch.full((rows, n_kv, d), 3.0, dtype=src, device="cuda")
           for _ in range(2)]
    tp.kv_cache_read(cache, dt, dl, *got, start=ds)
    tp.device_status()
    for g, x in zip(got, values):
        w = torch.full((rows, n_kv, d), 3.0, dtype=src)
        w[row] = x[row].to(src)
        assert (bits(g) == bits(w)).all()


def test_the_module_and_the_python_checks_make_the_same_calls(tp, monkeypatch):
    # write, read and attention by way of csrc/pycall.cpp and without it
    assert tp._load().__name__.endswith("._tpcall")
    for kind in ("bf16", "f16", "e4m3"):
        c = Cache([70, 0, 33], 16, 2, 128, kind, 6)
        x = torch.randn(3, 12, 128, device="cuda").bfloat16()
        k, v, q = x[:, :2], x[:, 2:4], x[:, 4:]
        start = torch.tensor([0, 2, 2, 3], dtype=torch.int32, device="cuda")
        results = []
        for module in (tp._load(), tp._EveryCallInPython):
            monkeypatch.setattr(tp, "_tpcall", module)
            cache = tuple(None if t is None else t.clone() for t in c.cache)
            args = cache, c.dev_table, c.dev_lens
            for s in (None, start):
                tp.kv_cache_write(k, v, *args, start=s)
                back = torch.zeros_like(k), torch.zeros_like(v)
                tp.kv_cache_read(*args, *back, start=s)
                out, lse = torch.zeros_like(q), torch.zeros(3, 8, device="cuda")
                tp.attn_decode(q, *args, out, lse=lse)
                out2 = torch.zeros_like(q)
                tp.attn_decode(q, *args, out2, scale=0.5,
                               ws=torch.empty(tp.attn_decode_workspace_bytes(
                                   *args, 3, 8), dtype=torch.uint8,
                                   device="cuda"))
                results.append((*cache, *back, out, lse, out2))
        tp.device_status()
        for a, w in zip(results[:2], results[2:]):
            for x1, x2 in zip(a, w):
                assert x1 is x2 is None or (bits(x1) == bits(x2)).all()
        monkeypatch.undo()


@pytest.mark.parametrize("module", [True, False])
def test_both_refuse_on_the_gpu(tp, monkeypatch, module):
    if not module:
        monkeypatch.setattr(tp, "_tpcall", tp._EveryCallInPython)
    c = Cache([5, 6], 4, 2, 64, "bf16", 7)
    x = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    n = tp.launch_count()
    for a, kind in (
            ((x.float(), x.float(), *c.args), TypeError),
            ((x, x.half(), *c.args), TypeError),
            ((x[:1], x, *c.args), ValueError),
            ((x[..., ::2], x[..., ::2], *c.args), ValueError),
            ((x, x, c.cache[:1] + (c.cache[1].half(),), *c.args[1:]),
             TypeError),
            ((x, x, c.cache, c.dev_table.long(), c.dev_lens), TypeError),
            ((x, x, c.cache, c.dev_table, c.dev_lens[:1]), ValueError),
            ((x, x, c.cache, c.dev_table.cpu(), c.dev_lens), ValueError),
            ((x[:, :, :40], x[:, :, :40], *c.args), ValueError)):
        with pytest.raises(kind):
            tp.kv_cache_write(*a)
    odd = torch.zeros(2 * 2 * 64 + 4, dtype=torch.bfloat16,
                      device="cuda")[4:].view(2, 2, 64)
    with pytest.raises(tp.TPError, match="TP_ERR_ARG"):
        tp.kv_cache_write(odd, x, *c.args)
    with pytest.raises(tp.TPError, match="TP_ERR_SHAPE"):   # written rows twice
        tp.kv_cache_read(*c.args, x[:1].expand(2, 2, 64), x)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    for kw, kind in ((dict(q=q.half(), out=q.half()), TypeError),
                     (dict(out=q[:, :2]), ValueError),
                     (dict(q=q[:, :3], out=q[:, :3]), ValueError),
                     (dict(lse=torch.zeros(2, 4, device="cuda").t()),
                      ValueError),
                     (dict(ws=torch.zeros(8, dtype=torch.uint8)), ValueError),
                     (dict(scale=float("nan")), tp.TPError)):
        a = dict(q=q, out=torch.empty_like(q), lse=None, ws=None, scale=None)
        a.update(kw)
        with pytest.raises(kind):
            tp.attn_decode(a["q"], *c.args, a["out"], lse=a["lse"],
                           scale=a["scale"], ws=a["ws"])
    assert tp.launch_count() == n
