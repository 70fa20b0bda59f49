"""Key-value cache without a GPU: pins of its oracle, where rows and pages are
found (the kernels' own code, compiled for the host), and the refusals of the C
entry points and of the binding (no call here launches)."""

import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import oracle
from oracle import kv_cache as okv
from test_fp8_block_device_host import On

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
NULL, SHAPE, DTYPE, WORKSPACE, UNSUPPORTED, ARG = 1, 2, 3, 4, 5, 8


# ------------------------------------------------------------------ oracle --
def test_tokens_of_rows():
    assert list(okv.tokens([3, 1, 0], 6)) == [
        (0, 0, 1), (1, 0, 2), (3, 1, 0)]
    assert list(okv.tokens([3, 1, 0], 9, [1, 4, 4, 6])) == [
        (1, 0, 0), (2, 0, 1), (3, 0, 2)]


def test_attend_is_the_last_rows_of_causal_attention():
    rng = np.random.default_rng(1)
    s, nq, nkv, d, h = 11, 4, 2, 8, 16
    X = rng.standard_normal((s, h))
    Wq, Wk, Wv = (rng.standard_normal((n * d, h)) * 0.3
                  for n in (nq, nkv, nkv))
    f = oracle.attention_forward(X, Wq, Wk, Wv, np.eye(nq * d), b=1, s=s,
                                 n_q=nq, n_kv=nkv, d=d)
    page, table = 4, np.array([[2, 0, 3]])
    pools = []
    for W in (Wk, Wv):
        x = np.full((4, page, nkv, d), np.nan)
        for t, row in enumerate((X @ W.T).reshape(s, nkv, d)):
            x[table[0][t // page], t % page] = row
        pools.append(x)
    out, _ = okv.attend((X[-3:] @ Wq.T).reshape(3, nq, d), *pools, table, [s],
                        d ** -0.5)
    assert np.allclose(out.reshape(3, -1), f["Out"][-3:], atol=1e-12)


def test_attend_by_hand_and_of_nothing():
    k = np.array([[[[1.0, 0.0]], [[0.0, 0.0]]]])
    v = np.array([[[[2.0, 1.0]], [[6.0, 5.0]]]])
    q = np.array([[[np.log(3.0), 9.0]], [[1.0, 1.0]]])
    out, lse = okv.attend(q, k, v, np.array([[0], [0]]), [2, 0], 1.0)
    # weights 3 and 1
    assert np.allclose(out[0, 0], [3.0, 2.0]) and np.isclose(lse[0, 0],
                                                             np.log(4.0))
    assert (out[1] == 0).all() and lse[1, 0] == -np.inf


def test_bounds_come_with_the_same_attention():
    from _kv_cache import Cache, attend_bounds
    for kind in ("bf16", "e4m3"):
        c = Cache([9, 0, 5], 4, 2, 64, kind, 3, device="cpu")
        q = np.random.default_rng(4).standard_normal((6, 6, 64))
        out, lse, eo, el = attend_bounds(c, q, 0.2, torch.bfloat16)
        with np.errstate(invalid="ignore"):
            want, wl = okv.attend(q, *c.values, c.table, c.lens, 0.2)
        assert np.allclose(out, want, rtol=1e-12, atol=1e-14)
        assert np.allclose(lse, wl, rtol=1e-12)
        seen = np.isfinite(lse)
        # of the size of the output's own rounding (values of up to 8)
        assert (eo[seen] <= 2.0 ** -8 * np.abs(out[seen]) + 2.0 ** -7).all()
        assert (el[seen] <= 2.0 ** -9).all() and (eo[~seen] == 0).all()


# ------------------------------------------------- the kernels' own indexing --
PLACE = r'''
#include "kv_place.h"
extern "C" int token_of(const tp_kv_cache* c, const int32_t* start, int per,
                        int64_t row, int* seq, int* pos) {
  return tp::kv_token_of(*c, start, per, row, seq, pos);
}
extern "C" int64_t page_of(const tp_kv_cache* c, int seq, int pos, int* off) {
  return tp::kv_page_of(*c, seq, pos, off);
}
'''


@pytest.fixture(scope="module")
def place(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no g++")
    d = tmp_path_factory.mktemp("place")
    (d / "p.cpp").write_text(PLACE)
    csrc = os.path.join(ROOT, "megatron_tensor_transformer_gate_gb300", "csrc")
    subprocess.run([cxx, "-O1", "-shared", "-fPIC", "-I", csrc,
                    str(d / "p.cpp"), "-o", str(d / "p.so")], check=True)
    L = ctypes.CDLL(str(d / "p.so"))
    L.page_of.restype = ctypes.c_int64
    return L


def i32(x):
    return np.ascontiguousarray(x, np.int32)


def addr(a):
    return a.ctypes.data_as(ctypes.c_void_p)


def desc(tp, table, lens, page=4, pages=10):
    c = tp.KvCache()
    c.b, c.page, c.table_cols, c.pages = len(lens), page, table.shape[1], pages
    c.table, c.table_stride = table.ctypes.data, table.shape[1]
    c.lens = lens.ctypes.data
    return c


def token(place, c, start, per, row):
    seq, pos = ctypes.c_int(), ctypes.c_int()
    ok = place.token_of(ctypes.byref(c), None if start is None else
                        addr(start), per, ctypes.c_int64(row),
                        ctypes.byref(seq), ctypes.byref(pos))
    return (seq.value, pos.value) if ok else None


@pytest.mark.parametrize("start", [None, [0, 3, 3, 4, 9], [2, 2, 5, 6, 7]])
def test_rows_as_the_oracle_says(tp, place, start):
    lens, table = i32([2, 0, 9, 3]), i32(np.zeros((4, 3)))
    rows = 12
    c = desc(tp, table, lens)
    s = None if start is None else i32(start)
    want = {r: (i, p) for r, i, p in okv.tokens(lens, rows, start)}
    for r in range(rows):
        assert token(place, c, s, 3, r) == want.get(r), r


def test_starts_that_are_wrong_name_places_of_the_batch(tp, place):
    rng = np.random.default_rng(2)
    lens, table = i32([7, 2 ** 31 - 1, -2 ** 31, 0, 5]), i32(np.zeros((5, 1)))
    c = desc(tp, table, lens)
    for _ in range(300):
        s = i32(rng.integers(-20, 40, 6))
        if rng.random() < 0.3:
            s[rng.integers(6)] = rng.choice([2 ** 31 - 1, -2 ** 31])
        for r in range(30):
            t = token(place, c, s, 1, r)
            assert t is None or (0 <= t[0] < 5 and 0 <= t[1] < lens[t[0]])


def test_pages_and_lengths_that_are_wrong_are_not_followed(tp, place):
    # rows of guards on both sides of the table: none is ever returned
    guard = np.full((5, 3), 7, np.int32)
    guard[1:4] = [[0, 9, -1], [10, 2 ** 31 - 1, -2 ** 31], [3, 4, 5]]
    table, lens = guard[1:4], i32([1, 1, 1])
    c = desc(tp, table, lens)
    off = ctypes.c_int()

    def page(seq, pos):
        return place.page_of(ctypes.byref(c), seq, pos, ctypes.byref(off))

    assert [page(0, p) for p in (0, 3, 4, 8, 11, 12, 2 ** 31 - 1)] == \
        [0, 0, 9, -1, -1, -1, -1]
    assert [page(1, p) for p in (0, 4, 8)] == [-1, -1, -1]
    assert [page(2, p) for p in (0, 4, 11, 12)] == [3, 4, 5, -1]
    assert page(2, 10) == 5 and off.value == 2


# --------------------------------------------------------- C entry refusals --
def good(tp, **kw):
    c = tp.KvCache()
    f = dict(dtype=1, b=2, n_kv=4, d=128, page=16, table_cols=3, pages=8,
             k=0x100000, v=0x200000, page_stride=16 * 512, token_stride=512,
             head_stride=128, ks=0x300000, vs=0x400000, s_page_stride=64,
             s_token_stride=4, s_head_stride=1, table=0x500000, table_stride=3,
             lens=0x600000)
    f.update(kw)
    for k, v in f.items():
        setattr(c, k, v)
    return c


def write(tp, c=None, dtype=1, rows=4, K=0x700000, kr=512, kh=128,
          V=0x800000, vr=512, vh=128, start=None, fn="tp_kv_cache_write",
          **kw):
    c = good(tp, **kw) if c is None else c
    return getattr(tp.lib(), fn)(ctypes.byref(c), dtype, rows, K, kr, kh, V,
                                 vr, vh, start, None)


BAD_CACHES = [
    (dict(dtype=0), DTYPE), (dict(dtype=7), DTYPE), (dict(b=0), SHAPE),
    (dict(b=70000), SHAPE), (dict(n_kv=0), SHAPE), (dict(page=0), SHAPE),
    (dict(table_cols=0), SHAPE), (dict(pages=0), SHAPE),
    (dict(pages=1 << 31), SHAPE), (dict(d=96), UNSUPPORTED),
    (dict(d=256), UNSUPPORTED), (dict(k=None), NULL), (dict(v=None), NULL),
    (dict(table=None), NULL), (dict(lens=None), NULL),
    (dict(dtype=2, ks=None), NULL), (dict(dtype=2, vs=None), NULL),
    (dict(page_stride=16 * 512 + 4), SHAPE),     # not on 16 bytes
    (dict(dtype=2, head_stride=136), SHAPE),     # of codes
    (dict(head_stride=64), SHAPE),               # heads overlap
    (dict(token_stride=256), SHAPE),             # tokens overlap
    (dict(page_stride=512), SHAPE), (dict(page_stride=-8192), SHAPE),
    (dict(page_stride=1 << 62), SHAPE),
    (dict(dtype=2, s_token_stride=3), SHAPE),
    (dict(dtype=2, s_head_stride=0), SHAPE),
    (dict(table_stride=2), SHAPE), (dict(k=0x100008), ARG),
    (dict(lens=0x600002), ARG), (dict(table=0x500001), ARG),
    (dict(dtype=2, ks=0x300002), ARG)]


@pytest.mark.parametrize("fn", ["tp_kv_cache_write", "tp_kv_cache_read"])
def test_moves_refuse(tp, fn):
    for kw, rc in BAD_CACHES:
        assert write(tp, good(tp, **kw), fn=fn) == rc, kw
    args = dict(fn=fn)
    for kw, rc in ((dict(dtype=0), DTYPE), (dict(dtype=2), DTYPE),
                   (dict(rows=0), SHAPE), (dict(rows=3), SHAPE),
                   (dict(rows=1 << 31), SHAPE), (dict(K=None), NULL),
                   (dict(V=None), NULL), (dict(kr=516), SHAPE),
                   (dict(vh=132), SHAPE), (dict(kr=-512), SHAPE),
                   (dict(V=0x800008), ARG), (dict(start=0x900002), ARG)):
        c = good(tp)
        assert write(tp, c, **args, **kw) == rc, kw
    assert getattr(tp.lib(), fn)(None, 1, 4, 0x700000, 512, 128, 0x800000, 512,
                                 128, None, None) == NULL
    if fn.endswith("read"):     # rows that are written lie apart
        assert write(tp, fn=fn, kr=256) == SHAPE
        assert write(tp, fn=fn, vh=0) == SHAPE


def decode(tp, c=None, dtype=1, rows=4, n_q=8, scale=0.1, q=0x700000, qr=1024,
           qh=128, o=0x800000, orow=1024, oh=128, lse=0xa00000, ws=0xb00000,
           size=1 << 40, **kw):
    c = good(tp, **kw) if c is None else c
    return tp.lib().tp_attn_decode(ctypes.byref(c), dtype, rows, n_q, scale, q,
                                   qr, qh, o, orow, oh, lse, ws, size, None)


def test_decode_refuses(tp):
    for kw, rc in BAD_CACHES:
        assert decode(tp, good(tp, **kw)) == rc, kw
    for kw, rc in ((dict(dtype=0), DTYPE), (dict(dtype=3), UNSUPPORTED),
                   (dict(rows=0), SHAPE), (dict(rows=5), SHAPE),
                   (dict(rows=1 << 30, n_q=8), SHAPE), (dict(n_q=6), SHAPE),
                   (dict(n_q=0), SHAPE), (dict(scale=float("nan")), ARG),
                   (dict(scale=float("inf")), ARG), (dict(q=None), NULL),
                   (dict(o=None), NULL), (dict(qr=1028), SHAPE),
                   (dict(oh=64), SHAPE), (dict(orow=512), SHAPE),
                   (dict(q=0x700004), ARG), (dict(lse=0xa00002), ARG),
                   (dict(ws=0xb00008), ARG)):
        assert decode(tp, **kw) == rc, kw
    c = good(tp)
    assert tp.lib().tp_attn_decode_workspace_bytes(None, 4, 8) == 0
    assert tp.lib().tp_attn_decode_workspace_bytes(ctypes.byref(c), 5, 8) == 0
    for kw in (dict(b=0), dict(n_kv=0), dict(page=0), dict(page=-64),
               dict(table_cols=-17), dict(table_cols=0), dict(d=80)):
        bad = good(tp, **kw)
        assert tp.lib().tp_attn_decode_workspace_bytes(ctypes.byref(bad), 4,
                                                       8) == 0, kw
    # more work than is counted in 31 bits, tokens beyond 2^30
    assert decode(tp, good(tp, b=2, n_kv=1024, page=1 << 20, table_cols=512,
                           token_stride=131072, page_stride=1 << 38,
                           s_token_stride=1024, table_stride=512),
                  n_q=1024, qr=1 << 17, orow=1 << 17) == SHAPE
    assert decode(tp, good(tp, page=1 << 20, table_cols=1025,
                           page_stride=512 << 20, table_stride=1025)) == SHAPE
    need = tp.lib().tp_attn_decode_workspace_bytes(ctypes.byref(c), 4, 8)
    if need:
        assert decode(tp, size=need - 1) == WORKSPACE
        assert decode(tp, ws=None) == NULL


# ---------------------------------------------------------- binding refusals --
@pytest.fixture
def make(tp, monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)

    def on(t, dev=0):
        return None if t is None else On(t, dev)

    def cache(kind=None, pages=6, page=4, n_kv=2, d=64, dev=0):
        return [on(t, dev) for t in tp.kv_cache_empty(
            pages, page, n_kv, d, tp.BF16 if kind is None else kind, "cpu")]

    def ints(*shape, dev=0, dtype=torch.int32):
        return On(torch.zeros(*shape, dtype=dtype), dev)

    return on, cache, ints


def test_room_for_a_cache(tp):
    k, v, ks, vs = tp.kv_cache_empty(5, 16, 2, 128, tp.FP8, "cpu")
    assert k.shape == (5, 16, 2, 128) and k.stride() == (4096, 128, 2048, 1)
    assert ks.shape == (5, 16, 2) and ks.stride() == (32, 1, 16)
    assert k.dtype == torch.float8_e4m3fn and v.stride() == k.stride()
    k, v, ks, vs = tp.kv_cache_empty(5, 16, 2, 128, tp.F16, "cpu")
    assert k.dtype == torch.float16 and ks is None and vs is None
    with pytest.raises(TypeError, match="dtype"):
        tp.kv_cache_empty(5, 16, 2, 128, tp.F32, "cpu")


def test_binding_refuses(tp, make):
    on, cache, ints = make
    b, m, nq = 3, 2, 4
    bf = torch.bfloat16
    rows = lambda heads=2, d=64, n=b * m, dev=0, dt=bf: On(
        torch.zeros(n, heads, d, dtype=dt), dev)
    base = dict(cache=cache(), table=ints(b, 5), lens=ints(b), q=rows(nq),
                out=rows(nq), k=rows(), v=rows(), lse=None, start=None,
                ws=None)
    both, move, att = ("move", "attend"), ("move",), ("attend",)
    c8 = cache(tp.FP8)
    cases = [
        (both, dict(cache=[On(t.t, 1) if t is not None else None
                           for t in cache()]), ValueError, "current device"),
        (both, dict(cache=[cache()[0], On(cache()[1].t, 1), None, None]),
         ValueError, "v: on"),
        (both, dict(cache=[on(torch.zeros(6, 4, 2, 64)), cache()[1]]),
         TypeError, "k: bfloat16"),
        (both, dict(cache=[cache()[0], cache(tp.F16)[1]]), TypeError, "^v:"),
        (both, dict(cache=[cache()[0], cache(pages=5)[1]]), ValueError,
         "^v: shape"),
        (both, dict(cache=[cache()[0],
                           on(torch.zeros(6, 4, 2, 64, dtype=bf))]),
         ValueError, "same strides"),
        (both, dict(cache=c8[:2]), ValueError, "codes without scales"),
        (both, dict(cache=cache()[:2] + c8[2:]), ValueError, "has none"),
        (both, dict(cache=c8[:3] + [on(torch.zeros(6, 4, 3))]), ValueError,
         "^vs: shape"),
        (both, dict(cache=c8[:3] + [on(torch.zeros(6, 4, 2))]), ValueError,
         "same strides"),
        (both, dict(table=ints(b, 5, dtype=torch.int64)), TypeError, "table"),
        (both, dict(table=ints(0, 5), lens=ints(0)), ValueError, "empty"),
        (both, dict(table=ints(b, 0)), ValueError, "empty"),
        (both, dict(cache=cache(pages=0)), ValueError, "empty"),
        (both, dict(cache=cache(n_kv=0)), ValueError, "empty"),
        (both, dict(table=ints(b * 5)), ValueError, "table: 2 axes"),
        (both, dict(table=ints(b, 5, dev=1)), ValueError, "table: on"),
        (both, dict(table=on(torch.zeros(5, b, dtype=torch.int32).t())),
         ValueError, "adjacent"),
        (both, dict(lens=ints(b + 1)), ValueError, "lens"),
        (both, dict(lens=ints(b, dtype=torch.int64)), TypeError, "lens"),
        (both, dict(lens=on(torch.zeros(2 * b, dtype=torch.int32)[::2])),
         ValueError, "lens"),
        (move, dict(k=rows(dt=torch.float32), v=rows(dt=torch.float32)),
         TypeError, "k rows"),
        (move, dict(v=rows(dt=torch.float16)), TypeError, "v rows"),
        (move, dict(k=rows(3)), ValueError, "k rows: shape"),
        (move, dict(v=rows(n=5)), ValueError, "v rows: shape"),
        (move, dict(k=rows(n=7), v=rows(n=7)), ValueError, "same number"),
        (move, dict(k=rows(dev=1)), ValueError, "k rows: on"),
        (move, dict(k=on(torch.zeros(6, 64, 2, dtype=bf).transpose(1, 2))),
         ValueError, "adjacent elements"),
        (move, dict(start=ints(b)), ValueError, "start"),
        (move, dict(start=ints(b + 1, dtype=torch.int64)), TypeError, "start"),
        (move, dict(start=ints(b + 1, dev=1)), ValueError, "start: on"),
        (att, dict(q=rows(5), out=rows(5)), ValueError, "5 heads"),
        (att, dict(q=rows(nq, n=7), out=rows(nq, n=7)), ValueError, "7 rows"),
        (att, dict(q=rows(nq, d=128)), ValueError, "^q: shape"),
        (att, dict(out=rows(nq, n=3)), ValueError, "^out: shape"),
        (att, dict(out=rows(nq, dt=torch.float16)), TypeError, "^out"),
        (att, dict(q=rows(nq, dt=torch.float16), out=rows(
            nq, dt=torch.float16)), TypeError, "over a bfloat16 cache"),
        (att, dict(q=rows(nq, dt=torch.float32)), TypeError, "^q: "),
        (att, dict(lse=on(torch.zeros(b * m, nq, dtype=bf))), TypeError,
         "lse"),
        (att, dict(lse=on(torch.zeros(b * m, nq + 1))), ValueError, "lse"),
        (att, dict(ws=On(torch.zeros(1 << 20, dtype=torch.uint8), 1)),
         ValueError, "^ws"),
    ]
    for calls, kw, kind, words in cases:
        a = dict(base, **kw)
        if "move" in calls:
            for fn in (lambda: tp.kv_cache_write(
                    a["k"], a["v"], a["cache"], a["table"], a["lens"],
                    start=a["start"]), lambda: tp.kv_cache_read(
                    a["cache"], a["table"], a["lens"], a["k"], a["v"],
                    start=a["start"])):
                with pytest.raises(kind, match=words):
                    fn()
        if "attend" in calls:
            with pytest.raises(kind, match=words):
                tp.attn_decode(a["q"], a["cache"], a["table"], a["lens"],
                               a["out"], lse=a["lse"], ws=a["ws"])
    with pytest.raises(ValueError, match="not on a GPU"):
        tp.kv_cache_write(rows().t, rows().t, [t if t is None else t.t for t in
                                               cache()], base["table"].t,
                          base["lens"].t)


def test_oracles_step_is_the_layers_attention(tp):
    # operands that E4M3 holds exactly leave only the bf16 roundings: the
    # step's output is the attention oracle's last row through Wo
    rng = np.random.default_rng(6)
    h, n_q, n_kv, d, page = 16, 4, 2, 64, 4
    n = 5
    x = rng.integers(-1, 2, (n, h)).astype(np.float64)
    x[:, 0] = 1.0
    W = {k: rng.integers(-1, 2, s).astype(np.float64) for k, s in
         (("Wq", (n_q * d, h)), ("Wk", (n_kv * d, h)), ("Wv", (n_kv * d, h)),
          ("Wo", (h, n_q * d)))}
    pools = [np.full((3, page, n_kv, d), np.nan) for _ in range(2)]
    table = np.array([[2, 0]])
    ys = []
    for t in range(n):
        # eps and gamma that make the norm's factor a power of two
        rms = np.mean(x[t] ** 2)
        eps = 1.0 - rms
        _, Z = okv.step(x[t:t + 1], None, np.ones(h), W, (*pools, False),
                        table, [t + 1], n_q, d, eps)
        ys.append(x[t])
    f = oracle.attention_forward(np.stack(ys), W["Wq"], W["Wk"], W["Wv"],
                                 np.eye(n_q * d), b=1, s=n, n_q=n_q,
                                 n_kv=n_kv, d=d)
    got = Z[0]
    # O once to bf16 and once to codes: 2^-8 and 2^-4 of its elements at most
    want = f["Out"][-1] @ W["Wo"].T
    slack = (2.0 ** -4 + 2.0 ** -7) * np.abs(f["Out"][-1]) @ np.abs(W["Wo"]).T
    assert (np.abs(got - want) <= slack + 1e-9).all()
    # whole numbers but for the scales' fp32 rounding, 2·2^-24 of 16 terms
    for t in range(n):
        assert np.allclose(pools[0][table[0][t // page], t % page],
                           (W["Wk"] @ x[t]).reshape(n_kv, d), rtol=0,
                           atol=16 * 2.0 ** -23)


@pytest.mark.parametrize("args", [
    (0, 256, 2, 1), (1, 252, 2, 1), (1, 16392, 2, 1), (1, 256, 3, 2),
    (1, 256, 2, 1, 96), (1, 256, 4, 2, 128, 4), (1, 256, 2, 2, 64, 2)])
def test_attention_block_refuses_sizes(args):
    from megatron_tensor_transformer_gate_gb300.blocks import \
        TPBlockFP8Attention
    with pytest.raises(ValueError):
        TPBlockFP8Attention(*args, device="cpu")


def test_attention_blocks_weights_that_failed_to_load_are_not_used(tp):
    from megatron_tensor_transformer_gate_gb300.blocks import \
        TPBlockFP8Attention
    blk = TPBlockFP8Attention(2, 256, 2, 1, device="cpu")
    W = [torch.zeros(256, 256), torch.zeros(128, 256), torch.zeros(128, 256),
         torch.zeros(256, 256)]
    with pytest.raises(ValueError, match="Wv"):
        blk.load_weights(W[0], W[1], W[0], W[3])
    with pytest.raises(ValueError, match="not on a GPU"):
        blk.load_weights(*W)
    with pytest.raises(RuntimeError, match="load_weights"):
        blk.forward(torch.zeros(2, 256), torch.ones(256), None, None, None)


def test_attention_block_refuses_another_batch():
    """A table of one sequence for two rows is not one with two new tokens."""
    from megatron_tensor_transformer_gate_gb300.blocks import \
        TPBlockFP8Attention
    blk = TPBlockFP8Attention(2, 256, 2, 1, device="cpu")
    blk.weights = ((None, None), (None, None))
    lens = torch.ones(1, dtype=torch.int32)
    for b in (1, 4):
        with pytest.raises(ValueError, match="2 sequences"):
            blk.forward(torch.zeros(2, 256), torch.ones(256),
                        (None, None, None, None),
                        torch.zeros(b, 3, dtype=torch.int32), lens)
