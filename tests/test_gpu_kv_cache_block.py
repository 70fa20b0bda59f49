"""The cache's operators as they are used together: TPBlockFP8Attention step by
step against the oracle, in front of a TPBlockFP8MLP, and after a prompt's
forward by TPAttention.

Each step is held to the oracle fed with what the device stored before it: Q, K,
V, O and Z are bf16 roundings of fp32 sums (2^-9 to 2^-8 relative, bound 1e-2),
what the cache takes is exact.

From end to end, codes amplify: where the value before them is off by ε (relative,
in the norm), one in Δ/ε of the codes moves by its step Δ, 2^-4 to 2^-3, which is
sqrt(ε·Δ) of the norm, 2^-1.5·sqrt(ε) at most; a rounding to bf16 likewise gives
sqrt(ε·2^-8).  Q, K and V differ in their last bf16 bit (2^-8) for a share of at
most 2^-5 of the elements (fp32 sums in another order): 2^-10.5.  Over a bf16
cache that moves the scores, of size 2 here, by 2^-9.5 and the weights, and with
them O, by as much; O rounded to bf16 is off by 2^-8.75, its codes and Z by
2^-5.85.  In a cache of codes one in 2^4 of the elements that differ moves by
2^-3: 2^-4.5·2^-3 = 2^-7.5 of K and V; K's moves the scores by 2^-6.5 and the
weights by as much, so that O is off by ε = 2^-6, its codes and Z by 2^-4.5."""

import numpy as np
import pytest
import torch

from oracle import fp8_block as ob
from oracle import kv_cache as okv
from megatron_tensor_transformer_gate_gb300 import inputs as I
from megatron_tensor_transformer_gate_gb300.blocks import (
    TPAttention, TPBlockFP8Attention, TPBlockFP8MLP)
from _kv_cache import HALF, page_table
from _parity import check_fro

pytestmark = pytest.mark.gpu
EPS = 1e-5
BF16 = torch.bfloat16


def weights(h, n_q, n_kv, d, seed, dtype=BF16):
    def n(shape, std, k):
        return I.normal(shape, std, seed + k, "cpu", dtype)
    return dict(Wq=n((n_q * d, h), 2 * h ** -0.5, 1),
                Wk=n((n_kv * d, h), h ** -0.5, 2),
                Wv=n((n_kv * d, h), h ** -0.5, 3),
                Wo=n((h, n_q * d), (n_q * d) ** -0.5, 4))


def gamma_of(h, seed):
    return I.normal((h,), 0.02, seed, "cpu", BF16, 1.0)


def check_stages(blk, W, cache, table, lens, Z, kind):
    """The last forward's steps, each against the oracle on the device's own
    input of it."""
    def value(q, s):
        return ob.dequantize(q.contiguous().view(torch.uint8).cpu().numpy(),
                             s.cpu().numpy())

    def deq(w):
        return ob.dequantize(*ob.quantize(w.float().numpy(), "block"))

    y = value(*blk.y)
    for name, got in (("Wq", blk.q), ("Wk", blk.k), ("Wv", blk.v)):
        check_fro(got.reshape(blk.T, -1), y @ deq(W[name]).T, name)
    pools = []
    for pool, scale, new in ((cache[0], cache[2], blk.k),
                             (cache[1], cache[3], blk.v)):
        new = new.float().cpu().numpy()
        if kind == "e4m3":
            codes = pool.view(torch.uint8).cpu().numpy()
            scale = scale.cpu().numpy()
            pools.append(okv.dequantize(codes, scale))
        else:
            pools.append(I.to_f64(pool))
        for row, i, p in okv.tokens(lens, blk.T):
            at = table[i][p // pool.shape[1]], p % pool.shape[1]
            if kind == "e4m3":
                q, s = okv.quantize(new[row])
                assert (codes[at] == q).all() and (scale[at] == s).all()
            else:
                assert (pools[-1][at] == new[row]).all()
    o, _ = okv.attend(I.to_f64(blk.q), *pools, table, lens, blk.d ** -0.5)
    check_fro(blk.o, o.reshape(blk.T, -1), "O")
    check_fro(Z, value(*blk.a) @ deq(W["Wo"]).T, "Z of the device's O")


@pytest.mark.parametrize("b,h,n_q,n_kv,d,n,new,kind,page,w_dtype", [
    (1, 256, 2, 1, 128, 1, 1, "bf16", 16, BF16),
    (3, 264, 8, 2, 128, 2, 1, "e4m3", 4, torch.float32),
    (5, 512, 4, 4, 64, 2, 2, "bf16", 7, BF16),
    (2, 1024, 8, 2, 128, 1, 4, "e4m3", 16, BF16)])
def test_steps(tp, b, h, n_q, n_kv, d, n, new, kind, page, w_dtype):
    W = weights(h, n_q, n_kv, d, 50 * b, w_dtype)
    gamma = gamma_of(h, 7)
    blk = TPBlockFP8Attention(b, h, n_q, n_kv, d, n, new=new, eps=EPS)
    blk.load_weights(**{k: v.cuda() for k, v in W.items()})
    lens = np.zeros(b, np.int64)
    idle = b - 1 if b > 2 else None          # a place without a sequence
    steps = 4
    table, pages = page_table([steps * new] * b, page,
                              np.random.default_rng(b))
    cache = tp.kv_cache_empty(pages, page, n_kv, d,
                              tp.FP8 if kind == "e4m3" else tp.BF16)
    for t in cache:
        if t is not None:
            t.view(torch.uint8).fill_(0xff) if t.element_size() == 1 \
                else t.fill_(float("nan"))
    dt = torch.from_numpy(table).cuda()
    dl = torch.zeros(b, dtype=torch.int32, device="cuda")
    pools = [np.full((pages, page, n_kv, d), np.nan) for _ in range(2)]
    o = {k: I.to_f64(v) for k, v in W.items()}
    for s in range(steps):
        x = I.normal((b * new, h), 1.0, 100 + s, "cpu", BF16)
        r = I.normal((b * new, h), 0.5, 200 + s, "cpu", BF16) if s % 2 else None
        lens += new
        if idle is not None:
            lens[idle] = 0
        dl.copy_(torch.from_numpy(lens))
        x1, Z = blk.forward(x.cuda(), gamma.cuda(), cache, dt, dl,
                            r=None if r is None else r.cuda())
        tp.device_status()
        w1, wZ = okv.step(I.to_f64(x), None if r is None else I.to_f64(r),
                          I.to_f64(gamma), o, (*pools, kind == "e4m3"), table,
                          lens, n_q, d, EPS)
        assert (I.to_f64(x1) == w1).all()
        if idle is not None:
            assert not Z[idle * new:].any()
        check_fro(Z, wZ, f"Z of step {s}",
                  2.0 ** -5.85 if kind == "bf16" else 2.0 ** -4.5)
        check_stages(blk, W, cache, table, lens, Z, kind)


def test_a_layer_that_generates_captured(tp):
    # attention and MLP block in one graph, replayed while the lengths grow,
    # against the same blocks called one by one
    b, h, f, n_q, n_kv, d = 4, 512, 768, 4, 2, 128
    W = {k: v.cuda() for k, v in weights(h, n_q, n_kv, d, 3).items()}
    W1 = I.normal((2 * f, h), h ** -0.5, 8, "cuda", BF16)
    W2 = I.normal((h, f), f ** -0.5, 9, "cuda", BF16)
    g1, g2 = gamma_of(h, 10).cuda(), gamma_of(h, 11).cuda()
    table = torch.randperm(16, generator=torch.Generator().manual_seed(1)) \
        .to(torch.int32).view(b, 4).cuda()

    class Layer:
        def __init__(self):
            self.attn = TPBlockFP8Attention(b, h, n_q, n_kv, d, eps=EPS)
            self.mlp = TPBlockFP8MLP(b, h, f, eps=EPS, train=False)
            self.attn.load_weights(**W)
            self.mlp.load_weights(W1, W2)
            self.cache = tp.kv_cache_empty(16, 8, n_kv, d, tp.FP8)
            self.lens = torch.zeros(b, dtype=torch.int32, device="cuda")
            self.x = torch.zeros(b, h, dtype=BF16, device="cuda")
            self.x1, self.z, self.x2, self.out = (
                torch.empty_like(self.x) for _ in range(4))

        def step(self):
            self.attn.forward(self.x, g1, self.cache, table, self.lens,
                              out=self.z)
            self.mlp.forward(self.x, g2, r=self.z, out=self.out, x1=self.x2)

    eager, held = Layer(), Layer()
    held.step()                      # every kernel once, with lengths of 0
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held.step()
    for s in range(32):
        x = I.normal((b, h), 1.0, 300 + s, "cuda", BF16)
        for L in (eager, held):
            L.x.copy_(x)
            L.lens += 1
        eager.step()
        graph.replay()
        assert torch.equal(eager.out, held.out), s
        assert torch.equal(eager.x2, held.x2), s
    tp.device_status()
    assert torch.isfinite(held.out).all()


@pytest.mark.parametrize("kind", ["f16", "e4m3"])
def test_after_a_prompts_forward(tp, kind):
    # K and V that the training attention saved go into the cache; the last
    # tokens' queries over it give what that forward gave for them
    b, s, h, n_q, n_kv, d, m = 3, 77, 256, 8, 2, 128, 2
    W = {k: v.cuda() for k, v in weights(h, n_q, n_kv, d, 13).items()}
    X = I.normal((b * s, h), 1.0, 14, "cuda", BF16)
    a = TPAttention(b, s, h, n_q, n_kv, d, 1)
    a.forward(X, W["Wq"], W["Wk"], W["Wv"], W["Wo"])
    S = a.saved()
    page, cols = 16, 5
    table = torch.randperm(b * cols, generator=torch.Generator()
                           .manual_seed(2)).to(torch.int32).view(b, cols) \
        .cuda()
    lens = torch.full((b,), s, dtype=torch.int32, device="cuda")
    cache = tp.kv_cache_empty(b * cols, page, n_kv, d,
                              tp.F16 if kind == "f16" else tp.FP8)
    K, V = (S[x].view(b * s, n_kv, d) for x in "KV")
    tp.kv_cache_write(K, V, cache, table, lens)
    q = S["Q"].view(b, s, n_q, d)[:, s - m:].reshape(b * m, n_q, d)
    out = torch.empty_like(q)
    lse = torch.empty(b * m, n_q, device="cuda")
    tp.attn_decode(q, cache, table, lens, out, lse=lse)
    back = torch.empty_like(K), torch.empty_like(V)
    tp.kv_cache_read(cache, table, lens, *back)
    tp.device_status()
    want = S["O"].view(b, s, n_q, d)[:, s - m:].reshape(b * m, n_q, d)
    wl = S["LSE"].view(b, n_q, s)[:, :, s - m:].permute(0, 2, 1) \
        .reshape(b * m, n_q)
    if kind == "f16":
        assert torch.equal(back[0], K) and torch.equal(back[1], V)
        # both round P to fp16 (2^-11 of Σ p|v| ≤ max|v|) and O to 16 bits,
        # the training forward to bf16
        bound = 2 * 2.0 ** -11 * V.abs().max().item()
        diff = (out.float() - want.float()).abs()
        assert (diff <= HALF[BF16] * want.float().abs() + bound).all()
        assert ((lse - wl).abs() <= 2.0 ** -10).all()
    else:
        # codes: K's half steps (2^-4) move a score by 2^-4·|x| at most, V's
        # an output by 2^-4 of the largest value
        assert ((back[1].float() - V.float()).abs() <=
                2.0 ** -4 * V.float().abs() +
                2.0 ** -10 * V.float().abs().amax(-1, keepdim=True)).all()
        check_fro(out, want.double().cpu().numpy(), "O over codes", 0.15)


def test_block_refuses(tp):
    for a in ((0, 256, 2, 1), (1, 252, 2, 1), (1, 256, 3, 2), (1, 256, 2, 1, 96),
              (1, 256, 2, 2, 64, 2), (1, 256, 4, 2, 128, 4)):
        with pytest.raises(ValueError):
            TPBlockFP8Attention(*a)
    blk = TPBlockFP8Attention(2, 256, 2, 1)
    cache = tp.kv_cache_empty(4, 8, 1, 128, tp.BF16)
    table = torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    lens = torch.ones(2, dtype=torch.int32, device="cuda")
    x = torch.zeros(2, 256, dtype=BF16, device="cuda")
    g = torch.ones(256, dtype=BF16, device="cuda")
    with pytest.raises(RuntimeError, match="load_weights"):
        blk.forward(x, g, cache, table, lens)
    W = {k: v.cuda() for k, v in weights(256, 2, 1, 128, 5).items()}
    with pytest.raises(ValueError, match="Wk"):
        blk.load_weights(W["Wq"], W["Wq"], W["Wv"], W["Wo"])
    blk.load_weights(**W)
    with pytest.raises(ValueError, match="k rows: shape"):   # of other heads
        blk.forward(x, g, tp.kv_cache_empty(4, 8, 2, 128, tp.BF16), table, lens)


def test_memory_made_in_a_call_is_of_its_stream(tp):
    from test_gpu_fp8_block_mlp import pool_of
    b, h, n_q, n_kv = 2, 256, 2, 1
    W = {k: v.cuda() for k, v in weights(h, n_q, n_kv, 128, 6).items()}
    x = I.normal((b, h), 1.0, 7, "cuda", BF16)
    r = I.normal((b, h), 1.0, 8, "cuda", BF16)
    g = gamma_of(h, 9).cuda()
    table = torch.arange(4, dtype=torch.int32, device="cuda").view(b, 2)
    lens = torch.ones(b, dtype=torch.int32, device="cuda")
    got = []
    side = torch.cuda.Stream()
    for stream in (None, side):
        blk = TPBlockFP8Attention(b, h, n_q, n_kv, eps=EPS)
        cache = tp.kv_cache_empty(4, 8, n_kv, 128, tp.FP8)
        torch.cuda.synchronize()
        blk.load_weights(**W, stream=stream)
        got.append(blk.forward(x, g, cache, table, lens, r=r, stream=stream))
        torch.cuda.synchronize()
    tp.device_status()
    for a, c in zip(*got):
        assert torch.equal(a, c)
        assert pool_of(c) == side.cuda_stream
