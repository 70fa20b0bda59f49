"""The logical shards of TPBlockFP8MLP, each quantized and multiplied on its own,
against the block's whole tensors: the same codes and scales, and partial
products whose sum over the shards (g in forward, f in backward) is the fused
product's.

Bound of a sum: the fused product and the shards' together round as in
tests/test_gpu_fp8_block.py, (72 + nb)·2^-24 of Σ|a||b| for each of the two and
half a step of the stored bf16 result, the partial products' own rounding to
fp32 within the first."""

import numpy as np
import pytest
import torch

from oracle import fp8_block as ob
from test_gpu_fp8_block import codes
from test_gpu_fp8_block_mlp import run, tensors

pytestmark = pytest.mark.gpu


def same(pair, whole, cols, rows=None):
    """A shard's pair is the whole's columns (and rows of blocks)."""
    q, s = pair
    wq, ws = whole
    k = slice(cols.start // 128, -(-cols.stop // 128))
    wq, ws = wq[:, cols], ws[k]
    if rows is not None:
        wq = wq[rows]
        ws = ws[:, rows.start // 128:-(-rows.stop // 128)]
    assert torch.equal(q.view(torch.uint8), wq.view(torch.uint8))
    assert torch.equal(s, ws)


def within(total, fused, a, b):
    args = [x for q, s in (a, b) for x in (codes(q), s.cpu().numpy())]
    exact, mag = ob.gemm(*args)
    tol = 2.0 ** -8 * np.abs(exact) + 2.1 * (72 + a[1].shape[0]) * \
        2.0 ** -24 * mag
    err = np.abs(total - fused.double().cpu().numpy())
    assert (err <= tol).all(), (err / np.maximum(tol, 1e-300)).max()


@pytest.mark.parametrize("T,h,f,n", [(70, 256, 1024, 8), (300, 520, 768, 3),
                                     (5, 384, 512, 2)])
def test_each_shard_is_a_slice_of_the_whole(tp, T, h, f, n):
    _, m, d = run(tensors(T, h, f, 30 + n), T, h, f, n)
    (w1, w1t), (w2, w2t) = m.weights
    each = f // n
    Z = torch.empty((T, h), dtype=torch.float32, device="cuda")
    dY, g_sum, f_sum = torch.empty_like(Z), 0.0, 0.0
    x1, out = torch.empty_like(d["x"]), torch.empty_like(d["x"])
    m.forward(d["x"], d["gamma"], r=d["r"], out=out, x1=x1)

    def pair(rows, cols, group=tp.FP8_ROW):
        return tp.fp8_block_empty(rows, cols, group)

    for i in range(n):
        own = slice(i * each, (i + 1) * each)
        up = slice(f + own.start, f + own.stop)
        gate_up = torch.cat((d["W1"][own], d["W1"][up]))
        v1 = pair(2 * each, h, tp.FP8_BLOCK), pair(h, 2 * each, tp.FP8_BLOCK)
        tp.quantize_fp8_block(gate_up, *v1[0], *v1[1])
        v2 = pair(h, each, tp.FP8_BLOCK), pair(each, h, tp.FP8_BLOCK)
        tp.quantize_fp8_block(d["W2"][:, own], *v2[0], *v2[1])
        whole = slice(0, h)
        for part, of in ((slice(0, each), own), (slice(each, 2 * each), up)):
            same((v1[0][0][part], v1[0][1][:, part.start // 128:
                                            part.stop // 128]), w1, whole, of)
            same((v1[1][0][:, part], v1[1][1][part.start // 128:
                                              part.stop // 128]), w1t, of)
        same(v2[0], w2, own)
        same(v2[1], w2t, whole, own)

        gu = torch.cat((m.gu[:, own], m.gu[:, up]), dim=1)
        a, at = pair(T, each), pair(each, T)
        tp.swiglu_fp8_fwd(gu, *a, *at)
        same(a, m.a, own)
        assert torch.equal(at[0].view(torch.uint8),
                           m.at[0][own].view(torch.uint8))
        tp.gemm_fp8_block(*a, *v2[0], Z)
        g_sum = g_sum + Z.double().cpu().numpy()

        dgu = pair(T, 2 * each)
        tp.swiglu_fp8_bwd(m.da[:, own], gu, *dgu)
        k = each // 128
        same((dgu[0][:, :each], dgu[1][:k]), m.dgu, own)
        same((dgu[0][:, each:], dgu[1][k:]), m.dgu, up)
        tp.gemm_fp8_block(*dgu, *v1[1], dY)
        f_sum = f_sum + dY.double().cpu().numpy()
    tp.device_status()
    within(g_sum, out, m.a, w2)
    within(f_sum, m.dy, m.dgu, w1t)
