"""Every form of the block-scaled product is reached: tiles, parts of K, groups
of scales, capture and streams, with the form that a case is meant for asserted.
Bounds: tests/test_gpu_fp8_block.py."""

import numpy as np
import pytest
import torch

from test_fp8_block_forms_host import FORMS
from test_gpu_fp8_block import GROUPS, activation, check_product, operand, room

pytestmark = pytest.mark.gpu

WIDE = (1080, 4330, 2600)   # 85 tiles: nine of 76 clusters have two; 21 blocks


def form(tp, M, N, K, group):
    return tp.gemm_fp8_block_form(M, N, K, GROUPS[group])[0]


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("gb", ["row", "block"])
@pytest.mark.parametrize("M,N,K,want", [f[:3] + (f[4],) for f in FORMS
                                        if f[1] * f[2] < 2 ** 25])
def test_form(tp, M, N, K, want, gb, out):
    assert tp.gemm_fp8_block_form(M, N, K, GROUPS[gb]) == want
    qa, sa = operand(tp, M, K, "row", M + K)
    qb, sb = operand(tp, N, K, gb, N + K)
    C = torch.full((M, N), float("nan"), dtype=out, device="cuda")
    tp.gemm_fp8_block(qa, sa, qb, sb, C)
    tp.device_status()
    check_product(C, qa, sa, qb, sb, f"{M}x{N}x{K} {want}")


def documented_sum(terms, form, split):
    """The K blocks' sums added in fp32 in the order that the header gives."""
    n = len(terms)
    if form == "thin":
        parts = [range(j, n, 8) for j in range(8)]
    else:
        parts = [range(n * j // split, n * (j + 1) // split)
                 for j in range(split)]
    sums = []
    for p in parts:
        v = np.float32(0)
        for b in p:
            v = np.float32(v + terms[b])
        sums.append(v)
    total = np.float32(0)
    for v in sums:
        total = np.float32(total + v)
    return total


@pytest.mark.parametrize("M,N,K", [(1, 100, 5000), (3, 100, 1), (8, 64, 1290),
                                   (9, 100, 4999), (37, 100, 900),
                                   (280, 3300, 2600), WIDE])
def test_order_of_the_blocks_sums(tp, M, N, K):
    # one product of 1·1 a block, so that its sum is the two scales' product
    name, _, split = tp.gemm_fp8_block_form(M, N, K, GROUPS["block"])
    nb = (K + 127) // 128
    qa, sa = tp.fp8_block_empty(M, K)
    qb, sb = tp.fp8_block_empty(N, K, GROUPS["block"])
    for q in (qa, qb):
        q.view(torch.uint8).zero_()
        q.view(torch.uint8)[:, ::128] = 0x38          # 1.0
    rng = np.random.default_rng(K)
    s = (rng.standard_normal(nb) * 10.0 ** rng.integers(-3, 4, nb)
         ).astype(np.float32)
    sa.copy_(torch.from_numpy(s).cuda()[:, None].expand_as(sa))
    sb.fill_(1.0)
    C = torch.empty((M, N), dtype=torch.float32, device="cuda")
    tp.gemm_fp8_block(qa, sa, qb, sb, C)
    want = documented_sum(s, name, split)
    assert bool((C == float(want)).all()), (name, split, want, C[0, 0])


@pytest.mark.parametrize("gb", ["row", "block"])
def test_wide_with_block_scaled_a(tp, gb):
    M, N, K = WIDE
    assert form(tp, M, N, K, gb) == "wide"
    qa, sa = operand(tp, M, K, "block", 1)
    qb, sb = operand(tp, N, K, gb, 2)
    C = torch.empty((M, N), dtype=torch.float32, device="cuda")
    tp.gemm_fp8_block(qa, sa, qb, sb, C)
    tp.device_status()
    check_product(C, qa, sa, qb, sb, "block-scaled A")


@pytest.mark.parametrize("gb", ["row", "block"])
def test_wide_with_nan_and_infinite_scales(tp, gb):
    M, N, K = WIDE
    assert form(tp, M, N, K, gb) == "wide"
    x, w = activation(M, K, 7), activation(N, K, 8)
    x[700, 130] = float("nan")
    w[4329, 2599] = float("inf")
    qa, sa = room(tp, M, K)
    qb, sb = room(tp, N, K, GROUPS[gb])
    tp.quantize_fp8_block(x, qa, sa)
    tp.quantize_fp8_block(w, qb, sb)
    C = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    tp.gemm_fp8_block(qa, sa, qb, sb, C)
    tp.device_status()
    poisoned = slice(4329, None) if gb == "row" else slice(4329 // 128 * 128,
                                                           None)
    bad = torch.isnan(C)
    assert bool(bad[700].all()) and bool(bad[:, poisoned].all())
    bad[700], bad[:, poisoned] = False, False
    assert not bool(bad.any())


@pytest.mark.parametrize("gb", ["row", "block"])
def test_wide_captured_and_replayed_next_to_an_eager_one(tp, gb):
    M, N, K = WIDE
    assert form(tp, M, N, K, gb) == "wide"
    qa, sa = operand(tp, M, K, "row", 1)
    qb, sb = operand(tp, N, K, gb, 2)
    C = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    E = torch.empty_like(C)
    tp.gemm_fp8_block(qa, sa, qb, sb, C)      # the kernel has run once
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tp.gemm_fp8_block(qa, sa, qb, sb, C)
    side = torch.cuda.Stream()
    for seed in (11, 12):
        tp.quantize_fp8_block(activation(M, K, seed), qa, sa)
        C.zero_(), E.zero_()
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        with torch.cuda.stream(side):
            tp.gemm_fp8_block(qa, sa, qb, sb, E)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        tp.device_status()
        check_product(C, qa, sa, qb, sb, "replayed")
        assert torch.equal(C, E)
