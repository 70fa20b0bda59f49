"""GPU parity of the block-scaled E4M3 operators against their 64-bit oracle.

Tolerances, by arithmetic:
* quantization of given values: codes and scales equal, every step being one
  IEEE fp32 operation or one E4M3 rounding;
* codes of a computed value v (SwiGLU, norm), read back as q·s: half an E4M3
  step, max(2^-4·|v|, 2^-10·s), for the device's own value v'; v' differs from
  v by ε·|v| with ε below 2^-18 for the norm (rsqrtf 2 ulp, three products)
  and below 2^-16 of the gate's and up's product for SwiGLU (an exponential of
  an argument up to 20: 2^-18, a division, four products), so the bound is
  taken with that much more; a scale is within ε of the exact one;
* the product: rounding of the output (2^-8 relative for bf16, 2^-24 for fp32)
  plus fp32 accumulation, (64 + 8 + nb)·2^-24 of Σ|a||b|: 128 products aligned
  to 2^-25 of the largest, four partial sums of a block truncated at 2^-23,
  and two roundings (sa·sb and the addition) for each of the nb blocks, the
  addition on a running sum that is itself below Σ|a||b|.
"""

import numpy as np
import pytest
import torch

from oracle import fp8_block as ob

pytestmark = pytest.mark.gpu

GROUPS = {"row": 0, "block": 1}


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def codes(q):
    return q.contiguous().view(torch.uint8).cpu().numpy()


def activation(rows, cols, seed, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, cols, generator=g)
    x *= torch.exp(torch.randn(rows, 1, generator=g))
    return x.to(dtype).cuda()


def room(tp, rows, cols, group=0, fill=0xAA):
    """A quantized matrix's room whose bytes, padding included, are `fill`."""
    q, s = tp.fp8_block_empty(rows, cols, group)
    q._base.view(torch.uint8).fill_(fill)
    s.fill_(-1.0)
    return q, s


def padding_kept(q, fill=0xAA):
    pad = q._base.view(torch.uint8)[:, q.shape[1]:]
    return bool((pad == fill).all())


def same_codes(q, s, want, what):
    wq, ws = want
    np.testing.assert_array_equal(s.cpu().numpy(), ws, err_msg=what)
    got = codes(q)
    bad = np.argwhere(got != wq)
    assert len(bad) == 0, f"{what}: {len(bad)} codes differ, e.g. {bad[:4]}"
    assert padding_kept(q), what


# ---------------------------------------------------------------- quantize --
SHAPES = [(1, 1), (1, 8), (1, 4096), (3, 130), (7, 129), (128, 128),
          (129, 257), (127, 1000), (300, 12), (777, 1000), (260, 384),
          (2500, 4100)]       # more tiles than four for each SM


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("group", ["row", "block"])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_quantize_bit_exact(tp, rows, cols, group, dtype):
    x = activation(rows, cols, rows * 31 + cols, dtype)
    g = GROUPS[group]
    q, s = room(tp, rows, cols, g)
    qt, st = room(tp, cols, rows, g)
    tp.quantize_fp8_block(x, q, s, qt, st)
    tp.device_status()
    xf = x.float().cpu().numpy()
    same_codes(q, s, ob.quantize(xf, group), "codes")
    same_codes(qt, st, ob.quantize(xf.T, group), "transpose")
    # each alone gives the same
    for kw in (dict(q=room(tp, rows, cols, g)), dict(qt=room(tp, cols, rows,
                                                             g))):
        a = {k: v[0] for k, v in kw.items()}
        a.update({"s" if k == "q" else "st": v[1] for k, v in kw.items()})
        tp.quantize_fp8_block(x, **a)
        for k, v in kw.items():
            other, os = (q, s) if k == "q" else (qt, st)
            assert torch.equal(v[0].view(torch.uint8),
                               other.view(torch.uint8))
            assert torch.equal(v[1], os)


@pytest.mark.parametrize("off", [1, 4, 8])
def test_quantize_column_slice(tp, off):
    # rows that start off 16 bytes, and a pitch that is not a multiple of 16
    big = activation(70, 301, 5)
    x = big[:, off:off + 200]
    q, s = room(tp, 70, 200)
    qt, st = room(tp, 200, 70)
    tp.quantize_fp8_block(x, q, s, qt, st)
    xf = x.float().cpu().numpy()
    same_codes(q, s, ob.quantize(xf, "row"), "codes")
    same_codes(qt, st, ob.quantize(xf.T, "row"), "transpose")


def test_quantize_zero_tiny_and_halfway_blocks(tp):
    x = torch.zeros(4, 512)
    x[1, 0] = 2.0 ** -126                     # below the floor
    x[1, 200] = -(2.0 ** -99)                 # above it
    x[2, :16] = 448.0 * torch.arange(16) / 16
    x[2, 128:128 + 15] = torch.tensor([448.0] + [17.0 + 2 * i
                                                 for i in range(14)])
    x[3, 384:] = -3.0e38
    x = x.to(torch.bfloat16)
    q, s = room(tp, 4, 512)
    tp.quantize_fp8_block(x.cuda(), q, s)
    same_codes(q, s, ob.quantize(x.float().numpy(), "row"), "codes")


@pytest.mark.parametrize("group", ["row", "block"])
def test_quantize_nan_keeps_its_place_and_inf_poisons_its_block(tp, group):
    x = activation(130, 300, 6)
    clean = x.float().cpu().numpy()
    x[3, 5] = float("nan")
    x[129, 299] = float("-inf")
    q, s = room(tp, 130, 300, GROUPS[group])
    qt, st = room(tp, 300, 130, GROUPS[group])
    tp.quantize_fp8_block(x, q, s, qt, st)
    clean[3, 5] = 0.0                         # a NaN does not enter amax
    for got, scale, ref, bad_at in ((q, s, clean, (129, 299)),
                                    (qt, st, clean.T, (299, 129))):
        wq, ws = ob.quantize(ref, group)
        at = (3, 5) if got is q else (5, 3)
        c, sc = codes(got), scale.cpu().numpy()
        assert c[at] & 0x7F == 0x7F
        e = ob.expand(sc, *c.shape)
        poisoned = ~np.isfinite(e)
        kb = bad_at[1] // 128
        n = min(128, c.shape[1] - kb * 128) * (1 if group == "row" else
                                               c.shape[0] - 128
                                               if c.shape[0] == 130 else
                                               c.shape[0] - 256)
        assert poisoned[bad_at] and poisoned.sum() == n
        keep = ~poisoned
        keep[at] = False
        assert (c[keep] == wq[keep]).all()
        with np.errstate(invalid="ignore"):
            v = got.float().cpu().numpy() * e
        assert np.isnan(v[poisoned]).all()


# --------------------------------------------------- codes of computed values --
def close_codes(q, s, v, slack, what, mag=None):
    """q·s is the E4M3 rounding of a value within slack·mag of v."""
    mag = np.abs(v) if mag is None else mag
    sc = s.cpu().numpy().astype(np.float64)
    big = ob.block_amax(mag, "row") / 448.0
    amax = ob.block_amax(v.astype(np.float32), "row").astype(np.float64)
    ws = np.where(amax == 0, 1.0, np.maximum(amax, 2.0 ** -100) / 448.0)
    assert (np.abs(sc - ws) <= slack * np.maximum(big, ws) + 2.0 ** -140
            ).all(), what + " scales"
    e = ob.expand(sc, *v.shape)
    got = f64(q) * e
    tol = np.maximum(2.0 ** -4 * np.abs(v), 2.0 ** -10 * e) * (1 + 2 * slack)
    assert (np.abs(got - v) <= tol + 2 * slack * mag).all(), what
    assert padding_kept(q), what


@pytest.mark.parametrize("T,f", [(1, 1), (1, 28), (1, 1376), (3, 130),
                                 (128, 128), (130, 264), (300, 77),
                                 (257, 344), (130, 256), (257, 384),
                                 (300, 12544), (1900, 2048),
                                 (2500, 4101), (2500, 4104)])
def test_swiglu_forward_and_backward(tp, T, f):
    gu = activation(T, 2 * f, T + f)
    gu[0, 0] = 120.0                          # σ = 1 and σ = 0 to the last bit
    gu[-1, f - 1] = -120.0
    dA = activation(T, f, T * f + 1) * 1e-3
    a, g = f64(gu), f64(dA)
    q, s = room(tp, T, f)
    qt, st = room(tp, f, T)
    tp.swiglu_fp8_fwd(gu, q, s, qt, st)
    v = ob.swiglu(a)
    close_codes(q, s, v, 2.0 ** -16, "A")
    close_codes(qt, st, v.T, 2.0 ** -16, "Aᵀ")
    q, s = room(tp, T, 2 * f)
    qt, st = room(tp, 2 * f, T)
    tp.swiglu_fp8_bwd(dA, gu, q, s, qt, st)
    tp.device_status()
    v = ob.swiglu_grad(g, a)
    # 1 + G(1 − σ) cancels near its zero: its error goes by what is added
    sig = 1.0 / (1.0 + np.exp(-a[:, :f]))
    mag = np.concatenate([np.abs(g * a[:, f:] * sig) *
                          (1.0 + np.abs(a[:, :f]) * (1.0 - sig)),
                          np.abs(v[:, f:])], axis=1)
    close_codes(q, s, v, 2.0 ** -16, "dGU", mag)
    close_codes(qt, st, v.T, 2.0 ** -16, "dGUᵀ", mag.T)


def test_swiglu_rows_of_a_wider_buffer(tp):
    T, f = 40, 96
    big = activation(T, 2 * f + 11, 3)
    gu = big[:, 3:3 + 2 * f]
    q, s = room(tp, T, f)
    tp.swiglu_fp8_fwd(gu, q, s)
    close_codes(q, s, ob.swiglu(f64(gu)), 2.0 ** -16, "A")


NORMS = [(T, h) for T in (1, 5) for h in (1, 7, 128, 130, 520, 1000, 1024,
                                          2048, 2056, 4100, 8192, 16384)]
# enough rows for each CTA to go round its ring of rows
NORMS += [(2500, 1032), (1900, 4096), (700, 4100), (1300, 8192), (700, 16384)]


@pytest.mark.parametrize("T,h", NORMS)
def test_add_rmsnorm(tp, T, h):
    x, r = activation(T, h, h), activation(T, h, h + 1) * 0.5
    gamma = (1.0 + 0.02 * torch.randn(h, generator=torch.Generator(
    ).manual_seed(h))).to(torch.bfloat16).cuda()
    x1, y = torch.empty_like(x), torch.empty_like(x)
    rstd = torch.empty(T, dtype=torch.float32, device="cuda")
    q, s = room(tp, T, h)
    tp.add_rmsnorm_fp8_fwd(x, r, gamma, x1, q, s, rstd, y=y, eps=1e-5)
    tp.device_status()
    assert torch.equal(x1, (x.float() + r.float()).to(torch.bfloat16))
    v = f64(x1)
    rs = 1.0 / np.sqrt((v * v).mean(axis=1) + 1e-5)
    np.testing.assert_allclose(rstd.cpu().numpy(), rs, rtol=2.0 ** -20)
    want = v * rs[:, None] * f64(gamma)
    close_codes(q, s, want, 2.0 ** -18, "codes")
    assert (np.abs(f64(y) - want) <= (2.0 ** -8 + 2.0 ** -18) *
            np.abs(want)).all()
    # without a residual: the norm of x itself, x1 written or not
    q2, s2 = room(tp, T, h)
    copy = torch.empty_like(x)
    tp.add_rmsnorm_fp8_fwd(x1, None, gamma, copy, q2, s2, rstd)
    assert torch.equal(copy, x1)
    assert torch.equal(q2.view(torch.uint8), q.view(torch.uint8))
    assert torch.equal(s2, s)
    tp.add_rmsnorm_fp8_fwd(x1, None, gamma, None, q2, s2, rstd)
    assert torch.equal(q2.view(torch.uint8), q.view(torch.uint8))


@pytest.mark.parametrize("T", [9, 2500])
@pytest.mark.parametrize("into", ["x", "r"])
def test_add_rmsnorm_in_place(tp, into, T):
    h = 1032
    x, r = activation(T, h, 1), activation(T, h, 2)
    gamma = torch.ones(h, dtype=torch.bfloat16, device="cuda")
    rstd = torch.empty(T, dtype=torch.float32, device="cuda")
    q, s = room(tp, T, h)
    x1 = torch.empty_like(x)
    tp.add_rmsnorm_fp8_fwd(x, r, gamma, x1, q, s, rstd)
    q2, s2 = room(tp, T, h)
    tp.add_rmsnorm_fp8_fwd(x, r, gamma, x if into == "x" else r, q2, s2, rstd)
    assert torch.equal(x if into == "x" else r, x1)
    assert torch.equal(q2.view(torch.uint8), q.view(torch.uint8))
    assert torch.equal(s2, s)


def test_add_rmsnorm_row_of_zeros_and_of_nan(tp):
    x = activation(3, 200, 4)
    x[1] = 0.0
    x[2, 17] = float("nan")
    gamma = torch.ones(200, dtype=torch.bfloat16, device="cuda")
    rstd = torch.empty(3, dtype=torch.float32, device="cuda")
    q, s = room(tp, 3, 200)
    tp.add_rmsnorm_fp8_fwd(x, None, gamma, None, q, s, rstd, eps=1e-5)
    c, sc = codes(q), s.cpu().numpy()
    assert (c[1] & 0x7F == 0).all() and (sc[:, 1] == 1.0).all()
    assert (c[2] & 0x7F == 0x7F).all() and np.isnan(rstd.cpu().numpy()[2])
    assert np.isfinite(f64(q[0:1])).all()


# ----------------------------------------------------------------- product --
def operand(tp, rows, k, group, seed):
    x = activation(rows, k, seed)
    q, s = room(tp, rows, k, GROUPS[group], fill=0x7F)   # NaN in the padding
    tp.quantize_fp8_block(x, q, s)
    return q, s


def check_product(C, qa, sa, qb, sb, what):
    c, mag = ob.gemm(codes(qa), sa.cpu().numpy(), codes(qb), sb.cpu().numpy())
    nb = sa.shape[0]
    half = 2.0 ** -8 if C.dtype == torch.bfloat16 else 2.0 ** -24
    tol = half * np.abs(c) + (1 + half) * (72 + nb) * 2.0 ** -24 * mag
    err = np.abs(C.double().cpu().numpy() - c)
    assert (err <= tol).all(), \
        f"{what}: {int((err > tol).sum())} of {err.size} off, worst " \
        f"{(err / np.maximum(tol, 1e-300)).max():.2f} of the bound"


PRODUCTS = [(1, 1, 1), (1, 16, 16), (1, 129, 130), (1, 1000, 4096),
            (8, 40, 2064), (7, 1030, 3333), (8, 17, 28700), (9, 130, 1300),
            (2, 256, 128), (5, 300, 77), (16, 136, 1000), (17, 520, 2100),
            (48, 384, 1376), (64, 256, 640), (65, 130, 260), (128, 128, 384),
            (129, 257, 513), (200, 1024, 512), (256, 256, 128),
            (300, 520, 208), (513, 384, 4096), (700, 260, 1100),
            (2600, 2400, 300), (2600, 2400, 40), (1000, 16, 512),
            (3000, 5, 300), (300, 5000, 128), (150, 700, 3000),
            # 256×256 tiles with rows of C off 16 bytes
            (2000, 2500, 700), (2000, 2501, 300), (2500, 2000, 40),
            (1500, 1450, 4100)]


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("ga,gb", [("row", "block"), ("row", "row")])
@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_product(tp, M, N, K, ga, gb, out):
    qa, sa = operand(tp, M, K, ga, M + K)
    qb, sb = operand(tp, N, K, gb, N + K + 1)
    C = torch.full((M, N), float("nan"), dtype=out, device="cuda")
    tp.gemm_fp8_block(qa, sa, qb, sb, C)
    tp.device_status()
    check_product(C, qa, sa, qb, sb, f"{M}x{N}x{K}")
    again = torch.empty_like(C)
    tp.gemm_fp8_block(qa, sa, qb, sb, again)
    assert torch.equal(C, again)              # no order of sums is left open


@pytest.mark.parametrize("gb", ["row", "block"])
@pytest.mark.parametrize("form,M,N,K", [
    ("wide", 1080, 4330, 2600),       # nine clusters go on to a second tile
    ("wide", 430, 4980, 9000), ("narrow", 40, 300, 28672),
    ("narrow", 128, 300, 28672), ("narrow", 300, 264, 16500)])
def test_product_whose_scales_go_round_their_ring(tp, form, M, N, K, gb):
    # K blocks that differ by powers of two: a block that met another's scales
    # would be off by far more than the bound
    def with_steps(rows, group, seed):
        q, s = operand(tp, rows, K, group, seed)
        g = torch.Generator().manual_seed(seed)
        s *= torch.exp2(torch.randint(-6, 7, (s.shape[0], 1), generator=g
                                      ).float()).cuda()
        return q, s

    assert tp.gemm_fp8_block_form(M, N, K, GROUPS[gb])[0] == form
    qa, sa = with_steps(M, "row", 21)
    qb, sb = with_steps(N, gb, 22)
    for out in (torch.float32, torch.bfloat16):
        C = torch.empty((M, N), dtype=out, device="cuda")
        tp.gemm_fp8_block(qa, sa, qb, sb, C)
        tp.device_status()
        check_product(C, qa, sa, qb, sb, f"{M}x{N}x{K}")


@pytest.mark.parametrize("ga,gb", [("block", "block"), ("block", "row")])
@pytest.mark.parametrize("M,N,K", [(3, 200, 300), (140, 270, 400),
                                   (600, 400, 900)])
def test_product_block_scaled_a(tp, M, N, K, ga, gb):
    qa, sa = operand(tp, M, K, ga, 1)
    qb, sb = operand(tp, N, K, gb, 2)
    C = torch.empty((M, N), dtype=torch.float32, device="cuda")
    tp.gemm_fp8_block(qa, sa, qb, sb, C)
    check_product(C, qa, sa, qb, sb, f"{M}x{N}x{K}")


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,N,K", [(3, 200, 300), (300, 270, 400),
                                   (2000, 2300, 200)])
@pytest.mark.parametrize("off", [0, 1, 8])
def test_product_into_a_slice_leaves_the_rest(tp, M, N, K, off, out):
    qa, sa = operand(tp, M, K, "row", 3)
    qb, sb = operand(tp, N, K, "block", 4)
    big = torch.full((M + 2, N + 21), 7.0, dtype=out, device="cuda")
    C = big[1:M + 1, off:off + N]
    tp.gemm_fp8_block(qa, sa, qb, sb, C)
    check_product(C, qa, sa, qb, sb, "slice")
    C.fill_(7.0)
    assert bool((big == 7.0).all())


@pytest.mark.parametrize("M,N", [(4, 200), (300, 400)])
def test_product_of_rows_and_columns_of_wider_matrices(tp, M, N):
    # operands with pitches of their own: rows of a longer matrix, columns
    # from a multiple of 128 on, with their scales
    qa, sa = operand(tp, M + 3, 800, "row", 5)
    qb, sb = operand(tp, N, 800, "row", 6)
    a, b = qa[2:2 + M, 256:600], qb[:, 256:600]
    sa, sb = sa[2:5, 2:2 + M], sb[2:5]
    C = torch.empty((M, N), dtype=torch.float32, device="cuda")
    tp.gemm_fp8_block(a, sa, b, sb, C)
    check_product(C, a, sa, b, sb, "wider")


@pytest.mark.parametrize("M,N", [(2, 130), (300, 400)])
def test_product_of_nan_and_infinite_scales(tp, M, N):
    x, w = activation(M, 300, 7), activation(N, 300, 8)
    x[1, 130] = float("nan")
    w[5, 299] = float("inf")
    qa, sa = room(tp, M, 300)
    qb, sb = room(tp, N, 300)
    tp.quantize_fp8_block(x, qa, sa)
    tp.quantize_fp8_block(w, qb, sb)
    C = torch.empty((M, N), dtype=torch.float32, device="cuda")
    tp.gemm_fp8_block(qa, sa, qb, sb, C)
    bad = torch.isnan(C)
    assert bool(bad[1].all()) and bool(bad[:, 5].all())
    bad[1], bad[:, 5] = False, False
    assert not bool(bad.any())


def test_products_on_a_side_stream_and_in_a_graph(tp):
    # decode-sized and wide products captured together, replayed twice on new
    # inputs, next to eager calls of the same kernels on another stream
    small = operand(tp, 3, 512, "row", 1) + operand(tp, 384, 512, "block", 2)
    wide = operand(tp, 300, 512, "row", 3) + operand(tp, 520, 512, "block", 4)
    cs = torch.empty((3, 384), dtype=torch.bfloat16, device="cuda")
    cw = torch.empty((300, 520), dtype=torch.float32, device="cuda")
    tp.gemm_fp8_block(*small, cs)
    tp.gemm_fp8_block(*wide, cw)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tp.gemm_fp8_block(*small, cs)
        tp.gemm_fp8_block(*wide, cw)
    side, es, ew = torch.cuda.Stream(), torch.empty_like(cs), \
        torch.empty_like(cw)
    for seed in (11, 12):
        tp.quantize_fp8_block(activation(3, 512, seed), small[0], small[1])
        tp.quantize_fp8_block(activation(300, 512, seed), wide[0], wide[1])
        cs.zero_(), cw.zero_()
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        with torch.cuda.stream(side):
            tp.gemm_fp8_block(*small, es)
            tp.gemm_fp8_block(*wide, ew)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        check_product(cs, *small, "graph, small")
        check_product(cw, *wide, "graph, wide")
        assert torch.equal(cs, es) and torch.equal(cw, ew)


@pytest.mark.parametrize("M", [1, 200])
def test_offsets_past_32_bits(tp, M):
    # 4.6 G elements: the last rows' codes, scales and products
    N, K, tail = 70000, 65536, 300
    gen = torch.Generator(device="cuda").manual_seed(9)
    w = torch.empty((N, K), dtype=torch.bfloat16, device="cuda")
    w.zero_()
    w[-tail:] = torch.randn((tail, K), generator=gen, device="cuda")
    q, s = tp.fp8_block_empty(N, K)
    tp.quantize_fp8_block(w, q, s)
    tp.device_status()
    wf = w[-tail:].float().cpu().numpy()
    del w
    wq, ws = ob.quantize(wf, "row")
    np.testing.assert_array_equal(s[:, -tail:].cpu().numpy(), ws)
    np.testing.assert_array_equal(codes(q[-tail:]), wq)
    qa, sa = operand(tp, M, K, "row", 1)
    C = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    tp.gemm_fp8_block(qa, sa, q, s, C)
    tp.device_status()
    assert not bool(C[:, :-tail].any())
    check_product(C[:, -tail:], qa, sa, q[-tail:], s[:, -tail:], "tail")


class NoFast:
    """Stands in for the CPython module: leaves every call to Python."""

    def __getattr__(self, name):
        return lambda *a: None


def test_both_ways_of_calling_agree(tp, monkeypatch):
    T, h = 5, 1000
    x, r, gu = activation(T, h, 1), activation(T, h, 2), activation(T, 2 * h, 3)
    gamma = torch.ones(h, dtype=torch.bfloat16, device="cuda")
    dA = activation(T, h, 4)
    w, ws = operand(tp, 300, h, "block", 5)

    def calls():
        out = []
        rstd = torch.empty(T, dtype=torch.float32, device="cuda")
        x1, y = torch.empty_like(x), torch.empty_like(x)
        q, s = room(tp, T, h)
        tp.add_rmsnorm_fp8_fwd(x, r, gamma, x1, q, s, rstd, y=y)
        C = torch.empty((T, 300), dtype=torch.bfloat16, device="cuda")
        tp.gemm_fp8_block(q, s, w, ws, C)
        out += [x1, y, rstd, q, s, C]
        for f, cols in ((lambda *a: tp.quantize_fp8_block(x, *a), h),
                        (lambda *a: tp.swiglu_fp8_fwd(gu, *a), h),
                        (lambda *a: tp.swiglu_fp8_bwd(dA, gu, *a), 2 * h)):
            both = room(tp, T, cols) + room(tp, cols, T)
            f(*both)
            out += both
        return out

    fast = calls()
    # the ordinary call is the module's: it returned a status, not None
    q, s = room(tp, T, h)
    assert tp._tpcall.quantize(x, q, s, None, None, None) == 0
    assert tp._tpcall.quantize(x, q, s, None, None,
                               torch.cuda.current_stream()) == 0
    for bad in ((x.cpu(), q, s), (x, q, None), (x, q[:, :-1], s),
                (x.half(), q, s), (x, q, s.double()), (x.t(), q, s), (1, q, s)):
        assert tp._tpcall.quantize(*bad, None, None, None) is None
    monkeypatch.setattr(tp, "_tpcall", NoFast())
    slow = calls()
    for a, b in zip(fast, slow):
        assert a.dtype == b.dtype
        v = torch.uint8 if a.element_size() == 1 else a.dtype
        assert torch.equal(a.view(v), b.view(v))
