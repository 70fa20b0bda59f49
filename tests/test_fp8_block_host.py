"""Block-scaled E4M3 without a GPU: pins of its oracle, and the refusals of
the C entry points and of the Python binding (no call here launches)."""

import ctypes

import numpy as np
import pytest
import torch

import oracle
from oracle import fp8 as ofp8
from oracle import fp8_block as ob

FAKE = ctypes.c_void_p(0x100000)   # an aligned address never dereferenced
ODD = ctypes.c_void_p(0x100001)
I64 = ctypes.c_int64
NULL, SHAPE, DTYPE, ARG = 1, 2, 3, 8


# ------------------------------------------------------------------ oracle --
def test_scales_of_hand_worked_blocks():
    x = np.zeros((2, 130), np.float32)
    x[0, 3], x[0, 129], x[1, 7] = -7.0, 14.0, 2.0 ** -130
    q, s = ob.quantize(x, "row")
    assert s.shape == (2, 2)
    assert s[0, 0] == np.float32(7.0) / np.float32(448.0) == 2.0 ** -6
    assert s[1, 0] == 2.0 ** -5
    assert s[0, 1] == np.float32(2.0 ** -100) / np.float32(448)   # the floor
    assert s[1, 1] == 1.0                                         # all zero
    v = ob.dequantize(q, s)
    assert v[0, 3] == -7.0 and v[0, 129] == 14.0
    assert v[1, 7] == 0.0                       # 448·2^-30 rounds to nothing
    qb, sb = ob.quantize(x, "block")
    assert sb.shape == (2, 1) and sb[0, 0] == 2.0 ** -6 and \
        sb[1, 0] == 2.0 ** -5


@pytest.mark.parametrize("group", ["row", "block"])
def test_a_value_is_within_half_a_step(group):
    rng = np.random.default_rng(5)
    x = (rng.standard_normal((150, 300)) *
         np.exp(2 * rng.standard_normal((150, 1)))).astype(np.float32)
    q, s = ob.quantize(x, group)
    step = np.maximum(np.abs(x) * 2.0 ** -4,
                      ob.expand(s, *x.shape) * 2.0 ** -10)
    # three fp32 roundings (r, x·r, s) beside E4M3's
    assert (np.abs(ob.dequantize(q, s) - x) <= step * (1 + 2.0 ** -20)).all()


def test_block_group_of_a_transpose_is_the_transpose():
    x = np.random.default_rng(6).standard_normal((200, 300)).astype(np.float32)
    q, s = ob.quantize(x, "block")
    qt, st = ob.quantize(x.T, "block")
    assert (qt == q.T).all() and (st == s.T).all()


def test_gemm_sums_blocks_of_128():
    rng = np.random.default_rng(7)
    qa, sa = ob.quantize(rng.standard_normal((5, 300)), "row")
    qb, sb = ob.quantize(rng.standard_normal((140, 300)), "block")
    c, _ = ob.gemm(qa, sa, qb, sb)
    a, b = ofp8.e4m3_decode(qa), ofp8.e4m3_decode(qb)
    want = np.zeros((5, 140))
    for kb in range(3):
        k = slice(kb * 128, kb * 128 + 128)
        for n in range(140):
            want[:, n] += a[:, k] @ b[n, k] * sa[kb] * float(sb[kb, n // 128])
    assert np.allclose(c, want, rtol=1e-12, atol=1e-12)


def test_swiglu_matches_the_mlp_oracle_and_differences():
    rng = np.random.default_rng(8)
    gu = rng.standard_normal((4, 12))
    assert np.allclose(ob.swiglu(gu), oracle.silu(gu[:, :6]) * gu[:, 6:],
                       rtol=1e-14)
    dA = rng.standard_normal((4, 6))
    grad, e = ob.swiglu_grad(dA, gu), 1e-6
    for i in range(4):
        for j in range(12):
            d = np.zeros_like(gu)
            d[i, j] = e
            num = ((ob.swiglu(gu + d) - ob.swiglu(gu - d)) * dA).sum() / (2 * e)
            assert abs(num - grad[i, j]) <= 1e-8


# ---------------------------------------------------------------- refusals --
def quantize(tp, dtype=1, group=0, rows=200, cols=300, x=FAKE, ldx=300,
             q=FAKE, ldq=304, s=FAKE, lds=200, qt=None, ldqt=0, st=None,
             ldst=0):
    return tp.lib().tp_quantize_fp8_block(dtype, group, rows, cols, x, ldx, q,
                                          ldq, s, lds, qt, ldqt, st, ldst,
                                          None)


def test_quantize_refusals(tp):
    assert quantize(tp, dtype=2) == DTYPE
    assert quantize(tp, group=2) == DTYPE
    assert quantize(tp, x=None) == NULL
    assert quantize(tp, q=None) == NULL                 # no output at all
    assert quantize(tp, s=None) == NULL
    assert quantize(tp, rows=0) == SHAPE
    assert quantize(tp, cols=0) == SHAPE
    assert quantize(tp, rows=1 << 31, lds=1 << 31) == SHAPE
    # 2^23 · 2^9 tiles of 128×128
    assert quantize(tp, rows=1 << 30, cols=1 << 16, ldx=1 << 16, ldq=1 << 16,
                    lds=1 << 30) == SHAPE
    assert quantize(tp, ldx=299) == SHAPE
    assert quantize(tp, ldq=300) == SHAPE               # not 16 bytes
    assert quantize(tp, ldq=288) == SHAPE               # < cols
    assert quantize(tp, lds=199) == SHAPE
    assert quantize(tp, group=1, lds=1) == SHAPE        # two row blocks
    assert quantize(tp, q=ctypes.c_void_p(0x100008)) == ARG
    assert quantize(tp, s=ctypes.c_void_p(0x100002)) == ARG
    assert quantize(tp, x=ODD) == ARG
    assert quantize(tp, dtype=0, x=ctypes.c_void_p(0x100002)) == ARG
    assert quantize(tp, qt=FAKE, ldqt=208, st=None, ldst=300) == NULL
    assert quantize(tp, qt=FAKE, ldqt=200, st=FAKE, ldst=300) == SHAPE
    assert quantize(tp, qt=FAKE, ldqt=208, st=FAKE, ldst=299) == SHAPE
    assert quantize(tp, q=None, s=None, qt=ODD, ldqt=208, st=FAKE,
                    ldst=300) == ARG


def test_swiglu_refusals(tp):
    L = tp.lib()

    def fwd(T=4, f=100, gu=FAKE, ldgu=200, q=FAKE, ldq=112, s=FAKE, lds=4,
            qt=None, ldqt=0, st=None, ldst=0):
        return L.tp_swiglu_fp8_fwd(T, f, gu, ldgu, q, ldq, s, lds, qt, ldqt,
                                   st, ldst, None)

    def bwd(T=4, f=100, da=FAKE, ldda=100, gu=FAKE, ldgu=200, q=FAKE, ldq=208,
            s=FAKE, lds=4, qt=None, ldqt=0, st=None, ldst=0):
        return L.tp_swiglu_fp8_bwd(T, f, da, ldda, gu, ldgu, q, ldq, s, lds,
                                   qt, ldqt, st, ldst, None)

    assert fwd(gu=None) == NULL and bwd(gu=None) == NULL
    assert bwd(da=None) == NULL
    assert fwd(q=None) == NULL and bwd(q=None) == NULL
    assert fwd(T=0) == SHAPE and bwd(T=0) == SHAPE
    assert fwd(f=0) == SHAPE and bwd(f=0) == SHAPE
    assert bwd(f=1 << 62) == SHAPE and fwd(f=1 << 62) == SHAPE
    assert fwd(ldgu=199) == SHAPE and bwd(ldgu=199) == SHAPE
    assert bwd(ldda=99) == SHAPE
    assert bwd(ldq=192) == SHAPE                # codes of [dG | dU]: 2f columns
    assert fwd(lds=3) == SHAPE
    assert fwd(gu=ODD) == ARG and bwd(da=ODD) == ARG


def test_norm_refusals(tp):
    L = tp.lib()

    def norm(T=4, h=100, x=FAKE, r=FAKE, g=FAKE, x1=FAKE, y=None, rstd=FAKE,
             q=FAKE, ldq=112, s=FAKE, lds=4):
        return L.tp_add_rmsnorm_fp8_fwd(T, h, 1e-5, x, r, g, x1, y, rstd, q,
                                        ldq, s, lds, None)

    assert norm(x=None) == NULL and norm(g=None) == NULL
    assert norm(rstd=None) == NULL and norm(q=None) == NULL
    assert norm(x1=None) == NULL                # a sum has to go somewhere
    assert norm(T=0) == SHAPE and norm(h=0) == SHAPE
    assert norm(h=16385, ldq=16400) == SHAPE
    assert norm(ldq=100) == SHAPE and norm(lds=3) == SHAPE
    assert norm(y=ODD) == ARG
    assert norm(rstd=ctypes.c_void_p(0x100002)) == ARG


def test_gemm_refusals(tp):
    L = tp.lib()

    def gemm(M=5, N=200, K=300, qa=FAKE, lda=304, sa=FAKE, ldsa=5, ag=0,
             qb=FAKE, ldb=304, sb=FAKE, ldsb=2, bg=1, od=1, C=FAKE, ldc=200):
        return L.tp_gemm_fp8_block(M, N, K, qa, lda, sa, ldsa, ag, qb, ldb,
                                   sb, ldsb, bg, od, C, ldc, None)

    assert gemm(od=2) == DTYPE and gemm(ag=3) == DTYPE and gemm(bg=-1) == DTYPE
    for k in ("qa", "sa", "qb", "sb", "C"):
        assert gemm(**{k: None}) == NULL, k
    for k in ("M", "N", "K"):
        assert gemm(**{k: 0}) == SHAPE, k
        assert gemm(**{k: -1}) == SHAPE, k
    assert gemm(lda=300) == SHAPE and gemm(ldb=288) == SHAPE
    assert gemm(ldsa=4) == SHAPE and gemm(ldsb=1) == SHAPE
    assert gemm(bg=0) == SHAPE                  # 200 row scales in rows of 2
    assert gemm(ldc=199) == SHAPE
    assert gemm(qa=ctypes.c_void_p(0x100008)) == ARG
    assert gemm(C=ODD) == ARG
    assert gemm(od=0, C=ctypes.c_void_p(0x100002)) == ARG


def test_binding_refuses_what_the_c_call_cannot_see(tp):
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="not on a GPU"):
        tp.quantize_fp8_block(x, *tp.fp8_block_empty(4, 256, device="cpu"))
    with pytest.raises(ValueError, match="columns"):
        tp._matrix(x.t(), "x")
    q, s = tp.fp8_block_empty(200, 300, tp.FP8_BLOCK, device="cpu")
    assert q.shape == (200, 300) and q.stride() == (304, 1)
    assert s.shape == (3, 2)
    with pytest.raises(TypeError, match="bfloat16"):
        tp._bf16(x.float(), "x")
    with pytest.raises(ValueError, match="shape"):
        tp._bf16(x, "x", (4, 255))
