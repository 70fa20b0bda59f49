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
             q=FAKE, ldq=112, s=FAKE, lds=4, eps=1e-5):
        return L.tp_add_rmsnorm_fp8_fwd(T, h, eps, x, r, g, x1, y, rstd, q,
                                        ldq, s, lds, None)

    assert norm(x=None) == NULL and norm(g=None) == NULL
    assert norm(rstd=None) == NULL and norm(q=None) == NULL
    assert norm(x1=None) == NULL                # a sum has to go somewhere
    assert norm(T=0) == SHAPE and norm(h=0) == SHAPE
    assert norm(h=16385, ldq=16400) == SHAPE
    assert norm(ldq=100) == SHAPE and norm(lds=3) == SHAPE
    assert norm(y=ODD) == ARG
    assert norm(eps=-1e-5) == ARG and norm(eps=float("nan")) == ARG
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
    q, s = tp.fp8_block_empty(4, 256, device="cpu")
    with pytest.raises(ValueError, match="not on a GPU"):
        tp.quantize_fp8_block(x, q, s)
    with pytest.raises(ValueError, match="a matrix"):
        tp.quantize_fp8_block(x[0], q, s)
    w, ws = tp.fp8_block_empty(200, 300, tp.FP8_BLOCK, device="cpu")
    assert w.shape == (200, 300) and w.stride() == (304, 1)
    assert ws.shape == (3, 2)


class OnDevice:
    """A CPU tensor that says it is on device 0: the binding's checks read
    nothing of its storage."""

    def __init__(self, t):
        self.t = t

    def get_device(self):
        return 0

    is_cuda = True

    def __getattr__(self, k):
        return getattr(self.t, k)


def test_binding_checks_types_shapes_strides_and_devices(tp, monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)

    def on(*shape, dtype=torch.bfloat16):
        return OnDevice(torch.zeros(*shape, dtype=dtype))

    def pair(rows, cols, group=0):
        return tuple(OnDevice(t) for t in
                     tp.fp8_block_empty(rows, cols, group, device="cpu"))

    q, s = pair(4, 256)
    assert tp._fp8_pair(q, s, "q", 4, 256, 0)[1::2] == (256, 4)
    assert tp._fp8_pair(*pair(200, 300, 1), "q", 200, 300, 0)[3:] == (2, 1)
    # a single row: any stride, the two groups are one
    one = OnDevice(torch.zeros(3, 40, dtype=torch.uint8)[1:2, :33])
    assert tp._fp8_pair(one, pair(1, 33)[1], "q", 1, 33, 0)[1] == 48
    for args, kind, words in (
            ((q, s, "q", 4, 255, 0), ValueError, "shape"),
            ((q, None, "q", 4, 256, 0), ValueError, "without scales"),
            ((on(4, 256), s, "q", 4, 256, 0), TypeError, "E4M3"),
            ((q, on(2, 4), "q", 4, 256, 0), TypeError, "float32"),
            ((q, on(3, 4, dtype=torch.float32), "q", 4, 256, 0), ValueError,
             "scales"),
            ((q, on(2, 3, dtype=torch.float32), "q", 4, 256, 0), ValueError,
             "scales"),
            ((q, s, "q", 4, 256, 1), ValueError, "not cuda:1"),
            ((OnDevice(torch.zeros(256, 4, dtype=torch.uint8).t()), s, "q", 4,
              256, 0), ValueError, "adjacent")):
        with pytest.raises(kind, match=words):
            tp._fp8_pair(*args)
    with pytest.raises(ValueError, match="adjacent"):
        tp._matrix(OnDevice(torch.zeros(6, 4).t()), "x")
    with pytest.raises(ValueError, match="different groups"):
        tp._fp8_outs(200, 300, 0, *pair(200, 300, 0), *pair(300, 200, 1))
    with pytest.raises(ValueError, match="neither"):
        tp._fp8_outs(200, 300, 0, None, None, None, None)
    with pytest.raises(ValueError, match="a scale for each row"):
        tp.swiglu_fp8_fwd(on(200, 600), *pair(200, 300, 1))
    with pytest.raises(ValueError, match="even"):
        tp.swiglu_fp8_fwd(on(4, 601), *pair(4, 300))
    with pytest.raises(ValueError, match="dA"):
        tp.swiglu_fp8_bwd(on(4, 299), on(4, 600), *pair(4, 600))
    x, g, rs = on(4, 256), on(256), on(4, dtype=torch.float32)
    for kw, kind, words in (
            (dict(x1=None), ValueError, "x1"),
            (dict(gamma=on(255)), ValueError, "gamma"),
            (dict(rstd=on(5, dtype=torch.float32)), ValueError, "rstd"),
            (dict(r=on(4, 256, dtype=torch.float32)), TypeError, "r: "),
            (dict(y=OnDevice(torch.zeros(4, 512, dtype=torch.bfloat16)
                             [:, ::2])), ValueError, "dense")):
        a = dict(x=x, r=x, gamma=g, x1=x, q=q, s=s, rstd=rs)
        a.update(kw)
        with pytest.raises(kind, match=words):
            tp.add_rmsnorm_fp8_fwd(**a)
    with pytest.raises(ValueError, match="qb: shape"):
        tp.gemm_fp8_block(q, s, *pair(8, 255), on(4, 8))
    with pytest.raises(ValueError, match="qa: shape"):
        tp.gemm_fp8_block(q, s, *pair(8, 256), on(5, 8))
