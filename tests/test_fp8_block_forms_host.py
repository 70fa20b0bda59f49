"""Which form a block-scaled product takes, on 152 SMs (no GPU needed): the GPU
tests of the forms rely on it."""

import ctypes

import pytest

FORMS = [  # M, N, K, b_group, form
    (1, 4096, 4096, 1, ("thin", 8, 1)), (8, 28672, 8192, 0, ("thin", 8, 1)),
    (9, 100, 100, 1, ("narrow", 16, 1)), (9, 100, 256, 1, ("narrow", 16, 2)),
    (16, 100, 384, 1, ("narrow", 16, 3)), (9, 4100, 900, 1, ("narrow", 16, 4)),
    (30, 100, 640, 1, ("narrow", 32, 5)), (23, 100, 768, 0, ("narrow", 32, 6)),
    (44, 100, 896, 1, ("narrow", 64, 7)), (37, 100, 900, 1, ("narrow", 64, 8)),
    (280, 3300, 384, 1, ("narrow", 128, 1)),
    (72, 100, 768, 1, ("narrow", 128, 6)),
    (1080, 4330, 2600, 1, ("wide", 256, 1)),
    (1080, 4330, 2600, 0, ("wide", 256, 1)),
    (8192, 8192, 28672, 1, ("wide", 256, 1))]


@pytest.mark.parametrize("M,N,K,b_group,form", FORMS)
def test_form(tp, M, N, K, b_group, form):
    assert tp.gemm_fp8_block_form(M, N, K, b_group, 152) == form


def test_refusals(tp):
    x = ctypes.c_int32()
    ok = [ctypes.byref(x)] * 3

    def rc(M=9, N=9, K=9, group=1, sms=152, out=ok):
        return tp.lib().tp_gemm_fp8_block_form(M, N, K, group, sms, *out)

    assert rc() == 0
    for i in range(3):
        assert rc(out=ok[:i] + [None] + ok[i + 1:]) == 1
    for k in ("M", "N", "K"):
        assert rc(**{k: 0}) == 2 and rc(**{k: (1 << 30) + 1}) == 2
    assert rc(group=2) == 3 and rc(sms=-1) == 8
