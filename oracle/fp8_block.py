"""Oracle for the block-scaled E4M3 operators (numpy).

Test infrastructure: see the package docstring.

Definition (include/tp.h, "FP8 with a scale per block"): a matrix [rows, cols]
is cut into 1×128 pieces of its rows (group "row") or 128×128 blocks (group
"block"), the last ones short; with amax a block's largest magnitude and every
operation rounded once to fp32,

    r = 448 / amax,   s = amax / 448,   q = e4m3(x·r),

amax = 0 giving s = 1 and an amax below 2^-100 counting as 2^-100; the value
is q·s.  Scales are stored [⌈cols/128⌉, rows] or [⌈cols/128⌉, ⌈rows/128⌉].

The gated activation and the norm are quantized from their exact values, so a
device result may differ from these codes where its fp32 value crosses a
rounding boundary; tests hold the dequantized value to E4M3's half step.

Pins: tests/test_fp8_block_host.py.
"""

import numpy as np

from .fp8 import E4M3_MAX, e4m3_decode, e4m3_encode, round_bf16

GROUP = 128
FLOOR = np.float32(2.0 ** -100)


def _cdiv(a, b):
    return (a + b - 1) // b


def block_amax(x, group):
    """[⌈cols/128⌉, rows or ⌈rows/128⌉] largest magnitudes (NaN left out)."""
    a = np.abs(np.asarray(x))
    a = np.where(np.isnan(a), 0, a)
    rows, cols = a.shape
    out = []
    for c in range(0, cols, GROUP):
        m = a[:, c:c + GROUP].max(axis=1)
        if group == "block":
            m = np.array([m[r:r + GROUP].max() for r in range(0, rows, GROUP)])
        out.append(m)
    return np.stack(out)


def expand(s, rows, cols):
    """The scale (or factor) of every element, [rows, cols]."""
    e = np.asarray(s).T
    if e.shape[0] != rows:
        e = np.repeat(e, GROUP, axis=0)[:rows]
    return np.repeat(e, GROUP, axis=1)[:, :cols]


def scales(amax):
    """(factor r, scale s) in fp32 of the blocks' amax."""
    amax = np.asarray(amax, np.float32)
    a = np.maximum(amax, FLOOR)
    r = (np.float32(E4M3_MAX) / a).astype(np.float32)
    s = np.where(amax == 0, np.float32(1), a / np.float32(E4M3_MAX))
    return r, s.astype(np.float32)


def quantize(x, group):
    """(codes uint8, scales fp32) of finite fp32 (or bf16-valued) x."""
    x = np.asarray(x, np.float32)
    r, s = scales(block_amax(x, group))
    prod = (x * expand(r, *x.shape)).astype(np.float32)
    return e4m3_encode(prod), s


def dequantize(q, s):
    q = np.asarray(q)
    return e4m3_decode(q) * expand(np.asarray(s, np.float64), *q.shape)


def gemm(qa, sa, qb, sb):
    """(C, Σ|a||b|) in float64: the product and what bounds its rounding."""
    a, b = dequantize(qa, sa), dequantize(qb, sb)
    return a @ b.T, np.abs(a) @ np.abs(b).T


def swiglu(gu):
    g, u = np.split(np.asarray(gu, np.float64), 2, axis=1)
    return g / (1.0 + np.exp(-g)) * u


def swiglu_grad(dA, gu):
    """[dG | dU]."""
    g, u = np.split(np.asarray(gu, np.float64), 2, axis=1)
    dA = np.asarray(dA, np.float64)
    s = 1.0 / (1.0 + np.exp(-g))
    return np.concatenate([dA * u * s * (1.0 + g * (1.0 - s)), dA * g * s],
                          axis=1)


def mlp(x, r, gamma, W1, W2, dZ, dx1, eps):
    """The residual + RMSNorm + SwiGLU MLP with block-scaled operands, forward
    and backward, each step's stored tensor rounded as the device stores it
    (bf16, or E4M3 codes of the values before any other rounding)."""
    from .norm import rmsnorm_backward, rmsnorm_forward
    x1 = round_bf16(x if r is None else x + r)
    y = rmsnorm_forward(x1, gamma, eps)["y"]

    def deq(v, group):
        return dequantize(*quantize(v, group))

    w1, w2 = deq(W1, "block"), deq(W2, "block")
    gu = round_bf16(deq(y, "row") @ w1.T)
    a = swiglu(gu)
    Z = deq(a, "row") @ w2.T
    dA = round_bf16(deq(dZ, "row") @ w2)
    dW2 = deq(dZ.T, "row") @ deq(a.T, "row").T
    dgu = swiglu_grad(dA, gu)
    dY = round_bf16(deq(dgu, "row") @ w1)
    dW1 = deq(dgu.T, "row") @ deq(round_bf16(y).T, "row").T
    n = rmsnorm_backward(dY, x1, gamma, eps, dres=dx1)
    return {"x1": x1, "Z": Z, "dX": n["dx"], "dgamma": n["dgamma"],
            "dW1": dW1, "dW2": dW2}
