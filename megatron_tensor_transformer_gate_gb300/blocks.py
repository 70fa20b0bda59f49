"""Convenience wrappers that own the workspaces of the TP block calls.

PyTorch only provides device memory here; every step runs in ``libtp.so``.
``TPMLP`` / ``TPAttention`` hold the forward workspace (saved activations)
and the backward scratch for one shape; ``TPLayer`` composes the pre-norm
layer  x1 = x + Attn(RMSNorm₁(x)),  out = x1 + MLP(RMSNorm₂(x1))  out of the
library's RMSNorm, attention and MLP entry points, which gives the layer's
four TP reductions (attention g and MLP g in forward, MLP f and attention f
in backward).
"""

import contextlib

import torch

from . import binding as B

_TD = {B.F32: torch.float32, B.BF16: torch.bfloat16,
       B.FP8: torch.bfloat16}   # FP8 mode stores bf16 tensors


def _buf(nbytes, device):
    return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=device)


def _views(ws, specs):
    """Tensors viewing consecutive 256-byte-aligned regions of a workspace
    (the layout include/tp.h documents); specs = [(name, shape, dtype)]."""
    out, off = {}, 0
    for name, shape, dt in specs:
        off = (off + 255) // 256 * 256
        n = 1
        for d in shape:
            n *= d
        nbytes = n * torch.empty((), dtype=dt).element_size()
        out[name] = ws[off:off + nbytes].view(dt).view(*shape)
        off += nbytes
    return out


class TPMLP:
    def __init__(self, T, h, h_ffn, n, *, dtype=B.BF16, act=B.GELU,
                 mode=B.FUSED, dropout_p=0.0, seed=0, device="cuda"):
        self.desc = B.mlp_desc(T, h, h_ffn, n, dtype, act, mode, dropout_p,
                               seed)
        self.T, self.h, self.f, self.act = T, h, h_ffn, act
        self.dtype = _TD[dtype]
        self.device = device
        self.ws = _buf(B.mlp_workspace_bytes(self.desc), device)
        self.scratch = _buf(B.mlp_bwd_scratch_bytes(self.desc), device)

    def forward(self, X, W1, W2, b1=None, b2=None, R=None, out=None,
                stream=None):
        if out is None:
            out = torch.empty((self.T, self.h), dtype=self.dtype,
                              device=self.device)
        B.mlp_fwd(self.desc, X, W1, W2, out, self.ws, b1=b1, b2=b2, R=R,
                  stream=stream)
        return out

    def backward(self, dOut, X, W1, W2, dres=None, want_db1=False,
                 want_db2=False, grads=None, stream=None):
        g = grads if grads is not None else self.alloc_grads(W1, W2,
                                                             want_db1,
                                                             want_db2)
        B.mlp_bwd(self.desc, dOut, X, W1, W2, self.ws, g["dX"], g["dW1"],
                  g["dW2"], self.scratch, db1=g.get("db1"), db2=g.get("db2"),
                  dres=dres, stream=stream)
        return g

    def saved(self):
        """Views of the activations the forward call saved for backward."""
        tf = (self.T, self.f)
        names = ("H", "A") if self.act == B.GELU else ("G", "U", "A")
        return _views(self.ws, [(n, tf, self.dtype) for n in names])

    def alloc_grads(self, W1, W2, want_db1=False, want_db2=False):
        kw = dict(dtype=self.dtype, device=self.device)
        g = {"dX": torch.empty((self.T, self.h), **kw),
             "dW1": torch.empty_like(W1), "dW2": torch.empty_like(W2)}
        if want_db1:
            g["db1"] = torch.empty((W1.shape[0],), **kw)
        if want_db2:
            g["db2"] = torch.empty((self.h,), **kw)
        return g


class TPAttention:
    """dtype B.BF16, or B.FP8: the projections of the forward on E4M3
    operands (bf16 storage and backward)."""

    def __init__(self, b, s, h, n_q, n_kv, d, n, *, causal=True, mode=B.FUSED,
                 dtype=B.BF16, device="cuda"):
        self.desc = B.attn_desc(b, s, h, n_q, n_kv, d, n, dtype, causal,
                                mode)
        self.T, self.h = b * s, h
        self.shape = (b, s, n_q, n_kv, d)
        self.device = device
        self.ws = _buf(B.attn_workspace_bytes(self.desc), device)
        self.scratch = _buf(B.attn_bwd_scratch_bytes(self.desc), device)

    def forward(self, X, Wq, Wk, Wv, Wo, bo=None, R=None, out=None,
                stream=None):
        if out is None:
            out = torch.empty((self.T, self.h), dtype=torch.bfloat16,
                              device=self.device)
        B.attn_fwd(self.desc, X, Wq, Wk, Wv, Wo, out, self.ws, bo=bo, R=R,
                   stream=stream)
        return out

    def backward(self, dOut, X, Wq, Wk, Wv, Wo, dres=None, want_dbo=False,
                 grads=None, stream=None):
        g = grads if grads is not None else self.alloc_grads(Wq, Wk, Wv, Wo,
                                                             want_dbo)
        B.attn_bwd(self.desc, dOut, X, Wq, Wk, Wv, Wo, self.ws, g["dX"],
                   g["dWq"], g["dWk"], g["dWv"], g["dWo"], self.scratch,
                   dbo=g.get("dbo"), dres=dres, stream=stream)
        return g

    def saved(self):
        """Views of Q, K, V (fp16), O (bf16) and LSE saved by the forward."""
        b, s, nq, nkv, d = self.shape
        T = b * s
        return _views(self.ws, [("Q", (T, nq * d), torch.float16),
                                ("K", (T, nkv * d), torch.float16),
                                ("V", (T, nkv * d), torch.float16),
                                ("O", (T, nq * d), torch.bfloat16),
                                ("LSE", (b, nq, s), torch.float32)])

    def alloc_grads(self, Wq, Wk, Wv, Wo, want_dbo=False):
        g = {"dX": torch.empty((self.T, self.h), dtype=torch.bfloat16,
                               device=self.device),
             "dWq": torch.empty_like(Wq), "dWk": torch.empty_like(Wk),
             "dWv": torch.empty_like(Wv), "dWo": torch.empty_like(Wo)}
        if want_dbo:
            g["dbo"] = torch.empty((self.h,), dtype=torch.bfloat16,
                                   device=self.device)
        return g


class TPLayer:
    """Pre-norm layer: RMSNorm → attention (+x) → RMSNorm → SwiGLU MLP (+x1),
    one tp_layer_fwd / tp_layer_bwd call per direction.  dtype B.FP8 runs
    every projection of the forward on E4M3 operands."""

    def __init__(self, b, s, h, h_ffn, n_q, n_kv, d, n, *, eps=1e-5,
                 act=B.SWIGLU, mode=B.FUSED, dtype=B.BF16, device="cuda"):
        if act != B.SWIGLU:
            raise ValueError("the layer's MLP is SwiGLU")
        self.T, self.h, self.eps = b * s, h, eps
        self.device = device
        self.desc = B.layer_desc(b, s, h, h_ffn, n_q, n_kv, d, n, dtype, mode,
                                 eps)
        self.ws = _buf(B.layer_workspace_bytes(self.desc), device)
        self.scratch = _buf(B.layer_bwd_scratch_bytes(self.desc), device)

    def forward(self, x, P, out=None, stream=None):
        if out is None:
            out = torch.empty((self.T, self.h), dtype=torch.bfloat16,
                              device=self.device)
        B.layer_fwd(self.desc, x, P, out, self.ws, stream)
        return out

    def alloc_grads(self, P):
        g = {k: torch.empty_like(P[k]) for k in ("g1", "Wq", "Wk", "Wv", "Wo",
                                                 "g2", "W1", "W2")}
        g = {"d" + k: v for k, v in g.items()}
        g["dX"] = torch.empty((self.T, self.h), dtype=torch.bfloat16,
                              device=self.device)
        return g

    def backward(self, dout, x, P, grads=None, stream=None):
        g = grads if grads is not None else self.alloc_grads(P)
        B.layer_bwd(self.desc, dout, x, P, self.ws, g, self.scratch, stream)
        return g


def _made_on(stream):
    """Memory that a call makes for itself belongs to the stream it runs on: of
    another stream's pool it may still be in use there."""
    return contextlib.nullcontext() if stream is None else \
        torch.cuda.stream(stream)


class TPBlockFP8MLP:
    """Residual + RMSNorm + SwiGLU MLP with every product, forward and
    backward, on block-scaled E4M3 operands:

        x1 = x + r,  Y = RMSNorm(x1)·γ,  [G | U] = Y·W1ᵀ,
        Z = (SiLU(G) ⊙ U)·W2ᵀ

    for T tokens (one for a generated token, or a batch).  Z is handed on
    without x1: the next norm adds it as its r.  Scales are 1×128 along each
    product's reduction axis for activations and gradients, 128×128 for
    weights; γ, x, r, x1, Z and the gradients are bf16 (weight gradients in
    ``grad_dtype``, bf16 or fp32).  Each operand's codes are made from fp32 values
    or from the bf16 tensor that the step before stores, with one exception: the
    codes of Yᵀ, for dW1, are of Y rounded to bf16 (those of Y, for the forward,
    are not), so that dW1's operand is rounded twice.

    W1 is [2·h_ffn, h] (gate rows, then up rows), W2 [h, h_ffn], both bf16 or
    fp32, unsharded.  Each of the n logical shards holds h_ffn/n hidden units,
    a multiple of 128 so that no block of 128 crosses a shard: quantizing the
    whole tensors is then quantizing each shard's, and the g and f sums are
    taken in the products' accumulation (the fused mode; no other).

    ``train=False`` keeps neither what the backward reads nor the transposed
    weights."""

    def __init__(self, T, h, h_ffn, n=1, *, eps=1e-5, train=True,
                 grad_dtype=torch.bfloat16, device="cuda"):
        if min(T, h, h_ffn, n) < 1 or h % 8 or h > 16384:
            raise ValueError("sizes: T, n ≥ 1, h a multiple of 8 up to 16384")
        if h_ffn % n or (h_ffn // n) % 128:
            raise ValueError("h_ffn/n: a multiple of 128")
        if grad_dtype not in (torch.bfloat16, torch.float32):
            raise ValueError("grad_dtype: bfloat16 or float32")
        self.T, self.h, self.f, self.n = T, h, h_ffn, n
        self.eps, self.train, self.grad_dtype = eps, train, grad_dtype
        self.device = device
        bf16 = dict(dtype=torch.bfloat16, device=device)
        pair = lambda r, c: B.fp8_block_empty(r, c, device=device)
        self.rstd = torch.empty(T, dtype=torch.float32, device=device)
        self.y, self.a = pair(T, h), pair(T, h_ffn)
        self.gu = torch.empty((T, 2 * h_ffn), **bf16)
        self.weights = None
        if train:
            self.x1 = None
            self.y16 = torch.empty((T, h), **bf16)
            self.yt, self.at = pair(h, T), pair(h_ffn, T)
            self.dz, self.dzt = pair(T, h), pair(h, T)
            self.dgu, self.dgut = pair(T, 2 * h_ffn), pair(2 * h_ffn, T)
            self.da = torch.empty((T, h_ffn), **bf16)
            self.dy = torch.empty((T, h), **bf16)
            self.norm_scratch = _buf(B.rmsnorm_bwd_scratch_bytes(T, h), device)

    def load_weights(self, W1, W2, stream=None):
        """Quantize W1 and W2 (after every update of them)."""
        if tuple(W1.shape) != (2 * self.f, self.h) or \
                tuple(W2.shape) != (self.h, self.f):
            raise ValueError(f"W1 {(2 * self.f, self.h)} and W2 "
                             f"{(self.h, self.f)}, got {tuple(W1.shape)} and "
                             f"{tuple(W2.shape)}")
        weights, self.weights = self.weights, None   # none, should a call fail
        if weights is None:
            with _made_on(stream):
                weights = [
                    [B.fp8_block_empty(*s, B.FP8_BLOCK, self.device)
                     if s is not None else (None, None) for s in
                     (W.shape, W.shape[::-1] if self.train else None)]
                    for W in (W1, W2)]
        for W, (q, qt) in zip((W1, W2), weights):
            B.quantize_fp8_block(W, *q, *qt, stream=stream)
        self.weights = weights

    def forward(self, x, gamma, r=None, out=None, x1=None, stream=None):
        """(x1, Z).  x1 may be given (x or r among it); without r it is x."""
        if self.weights is None:
            raise RuntimeError("load_weights comes first")
        if self.train:
            self.x1 = None   # what the last forward saved is overwritten
        with _made_on(stream):
            if r is None:
                x1 = x if x1 is None else x1
            elif x1 is None:
                x1 = torch.empty_like(x)
            if out is None:
                out = torch.empty((self.T, self.h), dtype=torch.bfloat16,
                                  device=self.device)
        (w1, _), (w2, _) = self.weights
        keep = self.train
        B.add_rmsnorm_fp8_fwd(x, r, gamma, None if x1 is x and r is None
                              else x1, *self.y, self.rstd,
                              y=self.y16 if keep else None, eps=self.eps,
                              stream=stream)
        B.gemm_fp8_block(*self.y, *w1, self.gu, stream=stream)
        B.swiglu_fp8_fwd(self.gu, *self.a, *(self.at if keep else ()),
                         stream=stream)
        B.gemm_fp8_block(*self.a, *w2, out, stream=stream)
        if keep:
            B.quantize_fp8_block(self.y16, qt=self.yt[0], st=self.yt[1],
                                 stream=stream)
            self.x1 = x1
        return x1, out

    def alloc_grads(self):
        kw = dict(device=self.device)
        return {"dX": torch.empty((self.T, self.h), dtype=torch.bfloat16, **kw),
                "dgamma": torch.empty(self.h, dtype=torch.bfloat16, **kw),
                "dW1": torch.empty((2 * self.f, self.h),
                                   dtype=self.grad_dtype, **kw),
                "dW2": torch.empty((self.h, self.f), dtype=self.grad_dtype,
                                   **kw)}

    def backward(self, dZ, gamma, dx1=None, grads=None, stream=None):
        """Gradients after a forward of the same inputs (x1 unchanged since):
        dX, of x and of r alike; dgamma, dW1, dW2.  dx1 is the gradient that
        reaches x1 past the norm (the residual stream's).  The quantizations
        pass gradients through."""
        if not self.train or self.x1 is None:
            raise RuntimeError("a forward of a block with train=True comes "
                               "first")
        with _made_on(stream):
            g = grads if grads is not None else self.alloc_grads()
        # what the norm's backward takes as it is (the products check theirs)
        dev = self.x1.get_device()
        for t, what, shape in ((gamma, "gamma", (self.h,)),
                               (dx1, "dx1", (self.T, self.h)),
                               (g["dX"], "dX", (self.T, self.h)),
                               (g["dgamma"], "dgamma", (self.h,))):
            if t is not None:
                B._dense(t, what, torch.bfloat16, shape, dev)
        (_, w1t), (_, w2t) = self.weights
        B.quantize_fp8_block(dZ, *self.dz, *self.dzt, stream=stream)
        B.gemm_fp8_block(*self.dz, *w2t, self.da, stream=stream)
        B.gemm_fp8_block(*self.dzt, *self.at, g["dW2"], stream=stream)
        B.swiglu_fp8_bwd(self.da, self.gu, *self.dgu, *self.dgut,
                         stream=stream)
        B.gemm_fp8_block(*self.dgu, *w1t, self.dy, stream=stream)
        B.gemm_fp8_block(*self.dgut, *self.yt, g["dW1"], stream=stream)
        B.rmsnorm_bwd(self.dy, self.x1, gamma, self.rstd, g["dX"],
                      g["dgamma"], self.norm_scratch, dres=dx1, eps=self.eps,
                      stream=stream)
        return g
