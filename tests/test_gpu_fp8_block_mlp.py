"""The block-scaled operators as they are used together: the residual + RMSNorm
+ SwiGLU MLP of blocks.TPBlockFP8MLP, forward and backward, against the oracle
that rounds what the device stores.

Bounds: a stored bf16 result's Frobenius error is 2^-9 to 2^-8 relative from
its own rounding; where an intermediate's last bits differ (fp32 accumulation,
approximate exponential) some codes move by one E4M3 step, 2^-4 to 2^-3 of the
element.  A bf16 intermediate differs in its last bit (2^-8) for a share of its
elements below 2^-5 (2^-24·√K·8 against 2^-9 for K ≤ 2^14 terms gives 2^-5);
of the codes made from those one in 2^4 moves by 2^-3: 2^-9 of the elements,
√2^-9·2^-3 = 2^-7.5 of the norm at the very most, so that the bf16 bound 1e-2
holds for every output, which is two such steps deep with its rounding
averaged over a product's K terms.
"""

import pytest
import torch

from oracle import fp8_block as ob
from megatron_tensor_transformer_gate_gb300 import inputs as I
from megatron_tensor_transformer_gate_gb300.blocks import TPBlockFP8MLP
from _parity import check_fro

pytestmark = pytest.mark.gpu
EPS = 1e-5


def tensors(T, h, f, seed, w_dtype=torch.bfloat16):
    def n(shape, std, k, dt=torch.bfloat16, mean=0.0):
        return I.normal(shape, std, seed + k, "cpu", dt, mean)
    return dict(x=n((T, h), 1.0, 1), r=n((T, h), 0.5, 2),
                gamma=n((h,), 0.02, 3, mean=1.0),
                W1=n((2 * f, h), h ** -0.5, 4, w_dtype),
                W2=n((h, f), f ** -0.5, 5, w_dtype),
                dZ=n((T, h), 1e-3, 6), dx1=n((T, h), 1e-3, 7))


def run(t, T, h, f, n=1, residual=True, grad_dtype=torch.bfloat16, **kw):
    d = {k: v.cuda() for k, v in t.items()}
    m = TPBlockFP8MLP(T, h, f, n, eps=EPS, grad_dtype=grad_dtype, **kw)
    m.load_weights(d["W1"], d["W2"])
    x1, Z = m.forward(d["x"], d["gamma"], r=d["r"] if residual else None)
    g = m.backward(d["dZ"], d["gamma"], dx1=d["dx1"] if residual else None) \
        if m.train else {}
    return dict(g, x1=x1, Z=Z), m, d


@pytest.mark.parametrize("T,h,f,n,residual,w_dtype,grad_dtype", [
    (1, 256, 256, 1, True, torch.bfloat16, torch.bfloat16),
    (5, 264, 128, 1, False, torch.bfloat16, torch.bfloat16),
    (100, 520, 512, 4, True, torch.float32, torch.float32),
    (130, 512, 1280, 2, True, torch.bfloat16, torch.float32),
    (515, 1024, 2816, 1, True, torch.bfloat16, torch.bfloat16)])
def test_mlp_forward_and_backward(tp, T, h, f, n, residual, w_dtype,
                                  grad_dtype):
    t = tensors(T, h, f, 100 * T, w_dtype)
    got, _, _ = run(t, T, h, f, n, residual, grad_dtype)
    tp.device_status()
    o = {k: I.to_f64(v) for k, v in t.items()}
    if not residual:
        o["r"] = o["dx1"] = None
    want = ob.mlp(eps=EPS, **o)
    assert (I.to_f64(got["x1"]) == want["x1"]).all()
    for k in ("Z", "dX", "dgamma", "dW1", "dW2"):
        assert got[k].dtype == (grad_dtype if k in ("dW1", "dW2")
                                else torch.bfloat16)
        check_fro(got[k], want[k], f"{k} at T={T} h={h} f={f}")


def test_shards_share_the_accumulation(tp):
    # the fused sum over shards is the product's own order of blocks
    t = tensors(70, 256, 1024, 3)
    a, _, _ = run(t, 70, 256, 1024, 1)
    b, _, _ = run(t, 70, 256, 1024, 8)
    assert all(torch.equal(a[k], b[k]) for k in a)


def test_serving_block_equals_the_training_forward(tp):
    t = tensors(3, 512, 768, 4)
    a, _, _ = run(t, 3, 512, 768)
    b, m, _ = run(t, 3, 512, 768, train=False)
    assert torch.equal(a["Z"], b["Z"]) and torch.equal(a["x1"], b["x1"])
    with pytest.raises(RuntimeError, match="train"):
        m.backward(a["Z"], t["gamma"].cuda())


def test_step_captured_and_replayed_next_to_an_eager_one(tp):
    # a captured step (weights quantized inside) replayed twice on new inputs
    # while an eager block of the same sizes works on another stream
    T, h, f = 150, 384, 512
    t = tensors(T, h, f, 5)
    _, m, d = run(t, T, h, f)
    eager, _, _ = run(t, T, h, f)            # every kernel has run once
    x1, Z, g = torch.empty_like(d["x"]), torch.empty_like(d["x"]), \
        m.alloc_grads()

    def step(blk, dev, x1, Z, g):
        blk.load_weights(dev["W1"], dev["W2"])
        blk.forward(dev["x"], dev["gamma"], r=dev["r"], out=Z, x1=x1)
        blk.backward(dev["dZ"], dev["gamma"], dx1=dev["dx1"], grads=g)

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(m, d, x1, Z, g)
    other = TPBlockFP8MLP(T, h, f, eps=EPS)
    side = torch.cuda.Stream()
    for seed in (6, 7):
        for k, v in tensors(T, h, f, seed).items():
            d[k].copy_(v.cuda())
        ex1, eZ, eg = torch.empty_like(x1), torch.empty_like(Z), \
            other.alloc_grads()
        side.wait_stream(torch.cuda.current_stream())
        graph.replay()
        with torch.cuda.stream(side):
            step(other, d, ex1, eZ, eg)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        assert torch.equal(x1, ex1) and torch.equal(Z, eZ)
        assert all(torch.equal(g[k], eg[k]) for k in g)
    tp.device_status()


def test_what_the_saved_codes_are_made_of(tp):
    # Yᵀ's codes are of the stored bf16 Y, Aᵀ's of the fp32 values of A's own
    T, h, f = 130, 264, 256
    _, m, _ = run(tensors(T, h, f, 9), T, h, f)
    yt, st = ob.quantize(m.y16.float().cpu().numpy().T, "row")
    assert (m.yt[0].contiguous().view(torch.uint8).cpu().numpy() == yt).all()
    assert (m.yt[1].cpu().numpy() == st).all()
    at = tp.fp8_block_empty(f, T)
    tp.swiglu_fp8_fwd(m.gu, qt=at[0], st=at[1])
    assert torch.equal(at[0].view(torch.uint8), m.at[0].view(torch.uint8))
    assert torch.equal(at[1], m.at[1])


def pool_of(t):
    """The stream whose memory pool a tensor is of."""
    return next(s["stream"] for s in torch.cuda.memory_snapshot()
                if 0 <= t.data_ptr() - s["address"] < s["total_size"])


def test_memory_made_in_a_call_is_of_its_stream(tp):
    T, h, f = 150, 384, 512
    t = tensors(T, h, f, 8)
    here, _, d = run(t, T, h, f)
    side = torch.cuda.Stream()
    m = TPBlockFP8MLP(T, h, f, eps=EPS)
    side.wait_stream(torch.cuda.current_stream())
    m.load_weights(d["W1"], d["W2"], stream=side)
    x1, Z = m.forward(d["x"], d["gamma"], r=d["r"], stream=side)
    g = m.backward(d["dZ"], d["gamma"], dx1=d["dx1"], stream=side)
    side.synchronize()
    tp.device_status()
    got = dict(g, x1=x1, Z=Z)
    for k, v in got.items():
        assert torch.equal(v, here[k]), k
        assert pool_of(v) == side.cuda_stream, k
    for pair in (p for w in m.weights for p in w):
        assert all(pool_of(v) == side.cuda_stream for v in pair)


def test_block_refuses(tp):
    for a in ((0, 256, 256), (4, 252, 256), (4, 256, 200), (4, 16392, 256)):
        with pytest.raises(ValueError):
            TPBlockFP8MLP(*a)
    with pytest.raises(ValueError):
        TPBlockFP8MLP(4, 256, 512, 8)        # shards of 64 units
    with pytest.raises(ValueError):
        TPBlockFP8MLP(4, 256, 256, grad_dtype=torch.float16)
    m = TPBlockFP8MLP(4, 256, 256)
    with pytest.raises(RuntimeError, match="load_weights"):
        m.forward(torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda"),
                  torch.ones(256, dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(ValueError, match="W1"):
        m.load_weights(torch.zeros(256, 256, device="cuda"),
                       torch.zeros(256, 256, device="cuda"))
