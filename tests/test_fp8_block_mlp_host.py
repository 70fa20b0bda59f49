"""What TPBlockFP8MLP refuses before its first call, and what is left of a call
that failed (no GPU needed: CPU tensors are refused)."""

import pytest
import torch

from megatron_tensor_transformer_gate_gb300.blocks import TPBlockFP8MLP
from test_fp8_block_device_host import On

T, H, F = 4, 256, 128


@pytest.mark.parametrize("which,bad,kind", [
    ("dx1", torch.zeros(T, H), TypeError),
    ("dx1", torch.zeros(T - 1, H, dtype=torch.bfloat16), ValueError),
    ("dx1", torch.zeros(T, 2 * H, dtype=torch.bfloat16)[:, ::2], ValueError),
    ("dx1", On(torch.zeros(T, H, dtype=torch.bfloat16), 1), ValueError),
    ("gamma", torch.zeros(H - 8, dtype=torch.bfloat16), ValueError),
    ("gamma", torch.zeros(H), TypeError),
    ("dX", torch.zeros(T, H // 2, dtype=torch.bfloat16), ValueError),
    ("dX", torch.zeros(H, T, dtype=torch.bfloat16).t(), ValueError),
    ("dgamma", torch.zeros(1, dtype=torch.bfloat16), ValueError),
    ("dgamma", torch.zeros(H), TypeError)])
def test_backward_refuses(tp, which, bad, kind):
    m = TPBlockFP8MLP(T, H, F, device="cpu")
    bf16 = torch.bfloat16
    m.x1 = torch.zeros(T, H, dtype=bf16)       # as after a forward
    m.weights = [[(None, None)] * 2] * 2
    a = dict(dZ=torch.zeros(T, H, dtype=bf16), gamma=torch.ones(H, dtype=bf16),
             dx1=torch.zeros(T, H, dtype=bf16), grads=m.alloc_grads())
    (a if which in a else a["grads"])[which] = bad
    with pytest.raises(kind, match=f"^{which}"):
        m.backward(**a)


def test_weights_that_failed_to_load_are_not_used(tp):
    m = TPBlockFP8MLP(T, H, F, device="cpu")
    x, gamma = torch.zeros(T, H, dtype=torch.bfloat16), \
        torch.ones(H, dtype=torch.bfloat16)
    for weights in (None, [[(None, None)] * 2] * 2):   # first, and an update
        m.weights = weights
        with pytest.raises(ValueError, match="not on a GPU"):
            m.load_weights(torch.zeros(2 * F, H), torch.zeros(H, F))
        with pytest.raises(RuntimeError, match="load_weights"):
            m.forward(x, gamma)


def test_no_backward_after_a_forward_that_failed(tp):
    m = TPBlockFP8MLP(T, H, F, device="cpu")
    x, gamma = torch.zeros(T, H, dtype=torch.bfloat16), \
        torch.ones(H, dtype=torch.bfloat16)
    m.x1 = x                                   # as after a forward
    m.weights = [[(None, None)] * 2] * 2
    with pytest.raises(ValueError, match="not on a GPU"):
        m.forward(x, gamma)
    with pytest.raises(RuntimeError, match="forward"):
        m.backward(x, gamma)
