"""Block-scaled calls with tensors that are not on the current device, or on
two devices, are refused (no GPU needed: the checks read nothing of a tensor's
storage)."""

import pytest
import torch


class On:
    """A CPU tensor that says it is on a device."""

    is_cuda = True

    def __init__(self, t, dev):
        self.t, self.device, self.dev = t, f"cuda:{dev}", dev

    def get_device(self):
        return self.dev

    def __getattr__(self, k):
        return getattr(self.t, k)


@pytest.fixture
def make(tp, monkeypatch):
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)

    def tensor(*shape, dev=0, dtype=torch.bfloat16):
        return On(torch.zeros(*shape, dtype=dtype), dev)

    def pair(rows, cols, group=0, dev=0):
        return tuple(On(t, dev) for t in
                     tp.fp8_block_empty(rows, cols, group, device="cpu"))

    return tensor, pair


CURRENT = "current device is cuda:0"


def test_all_on_another_device(tp, make):
    t, pair = make
    on1 = dict(dev=1)
    with pytest.raises(ValueError, match=CURRENT):
        tp.quantize_fp8_block(t(4, 256, **on1), *pair(4, 256, **on1))
    with pytest.raises(ValueError, match=CURRENT):
        tp.swiglu_fp8_fwd(t(4, 512, **on1), *pair(4, 256, **on1))
    with pytest.raises(ValueError, match=CURRENT):
        tp.swiglu_fp8_bwd(t(4, 256, **on1), t(4, 512, **on1),
                          *pair(4, 512, **on1))
    with pytest.raises(ValueError, match=CURRENT):
        tp.add_rmsnorm_fp8_fwd(t(4, 256, **on1), None, t(256, **on1), None,
                               *pair(4, 256, **on1),
                               t(4, dtype=torch.float32, **on1))
    with pytest.raises(ValueError, match=CURRENT):
        tp.gemm_fp8_block(*pair(4, 256, **on1), *pair(8, 256, 1, **on1),
                          t(4, 8, **on1))


def test_one_operand_on_another_device(tp, make):
    t, pair = make
    q, s = pair(4, 256)
    far_q, far_s = pair(4, 256, dev=1)
    x = t(4, 256)
    for a in ((far_q, s), (q, far_s)):
        with pytest.raises(ValueError, match="not cuda:0"):
            tp.quantize_fp8_block(x, *a)
        with pytest.raises(ValueError, match="not cuda:0"):
            tp.gemm_fp8_block(*a, *pair(8, 256, 1), t(4, 8))
        with pytest.raises(ValueError, match="not cuda:0"):
            tp.gemm_fp8_block(*pair(8, 256), *a, t(8, 4))
    with pytest.raises(ValueError, match=CURRENT):
        tp.swiglu_fp8_bwd(t(4, 128, dev=1), x, q, s)
    rs = t(4, dtype=torch.float32)
    for i in (1, 2, 3, 6, 7):   # r, gamma, x1, rstd, y
        a = [x, x, t(256), x, q, s, rs, x]
        a[i] = On(a[i].t, 1)
        with pytest.raises(ValueError, match="not cuda:0"):
            tp.add_rmsnorm_fp8_fwd(*a)
