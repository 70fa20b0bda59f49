"""Block-scaled calls from several threads at once, each on a stream of its own.
In a process of its own, so that the first call of every kernel (which sets its
attributes and loads the binding's module) is among them."""

import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

THREADS, ROUNDS = 4, 5


def work(tp, seed, sizes):
    """Every call once: SwiGLU both ways, the norm, three forms of product."""
    T, h, f = sizes
    g = torch.Generator(device="cuda").manual_seed(seed)

    def rand(*shape):
        return torch.randn(shape, generator=g, device="cuda").bfloat16()

    x, r, gu, dA, w = rand(T, h), rand(T, h), rand(T, 2 * f), rand(T, f), \
        rand(f, h)
    gamma = torch.ones(h, dtype=torch.bfloat16, device="cuda")
    out = []

    def pair(rows, cols, group=tp.FP8_ROW):
        q, s = tp.fp8_block_empty(rows, cols, group)
        out.extend((q.view(torch.uint8), s))
        return q, s

    def like(*shape, dtype=torch.bfloat16):
        out.append(torch.empty(shape, dtype=dtype, device="cuda"))
        return out[-1]

    wq, y, a = pair(f, h, tp.FP8_BLOCK), pair(T, h), pair(T, f)
    tp.quantize_fp8_block(w, *wq, *pair(h, f, tp.FP8_BLOCK))
    tp.add_rmsnorm_fp8_fwd(x, r, gamma, like(T, h), *y,
                           like(T, dtype=torch.float32), y=like(T, h))
    tp.gemm_fp8_block(*y, *wq, like(T, f))
    few = y[0][:3], y[1][:, :3]
    tp.gemm_fp8_block(*few, *wq, like(min(3, T), f))
    tp.swiglu_fp8_fwd(gu, *a, *pair(f, T))
    tp.swiglu_fp8_bwd(dA, gu, *pair(T, 2 * f), *pair(2 * f, T))
    tp.gemm_fp8_block(*pair_of(tp, x, out), *pair_of(tp, w, out),
                      like(T, f, dtype=torch.float32))
    return out


def pair_of(tp, t, out):
    q, s = tp.fp8_block_empty(*t.shape)
    tp.quantize_fp8_block(t, q, s)
    out.extend((q.view(torch.uint8), s))
    return q, s


SIZES = [(300, 640, 512), (2100, 1032, 2560), (40, 2056, 384), (1, 512, 768)]


def main():
    import threading

    from megatron_tensor_transformer_gate_gb300 import binding as tp
    start = threading.Barrier(THREADS)
    results, errors = [[] for _ in range(THREADS)], []

    def run(i):
        try:
            stream = torch.cuda.Stream()
            start.wait()
            with torch.cuda.stream(stream):
                for k in range(ROUNDS):
                    results[i].append(work(tp, 10 * i + k, SIZES[i]))
            stream.synchronize()
        except Exception as e:   # told to the main thread
            errors.append(repr(e))

    torch.zeros(1, device="cuda")
    threads = [threading.Thread(target=run, args=(i,)) for i in range(THREADS)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    tp.device_status()
    for i in range(THREADS):
        for k in range(ROUNDS):
            alone = work(tp, 10 * i + k, SIZES[i])
            for a, b in zip(results[i][k], alone):
                assert torch.equal(a.contiguous().view(torch.uint8),
                                   b.contiguous().view(torch.uint8)), (i, k)
    print("same results")


def test_first_calls_from_several_threads(tp):
    r = subprocess.run([sys.executable, os.path.abspath(__file__)], cwd=ROOT,
                       capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, PYTHONPATH=ROOT))
    assert r.returncode == 0 and "same results" in r.stdout, r.stderr[-3000:]


if __name__ == "__main__":
    main()
