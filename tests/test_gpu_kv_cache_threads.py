"""Calls of the key-value cache from several threads at once, each on a stream of
its own.  In a process of its own, so that the first call of every kernel (which
sets its attributes and loads the binding's module) is among them."""

import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

THREADS, ROUNDS = 4, 5
SIZES = [(3, 500, 8, 2, 128), (1, 3000, 32, 1, 64), (40, 20, 4, 4, 128),
         (2, 700, 16, 4, 64)]     # b, s, n_q, n_kv, d


def work(tp, seed, sizes):
    b, s, n_q, n_kv, d = sizes
    g = torch.Generator(device="cuda").manual_seed(seed)
    page, out = 16, []
    cols = (s + page - 1) // page
    table = torch.arange(b * cols, dtype=torch.int32, device="cuda").view(b,
                                                                          cols)
    lens = torch.full((b,), s, dtype=torch.int32, device="cuda")
    x = torch.randn((b * s, 2 * n_kv, d), generator=g, device="cuda").bfloat16()
    q = torch.randn((b, n_q, d), generator=g, device="cuda").bfloat16()
    for dtype in (tp.BF16, tp.F16, tp.FP8):
        cache = tp.kv_cache_empty(b * cols, page, n_kv, d, dtype)
        tp.kv_cache_write(x[:, :n_kv], x[:, n_kv:], cache, table, lens)
        for t in range(2):
            out.append(torch.empty((b * s, n_kv, d), dtype=torch.bfloat16,
                                   device="cuda"))
        tp.kv_cache_read(cache, table, lens, *out[-2:])
        out.append(torch.empty_like(q))
        tp.attn_decode(q, cache, table, lens, out[-1])
    return out


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
            for a, b in zip(results[i][k], work(tp, 10 * i + k, SIZES[i])):
                assert torch.equal(a, b), (i, k)
    print("same results")


def test_first_calls_from_several_threads(tp):
    r = subprocess.run([sys.executable, os.path.abspath(__file__)], cwd=ROOT,
                       capture_output=True, text=True, timeout=300,
                       env=dict(os.environ, PYTHONPATH=ROOT))
    assert r.returncode == 0 and "same results" in r.stdout, r.stderr[-3000:]


if __name__ == "__main__":
    main()
