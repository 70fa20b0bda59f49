"""Rules on the device code that its text alone can show."""

import glob
import os
import re

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def asm_strings(text):
    """String literals, adjacent ones joined as the compiler joins them."""
    return re.findall(r'"((?:[^"\\]|\\.)*)"', re.sub(r'"\s*"', "", text))


def multicast_loads(text):
    return [s for s in asm_strings(text)
            if "cp.async.bulk" in s and ".multicast" in s]


def test_the_search_sees_a_split_instruction():
    load = ('asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.tile"'
            '\n  ".mbarrier::complete_tx::bytes.multicast::cluster [%0];");')
    commit = ('asm("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::'
              'cluster."\n "multicast::cluster.b64 [%0], %1;");')
    assert len(multicast_loads(load)) == 1 and not multicast_loads(commit)


def test_no_load_is_multicast_to_a_cluster():
    # One library serves every rank of a run on several GPUs, and a multicast
    # load is for one GPU's own memory alone.
    files = [f for d in ("include", "megatron_tensor_transformer_gate_gb300")
             for f in glob.glob(os.path.join(ROOT, d, "**", "*"),
                                recursive=True)
             if f.endswith((".cu", ".cuh", ".h", ".cpp"))]
    assert len(files) > 10
    for f in files:
        with open(f, encoding="utf-8") as fh:
            assert not multicast_loads(fh.read()), os.path.relpath(f, ROOT)
