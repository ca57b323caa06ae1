"""GPU: paged_kv_check_status over the error words of both units of kernels, in a process of its
own: the second is read once its unit has launched something, by a captured graph too."""
import subprocess
import sys
import textwrap

import pytest
import torch

from paged_kv_cache_26_gb300 import build as pkv_build

pytestmark = pytest.mark.gpu

PROGRAM = textwrap.dedent("""
    import torch
    import paged_kv_cache_26_gb300 as pkv

    def flagged():
        try:
            pkv.paged_kv_check_status()
        except pkv.PagedKVError as e:
            assert e.code == -6, e
            return str(e)
        return ""

    x = torch.randn(3, 1, 64, device="cuda").half()
    pools = [torch.zeros(2, 1, 16, 64, dtype=torch.float16, device="cuda") for _ in range(2)]
    slots = torch.tensor([1, 2, 32], dtype=torch.int32, device="cuda")
    assert flagged() == ""
    pkv.paged_kv_append(x, x, slots, *pools)                       # the first unit alone
    assert "slot" in flagged() and flagged() == ""
    rope = pkv.make_rope([0.5] * 32, 64)
    pos = torch.arange(3, dtype=torch.int32, device="cuda")
    slots[2] = 3
    torch.cuda.synchronize()
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(x)
    with torch.cuda.graph(graph):                                  # the second unit's first launch is a captured one
        pkv.paged_kv_append_rope(x, x, x, pos, rope, slots, *pools, q_out=out)
    graph.replay()
    assert flagged() == ""
    slots[2] = 32
    graph.replay()
    assert "slot" in flagged() and flagged() == ""
    graph.replay()                                                 # both at once, each other bits
    pkv.paged_decode_attention(x, *pools, torch.full((3, 1), 9, dtype=torch.int32, device="cuda"), pos + 1, 0.1)
    both = flagged()
    assert "slot" in both and "block id" in both and flagged() == ""
    print("fine")
""")


def test_both_words():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkv_build.build()
    r = subprocess.run([sys.executable, "-c", PROGRAM], capture_output=True, text=True, cwd=pkv_build.ROOT, timeout=300)
    assert r.returncode == 0 and r.stdout.strip() == "fine", r.stdout + r.stderr
