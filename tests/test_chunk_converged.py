"""CPU: in chunk_row_product, whose lanes part where their rows end, every access to tensor
memory (a warp's instruction, all lanes together) has a warp barrier before it."""
import os
import re

from paged_kv_cache_26_gb300 import build as pkv_build

SRC = open(os.path.join(pkv_build.CSRC, "chunk_attention.cuh"), encoding="utf-8").read()


def test_tensor_memory_is_accessed_by_whole_warps():
    body = SRC[SRC.index("void chunk_row_product("):]
    body = body[:body.index("\n}\n")]
    skip = body.index("if (t0 + t >= vis) continue;")
    loop = body.rindex("for (int t0 = 0;", 0, skip)
    inner, after = body[loop:skip], body[skip:]
    # the loop comes round to its loads, and leaves for the stores
    assert inner.index("__syncwarp();") < inner.index("tmem_ld32(")
    assert after.index("__syncwarp();") < after.index("tmem_st32(")
    assert len(re.findall(r"tmem_(?:ld|st)\d+\(", body)) == 3
