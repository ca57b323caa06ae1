"""The README's example of prompts in chunks and block-sparse steps runs as it stands."""
import os
import re

import numpy as np
import pytest
import torch

import paged_kv_cache_26_gb300 as pkv
from oracle import long_context as lc
from long_context_helpers import DEV, assert_within, f64, i32, tolerance
from paged_kv_cache_26_gb300 import build as pkv_build

TEXT = open(os.path.join(pkv_build.ROOT, "README.md"), encoding="utf-8").read()
BLOCKS = re.findall(r"```py\n(.*?)```", TEXT, re.S)


def test_names():
    assert len(BLOCKS) == 1
    names = set(re.findall(r"\bpkv\.(\w+)", BLOCKS[0]))
    assert names <= set(pkv.__all__) and {"paged_chunk_attention", "paged_select_blocks"} <= names


@pytest.mark.gpu
def test_example():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkv_build.build()
    B, Hq, Hkv, D, NB, MB = 2, 8, 2, 128, 220, 100
    lens = np.array([1300, 45])
    T = int(lens.sum())
    g = torch.Generator().manual_seed(0)

    def rand(*shape):
        return torch.randn(*shape, generator=g).bfloat16().to(DEV)

    env = dict(torch=torch, pkv=pkv, D=D, Hkv=Hkv, T=T, num_blocks=NB, k_cache=rand(NB, Hkv, 16, D), v_cache=rand(NB, Hkv, 16, D),
               q_chunk=rand(T, Hq, D), k_chunk=rand(T, Hkv, D), v_chunk=rand(T, Hkv, D),
               positions=i32(np.concatenate([np.arange(n) for n in lens])), context_lens=i32([0, 0]), new_lens=i32(lens),
               block_tables=i32(np.full((B, MB), -1)), free_blocks=i32(np.random.default_rng(0).permutation(NB)),
               num_free=i32([NB]), slots=i32(np.zeros(T)), offsets=i32(np.zeros(B + 1)), step_slots=i32(np.zeros(B)),
               q=rand(B, Hq, D), k_new=rand(B, Hkv, D), v_new=rand(B, Hkv, D))
    exec(BLOCKS[0], env)
    assert env["context_lens"].tolist() == (lens + 1).tolist()
    kp, vp, Q = f64(env["k_cache"]), f64(env["v_cache"]), f64(env["q_turned"])
    tab, sel = env["block_tables"].cpu().numpy(), env["blocks"].cpu().numpy()
    assert (sel[0] >= 0).all() and (sel[1, :, 3:] == -1).all()
    ref, mag = lc.sparse_attention(Q, kp, vp, tab, lens + 1, sel, D ** -0.5)
    assert_within(f64(env["out"]), ref, tolerance(ref, mag, torch.bfloat16, Q, kp, vp, D ** -0.5, 16 * 64, 16))
