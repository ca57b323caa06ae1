"""The README's Python runs: its names exist, and its examples do what they say."""
import os
import re

import numpy as np
import pytest
import torch

import paged_kv_cache_26_gb300 as pkv
from oracle import int4, serving
from paged_kv_cache_26_gb300 import build as pkv_build
from parity_helpers import bits, widen_out

TEXT = open(os.path.join(pkv_build.ROOT, "README.md"), encoding="utf-8").read()
BLOCKS = re.findall(r"```python\n(.*?)```", TEXT, re.S)
DEV = "cuda"


def test_every_name_is_public():
    names = set(re.findall(r"\bpkv\.(\w+)", TEXT))
    assert len(BLOCKS) == 3 and names
    assert names <= set(pkv.__all__) and all(hasattr(pkv, n) for n in pkv.__all__)


def test_a_workspace_is_not_made_in_a_call():
    assert not re.search(r"=\s*pkv\.make_workspace\w*\([^)]*\)\s*\)", TEXT)


@pytest.mark.gpu
def test_examples():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkv_build.build()
    B, Hq, Hkv, D, K, V, MB, NB = 3, 8, 2, 128, 3, 211, 6, 40
    g = torch.Generator().manual_seed(0)

    def rand(*shape):
        return torch.randn(*shape, generator=g).bfloat16().to(DEV)

    def i32(x):
        return torch.from_numpy(np.ascontiguousarray(x, np.int32)).to(DEV)

    # the first example over tables of its own
    env = dict(q=rand(B, Hq, D), k_new=rand(B, Hkv, D), v_new=rand(B, Hkv, D), D=D, Hkv=Hkv, K=K, num_blocks=NB,
               k_cache=rand(NB, Hkv, 16, D), v_cache=rand(NB, Hkv, 16, D),
               block_tables=i32(np.arange(B * MB).reshape(B, MB)), context_lens=i32([5, 40, 16]))
    exec(BLOCKS[0], env)
    assert env["out"].shape == (B, Hq, D) and torch.isfinite(env["out"].float()).all()
    # the second: empty sequences, then prompts
    lens = np.array([5, 40, 16])
    total = int(lens.sum())
    perm = np.random.default_rng(0).permutation(NB)
    env.update(block_tables=i32(np.full((B, MB), -1)), context_lens=i32([0] * B), new_lens=i32(lens),
               free_blocks=i32(perm), num_free=i32([NB]), slots=i32(np.zeros(total)), k_prompt=rand(total, Hkv, D),
               v_prompt=rand(total, Hkv, D))
    exec(BLOCKS[1], env)
    pkv.paged_kv_check_status()
    s, _, t, free, n = serving.resize_tables([0] * B, lens, np.full((B, MB), -1), perm, NB)
    s1, _, t, free, n = serving.resize_tables(lens, lens + 1, t, free, n)
    rk = rv = np.zeros((NB, Hkv, 16, 68), np.uint8)
    rk, rv = int4.kv_append_int4(rk, rv, bits(env["k_prompt"]), bits(env["v_prompt"]), s, "bf16")
    val = [int4.values(p, f).transpose(0, 2, 1, 3).reshape(NB * 16, Hkv, D)[s] for p, f in ((rk, False), (rv, True))]
    for name, x in zip("kv", val):
        assert torch.equal(env[name].cpu(), torch.from_numpy(x.astype(np.float32)).bfloat16())
    rk, rv = int4.kv_append_int4(rk, rv, bits(env["k_new"]), bits(env["v_new"]), s1, "bf16")
    assert np.array_equal(env["kc"].cpu().numpy(), rk) and np.array_equal(env["vc"].cpu().numpy(), rv)
    ref = int4.decode_attention(widen_out(env["q"].cpu(), "bf16"), rk, rv, t, lens + 1, D ** -0.5)
    assert np.abs(widen_out(env["out"].cpu(), "bf16") - ref).max() < 0.03
    # the third
    target, draft = (torch.softmax(2 * torch.randn(B, m, V, generator=g), -1).to(DEV) for m in (K + 1, K))
    env.update(q_multi=rand(B, K + 1, Hq, D), k_multi=rand(B, K + 1, Hkv, D), v_multi=rand(B, K + 1, Hkv, D),
               target_probs=target, draft_probs=draft,
               draft_tokens=torch.randint(0, V, (B, K), generator=g, dtype=torch.int32).to(DEV),
               accept_u=torch.rand(B, K, generator=g).to(DEV), sample_u=torch.rand(B, generator=g).to(DEV))
    exec(BLOCKS[2], env)
    assert torch.equal(env["context_lens"], env["lens"])
    assert (env["lens"].cpu().numpy() == lens + 2 + env["accepted"].cpu().numpy()).all()
