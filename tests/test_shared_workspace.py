"""One workspace for calls of different shapes and pool formats: sizes on the
CPU, and on the GPU the results of a fresh workspace, whatever ran before."""
import ctypes

import numpy as np
import pytest
import torch

import paged_kv_cache_26_gb300 as pkv
import workloads as wl
from paged_kv_cache_26_gb300 import build as pkv_build
from paged_kv_cache_26_gb300._native import PkvDims, lib

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    pkv_build.build()


def align(n):
    return -(-n // 256) * 256


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count if torch.cuda.is_available() else 1


def dims(**kw):
    d = dict(num_seqs=64, num_q_heads=32, num_kv_heads=8, head_dim=128, block_size=16, num_blocks=9,
             max_blocks_per_seq=40, dtype=1)
    d.update(kw)
    return PkvDims(**d)


def automatic_bytes(d):
    """Partials and log-sum-exps of five segments per warp, counters, publication: the automatic path's size since
    the 16-bit and E4M3 pools were all there was."""
    seg = sms() * 12 * 5
    return align(seg * 16 * d.head_dim * 4) + align(seg * 16 * 4) + 256 + align((2 * d.num_seqs + 2) * 4)


# ------------------------------------------------------------------ sizes

@pytest.mark.parametrize("kw", [{}, dict(num_seqs=1, num_kv_heads=1, num_q_heads=1), dict(num_seqs=2048),
                                dict(head_dim=64, num_seqs=300), dict(num_seqs=2048, num_kv_heads=32)])
def test_the_16_bit_calls_need_no_room_for_4_bit_ones(kw):
    """Called without a GPU: a workspace one byte short is refused for its size, one of the size is not."""
    d = dims(**kw)
    need = automatic_bytes(d)
    p, null = ctypes.c_void_p(1 << 20), ctypes.c_void_p(0)
    got = lib().paged_decode_workspace_bytes(ctypes.byref(d), 0)
    assert got == need or got > need and d.num_seqs * d.num_kv_heads * 8 > need // 2  # more units than fit, on one SM

    def attend(n):
        if torch.cuda.is_available():
            pytest.skip("made-up pointers: refusals only, without a GPU")
        return lib().paged_decode_attention(p, p, p, p, p, 0.1, p, 0, p, n, ctypes.byref(d), null)

    assert attend(need - 1) == -1 and "too small" in lib().paged_kv_last_error().decode()
    assert attend(need) not in (0, -1)                      # on to the driver, which is not there


def test_split_and_multi_token_calls_ask_for_the_header_and_do_without():
    d = dims()
    p, null = ctypes.c_void_p(1 << 20), ctypes.c_void_p(0)
    L = lib()
    rows = 64 * 32 * 4
    need = align(rows * 128 * 4) + align(rows * 4)
    assert L.paged_decode_workspace_bytes(ctypes.byref(d), 4) == need + 256
    assert L.paged_decode_workspace_bytes(ctypes.byref(d), 1) == 0
    rows *= 3
    multi = align(rows * 128 * 4) + align(rows * 4)
    assert L.paged_decode_multi_workspace_bytes(ctypes.byref(d), 3, 4) == multi + 256
    assert L.paged_decode_multi_workspace_bytes(ctypes.byref(d), 3, 1) == 0
    if not torch.cuda.is_available():
        assert L.paged_decode_attention(p, p, p, p, p, 0.1, p, 4, p, need - 1, ctypes.byref(d), null) == -1
        assert L.paged_decode_attention(p, p, p, p, p, 0.1, p, 4, p, need, ctypes.byref(d), null) not in (0, -1)
        assert L.paged_decode_attention_multi(p, p, p, p, p, 3, 0.1, p, 4, p, multi - 1, ctypes.byref(d), null) == -1
        assert L.paged_decode_attention_multi(p, p, p, p, p, 3, 0.1, p, 4, p, multi, ctypes.byref(d), null) not in (0, -1)


# ------------------------------------------------------------------ calls

def batch(name, B, n, d, heads=(16, 8), seed=0):
    """A call of this shape as f(workspace) -> out; the pools are shared."""
    H, hk = heads
    g = torch.Generator(DEV).manual_seed(seed + B + d)
    MB = -(-n // 16)
    nb = 512
    bt = torch.randint(0, nb, (B, MB), generator=g, device=DEV, dtype=torch.int32)
    cl = torch.randint(max(1, n - 40), n + 1, (B,), generator=g, device=DEV, dtype=torch.int32)
    q = torch.randn(B, H, d, generator=g, device=DEV).bfloat16()
    if name in ("16-bit", "split", "multi"):
        kc, vc = (torch.randn(nb, hk, 16, d, generator=g, device=DEV).bfloat16() for _ in range(2))
        if name == "multi":
            qm = torch.randn(B, 3, H, d, generator=g, device=DEV).bfloat16()
            return lambda ws: pkv.paged_decode_attention_multi(qm, kc, vc, bt, cl, d ** -0.5, num_splits=4, workspace=ws)
        n_split = 3 if name == "split" else 0
        return lambda ws: pkv.paged_decode_attention(q, kc, vc, bt, cl, d ** -0.5, num_splits=n_split, workspace=ws)
    if name == "E4M3":
        kc, vc = (torch.randn(nb, hk, 16, d, generator=g, device=DEV).to(torch.float8_e4m3fn) for _ in range(2))
        s = torch.full((hk,), 0.02, device=DEV)
        return lambda ws: pkv.paged_decode_attention_fp8(q, kc, vc, s, s, bt, cl, d ** -0.5, workspace=ws)
    kc, vc = (torch.zeros(nb, hk, 16, d // 2 + 4, dtype=torch.uint8, device=DEV) for _ in range(2))
    k, v = (torch.randn(nb * 16, hk, d, generator=g, device=DEV).bfloat16() for _ in range(2))
    pkv.paged_kv_append_int4(k, v, torch.arange(nb * 16, dtype=torch.int32, device=DEV), kc, vc)
    return lambda ws: pkv.paged_decode_attention_int4(q, kc, vc, bt, cl, d ** -0.5, workspace=ws)


@pytest.mark.gpu
def test_results_do_not_depend_on_the_calls_before():
    """Batches that grow and shrink, two head sizes, all pool formats, splits and several tokens, on one workspace.
    The larger 16-bit and E4M3 batches hand out tails from the counters (shares of 48 blocks and more)."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    calls = [batch(*a) for a in (("4-bit", 64, 700, 128), ("16-bit", 300, 600, 128), ("16-bit", 64, 4000, 128),
                                 ("4-bit", 2000, 40, 128), ("E4M3", 300, 1200, 128), ("16-bit", 300, 600, 64),
                                 ("split", 40, 900, 128), ("16-bit", 100, 1700, 128), ("multi", 40, 900, 128),
                                 ("E4M3", 200, 1300, 128), ("4-bit", 33, 500, 64), ("16-bit", 1000, 200, 64),
                                 ("16-bit", 1, 30, 128))]
    want = []
    for c in calls:
        ws = torch.zeros(96 << 20, dtype=torch.uint8, device=DEV)
        want.append(c(ws).clone())
        assert not ws[:8].any()                             # the counters
    shared = torch.zeros(96 << 20, dtype=torch.uint8, device=DEV)
    rng = np.random.default_rng(0)
    for i in list(range(len(calls))) * 2 + list(rng.permutation(len(calls))):
        assert torch.equal(calls[i](shared), want[i]), i
        assert not shared[:8].any()
    pkv.paged_kv_check_status()


@pytest.mark.gpu
def test_workspaces_of_the_size_before_4_bit_pools():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    c = batch("16-bit", 300, 600, 128)
    d = dims(num_seqs=300, num_q_heads=16, max_blocks_per_seq=38)
    a, b = c(torch.zeros(automatic_bytes(d), dtype=torch.uint8, device=DEV)), c(None)
    assert torch.equal(a, b)
    for name, rows in (("split", 40 * 16 * 3), ("multi", 40 * 3 * 16 * 4)):
        c = batch(name, 40, 900, 128)
        exact = torch.empty(align(rows * 128 * 4) + align(rows * 4), dtype=torch.uint8, device=DEV)
        assert torch.equal(c(exact), c(None))
    pkv.paged_kv_check_status()
