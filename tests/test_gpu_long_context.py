"""GPU: the operators together, as a serving loop uses them: prompts enter in chunks
(tables grown on the GPU, keys turned on their way into the cache, attention of the
chunk, bounds of its blocks), then tokens are decoded over selected blocks, in one
captured step."""
import numpy as np
import pytest
import torch

import paged_kv_cache_26_gb300 as pkv
from long_context_helpers import DEV, assert_within, f64, i32, tolerance
from oracle import long_context as lc
from paged_kv_cache_26_gb300 import build as pkv_build

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("d,hq,hk", [(64, 4, 2), (128, 8, 1)])
def test_prompts_in_chunks_then_sparse_steps(dtype, d, hq, hk):
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkv_build.build()
    B, MB, NB, num, steps = 3, 80, 200, 9, 20
    prompts = np.array([700, 33, 260])
    gen = torch.Generator().manual_seed(1)
    total = prompts + steps
    q, k, v = ([torch.randn(int(n), h, d, generator=gen).to(dtype) for n in total] for h in (hq, hk, hk))
    inv = [10000.0 ** (-i / (d // 2)) for i in range(d // 2)]
    rope = pkv.make_rope(inv, d)
    scale = d ** -0.5
    # what attention should see: turned once, rounded once
    turned = [[torch.from_numpy(lc.rope(f64(x), np.arange(x.shape[0])[None], inv)).to(dtype) for x in xs] for xs in (q, k)]

    kc, vc = (torch.full((NB, hk, 16, d), float("nan"), dtype=dtype, device=DEV) for _ in range(2))
    bounds, scales = torch.zeros(NB, hk, 2, d, dtype=torch.int8, device=DEV), torch.zeros(NB, hk, device=DEV)
    tables, lens = i32(np.full((B, MB), -1)), i32([0] * B)
    free, num_free = i32(np.random.default_rng(0).permutation(NB)), i32([NB])

    def rows(xs, at, n):
        return torch.cat([x[a:a + m] for x, a, m in zip(xs, at, n)]).to(DEV)

    at = np.zeros(B, int)
    chunk_out = [[] for _ in range(B)]
    while (at < prompts).any():
        n = np.minimum(prompts - at, [256, 20, 130])
        T = int(n.sum())
        slots, offsets = torch.empty(T, dtype=torch.int32, device=DEV), torch.empty(B + 1, dtype=torch.int32, device=DEV)
        pkv.paged_kv_resize_tables(lens, i32(at + n), tables, free, num_free, slot_mapping=slots, token_offsets=offsets)
        pos = i32(np.concatenate([a + np.arange(m) for a, m in zip(at, n)]))
        qt = pkv.paged_kv_append_rope(rows(q, at, n), rows(k, at, n), rows(v, at, n), pos, rope, slots, kc, vc)
        out = pkv.paged_chunk_attention(qt, kc, vc, tables, lens, offsets, scale)
        pkv.paged_kv_update_bounds(kc, tables, lens, bounds, scales, offsets, T)
        pkv.paged_kv_check_status()
        for b, part in enumerate(out.split(n.tolist())):
            chunk_out[b].append(part)
        at += n
    # the cache holds the turned keys; the rotation is off by less than a rounding
    kp, vp, tab = f64(kc), f64(vc), tables.cpu().numpy()
    u = torch.finfo(dtype).eps / 2
    for b in range(B):
        got = np.stack([lc.gather(kp, tab[b], prompts[b], x) for x in range(hk)], 1)
        want = f64(turned[1][b][:prompts[b]])
        assert (np.abs(got - want) <= 2 * u * np.abs(want) + 2.0 ** -18).all()
        Q = f64(turned[0][b][:prompts[b]])
        off = np.array([0, prompts[b]])
        ref, mag = lc.chunk_attention(Q, kp, vp, tab[b:b + 1], prompts[b:b + 1], off, scale)
        # (queries off by a rounding as well: a logit moves by 2 u of its sum of magnitudes)
        K = np.nan_to_num(kp)
        S = scale * np.sqrt((Q ** 2).sum(-1)).max() * np.sqrt((K ** 2).sum(-1)).max()
        tol = tolerance(ref, mag, dtype, Q, kp, vp, scale, int(prompts[b])) + 4 * u * S * mag * 2
        assert_within(f64(torch.cat(chunk_out[b])), ref, tol)
    eb, es = lc.update_bounds(kc.float().cpu().numpy(), tab, prompts, np.concatenate([[0], np.cumsum(prompts)]),
                              np.zeros((NB, hk, 2, d), np.int8), np.zeros((NB, hk), np.float32))
    assert np.array_equal(bounds.cpu().numpy(), eb) and np.array_equal(scales.cpu().numpy(), es)

    # decode: one captured step, its inputs written into place
    sq, sk, sv = (torch.zeros(B, h, d, dtype=dtype, device=DEV) for h in (hq, hk, hk))
    slots, pos, new = i32([0] * B), i32([0] * B), lens.clone()
    sel, out = i32(np.zeros((B, hk, num))), torch.zeros(B, hq, d, dtype=dtype, device=DEV)
    qt = torch.empty_like(sq)
    ws = torch.empty(1 << 20, dtype=torch.uint8, device=DEV)

    def step():
        pos.copy_(lens)
        torch.add(lens, 1, out=new)
        pkv.paged_kv_resize_tables(lens, new, tables, free, num_free, slot_mapping=slots)
        pkv.paged_kv_append_rope(sq, sk, sv, pos, rope, slots, kc, vc, q_out=qt)
        pkv.paged_kv_update_bounds(kc, tables, lens, bounds, scales)
        pkv.paged_select_blocks(qt, bounds, scales, tables, lens, num, 1, 2, selected=sel, workspace=ws)
        pkv.paged_decode_attention_sparse(qt, kc, vc, tables, lens, sel, scale, out=out)

    def load(i):
        for dst, src in ((sq, q), (sk, k), (sv, v)):
            dst.copy_(torch.stack([x[p + i] for x, p in zip(src, prompts)]))

    load(0)
    step()
    pkv.paged_kv_check_status()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for i in range(1, steps):
        load(i)
        graph.replay()
    pkv.paged_kv_check_status()
    end = prompts + steps
    assert lens.tolist() == end.tolist()
    kp, vp, tab = f64(kc), f64(vc), tables.cpu().numpy()
    eb, es = lc.update_bounds(kc.float().cpu().numpy(), tab, end, np.concatenate([[0], np.cumsum(end)]), eb, es)
    assert np.array_equal(bounds.cpu().numpy(), eb) and np.array_equal(scales.cpu().numpy(), es)
    Q = f64(qt)
    assert np.array_equal(sel.cpu().numpy(), lc.select_blocks(qt.float().cpu().numpy(), eb, es, tab, end, num, 1, 2))
    ref, mag = lc.sparse_attention(Q, kp, vp, tab, end, sel.cpu().numpy(), scale)
    assert_within(f64(out), ref, tolerance(ref, mag, dtype, Q, kp, vp, scale, 16 * num, 11 if dtype == torch.float16 else 16))
