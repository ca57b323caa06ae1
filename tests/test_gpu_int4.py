"""GPU parity of the 4-bit KV cache against the float64 oracle.

Append: the whole pool bit for bit.  Read-back: the oracle's values rounded
once, bit for bit.  Attention against the oracle over the dequantised pool,
elementwise |gpu - ref| <= u |ref| + w + 2^-11 H + 2^-13 A with
  u = eps/2 of the output's type (its one rounding),
  w = half of the type's smallest subnormal: a value below the smallest normal
      one (2^-14 in float16) is rounded to a multiple of eps * 2^-14 = 2^-24,
      so its one rounding moves it by up to 2^-25 whatever its size,
  H = the largest 7.5 * scale among the V rows attended (half a row's range):
      each weight is rounded to float16 (at most 2^-11 of it) and multiplies
      c - 7.5 steps, so the weighted mean moves by at most 2^-11 H,
  A = the largest |V| attended: the weights' own errors.  A logit is a float32
      sum of 128 products whose magnitudes add up to at most about 100 here
      (each partial sum rounded, 2^-24 of it: below 2^-14 in all), ex2.approx
      is good to 2^-22, and a weight's error counts twice (numerator and
      normaliser).
"""
import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_26_gb300 as pkv
import workloads as wl
from oracle import int4
from paged_kv_cache_26_gb300 import build as pkv_build
from paged_kv_cache_26_gb300.loop import DecodeLoop
from parity_helpers import bits, widen_out

pytestmark = pytest.mark.gpu
DEV = "cuda"
NAMES = {torch.float16: "fp16", torch.bfloat16: "bf16"}


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkv_build.build()


def oracle_store(k, v, slots, kp, vp):
    """int4_caches' store by the oracle (CPU)."""
    dt = NAMES[k.dtype]
    a, b = int4.kv_append_int4(kp.cpu().numpy(), vp.cpu().numpy(), bits(k), bits(v), slots.cpu().numpy(), dt)
    return [torch.from_numpy(a).to(kp.device), torch.from_numpy(b).to(vp.device)]


def gpu_store(k, v, slots, kp, vp):
    pkv.paged_kv_append_int4(k, v, slots, kp, vp)


def assert_attention(out, ref, dtype, kp_v, tables, lens, what=""):
    """out: GPU tensor [B][Hq][D]; ref float64; kp_v: V pool (numpy) as attended."""
    got = widen_out(out, NAMES[dtype])
    assert np.isfinite(got).all(), f"{what}: non-finite output"
    hk = kp_v.shape[1]
    g = ref.shape[1] // hk
    d = ref.shape[2]
    pairs = np.ascontiguousarray(int4.tiles(kp_v)[:, :, 8 * d:]).view(np.float16).reshape(kp_v.shape[0], hk, 16, 2)
    u = torch.finfo(dtype).eps / 2
    w = torch.finfo(dtype).smallest_normal * u
    for b in range(ref.shape[0]):
        n = int(lens[b])
        if n == 0:
            assert not got[b].any(), f"{what}: an empty context gives zeros"
            continue
        ids = np.asarray(tables[b, :-(-n // 16)], np.int64)
        pr = pairs[ids].astype(np.float64).transpose(0, 2, 1, 3).reshape(-1, hk, 2)[:n]
        H = (7.5 * pr[..., 0]).max(0)
        A = np.maximum(np.abs(pr[..., 1]), np.abs(pr[..., 1] + 15 * pr[..., 0])).max(0)
        tol = (2.0 ** -11 * H + 2.0 ** -13 * A).repeat(g)[:, None] + u * np.abs(ref[b]) + w
        err = np.abs(got[b] - ref[b])
        assert (err <= tol).all(), (what, b, n, float((err / tol).max()))


def check_step(w, caches, layer=0, fused=True):
    """One step through the GPU and the oracle: pools bit for bit, attention within the bound."""
    dtype = wl.DTYPES[w.spec.dtype]
    kc, vc = caches.k_cache[layer].to(DEV, copy=True), caches.v_cache[layer].to(DEV, copy=True)
    q, kn, vn = (t[layer].to(DEV) for t in (w.q, w.k_new, w.v_new))
    bt, cl = torch.from_numpy(w.block_tables).to(DEV), torch.from_numpy(w.context_lens).to(DEV)
    slots = pkv.paged_kv_slot_mapping(w.block_tables, w.context_lens)
    if fused:
        out = pkv.paged_decode_step_int4(q, kn, vn, kc, vc, bt, cl, w.scale)
    else:
        pkv.paged_kv_append_int4(kn, vn, torch.from_numpy(slots).to(DEV), kc, vc)
        out = pkv.paged_decode_attention_int4(q, kc, vc, bt, cl, w.scale)
    pkv.paged_kv_check_status()
    rk, rv = int4.kv_append_int4(caches.k_cache[layer].cpu().numpy(), caches.v_cache[layer].cpu().numpy(),
                                 bits(kn), bits(vn), slots, w.spec.dtype)
    assert np.array_equal(kc.cpu().numpy(), rk), "K pool differs from the oracle's append"
    assert np.array_equal(vc.cpu().numpy(), rv), "V pool differs from the oracle's append"
    ref = int4.decode_attention(widen_out(q.cpu(), w.spec.dtype), rk, rv, w.block_tables, w.context_lens, w.scale)
    assert_attention(out.cpu(), ref, dtype, rv, w.block_tables, w.context_lens, w.spec.name)
    return out


# ------------------------------------------------------------------ append and read

@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16], ids=["fp16", "bf16"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [1, 2, 3, 37, 160])
def test_append_and_read_bit_exact(n, d, dtype):
    g = torch.Generator().manual_seed(n + d)
    hk, nb = 3, 12
    mag = torch.exp(torch.empty(n, hk, 1).uniform_(-16, 9, generator=g))
    k = (torch.randn(n, hk, d, generator=g) * mag).to(dtype)
    v = (torch.randn(n, hk, d, generator=g) + 3 * torch.randn(n, hk, 1, generator=g)).to(dtype)
    k[0, 0] = 0.75                                              # a row of equal values
    v[-1, 1, :5] = torch.tensor([float("inf"), -float("inf"), 6e4, -0.0, 1e-30])
    slots = np.random.default_rng(n).permutation(nb * 16)[:n].astype(np.int32)
    if n > 30:
        slots[:24] = 32 + np.arange(24)                         # a run of tokens in order, as a prompt has
        slots[30] = -1
        rest = np.setdiff1d(np.arange(nb * 16), 32 + np.arange(24))
        slots[24:30], slots[31:] = rest[:6], rest[6:6 + n - 31]
    rng = np.random.default_rng(0)
    kp, vp = (rng.integers(0, 256, (nb, hk, 16, d // 2 + 4)).astype(np.uint8) for _ in range(2))
    rk, rv = int4.kv_append_int4(kp, vp, bits(k), bits(v), slots, NAMES[dtype])
    kd, vd = torch.from_numpy(kp).to(DEV), torch.from_numpy(vp).to(DEV)
    pkv.paged_kv_append_int4(k.to(DEV), v.to(DEV), torch.from_numpy(slots).to(DEV), kd, vd)
    pkv.paged_kv_check_status()
    assert np.array_equal(kd.cpu().numpy(), rk) and np.array_equal(vd.cpu().numpy(), rv)
    ko, vo = pkv.paged_kv_read_int4(torch.from_numpy(slots).to(DEV), kd, vd, dtype)
    pkv.paged_kv_check_status()
    for out, pool, is_v in ((ko, rk, False), (vo, rv, True)):
        val = int4.values(pool, is_v).transpose(0, 2, 1, 3).reshape(nb * 16, hk, d)[np.maximum(slots, 0)]
        val[slots < 0] = 0
        # the kernel rounds to float32 first; a second rounding to 16 bits may differ from the direct one only at a tie
        ref = torch.from_numpy(val.astype(np.float32)).to(dtype)
        assert torch.equal(out.cpu(), ref)


def test_append_across_blocks_as_a_prompt():
    """Odd starts, odd ends and block borders of prompt appends, several KV heads."""
    d, hk, nb, dtype = 128, 5, 20, torch.bfloat16
    table = np.random.default_rng(3).permutation(nb).astype(np.int32)
    for start, stop in ((0, 16), (0, 33), (5, 6), (7, 40), (15, 49), (1, 300)):
        pos = np.arange(start, stop)
        slots = (table[pos // 16] * 16 + pos % 16).astype(np.int32)
        g = torch.Generator().manual_seed(start)
        k, v = (torch.randn(len(pos), hk, d, generator=g).to(dtype) for _ in range(2))
        kp, vp = (np.full((nb, hk, 16, 68), 0xA5, np.uint8) for _ in range(2))
        rk, rv = int4.kv_append_int4(kp, vp, bits(k), bits(v), slots, "bf16")
        kd, vd = torch.from_numpy(kp).to(DEV), torch.from_numpy(vp).to(DEV)
        pkv.paged_kv_append_int4(k.to(DEV), v.to(DEV), torch.from_numpy(slots).to(DEV), kd, vd)
        assert np.array_equal(kd.cpu().numpy(), rk) and np.array_equal(vd.cpu().numpy(), rv), (start, stop)


def test_slots_past_the_pool_are_skipped_and_flagged():
    k = torch.ones(2, 2, 64, dtype=torch.float16, device=DEV)
    kp = torch.zeros(2, 2, 16, 36, dtype=torch.uint8, device=DEV)
    vp = torch.zeros_like(kp)
    for slots in ([32, 0], [-1, 1 << 30]):
        s = torch.tensor(slots, dtype=torch.int32, device=DEV)
        pkv.paged_kv_append_int4(k, k, s, kp, vp)
        with pytest.raises(pkv.PagedKVError) as e:
            pkv.paged_kv_check_status()
        assert e.value.code == -6
        ko, vo = pkv.paged_kv_read_int4(s, kp, vp, torch.float16)
        with pytest.raises(pkv.PagedKVError):
            pkv.paged_kv_check_status()
        assert not ko[s >= 32].any() and not ko[s < 0].any()
    assert kp[1].sum() == 0


# ------------------------------------------------------------------ attention

REDUCED = [
    wl.TINY,
    wl.TINY.replace(name="tiny_bf16", dtype="bf16", num_q_heads=6),
    wl.TINY.replace(name="tiny_d128_mqa7", head_dim=128, num_kv_heads=1, num_q_heads=7, pool=("factor", 2.0)),
    wl.LLAMA3_8B.replace(name="llama8b_small", batch=6, lengths=("uniform", 1, 700)),
    wl.MHA_7B_B16.replace(name="mha_small", batch=3, lengths=("constant", 333), num_layers=2),
    wl.LLAMA70B_TAIL.replace(name="70b_small", batch=24, lengths=("lognormal", 200.0, 1.0, 1, 900),
                             shared_prefix=(4, 64)),
    wl.LONG_CTX.replace(name="long_small", batch=2, lengths=("constant", 2100)),
    wl.LLAMA3_8B.replace(name="group5_fp16", batch=5, num_q_heads=15, num_kv_heads=3, dtype="fp16",
                         lengths=("uniform", 1, 1500)),
]


@pytest.mark.parametrize("fused", [True, False])
@pytest.mark.parametrize("spec", REDUCED, ids=lambda s: s.name)
def test_reduced_configs_every_output(spec, fused):
    w = wl.generate(spec, seed=5)
    caches = wl.int4_caches(w, oracle_store)
    for layer in range(len(w.q)):
        check_step(w, caches, layer, fused)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [(1,), (2, 1), (5, 0, 7), (15, 16, 17), (31, 32, 33, 48, 49), (4096, 1, 1, 1), (0, 0)])
def test_edge_lengths(lens, d):
    spec = wl.LLAMA3_8B.replace(name="custom", batch=len(lens), lengths=("fixed", tuple(lens)), head_dim=d,
                                pool=("factor", 1.5), num_q_heads=16, num_kv_heads=2)
    w = wl.generate(spec, seed=2)
    check_step(w, wl.int4_caches(w, oracle_store))


@pytest.mark.parametrize("spec", [wl.LLAMA3_8B, wl.LONG_CTX.replace(batch=2), wl.MHA_7B_B16.replace(batch=2)],
                         ids=lambda s: s.name)
def test_full_lengths_every_output(spec):
    w = wl.generate(spec, seed=0, device=DEV, layers=1)
    check_step(w, wl.int4_caches(w, gpu_store))


def test_maximum_batch():
    spec = wl.LLAMA3_8B.replace(name="b2048", batch=2048, lengths=("uniform", 1, 40), num_q_heads=8, num_kv_heads=2)
    w = wl.generate(spec, seed=4, device=DEV)
    check_step(w, wl.int4_caches(w, gpu_store))


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("mag", [2e-6, 1e-3, 300.0])
def test_magnitudes_of_v(mag, dtype):
    """Scales from float16 subnormals upwards, rows of very different scales in one context."""
    spec = wl.LLAMA3_8B.replace(name=f"mag{mag}", batch=3, lengths=("fixed", (3, 70, 600)), dtype=dtype,
                                num_q_heads=8, num_kv_heads=2, pool=("factor", 1.5))
    w = wl.generate(spec, seed=8)
    g = torch.Generator().manual_seed(1)
    f = torch.exp(torch.empty(w.v_cache[0].shape[:3] + (1,)).uniform_(-3, 3, generator=g)) * mag
    w.v_cache[0] = (w.v_cache[0].float() * f).to(w.v_cache[0].dtype)
    w.v_new[0] = (w.v_new[0].float() * mag).to(w.v_new[0].dtype)
    check_step(w, wl.int4_caches(w, oracle_store))


def test_offset_rows_long_context():
    """A common offset many times the spread, over a long context: the part
    that cancels must not cost the output its low bits."""
    spec = wl.LLAMA3_8B.replace(name="offset", batch=1, lengths=("constant", 20000), num_q_heads=8, num_kv_heads=1)
    w = wl.generate(spec, seed=3, device=DEV)
    w.v_cache[0] += 4.0
    w.k_cache[0] += 1.0
    check_step(w, wl.int4_caches(w, gpu_store))


def test_constant_rows_have_scale_zero():
    spec = wl.LLAMA3_8B.replace(name="const", batch=2, lengths=("fixed", (40, 9)), num_q_heads=8, num_kv_heads=2,
                                pool=("factor", 1.5))
    w = wl.generate(spec, seed=1)
    w.v_cache[0] = torch.where(torch.isnan(w.v_cache[0]), w.v_cache[0], torch.full_like(w.v_cache[0], 1.5))
    w.v_new[0].fill_(1.5)
    out = check_step(w, wl.int4_caches(w, oracle_store))
    assert torch.equal(out.cpu(), torch.full_like(out.cpu(), 1.5))


def test_one_token_returns_its_row():
    spec = wl.TINY.replace(name="one", batch=3, lengths=("constant", 1), pool=("fixed", 8))
    w = wl.generate(spec, seed=1)
    caches = wl.int4_caches(w, oracle_store)
    out = check_step(w, caches)
    slots = pkv.paged_kv_slot_mapping(w.block_tables, w.context_lens)
    _, rv = int4.kv_append_int4(caches.k_cache[0].numpy(), caches.v_cache[0].numpy(), bits(w.k_new[0]),
                                bits(w.v_new[0]), slots, "fp16")
    val = int4.values(rv, True).transpose(0, 2, 1, 3).reshape(-1, 2, 64)[slots]
    ref = torch.from_numpy(val).half().repeat_interleave(4, 1)
    assert (out.cpu().float() - ref.float()).abs().max() <= 2.0 ** -11 * ref.float().abs().max()


def test_fused_and_separate_give_identical_bits():
    w = wl.generate(REDUCED[3], seed=9)
    caches = wl.int4_caches(w, oracle_store)
    a, b = check_step(w, caches, fused=True), check_step(w, caches, fused=False)
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_repeated_calls_give_identical_bits_and_a_reusable_workspace():
    w = wl.generate(wl.LLAMA3_8B.replace(batch=9), seed=9, device=DEV)
    c = wl.int4_caches(w, gpu_store)
    bt, cl = torch.from_numpy(w.block_tables).to(DEV), torch.from_numpy(w.context_lens - 1).to(DEV)
    ws = pkv.make_workspace_int4(w.q[0], c.k_cache[0], bt)
    outs = [pkv.paged_decode_attention_int4(w.q[0], c.k_cache[0], c.v_cache[0], bt, cl, w.scale, workspace=ws).clone()
            for _ in range(3)]
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


# ------------------------------------------------------------------ bad inputs, streams, graphs

def test_bad_block_ids_and_lengths_are_flagged_and_read_as_zeros():
    spec = wl.LLAMA3_8B.replace(name="bad", batch=3, lengths=("fixed", (70, 40, 90)), num_q_heads=8, num_kv_heads=2,
                                pool=("factor", 1.5))
    w = wl.generate(spec, seed=1)
    c = wl.int4_caches(w, oracle_store)
    kc, vc = c.k_cache[0].to(DEV), c.v_cache[0].to(DEV)
    for bad in (-1, w.num_blocks, 1 << 30):
        tables = w.block_tables.copy()
        tables[0, 1], tables[2, 2], tables[2, 3] = bad, bad, bad
        lens = (w.context_lens - 1).astype(np.int32)
        out = pkv.paged_decode_attention_int4(w.q[0].to(DEV), kc, vc, torch.from_numpy(tables).to(DEV),
                                              torch.from_numpy(lens).to(DEV), w.scale)
        with pytest.raises(pkv.PagedKVError) as e:
            pkv.paged_kv_check_status()
        assert e.value.code == -6
        kz, vz = (np.concatenate([p.cpu().numpy(), np.zeros_like(p[:1].cpu().numpy())]) for p in (kc, vc))
        tables[tables == bad] = w.num_blocks
        ref = int4.decode_attention(widen_out(w.q[0], "bf16"), kz, vz, tables, lens, w.scale)
        assert_attention(out.cpu(), ref, torch.bfloat16, vz, tables, lens, f"id {bad}")
    lens = np.array([w.max_blocks * 16 + 5, -3, 40], np.int32)
    tables = np.where(w.block_tables < 0, 0, w.block_tables).astype(np.int32)
    kz, vz = (torch.where(p == 0xFF, torch.zeros_like(p), p) for p in (kc, vc))  # the unused slots, without NaN pairs
    out = pkv.paged_decode_attention_int4(w.q[0].to(DEV), kz, vz, torch.from_numpy(tables).to(DEV),
                                          torch.from_numpy(lens).to(DEV), w.scale)
    with pytest.raises(pkv.PagedKVError):
        pkv.paged_kv_check_status()
    assert not out[1].any() and torch.isfinite(out.float()).all()


def test_bf16_query_beyond_fp16_range_is_flagged():
    spec = wl.LLAMA3_8B.replace(name="qbig", batch=2, lengths=("fixed", (20, 40)), pool=("factor", 1.5))
    w = wl.generate(spec, seed=1)
    c = wl.int4_caches(w, oracle_store)
    w.q[0][1, 3, 5] = 1.0e5
    with pytest.raises(pkv.PagedKVError) as e:
        check_step(w, c)
    assert e.value.code == -6 and "fp16 range" in str(e.value)
    pkv.paged_kv_check_status()


def test_inputs_written_on_the_stream_right_before_the_step():
    """A serving loop that advances lengths and tables on the GPU between steps."""
    B, hk, h, d, nb = 6, 2, 8, 128, 64
    g = torch.Generator().manual_seed(0)
    perm = torch.randperm(nb, generator=g).int()
    lens = torch.tensor([0, 14, 15, 16, 31, 47], dtype=torch.int32)
    tables = torch.full((B, 6), -1, dtype=torch.int32)
    full = perm[:B * 6].view(B, 6)
    kp, vp = (torch.full((nb, hk, 16, 68), 0xFF, dtype=torch.uint8, device=DEV) for _ in range(2))
    rows, slots = [], []
    for b in range(B):
        n = -(-int(lens[b]) // 16)
        tables[b, :n] = full[b, :n]
        slots += [int(full[b, p // 16]) * 16 + p % 16 for p in range(int(lens[b]))]
    k0, v0 = (torch.randn(len(slots), hk, d, generator=g).bfloat16() for _ in range(2))
    st = torch.tensor(slots, dtype=torch.int32)
    pkv.paged_kv_append_int4(k0.to(DEV), v0.to(DEV), st.to(DEV), kp, vp)
    rk, rv = int4.kv_append_int4(np.full(kp.shape, 0xFF, np.uint8), np.full(kp.shape, 0xFF, np.uint8), bits(k0),
                                 bits(v0), slots, "bf16")
    lens_d, tables_d, full_d = lens.to(DEV), tables.to(DEV), full.to(DEV)
    seqs = torch.arange(B, device=DEV)
    q = torch.randn(20, B, h, d, generator=g).bfloat16()
    kn, vn = (torch.randn(20, B, hk, d, generator=g).bfloat16() for _ in range(2))
    qd, knd, vnd = q.to(DEV), kn.to(DEV), vn.to(DEV)
    ws = pkv.make_workspace_int4(qd[0], kp, tables_d)
    outs = []
    for i in range(20):
        j = (lens_d // 16).long()
        tables_d.index_put_((seqs, j), full_d[seqs, j])
        lens_d.add_(1)
        outs.append(pkv.paged_decode_step_int4(qd[i], knd[i], vnd[i], kp, vp, tables_d, lens_d, d ** -0.5,
                                               workspace=ws))
    pkv.paged_kv_check_status()
    for i in range(20):
        n = (lens + 1 + i).numpy()
        sl = [int(full[b, (n[b] - 1) // 16]) * 16 + (n[b] - 1) % 16 for b in range(B)]
        rk, rv = int4.kv_append_int4(rk, rv, bits(kn[i]), bits(vn[i]), sl, "bf16")
        ref = int4.decode_attention(widen_out(q[i], "bf16"), rk, rv, full.numpy(), n, d ** -0.5)
        assert_attention(outs[i].cpu(), ref, torch.bfloat16, rv, full.numpy(), n, f"step {i}")
    assert np.array_equal(kp.cpu().numpy(), rk) and np.array_equal(vp.cpu().numpy(), rv)


@pytest.mark.parametrize("batch", [6, 40, 200])
@pytest.mark.parametrize("kind", ["lengths", "tables", "garbage", "zeros"])
def test_stale_inputs_before_the_grid_wait_are_rebuilt(kind, batch):
    """The prologue is handed other lengths and tables than the real ones: outputs and pools are the normal step's."""
    spec = wl.LLAMA3_8B.replace(name="stale", batch=batch, lengths=("uniform", 1, 900), num_q_heads=8, num_kv_heads=2)
    w = wl.generate(spec, seed=batch)
    c = wl.int4_caches(w, oracle_store)
    q, kn, vn = (t[0].to(DEV) for t in (w.q, w.k_new, w.v_new))
    bt, cl = torch.from_numpy(w.block_tables).to(DEV), torch.from_numpy(w.context_lens).to(DEV)
    g = torch.Generator().manual_seed(1)
    sl, st = cl.clone(), bt.clone()
    if kind == "lengths":
        sl = (cl - 1).clamp(min=0)
    elif kind == "tables":
        st[:, 0] = st[:, 0].roll(1)
    elif kind == "garbage":
        sl = torch.randint(-50, 4 * 900, cl.shape, generator=g, dtype=torch.int32).to(DEV)
        st = torch.randint(-5, w.num_blocks + 5, bt.shape, generator=g, dtype=torch.int32).to(DEV)
    else:
        sl.zero_()
    for append in (True, False):
        kc, vc = c.k_cache[0].to(DEV, copy=True), c.v_cache[0].to(DEV, copy=True)
        if not append:
            pkv.paged_kv_append_int4(kn, vn, torch.from_numpy(pkv.paged_kv_slot_mapping(w.block_tables, w.context_lens)
                                                              ).to(DEV), kc, vc)
        k2, v2 = kc.clone(), vc.clone()
        if append:
            want = pkv.paged_decode_step_int4(q, kn, vn, kc, vc, bt, cl, w.scale)
        else:
            want = pkv.paged_decode_attention_int4(q, kc, vc, bt, cl, w.scale)
        got = pkv.paged_kv_selftest_stale_prologue_int4(q, kn if append else None, vn if append else None, k2, v2, bt,
                                                        cl, st, sl, w.scale)
        pkv.paged_kv_check_status()
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))
        assert torch.equal(kc, k2) and torch.equal(vc, v2)


def test_offsets_past_32_bits():
    """Pools of more than 4 GB: blocks near their end, through every call that addresses them."""
    hk, d, nb = 8, 128, 520_000                    # 4.5 GB each
    kc, vc = (torch.empty(nb, hk, 16, 68, dtype=torch.uint8, device=DEV) for _ in range(2))
    assert kc.numel() > 1 << 32
    lens = [100, 33]
    ids = torch.tensor([[nb - 1, 3, nb - 7, nb - 2, nb - 3, nb - 4, 9], [nb - 5, nb - 6, nb - 9, -1, -1, -1, -1]],
                       dtype=torch.int32)
    ks, vs = (torch.zeros(10, hk, 16, 68, dtype=torch.uint8, device=DEV) for _ in range(2))
    ids_s = torch.tensor([[0, 1, 2, 3, 4, 5, 6], [7, 8, 9, -1, -1, -1, -1]], dtype=torch.int32)  # a small pool
    g = torch.Generator().manual_seed(0)
    for b, n in enumerate(lens):
        k, v = (torch.randn(n, hk, d, generator=g).bfloat16().to(DEV) for _ in range(2))
        pos = torch.arange(n)
        for t, kp, vp in ((ids, kc, vc), (ids_s, ks, vs)):
            slots = (t[b, pos // 16] * 16 + pos % 16).int().to(DEV)
            pkv.paged_kv_append_int4(k, v, slots, kp, vp)
            ko, vo = pkv.paged_kv_read_int4(slots, kp, vp, torch.bfloat16)
            if kp is kc:
                far = (ko, vo)
        assert torch.equal(ko, far[0]) and torch.equal(vo, far[1])
    q = torch.randn(2, 16, d, generator=g).bfloat16().to(DEV)
    kn, vn = (torch.randn(2, hk, d, generator=g).bfloat16().to(DEV) for _ in range(2))
    cl = torch.tensor(lens, dtype=torch.int32, device=DEV) + 1
    outs = [pkv.paged_decode_step_int4(q, kn, vn, kp, vp, t.to(DEV), cl, d ** -0.5)
            for t, kp, vp in ((ids, kc, vc), (ids_s, ks, vs))]
    pkv.paged_kv_check_status()
    assert torch.equal(outs[0], outs[1])
    pkv.paged_kv_copy_blocks(kc, vc, torch.tensor([[nb - 1, nb - 8]], dtype=torch.int32, device=DEV))
    pkv.paged_kv_check_status()
    assert torch.equal(kc[nb - 8], ks[0]) and torch.equal(vc[nb - 8], vs[0])


def test_another_stream_and_captured_graphs():
    w = wl.generate(REDUCED[3], seed=4)
    c = wl.int4_caches(w, oracle_store)
    kc, vc = c.k_cache[0].to(DEV), c.v_cache[0].to(DEV)
    bt, cl = torch.from_numpy(w.block_tables).to(DEV), torch.from_numpy(w.context_lens - 1).to(DEV)
    q = w.q[0].to(DEV)
    want = pkv.paged_decode_attention_int4(q, kc, vc, bt, cl, w.scale)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = pkv.paged_decode_attention_int4(q, kc, vc, bt, cl, w.scale, stream=side,
                                          workspace=pkv.make_workspace_int4(q, kc, bt))
    side.synchronize()
    assert torch.equal(got, want)
    graphs, outs = [], []
    for _ in range(2):
        ws, out = pkv.make_workspace_int4(q, kc, bt), torch.empty_like(q)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            pkv.paged_decode_attention_int4(q, kc, vc, bt, cl, w.scale, out=out, workspace=ws)
        graphs.append(gr)
        outs.append((out, ws))
    for gr in graphs * 3:
        gr.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for o, _ in outs)
    q.mul_(0.5)
    cl.sub_(1)
    want = pkv.paged_decode_attention_int4(q, kc, vc, bt, cl, w.scale)
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0][0], want)
    pkv.paged_kv_check_status()


# ------------------------------------------------------------------ block copies and the decode loop

@pytest.mark.parametrize("d", [64, 128])
def test_copy_blocks(d):
    rng = np.random.default_rng(0)
    kp, vp = (torch.from_numpy(rng.integers(0, 256, (9, 3, 16, d // 2 + 4)).astype(np.uint8)) for _ in range(2))
    pairs = torch.tensor([[0, 4], [2, 8], [0, 5]], dtype=torch.int32)
    kd, vd = kp.to(DEV), vp.to(DEV)
    pkv.paged_kv_copy_blocks(kd, vd, pairs.to(DEV))
    pkv.paged_kv_check_status()
    for a, b in ((kp, kd), (vp, vd)):
        a = a.clone()
        a[[4, 8, 5]] = a[[0, 2, 0]]
        assert torch.equal(a, b.cpu())


@pytest.mark.parametrize("d", [64, 128])
def test_decode_loop_over_a_4bit_pool(d):
    """Admission, steps, a fork with copy-on-write and block reuse, every step against the oracle."""
    H, hk, B, dtype = 8, 2, 4, torch.bfloat16
    loop = DecodeLoop(num_blocks=40, num_q_heads=H, num_kv_heads=hk, head_dim=d, max_batch=B, max_context=128,
                      dtype=dtype, int4=True)
    g = torch.Generator().manual_seed(d)
    hist = {}                                   # batch slot -> list of (k, v) rows
    def admit(p, gen):
        k, v = (torch.randn(p, hk, d, generator=g).to(dtype) for _ in range(2))
        s = loop.admit(k.to(DEV), v.to(DEV), gen)
        torch.cuda.synchronize()
        hist[s] = [k, v]
    admit(21, 9)
    admit(1, 30)
    for step in range(24):
        if step == 5:
            f = loop.fork(0, 12)
            hist[f] = [x.clone() for x in hist[0]]
        if step in (10, 13) and loop.num_free_slots:
            admit(17 + step, 6)
        q = torch.randn(B, H, d, generator=g).to(dtype)
        kn, vn = (torch.randn(B, hk, d, generator=g).to(dtype) for _ in range(2))
        out = loop.step(q.to(DEV), kn.to(DEV), vn.to(DEV)).cpu()
        torch.cuda.synchronize()
        pkv.paged_kv_check_status()
        for s in range(B):
            if s not in hist:
                assert not out[s].any()
                continue
            hist[s] = [torch.cat([hist[s][0], kn[s:s + 1]]), torch.cat([hist[s][1], vn[s:s + 1]])]
            n = hist[s][0].shape[0]
            nb = -(-n // 16)
            pools = [np.zeros((nb, hk, 16, d // 2 + 4), np.uint8) for _ in range(2)]
            rk, rv = int4.kv_append_int4(*pools, bits(hist[s][0]), bits(hist[s][1]), np.arange(n), "bf16")
            t = np.arange(nb)[None]
            ref = int4.decode_attention(widen_out(q[s:s + 1], "bf16"), rk, rv, t, [n], d ** -0.5)
            assert_attention(out[s:s + 1], ref, dtype, rv, t, [n], f"step {step} slot {s}")
        for s in loop.finish_step():
            del hist[s]
    assert loop.stats()["copied_blocks"] >= 1
    with pytest.raises(ValueError):
        DecodeLoop(num_blocks=4, num_q_heads=8, num_kv_heads=2, head_dim=128, max_batch=1, max_context=16, int4=True,
                   k_scale=torch.ones(2, device=DEV), v_scale=torch.ones(2, device=DEV))


def test_wrong_shapes_are_refused():
    q = torch.zeros(2, 8, 128, dtype=torch.bfloat16, device=DEV)
    kc = torch.zeros(4, 2, 16, 68, dtype=torch.uint8, device=DEV)
    bt, cl = torch.zeros(2, 1, dtype=torch.int32, device=DEV), torch.ones(2, dtype=torch.int32, device=DEV)
    ok = dict(q=q, k_cache=kc, v_cache=kc.clone(), block_tables=bt, context_lens=cl, scale=0.1)
    for bad in (dict(q=q[:, :, :64].contiguous()), dict(q=q.float()), dict(k_cache=kc.view(torch.int8)),
                dict(k_cache=kc[:, :, :, :36].contiguous()), dict(block_tables=bt[:1]), dict(context_lens=cl[:1]),
                dict(q=q.transpose(0, 1)), dict(block_tables=bt.long()), dict(out=torch.empty_like(q).half())):
        with pytest.raises(ValueError):
            pkv.paged_decode_attention_int4(**{**ok, **bad})
    with pytest.raises(pkv.PagedKVError) as e:
        pkv.paged_decode_attention_int4(**{**ok, "q": torch.zeros(2, 18, 128, dtype=torch.bfloat16, device=DEV)})
    assert e.value.code == -2


def test_a_strided_workspace_is_refused():
    kc, vc, q = (torch.zeros(4, 2, 16, 68, dtype=torch.uint8, device=DEV), torch.zeros(4, 2, 16, 68, dtype=torch.uint8,
                 device=DEV), torch.zeros(1, 8, 128, dtype=torch.half, device=DEV))
    bt, cl = torch.zeros(1, 2, dtype=torch.int32, device=DEV), torch.zeros(1, dtype=torch.int32, device=DEV)
    ws = torch.zeros(2 * pkv.make_workspace_int4(q, kc, bt).numel(), dtype=torch.uint8, device=DEV)
    with pytest.raises(ValueError):
        pkv.paged_decode_attention_int4(q, kc, vc, bt, cl, 0.1, workspace=ws[::2])


@pytest.mark.parametrize("group", [3, 4, 5, 8])
def test_many_units_merged_four_heads_at_a_time(group):
    """More heads than warps run at once: groups that four does not divide, units cut once or not at all, and one
    long sequence whose units have many pieces."""
    lens = np.random.default_rng(group).integers(0, 330, 450)
    lens[7], lens[100] = 5000, 0
    spec = wl.LLAMA3_8B.replace(name="many", batch=450, lengths=("fixed", tuple(int(max(n, 1)) for n in lens)),
                                num_q_heads=2 * group, num_kv_heads=2)
    w = wl.generate(spec, seed=group)
    check_step(w, wl.int4_caches(w, oracle_store))


@pytest.mark.parametrize("group", [1, 3, 8])
def test_one_head_in_many_pieces(group):
    spec = wl.LLAMA3_8B.replace(name="one", batch=2, lengths=("fixed", (20011, 3)), num_q_heads=group, num_kv_heads=1)
    w = wl.generate(spec, seed=group)
    check_step(w, wl.int4_caches(w, oracle_store))
