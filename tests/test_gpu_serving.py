"""GPU block tables and draft verification against the oracle: whole numbers,
so every comparison is for equality."""
import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_26_gb300 as pkv
from oracle import serving
from paged_kv_cache_26_gb300 import build as pkv_build
from parity_helpers import assert_close, bits, widen_out

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def built():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    pkv_build.build()


def i32(x):
    return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(DEV)


# ------------------------------------------------------------------ block tables

def pool_state(lens, MB, num_blocks, seed):
    rng = np.random.default_rng(seed)
    perm = rng.permutation(num_blocks).astype(np.int32)
    tables = np.full((len(lens), MB), -1, np.int32)
    at = 0
    for b, n in enumerate(-(-np.asarray(lens) // 16)):
        tables[b, :n] = perm[at:at + n]
        at += n
    free = np.full(num_blocks, -1, np.int32)
    free[:num_blocks - at] = perm[at:]
    return tables, free, num_blocks - at


def check_resize(lens, new, tables, free, num_free, spare=3, offset=0):
    d = dict(lens=i32(lens), tables=i32(tables), free=i32(free), num=i32([num_free]))
    total = int(np.maximum(np.asarray(new) - np.asarray(lens), 0).sum())
    slots = torch.full((total + spare + offset,), -7, dtype=torch.int32, device=DEV)
    offs = torch.empty(len(lens) + 1, dtype=torch.int32, device=DEV)
    pkv.paged_kv_resize_tables(d["lens"], i32(new), d["tables"], d["free"], d["num"], slot_mapping=slots[offset:],
                               token_offsets=offs)
    pkv.paged_kv_check_status()
    rs, ro, rt, rf, rn = serving.resize_tables(lens, new, tables, free, num_free)
    assert (slots[:offset] == -7).all()
    assert slots[offset:].tolist() == rs + [-1] * spare
    assert offs.tolist() == ro
    assert np.array_equal(d["tables"].cpu().numpy(), rt)
    assert d["num"].item() == rn and d["free"].tolist()[:rn] == rf[:rn]
    assert d["free"].tolist()[max(rn, num_free):] == list(free[max(rn, num_free):])  # behind the list: untouched
    assert d["lens"].tolist() == list(map(int, new))
    return rt, np.array(rf, np.int32), rn


@pytest.mark.parametrize("B,top,grow", [(1, 1, 1), (1, 40, 17), (3, 16, 16), (64, 500, 5), (200, 90, 40),
                                        (1000, 40, 20), (1025, 33, 3), (8192, 20, 2)])
def test_resize_grow_shrink_and_mixtures(B, top, grow):
    rng = np.random.default_rng(B)
    lens = rng.integers(0, top + 1, B)
    MB = -(-(top + grow) // 16) + 1
    nb = B * MB + 5
    t, f, n = pool_state(lens, MB, nb, B)
    new = lens + rng.integers(0, grow + 1, B)
    t, f, n = check_resize(lens, new, t, f, n, spare=5)
    mixed = rng.integers(0, MB * 16 + 1, B)                          # some grow, some shrink, some stay
    mixed[rng.random(B) < 0.2] = 0
    t, f, n = check_resize(new, mixed, t, f, n, spare=0, offset=1)   # an unaligned slot map
    t, f, n = check_resize(mixed, mixed, t, f, n)
    t, f, n = check_resize(mixed, np.zeros(B, int), t, f, n)
    assert n == nb and sorted(f) == list(range(nb))
    check_resize(np.zeros(B, int), np.full(B, MB * 16), t, f, n)     # to the table's last slot


def test_resize_prompts_of_many_tokens():
    rng = np.random.default_rng(1)
    lens = np.zeros(96, int)
    new = np.minimum(8192, np.rint(1000 * np.exp(rng.standard_normal(96)))).astype(int)
    new[::9] = 0
    t, f, n = pool_state(lens, 512, 20000, 2)
    check_resize(lens, new, t, f, n, spare=2)


def test_resize_growth_that_is_taken_back_leaves_the_list():
    lens = np.array([0, 15, 16, 31, 100])
    t, f, n = pool_state(lens, 10, 60, 3)
    t2, f2, n2 = check_resize(lens, lens + 21, t, f, n)
    _, f3, n3 = check_resize(lens + 21, lens, t2, f2, n2)
    assert n3 == n and np.array_equal(f3[:n], f[:n])


def test_resize_without_slots_and_without_sequences():
    lens = np.array([40, 3])
    t, f, n = pool_state(lens, 4, 20, 3)
    d = [i32(lens), i32(t), i32(f), i32([n])]
    assert pkv.paged_kv_resize_tables(d[0], i32([10, 30]), d[1], d[2], d[3]) == (None, None)
    pkv.paged_kv_check_status()
    _, _, rt, rf, rn = serving.resize_tables(lens, [10, 30], t, f, n)
    assert np.array_equal(d[1].cpu().numpy(), rt) and d[3].item() == rn and d[2].tolist()[:rn] == rf[:rn]
    none = i32(np.zeros((0,)))
    slots, offs = torch.zeros(5, dtype=torch.int32, device=DEV), torch.ones(1, dtype=torch.int32, device=DEV)
    pkv.paged_kv_resize_tables(none, none, i32(np.zeros((0, 4))), d[2], d[3], slots, offs)
    pkv.paged_kv_check_status()
    assert slots.tolist() == [-1] * 5 and offs.tolist() == [0] and d[3].item() == rn


@pytest.mark.parametrize("cluster", [False, True])
def test_resize_failures_change_nothing(cluster):
    lens = np.array([16, 5, 30])
    t, f, n = pool_state(lens, 40, 30, 3)
    many = 5000 if cluster else 600                                   # more than one CTA's pass of slots
    cases = [([16 + 16 * (n + 1), 5, 30], n, many, -5),               # one block too many
             ([16, 5, 641], n, many, -6), ([16, -1, 30], n, many, -6),
             ([17, 9, 31], n, 5, -6),                                 # six tokens, room for five
             ([17, 5, 30], -1, many, -6), ([17, 5, 30], 31, many, -6),
             ([0, 0, 0], 30, many, -6)]                               # more given than the list can hold
    for new, count, room, code in cases:
        d = [i32(lens), i32(t), i32(f), i32([count])]
        slots = torch.full((room,), 9, dtype=torch.int32, device=DEV)
        offs = torch.full((4,), 9, dtype=torch.int32, device=DEV)
        pkv.paged_kv_resize_tables(d[0], i32(new), d[1], d[2], d[3], slots, offs)
        with pytest.raises(pkv.PagedKVError) as e:
            pkv.paged_kv_check_status()
        assert e.value.code == code, new
        assert (slots == -1).all() and (offs == 0).all()
        for a, b in zip(d, (lens, t, f, [count])):
            assert np.array_equal(a.cpu().numpy(), np.asarray(b, np.int32))
    # exactly as many blocks as there are
    check_resize(lens, [16 + 16 * min(n, 39), 5, 30], t, f, n) if n <= 39 else None
    # ids outside the pool give slot -1 and a flag
    f2 = f.copy()
    f2[n - 1] = 30
    d = [i32(lens), i32(t), i32(f2), i32([n])]
    slots, _ = pkv.paged_kv_resize_tables(d[0], i32([18, 5, 30]), d[1], d[2], d[3], torch.zeros(
        2, dtype=torch.int32, device=DEV))
    with pytest.raises(pkv.PagedKVError) as e:
        pkv.paged_kv_check_status()
    assert e.value.code == -6 and slots.tolist() == [-1, -1]


def test_resize_wrong_shapes_are_refused():
    ok = [i32([1, 2]), i32([1, 2]), i32(np.zeros((2, 3))), i32(np.arange(6)), i32([6])]
    for k, bad in ((0, i32([1])), (1, i32([1, 2, 3])), (2, i32(np.zeros((3, 3)))), (2, i32(np.zeros(3))),
                   (3, i32(np.zeros((2, 3)))), (4, i32([1, 2])), (0, ok[0].long()), (2, ok[2].t())):
        args = list(ok)
        args[k] = bad
        with pytest.raises(ValueError):
            pkv.paged_kv_resize_tables(*args)
    for kw in (dict(slot_mapping=i32(np.zeros((2, 2)))), dict(token_offsets=i32([0, 0]))):
        with pytest.raises(ValueError):
            pkv.paged_kv_resize_tables(*ok, **kw)


def test_resize_in_a_captured_loop_on_another_stream():
    """A graph that grows every sequence by one token, replayed over block borders."""
    lens = np.array([0, 15, 40, 100])
    t, f, n = pool_state(lens, 12, 60, 5)
    d = [i32(lens), i32(t), i32(f), i32([n])]
    new, slots = i32(lens), torch.empty(6, dtype=torch.int32, device=DEV)
    log = torch.zeros(40, 6, dtype=torch.int32, device=DEV)
    step = torch.zeros(1, dtype=torch.int64, device=DEV)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            new.add_(1)
            pkv.paged_kv_resize_tables(d[0], new, d[1], d[2], d[3], slots)
            log.index_copy_(0, step, slots[None])
            step.add_(1)
        for _ in range(40):
            g.replay()
    side.synchronize()
    pkv.paged_kv_check_status()
    for i in range(40):
        s, _, t, f, n = serving.resize_tables(lens, lens + 1, t, f, n)
        lens = lens + 1
        assert log[i].tolist() == s + [-1, -1]
    assert np.array_equal(d[1].cpu().numpy(), t) and d[3].item() == n and d[2].tolist()[:n] == f[:n]


# ------------------------------------------------------------------ verification

def check_verify(target, draft, tokens, au, su, n=None, ctx=None, lens=None):
    a, out, new = pkv.paged_verify_draft(target, draft, tokens, au, su, draft_lens=n, context_lens=ctx)
    pkv.paged_kv_check_status()
    B, K = tokens.shape
    T, D = target.float().cpu().numpy(), draft.float().cpu().numpy() if draft is not None else None
    x, AU, SU = tokens.cpu().numpy(), au.cpu().numpy(), su.cpu().numpy()
    for b in range(B):
        if ctx is not None and ctx[b] <= 0:
            assert a[b] == 0 and (out[b] == -1).all() and new[b] == 0
            continue
        acc, tok = serving.verify_one(T[b], None if D is None else D[b], x[b], K if n is None else int(n[b]), AU[b],
                                      SU[b])
        want = list(x[b, :acc]) + [tok] + [-1] * (K - acc)
        assert a[b].item() == acc and out[b].tolist() == want, (b, a[b].item(), acc, out[b].tolist(), want)
        if ctx is not None:
            assert new[b].item() == max(int(ctx[b]) - (K - acc), 0)
    return a


def probabilities(gen, shape, dtype, sharp=2.0):
    return torch.softmax(sharp * torch.randn(shape, generator=gen), -1).to(dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16], ids=["fp32", "fp16", "bf16"])
@pytest.mark.parametrize("V", [1, 2, 3, 127, 128, 129, 2047, 4099, 16385])
def test_verify_vocabularies_and_types(V, dtype):
    g = torch.Generator().manual_seed(V)
    B, K = 6, 3
    t, d = probabilities(g, (B, K + 1, V), dtype), probabilities(g, (B, K, V), dtype)
    d[::2] = t[::2, :K]                                         # half of the sequences agree with their draft
    tok = torch.randint(0, V, (B, K), generator=g, dtype=torch.int32)
    if V > 3:
        tok[1] = t[1, :K].argmax(-1).int()
    au, su = torch.rand(B, K, generator=g), torch.rand(B, generator=g)
    su[:2] = torch.tensor([0.0, 1.0 - 2.0 ** -24])
    n = torch.tensor([3, 0, 1, 2, 3, 3], dtype=torch.int32)
    ctx = torch.tensor([4, 10, 0, 100, 7, 4], dtype=torch.int32)
    t, d, tok, au, su, n, ctx = (v.to(DEV) for v in (t, d, tok, au, su, n, ctx))
    a = check_verify(t, d, tok, au, su)
    assert a[0] == K                                            # u q < p always holds for p = q > 0
    check_verify(t, None, tok, au, su, n, ctx)
    check_verify(t, d, tok, au, su, n, ctx)


@pytest.mark.parametrize("V", [50257, 131072])
def test_verify_large_vocabularies(V):
    g = torch.Generator().manual_seed(V)
    B, K = 3, 2
    t, d = probabilities(g, (B, K + 1, V), torch.float32, 4.0), probabilities(g, (B, K, V), torch.float32, 4.0)
    tok = d.argmax(-1).int()
    au, su = torch.rand(B, K, generator=g), torch.rand(B, generator=g)
    check_verify(*(v.to(DEV) for v in (t, d, tok, au, su)))


def test_verify_the_largest_vocabulary():
    V = 1 << 22
    p = torch.zeros(1, 1, V)
    at = [0, 5, 127, 128, 1 << 20, V - 129, V - 1]
    p[0, 0, at] = torch.tensor([0.1, 0.2, 0.05, 0.25, 0.1, 0.2, 0.1])
    w = [serving.weight(float(v)) for v in p[0, 0, at]]
    us = [0.0, 0.05, 0.2, 0.31, 0.349, 0.5, 0.65, 0.8, 0.95, 0.999999]
    t = p.to(DEV).expand(len(us), 1, V)
    _, out, _ = pkv.paged_verify_draft(t, None, torch.empty(len(us), 0, dtype=torch.int32, device=DEV),
                                       torch.empty(len(us), 0, device=DEV), torch.tensor(us, device=DEV))
    u32 = np.array(us, np.float32)
    assert out[:, 0].tolist() == [at[serving.draw(w, float(u))] for u in u32]


def test_verify_many_drafts_and_none():
    g = torch.Generator().manual_seed(0)
    for K in (0, 1, 7, 31):
        t, d = probabilities(g, (4, K + 1, 50), torch.float32), probabilities(g, (4, K, 50), torch.float32)
        d[:3] = t[:3, :K] * 0.999
        tok = torch.randint(0, 50, (4, K), generator=g, dtype=torch.int32)
        au, su = torch.rand(4, K, generator=g), torch.rand(4, generator=g)
        ctx = torch.tensor([K + 1, 40, 99, 0], dtype=torch.int32)
        a = check_verify(*(v.to(DEV) for v in (t, d, tok, au, su)), ctx=ctx.to(DEV))
        assert a[:3].tolist() == [K] * 3


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16], ids=["fp32", "bf16"])
@pytest.mark.parametrize("shift", [0, 1, 4])
def test_verify_rows_inside_a_padded_vocabulary(shift, dtype):
    """Views: padded rows, sequences far apart, starts off the vector width; the padding holds NaN."""
    g = torch.Generator().manual_seed(shift)
    B, K, V = 3, 2, 1000
    big_t = torch.full((B + 1, K + 2, V + 11), float("nan"), dtype=dtype)
    big_d = torch.full((B, K + 5, V + 6), float("nan"), dtype=dtype)
    big_t[1:, 1:, shift:shift + V] = probabilities(g, (B, K + 1, V), dtype)
    big_d[:, :K, shift:shift + V] = probabilities(g, (B, K, V), dtype)
    big_t, big_d = big_t.to(DEV), big_d.to(DEV)
    t, d = big_t[1:, 1:, shift:shift + V], big_d[:, :K, shift:shift + V]
    tok = torch.randint(0, V, (B, K), generator=g, dtype=torch.int32).to(DEV)
    check_verify(t, d, tok, torch.rand(B, K, generator=g).to(DEV), torch.rand(B, generator=g).to(DEV))
    # one distribution for every row of a sequence
    check_verify(t[:, :1].expand(B, K + 1, V), None, tok, torch.rand(B, K, generator=g).to(DEV),
                 torch.rand(B, generator=g).to(DEV))


def test_verify_borders_of_the_draw():
    """u at every border of the running sum: the token is the first whose sum exceeds it."""
    p = torch.tensor([0.0, 0.25, 0.0, 0.5, 0.125, 0.125, 0.0])
    for u, want in ((0.0, 1), (0.25 - 2.0 ** -25, 1), (0.25, 3), (0.75 - 2.0 ** -24, 3), (0.75, 4), (0.875, 5),
                    (1.0 - 2.0 ** -24, 5), (1.0, 5), (7.0, 5), (-1.0, 1), (float("nan"), 1), (float("inf"), 5)):
        t = p.expand(1, 1, 7).contiguous().to(DEV)
        _, out, _ = pkv.paged_verify_draft(t, None, torch.empty(1, 0, dtype=torch.int32, device=DEV),
                                           torch.empty(1, 0, device=DEV), torch.tensor([u], device=DEV))
        assert out.item() == want, u
    # acceptance is strict: u q < p
    t = torch.tensor([[[0.25, 0.75], [0.5, 0.5]]], device=DEV)
    d = torch.tensor([[[0.5, 0.5]]], device=DEV)
    for u, want in ((0.5, 0), (0.5 - 2.0 ** -24, 1)):
        a, out, _ = pkv.paged_verify_draft(t, d, torch.zeros(1, 1, dtype=torch.int32, device=DEV),
                                           torch.tensor([[u]], device=DEV), torch.tensor([0.9], device=DEV))
        assert a.item() == want and out.tolist() == ([[0, 1]] if want else [[1, -1]])


def test_verify_weights_around_the_small_entries_border():
    """Entries around 2^-17, 2^-40 and ties of the rounding: the draw counts them as the oracle does."""
    small = np.float32(2.0 ** -17)
    vals = [np.nextafter(small, np.float32(0)), small, np.nextafter(small, np.float32(1)), 2.0 ** -41, 1.5 * 2.0 ** -40,
            2.5 * 2.0 ** -40, 3.5 * 2.0 ** -40, 2.0 ** -40, 2.0 ** -126, 1e-45, 0.0, 1.0, np.nextafter(np.float32(1), np.float32(0))]
    g = np.random.default_rng(0)
    p = np.array([vals[i] for i in g.integers(0, len(vals) - 3, 700)], np.float32)   # small ones only
    p[::97] = 2.0 ** -20
    w = [serving.weight(float(v)) for v in p]
    total = sum(w)
    us = np.concatenate([g.random(200), [0.0, 1 - 2.0 ** -24]]).astype(np.float32)
    t = torch.from_numpy(p).to(DEV).expand(len(us), 1, 700)
    _, out, _ = pkv.paged_verify_draft(t, None, torch.empty(len(us), 0, dtype=torch.int32, device=DEV),
                                       torch.empty(len(us), 0, device=DEV), torch.from_numpy(us).to(DEV))
    assert out[:, 0].tolist() == [serving.draw(w, float(u)) for u in us]
    for v in vals:                                             # one entry alone, another of the same weight after it
        q = np.array([v, v, 0.0], np.float32)
        w = [serving.weight(float(x)) for x in q]
        us = np.array([0.49999, 0.5, 0.75], np.float32)
        t = torch.from_numpy(q).to(DEV).expand(3, 1, 3)
        _, out, _ = pkv.paged_verify_draft(t, None, torch.empty(3, 0, dtype=torch.int32, device=DEV),
                                           torch.empty(3, 0, device=DEV), torch.from_numpy(us).to(DEV))
        assert out[:, 0].tolist() == [serving.draw(w, float(u)) for u in us], v
    assert total > 0


def test_verify_rows_without_a_residual_and_without_mass():
    V = 300
    t = torch.full((3, 2, V), 0.0)
    d = torch.full((3, 1, V), 0.0)
    t[0, 0, 7], d[0, 0, 7], d[0, 0, 9] = 0.25, 0.5, 0.5            # p <= q everywhere: drawn from p
    t[1, :, 3] = 2.0                                               # above 1 counts as 1
    d[1, 0, 5] = 1.0
    t[2, 0] = float("nan")                                         # no mass at all
    t[2, 0, 4] = -1.0
    tok = torch.tensor([[9], [5], [1]], dtype=torch.int32)
    au, su = torch.full((3, 1), 0.9), torch.tensor([0.999, 0.5, 0.5])
    a, out, _ = pkv.paged_verify_draft(*(v.to(DEV) for v in (t, d, tok, au, su)))
    pkv.paged_kv_check_status()
    assert a.tolist() == [0, 0, 0] and out.tolist() == [[7, -1], [3, -1], [-1, -1]]


def test_verify_bad_tokens_and_lengths_are_flagged():
    g = torch.Generator().manual_seed(0)
    t = probabilities(g, (4, 3, 100), torch.float32).to(DEV)
    tok = torch.tensor([[100, 1], [-1, 1], [5, 6], [5, 6]], dtype=torch.int32, device=DEV)
    n = torch.tensor([2, 2, 3, -2], dtype=torch.int32, device=DEV)
    au, su = torch.zeros(4, 2, device=DEV), torch.full((4,), 0.5, device=DEV)
    a, out, _ = pkv.paged_verify_draft(t, None, tok, au, su, draft_lens=n)
    with pytest.raises(pkv.PagedKVError) as e:
        pkv.paged_kv_check_status()
    assert e.value.code == -6
    assert a.tolist() == [0, 0, 2, 0] and (out[:2, 0] >= 0).all()
    T = t.cpu().numpy()
    assert out[0, 0].item() == serving.draw([serving.weight(v) for v in T[0, 0]], 0.5)


def test_verify_wrong_shapes_are_refused():
    t, d = torch.zeros(2, 3, 8, device=DEV), torch.zeros(2, 2, 8, device=DEV)
    x, au, su = torch.zeros(2, 2, dtype=torch.int32, device=DEV), torch.zeros(2, 2, device=DEV), torch.zeros(2, device=DEV)
    ok = dict(target_probs=t, draft_probs=d, draft_tokens=x, accept_u=au, sample_u=su)
    for bad in (dict(target_probs=t[:, :2]), dict(target_probs=t.double()), dict(draft_probs=d.half()),
                dict(draft_probs=d[:, :, :7]), dict(target_probs=t.transpose(1, 2)), dict(draft_tokens=x.long()),
                dict(accept_u=au[:1]), dict(sample_u=su[:1]), dict(draft_lens=x[0, :1]), dict(context_lens=su),
                dict(target_probs=torch.zeros(2, 3, 16, device=DEV)[:, :, ::2])):
        with pytest.raises(ValueError):
            pkv.paged_verify_draft(**{**ok, **bad})


# ------------------------------------------------------------------ all of it together

def test_speculative_rounds_on_the_gpu():
    """Reserve, attend and append the drafts (multi-token step), verify, give
    back: every round's tables, attention and tokens against the oracle, the
    host never reading a length."""
    B, H, hk, D, K, V, MB = 5, 8, 2, 64, 3, 257, 12
    rng = np.random.default_rng(0)
    g = torch.Generator().manual_seed(0)
    lens = np.array([0, 14, 31, 48, 5])
    t, f, n = pool_state(lens, MB, 50, 1)
    kc, vc = (torch.randn(50, hk, 16, D, generator=g).half() for _ in range(2))
    d = dict(lens=i32(lens), tables=i32(t), free=i32(f), num=i32([n]))
    kd, vd = kc.to(DEV), vc.to(DEV)
    kb, vb = bits(kc), bits(vc)
    slots = torch.empty(B * (K + 1), dtype=torch.int32, device=DEV)
    scale = D ** -0.5
    for step in range(8):
        q = torch.randn(B, K + 1, H, D, generator=g).half()
        kn, vn = (torch.randn(B, K + 1, hk, D, generator=g).half() for _ in range(2))
        target, draft = probabilities(g, (B, K + 1, V), torch.float32), probabilities(g, (B, K, V), torch.float32)
        draft[::2] = target[::2, :K]
        x = torch.randint(0, V, (B, K), generator=g, dtype=torch.int32)
        au, su = torch.rand(B, K, generator=g), torch.rand(B, generator=g)
        want_lens = d["lens"] + (K + 1)
        pkv.paged_kv_resize_tables(d["lens"], want_lens, d["tables"], d["free"], d["num"], slot_mapping=slots)
        out = pkv.paged_decode_step_multi(q.to(DEV), kn.to(DEV), vn.to(DEV), kd, vd, d["tables"], d["lens"], scale)
        a, tok, new = pkv.paged_verify_draft(target.to(DEV), draft.to(DEV), x.to(DEV), au.to(DEV), su.to(DEV),
                                             context_lens=d["lens"])
        pkv.paged_kv_resize_tables(d["lens"], new, d["tables"], d["free"], d["num"])
        pkv.paged_kv_check_status()
        # the same round on the CPU
        s, _, t, f, n = serving.resize_tables(lens, lens + K + 1, t, f, n)
        assert slots.tolist() == s
        full = lens + K + 1
        kb, vb = oracle.kv_append(kb, vb, bits(kn).reshape(-1, hk, D), bits(vn).reshape(-1, hk, D), np.array(s), 16)
        ref = oracle.decode_attention_multi(bits(q), kb, vb, np.where(t < 0, 0, t), full, K + 1, scale, "fp16", 16)
        assert_close(widen_out(out.cpu(), "fp16"), ref, f"round {step}")
        acc = []
        for b in range(B):
            r = serving.verify_one(target[b].numpy(), draft[b].numpy(), x[b].numpy(), K, au[b].numpy(), float(su[b]))
            assert (a[b].item(), tok[b, r[0]].item()) == r
            acc.append(r[0])
        lens = full - K + np.array(acc)
        _, _, t, f, n = serving.resize_tables(full, lens, t, f, n)
        assert d["lens"].tolist() == list(lens) and np.array_equal(d["tables"].cpu().numpy(), t)
        assert d["num"].item() == n and d["free"].tolist()[:n] == f[:n]
    assert np.array_equal(bits(kd), kb) and np.array_equal(bits(vd), vb)


def test_4bit_steps_over_tables_built_on_the_gpu():
    """A decode loop without host work: lengths advance, tables grow and the
    4-bit step runs inside one captured graph."""
    from oracle import int4
    from test_gpu_int4 import assert_attention
    B, H, hk, D, MB = 4, 8, 2, 128, 4
    g = torch.Generator().manual_seed(0)
    t, f, n = pool_state([0] * B, MB, 20, 1)
    d = [i32([0] * B), i32(t), i32(f), i32([n])]
    kp, vp = (torch.full((20, hk, 16, 68), 0xFF, dtype=torch.uint8, device=DEV) for _ in range(2))
    q, kn, vn = (torch.randn(B, x, D, generator=g).bfloat16().to(DEV) for x in (H, hk, hk))
    new, out = i32([0] * B), torch.empty(B, H, D, dtype=torch.bfloat16, device=DEV)
    ws = pkv.make_workspace_int4(q, kp, d[1])
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        new.add_(1)
        pkv.paged_kv_resize_tables(d[0], new, d[1], d[2], d[3])
        pkv.paged_decode_step_int4(q, kn, vn, kp, vp, d[1], d[0], D ** -0.5, out=out, workspace=ws)
    rk = rv = np.full((20, hk, 16, 68), 0xFF, np.uint8)
    for i in range(40):
        qi, ki, vi = (torch.randn(x.shape, generator=g).bfloat16() for x in (q, kn, vn))
        q.copy_(qi), kn.copy_(ki), vn.copy_(vi)
        gr.replay()
        torch.cuda.synchronize()
        s, _, t, f, n = serving.resize_tables([i] * B, [i + 1] * B, t, f, n)
        rk, rv = int4.kv_append_int4(rk, rv, bits(ki), bits(vi), s, "bf16")
        ref = int4.decode_attention(widen_out(qi, "bf16"), rk, rv, t, [i + 1] * B, D ** -0.5)
        assert_attention(out.cpu(), ref, torch.bfloat16, rv, t, [i + 1] * B, f"step {i}")
    pkv.paged_kv_check_status()
    assert np.array_equal(kp.cpu().numpy(), rk) and np.array_equal(vp.cpu().numpy(), rv)


@pytest.mark.parametrize("by_handle", [False, True])
def test_new_tensors_belong_to_the_calls_stream(by_handle):
    """Tensors a call makes when it is given a stream: not memory that work still
    queued on the current stream writes to."""
    rng = np.random.default_rng(6)
    gen = torch.Generator(DEV).manual_seed(6)
    kc, vc = (torch.zeros(24, 2, 16, 68, dtype=torch.uint8, device=DEV) for _ in range(2))
    k, v = (torch.randn(90, 2, 128, generator=gen, device=DEV).half() for _ in range(2))
    pkv.paged_kv_append_int4(k, v, i32(np.arange(90)), kc, vc)
    q = torch.randn(3, 8, 128, generator=gen, device=DEV).half()
    bt, cl = i32([[0, 1], [2, 3], [4, 5]]), i32([30, 9, 20])
    slots = i32(rng.permutation(90)[:33])
    p = torch.softmax(torch.randn(3, 4, 500, generator=gen, device=DEV), -1)
    d = torch.softmax(torch.randn(3, 3, 500, generator=gen, device=DEV), -1)
    tokens, u, su = i32(rng.integers(0, 500, (3, 3))), torch.full((3, 3), 0.2, device=DEV), torch.full((3,), 0.5, device=DEV)
    calls = [lambda s: pkv.paged_kv_read_int4(slots, kc, vc, torch.float16, stream=s),
             lambda s: (pkv.paged_decode_attention_int4(q, kc, vc, bt, cl, 0.1, stream=s),),
             lambda s: pkv.paged_verify_draft(p, d, tokens, u, su, context_lens=cl, stream=s)]
    side = torch.cuda.Stream()
    for call in calls:
        want = [t.clone() for t in call(None)]
        stale = [torch.empty_like(t) for t in want]
        torch.cuda.synchronize()
        torch.cuda._sleep(40_000_000)
        for t in stale:
            t.fill_(7)
        del stale
        got = call(side.cuda_stream if by_handle else side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
    pkv.paged_kv_check_status()
