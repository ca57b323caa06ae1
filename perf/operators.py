"""Cases of the 4-bit KV cache, the GPU block tables and the draft verification.

Three operators of a serving loop over a paged KV cache, each in its plain form
(elementary torch operations) and, where ``own`` is true, as the package's calls:

* the 4-bit cache: a slot-mapped quantising append, reading rows back, and
  decode attention (with or without the fused append of the step's token);
* block tables and slot maps built on the GPU from the requests' lengths;
* verification of drafted tokens against the target's probabilities.

4-bit pools are uint8[num_blocks][Hkv][16][D/2 + 4].  The 16 * (D/2 + 4) bytes
of one (block, KV head) are its codes, then 16 float16 pairs (scale, minimum),
one per token; a value is scale * code + minimum with a code of 0..15.
  K codes: byte (D/2) t + d/2 holds dims d (low four bits) and d + 1 of token t.
  V codes: with G = D/8, the byte of (token t, dim d) is
    (t/8) 4D + (d/G) 4G + (t/2 % 4) G + (d%G)/4 * 4 + (t%2) 2 + (d%4)/2,
    low four bits first.
Row quantisation, in IEEE float32: x limited to +-65504, minimum =
float16(min x), scale = float16((max x - minimum) / 15), code =
round((x - minimum) * (1 / scale)) limited to 0..15 (0 where the scale is 0).
"""
import math
import statistics

import numpy as np
import torch

own = False

BLOCK = 16
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}
F16_MAX = 65504.0


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # a handful of short chats on a small model: launch latency decides
        dict(name="step tiny", op="step", batch=4, q_heads=8, kv_heads=2, head_dim=64, dtype="fp16",
             lengths="uniform", lo=17, hi=100, empty=0),
        # 64 chats on an 8-billion-parameter grouped-query model, the usual serving batch
        dict(name="step b64", op="step", batch=64, q_heads=32, kv_heads=8, head_dim=128, dtype="bf16",
             lengths="uniform", lo=512, hi=4096, empty=0),
        # multi-head attention of a 7-billion-parameter model, equal lengths
        dict(name="step mha", op="step", batch=16, q_heads=32, kv_heads=32, head_dim=128, dtype="fp16",
             lengths="uniform", lo=2048, hi=2048, empty=0),
        # eight long documents
        dict(name="attention long", op="attention", batch=8, q_heads=32, kv_heads=8, head_dim=128, dtype="bf16",
             lengths="uniform", lo=32768, hi=32768, empty=0),
        # 256 requests with a long tail of lengths, eight query heads to a KV head, a few slots empty
        dict(name="attention tail", op="attention", batch=256, q_heads=64, kv_heads=8, head_dim=128, dtype="bf16",
             lengths="lognormal", lo=80, hi=8192, empty=3),
        # prompts of eight requests enter the pool, and their rows are read back
        dict(name="append prompts", op="append", batch=8, kv_heads=8, head_dim=128, dtype="bf16", lo=517, hi=4001),
        # one token each of 61 requests, an odd number of heads
        dict(name="append rows", op="append", batch=61, kv_heads=5, head_dim=64, dtype="fp16", lo=1, hi=1),
        # 64 requests reserve room for five tokens (one and four drafts) and give it back
        dict(name="tables reserve", op="tables", batch=64, lo=512, hi=4096, grow=5, max_blocks=320),
        # 256 prompts are admitted at once, and leave again
        dict(name="tables admit", op="tables", batch=256, lo=0, hi=0, grow=0, max_blocks=512),
        # one request's four drafts
        dict(name="verify one", op="verify", batch=1, drafts=4, vocab=32768, dtype="fp32", ragged=False, certain=False),
        # 64 requests with seven drafts each
        dict(name="verify b64", op="verify", batch=64, drafts=7, vocab=131072, dtype="fp32", ragged=False,
             certain=False),
        # padded drafts looked up in the prompt (no draft probabilities), odd vocabulary, 16-bit probabilities
        dict(name="verify lookup", op="verify", batch=17, drafts=3, vocab=50257, dtype="bf16", ragged=True,
             certain=True),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["step", "attention", "append", "tables", "verify"])
    dtype = rng.choice(["fp16", "bf16"])
    if op in ("step", "attention"):
        head_dim = rng.choice([64, 128])
        kv_heads = _log_int(rng, 1, 32)
        group = rng.randint(1, 8)
        batch = _log_int(rng, 1, 300)
        # as many cached values as the longest listed batch at most
        most = 8 * 32768 * 8 * 128 // (batch * kv_heads * head_dim)
        hi = _log_int(rng, 1, min(40000, most))
        lo = rng.randint(1, hi) if rng.random() < 0.7 else hi
        lengths = "lognormal" if hi > 400 and rng.random() < 0.3 else "uniform"
        return dict(op=op, batch=batch, q_heads=kv_heads * group, kv_heads=kv_heads, head_dim=head_dim, dtype=dtype,
                    lengths=lengths, lo=lo, hi=hi, empty=rng.randint(0, batch // 4))
    if op == "append":
        head_dim = rng.choice([64, 128])
        kv_heads = _log_int(rng, 1, 32)
        batch = _log_int(rng, 1, 128)
        most = max(1, 8 * 2259 * 8 * 128 // (batch * kv_heads * head_dim))
        hi = _log_int(rng, 1, most)
        return dict(op=op, batch=batch, kv_heads=kv_heads, head_dim=head_dim, dtype=dtype,
                    lo=rng.randint(1, hi), hi=hi)
    if op == "tables":
        batch = _log_int(rng, 1, 256)
        hi = _log_int(rng, 1, 4096)
        return dict(op=op, batch=batch, lo=rng.randint(0, hi), hi=hi, grow=_log_int(rng, 1, 700),
                    max_blocks=rng.randint(300, 400))
    batch = _log_int(rng, 1, 64)
    return dict(op=op, batch=batch, drafts=rng.randint(1, 7), vocab=_log_int(rng, 1000, 131072),
                dtype=rng.choice(["fp32", "fp32", "bf16", "fp16"]), ragged=rng.random() < 0.5,
                certain=rng.random() < 0.25)


def _lengths(case, seed=None):
    """The batch's lengths: quantiles of the case's distribution, so that every
    seed has the same work, in the seed's order."""
    n = case["batch"]
    lo, hi = case["lo"], case["hi"]
    if case.get("lengths") == "lognormal":  # median and spread as of chat traffic, cut at both ends
        z = [statistics.NormalDist().inv_cdf((i + 0.5) / n) for i in range(n)]
        lens = [min(hi, max(lo, int(round(min(1000.0, hi / 8) * math.exp(v))))) for v in z]
    else:
        lens = [lo + int(round((hi - lo) * (i + 0.5) / n)) for i in range(n)]
    lens = np.asarray(lens, np.int64)
    lens[:case.get("empty", 0)] = 0
    return lens if seed is None else np.random.default_rng(seed).permutation(lens)


def _grown(case, seed=None):
    """Lengths of the tables' cases before and after their growth."""
    old = _lengths(case)
    n = case["batch"]
    if case["grow"]:
        new = old + case["grow"]
    else:  # admission: prompts with a long tail
        z = [statistics.NormalDist().inv_cdf((i + 0.5) / n) for i in range(n)]
        new = np.asarray([min(8192, max(80, int(round(1000 * math.exp(v))))) for v in z], np.int64)
    if seed is None:
        return old, new
    p = np.random.default_rng(seed).permutation(n)
    return old[p], new[p]


#: share of the verified sequences whose drafts are rejected somewhere, in these inputs
REJECTED = 0.75


def work(case):
    op = case["op"]
    if op in ("step", "attention"):
        lens = _lengths(case)
        tokens, blocks, b = int(lens.sum()), int((-(-lens // BLOCK)).sum()), case["batch"]
        d, h, hk = case["head_dim"], case["q_heads"], case["kv_heads"]
        row = d // 2 + 4
        n = 2 * tokens * hk * row + 2 * b * h * d * 2 + 4 * blocks + 4 * b
        if op == "step":
            n += 2 * b * hk * (2 * d + row)
        return {"bytes": n, "flops": 4 * tokens * h * d}
    if op == "append":
        d, hk, tokens = case["head_dim"], case["kv_heads"], int(_lengths(case).sum())
        # appended: values in, codes out; read back: codes in, values out
        return {"bytes": 2 * (2 * tokens * hk * (2 * d + d // 2 + 4) + 4 * tokens), "flops": 2 * 8 * tokens * hk * d}
    if op == "tables":
        old, new = _grown(case)
        tokens, taken = int((new - old).sum()), int((-(-new // BLOCK) + (-old // BLOCK)).sum())
        # growth: lengths in and out, blocks off the list and into the tables, slots and offsets out; then back
        return {"bytes": 2 * 12 * case["batch"] + 16 * taken + 4 * tokens + 4 * case["batch"], "flops": 0}
    size = 4 if case["dtype"] == "fp32" else 2
    b, k, v = case["batch"], case["drafts"], case["vocab"]
    rows = 1.0 if case["certain"] else 1.0 + REJECTED
    return {"bytes": int(rows * b * v * size) + b * k * (2 * size + 8) + b * (k + 1) * 4 + 16 * b, "flops": 0}


# ------------------------------------------------------------------ the 4-bit format, plainly

def _quantise(x):
    """Codes (uint8 [..., D]) and float16 pairs [..., 2] of rows [..., D]."""
    x = x.float().clamp(-F16_MAX, F16_MAX)
    low = x.amin(-1, keepdim=True).half()
    scale = ((x.amax(-1, keepdim=True) - low.float()) / 15.0).half()
    inv = torch.where(scale > 0, 1.0 / scale.float(), torch.zeros_like(x[..., :1]))
    codes = ((x - low.float()) * inv).round().clamp(0, 15).to(torch.uint8)
    return codes, torch.cat([scale, low], -1)


def _k_bytes(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def _views(pool, d):
    """The codes as K and as V order them, and the float16 pairs, of a pool."""
    nb, hk = pool.shape[:2]
    flat = pool.view(nb, hk, BLOCK * (d // 2 + 4))
    n = BLOCK * d // 2
    return (flat[..., :n].unflatten(-1, (BLOCK, d // 2)), flat[..., :n].unflatten(-1, (2, 8, 4, d // 32, 2, 2)),
            flat.view(torch.float16)[..., n // 2:].unflatten(-1, (BLOCK, 2)))


def _store(k_new, v_new, slots, k_cache, v_cache):
    """Plain append: rows [T][Hkv][D] at their slots; all slots are >= 0."""
    d = k_new.shape[-1]
    blk, t = slots.long() // BLOCK, slots.long() % BLOCK
    for x, pool, is_v in ((k_new, k_cache, False), (v_new, v_cache, True)):
        codes, pairs = _quantise(x)
        as_k, as_v, meta = _views(pool, d)
        b = _k_bytes(codes)
        if is_v:
            as_v[blk, :, t // 8, :, t // 2 % 4, :, t % 2] = b.unflatten(-1, (8, d // 32, 2))
        else:
            as_k[blk, :, t] = b
        meta[blk, :, t] = pairs


def _values(pool, d, is_v):
    """Every value of a pool: float32 [NB][Hkv][16][D]."""
    as_k, as_v, meta = _views(pool, d)
    if is_v:  # [half][dim group][pair][quad][parity][byte] -> [half][pair][parity][group][quad][byte]
        as_k = as_v.permute(0, 1, 2, 4, 6, 3, 5, 7).reshape(as_k.shape)
    codes = torch.stack([as_k & 15, as_k >> 4], -1).flatten(-2)
    return codes.float() * meta[..., :1].float() + meta[..., 1:].float()


def _rows(slots, pool, d, is_v, dtype):
    blk, t = slots.long() // BLOCK, slots.long() % BLOCK
    as_k, as_v, meta = _views(pool, d)
    b = as_v[blk, :, t // 8, :, t // 2 % 4, :, t % 2].flatten(-3) if is_v else as_k[blk, :, t]
    pairs = meta[blk, :, t].float()
    codes = torch.stack([b & 15, b >> 4], -1).flatten(-2)
    return (codes.float() * pairs[..., :1] + pairs[..., 1:]).to(dtype)


def _attend(q, k_cache, v_cache, tables, lens, scale):
    b, h, d = q.shape
    hk = k_cache.shape[1]
    idx = tables.long().clamp(min=0)
    n = idx.shape[1] * BLOCK
    live = torch.arange(n, device=q.device) < lens[:, None]                     # [B][N]
    k = _values(k_cache, d, False)[idx].transpose(1, 2).reshape(b, hk, n, d)
    k = torch.where(live[:, None, :, None], k, torch.zeros_like(k[:1, :1, :1, :1]))
    s = torch.matmul(q.float().view(b, hk, h // hk, d), k.transpose(-1, -2)) * scale
    del k
    s = torch.where(live[:, None, None], s, torch.full_like(s[:1, :1, :1, :1], -math.inf))
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    p = p / p.sum(-1, keepdim=True).clamp(min=1e-30)
    v = _values(v_cache, d, True)[idx].transpose(1, 2).reshape(b, hk, n, d)
    v = torch.where(live[:, None, :, None], v, torch.zeros_like(v[:1, :1, :1, :1]))
    return torch.matmul(p, v).view(b, h, d).to(q.dtype)


# ------------------------------------------------------------------ block tables, plainly

def _resize(lens, new_lens, tables, free, num_free, slots):
    """Gives every sequence the blocks of its new length and returns the slots
    of the tokens it gained (packed by sequence, -1 behind them) and their
    offsets.  Blocks taken come off the top of the free list in order of
    sequence and block; blocks given back go on it so that growing and
    shrinking again leaves the list as it was."""
    width = tables.shape[1]
    old, new = lens.long(), new_lens.long()
    nb_old, nb_new = (old + BLOCK - 1) // BLOCK, (new + BLOCK - 1) // BLOCK
    give, take = (nb_old - nb_new).clamp(min=0), (nb_new - nb_old).clamp(min=0)
    col = torch.arange(width, device=lens.device)
    count, gives = num_free.long(), give.sum()
    out = (col >= nb_new[:, None]) & (col < nb_old[:, None])
    rank = torch.cumsum(out.flatten(), 0).view_as(out) - 1
    here = torch.where(out, count + gives - 1 - rank, torch.full_like(rank, free.numel()))
    pool = torch.cat([free, free.new_zeros(1)])
    pool[here.flatten().clamp(max=free.numel())] = tables.flatten()
    got = (col >= nb_old[:, None]) & (col < nb_new[:, None])
    rank = torch.cumsum(got.flatten(), 0).view_as(got) - 1
    ids = pool[(count + gives - 1 - rank).clamp(min=0, max=free.numel())]
    tables.copy_(torch.where(got, ids, tables))
    free.copy_(pool[:-1])
    num_free.copy_((count + gives - take.sum()).int().view_as(num_free))
    gained = (new - old).clamp(min=0)
    offsets = torch.cat([gained.new_zeros(1), torch.cumsum(gained, 0)])
    at = torch.arange(slots.numel(), device=lens.device)
    seq = torch.searchsorted(offsets, at, right=True).sub(1).clamp(max=lens.numel() - 1)
    pos = old[seq] + at - offsets[seq]
    where = tables[seq, (pos // BLOCK).clamp(max=width - 1)] * BLOCK + pos % BLOCK
    slots.copy_(torch.where(at < offsets[-1], where, torch.full_like(where, -1)).int())
    lens.copy_(new_lens)
    return slots, offsets.int()


# ------------------------------------------------------------------ verification, plainly

SCALE_BITS, U_BITS = 40, 30


def _weights(p):
    """Probabilities as whole numbers of 2^-40."""
    p = torch.where(p > 0, p, torch.zeros_like(p)).double().clamp(max=1.0)
    return (p * 2.0 ** SCALE_BITS).round().long()


def _verify(target, draft, tokens, draft_lens, accept_u, sample_u, lens):
    b, k = tokens.shape
    seq = torch.arange(b, device=tokens.device)
    row = torch.arange(k, device=tokens.device)
    t = tokens.long()
    p = target[seq[:, None], row, t].double()
    q = draft[seq[:, None], row, t].double() if draft is not None else torch.ones_like(p)
    n = draft_lens.long() if draft_lens is not None else torch.full_like(seq, k)
    ok = (accept_u.double() * q < p) & (row < n[:, None])
    a = torch.cumprod(ok.long(), 1).sum(1)
    rejected = a < n
    at = a.clamp(max=k - 1)
    w = _weights(target[seq, a].float())
    if draft is not None:
        off = _weights(draft[seq, at].float())
    else:
        off = torch.zeros_like(w).scatter_(1, t[seq, at][:, None], 1 << SCALE_BITS)
    rest = torch.where(rejected[:, None], (w - off).clamp(min=0), w)
    w = torch.where(rest.sum(1, keepdim=True) > 0, rest, w)
    cum = torch.cumsum(w, 1)
    total = cum[:, -1]
    u = (sample_u.double().clamp(0, 1) * (1 << U_BITS)).floor().long().clamp(max=(1 << U_BITS) - 1)
    goal = ((total >> 32) * u << (32 - U_BITS)) + ((total & 0xFFFFFFFF) * u >> U_BITS)
    token = (cum <= goal[:, None]).sum(1)
    token = torch.where(total > 0, token, torch.full_like(token, -1))
    out = torch.where(torch.arange(k + 1, device=t.device) < a[:, None],
                      torch.cat([t, t[:, :1]], 1), torch.full_like(t[:, :1], -1))
    out[seq, a] = token
    return a.int(), out.int(), (lens - (k - a)).clamp(min=0).int()


# ------------------------------------------------------------------ inputs and one pass

def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _randn(gen, shape, dtype, dev, mean=None):
    x = torch.randn(shape, generator=gen, device=dev)
    return (x if mean is None else x + mean).to(dtype)


def _tables_for(lens, seed, dev, spare=1.25):
    """Scattered block tables for these lengths (-1 behind the last block)."""
    rng = np.random.default_rng(seed + 17)
    nblk = -(-lens // BLOCK)
    total = int(nblk.sum())
    num_blocks = max(1, int(math.ceil(total * spare)))
    perm = rng.permutation(num_blocks).astype(np.int32)
    width = max(1, int(nblk.max()))
    first = np.concatenate([[0], np.cumsum(nblk)])[:-1]
    col = np.arange(width)
    tables = np.where(col < nblk[:, None], perm[np.minimum(first[:, None] + col, num_blocks - 1)], -1)
    return torch.from_numpy(tables.astype(np.int32)).to(dev), num_blocks


def _prepare_cache(case, seed):
    dev = _device()
    gen = torch.Generator(device=dev).manual_seed(seed)
    lens = _lengths(case, seed)
    b, hk, d, dt = case["batch"], case["kv_heads"], case["head_dim"], DTYPES[case["dtype"]]
    h = case["q_heads"]
    tables, num_blocks = _tables_for(lens, seed, dev)
    pools = []
    for is_v in (False, True):
        # keys have a mean of their own in each channel
        mean = None if is_v else 0.5 * torch.randn((hk, 1, d), generator=gen, device=dev)
        pool = torch.empty((num_blocks, hk, BLOCK, d // 2 + 4), dtype=torch.uint8, device=dev)
        as_k, as_v, meta = _views(pool, d)
        for i in range(0, num_blocks, 4096):
            m = min(4096, num_blocks - i)
            codes, pairs = _quantise(_randn(gen, (m, hk, BLOCK, d), dt, dev, mean))
            codes = _k_bytes(codes)
            if is_v:
                as_v[i:i + m] = codes.unflatten(-1, (8, d // 32, 2)).unflatten(2, (2, 4, 2)).permute(0, 1, 2, 5, 3, 6, 4, 7)
            else:
                as_k[i:i + m] = codes
            meta[i:i + m] = pairs
        # slots that hold no token: NaN pairs
        live = torch.zeros((num_blocks, BLOCK), dtype=torch.bool, device=dev)
        n = tables.shape[1] * BLOCK
        at = torch.arange(n, device=dev)
        have = torch.from_numpy(np.maximum(lens - (case["op"] == "step"), 0)).to(dev)
        ids = tables.long().clamp(min=0).repeat_interleave(BLOCK, 1)
        mask = at < have[:, None]
        live[ids[mask], (at % BLOCK).expand(b, n)[mask]] = True
        meta.masked_fill_(~live[:, None, :, None], float("nan"))
        pools.append(pool)
    st = dict(op=case["op"], q=_randn(gen, (b, h, d), dt, dev), k_cache=pools[0], v_cache=pools[1], tables=tables,
              lens=torch.from_numpy(lens.astype(np.int32)).to(dev), scale=1.0 / math.sqrt(d),
              out=torch.empty((b, h, d), dtype=dt, device=dev), workspace=None)
    if case["op"] == "step":
        st["k_new"] = _randn(gen, (b, hk, d), dt, dev)
        st["v_new"] = _randn(gen, (b, hk, d), dt, dev)
        last = torch.from_numpy(np.maximum(lens - 1, 0)).to(dev)
        blk = tables.long().gather(1, (last // BLOCK)[:, None])[:, 0]
        st["rows"] = torch.nonzero(st["lens"] > 0)[:, 0]
        st["slots"] = (blk * BLOCK + last % BLOCK)[st["rows"]]
    if own:
        import paged_kv_cache_26_gb300 as pkv
        st["workspace"] = pkv.make_workspace_int4(st["q"], st["k_cache"], st["tables"])
    return st


def _prepare_append(case, seed):
    dev = _device()
    gen = torch.Generator(device=dev).manual_seed(seed)
    lens = _lengths(case, seed)
    hk, d, dt = case["kv_heads"], case["head_dim"], DTYPES[case["dtype"]]
    n = int(lens.sum())
    if case["hi"] == 1:  # one token of each request, anywhere in its block
        slots = np.random.default_rng(seed).permutation(2 * n)[:n] * BLOCK
        slots = slots + np.random.default_rng(seed + 1).integers(0, BLOCK, n)
        num_blocks = 2 * n
    else:
        tables, num_blocks = _tables_for(lens, seed, "cpu")
        tables = tables.numpy()
        slots = np.concatenate([tables[i, np.arange(m) // BLOCK] * BLOCK + np.arange(m) % BLOCK
                                for i, m in enumerate(lens)])
    pool = torch.zeros((2, num_blocks, hk, BLOCK, d // 2 + 4), dtype=torch.uint8, device=dev)
    mean = 0.5 * torch.randn((hk, d), generator=gen, device=dev)
    return dict(op="append", k_new=_randn(gen, (n, hk, d), dt, dev, mean), v_new=_randn(gen, (n, hk, d), dt, dev),
                slots=torch.from_numpy(slots.astype(np.int32)).to(dev), k_cache=pool[0], v_cache=pool[1],
                k_out=torch.empty((n, hk, d), dtype=dt, device=dev), v_out=torch.empty((n, hk, d), dtype=dt, device=dev))


def _prepare_tables(case, seed):
    dev = _device()
    rng = np.random.default_rng(seed)
    old, new = _grown(case, seed)
    nb_old, nb_new = -(-old // BLOCK), -(-new // BLOCK)
    held, taken = int(nb_old.sum()), int((nb_new - nb_old).sum())
    num_blocks = int(1.25 * (held + taken)) + 1
    perm = rng.permutation(num_blocks).astype(np.int32)
    tables = np.full((case["batch"], case["max_blocks"]), -1, np.int32)
    first = 0
    for b, n in enumerate(nb_old):
        tables[b, :n] = perm[first:first + n]
        first += n
    free = np.full(num_blocks, -1, np.int32)
    free[:num_blocks - held] = perm[held:]
    slots = int((new - old).sum())

    def i32(x):
        return torch.from_numpy(np.ascontiguousarray(x, dtype=np.int32)).to(dev)

    return dict(op="tables", lens=i32(old), old=i32(old), new=i32(new), tables=i32(tables), free=i32(free),
                num_free=i32([num_blocks - held]), slots=torch.empty(slots + 7, dtype=torch.int32, device=dev),
                offsets=torch.empty(case["batch"] + 1, dtype=torch.int32, device=dev))


def _prepare_verify(case, seed):
    dev = _device()
    gen = torch.Generator(device=dev).manual_seed(seed)
    b, k, v, dt = case["batch"], case["drafts"], case["vocab"], DTYPES[case["dtype"]]
    # peaked as a model's next-token distributions are (one token has about half of the mass, sometimes most of
    # it); the draft's are the target's with an error
    logits = 2.5 * torch.randn((b, k + 1, v), generator=gen, device=dev)
    first = torch.randint(0, v, (b, k + 1, 1), generator=gen, device=dev)
    top = torch.logsumexp(logits, -1, keepdim=True) + 1.5 * torch.randn((b, k + 1, 1), generator=gen, device=dev)
    logits.scatter_(-1, first, top)
    target = torch.softmax(logits, -1).to(dt)
    draft = torch.softmax(logits[:, :k] + 0.6 * torch.randn((b, k, v), generator=gen, device=dev), -1).to(dt)
    if case["certain"]:  # drafts without probabilities: the likeliest or the second likeliest token
        tokens = torch.topk(logits[:, :k], 2).indices
        pick = torch.rand((b, k), generator=gen, device=dev) < 0.5
        tokens = torch.where(pick, tokens[..., 0], tokens[..., 1]).int()
    else:
        cum = torch.cumsum(draft.double(), -1)
        u = torch.rand((b, k, 1), generator=gen, device=dev, dtype=torch.float64) * cum[..., -1:]
        tokens = (cum <= u).sum(-1).clamp(max=v - 1).int()
        del cum
    st = dict(op="verify", target=target, draft=None if case["certain"] else draft, tokens=tokens, draft_lens=None,
              accept_u=torch.rand((b, k), generator=gen, device=dev), sample_u=torch.rand(b, generator=gen, device=dev),
              lens=torch.randint(k + 1, 4096, (b,), generator=gen, device=dev, dtype=torch.int32))
    if case["ragged"]:
        st["draft_lens"] = torch.randint(0, k + 1, (b,), generator=gen, device=dev, dtype=torch.int32)
    return st


def prepare(case, seed):
    return {"step": _prepare_cache, "attention": _prepare_cache, "append": _prepare_append,
            "tables": _prepare_tables, "verify": _prepare_verify}[case["op"]](case, seed)


def run(state):
    s = state
    if own:
        import paged_kv_cache_26_gb300 as pkv
        if s["op"] == "step":
            out = pkv.paged_decode_step_int4(s["q"], s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["tables"],
                                             s["lens"], s["scale"], out=s["out"], workspace=s["workspace"])
            return {"out": out, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        if s["op"] == "attention":
            return {"out": pkv.paged_decode_attention_int4(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"],
                                                           s["scale"], out=s["out"], workspace=s["workspace"])}
        if s["op"] == "append":
            pkv.paged_kv_append_int4(s["k_new"], s["v_new"], s["slots"], s["k_cache"], s["v_cache"])
            k, v = pkv.paged_kv_read_int4(s["slots"], s["k_cache"], s["v_cache"], k_out=s["k_out"], v_out=s["v_out"])
            return {"k": k, "v": v}
        if s["op"] == "tables":
            slots, offsets = pkv.paged_kv_resize_tables(s["lens"], s["new"], s["tables"], s["free"], s["num_free"],
                                                        slot_mapping=s["slots"], token_offsets=s["offsets"])
            pkv.paged_kv_resize_tables(s["lens"], s["old"], s["tables"], s["free"], s["num_free"])
            return {"slots": slots, "offsets": offsets, "tables": s["tables"], "free": s["free"],
                    "num_free": s["num_free"], "lens": s["lens"]}
        accepted, tokens, lens = pkv.paged_verify_draft(s["target"], s["draft"], s["tokens"], s["accept_u"],
                                                        s["sample_u"], draft_lens=s["draft_lens"],
                                                        context_lens=s["lens"])
        return {"accepted": accepted, "tokens": tokens, "lens": lens}
    if s["op"] == "step":
        # the pools are fixed bit for bit by their format: they come back as the bytes that they are
        _store(s["k_new"][s["rows"]], s["v_new"][s["rows"]], s["slots"], s["k_cache"], s["v_cache"])
        out = _attend(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["scale"])
        return {"out": out, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if s["op"] == "attention":
        return {"out": _attend(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["scale"])}
    if s["op"] == "append":
        d, dt = s["k_new"].shape[-1], s["k_new"].dtype
        _store(s["k_new"], s["v_new"], s["slots"], s["k_cache"], s["v_cache"])
        return {"k": _rows(s["slots"], s["k_cache"], d, False, dt), "v": _rows(s["slots"], s["v_cache"], d, True, dt)}
    if s["op"] == "tables":
        slots, offsets = _resize(s["lens"], s["new"], s["tables"], s["free"], s["num_free"], s["slots"])
        _resize(s["lens"], s["old"], s["tables"], s["free"], s["num_free"], torch.empty_like(s["slots"][:0]))
        return {"slots": slots, "offsets": offsets, "tables": s["tables"], "free": s["free"],
                "num_free": s["num_free"], "lens": s["lens"]}
    accepted, tokens, lens = _verify(s["target"], s["draft"], s["tokens"], s["draft_lens"], s["accept_u"],
                                     s["sample_u"], s["lens"])
    return {"accepted": accepted, "tokens": tokens, "lens": lens}


# ------------------------------------------------------------------ the definitions in 64 bits

def _code_at(d, is_v, dev):
    """Byte of every (token, dim) within a tile, and its shift."""
    t = torch.arange(BLOCK, device=dev)[:, None]
    i = torch.arange(d, device=dev)[None]
    if not is_v:
        return t * (d // 2) + i // 2, (i % 2 * 4).expand(BLOCK, d)
    g = d // 8
    at = (t // 8) * (4 * d) + (i // g) * (4 * g) + (t // 2 % 4) * g + (i % g) // 4 * 4 + (t % 2) * 2 + i % 4 // 2
    return at, (i % 2 * 4).expand(BLOCK, d)


def _tile_values(tiles, d, is_v):
    """float64 [n][16][D] of tiles uint8 [n][16 (D/2 + 4)]."""
    at, shift = _code_at(d, is_v, tiles.device)
    code = (tiles[:, at.flatten()].long().view(-1, BLOCK, d) >> shift) & 15
    pairs = tiles[:, BLOCK * d // 2:].contiguous().view(torch.float16).view(-1, BLOCK, 2).double()
    return code.double() * pairs[..., :1] + pairs[..., 1:]


def _row_values(x):
    """What rows [..., D] are once they are held in 4 bits: float64."""
    x = x.float().cpu().numpy().clip(-F16_MAX, F16_MAX).astype(np.float32)
    low = x.min(-1, keepdims=True).astype(np.float16).astype(np.float32)
    scale = ((x.max(-1, keepdims=True) - low) / np.float32(15)).astype(np.float16).astype(np.float32)
    inv = np.divide(np.float32(1), scale, out=np.zeros_like(scale), where=scale > 0)
    code = np.clip(np.rint((x - low) * inv), 0, 15)
    return code.astype(np.float64) * scale.astype(np.float64) + low.astype(np.float64)


def _exact_attention(case, seed):
    st = prepare(case, seed)
    q, d, h, hk = st["q"].double(), case["head_dim"], case["q_heads"], case["kv_heads"]
    out = torch.zeros_like(q)
    lens, tables = st["lens"].tolist(), st["tables"].cpu()
    k_row = v_row = None
    if case["op"] == "step":
        k_row, v_row = (torch.from_numpy(_row_values(st[n])).to(q.device) for n in ("k_new", "v_new"))
    for b, n in enumerate(lens):
        if n == 0:
            continue
        ids = tables[b, :-(-n // BLOCK)].long().to(q.device)
        for x in range(hk):
            k, v = (_tile_values(st[c][ids, x].flatten(1), d, c == "v_cache").reshape(-1, d)[:n]
                    for c in ("k_cache", "v_cache"))
            if k_row is not None:
                k[n - 1], v[n - 1] = k_row[b, x], v_row[b, x]
            g = slice(x * (h // hk), (x + 1) * (h // hk))
            out[b, g] = torch.softmax(q[b, g] @ k.T * st["scale"], -1) @ v
    return {"out": out, "k_cache": None, "v_cache": None} if case["op"] == "step" else {"out": out}


def _exact_tables(case, seed):
    st = prepare(case, seed)
    tables, free = st["tables"].cpu().numpy().copy(), st["free"].tolist()
    stack = free[:int(st["num_free"])]
    slots, offsets = [], [0]
    for b, (old, new) in enumerate(zip(st["old"].tolist(), st["new"].tolist())):
        for pos in range(old, new):
            if pos % BLOCK == 0:
                tables[b, pos // BLOCK] = stack.pop()
            slots.append(int(tables[b, pos // BLOCK]) * BLOCK + pos % BLOCK)
        offsets.append(len(slots))
    slots += [-1] * (st["slots"].numel() - len(slots))
    return {"slots": np.asarray(slots, np.int32), "offsets": np.asarray(offsets, np.int32), "tables": tables,
            "free": np.asarray(free, np.int32), "num_free": st["num_free"].cpu().numpy(), "lens": st["old"].cpu().numpy()}


def _exact_verify(case, seed):
    st = prepare(case, seed)
    b, k = st["tokens"].shape
    accepted, tokens = np.zeros(b, np.int32), np.full((b, k + 1), -1, np.int32)
    one = 1 << SCALE_BITS

    def whole(p):
        return np.rint(np.clip(p.float().cpu().numpy().astype(np.float64), 0, 1) * one).astype(np.int64)

    for i in range(b):
        n = k if st["draft_lens"] is None else int(st["draft_lens"][i])
        a = 0
        while a < n:
            x = int(st["tokens"][i, a])
            q = 1.0 if st["draft"] is None else float(st["draft"][i, a, x])
            if not float(st["accept_u"][i, a]) * q < float(st["target"][i, a, x]):
                break
            tokens[i, a] = x
            a += 1
        accepted[i] = a
        w = whole(st["target"][i, a])
        if a < n:
            if st["draft"] is None:
                rest = w.copy()
                rest[int(st["tokens"][i, a])] = 0
            else:
                rest = np.maximum(w - whole(st["draft"][i, a]), 0)
            w = rest if rest.any() else w
        cum = np.cumsum(w)
        goal = int(cum[-1]) * min(int(float(st["sample_u"][i]) * (1 << U_BITS)), (1 << U_BITS) - 1) >> U_BITS
        tokens[i, a] = int(np.searchsorted(cum, goal, side="right")) if cum[-1] else -1
    lens = np.maximum(st["lens"].cpu().numpy() - (k - accepted), 0).astype(np.int32)
    return {"accepted": accepted, "tokens": tokens, "lens": lens}


def exact(case, seed):
    if case["op"] in ("step", "attention"):
        return _exact_attention(case, seed)
    if case["op"] == "append":
        st = _prepare_append(case, seed)
        return {"k": _row_values(st["k_new"]), "v": _row_values(st["v_new"])}
    return _exact_tables(case, seed) if case["op"] == "tables" else _exact_verify(case, seed)
