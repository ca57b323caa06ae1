"""Cases of the rotary append, chunked prefill attention and block-sparse decode.

Operators of a serving loop over a paged KV cache, each in its plain form
(elementary torch operations) and, where ``own`` is true, as the package's calls:

* rope: queries and keys turned to their positions (pairs of dims rotated by
  position times frequency; up to four position axes), the queries returned, the
  keys and values stored at their slots of the paged caches;
* chunk: causal attention of a ragged batch of new tokens, already in the cache,
  over their whole context (chunked prefill; single tokens among them);
* bounds: for the blocks that new tokens touched, the per-dim largest and
  smallest key in 8 bits with one scale for a (block, KV head);
* sparse: the blocks whose bounds promise the largest logits are chosen for each
  (sequence, KV head), and the new token attends to them alone.

Bounds of the n valid keys of a (block, KV head), in IEEE float32: scale =
max |K| * float32(1/127); upper = ceil(max K / scale), lower = floor(min K / scale),
limited to +-127 (0 where the scale is 0); with a value that is not finite
the scale is infinite, upper 127 and lower -127.  They are int8
[num_blocks][Hkv][2][D] (upper, lower) and float32 [num_blocks][Hkv].
Score of a block: with c = round_half_even(q / s), s = max |q| * float32(1/127)
(c = 0 where s is 0 or not finite), the largest over the group's heads of
(sum_d max(c upper, c lower)) * scale * s, the sum in whole numbers, then two
float32 products, a NaN as +infinity.  Chosen: the first and the last blocks that
are always kept, then by falling score, the lowest block first among equals.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 16
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # the next token of 64 chats: launch latency decides
        dict(name="rope step", op="rope", batch=64, lo=1, hi=1, base=4000, q_heads=32, kv_heads=8, head_dim=128,
             rot_dim=128, axes=1, interleaved=False, dtype="bf16"),
        # prompts of eight requests, as chunks of documents that began far before
        dict(name="rope prompts", op="rope", batch=8, lo=1031, hi=3065, base=900000, q_heads=32, kv_heads=8,
             head_dim=128, rot_dim=128, axes=1, interleaved=False, dtype="bf16"),
        # a prompt with images: time, height and width positions, seven query heads to a KV head
        dict(name="rope axes", op="rope", batch=1, lo=1237, hi=1237, base=300, q_heads=28, kv_heads=4,
             head_dim=128, rot_dim=128, axes=3, interleaved=False, dtype="fp16"),
        # three short turns of chats on a small model: latency
        dict(name="chunk tiny", op="chunk", batch=3, lo=5, hi=60, before_lo=0, before_hi=200, singles=0, q_heads=8,
             kv_heads=2, head_dim=64, dtype="fp16"),
        # four whole prompts on an 8-billion-parameter grouped-query model
        dict(name="chunk prompts", op="chunk", batch=4, lo=2500, hi=5600, before_lo=0, before_hi=0, singles=0,
             q_heads=32, kv_heads=8, head_dim=128, dtype="bf16"),
        # one chunk at the end of a long document
        dict(name="chunk long", op="chunk", batch=1, lo=2048, hi=2048, before_lo=63001, before_hi=63001, singles=0,
             q_heads=32, kv_heads=8, head_dim=128, dtype="bf16"),
        # a serving step that mixes four chunks with 36 sequences that decode one token
        dict(name="chunk mixed", op="chunk", batch=40, lo=200, hi=700, before_lo=512, before_hi=4096, singles=36,
             q_heads=64, kv_heads=8, head_dim=128, dtype="bf16"),
        # the bounds of eight prompts' blocks
        dict(name="bounds prompts", op="bounds", batch=8, lo=517, hi=4001, before_lo=0, before_hi=0, kv_heads=8,
             head_dim=128, dtype="bf16"),
        # one new token of 61 requests, an odd number of heads
        dict(name="bounds step", op="bounds", batch=61, lo=1, hi=1, before_lo=0, before_hi=2000, kv_heads=5,
             head_dim=64, dtype="fp16"),
        # one long document, eight query heads to a KV head
        dict(name="sparse one", op="sparse", batch=1, lo=131072, hi=131072, q_heads=64, kv_heads=8, head_dim=128,
             chosen=128, sink=1, recent=2, dtype="bf16"),
        # 32 documents of many lengths
        dict(name="sparse b32", op="sparse", batch=32, lo=8192, hi=32768, q_heads=32, kv_heads=8, head_dim=128,
             chosen=128, sink=1, recent=2, dtype="bf16"),
        # a few chats on a small model, some shorter than what may be chosen
        dict(name="sparse small", op="sparse", batch=5, lo=100, hi=2900, q_heads=8, kv_heads=2, head_dim=64,
             chosen=21, sink=1, recent=1, dtype="fp16"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["rope", "chunk", "chunk", "bounds", "sparse", "sparse"])
    dtype = rng.choice(["fp16", "bf16"])
    head_dim = rng.choice([64, 128])
    kv_heads = _log_int(rng, 1, 32)
    q_heads = kv_heads * rng.randint(1, 8)
    heads = dict(kv_heads=kv_heads, head_dim=head_dim, dtype=dtype)
    if op == "rope":
        batch = _log_int(rng, 1, 256)
        most = max(1, 16384 * 48 * 128 // (batch * (q_heads + 2 * kv_heads) * head_dim))
        hi = _log_int(rng, 1, min(16384, most))
        return dict(op=op, batch=batch, lo=rng.randint(1, hi), hi=hi, base=_log_int(rng, 1, 1000000),
                    q_heads=q_heads, rot_dim=rng.choice([head_dim, head_dim, head_dim // 2]),
                    axes=rng.choice([1, 1, 2, 3, 4]), interleaved=rng.random() < 0.4, **heads)
    if op == "chunk":
        batch = _log_int(rng, 1, 64)
        # as much work as the listed chunk of a long document at most, and 4 GB of cache
        cells = 2048 * 64000 * 32 * 128 // (batch * q_heads * head_dim)
        hi = _log_int(rng, 1, max(1, min(6000, int(math.sqrt(cells)))))
        room = min(cells // hi, (4 << 30) // (4 * batch * kv_heads * head_dim), 66000)
        before_hi = _log_int(rng, 1, max(1, room - hi)) if rng.random() < 0.7 else 0
        return dict(op=op, batch=batch, lo=rng.randint(1, hi), hi=hi, before_lo=rng.randint(0, before_hi),
                    before_hi=before_hi, singles=rng.randint(0, batch) if rng.random() < 0.3 else 0, q_heads=q_heads,
                    **heads)
    if op == "bounds":
        batch = _log_int(rng, 1, 128)
        hi = _log_int(rng, 1, max(1, 8 * 2259 * 8 * 128 // (batch * kv_heads * head_dim)))
        return dict(op=op, batch=batch, lo=rng.randint(1, hi), hi=hi, before_lo=0,
                    before_hi=rng.randint(0, 4000), **heads)
    batch = _log_int(rng, 1, 64)
    hi = _log_int(rng, 1, min(131072, max(1, 32 * 20480 * 8 * 128 // (batch * kv_heads * head_dim))))
    sink, recent = rng.randint(0, 3), rng.randint(1, 4)
    chosen = sink + recent + _log_int(rng, 1, 250)
    return dict(op=op, batch=batch, lo=rng.randint(1, hi), hi=hi, q_heads=q_heads, chosen=chosen, sink=sink,
                recent=recent, **heads)


def _between(lo, hi, n):
    """n lengths from lo to hi, the same for every seed."""
    return np.asarray([lo + int(round((hi - lo) * (i + 0.5) / n)) for i in range(n)], np.int64)


def _lengths(case, seed=None):
    """New tokens and context lengths (with the new tokens) of every sequence."""
    n = case["batch"]
    new = _between(case["lo"], case["hi"], n)
    new[:case.get("singles", 0)] = 1
    if case["op"] == "sparse":
        new, ctx = np.ones_like(new), new
    else:
        before = _between(case.get("before_lo", 0), case.get("before_hi", 0), n)
        ctx = new + before[::-1]
    p = np.arange(n) if seed is None else np.random.default_rng(seed).permutation(n)
    return new[p], ctx[p]


def _touched(new, ctx):
    """Blocks that hold a new token, of every sequence."""
    return (ctx + BLOCK - 1) // BLOCK - (ctx - new) // BLOCK


def work(case):
    new, ctx = _lengths(case)
    tokens, d, hk = int(new.sum()), case["head_dim"], case["kv_heads"]
    if case["op"] == "rope":
        rows = tokens * (case["q_heads"] + 2 * hk)
        return {"bytes": 2 * rows * d * 2 + tokens * (4 * case["axes"] + 4),
                "flops": 3 * tokens * (case["q_heads"] + hk) * case["rot_dim"]}
    if case["op"] == "chunk":
        seen = int((new * (2 * ctx - new + 1) // 2).sum())
        n = 2 * int(ctx.sum()) * hk * d * 2 + 2 * tokens * case["q_heads"] * d * 2
        return {"bytes": n + 4 * int(((ctx + BLOCK - 1) // BLOCK).sum()), "flops": 4 * seen * case["q_heads"] * d}
    if case["op"] == "bounds":
        blocks = int(_touched(new, ctx).sum())
        return {"bytes": blocks * (hk * (BLOCK * d * 2 + 2 * d + 4) + 4), "flops": 3 * blocks * hk * BLOCK * d}
    blocks = (ctx + BLOCK - 1) // BLOCK
    some = int(np.minimum(blocks, case["chosen"]).sum())
    b, h = case["batch"], case["q_heads"]
    n = int(blocks.sum()) * (hk * (2 * d + 4) + 4) + some * hk * (2 * BLOCK * d * 2 + 4) + 2 * b * h * d * 2
    return {"bytes": n, "flops": 2 * int(blocks.sum()) * h * d + 4 * some * BLOCK * h * d}


# ------------------------------------------------------------------ plain forms

def _rotate(x, cos, sin, rot, interleaved):
    """x [T][H][D] float32, cos / sin [T][rot/2] float32."""
    cos, sin = cos[:, None], sin[:, None]
    head, tail = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        head = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([head, tail], -1)


def _angles(positions, inv_freq, axis):
    """[T][rot/2] in float64: far positions need more than 24 bits."""
    return positions.double()[axis].T * inv_freq


def _rope(st):
    q, k, v = st["q"], st["k"], st["v"]
    angle = _angles(st["positions"], st["inv_freq"], st["axis"])
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    turned = [_rotate(x.float(), cos, sin, st["rot"], st["interleaved"]).to(x.dtype) for x in (q, k)]
    blk, t = st["slots"].long() // BLOCK, st["slots"].long() % BLOCK
    st["k_cache"][blk, :, t] = turned[1]
    st["v_cache"][blk, :, t] = v
    return turned[0]


def _chunk(st):
    q, scale = st["q"], st["scale"]
    h, d = q.shape[1:]
    hk = st["k_cache"].shape[1]
    out = torch.empty_like(q)
    at = 0
    for b, (n, ctx) in enumerate(zip(st["new_host"], st["ctx_host"])):
        ids = st["tables"][b, :-(-ctx // BLOCK)].long()
        seen = torch.arange(ctx, device=q.device) <= torch.arange(ctx - n, ctx, device=q.device)[:, None]
        for x in range(hk):
            k, v = (st[c][ids, x].flatten(0, 1)[:ctx].float() for c in ("k_cache", "v_cache"))
            g = slice(x * (h // hk), (x + 1) * (h // hk))
            s = torch.matmul(q[at:at + n, g].float().transpose(0, 1), k.T) * scale      # [g][n][ctx]
            s = s.masked_fill_(~seen, -math.inf)
            s = torch.exp(s.sub_(s.amax(-1, keepdim=True)))
            out[at:at + n, g] = (torch.matmul(s, v) / s.sum(-1, keepdim=True)).transpose(0, 1).to(q.dtype)
        at += n
    return out


def _inv127(x):
    return torch.full_like(x, np.float32(1) / np.float32(127))


def _bounds_of(k, valid):
    """k [n][Hkv][16][D], valid [n] tokens: int8 [n][Hkv][2][D] and float32 [n][Hkv]."""
    k = k.float()
    live = (torch.arange(BLOCK, device=k.device) < valid[:, None])[:, None, :, None]
    finite = (torch.isfinite(k) | ~live).flatten(2).all(-1)
    k = torch.where(finite[..., None, None], k, torch.ones_like(k))
    hi = torch.where(live, k, torch.full_like(k, -math.inf)).amax(2)
    lo = torch.where(live, k, torch.full_like(k, math.inf)).amin(2)
    top = torch.maximum(hi.abs(), lo.abs()).amax(-1)
    scale = top * _inv127(top)
    s = scale[..., None]
    zero = torch.zeros_like(hi)
    hi = torch.where(s > 0, torch.ceil(hi / s).clamp(-127, 127), zero)
    lo = torch.where(s > 0, torch.floor(lo / s).clamp(-127, 127), zero)
    hi = torch.where(finite[..., None], hi, zero + 127)
    lo = torch.where(finite[..., None], lo, zero - 127)
    scale = torch.where(finite, scale, torch.full_like(scale, math.inf))
    return torch.stack([hi, lo], 2).to(torch.int8), scale


def _bounds(st):
    seq, blk = st["touched"]
    phys = st["tables"][seq, blk].long()
    valid = (st["lens"][seq] - blk * BLOCK).clamp(max=BLOCK)
    st["bounds"][phys], st["scales"][phys] = _bounds_of(st["k_cache"][phys], valid)
    return st["bounds"], st["scales"]


def _select(q, bounds, scales, tables, lens, chosen, sink, recent):
    b, h, d = q.shape
    hk, width = bounds.shape[1], tables.shape[1]
    x = q.float()
    top = x.abs().amax(-1, keepdim=True)
    s = top * _inv127(top)
    c = torch.where((s > 0) & torch.isfinite(s), torch.round(x / s), torch.zeros_like(x)).view(b, hk, -1, d)
    idx = tables.long().clamp(min=0)
    e = bounds[idx].float().permute(0, 2, 3, 4, 1)                                  # [B][Hkv][2][D][N]
    dot = torch.matmul(c.clamp(min=0), e[:, :, 0]) + torch.matmul(c.clamp(max=0), e[:, :, 1])
    score = dot * scales[idx].permute(0, 2, 1)[:, :, None] * s.view(b, hk, -1, 1)
    score = torch.where(torch.isnan(score), torch.full_like(score, math.inf), score).amax(2)
    nb = ((lens.long() + BLOCK - 1) // BLOCK)[:, None, None]
    col = torch.arange(width, device=q.device)
    kept = ((col < sink) | (col >= nb - recent)) & (col < nb)
    # by falling rank of (kept, score), the lowest block first: two stable sorts
    order = torch.argsort(score, dim=-1, descending=True, stable=True)
    rank = torch.where(kept, 0, 1) + torch.where(col < nb, 0, 2)
    order = order.gather(-1, torch.argsort(rank.expand_as(score).gather(-1, order), dim=-1, stable=True))
    n = min(chosen, width)
    first = order[..., :n]
    first = torch.where(torch.arange(n, device=q.device) < nb, first, torch.full_like(first, width)).sort(-1).values
    out = torch.full((b, hk, chosen), -1, dtype=torch.int32, device=q.device)
    out[..., :n] = torch.where(first < width, first, torch.full_like(first, -1)).int()
    return out


def _attend_chosen(q, k_cache, v_cache, tables, lens, chosen, scale):
    b, h, d = q.shape
    hk, n = k_cache.shape[1], chosen.shape[2]
    j = chosen.long().clamp(min=0)
    phys = tables.long()[torch.arange(b, device=q.device)[:, None, None], j].clamp(min=0)
    head = torch.arange(hk, device=q.device)[None, :, None]
    pos = j[..., None] * BLOCK + torch.arange(BLOCK, device=q.device)
    live = ((pos < lens[:, None, None, None]) & (chosen >= 0)[..., None]).flatten(2)  # [B][Hkv][n * 16]
    k, v = (torch.where(live[..., None], c[phys, head].flatten(2, 3).float(), torch.zeros((), device=q.device))
            for c in (k_cache, v_cache))
    s = torch.matmul(q.float().view(b, hk, -1, d), k.transpose(-1, -2)) * scale
    s = torch.where(live[:, :, None], s, torch.full_like(s, -math.inf))
    p = torch.exp(s - s.amax(-1, keepdim=True))
    return (torch.matmul(p, v) / p.sum(-1, keepdim=True)).view(b, h, d).to(q.dtype)


# ------------------------------------------------------------------ inputs and one pass

def _device():
    return torch.device("cuda" if torch.cuda.is_available() else "cpu")


def _paged(case, seed, ctx):
    """Tables over a scattered pool, on the device, and the pool's size in blocks."""
    blocks = -(-ctx // BLOCK)
    total, width = int(blocks.sum()), max(1, int(blocks.max()))
    num_blocks = total + total // 8 + 1
    perm = np.random.default_rng(seed + 7).permutation(num_blocks)[:total].astype(np.int32)
    tables = np.full((len(ctx), width), -1, np.int32)
    at = 0
    for b, n in enumerate(blocks):
        tables[b, :n] = perm[at:at + n]
        at += n
    return tables, num_blocks


def _keys(shape, gen, dtype, dev):
    """Keys as a projection gives them: dims with means and spreads of their own,
    neighbouring tokens (a block's) alike."""
    nb, hk, n, d = shape
    spread = torch.exp(0.5 * torch.randn(hk, 1, d, generator=gen, device=dev))
    mean = torch.randn(hk, 1, d, generator=gen, device=dev)
    out = torch.empty(shape, dtype=dtype, device=dev)
    for at in range(0, nb, 8192):                                   # in pieces: float32 of a large pool is large
        m = min(8192, nb - at)
        topic = torch.randn(m, hk, 1, d, generator=gen, device=dev)
        x = torch.randn(m, hk, n, d, generator=gen, device=dev)
        out[at:at + m] = ((0.7 * x + 0.7 * topic) * spread + mean).to(dtype)
    return out


def _values(shape, gen, dtype, dev):
    out = torch.empty(shape, dtype=dtype, device=dev)
    for at in range(0, shape[0], 8192):
        out[at:at + 8192] = torch.randn(out[at:at + 8192].shape, generator=gen, device=dev).to(dtype)
    return out


def _axis_of(case):
    """Position axis of every frequency: the axes in sections, the later ones larger."""
    half, n = case["rot_dim"] // 2, case["axes"]
    if n == 1:
        return [0] * half
    first = half // (n + 1)
    rest = half - first
    return [0] * first + [1 + i * (n - 1) // rest for i in range(rest)]


def _positions(case, seed, new, ctx):
    """[axes][tokens]: text advances every axis; with several axes a third of each
    prompt is an image whose tokens share the first axis and lie on a grid."""
    rng = np.random.default_rng(seed + 3)
    rows = []
    for n, base in zip(new, rng.integers(0, case["base"] + 1, len(new))):
        p = np.tile(base + np.arange(n), (case["axes"], 1))
        side = int(math.isqrt(n // 3))
        if case["axes"] > 1 and side > 1:
            at, m = n // 3, side * side
            grid = np.arange(m)
            p[:, at:at + m] = base + at
            p[-1, at:at + m] += grid % side
            p[-2, at:at + m] += grid // side
            p[:, at + m:] = base + at + side + np.arange(n - at - m)
        rows.append(p)
    return np.concatenate(rows, 1).astype(np.int32)


def _prepare_rope(case, seed):
    dev, dt = _device(), DTYPES[case["dtype"]]
    gen = torch.Generator(device=dev).manual_seed(seed)
    new, ctx = _lengths(case, seed)
    tables, num_blocks = _paged(case, seed, ctx)
    h, hk, d, tokens = case["q_heads"], case["kv_heads"], case["head_dim"], int(new.sum())
    # one fused projection's output: queries, keys and values of a token side by side
    qkv = torch.randn(tokens, (h + 2 * hk) * d, generator=gen, device=dev).to(dt)
    q, k, v = (x.view(tokens, -1, d) for x in qkv.split([h * d, hk * d, hk * d], -1))
    slots = np.concatenate([tables[b, p // BLOCK] * BLOCK + p % BLOCK
                            for b, p in enumerate(np.arange(c - n, c) for n, c in zip(new, ctx))]).astype(np.int32)
    pool = [torch.randn(num_blocks, hk, BLOCK, d, generator=gen, device=dev).to(dt) for _ in range(2)]
    inv = [500000.0 ** (-2.0 * i / case["rot_dim"]) for i in range(case["rot_dim"] // 2)]
    axis = _axis_of(case)
    st = dict(case=case, q=q, k=k, v=v, k_cache=pool[0], v_cache=pool[1], slots=torch.from_numpy(slots).to(dev),
              positions=torch.from_numpy(_positions(case, seed, new, ctx)).to(dev), rot=case["rot_dim"],
              interleaved=case["interleaved"], inv_freq=torch.tensor(inv, dtype=torch.float64, device=dev),
              axis=torch.tensor(axis, device=dev), q_out=torch.empty(tokens, h, d, dtype=dt, device=dev))
    if own:
        import paged_kv_cache_26_gb300 as pkv
        st["rope"] = pkv.make_rope(inv, d, axes=axis, interleaved=case["interleaved"])
    return st


def prepare(case, seed):
    if case["op"] == "rope":
        return _prepare_rope(case, seed)
    dev, dt = _device(), DTYPES[case["dtype"]]
    gen = torch.Generator(device=dev).manual_seed(seed)
    new, ctx = _lengths(case, seed)
    tables, num_blocks = _paged(case, seed, ctx)
    hk, d = case["kv_heads"], case["head_dim"]
    shape = (num_blocks, hk, BLOCK, d)
    st = dict(case=case, tables=torch.from_numpy(tables).to(dev), lens=torch.from_numpy(ctx.astype(np.int32)).to(dev),
              k_cache=_keys(shape, gen, dt, dev), scale=d ** -0.5)
    if case["op"] != "sparse":
        st["offsets"] = torch.from_numpy(np.concatenate([[0], np.cumsum(new)]).astype(np.int32)).to(dev)
    if case["op"] == "bounds":
        st["tokens"] = int(new.sum())
        many = _touched(new, ctx)
        seq = np.repeat(np.arange(len(new)), many)
        first = np.repeat((ctx - new) // BLOCK - np.concatenate([[0], np.cumsum(many)[:-1]]), many)
        st["touched"] = tuple(torch.from_numpy(x).to(dev) for x in (seq, first + np.arange(len(seq))))
        st["bounds"] = torch.zeros(num_blocks, hk, 2, d, dtype=torch.int8, device=dev)
        st["scales"] = torch.zeros(num_blocks, hk, device=dev)
        return st
    h = case["q_heads"]
    st["v_cache"] = _values(shape, gen, dt, dev)
    st["q"] = torch.randn(int(new.sum()), h, d, generator=gen, device=dev).to(dt)
    if case["op"] == "chunk":
        st.update(new_host=new.tolist(), ctx_host=ctx.tolist(), out=torch.empty_like(st["q"]))
        if own:
            import paged_kv_cache_26_gb300 as pkv
            st["workspace"] = pkv.make_workspace_chunk(st["q"], st["k_cache"], st["tables"])
        return st
    # the bounds that the loop has kept, of whole blocks but the last
    valid = torch.full((num_blocks,), BLOCK, device=dev)
    last = torch.from_numpy(tables[np.arange(len(ctx)), (ctx - 1) // BLOCK].astype(np.int64)).to(dev)
    valid[last] = torch.from_numpy((ctx - 1) % BLOCK + 1).to(dev)
    parts = [_bounds_of(st["k_cache"][i:i + 4096], valid[i:i + 4096]) for i in range(0, num_blocks, 4096)]
    st["bounds"], st["scales"] = (torch.cat(x) for x in zip(*parts))
    return st


def run(state):
    st, op = state, state["case"]["op"]
    if own:
        import paged_kv_cache_26_gb300 as pkv
    if op == "rope":
        if own:
            q = pkv.paged_kv_append_rope(st["q"], st["k"], st["v"], st["positions"], st["rope"], st["slots"],
                                         st["k_cache"], st["v_cache"], q_out=st["q_out"])
        else:
            q = _rope(st)
        return {"q": q, "k_cache": st["k_cache"], "v_cache": st["v_cache"]}
    if op == "chunk":
        if own:
            return {"out": pkv.paged_chunk_attention(st["q"], st["k_cache"], st["v_cache"], st["tables"], st["lens"],
                                                     st["offsets"], st["scale"], out=st["out"],
                                                     workspace=st["workspace"])}
        return {"out": _chunk(st)}
    if op == "bounds":
        if own:
            pkv.paged_kv_update_bounds(st["k_cache"], st["tables"], st["lens"], st["bounds"], st["scales"],
                                       q_offsets=st["offsets"], num_tokens=st["tokens"])
            return {"bounds": st["bounds"], "scales": st["scales"]}
        bounds, scales = _bounds(st)
        return {"bounds": bounds, "scales": scales}
    c = st["case"]
    if own:
        chosen = pkv.paged_select_blocks(st["q"], st["bounds"], st["scales"], st["tables"], st["lens"], c["chosen"],
                                         sink_blocks=c["sink"], recent_blocks=c["recent"])
        out = pkv.paged_decode_attention_sparse(st["q"], st["k_cache"], st["v_cache"], st["tables"], st["lens"], chosen,
                                                st["scale"])
    else:
        chosen = _select(st["q"], st["bounds"], st["scales"], st["tables"], st["lens"], c["chosen"], c["sink"],
                         c["recent"])
        out = _attend_chosen(st["q"], st["k_cache"], st["v_cache"], st["tables"], st["lens"], chosen, st["scale"])
    return {"chosen": chosen, "out": out}


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_rope(case, seed):
    st = prepare(case, seed)
    rot, half = case["rot_dim"], case["rot_dim"] // 2
    inv, axis = st["inv_freq"].cpu().numpy(), st["axis"].cpu().numpy()
    angle = st["positions"].cpu().numpy()[axis].T.astype(np.float64) * inv
    turn = torch.from_numpy(np.exp(1j * angle)).to(st["q"].device)[:, None]

    def turned(x):
        y = x.double().clone()
        first, second = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(half), slice(half, rot))
        z = torch.complex(y[..., first], y[..., second]) * turn
        y[..., first], y[..., second] = z.real, z.imag
        return y

    k_cache, v_cache = st["k_cache"].double(), st["v_cache"].double()
    rows = st["slots"].long()
    for pool, x in ((k_cache, turned(st["k"])), (v_cache, st["v"].double())):
        flat = pool.transpose(1, 2).reshape(-1, *x.shape[1:])
        flat[rows] = x
        pool.copy_(flat.view(pool.shape[0], BLOCK, *x.shape[1:]).transpose(1, 2))
    return {"q": turned(st["q"]), "k_cache": k_cache, "v_cache": v_cache}


def _exact_chunk(case, seed):
    st = prepare(case, seed)
    q, (h, d), hk = st["q"].double(), st["q"].shape[1:], case["kv_heads"]
    out = torch.empty_like(q)
    offsets = st["offsets"].tolist()
    for b, ctx in enumerate(st["lens"].tolist()):
        at, n = offsets[b], offsets[b + 1] - offsets[b]
        slots = torch.arange(ctx, device=q.device)
        ids = st["tables"][b].long()[slots // BLOCK]
        for x in range(h):
            k, v = (st[c][ids, x // (h // hk), slots % BLOCK].double() for c in ("k_cache", "v_cache"))
            for i in range(0, n, 1024):
                m = min(1024, n - i)
                top = ctx - n + i + m                                  # keys that this part sees at all
                s = (q[at + i:at + i + m, x] * st["scale"]) @ k[:top].T
                s += torch.full_like(s, -math.inf).triu_(top - m + 1)
                out[at + i:at + i + m, x] = torch.softmax(s, -1) @ v[:top]
    return {"out": out}


def _exact_bounds_block(k):
    """One (block, KV head) of finite keys [n][D] (numpy float32)."""
    hi, lo = k.max(0), k.min(0)
    scale = np.float32(np.abs(k).max()) * (np.float32(1) / np.float32(127))
    if scale == 0:
        return np.zeros((2, k.shape[1]), np.int8), scale
    both = np.stack([np.ceil(hi / scale), np.floor(lo / scale)])
    return np.clip(both, -127, 127).astype(np.int8), scale


def _exact_bounds(case, seed):
    st = prepare(case, seed)
    bounds, scales = st["bounds"].cpu().numpy(), st["scales"].cpu().numpy()
    keys, tables, offsets = st["k_cache"].float().cpu().numpy(), st["tables"].cpu().numpy(), st["offsets"].tolist()
    for b, ctx in enumerate(st["lens"].tolist()):
        start = ctx - (offsets[b + 1] - offsets[b])
        for j in range(start // BLOCK, -(-ctx // BLOCK)):
            phys = tables[b, j]
            for x in range(case["kv_heads"]):
                bounds[phys, x], scales[phys, x] = _exact_bounds_block(keys[phys, x, :min(BLOCK, ctx - j * BLOCK)])
    return {"bounds": bounds, "scales": scales}


def _exact_sparse(case, seed):
    st = prepare(case, seed)
    q, d, h, hk = st["q"], case["head_dim"], case["q_heads"], case["kv_heads"]
    g, n = h // hk, case["chosen"]
    tables, one = st["tables"].cpu().numpy(), np.float32(1) / np.float32(127)
    chosen = np.full((case["batch"], hk, n), -1, np.int32)
    out = torch.zeros_like(q, dtype=torch.float64)
    x32 = q.float().cpu().numpy()
    for b, ctx in enumerate(st["lens"].tolist()):
        nb = -(-ctx // BLOCK)
        ids = torch.from_numpy(tables[b, :nb].astype(np.int64)).to(q.device)
        edge, step = st["bounds"][ids].cpu().numpy().astype(np.float64), st["scales"][ids].cpu().numpy()
        for x in range(hk):
            score = np.full(nb, -np.inf, np.float32)
            for y in range(x * g, (x + 1) * g):
                s = np.abs(x32[b, y]).max() * one
                c = np.rint(x32[b, y] / s).astype(np.float64) if s > 0 else np.zeros(d)
                dot = edge[:, x, 0] @ np.maximum(c, 0) + edge[:, x, 1] @ np.minimum(c, 0)
                score = np.maximum(score, dot.astype(np.float32) * step[:, x] * s)
            keep = set(range(min(case["sink"], nb))) | set(range(max(0, nb - case["recent"]), nb))
            rest = sorted((j for j in range(nb) if j not in keep), key=lambda j: (-score[j], j))
            some = sorted((sorted(keep) + rest)[:n])
            chosen[b, x, :len(some)] = some
            pos = np.concatenate([np.arange(j * BLOCK, min((j + 1) * BLOCK, ctx)) for j in some])
            at = torch.from_numpy(tables[b, pos // BLOCK].astype(np.int64)).to(q.device)
            t = torch.from_numpy(pos % BLOCK).to(q.device)
            k, v = (st[p][at, x, t].double() for p in ("k_cache", "v_cache"))
            heads = slice(x * g, (x + 1) * g)
            out[b, heads] = torch.softmax(q[b, heads].double() @ k.T * st["scale"], -1) @ v
    return {"chosen": chosen, "out": out}


def exact(case, seed):
    return {"rope": _exact_rope, "chunk": _exact_chunk, "bounds": _exact_bounds, "sparse": _exact_sparse}[case["op"]](
        case, seed)
