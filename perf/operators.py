"""Cases and plain forms of the operators on the paged 8-bit K/V cache.

The cache: K and V pools of e4m3 values [num_blocks, kv_heads, block, head_dim]
with one fp32 scale per block and head, reached through a block table per
request. Four operators work on it: `append` writes a step's new tokens,
`attention` reads it, `weigh` adds up the attention weight each cached token
received, and `evict` keeps the tokens with the most weight in fewer pages.

Rows of a call are ragged: request i owns rows row_begin[i] .. row_begin[i + 1]
and its row j sits at slot context_lens[i] - n_i + j.
"""

import itertools
import math

import torch

own = False

F8 = torch.float8_e4m3fn
F8_MAX = 448.0


# ------------------------------------------------------------------ the cases

def listed():
    base = dict(head_dim=128, long=0)
    return [
        # one decode step of 64 requests: a token each into pages that already hold some
        dict(base, name="append_step", op="append", bs=64, rows_lo=1, rows_hi=1, ctx_lo=1,
             ctx_hi=1024, heads=32, kv_heads=8, block=64),
        # a scheduler step that mixes prompt chunks: thousands of new tokens, ragged, behind earlier ones
        dict(base, name="append_chunks", op="append", bs=6, rows_lo=700, rows_hi=4096, ctx_lo=1000,
             ctx_hi=8192, heads=32, kv_heads=8, block=64),
        # one chat at its start: the smallest call, where latency counts
        dict(base, name="decode_single", op="attention", bs=1, rows_lo=1, rows_hi=1, ctx_lo=500,
             ctx_hi=500, heads=32, kv_heads=8, block=16),
        # batch decode with contexts of a few thousand to 32 k tokens
        dict(base, name="decode_batch", op="attention", bs=64, rows_lo=1, rows_hi=1, ctx_lo=4096,
             ctx_hi=32768, heads=64, kv_heads=8, block=64),
        # speculative verify, four draft rows, long contexts, few K/V heads
        dict(base, name="decode_verify", op="attention", bs=32, rows_lo=4, rows_hi=4, ctx_lo=16384,
             ctx_hi=65536, heads=16, kv_heads=2, block=64),
        # chunked prefill: prompt chunks of up to 2 k tokens behind up to 8 k cached ones
        dict(base, name="prompt_chunks", op="attention", bs=4, rows_lo=1100, rows_hi=2048,
             ctx_lo=2048, ctx_hi=8192, heads=32, kv_heads=8, block=64),
        # a mixed step: two prompts among decoding requests, narrow heads, pages of 48 tokens
        dict(base, name="mixed_step", op="attention", bs=18, rows_lo=1, rows_hi=900, long=2,
             ctx_lo=1, ctx_hi=4096, heads=24, kv_heads=8, block=48, head_dim=64),
        # the weights of a decode step, batch of 32
        dict(base, name="weigh_step", op="weigh", bs=32, rows_lo=1, rows_hi=1, ctx_lo=4096,
             ctx_hi=16384, heads=32, kv_heads=8, block=64),
        # the weights of the last 64 rows of long prompts (an observation window before evicting)
        dict(base, name="weigh_window", op="weigh", bs=4, rows_lo=64, rows_hi=64, ctx_lo=16384,
             ctx_hi=32768, heads=32, kv_heads=8, block=64),
        # one short chat cut to 512 tokens
        dict(base, name="evict_single", op="evict", bs=1, rows_lo=1, rows_hi=1, ctx_lo=1500,
             ctx_hi=1500, heads=32, kv_heads=8, block=16, keep=512, sinks=4, recent=64),
        # a batch of long requests cut to 4 k tokens each
        dict(base, name="evict_batch", op="evict", bs=16, rows_lo=1, rows_hi=1, ctx_lo=2000,
             ctx_hi=65536, heads=32, kv_heads=8, block=64, keep=4096, sinks=16, recent=512),
    ]


def draw(rng):
    def logint(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["append", "append", "attention", "attention", "attention", "attention",
                     "weigh", "weigh", "evict", "evict"])
    kv_heads = rng.choice([1, 2, 3, 4, 5, 8])
    c = dict(op=op, kv_heads=kv_heads,
             heads=kv_heads * rng.choice([g for g in (1, 2, 3, 4, 5, 8) if kv_heads * g <= 32]),
             head_dim=rng.choice([64, 128, 128]), block=rng.choice([1, 8, 16, 24, 32, 48, 64, 128]),
             long=0)
    if op == "append":
        if rng.random() < 0.5:
            c.update(bs=logint(1, 128), rows_lo=1, rows_hi=rng.choice([1, 2, 4]), ctx_lo=1,
                     ctx_hi=logint(8, 1024))
        else:
            hi = logint(8, 4096)
            c.update(bs=logint(1, 6), rows_lo=max(1, hi // 5), rows_hi=hi, ctx_lo=1,
                     ctx_hi=logint(hi, 2 * hi))
    elif op == "attention":
        kind = rng.choice(["decode", "decode", "prompt", "mixed"])
        if kind == "decode":
            n = rng.choice([1, 1, 2, 3, 4])
            hi = logint(64, 65536)
            c.update(bs=logint(1, max(1, min(64, 900000 // hi))), rows_lo=n, rows_hi=n,
                     ctx_lo=max(1, hi // 8), ctx_hi=hi)
        elif kind == "prompt":
            hi = logint(33, 1700)
            c.update(bs=logint(1, 4), rows_lo=max(1, hi // 2), rows_hi=hi, ctx_lo=1,
                     ctx_hi=logint(hi, 4 * hi))
        else:
            c.update(bs=logint(4, 24), rows_lo=1, rows_hi=logint(40, 900), long=2, ctx_lo=1,
                     ctx_hi=logint(100, 4096))
    elif op == "weigh":
        if rng.random() < 0.5:
            hi = logint(64, 16384)
            c.update(bs=logint(1, 32), rows_lo=1, rows_hi=rng.choice([1, 2, 4]),
                     ctx_lo=max(1, hi // 4), ctx_hi=hi)
        else:
            hi = logint(300, 32768)
            c.update(bs=logint(1, 4), rows_lo=8, rows_hi=logint(16, 64), ctx_lo=max(1, hi // 2),
                     ctx_hi=hi)
    else:
        hi = logint(100, 65536)
        keep = logint(24, 4096)
        c.update(bs=logint(1, 16), rows_lo=1, rows_hi=1, ctx_lo=max(1, hi // 16), ctx_hi=hi,
                 keep=keep, sinks=rng.randint(0, keep // 8), recent=rng.randint(0, keep // 4))
    return c


def _spread(lo, hi, n, turn):
    """n whole numbers over [lo, hi], the same for every call (golden-ratio steps)."""
    return [lo + int((hi - lo + 1) * ((0.5 + (i + turn) * 0.6180339887498949) % 1.0))
            for i in range(n)]


def _lens(case):
    """New rows and context length (with the new rows) of every request."""
    bs = case["bs"]
    rows = _spread(case["rows_lo"], case["rows_hi"], bs, 3)
    if case["long"]:
        rows = [case["rows_hi"] - 37 * i if i < case["long"] else case["rows_lo"]
                for i in range(bs)]
        rows = [max(1, r) for r in rows]
    ctx = _spread(case["ctx_lo"], case["ctx_hi"], bs, 0)
    return rows, [max(c, r) for c, r in zip(ctx, rows)]


# ------------------------------------------------------------------ inputs

def _pow2_scale(amax):
    """The power of two s with amax / s in (224, 448]: 2^ceil(log2(amax / 448))."""
    m, e = torch.frexp(amax)  # amax = m 2^e with m in [0.5, 1), and 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(amax > 0, e, torch.full_like(e, -100))
    return torch.ldexp(torch.ones_like(amax), e.clamp(min=-100))


def _fill_pool(gen, blocks, kv_heads, block, head_dim, device, spread):
    """A pool as `append` leaves it: normal values whose size differs by channel
    and block, quantised with each (block, head)'s own power-of-two scale."""
    x = torch.randn((blocks, kv_heads, block, head_dim), generator=gen, device=device)
    x *= torch.exp2(torch.randn((1, kv_heads, 1, head_dim), generator=gen, device=device) * spread)
    x *= torch.exp2(torch.randn((blocks, kv_heads, 1, 1), generator=gen, device=device) * 0.3)
    s = _pow2_scale(x.abs().amax((2, 3)).clamp(min=1e-20))
    x /= s[:, :, None, None]
    return x.to(F8), s.contiguous()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    rows, ctx = _lens(case)
    bs, P, H, Hq, D = case["bs"], case["block"], case["kv_heads"], case["heads"], case["head_dim"]
    pages = [-(-c // P) for c in ctx]
    W = max(pages) + 1
    keep_pages = -(-case["keep"] // P) if case["op"] == "evict" else 0
    blocks = sum(pages) + bs * keep_pages + 3
    perm = torch.randperm(blocks, generator=gen, device=dev).to(torch.int32)
    tables = torch.full((bs, W), -1, dtype=torch.int32, device=dev)
    at = 0
    for i, n in enumerate(pages):
        tables[i, :n] = perm[at:at + n]
        at += n
    st = dict(op=case["op"], tables=tables,
              ctx=torch.tensor(ctx, dtype=torch.int32, device=dev), max_rows=max(rows),
              row_begin=torch.tensor([0] + list(itertools.accumulate(rows)), dtype=torch.int32, device=dev))
    st["kc"], st["ks"] = _fill_pool(gen, blocks, H, P, D, dev, 0.5)
    st["vc"], st["vs"] = _fill_pool(gen, blocks, H, P, D, dev, 0.3)
    total = sum(rows)
    if case["op"] == "append":
        st["k"] = torch.randn((total, H, D), generator=gen, device=dev).to(torch.bfloat16)
        st["v"] = torch.randn((total, H, D), generator=gen, device=dev).to(torch.bfloat16)
    if case["op"] in ("attention", "weigh"):
        # a few channels carry most of the score, as in trained models
        q = torch.randn((total, Hq, D), generator=gen, device=dev)
        q *= torch.exp2(torch.randn((1, Hq, D), generator=gen, device=dev) * 0.5)
        st["q"] = q.to(torch.bfloat16)
        st["sm_scale"] = D ** -0.5
    if case["op"] == "weigh":
        st["mass_in"] = torch.rand((bs, H, W * P), generator=gen, device=dev)
        st["mass"] = st["mass_in"].clone()
        st["lse"] = _plain_attention(st, values=False)
    if case["op"] == "evict":
        # accumulated weight is heavy-tailed, and zero for tokens never looked at
        m = torch.exp2(torch.randn((bs, H, W * P), generator=gen, device=dev) * 3.0)
        st["mass"] = torch.where(torch.rand(m.shape, generator=gen, device=dev) < 0.3,
                                 torch.zeros_like(m), m)
        st["keep"], st["sinks"], st["recent"] = case["keep"], case["sinks"], case["recent"]
        st["new_tables"] = perm[at:at + bs * keep_pages].reshape(bs, keep_pages).contiguous()
    # the scratch memory that a program keeps beside its cache
    st["ws"] = torch.zeros(32 << 20, dtype=torch.uint8, device=dev)
    return st


# ------------------------------------------------------------------ plain forms

def _paged(pool, scale, tables):
    """The tokens behind the tables, dequantised: fp32 [bs, kv_heads, W * block, head_dim]."""
    t = tables.long().clamp(min=0)
    x = pool[t].float() * scale[t][..., None, None]
    bs, W, H, P, D = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(bs, H, W * P, D)


def _padded(st, x):
    """Rows [rows, ...] -> [bs, max_rows, ...] (padding repeats row 0), and which are rows."""
    n = st["row_begin"][1:] - st["row_begin"][:-1]
    j = torch.arange(st["max_rows"], device=x.device)
    real = j[None, :] < n[:, None]
    at = torch.where(real, st["row_begin"][:-1, None] + j[None, :], 0).long()
    return x[at], real, n, j


def _scores(st):
    """Scores [bs, kv_heads, max_rows, group, slots] with -inf outside the mask, and the rows that are rows."""
    q, real, n, j = _padded(st, st["q"])
    k = _paged(st["kc"], st["ks"], st["tables"])
    bs, R, Hq, D = q.shape
    H = k.shape[1]
    q = q.float().reshape(bs, R, H, Hq // H, D).permute(0, 2, 1, 3, 4).reshape(bs, H, -1, D)
    s = torch.matmul(q, k.transpose(2, 3)).mul_(st["sm_scale"]).reshape(bs, H, R, Hq // H, -1)
    t = torch.arange(k.shape[2], device=q.device)
    last = st["ctx"][:, None] - n[:, None] + j[None, :]
    seen = (t[None, None, :] <= last[:, :, None]) & real[:, :, None]
    return s.masked_fill_(~seen[:, None, :, None, :], -math.inf), real


def _plain_attention(st, values=True):
    s, real = _scores(st)
    bs, H, R, G, _ = s.shape
    top = s.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    s = s.sub_(top).exp_()
    total = s.sum(-1, keepdim=True)
    lse = (top + total.log()).squeeze(-1).permute(0, 2, 1, 3).reshape(bs, R, H * G)[real]
    if not values:
        return lse
    v = _paged(st["vc"], st["vs"], st["tables"])
    o = torch.matmul(s.reshape(bs, H, R * G, -1), v).reshape(bs, H, R, G, -1)
    o = o / torch.where(total > 0, total, torch.ones_like(total))
    o = o.permute(0, 2, 1, 3, 4).reshape(bs, R, H * G, -1)[real]
    return o.to(torch.bfloat16), lse


def _plain_weigh(st):
    s, real = _scores(st)
    bs, H, R, G, _ = s.shape
    lse, _, _, _ = _padded(st, st["lse"])
    lse = lse.reshape(bs, R, H, G).permute(0, 2, 1, 3)
    w = s.sub_(lse[..., None]).exp_().sum((2, 3))
    t = torch.arange(w.shape[-1], device=w.device)
    held = t[None, None, :] < st["ctx"][:, None, None]
    return torch.where(held, st["mass_in"] + w, st["mass"])


def _plain_append_one(st, x, pool, scale):
    P = pool.shape[2]
    rb, ctx, tables = st["row_begin"].long(), st["ctx"].long(), st["tables"].long()
    n = rb[1:] - rb[:-1]
    r = torch.arange(x.shape[0], device=x.device)
    req = torch.searchsorted(rb[1:].contiguous(), r, right=True)
    slot = ctx[req] - n[req] + r - rb[req]
    page, off = tables[req, slot // P], slot % P
    x = x.float()
    # new scales: the largest new value of each page and head, against the earlier tokens' scale
    amax = torch.zeros_like(scale).index_reduce_(0, page, x.abs().amax(2), "amax")
    hit = torch.zeros(scale.shape[0], dtype=torch.bool, device=x.device).index_fill_(0, page, True)
    fresh = _pow2_scale(amax)
    first = ctx - n  # the first new slot: its page holds earlier tokens where it is not the page's first
    old_page = tables.gather(1, (first // P)[:, None]).squeeze(1)
    mixed = torch.zeros_like(hit).index_fill_(0, old_page[(first % P > 0) & (n > 0)], True)
    new = torch.where(mixed[:, None], torch.maximum(scale, fresh), fresh)
    new = torch.where(hit[:, None], new, scale)
    # earlier tokens of a page whose scale grew
    before = pool[old_page].float() * scale[old_page][..., None, None]
    again = (before / new[old_page][..., None, None]).clamp(-F8_MAX, F8_MAX).to(F8)
    o = torch.arange(P, device=x.device)
    moved = (o[None, :] < (first % P)[:, None])[:, None, :] & (new != scale)[old_page][:, :, None]
    bytes_ = torch.where(moved[..., None], again.view(torch.uint8), pool[old_page].view(torch.uint8))
    touched = n > 0
    pool.view(torch.uint8)[old_page[touched]] = bytes_[touched]
    code = (x / new[page][..., None]).clamp(-F8_MAX, F8_MAX).to(F8)
    pool.view(torch.uint8)[page, :, off] = code.view(torch.uint8)
    scale.copy_(new)


def _plain_append(st):
    _plain_append_one(st, st["k"], st["kc"], st["ks"])
    _plain_append_one(st, st["v"], st["vc"], st["vs"])
    return st["kc"], st["vc"], st["ks"], st["vs"]


def _plain_evict_one(st, pool, scale, kept, new_len):
    bs, H, keep = kept.shape
    P, D = pool.shape[2], pool.shape[3]
    W = st["new_tables"].shape[1]
    there = kept >= 0
    slot = kept.clamp(min=0)
    page = st["tables"].long()[torch.arange(bs, device=pool.device)[:, None, None], slot // P]
    h = torch.arange(H, device=pool.device)[None, :, None]
    x = pool[page, h, slot % P].float() * scale[page, h][..., None]
    x = torch.where(there[..., None], x, torch.zeros_like(x))
    x = torch.nn.functional.pad(x, (0, 0, 0, W * P - keep)).reshape(bs, H, W, P, D)
    s = _pow2_scale(x.abs().amax((3, 4)))
    code = (x / s[..., None, None]).clamp(-F8_MAX, F8_MAX).to(F8).view(torch.uint8)
    slots = torch.arange(W * P, device=pool.device).reshape(W, P)
    in_use = slots[None] < new_len[:, None, None]
    dst = st["new_tables"].long()
    at_page = dst[:, :, None].expand(bs, W, P)[in_use]
    at_off = (slots % P)[None].expand(bs, W, P)[in_use]
    pool.view(torch.uint8)[at_page, :, at_off] = code.permute(0, 2, 3, 1, 4)[in_use]
    used_page = in_use.any(2)
    scale[dst[used_page]] = s.permute(0, 2, 1)[used_page]


def _plain_evict(st):
    mass, ctx, keep = st["mass"], st["ctx"].long(), st["keep"]
    bs, H, L = mass.shape
    t = torch.arange(L, device=mass.device)
    held = t[None, :] < ctx[:, None]
    safe = held & ((t[None, :] < st["sinks"]) | (t[None, :] >= ctx[:, None] - st["recent"]))
    rank = torch.where(safe[:, None], math.inf, mass)
    rank = torch.where(held[:, None], rank, -math.inf)
    rank = torch.nn.functional.pad(rank, (0, max(0, keep - L)), value=-math.inf)
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :keep]
    new_len = ctx.clamp(max=keep)
    i = torch.arange(keep, device=mass.device)
    there = i[None, None, :] < new_len[:, None, None]
    kept = torch.where(there, order, 2 ** 31 - 1).sort(-1).values
    kept = torch.where(there, kept, -1)
    m = torch.where(there, mass.gather(2, kept.clamp(min=0)), torch.zeros((), device=mass.device))
    mass_out = torch.nn.functional.pad(m, (0, max(0, L - keep)))[..., :L].contiguous()
    _plain_evict_one(st, st["kc"], st["ks"], kept, new_len)
    _plain_evict_one(st, st["vc"], st["vs"], kept, new_len)
    return kept.to(torch.int32), new_len.to(torch.int32), mass_out


def _evict_outputs(st, kept, new_len, mass_out):
    # the pages that the call wrote, with what their slots and scales now hold
    t = st["new_tables"].long()
    return kept, new_len, mass_out, st["kc"][t], st["vc"][t], st["ks"][t], st["vs"][t]


# ------------------------------------------------------------------ one pass

def run(state):
    st = state
    if own:
        return _run_own(st)
    if st["op"] == "append":
        return _plain_append(st)
    if st["op"] == "attention":
        return _plain_attention(st)
    if st["op"] == "weigh":
        return _plain_weigh(st)
    return _evict_outputs(st, *_plain_evict(st))


def _run_own(st):
    from sparse_attention_indexer_pmqa_gb300 import pmqa
    cache = (st["kc"], st["vc"], st["ks"], st["vs"], st["tables"], st["ctx"])
    if st["op"] == "append":
        pmqa.pmqa_cache_append(st["k"], st["v"], *cache, st["row_begin"], st["max_rows"],
                               ws=st["ws"])
        return st["kc"], st["vc"], st["ks"], st["vs"]
    if st["op"] == "attention":
        return pmqa.pmqa_cache_attention(st["q"], *cache, st["row_begin"], st["max_rows"],
                                         st["sm_scale"], want_lse=True, ws=st["ws"])
    if st["op"] == "weigh":
        return pmqa.pmqa_cache_weigh(st["q"], st["kc"], st["ks"], st["tables"], st["ctx"],
                                     st["row_begin"], st["max_rows"], st["sm_scale"], st["lse"],
                                     st["mass_in"], mass_out=st["mass"], ws=st["ws"])
    kept, new_len, mass_out = pmqa.pmqa_cache_evict(
        *cache, st["mass"], st["keep"], st["sinks"], st["recent"], st["new_tables"], ws=st["ws"])
    return _evict_outputs(st, kept, new_len, mass_out)


def work(case):
    rows, ctx = _lens(case)
    H, Hq, D, P = case["kv_heads"], case["heads"], case["head_dim"], case["block"]
    total = sum(rows)
    pages = sum(-(-c // P) for c in ctx)
    # slots seen by row j of n rows behind c slots in all: c - n + j + 1
    seen = sum(n * (c - n) + n * (n + 1) // 2 for n, c in zip(rows, ctx))
    if case["op"] == "append":
        touched = sum((c - 1) // P - (c - n) // P + 1 for n, c in zip(rows, ctx))
        return {"bytes": 2 * total * H * D * 3 + 2 * touched * (8 * H + 4), "flops": 0}
    if case["op"] == "attention":
        b = 2 * H * D * sum(ctx) + pages * (8 * H + 4) + total * Hq * (4 * D + 4)
        return {"bytes": b, "flops": 4 * D * Hq * seen}
    if case["op"] == "weigh":
        b = H * D * sum(ctx) + pages * (4 * H + 4) + total * Hq * (2 * D + 4) + 8 * H * sum(ctx)
        return {"bytes": b, "flops": 2 * D * Hq * seen}
    new = sum(min(c, case["keep"]) for c in ctx)
    L = (max(-(-c // P) for c in ctx) + 1) * P
    return {"bytes": H * (4 * sum(ctx) + 4 * D * new + 4 * L * case["bs"]
                          + 4 * case["keep"] * case["bs"]), "flops": 0}


# ------------------------------------------------------------------ 64-bit definition

def _e4m3(x):
    """The e4m3 value nearest to each fp64 value (ties to even), at most 448."""
    a = x.abs().clamp(max=F8_MAX)
    step = torch.exp2(torch.floor(torch.log2(a.clamp(min=2.0 ** -6))) - 3)
    return torch.sign(x) * torch.round(a / step) * step


def _scale_of(amax):
    e = torch.round(torch.log2(amax) - math.log2(F8_MAX))
    e = torch.where(F8_MAX * torch.exp2(e) >= amax, e, e + 1)
    return torch.where(amax > 0, torch.exp2(e), torch.zeros_like(amax)).clamp(min=2.0 ** -100)


def _exact_append(st, x, pool, scale, rows, ctx, P):
    pool, scale, tables = pool.double(), scale.double(), st["tables"].tolist()
    at = 0
    for i, (n, c) in enumerate(zip(rows, ctx)):
        first, new = c - n, x[at:at + n].double()  # [n, heads, dim]
        at += n
        for b in range(first // P, (c - 1) // P + 1):
            page, lo, hi = tables[i][b], max(first, b * P), min(c, (b + 1) * P)
            part = new[lo - first:hi - first].transpose(0, 1)
            s, held = _scale_of(part.abs().amax((1, 2))), lo - b * P
            if held:
                s = torch.maximum(s, scale[page])
                old = pool[page, :, :held] * (scale[page] / s)[:, None, None]
                grew = (s != scale[page])[:, None, None]
                pool[page, :, :held] = torch.where(grew, _e4m3(old), pool[page, :, :held])
            pool[page, :, held:hi - b * P] = _e4m3(part / s[:, None, None])
            scale[page] = s
    return pool, scale


def _exact_evict(st, ctx, P):
    keep, sinks, recent = st["keep"], st["sinks"], st["recent"]
    mass, tables, new_tables = st["mass"], st["tables"].long(), st["new_tables"].long()
    out_mass = torch.zeros_like(mass, dtype=torch.float64)
    pools = [[p.double(), s.double()] for p, s in ((st["kc"], st["ks"]), (st["vc"], st["vs"]))]
    H, W = mass.shape[1], new_tables.shape[1]
    heads = torch.arange(H, device=mass.device)[:, None]
    for i, c in enumerate(ctx):
        n = min(c, keep)
        rank = mass[i, :, :c].clone()
        rank[:, :sinks] = math.inf
        rank[:, max(0, c - recent):] = math.inf
        kept = (-rank.double()).argsort(dim=1, stable=True)[:, :n].sort(1).values
        out_mass[i, :, :n] = mass[i].double().gather(1, kept)
        page = tables[i][kept // P]
        for pool, scale in pools:
            x = pool[page, heads, kept % P] * scale[page, heads][..., None]
            x = torch.nn.functional.pad(x, (0, 0, 0, W * P - n)).reshape(H, W, P, -1)
            s = _scale_of(x.abs().amax((2, 3)))
            x = _e4m3(x / s[..., None, None])
            for b in range(-(-n // P)):
                m = min(P, n - b * P)
                pool[new_tables[i, b], :, :m] = x[:, b, :m]
                scale[new_tables[i, b]] = s[:, b]
    t = new_tables
    (k, ks), (v, vs) = pools
    return None, None, out_mass, k[t], v[t], ks[t], vs[t]


def exact(case, seed):
    """What `run` returns, in 64 bits from the definition, request by request."""
    rows, ctx = _lens(case)
    if case["op"] in ("attention", "weigh"):
        seen = sum(n * c for n, c in zip(rows, ctx))
        if seen * case["heads"] * case["head_dim"] > 5e11:
            return None
    st = prepare(case, seed)
    P, H, G = case["block"], case["kv_heads"], case["heads"] // case["kv_heads"]
    if case["op"] == "append":
        k, ks = _exact_append(st, st["k"], st["kc"], st["ks"], rows, ctx, P)
        v, vs = _exact_append(st, st["v"], st["vc"], st["vs"], rows, ctx, P)
        return k, v, ks, vs
    if case["op"] == "evict":
        return _exact_evict(st, ctx, P)
    tables = st["tables"].cpu()

    def tokens(pool, scale, i, c):
        ids = tables[i, :-(-c // P)].long().cuda()
        x = pool[ids].double() * scale[ids].double()[:, :, None, None]
        return x.transpose(0, 1).reshape(H, -1, x.shape[-1])[:, :c]

    outs, lses, at = [], [], 0
    mass = st["mass"].double() if case["op"] == "weigh" else None
    for i, (n, c) in enumerate(zip(rows, ctx)):
        q = st["q"][at:at + n].double().reshape(n, H, G, -1)
        s = torch.einsum("nhgd,htd->hgnt", q, tokens(st["kc"], st["ks"], i, c)) * st["sm_scale"]
        slot = torch.arange(c, device="cuda")
        s.masked_fill_(slot[None, :] > slot[c - n:, None], -math.inf)
        if mass is not None:
            lse = st["lse"][at:at + n].double().reshape(n, H, G).permute(1, 2, 0)
            w = (s - lse[..., None]).exp().sum((1, 2))
            mass[i, :, :c] = st["mass_in"][i, :, :c].double() + w
        else:
            lse = torch.logsumexp(s, -1)
            o = torch.einsum("hgnt,htd->nhgd", (s - lse[..., None]).exp(),
                             tokens(st["vc"], st["vs"], i, c))
            outs.append(o.reshape(n, H * G, -1))
            lses.append(lse.permute(2, 0, 1).reshape(n, H * G))
        at += n
    return mass if mass is not None else (torch.cat(outs), torch.cat(lses))
