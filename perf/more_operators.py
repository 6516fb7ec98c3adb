"""Cases and plain forms of the operators around the sparse-MLA step: what writes
its caches and what attends to all of a latent cache.

`rope` rotates query and key heads; `index_append` normalises, rotates and
quantises a step's new indexer keys into the paged cache of 132-byte rows (128
e4m3 values and an fp32 scale) and its queries into fp8 with their scales folded
into the head weights; `index_read` gives cached keys back as contiguous rows;
`latent_append` writes the latent cache (576 e4m3 values a token, one scale for
all) and its queries; `latent_attention` attends to every cached token.

Rows of a call are ragged: request i owns rows row_begin[i] .. row_begin[i + 1]
and its row j sits at slot context_lens[i] - n_i + j.
"""

import itertools
import math

import torch

own = False

F8 = torch.float8_e4m3fn
F8_MAX = 448.0
TINY = 2.0 ** -100
LATENT, VALUES, ROTARY = 576, 512, 64


# ------------------------------------------------------------------ the cases

def listed():
    rot = dict(interleaved=False, factor=1.0, base=10000.0)
    yarn = dict(interleaved=True, factor=40.0, base=10000.0)
    return [
        # one decode step of 64 requests, all of each head rotated: latency counts
        dict(rot, name="rope_step", op="rope", rows=64, heads=32, kv_heads=8, head_dim=128, begin=0,
             dim=128, far=32768),
        # a scheduler step of 12 k prompt tokens, the last 64 of 192 values of each head, long contexts
        dict(yarn, name="rope_prompts", op="rope", rows=12000, heads=32, kv_heads=1, head_dim=192,
             begin=128, dim=64, far=150000),
        # the indexer's inputs of a speculative decode step: 32 requests of 4 rows, pages of one token
        dict(yarn, name="index_step", op="index_append", bs=32, rows_lo=4, rows_hi=4, ctx_lo=16384,
             ctx_hi=65536, heads=64, block=1, norm=1),
        # the same of prompt chunks, thousands of rows
        dict(yarn, name="index_prompts", op="index_append", bs=6, rows_lo=700, rows_hi=4096,
             ctx_lo=1000, ctx_hi=8192, heads=64, block=64, norm=1),
        # the cached keys of one request, for the prefill logits of its next chunk
        dict(name="read_single", op="index_read", bs=1, ctx_lo=8192, ctx_hi=8192, block=1),
        # the keys of a batch of long requests
        dict(name="read_batch", op="index_read", bs=32, ctx_lo=16384, ctx_hi=65536, block=64),
        # latent rows and queries of a decode step
        dict(yarn, name="latent_step", op="latent_append", bs=32, rows_lo=4, rows_hi=4, ctx_lo=16384,
             ctx_hi=65536, heads=16, block=1, norm=2),
        # the same of prompt chunks
        dict(yarn, name="latent_prompts", op="latent_append", bs=6, rows_lo=700, rows_hi=4096,
             ctx_lo=1000, ctx_hi=8192, heads=16, block=64, norm=2),
        # one chat at its start: the smallest attention, where latency counts
        dict(name="attend_single", op="latent_attention", bs=1, rows_lo=1, rows_hi=1, ctx_lo=500,
             ctx_hi=500, heads=16, block=16, long=0),
        # batch decode, all 128 heads on one GPU
        dict(name="attend_batch", op="latent_attention", bs=64, rows_lo=1, rows_hi=1, ctx_lo=4096,
             ctx_hi=32768, heads=128, block=64, long=0),
        # speculative verify of four draft rows, 16 heads a GPU, long contexts
        dict(name="attend_verify", op="latent_attention", bs=32, rows_lo=4, rows_hi=4, ctx_lo=16384,
             ctx_hi=65536, heads=16, block=1, long=0),
        # prompt chunks behind cached tokens
        dict(name="attend_prompts", op="latent_attention", bs=3, rows_lo=700, rows_hi=1200, ctx_lo=1500,
             ctx_hi=6000, heads=128, block=64, long=0),
    ]


def draw(rng):
    def logint(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["rope", "index_append", "index_read", "latent_append", "latent_attention",
                     "latent_attention", "latent_attention"])
    block = rng.choice([1, 1, 8, 16, 24, 48, 64, 64, 128])
    rot = dict(interleaved=rng.random() < 0.5, factor=rng.choice([1.0, 4.0, 40.0]),
               base=rng.choice([10000.0, 500000.0]))
    if op == "rope":
        head_dim = rng.choice([64, 80, 96, 128, 192])
        dim = rng.choice([d for d in (16, 32, 64, 80, 96, 128, 192) if d <= head_dim])
        return dict(rot, op=op, rows=logint(1, 8000), heads=rng.randint(1, 40),
                    kv_heads=rng.randint(1, 8), head_dim=head_dim, dim=dim,
                    begin=8 * rng.randint(0, (head_dim - dim) // 8), far=logint(100, 1000000))
    if op == "index_read":
        hi = logint(64, 65536)
        return dict(op=op, bs=logint(1, 32), ctx_lo=max(1, hi // 8), ctx_hi=hi, block=block)
    if op in ("index_append", "latent_append"):
        index = op == "index_append"
        c = dict(rot, op=op, block=block, norm=rng.choice([0, 1, 2]),
                 heads=rng.choice([16, 32, 64]) if index else rng.choice([8, 16, 24, 32]))
        if rng.random() < 0.5:
            return dict(c, bs=logint(1, 128), rows_lo=1, rows_hi=rng.choice([1, 2, 4]), ctx_lo=1,
                        ctx_hi=logint(8, 16384))
        hi = logint(8, 2500)
        return dict(c, bs=logint(1, 5), rows_lo=max(1, hi // 5), rows_hi=hi, ctx_lo=1,
                    ctx_hi=logint(hi, 3 * hi))
    c = dict(op=op, block=block, heads=rng.choice([1, 5, 8, 16, 16, 20, 32, 40, 64, 96, 128]), long=0)
    kind = rng.choice(["decode", "decode", "prompt", "mixed"])
    if kind == "decode":
        n = rng.choice([1, 1, 2, 3, 4])
        hi = logint(64, 65536)
        most = min(64, 1200000 // hi, 12000000 // (hi * n * c["heads"] // 16 + 1))
        return dict(c, bs=logint(1, max(1, most)), rows_lo=n, rows_hi=n, ctx_lo=max(1, hi // 8), ctx_hi=hi)
    if kind == "prompt":
        hi = logint(17, 700)
        return dict(c, bs=logint(1, 3), rows_lo=max(1, hi // 2), rows_hi=hi, ctx_lo=1,
                    ctx_hi=logint(hi, 4 * hi))
    return dict(c, heads=min(c["heads"], 40), bs=logint(4, 20), rows_lo=1, rows_hi=logint(40, 500),
                long=2, ctx_lo=1, ctx_hi=logint(100, 4096))


def _spread(lo, hi, n, turn):
    """n whole numbers over [lo, hi], the same for every call (golden-ratio steps)."""
    return [lo + int((hi - lo + 1) * ((0.5 + (i + turn) * 0.6180339887498949) % 1.0))
            for i in range(n)]


def _lens(case):
    """New rows and context length (with the new rows) of every request."""
    bs = case["bs"]
    ctx = _spread(case["ctx_lo"], case["ctx_hi"], bs, 0)
    if case["op"] == "index_read":
        return ctx, ctx
    rows = _spread(case["rows_lo"], case["rows_hi"], bs, 3)
    if case.get("long"):
        rows = [case["rows_hi"] - 37 * i if i < case["long"] else case["rows_lo"] for i in range(bs)]
        rows = [max(1, r) for r in rows]
    return rows, [max(c, r) for c, r in zip(ctx, rows)]


# ------------------------------------------------------------------ inputs

def _inv_freq(case, dim):
    """Radians per position of each pair, fp64: base^(-2 i / dim), slowed by `factor` where the
    pair turns less than once over 4096 positions, kept where more than 32 times, between them in
    parts."""
    i = torch.arange(dim // 2, dtype=torch.float64)
    f = case["base"] ** (-2.0 * i / dim)
    if case["factor"] == 1.0:
        return f
    at = [dim * math.log(4096 / (2 * math.pi * turns)) / (2 * math.log(case["base"])) for turns in (32, 1)]
    lo, hi = max(0, math.floor(at[0])), min(dim - 1, math.ceil(at[1]))
    slowed = ((i - lo) / max(hi - lo, 0.001)).clamp(0, 1)
    return f * (1 - slowed) + f / case["factor"] * slowed


def _rotary_scale(case):
    return 1.0 if case["factor"] == 1.0 else 0.1 * math.log(case["factor"]) + 1.0


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def randn(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    def heads(rows, n, dim, spread=0.5):
        # channels of different size, as trained projections give
        return (randn(rows, n, dim) * torch.exp2(randn(1, n, dim) * spread)).to(torch.bfloat16)

    op = case["op"]
    st = dict(op=op)
    if op in ("rope", "index_append", "latent_append"):
        st["dim"] = case["dim"] if op == "rope" else ROTARY
        st["begin"] = case["begin"] if op == "rope" else 0
        st["inv_freq"] = _inv_freq(case, st["dim"]).to(dev)
        st["interleaved"], st["scale"] = case["interleaved"], _rotary_scale(case)
    if op == "rope":
        n, D = case["rows"], case["head_dim"]
        st["positions"] = torch.randint(0, case["far"], (n,), generator=gen, device=dev, dtype=torch.int32)
        st["q"], st["k"] = heads(n, case["heads"], D), heads(n, case["kv_heads"], D)
        return st
    rows, ctx = _lens(case)
    bs, P, total = case["bs"], case["block"], sum(rows)
    pages = [-(-c // P) for c in ctx]
    blocks = sum(pages) + 3
    perm = torch.randperm(blocks, generator=gen, device=dev).to(torch.int32)
    tables = torch.full((bs, max(pages) + 1), -1, dtype=torch.int32, device=dev)
    at = 0
    for i, n in enumerate(pages):
        tables[i, :n] = perm[at:at + n]
        at += n
    st.update(tables=tables, ctx=torch.tensor(ctx, dtype=torch.int32, device=dev), max_rows=max(rows),
              row_begin=torch.tensor([0] + list(itertools.accumulate(rows)), dtype=torch.int32, device=dev))
    if op in ("index_append", "index_read"):
        st["kv"] = _index_pool(gen, blocks, P, dev)
    else:
        st["kv"], st["kv_scale"] = _latent_pool(gen, blocks, P, dev)
    if op == "index_append":
        st["k"] = heads(total, 1, 128, 0.3)[:, 0]
        st["q"], st["w"] = heads(total, case["heads"], 128), randn(total, case["heads"])
        st["weight_scale"] = (128 * case["heads"]) ** -0.5
        st["norm"] = _norm(case["norm"], randn, 128)
    if op == "latent_append":
        # the projection gives a row's latent and rotary parts side by side
        st["kv_new"] = heads(total, 1, LATENT, 0.3)[:, 0].contiguous()
        st["norm"] = _norm(case["norm"], randn, VALUES)
        st["q_c"], st["q_pe"] = heads(total, case["heads"], VALUES), heads(total, case["heads"], ROTARY)
        st["q_scale"] = 0.0375
    if op == "latent_attention":
        x = randn(total, case["heads"], LATENT) * torch.exp2(randn(1, case["heads"], LATENT) * 0.5)
        st["q_scale"], st["sm_scale"] = 0.05, 192 ** -0.5
        st["q"] = (x / st["q_scale"]).clamp(-F8_MAX, F8_MAX).to(F8)
    if op != "index_read":
        # the scratch memory that a program keeps beside its cache
        st["ws"] = torch.zeros(48 << 20, dtype=torch.uint8, device=dev)
    else:
        st["ws"] = torch.zeros(256, dtype=torch.uint8, device=dev)
    st["total"] = total
    return st


def _norm(kind, randn, n):
    """(kind, weight, bias): 0 none, 1 layer norm, 2 root mean square."""
    weight = 1.0 + 0.1 * randn(n) if kind else None
    return kind, weight, 0.1 * randn(n) if kind == 1 else None


def _index_pool(gen, blocks, P, dev):
    x = torch.randn((blocks * P, 128), generator=gen, device=dev)
    s = x.abs().amax(1, keepdim=True) / F8_MAX
    pool = torch.empty((blocks * P, 132), dtype=torch.uint8, device=dev)
    pool[:, :128] = (x / s).to(F8).view(torch.uint8)
    pool[:, 128:] = s.view(torch.uint8)
    return pool.reshape(blocks, P, 132)


def _latent_pool(gen, blocks, P, dev):
    x = torch.randn((blocks, P, LATENT), generator=gen, device=dev)
    x *= torch.exp2(torch.randn((1, 1, LATENT), generator=gen, device=dev) * 0.5)
    return (x / 0.03).clamp_(-F8_MAX, F8_MAX).to(F8), 0.03


# ------------------------------------------------------------------ plain forms

def _rotate(st, x, positions, begin):
    """fp32 x [rows, heads, D] with dims begin .. begin + dim of each head rotated."""
    d = st["dim"]
    angle = positions.double()[:, None] * st["inv_freq"]
    cos, sin = (angle.cos() * st["scale"]).float()[:, None], (angle.sin() * st["scale"]).float()[:, None]
    r = x[..., begin:begin + d]
    if st["interleaved"]:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = r[..., :d // 2], r[..., d // 2:]
        r = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((x[..., :begin], r, x[..., begin + d:]), -1)


def _normed(norm, x, eps=1e-6):
    kind, weight, bias = norm
    if kind == 1:
        x = x - x.mean(-1, keepdim=True)
    if kind:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * weight
    return x if bias is None else x + bias


def _slots(st):
    """The position of every row in its request, and its place in the pool."""
    rb, ctx, tables = st["row_begin"].long(), st["ctx"].long(), st["tables"].long()
    r = torch.arange(st["total"], device=rb.device)
    req = torch.searchsorted(rb[1:].contiguous(), r, right=True)
    slot = ctx[req] - (rb[1:] - rb[:-1])[req] + r - rb[req]
    P = st["kv"].shape[1]
    return slot, tables[req, slot // P] * P + slot % P


def _coded(x, s):
    return (x / s).clamp(-F8_MAX, F8_MAX).to(F8)


def _index_views(st):
    """The pool's codes and scales, as they lie."""
    return st["kv"].view(F8)[..., :128], st["kv"].view(torch.float32)[..., 32]


def _plain_index_append(st):
    slot, at = _slots(st)
    k = _rotate(st, _normed(st["norm"], st["k"].float())[:, None], slot, 0)[:, 0]
    s = k.abs().amax(1).clamp(min=TINY) / F8_MAX
    rows = st["kv"].reshape(-1, 132)
    rows[at, :128] = _coded(k, s[:, None]).view(torch.uint8)
    rows.view(torch.float32)[at, 32] = s
    q = _rotate(st, st["q"].float(), slot, 0)
    s = q.abs().amax(2).clamp(min=TINY) / F8_MAX
    return (*_index_views(st), _coded(q, s[..., None]), st["w"] * s * st["weight_scale"])


def _plain_index_read(st):
    _, at = _slots(st)
    rows = st["kv"].reshape(-1, 132)
    return rows[at, :128].view(F8), rows.view(torch.float32)[at, 32]


def _plain_latent_append(st):
    slot, at = _slots(st)
    c = _normed(st["norm"], st["kv_new"][:, :VALUES].float())
    pe = _rotate(st, st["kv_new"][:, None, VALUES:].float(), slot, 0)[:, 0]
    code = _coded(torch.cat((c, pe), -1), st["kv_scale"])
    st["kv"].view(torch.uint8).reshape(-1, LATENT)[at] = code.view(torch.uint8)
    q = torch.cat((st["q_c"].float(), _rotate(st, st["q_pe"].float(), slot, 0)), -1)
    return st["kv"], _coded(q, st["q_scale"])


def _plain_latent_attention(st):
    rb, R = st["row_begin"], st["max_rows"]
    n = rb[1:] - rb[:-1]
    j = torch.arange(R, device=rb.device)
    real = j[None, :] < n[:, None]
    q = st["q"].view(torch.uint8)[torch.where(real, rb[:-1, None] + j[None, :], 0).long()].view(F8)
    bs, _, H, _ = q.shape
    k = st["kv"][st["tables"].long().clamp(min=0)].float().reshape(bs, -1, LATENT)
    factor = st["sm_scale"] * st["q_scale"] * st["kv_scale"]
    s = torch.matmul(q.float().reshape(bs, R * H, LATENT), k.transpose(1, 2)).mul_(factor).reshape(bs, R, H, -1)
    t = torch.arange(k.shape[1], device=rb.device)
    last = st["ctx"][:, None] - n[:, None] + j[None, :]
    seen = (t[None, None, :] <= last[:, :, None]) & real[:, :, None]
    s.masked_fill_(~seen[:, :, None, :], -math.inf)
    top = s.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)
    s = s.sub_(top).exp_()
    total = s.sum(-1, keepdim=True)
    lse = (top + total.log()).squeeze(-1)[real]
    o = torch.matmul(s.reshape(bs, R * H, -1), k[..., :VALUES]).reshape(bs, R, H, VALUES)
    o = o * st["kv_scale"] / torch.where(total > 0, total, torch.ones_like(total))
    return o[real].to(torch.bfloat16), lse


def _plain_rope(st):
    return tuple(_rotate(st, st[x].float(), st["positions"], st["begin"]).to(torch.bfloat16) for x in "qk")


# ------------------------------------------------------------------ one pass

def run(state):
    st = state
    if own:
        return _run_own(st)
    return {"rope": _plain_rope, "index_append": _plain_index_append, "index_read": _plain_index_read,
            "latent_append": _plain_latent_append, "latent_attention": _plain_latent_attention}[st["op"]](st)


def _run_own(st):
    from sparse_attention_indexer_pmqa_gb300 import pmqa
    if st["op"] == "rope":
        rotary = pmqa.Rotary(st["inv_freq"], st["begin"], st["interleaved"], st["scale"])
        return pmqa.pmqa_rope(st["q"], st["positions"], rotary, other=st["k"])
    cache = (st["kv"], st["tables"], st["ctx"], st["row_begin"], st["max_rows"])
    if st["op"] == "index_append":
        rotary = pmqa.Rotary(st["inv_freq"], 0, st["interleaved"], st["scale"])
        q, w = pmqa.pmqa_index_append(st["k"], *cache, q=st["q"], weights=st["w"],
                                      weight_scale=st["weight_scale"], norm=pmqa.Norm(*st["norm"]),
                                      rotary=rotary, ws=st["ws"])
        return (*_index_views(st), q, w)
    if st["op"] == "index_read":
        return pmqa.pmqa_index_read(st["kv"], st["tables"], st["row_begin"], st["total"], ws=st["ws"])
    if st["op"] == "latent_append":
        rotary = pmqa.Rotary(st["inv_freq"], 0, st["interleaved"], st["scale"])
        q = pmqa.pmqa_latent_append(st["kv_new"][:, :VALUES], st["kv_new"][:, VALUES:], *cache,
                                    st["kv_scale"], q_c=st["q_c"], q_pe=st["q_pe"],
                                    q_scale=st["q_scale"], norm=pmqa.Norm(*st["norm"]), rotary=rotary,
                                    ws=st["ws"])
        return st["kv"], q
    return pmqa.pmqa_latent_attention(st["q"], *cache, st["q_scale"], st["kv_scale"], st["sm_scale"],
                                      want_lse=True, ws=st["ws"])


def work(case):
    if case["op"] == "rope":
        n, D = (case["heads"] + case["kv_heads"]) * case["head_dim"], case["dim"]
        return {"bytes": case["rows"] * (4 * n + 4), "flops": 6 * case["rows"] * n // case["head_dim"] * D}
    rows, ctx = _lens(case)
    total, H = sum(rows), case.get("heads", 0)
    pages = sum(-(-c // case["block"]) for c in ctx)
    touched = sum((c - 1) // case["block"] - (c - n) // case["block"] + 1 for n, c in zip(rows, ctx))
    if case["op"] == "index_read":
        return {"bytes": 264 * total + 4 * pages, "flops": 0}
    if case["op"] == "index_append":
        return {"bytes": total * (256 + 132 + H * (256 + 128 + 8)) + 4 * touched, "flops": 0}
    if case["op"] == "latent_append":
        return {"bytes": total * (1 + H) * (2 * LATENT + LATENT) + 4 * touched, "flops": 0}
    # slots seen by row j of n rows behind c slots in all: c - n + j + 1
    seen = sum(n * (c - n) + n * (n + 1) // 2 for n, c in zip(rows, ctx))
    return {"bytes": LATENT * sum(ctx) + 4 * pages + total * H * (LATENT + 2 * VALUES + 4),
            "flops": 2 * (LATENT + VALUES) * H * seen}


# ------------------------------------------------------------------ 64-bit definition

def _turned(st, x, positions, begin):
    """x with its pairs as complex numbers turned by scale * e^(i position frequency)."""
    half, d = st["dim"] // 2, st["dim"]
    i = torch.arange(half, device=x.device)
    a, b = (begin + 2 * i, begin + 2 * i + 1) if st["interleaved"] else (begin + i, begin + half + i)
    turn = torch.polar(torch.full((1, d // 2), st["scale"], dtype=torch.float64, device=x.device),
                       positions.double()[:, None] * st["inv_freq"])[:, None]
    z = torch.complex(x[..., a], x[..., b]) * turn
    y = x.clone()
    y[..., a], y[..., b] = z.real, z.imag
    return y


def _exact_norm(norm, x, eps=1e-6):
    kind, weight, bias = norm
    if kind == 0:
        return x
    if kind == 1:
        var, mean = torch.var_mean(x, -1, unbiased=False, keepdim=True)
        return (x - mean) / (var + eps).sqrt() * weight.double() + bias.double()
    return x / ((x ** 2).mean(-1, keepdim=True) + eps).sqrt() * weight.double()


def exact(case, seed):
    """What `run` returns, in 64 bits from the definition, request by request; what is held in 8
    bits before its rounding."""
    op = case["op"]
    if op == "rope":
        st = prepare(case, seed)
        return tuple(_turned(st, st[x].double(), st["positions"], st["begin"]) for x in "qk")
    rows, ctx = _lens(case)
    if op == "latent_attention":
        seen = sum(n * c for n, c in zip(rows, ctx))
        if seen * case["heads"] * (LATENT + VALUES) * 2 > 5e12:
            return None
    st = prepare(case, seed)
    P, tables = case["block"], st["tables"].cpu().long()

    def places(i, lo, hi):
        t = torch.arange(lo, hi)
        return (tables[i, t // P] * P + t % P).cuda()

    if op == "index_read":
        at = torch.cat([places(i, 0, c) for i, c in enumerate(ctx)])
        raw = st["kv"].reshape(-1, 132)[at]
        return raw[:, :128].contiguous().view(F8).double(), raw[:, 128:].contiguous().view(torch.float32)[:, 0].double()
    if op in ("index_append", "latent_append"):
        pos = torch.cat([torch.arange(c - n, c) for n, c in zip(rows, ctx)]).cuda()
        at = torch.cat([places(i, c - n, c) for i, (n, c) in enumerate(zip(rows, ctx))])
    if op == "index_append":
        codes, scales = (x.double().reshape(-1, *x.shape[2:]) for x in _index_views(st))
        k = _turned(st, _exact_norm(st["norm"], st["k"].double())[:, None], pos, 0)[:, 0]
        scales[at] = k.abs().amax(1) / F8_MAX
        codes[at] = k / scales[at][:, None]
        q = _turned(st, st["q"].double(), pos, 0)
        s = q.abs().amax(2) / F8_MAX
        shape = st["kv"].shape[:2]
        return (codes.reshape(*shape, 128), scales.reshape(shape), q / s[..., None],
                st["w"].double() * s * st["weight_scale"])
    if op == "latent_append":
        new = st["kv_new"].double()
        c = _exact_norm(st["norm"], new[:, :VALUES])
        pe = _turned(st, new[:, None, VALUES:], pos, 0)[:, 0]
        pool = st["kv"].double().reshape(-1, LATENT)
        pool[at] = (torch.cat((c, pe), 1) / st["kv_scale"]).clamp(-F8_MAX, F8_MAX)
        q = torch.cat((st["q_c"].double(), _turned(st, st["q_pe"].double(), pos, 0)), 2) / st["q_scale"]
        return pool.reshape(st["kv"].shape), q.clamp(-F8_MAX, F8_MAX)
    outs, lses, at = [], [], 0
    pool = st["kv"].reshape(-1, LATENT)
    for i, (n, c) in enumerate(zip(rows, ctx)):
        k = pool.view(torch.uint8)[places(i, 0, c)].view(F8).double() * st["kv_scale"]
        q = st["q"][at:at + n].double() * st["q_scale"]
        s = torch.einsum("nhd,td->nht", q, k) * st["sm_scale"]
        slot = torch.arange(c, device="cuda")
        s.masked_fill_((slot[None, :] > slot[c - n:, None])[:, None], -math.inf)
        lse = torch.logsumexp(s, -1)
        outs.append(torch.einsum("nht,td->nhd", (s - lse[..., None]).exp(), k[:, :VALUES]))
        lses.append(lse)
        at += n
    return torch.cat(outs), torch.cat(lses)
