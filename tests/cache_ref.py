"""Plain 64-bit forms of the operators on the 8-bit K/V cache, request by
request, with the error bounds of the kernels' number formats, and the random
problems that the tests run them on (torch on the CPU)."""

import math
from types import SimpleNamespace

import torch

F8 = torch.float8_e4m3fn
NAN8 = 0x7F


def scale_of(amax: torch.Tensor) -> torch.Tensor:
    """2^ceil(log2(a / 448)), at least 2^-100, for fp64 a >= 0."""
    m, e = torch.frexp(amax)  # a = m 2^e, 448 = 0.875 * 2^9
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=-100)
    e = torch.where(amax > 0, e, torch.full_like(e, -100))
    return torch.ldexp(torch.ones_like(amax), e)


def to_code(x: torch.Tensor) -> torch.Tensor:
    """uint8 e4m3 codes of fp64 values, nearest even, saturated (through fp32,
    in which every value handed in here is exact)."""
    return x.float().clamp(-448.0, 448.0).to(F8).view(torch.uint8)


def value(code: torch.Tensor) -> torch.Tensor:
    return code.view(F8).double()


def make(rows, ctx, *, kv_heads, group, head_dim, block, seed=0, spare=3, poison=True, lead=0,
         tail=0, scales="pow2"):
    """A cache with the requests' tokens in a random set of blocks. poison: NaN
    in every slot and scale that no request holds. lead / tail: rows of no
    request before and behind the requests' own."""
    g = torch.Generator().manual_seed(seed)
    bs = len(ctx)
    pages = [-(-c // block) for c in ctx]
    W = max(pages + [1]) + 1
    nb = sum(pages) + spare
    perm = torch.randperm(nb, generator=g).to(torch.int32)
    bt = torch.full((bs, W), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(pages):
        bt[i, :n] = perm[at:at + n]
        at += n

    def pool():
        x = torch.randn((nb, kv_heads, block, head_dim), generator=g, dtype=torch.float64)
        x *= torch.exp2(torch.randn((nb, kv_heads, 1, 1), generator=g, dtype=torch.float64))
        s = scale_of(x.abs().amax((2, 3)))
        if scales == "any":  # scales that no append made
            s = (s * (1.0 + torch.rand(s.shape, generator=g, dtype=torch.float64))).float().double()
        code = to_code(x / s[:, :, None, None])
        s = s.float()
        if poison:
            held = torch.zeros((nb, block), dtype=torch.bool)
            for i, c in enumerate(ctx):
                for t in range(c):
                    held[bt[i, t // block], t % block] = True
            code[~held[:, None, :].expand(nb, kv_heads, block)] = NAN8
            s[~held.any(1)] = math.nan
        return code, s

    kc, ks = pool()
    vc, vs = pool()
    rb = [lead]
    for n in rows:
        rb.append(rb[-1] + n)
    total = rb[-1] + tail
    q = torch.randn((total, kv_heads * group, head_dim), generator=g)
    return SimpleNamespace(
        kc=kc, ks=ks, vc=vc, vs=vs, bt=bt, ctx=torch.tensor(ctx, dtype=torch.int32),
        rb=torch.tensor(rb, dtype=torch.int32), max_rows=max(list(rows) + [1]), q=q.to(torch.bfloat16),
        k_new=torch.randn((total, kv_heads, head_dim), generator=g).to(torch.bfloat16),
        v_new=torch.randn((total, kv_heads, head_dim), generator=g).to(torch.bfloat16),
        free=perm[at:], rows=list(rows), H=kv_heads, G=group, D=head_dim, P=block, bs=bs,
        sm=head_dim ** -0.5, gen=g)


def tokens(code, scale, bt, i, c, P):
    """The c cached tokens of request i, fp64 [H, c, D], and each one's scale [H, c]."""
    ids = bt[i, :-(-c // P)].long()
    x = value(code[ids]) * scale[ids].double()[:, :, None, None]
    H, D = code.shape[1], code.shape[3]
    s = scale[ids].double()[:, :, None].expand(-1, -1, P)
    return (x.transpose(0, 1).reshape(H, -1, D)[:, :c], s.transpose(0, 1).reshape(H, -1)[:, :c])


def _scores(p, i):
    """Scores of request i, fp64 [H, G, n, c] with -inf where a row does not see
    a token, and a bound of the kernels' error in them."""
    n, c = p.rows[i], int(p.ctx[i])
    r0 = int(p.rb[i])
    q = p.q[r0:r0 + n].double().reshape(n, p.H, p.G, p.D)
    k, _ = tokens(p.kc, p.ks, p.bt, i, c, p.P)
    s = torch.einsum("nhgd,htd->hgnt", q, k) * p.sm
    # fp32 accumulation of D products, each sum off by at most one unit of 2^-23 of
    # the absolute products' sum; q split or scaled loses at most 2^-17 of its
    # row's largest value per element; three fp32 multiplications of the score
    mag = torch.einsum("nhgd,htd->hgnt", q.abs(), k.abs()) * abs(p.sm)
    top = torch.einsum("nhg,ht->hgnt", q.abs().amax(-1), k.abs().sum(-1)) * abs(p.sm)
    err = mag * (p.D + 4) * 2.0 ** -23 + top * 2.0 ** -17
    j = torch.arange(n)[:, None]
    late = torch.arange(c)[None, :] > c - n + j
    return s.masked_fill(late, -math.inf), err.masked_fill(late, 0.0)


def attention(p):
    """(out, lse, tolerance of out, tolerance of lse) over all rows; NaN where
    no request has a row."""
    total, Hq = p.q.shape[0], p.H * p.G
    out = torch.full((total, Hq, p.D), math.nan, dtype=torch.float64)
    lse = torch.full((total, Hq), math.nan, dtype=torch.float64)
    tol, ltol = out.clone(), lse.clone()
    for i in range(p.bs):
        n, c = p.rows[i], int(p.ctx[i])
        if n == 0:
            continue
        r0 = int(p.rb[i])
        if c == 0:
            out[r0:r0 + n], lse[r0:r0 + n] = 0.0, -math.inf
            tol[r0:r0 + n], ltol[r0:r0 + n] = 0.0, 0.0
            continue
        s, err = _scores(p, i)
        l = torch.logsumexp(s, -1)
        w = torch.where(torch.isinf(l)[..., None], torch.zeros_like(s), (s - l[..., None]).exp())
        v, vs = tokens(p.vc, p.vs, p.bt, i, c, p.P)
        o = torch.einsum("hgnt,htd->nhgd", w, v)
        # a weight is off by its score's error, 2^-20 for the exponential and its
        # argument (|x| < 2^6 in base 2, fp32), and 2^-11 for its f16 rounding
        # or 2^-25 of the largest weight (the f16 subnormal step, under a block
        # scale of up to 32 times the token's)
        de = err.amax(-1) + 2.0 ** -18
        spread = torch.einsum("hgnt,htd->nhgd", w * (2.0 ** -11 + 2.0 * (err + de[..., None])), v.abs())
        floor = c * 2.0 ** -25 * 32.0 * 448.0 * vs.amax(-1)  # [H]
        d = o.abs() * 2.0 ** -8 + spread + floor[None, :, None, None]
        out[r0:r0 + n] = o.reshape(n, Hq, p.D)
        tol[r0:r0 + n] = d.reshape(n, Hq, p.D)
        lse[r0:r0 + n] = l.permute(2, 0, 1).reshape(n, Hq)
        e = de + torch.where(torch.isinf(l), torch.zeros_like(l), l.abs()) * 2.0 ** -21
        ltol[r0:r0 + n] = e.permute(2, 0, 1).reshape(n, Hq)
    return out, lse, tol, ltol


def weigh(p, lse, mass_in):
    """(mass_out, tolerance): entries of cached tokens; the others NaN."""
    out = torch.full(mass_in.shape, math.nan, dtype=torch.float64)
    tol = torch.zeros_like(out)
    for i in range(p.bs):
        n, c = p.rows[i], min(int(p.ctx[i]), mass_in.shape[2])
        had = mass_in[i, :, :c].double()
        out[i, :, :c] = had
        if n == 0 or c == 0:
            continue
        s, err = _scores(p, i)
        r0 = int(p.rb[i])
        l = lse[r0:r0 + n].double().reshape(n, p.H, p.G).permute(1, 2, 0)[..., None]
        w = torch.where(torch.isinf(s), torch.zeros_like(s), (s - l).exp())
        # the exponent's error, 2^-20 for the exponential and lse in base 2, the fp32
        # sum, and 2^-126 where a weight below the normal range is taken for 0
        d = w * (err + 2.0 ** -18 + l.abs().nan_to_num(0, 0, 0) * 2.0 ** -22)
        out[i, :, :c] += w.sum((1, 2))[:, :c]
        tol[i, :, :c] = d.sum((1, 2))[:, :c] + out[i, :, :c].abs() * (n * p.G + 2) * 2.0 ** -24
        tol[i, :, :c] += n * p.G * 2.0 ** -126
    return out, tol


def append(p):
    """Codes and scales of both pools after the call."""
    res = []
    for code, scale, new in ((p.kc, p.ks, p.k_new), (p.vc, p.vs, p.v_new)):
        code, scale = code.clone(), scale.clone()
        for i in range(p.bs):
            n, c = p.rows[i], int(p.ctx[i])
            first, r0 = c - n, int(p.rb[i])
            lo0 = max(first, 0)
            for b in range(lo0 // p.P, (c - 1) // p.P + 1) if n and c else ():
                page, lo, hi = int(p.bt[i, b]), max(lo0, b * p.P), min(c, (b + 1) * p.P)
                x = new[r0 + lo - first:r0 + hi - first].double().transpose(0, 1)  # [H, m, D]
                a = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax((1, 2))
                s, held = scale_of(a), lo - b * p.P
                if held:
                    old = scale[page].double()
                    s = torch.maximum(s, old)
                    back = to_code(value(code[page, :, :held]) * old[:, None, None] / s[:, None, None])
                    grew = (s != old)[:, None, None]
                    code[page, :, :held] = torch.where(grew, back, code[page, :, :held])
                # x / s in fp32, the nearest value, then the nearest code
                y = (x / s[:, None, None]).float().double()
                code[page, :, held:hi - b * p.P] = to_code(y)
                scale[page] = s.float()
        res += [code, scale]
    return res


def evict(p, mass, keep, sinks, recent, new_tables):
    """(kept, lens, mass_out, kc, ks, vc, vs)."""
    bs, H, width = mass.shape
    kept = torch.full((bs, H, keep), -1, dtype=torch.int32)
    mass_out = torch.zeros_like(mass)
    lens = torch.clamp(p.ctx, max=keep)
    pools = [[p.kc.clone(), p.ks.clone()], [p.vc.clone(), p.vs.clone()]]
    for i in range(bs):
        c, n = int(p.ctx[i]), int(lens[i])
        for h in range(H):
            def rank(t):
                m = float(mass[i, h, t])
                if t < sinks or t >= c - recent:
                    return (-2, 0.0, t)
                return (0, 0.0, t) if math.isnan(m) else (-1, -m, t)

            slots = sorted(sorted(range(c), key=rank)[:n])
            kept[i, h, :n] = torch.tensor(slots, dtype=torch.int32)
            mass_out[i, h, :n] = mass[i, h, slots]
            for pool in pools:
                code, scale = pool
                for b in range(-(-n // p.P)):
                    part = slots[b * p.P:(b + 1) * p.P]
                    ids = p.bt[i, [t // p.P for t in part]].long()
                    off = torch.tensor([t % p.P for t in part])
                    x = value(code[ids, h, off]) * scale[ids, h].double()[:, None]
                    a = torch.where(torch.isfinite(x), x.abs(), torch.zeros_like(x)).amax()
                    s = scale_of(a)
                    d = int(new_tables[i, b])
                    code[d, h, :len(part)] = to_code((x / s).float().double())
                    scale[d, h] = s.float()
    return kept, lens, mass_out, pools[0][0], pools[0][1], pools[1][0], pools[1][1]
