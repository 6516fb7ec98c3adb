"""Plain 64-bit forms of the operators around the sparse-MLA step (rope, index
append and read, latent append and attention), request by request, with the error
bounds of the kernels' number formats, and the random problems that the tests run
them on (torch on the CPU).

Roundings: half a step, bf16 2^-8 and e4m3 2^-4 of the value (e4m3 2^-10 below its
smallest normal value 2^-6), fp32 2^-24. A rotated value a cos - b sin in fp32 is off
by at most 2^-20 (|a| + |b|) scale: the angle by pi 2^-25, cosine and sine by two
units, three roundings."""

import math
from types import SimpleNamespace

import torch

F8 = torch.float8_e4m3fn
NAN8 = 0x7F
TINY = 2.0 ** -100
LATENT, VALUES = 576, 512


def value(code):
    return code.view(F8).double()


def half_step(x):
    """Half a step of e4m3 at |x|, which may be off by a little."""
    return (x.abs() * 2.0 ** -4).clamp(min=2.0 ** -10)


def layout(rows, ctx, block, seed=0, lead=0, tail=0, spare=3):
    """Requests of rows[i] rows and ctx[i] tokens in a random set of blocks. lead / tail:
    rows of no request before and behind the requests' own."""
    g = torch.Generator().manual_seed(seed)
    pages = [-(-c // block) for c in ctx]
    nb = sum(pages) + spare
    perm = torch.randperm(nb, generator=g).to(torch.int32)
    bt = torch.full((len(ctx), max(pages + [1]) + 1), -1, dtype=torch.int32)
    at = 0
    for i, n in enumerate(pages):
        bt[i, :n] = perm[at:at + n]
        at += n
    rb = [lead]
    for n in rows:
        rb.append(rb[-1] + n)
    return SimpleNamespace(bt=bt, ctx=torch.tensor(ctx, dtype=torch.int32), nb=nb, P=block, gen=g,
                           rb=torch.tensor(rb, dtype=torch.int32), rows=list(rows),
                           total=rb[-1] + tail, max_rows=max(list(rows) + [1]), bs=len(ctx))


def places(p, i, lo, hi):
    """Pool rows of slots lo .. hi of request i."""
    t = torch.arange(lo, hi)
    return p.bt[i, t // p.P].long() * p.P + t % p.P


def slots(p):
    """(row, request, slot) of every row of a request."""
    return [(int(p.rb[i]) + j, i, int(p.ctx[i]) - n + j) for i, n in enumerate(p.rows) for j in range(n)]


# ------------------------------------------------------------------ rotary

def rotate(x, positions, inv_freq, begin=0, interleaved=False, scale=1.0):
    """x [rows, heads, D] in 64 bits, and the bound of an fp32 kernel's error."""
    half = inv_freq.numel()
    i = torch.arange(half)
    a, b = (begin + 2 * i, begin + 2 * i + 1) if interleaved else (begin + i, begin + half + i)
    th = positions.double()[:, None, None] * inv_freq
    c, s = th.cos() * scale, th.sin() * scale
    y, e = x.clone(), torch.zeros_like(x)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., b] * c + x[..., a] * s
    e[..., a] = e[..., b] = (x[..., a].abs() + x[..., b].abs()) * abs(scale) * 2.0 ** -20
    return y, e


def norm(x, kind, weight, bias, eps):
    """Normalised rows in 64 bits and the bound of an fp32 kernel's error: mean and variance
    of n values are sums of at most 16 + 5 roundings, 2^-19 of the largest value; then a
    reciprocal root and three roundings."""
    if kind == 0:
        return x, torch.zeros_like(x)
    w = torch.ones(x.shape[-1], dtype=torch.float64) if weight is None else weight.double()
    b = torch.zeros(x.shape[-1], dtype=torch.float64) if bias is None else bias.double()
    top = x.abs().amax(-1, keepdim=True)
    if kind == 1:
        x = x - x.mean(-1, keepdim=True)
    f = 1.0 / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    y = x * f * w
    return y + b, top * f * w.abs() * 2.0 ** -18 + y.abs() * 2.0 ** -19 + b.abs() * 2.0 ** -23


def coded(y, e, inv):
    """What a value y known to e becomes as a code times its scale 1 / inv: bounds of the code's
    value, in 64 bits."""
    x = (y * inv).clamp(-448.0, 448.0)
    return x, half_step(x.abs() + e * inv) + e * inv + x.abs() * 2.0 ** -22


# ------------------------------------------------------------------ attention

def attention_problem(rows, ctx, heads, block, seed=0, poison=True, **kw):
    """poison: NaN in every slot that no request holds."""
    p = layout(rows, ctx, block, seed, **kw)
    x = torch.randn((p.nb * block, LATENT), generator=p.gen) * torch.exp2(0.5 * torch.randn((1, LATENT), generator=p.gen))
    p.kv_scale, p.q_scale, p.sm = 0.03, 0.05, 192 ** -0.5
    code = (x / p.kv_scale).clamp(-448, 448).to(F8).view(torch.uint8)
    if poison:
        held = torch.zeros(p.nb * block, dtype=torch.bool)
        for i, c in enumerate(ctx):
            held[places(p, i, 0, c)] = True
        code[~held] = NAN8
    p.kv = code.reshape(p.nb, block, LATENT)
    q = torch.randn((p.total, heads, LATENT), generator=p.gen) * torch.exp2(0.5 * torch.randn((1, heads, LATENT), generator=p.gen))
    p.q = (q / p.q_scale).clamp(-448, 448).to(F8).view(torch.uint8)
    p.heads = heads
    return p


def attention(p, leave=None):
    """(out, lse) in 64 bits and their bounds. Rows of no request are NaN. leave: (request, slot)
    pairs that no row attends to.

    A score's error: fp32 sums of 576 exact products, one unit of 2^-23 of their absolute
    sum each, and its scaling. A weight, in a unit in which the row's largest is at least 1,
    as an e4m3 term, off by 2^-4 of the weight, or by 2^-10 below 2^-6, and a term for that
    remainder: e4m3 of 16 times it with up to 32 packed rows (query tokens x heads), off by 2^-4
    of the remainder, 2^-8 of the weight, or by 2^-10 / 16 = 2^-14; e5m2 with more, off by 2^-3 of
    it, 2^-7 of the weight or 2^-13 (a remainder of at most 2^-10). Through f16, 2^-11. exp2
    and the sums in fp32: 2^-18. The result is rounded to bf16."""
    few = min(p.max_rows, p.total) * p.heads <= 32
    part, floor = (2.0 ** -8, 2.0 ** -14) if few else (2.0 ** -7, 2.0 ** -13)
    out = torch.full((p.total, p.heads, VALUES), math.nan, dtype=torch.float64)
    lse = torch.full((p.total, p.heads), math.nan, dtype=torch.float64)
    tol, ltol = torch.zeros_like(out), torch.zeros_like(lse)
    pool = value(p.kv.reshape(-1, LATENT)) * p.kv_scale
    q = value(p.q) * p.q_scale
    for i, n in enumerate(p.rows):
        c, r0 = int(p.ctx[i]), int(p.rb[i])
        if n == 0:
            continue
        k = pool[places(p, i, 0, c)]
        x = q[r0:r0 + n].reshape(n * p.heads, LATENT)
        s = (x @ k.T * p.sm).reshape(n, p.heads, c)
        mag = (x.abs() @ k.abs().T * abs(p.sm)).reshape(n, p.heads, c)
        seen = torch.arange(c)[None, :] <= c - n + torch.arange(n)[:, None]
        if leave:
            for j, t in leave:
                if j == i:
                    seen[:, t] = False
        s = s.masked_fill(~seen[:, None], -math.inf)
        d = (mag * 580 * 2.0 ** -23 + s.abs() * 2.0 ** -20 + 2.0 ** -18).masked_fill(~seen[:, None], 0.0)
        l = torch.logsumexp(s, -1) if c else torch.full((n, p.heads), -math.inf, dtype=torch.float64)
        w = torch.where(seen[:, None], (s - l[..., None]).exp(), torch.zeros_like(s))
        v = k[:, :VALUES]
        # a token that a row does not see takes no part, whatever it holds
        v0 = torch.where(v.isnan(), torch.zeros_like(v), v)
        o = (w.reshape(n * p.heads, c) @ v0).reshape(n, p.heads, VALUES)
        dtop = d.amax(-1, keepdim=True) if c else torch.zeros((n, p.heads, 1), dtype=torch.float64)
        e = w * (part + 2.0 ** -11 + d + dtop)
        if c:
            e = e + torch.where(seen[:, None], w.amax(-1, keepdim=True) * floor, torch.zeros_like(w))
        e = (e.nan_to_num(0.0).reshape(n * p.heads, c) @ v0.abs()).reshape(n, p.heads, VALUES)
        none = ~seen.any(-1)
        o[none], l[none] = 0.0, -math.inf
        out[r0:r0 + n], lse[r0:r0 + n] = o, l
        tol[r0:r0 + n] = e + (o.abs() + e) * 2.0 ** -8
        ltol[r0:r0 + n] = dtop[..., 0] + l.abs().nan_to_num(0.0, 0.0, 0.0) * 2.0 ** -21 + 2.0 ** -18
    return out, lse, tol, ltol
