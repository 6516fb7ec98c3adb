"""Plain 64-bit attention on the 8-bit K/V cache with bounds that stay a small
part of the outputs at any context length, and with tokens that may be left
out (torch on the CPU). Beside the bounds of each value there is one of the
root mean square of their errors, in which independent roundings add up as
squares."""

import math

import torch

from tests import cache_ref as ref


def _tokens(p, code, scale, i, there):
    """The cached tokens of request i and their scales, zeros where one is left out."""
    x, s = ref.tokens(code, scale, p.bt.clamp(0, code.shape[0] - 1), i, int(p.ctx[i]), p.P)
    return (torch.where(there[None, :, None], x, torch.zeros_like(x)),
            torch.where(there[None, :], s, torch.zeros_like(s)))


def _scores(p, i, there, split):
    """Scores of request i, fp64 [H, G, n, c], a bound of their errors, and the tokens
    that a row does not see (-inf, no error)."""
    n, c, r0 = p.rows[i], int(p.ctx[i]), int(p.rb[i])
    q = p.q[r0:r0 + n].double().reshape(n, p.H, p.G, p.D)
    k, _ = _tokens(p, p.kc, p.ks, i, there)
    s = torch.einsum("nhgd,htd->hgnt", q, k) * p.sm
    mag = torch.einsum("nhgd,htd->hgnt", q.abs(), k.abs()) * abs(p.sm)
    top = torch.einsum("nhg,ht->hgnt", q.abs().amax(-1), k.abs().sum(-1)) * abs(p.sm)
    # D products summed in fp32 in any order, three fp32 multiplications of the
    # sum, and what q loses of its row's largest value
    err = mag * (p.D + 4) * 2.0 ** -23 + top * split
    hidden = (torch.arange(c)[None, :] > c - n + torch.arange(n)[:, None]) | ~there[None, :]
    return s.masked_fill(hidden, -math.inf), err.masked_fill(hidden, 0.0), hidden


def attention(p, gone=None, split=2.0 ** -21):
    """(out, lse, bound of out, bound of lse, bound of out's rms error) of every
    row of a request; the rows of none are NaN. gone: bool [bs, slots], tokens that
    take no part. split: what q may lose of its row's largest value.

    A weight p = 2^(x - m) is rounded to f16: off by 2^-11 of itself, or by 2^-25
    where that is more. m is a score of the row, not above its largest one, so
    that with the weights' sum l the step of a weight p / l is 2^-25 / l <= 2^-25
    e^(largest score - lse). Where few rows share a tile, p is multiplied by its
    token's scale over one that is at most 32 times the largest among 32 tokens, and
    the step is that scale's; where many do, the values are, over the largest scale
    so far: off by 2^-11 of themselves, or by 2^-31 of that scale where that is more."""
    total, Hq = p.q.shape[0], p.H * p.G
    out = torch.full((total, Hq, p.D), math.nan, dtype=torch.float64)
    lse = torch.full((total, Hq), math.nan, dtype=torch.float64)
    tol, rms, ltol = out.clone(), out.clone(), lse.clone()
    for i in range(p.bs):
        n, c, r0 = p.rows[i], int(p.ctx[i]), int(p.rb[i])
        if n == 0:
            continue
        where = slice(r0, r0 + n)
        if c == 0:
            out[where], tol[where], rms[where] = 0.0, 0.0, 0.0
            lse[where], ltol[where] = -math.inf, 0.0
            continue
        there = torch.ones(c, dtype=torch.bool) if gone is None else ~gone[i, :c]
        s, err, hidden = _scores(p, i, there, split)
        v, vs = _tokens(p, p.vc, p.vs, i, there)
        l = torch.logsumexp(s, -1)
        some = ~torch.isinf(l)
        w = torch.where(some[..., None], (s - l[..., None]).exp(), torch.zeros_like(s))
        high = torch.where(some, (s.amax(-1) - l).exp(), torch.zeros_like(l))  # 1 / l at most
        o = torch.einsum("hgnt,htd->nhgd", w, v)
        few = n * p.G <= 32
        # the weights' relative error: their own rounding (2^-11) and, of many rows, the
        # values', their score's, and that of the exponential and its argument (|x| < 2^6)
        rel = (2.0 ** -11 if few else 2.0 ** -10) + 2.0 * (err + 2.0 ** -18)
        if few:
            near = torch.nn.functional.pad(vs.abs(), (0, -c % 32)).reshape(p.H, -1, 32)
            near = near.amax(-1).repeat_interleave(32, 1)[:, :c]  # the largest of its 32 tokens
            step = 2.0 ** -25 * 32.0 * (near / torch.where(there, vs.abs(), 1.0)).clamp(min=1.0)
            low = torch.zeros_like(vs)
        else:
            step = torch.full_like(vs, 2.0 ** -25)
            low = 2.0 ** -31 * vs.abs().amax(-1, keepdim=True).expand_as(vs)
        each = w * rel + ~hidden * high[..., None] * step[:, None, None]
        half = o.abs() * 2.0 ** -8
        # and the sums in fp32, 16 tokens a product: of all of them one behind the other,
        # or of each quarter and then of the parts (of 128 tokens or more)
        sums = c / 64 + c / 128 + 8 if few else c / 16 + 8
        body = torch.einsum("hgnt,htd->nhgd", each + w * sums * 2.0 ** -23, v.abs())
        body += torch.einsum("hgnt,ht->nhg", w, low)[..., None]
        square = torch.einsum("hgnt,htd->nhgd", each ** 2, v ** 2)
        square += torch.einsum("hgnt,ht->nhg", w ** 2, low ** 2)[..., None]
        out[where] = o.reshape(n, Hq, p.D)
        tol[where] = (half + body).reshape(n, Hq, p.D)
        rms[where] = (half ** 2 + square).sqrt().reshape(n, Hq, p.D)
        lse[where] = l.permute(2, 0, 1).reshape(n, Hq)
        # lse: the weighted mean of the scores' errors, the sum of the weights, and
        # the logarithm and its product with ln 2
        e = (w * err).sum(-1) + 2.0 ** -18 + torch.where(some, l.abs(), torch.zeros_like(l)) * 2.0 ** -21
        ltol[where] = torch.where(some, e, torch.zeros_like(e)).permute(2, 0, 1).reshape(n, Hq)
    return out, lse, tol, ltol, rms


def weigh(p, lse, mass_in, split=2.0 ** -21):
    """(mass_out, bound) of cached tokens; the others NaN."""
    out = torch.full(mass_in.shape, math.nan, dtype=torch.float64)
    tol = torch.zeros_like(out)
    for i in range(p.bs):
        n, c, r0 = p.rows[i], int(p.ctx[i]), int(p.rb[i])
        out[i, :, :c] = mass_in[i, :, :c].double()
        if n == 0 or c == 0:
            continue
        s, err, _ = _scores(p, i, torch.ones(c, dtype=torch.bool), split)
        l = lse[r0:r0 + n].double().reshape(n, p.H, p.G).permute(1, 2, 0)[..., None]
        w = torch.where(torch.isinf(s), torch.zeros_like(s), (s - l).exp())
        # the score's error, the exponential and its argument, lse in base 2, the sum
        d = w * (err + 2.0 ** -18 + l.abs() * 2.0 ** -22)
        out[i, :, :c] += w.sum((1, 2))
        tol[i, :, :c] = d.sum((1, 2)) + out[i, :, :c].abs() * (n * p.G + 2) * 2.0 ** -24
    return out, tol


def root_mean_square(x: torch.Tensor) -> float:
    return float(x.double().square().mean().sqrt())


def matches(p, got, lse, **kw):
    """Every row of a request within its bounds, and their errors together."""
    want, want_l, tol, ltol, rms = attention(p, **kw)
    r0, r1 = int(p.rb[0]), int(p.rb[-1])
    d = got.double().cpu()[r0:r1] - want[r0:r1]
    over = d.abs() - tol[r0:r1]
    assert float(over.max()) <= 0.0, float(over.max())
    assert root_mean_square(d) <= root_mean_square(rms[r0:r1])
    w, g = want_l[r0:r1], lse.double().cpu()[r0:r1]
    inf = torch.isinf(w)
    assert torch.equal(g[inf], w[inf])
    over = (g[~inf] - w[~inf]).abs() - ltol[r0:r1][~inf]
    assert over.numel() == 0 or float(over.max()) <= 0.0, float(over.max())
