"""The bounds that long contexts are checked with: they agree with the plain form,
they are a small part of the outputs, and results with a part lost, counted twice
or left out lie outside them (mistakes planted in the plain form)."""

import math

import pytest
import torch

from tests import cache_bounds as cb
from tests import cache_ref as ref

LONG = [
    # rows, ctx, kv_heads, group, head_dim, block
    ([2], [20000], 1, 4, 64, 64),
    ([40], [5000], 1, 1, 128, 64),
    ([5, 1], [3100, 2049], 2, 8, 64, 48),
    ([1], [60000], 1, 8, 128, 64),
]


def make(case, **kw):
    rows, ctx, H, G, D, P = case
    return ref.make(rows, ctx, kv_heads=H, group=G, head_dim=D, block=P, poison=False, **kw)


@pytest.mark.parametrize("case", LONG)
def test_bounds_are_a_small_part_of_the_output(case):
    p = make(case, seed=31)
    out, lse, tol, ltol, rms = cb.attention(p)
    want, want_l, _, _ = ref.attention(p)
    torch.testing.assert_close(out, want)
    torch.testing.assert_close(lse, want_l)
    size = cb.root_mean_square(out)
    assert cb.root_mean_square(tol) < 0.06 * size
    assert cb.root_mean_square(rms) < 0.01 * size
    assert float(ltol.max()) < 2e-3
    cb.matches(p, out.to(torch.bfloat16), lse.float())


def refused(p, out, lse, **kw):
    try:
        cb.matches(p, out.to(torch.bfloat16), lse.float(), **kw)
    except AssertionError:
        return True
    return False


@pytest.mark.parametrize("case", LONG)
def test_a_lost_part_lies_outside_the_bounds(case):
    """The values of some tokens missing from `out`, or there twice, with the sums (and
    lse) as they should be: what a wrong join of cut contexts would give."""
    p = make(case, seed=32)
    p.q *= 0.125  # every token has some of the weight
    out, lse, _, _, rms = cb.attention(p)
    assert cb.root_mean_square(rms) < 0.01 * cb.root_mean_square(out)
    assert not refused(p, out, lse)
    assert refused(p, torch.zeros_like(out), lse)
    c = int(p.ctx[0])
    for a, b in ((0, c // 10), (c // 2, c // 2 + 128), (c - 300, c - 200)):
        kept = p.vc.clone()
        for t in range(a, b):
            p.vc[p.bt[0, t // p.P], :, t % p.P] = 0
        less = cb.attention(p)[0]
        p.vc = kept
        assert refused(p, less, lse)
        assert refused(p, 2 * out - less, lse)


def test_left_out_tokens():
    """Tokens of a block that is left out: the others' slots stay what they are."""
    p = make(([3], [50], 1, 2, 64, 16), seed=33)
    gone = torch.zeros((1, 64), dtype=torch.bool)
    gone[0, 16:32] = True
    out, lse, _, _, _ = cb.attention(p, gone=gone)
    k, _ = ref.tokens(p.kc, p.ks, p.bt, 0, 50, 16)
    v, _ = ref.tokens(p.vc, p.vs, p.bt, 0, 50, 16)
    for j in range(3):
        seen = [t for t in range(48 + j) if not 16 <= t < 32]
        for g in range(2):
            s = (k[0, seen] @ p.q[j, g].double()) * p.sm
            torch.testing.assert_close(out[j, g], torch.softmax(s, 0) @ v[0, seen])
            torch.testing.assert_close(lse[j, g], torch.logsumexp(s, 0))
    # counted with score 0 and no value, as zero-filled tokens would be, they show
    full = torch.logaddexp(lse, torch.full_like(lse, math.log(16.0)))
    assert not refused(p, out, lse, gone=gone)
    assert refused(p, out * (lse - full).exp()[..., None], full, gone=gone)
