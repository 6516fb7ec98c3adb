"""Values of the cache operators inside bounds that stay a small part of them."""

import pytest
import torch

from tests import cache_bounds as cb
from tests import cache_ref as ref
from tests.test_gpu_cache import cuda, status_is
from tests.test_gpu_cache_paths import attend

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------- long contexts

LONG = [
    # rows, ctx, kv_heads, group, head_dim, block
    ([2], [20000], 1, 4, 64, 64),
    ([1], [60000], 1, 8, 128, 64),
    ([1, 2], [30000, 9000], 2, 12, 128, 48),
    ([40], [5000], 1, 1, 128, 64),
    ([5, 1, 5], [3100, 700, 2049], 2, 8, 64, 48),
    ([9, 12], [9000, 12345], 1, 6, 128, 24),
]


@pytest.mark.parametrize("flat", [False, True])
@pytest.mark.parametrize("case", LONG)
def test_values_of_long_contexts(cuda_lib, case, flat):
    rows, ctx, H, G, D, P = case
    p = ref.make(rows, ctx, kv_heads=H, group=G, head_dim=D, block=P, seed=41)
    if flat:
        p.q *= 0.125  # every token has some of the weight: a lost part shows
    ws = cuda_lib.cache_workspace()
    out, lse = attend(cuda_lib, p, ws=ws)
    status_is(cuda_lib, ws)
    cb.matches(p, out, lse)


# ------------------------------------------------------------- blocks left out

@pytest.mark.parametrize("rows,ctx,bad", [
    ([60, 1], [150, 20], 1),           # many rows, uncut or in few pieces
    ([50, 40], [3000, 2500], 40),      # cut over the SMs
    ([33] * 150, [70] * 150, 0),       # more row blocks than SMs
    ([2, 1], [150, 20], 2),            # few rows
    ([1], [4000], 60),                 # few rows, cut
])
def test_tokens_of_a_bad_block_take_no_part(cuda_lib, rows, ctx, bad):
    """Their weight is in no sum: not as tokens of score 0 either."""
    p = ref.make(rows, ctx, kv_heads=2, group=1, head_dim=128, block=32, seed=42, poison=False)
    ws = cuda_lib.cache_workspace()
    d = cuda(p)
    d[4] = d[4].clone()
    d[4][0, bad] = p.kc.shape[0]
    gone = torch.zeros((p.bs, p.bt.shape[1] * 32), dtype=torch.bool)
    gone[0, 32 * bad:32 * bad + 32] = True
    out, lse = attend(cuda_lib, p, d, ws)
    status_is(cuda_lib, ws, cuda_lib.PMQA_DEV_BAD_BLOCK_ID)
    cb.matches(p, out, lse, gone=gone)


# ------------------------------------------------------------- queries with a large channel

def large_channel(rows, ctx, D, power, seed):
    """Queries with one channel of 2^power that meets zeros, the others 1 to 2 with all
    eight bits of their significands in use, and keys of 1 and -1: every product and
    sum of products is exact in fp32."""
    p = ref.make(rows, ctx, kv_heads=2, group=2, head_dim=D, block=16, seed=seed, poison=False)
    g = p.gen
    p.kc = torch.where(torch.rand(p.kc.shape, generator=g) < 0.5, 0x38, 0xB8).to(torch.uint8)
    p.kc[..., 5] = 0
    p.ks = torch.ones_like(p.ks)
    sign = torch.where(torch.rand(p.q.shape, generator=g) < 0.5, 1.0, -1.0)
    q = sign * (128 + torch.randint(0, 128, p.q.shape, generator=g)) / 128.0
    q[..., 5] = 2.0 ** power
    p.q = q.to(torch.bfloat16)
    assert torch.equal(p.q.float(), q)
    return p


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows", [2, 40])
@pytest.mark.parametrize("power,split", [(6, 0.0), (10, 0.0), (13, 0.0), (16, 2.0 ** -21)])
def test_queries_with_a_large_channel(cuda_lib, rows, D, power, split):
    """Values of 2^-13 of their row's largest and more keep every bit, for many rows as
    for few; smaller ones are off by 2^-21 of it at most."""
    p = large_channel([rows, 1], [rows + 70, 40], D, power, seed=43)
    split = split if rows == 40 else 0.0
    ws = cuda_lib.cache_workspace()
    out, lse = attend(cuda_lib, p, ws=ws)
    cb.matches(p, out, lse, split=split)
    mass = cuda_lib.pmqa_cache_weigh(p.q.cuda(), *[t.cuda() for t in (p.kc, p.ks, p.bt, p.ctx, p.rb)],
                                     p.max_rows, p.sm, lse, ws=ws)
    want, tol = cb.weigh(p, lse.cpu(), torch.zeros(mass.shape), split=split)
    held = ~torch.isnan(want)
    over = (mass.double().cpu()[held] - want[held]).abs() - tol[held]
    assert float(over.max()) <= 0.0, float(over.max())
    status_is(cuda_lib, ws)


# ------------------------------------------------------------- scales far apart

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("power", [-12, -20, -25, -28, -32])
@pytest.mark.parametrize("scales", ["pow2", "any"])
def test_value_scales_far_apart(cuda_lib, scales, power, D):
    """The last block's values are 2^-power times as large as the others': rows that do
    not see it keep theirs, to 2^-31 of the largest scale."""
    p = ref.make([40], [304], kv_heads=2, group=1, head_dim=D, block=16, seed=44, poison=False,
                 scales=scales)
    p.vs[p.bt[0, :18].long()] *= 2.0 ** power
    ws = cuda_lib.cache_workspace()
    out, lse = attend(cuda_lib, p, ws=ws)
    status_is(cuda_lib, ws)
    want, _, tol, _, _ = cb.attention(p)
    assert float((tol[:24] / want[:24].abs().mean()).max()) < 0.5  # the bound says something
    cb.matches(p, out, lse)
