"""The operators on the 8-bit K/V cache against their plain 64-bit forms."""

import math

import pytest
import torch

from tests import cache_ref as ref

pytestmark = pytest.mark.gpu

# rows, ctx, kv_heads, group, head_dim, block
SHAPES = [
    ("one_token", [1], [1], 1, 1, 128, 1),
    ("single", [1], [500], 8, 4, 128, 16),
    ("group8", [1, 1, 1], [129, 1, 300], 2, 8, 128, 64),
    ("empty_context", [1, 1, 0, 1], [0, 65, 40, 64], 2, 4, 128, 64),
    ("verify", [4, 4], [203, 70], 2, 8, 128, 64),
    ("verify_before_slot_0", [4, 3], [2, 3], 2, 3, 128, 8),
    ("multi_head", [1, 2], [77, 140], 5, 1, 64, 24),
    ("odd_group", [2, 1, 3], [100, 33, 260], 3, 5, 64, 48),
    ("wide_group", [1, 1], [190, 517], 1, 32, 128, 128),
    ("widest_group", [1, 2], [90, 200], 1, 128, 128, 32),
    ("narrow_pages", [1, 3], [19, 133], 2, 2, 128, 1),
    ("odd_pages", [2, 1], [64, 211], 1, 6, 64, 5),
    ("big_pages", [1, 1], [700, 1100], 1, 4, 128, 1024),
    ("prompt", [70], [70], 2, 4, 128, 64),
    ("chunks", [130, 37, 200], [300, 37, 513], 2, 4, 128, 64),
    ("mixed", [90, 1, 1, 0, 150, 1], [400, 17, 260, 30, 150, 129], 3, 3, 64, 48),
    ("mixed_odd", [61, 1, 2], [61, 500, 300], 1, 7, 128, 24),
    ("many", [1] * 200, [(37 * i) % 150 for i in range(200)], 1, 4, 64, 16),
]
IDS = [s[0] for s in SHAPES]


def problem(shape, **kw):
    _, rows, ctx, H, G, D, P = shape
    return ref.make(rows, ctx, kv_heads=H, group=G, head_dim=D, block=P, **kw)


def cuda(p):
    return [t.cuda() for t in (p.kc, p.vc, p.ks, p.vs, p.bt, p.ctx)]


def status_is(lib, ws, want=0):
    assert lib.pmqa_read_device_status(ws) == want


def check(got, want, tol):
    """Within tolerance everywhere, NaN exactly where the reference has it."""
    got = got.double()
    assert torch.equal(torch.isnan(got), torch.isnan(want))
    fin = torch.isfinite(want)
    assert torch.equal(got[~fin & ~torch.isnan(want)], want[~fin & ~torch.isnan(want)])
    over = (got[fin] - want[fin]).abs() - tol[fin]
    assert over.numel() == 0 or float(over.max()) <= 0.0, float(over.max())


def expects_drop(p):
    return any(n > c for n, c in zip(p.rows, p.ctx.tolist()))


@pytest.mark.parametrize("scales", ["pow2", "any"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_attention(cuda_lib, shape, scales):
    p = problem(shape, seed=3, lead=2, tail=3, scales=scales)
    ws = cuda_lib.cache_workspace()
    q = p.q.cuda()
    out = torch.full_like(q, math.nan)
    lse = torch.full(q.shape[:2], math.nan, device="cuda")
    got, got_l = cuda_lib.pmqa_cache_attention(q, *cuda(p), p.rb.cuda(), p.max_rows, p.sm, out=out,
                                               lse=lse, ws=ws)
    status_is(cuda_lib, ws)
    want, want_l, tol, ltol = ref.attention(p)
    check(got.cpu(), want, tol)
    check(got_l.cpu(), want_l, ltol)


@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_weigh(cuda_lib, shape):
    p = problem(shape, seed=4, lead=1, tail=2)
    _, lse, _, _ = ref.attention(p)
    lse = lse.float()
    width = p.bt.shape[1] * p.P
    mass = torch.rand((p.bs, p.H, width), generator=p.gen)
    want, tol = ref.weigh(p, lse, mass)
    kc, _, ks, _, bt, ctx = cuda(p)
    ws = cuda_lib.cache_workspace()
    args = (p.q.cuda(), kc, ks, bt, ctx, p.rb.cuda(), p.max_rows, p.sm, lse.cuda())
    out = torch.full(mass.shape, math.nan, device="cuda")
    cuda_lib.pmqa_cache_weigh(*args, mass.cuda(), mass_out=out, ws=ws)
    status_is(cuda_lib, ws)
    check(out.cpu(), want, tol)
    # in place: the same sums, other entries kept
    there = mass.cuda()
    cuda_lib.pmqa_cache_weigh(*args, there, mass_out=there, ws=ws)
    held = ~torch.isnan(want)
    assert torch.equal(there.cpu()[held], out.cpu()[held])
    assert torch.equal(there.cpu()[~held], mass[~held])
    # without earlier masses
    fresh = cuda_lib.pmqa_cache_weigh(*args, ws=ws)
    want0, tol0 = ref.weigh(p, lse, torch.zeros_like(mass))
    check(fresh.cpu(), want0.nan_to_num(0.0), tol0)


@pytest.mark.parametrize("scales", ["pow2", "any"])
@pytest.mark.parametrize("shape", SHAPES, ids=IDS)
def test_append(cuda_lib, shape, scales):
    p = problem(shape, seed=5, lead=2, tail=1, scales=scales)
    r0 = int(p.rb[0])
    if p.rows[0] and int(p.ctx[0]):
        last = r0 + p.rows[0] - 1
        p.k_new[last, 0, :4] = torch.tensor([math.nan, math.inf, -math.inf, 0.0])
        p.v_new[last] = 0.0
        p.k_new[last, -1] *= 200.0  # makes the block's scale grow
    want = ref.append(p)
    d = cuda(p)
    ws = cuda_lib.cache_workspace()
    cuda_lib.pmqa_cache_append(p.k_new.cuda(), p.v_new.cuda(), *d, p.rb.cuda(), p.max_rows, ws=ws)
    status_is(cuda_lib, ws, cuda_lib.PMQA_DEV_BAD_CONTEXT if expects_drop(p) else 0)
    for got, w in zip((d[0], d[2], d[1], d[3]), want):
        g = got.cpu()
        if w.dtype == torch.uint8:
            # both signs of NaN are NaN
            g, w = g.clone(), w.clone()
            g[g == 0xFF], w[w == 0xFF] = 0x7F, 0x7F
            assert torch.equal(g, w)
        else:
            assert torch.equal(g.nan_to_num(-1.0), w.nan_to_num(-1.0))


EVICT = [
    # ctx, kv_heads, head_dim, block, keep, sinks, recent
    ([1], 1, 128, 1, 1, 0, 0),
    ([100, 7, 0, 33], 2, 128, 16, 33, 2, 8),
    ([300, 129], 3, 64, 48, 100, 0, 0),
    ([300, 299], 1, 128, 64, 65, 30, 35),  # nothing left to choose
    ([700], 2, 64, 5, 64, 4, 0),
    ([1500, 40], 1, 128, 128, 512, 4, 64),
    ([2600], 1, 64, 1024, 1030, 0, 7),
    ([9000], 2, 64, 64, 200, 3, 5),
]


@pytest.mark.parametrize("kind", ["random", "ties", "odd"])
@pytest.mark.parametrize("case", EVICT)
def test_evict(cuda_lib, case, kind):
    ctx, H, D, P, keep, sinks, recent = case
    per = -(-keep // P)
    p = ref.make([1] * len(ctx), ctx, kv_heads=H, group=1, head_dim=D, block=P, seed=6,
                 spare=per * len(ctx) + 2, scales="any" if kind == "odd" else "pow2")
    width = max(ctx) + 3
    mass = torch.exp2(torch.randn((len(ctx), H, width), generator=p.gen) * 3)
    if kind == "ties":
        mass = (mass * 2).floor().clamp(max=2.0)  # three values only
        mass[:, :, ::5] = -0.0
    if kind == "odd":
        mass -= 1.0
        mass[:, :, ::7] = math.nan
        mass[:, :, 1::11] = math.inf
        mass[:, :, 2::11] = -math.inf
    new = p.free[:per * len(ctx)].reshape(len(ctx), per).contiguous()
    want = ref.evict(p, mass, keep, sinks, recent, new)
    d = cuda(p)
    ws = cuda_lib.cache_workspace()
    kept, lens, mout = cuda_lib.pmqa_cache_evict(*d, mass.cuda(), keep, sinks, recent, new.cuda(),
                                                 ws=ws)
    status_is(cuda_lib, ws)
    assert torch.equal(kept.cpu(), want[0])
    assert torch.equal(lens.cpu(), want[1])
    assert torch.equal(mout.cpu().nan_to_num(-5.0), want[2].nan_to_num(-5.0))
    for got, w in zip((d[0], d[2], d[1], d[3]), want[3:]):
        g = got.cpu()
        assert torch.equal(g, w) if w.dtype == torch.uint8 else \
            torch.equal(g.nan_to_num(-1.0), w.nan_to_num(-1.0))
