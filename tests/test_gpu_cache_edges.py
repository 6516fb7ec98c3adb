"""Inputs at the edges of what the cache operators' documentation allows: lengths and
rows past their arrays, requests without rows, the largest `keep`, streams."""

import math

import pytest
import torch

from tests import cache_ref as ref
from tests.test_gpu_cache import cuda, status_is
from tests.test_gpu_cache_paths import attend, matches

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------- rows past their arrays

def appended(lib, p, ctx, rb, max_rows):
    """Both pools and scales after an append with these lengths, and the status."""
    ws = lib.cache_workspace()
    d = cuda(p)
    d[5] = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    lib.pmqa_cache_append(p.k_new.cuda(), p.v_new.cuda(), *d,
                          torch.tensor(rb, dtype=torch.int32, device="cuda"), max_rows, ws=ws)
    return [d[i].cpu() for i in (0, 2, 1, 3)], lib.pmqa_read_device_status(ws)


def full_table(n, block):
    """Two requests, the first with all of its table's blocks in use, and n new rows."""
    p = ref.make([n, min(n, 2)], [4 * block, 30], kv_heads=2, group=1, head_dim=128, block=block,
                 seed=51, poison=False)
    p.bt = p.bt[:, :4].contiguous()
    return p


def only(p, runs):
    """Leave each request the `count` new rows from `first` on."""
    keep = torch.cat([torch.arange(first, first + count) for first, count in runs])
    p.k_new, p.v_new = p.k_new[keep], p.v_new[keep]
    p.rows = [count for _, count in runs]
    p.rb = torch.tensor([0, runs[0][1], runs[0][1] + runs[1][1]], dtype=torch.int32)


@pytest.mark.parametrize("n,block", [(1, 16), (3, 16), (150, 64), (40, 8)])
@pytest.mark.parametrize("past", [1, 2, 1000, 2 ** 31 - 1])
def test_rows_past_the_table_are_dropped(cuda_lib, n, block, past):
    """A length past the table: rows whose slots the table has go there, the others
    nowhere, and no earlier token is overwritten."""
    p = full_table(n, block)
    cap = 4 * block
    ctx = min(cap + past, 2 ** 31 - 1)
    got, status = appended(cuda_lib, p, [ctx, 30], p.rb.tolist(), n)
    assert status == cuda_lib.PMQA_DEV_BAD_CONTEXT
    kept = max(0, n - (ctx - cap))
    p.ctx = torch.tensor([cap if kept else 0, 30], dtype=torch.int32)
    only(p, [(0, kept), (n, p.rows[1])])
    for g, w in zip(got, ref.append(p)):
        assert torch.equal(g, w)


@pytest.mark.parametrize("max_rows", [1, 2, 100])
def test_rows_past_max_rows_are_dropped(cuda_lib, max_rows):
    """More rows than max_rows: the first ones go to their own slots."""
    n, ctx = 130, 250
    p = full_table(n, 64)
    got, status = appended(cuda_lib, p, [ctx, 30], p.rb.tolist(), max_rows)
    assert status == cuda_lib.PMQA_DEV_BAD_CONTEXT
    m1, m2 = min(n, max_rows), min(2, max_rows)
    p.ctx = torch.tensor([ctx - n + m1, 30 - 2 + m2], dtype=torch.int32)
    only(p, [(0, m1), (n, m2)])
    for g, w in zip(got, ref.append(p)):
        assert torch.equal(g, w)


@pytest.mark.parametrize("max_rows", [1, 40])
def test_rows_outside_the_call_are_dropped(cuda_lib, max_rows):
    """row_begin outside [0, rows]: rows that exist keep their slots."""
    # request 0 begins three rows before the first; request 1 ends past the last
    p = full_table(1, 16)
    got, status = appended(cuda_lib, p, [60, 30], [-3, 1, 60], max_rows)
    assert status == cuda_lib.PMQA_DEV_BAD_CONTEXT
    p.ctx = torch.tensor([60, 0], dtype=torch.int32)  # request 1's row would be slot 30 - 59
    only(p, [(0, 1), (1, 0)])
    for g, w in zip(got, ref.append(p)):
        assert torch.equal(g, w)
    p = full_table(3, 16)
    got, status = appended(cuda_lib, p, [60, 30], [0, 3, 8], max_rows)
    assert status == cuda_lib.PMQA_DEV_BAD_CONTEXT
    m = [min(3, max_rows), min(2, max_rows)]
    p.ctx = torch.tensor([60 - 3 + m[0], 30 - 5 + m[1]], dtype=torch.int32)
    only(p, [(0, m[0]), (3, m[1])])
    for g, w in zip(got, ref.append(p)):
        assert torch.equal(g, w)


@pytest.mark.parametrize("n", [1, 40])
def test_a_negative_length_appends_nothing(cuda_lib, n):
    p = full_table(n, 16)
    got, status = appended(cuda_lib, p, [-7, 30], p.rb.tolist(), max(n, 2))
    assert status == cuda_lib.PMQA_DEV_BAD_CONTEXT
    p.ctx = torch.tensor([0, 30], dtype=torch.int32)
    only(p, [(0, 0), (n, p.rows[1])])
    for g, w in zip(got, ref.append(p)):
        assert torch.equal(g, w)


# ------------------------------------------------------------- requests without rows

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,G", [(1, 4), (2, 8), (40, 1)])
@pytest.mark.parametrize("bad", ["codes", "scales", "both"])
def test_weigh_of_a_request_without_rows(cuda_lib, bad, n, G, D):
    """A sum over no rows adds nothing, whatever the cached keys are."""
    p = ref.make([0, n], [150, 100], kv_heads=2, group=G, head_dim=D, block=16, seed=52)
    if bad != "scales":
        p.kc[p.bt[0, :9].long()] = ref.NAN8
    if bad != "codes":
        p.ks[p.bt[0, :9].long()] = math.nan
    _, lse, _, _ = ref.attention(p)
    width = p.bt.shape[1] * 16
    mass = torch.rand((2, 2, width), generator=p.gen)
    kc, _, ks, _, bt, ctx = cuda(p)
    ws = cuda_lib.cache_workspace()
    args = (p.q.cuda(), kc, ks, bt, ctx, p.rb.cuda(), p.max_rows, p.sm, lse.float().cuda())
    got = cuda_lib.pmqa_cache_weigh(*args, mass.cuda(), mass_out=torch.zeros_like(mass).cuda(),
                                    ws=ws).cpu()
    fresh = cuda_lib.pmqa_cache_weigh(*args, ws=ws).cpu()
    status_is(cuda_lib, ws)
    assert torch.equal(got[0, :, :150], mass[0, :, :150]) and torch.all(got[0, :, 150:] == 0.0)
    assert torch.all(fresh[0] == 0.0)
    # a table entry outside the pool is still reported
    bt[0, 1] = -1
    got = cuda_lib.pmqa_cache_weigh(*args, mass.cuda(), ws=ws).cpu()
    status_is(cuda_lib, ws, cuda_lib.PMQA_DEV_BAD_BLOCK_ID)
    assert torch.equal(got[0], mass[0])


# ------------------------------------------------------------- clamps of requests without rows

@pytest.mark.parametrize("G", [2, 40])
@pytest.mark.parametrize("rows,ctx,rb", [
    ([0, 1], [10 ** 6, 30], [0, 0, 1]),   # a context past its table
    ([0, 1], [-1, 30], [0, 0, 1]),
    ([1, 0], [30, 20], [0, 1, 0]),        # row_begin falls
    ([1, 0], [30, 20], [0, 1, 9]),        # and runs past the rows
])
def test_clamps_are_reported_for_requests_without_rows(cuda_lib, rows, ctx, rb, G):
    """Whatever the heads per kv head: a request that no kernel works on is looked at."""
    p = ref.make(rows, [30, 30], kv_heads=1, group=G, head_dim=64, block=16, seed=53)
    ws = cuda_lib.cache_workspace()
    d = cuda(p)
    d[5] = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    out, lse = cuda_lib.pmqa_cache_attention(p.q.cuda(), *d, torch.tensor(rb, dtype=torch.int32).cuda(),
                                             1, p.sm, want_lse=True, ws=ws)
    status_is(cuda_lib, ws, cuda_lib.PMQA_DEV_BAD_CONTEXT)
    matches(p, out, lse)


@pytest.mark.parametrize("extra,H", [(100, 2), (200, 1)])
def test_clamps_are_reported_where_nothing_is_cut(cuda_lib, extra, H):
    """More row blocks than SMs, in order of length (up to 128 requests) or of rows."""
    p = ref.make([0] + [1] * extra, [30] * (1 + extra), kv_heads=H, group=40, head_dim=64, block=16,
                 seed=54)
    ws = cuda_lib.cache_workspace()
    d = cuda(p)
    d[5][0] = 10 ** 6
    out, lse = attend(cuda_lib, p, d, ws)
    status_is(cuda_lib, ws, cuda_lib.PMQA_DEV_BAD_CONTEXT)
    matches(p, out, lse)


@pytest.mark.parametrize("P", [1, 16])
def test_append_reports_rows_that_fall(cuda_lib, P):
    """row_begin that falls in the middle: that request has no rows, and is reported."""
    p = ref.make([5, 0, 1], [30, 30, 30], kv_heads=2, group=1, head_dim=64, block=P, seed=56,
                 poison=False)
    got, status = appended(cuda_lib, p, [30, 30, 30], [0, 5, 3, 4], 5)
    assert status == cuda_lib.PMQA_DEV_BAD_CONTEXT
    p.k_new[5], p.v_new[5] = p.k_new[3], p.v_new[3]
    for g, w in zip(got, ref.append(p)):
        assert torch.equal(g, w)


# ------------------------------------------------------------- the largest keep

def test_evict_with_the_largest_keep(cuda_lib):
    """keep = 2^31 - 1: nothing is dropped, everything moves."""
    keep, P, c = 2 ** 31 - 1, 1024, 1500
    p = ref.make([1], [c], kv_heads=1, group=1, head_dim=64, block=P, seed=55, spare=2, poison=False)
    new = torch.full((1, -(-keep // P)), -1, dtype=torch.int32)
    new[0, :2] = p.free[:2]
    mass = torch.rand((1, 1, c), generator=p.gen)
    d = cuda(p)
    ws = cuda_lib.cache_workspace()
    kept, lens, out = cuda_lib.pmqa_cache_evict(*d, mass.cuda(), keep, 4, 8, new.cuda(), ws=ws)
    status_is(cuda_lib, ws)
    assert int(lens[0]) == c and torch.equal(out.cpu(), mass)
    assert torch.equal(kept[0, 0, :c].cpu(), torch.arange(c, dtype=torch.int32))
    assert bool((kept[0, 0, c:] == -1).all())
    want = ref.evict(p, mass, c, 4, 8, new[:, :2])
    for got, w in zip((d[0], d[2], d[1], d[3]), want[3:]):
        assert torch.equal(got.cpu(), w)


# ------------------------------------------------------------- a workspace made on a stream

def test_a_workspace_made_on_a_stream_is_that_streams(cuda_lib):
    """Memory that the current stream still reads is not handed to another stream."""
    n = cuda_lib.pmqa_cache_workspace_bytes()
    side = torch.cuda.Stream()
    x = torch.full((n,), 7, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(50_000_000)  # about 25 ms on the current stream
    y = x + 0
    del x
    ws = cuda_lib.cache_workspace(stream=side)
    torch.cuda.synchronize()
    assert bool((y == 7).all())
    assert cuda_lib.pmqa_read_device_status(ws, stream=side) == 0


# ------------------------------------------------------------- sizes that no other test has

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("P", [1, 5, 7, 100, 1024])
def test_many_rows_with_blocks_of_any_size(cuda_lib, P, D):
    """Blocks that end inside a tile, one token long and longer than a tile."""
    p = ref.make([45, 300, 2], [333, 300, 150], kv_heads=2, group=2, head_dim=D, block=P, seed=57)
    ws = cuda_lib.cache_workspace()
    d = cuda(p)
    out, lse = attend(cuda_lib, p, d, ws)
    matches(p, out, lse)
    mass = cuda_lib.pmqa_cache_weigh(p.q.cuda(), d[0], d[2], d[4], d[5], p.rb.cuda(), p.max_rows, p.sm,
                                     lse, ws=ws).cpu()
    want, tol = ref.weigh(p, lse.cpu(), torch.zeros(mass.shape))
    held = ~torch.isnan(want)
    assert bool(((mass.double() - want).abs() <= tol)[held].all())
    status_is(cuda_lib, ws)


@pytest.mark.parametrize("rows", [1, 3, 80])
@pytest.mark.parametrize("width", [1, 70, 129])
def test_masses_narrower_than_the_context(cuda_lib, width, rows):
    """Tokens past mass_width are weighed by no one and written nowhere."""
    p = ref.make([rows, 1], [150, 60], kv_heads=2, group=4, head_dim=128, block=16, seed=58)
    _, lse, _, _ = ref.attention(p)
    mass = torch.rand((2, 2, width), generator=p.gen)
    wide = torch.rand((2, 2, 160), generator=p.gen)
    wide[..., :width] = mass
    kc, _, ks, _, bt, ctx = cuda(p)
    args = (p.q.cuda(), kc, ks, bt, ctx, p.rb.cuda(), p.max_rows, p.sm, lse.float().cuda())
    ws = cuda_lib.cache_workspace()
    got = cuda_lib.pmqa_cache_weigh(*args, mass.cuda(), ws=ws)
    full = cuda_lib.pmqa_cache_weigh(*args, wide.cuda(), ws=ws)
    assert torch.equal(got, full[..., :width])
    status_is(cuda_lib, ws)


@pytest.mark.parametrize("H,G", [(40, 1), (1, 24), (16, 8)])
def test_head_counts(cuda_lib, H, G):
    p = ref.make([1, 60, 3], [200, 140, 9], kv_heads=H, group=G, head_dim=64, block=32, seed=59)
    ws = cuda_lib.cache_workspace()
    out, lse = attend(cuda_lib, p, ws=ws)
    matches(p, out, lse)
    status_is(cuda_lib, ws)


def test_rows_of_no_request_may_hold_anything(cuda_lib):
    """NaN queries and new tokens in front of, between and behind the requests' rows."""
    p = ref.make([2, 50], [80, 90], kv_heads=2, group=4, head_dim=128, block=16, seed=60, lead=5,
                 tail=6, poison=False)
    for t in (p.q, p.k_new, p.v_new):
        t[:5], t[57:] = math.nan, math.nan
    want = ref.append(p)
    d = cuda(p)
    ws = cuda_lib.cache_workspace()
    cuda_lib.pmqa_cache_append(p.k_new.cuda(), p.v_new.cuda(), *d, p.rb.cuda(), 50, ws=ws)
    for g, w in zip((d[0], d[2], d[1], d[3]), want):
        assert torch.equal(g.cpu(), w)
    p.kc, p.ks, p.vc, p.vs = want
    out, lse = attend(cuda_lib, p, d, ws)
    matches(p, out, lse)
    status_is(cuda_lib, ws)


# ------------------------------------------------------------- infinite queries

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows,G", [(1, 4), (3, 8), (40, 1)])
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_an_infinite_query_makes_its_row_nan(cuda_lib, bad, rows, G, D):
    """For few rows as for many, also where every score would be -inf; no other row changes."""
    p = ref.make([rows, 1], [90, 40], kv_heads=2, group=G, head_dim=D, block=16, seed=61, poison=False)
    p.kc[..., 7] = 0xB8  # -1 for every token
    ws = cuda_lib.cache_workspace()
    d = cuda(p)
    out, lse = attend(cuda_lib, p, d, ws)
    args = (d[0], d[2], d[4], d[5], p.rb.cuda(), p.max_rows, p.sm)
    mass = cuda_lib.pmqa_cache_weigh(p.q.cuda(), *args, lse, ws=ws)
    j = rows - 1
    p.q[j, 0, 7] = bad
    got, got_l = attend(cuda_lib, p, d, ws)
    assert bool(torch.isnan(got[j, 0]).all()) and bool(torch.isnan(got_l[j, 0]))
    same = torch.ones(p.q.shape[:2], dtype=torch.bool)
    same[j, 0] = False
    assert torch.equal(got.cpu()[same], out.cpu()[same])
    assert torch.equal(got_l.cpu()[same], lse.cpu()[same])
    weighed = cuda_lib.pmqa_cache_weigh(p.q.cuda(), *args, lse, ws=ws)
    assert bool(torch.isnan(weighed[0, 0, :90]).all())
    assert torch.equal(weighed[0, 1], mass[0, 1]) and torch.equal(weighed[1], mass[1])
    status_is(cuda_lib, ws)
