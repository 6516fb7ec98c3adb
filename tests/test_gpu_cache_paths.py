"""How the operators on the 8-bit K/V cache are used together, and the inputs
that their documentation allows at the edges."""

import math

import pytest
import torch

from tests import cache_ref as ref
from tests.test_gpu_cache import check, cuda, status_is

pytestmark = pytest.mark.gpu


def attend(lib, p, d=None, ws=None, **kw):
    d = cuda(p) if d is None else d
    return lib.pmqa_cache_attention(p.q.cuda(), *d, p.rb.cuda(), p.max_rows, p.sm, want_lse=True,
                                    ws=ws, **kw)


def matches(p, got, lse):
    want, want_l, tol, ltol = ref.attention(p)
    r0, r1 = int(p.rb[0]), int(p.rb[-1])
    check(got.cpu()[r0:r1], want[r0:r1], tol[r0:r1])
    check(lse.cpu()[r0:r1], want_l[r0:r1], ltol[r0:r1])


@pytest.mark.parametrize("H,G,D,P", [(2, 4, 128, 16), (3, 2, 64, 5)])
def test_a_serving_run(cuda_lib, H, G, D, P):
    """Prompts written and attended to, weighed, evicted, then decode steps on
    what was kept, everything in one workspace on one stream."""
    lib = cuda_lib
    keep, steps = 48, 3
    n = [70, 41, 20]
    p = ref.make(n, n, kv_heads=H, group=G, head_dim=D, block=P, seed=8, poison=False,
                 spare=3 * (-(-(keep + steps) // P)) + 2)
    ws = lib.cache_workspace()
    d = cuda(p)
    width = p.bt.shape[1] * P
    # the prompt
    want = ref.append(p)
    lib.pmqa_cache_append(p.k_new.cuda(), p.v_new.cuda(), *d, p.rb.cuda(), p.max_rows, ws=ws)
    p.kc, p.ks, p.vc, p.vs = want
    for got, w in zip((d[0], d[2], d[1], d[3]), want):
        assert torch.equal(got.cpu(), w)
    out, lse = attend(lib, p, d, ws)
    matches(p, out, lse)
    mass = lib.pmqa_cache_weigh(p.q.cuda(), d[0], d[2], d[4], d[5], p.rb.cuda(), p.max_rows, p.sm,
                                lse, mass_width=width, ws=ws)
    wm, tol = ref.weigh(p, lse.cpu(), torch.zeros((3, H, width)))
    check(mass.cpu(), wm.nan_to_num(0.0), tol)
    # the eviction, from the masses that the call before computed
    per = -(-(keep + steps) // P)
    new = p.free[:3 * per].reshape(3, per).contiguous()
    gone = ref.evict(p, mass.cpu(), keep, 4, 16, new)
    kept, lens, mass = lib.pmqa_cache_evict(*d, mass, keep, 4, 16, new.cuda(), ws=ws)
    assert torch.equal(kept.cpu(), gone[0]) and torch.equal(lens.cpu(), gone[1])
    p.kc, p.ks, p.vc, p.vs = gone[3:]
    for got, w in zip((d[0], d[2], d[1], d[3]), gone[3:]):
        assert torch.equal(got.cpu(), w)
    # decode steps behind the kept tokens
    p.bt, ctx = new, gone[1]
    for step in range(steps):
        ctx = ctx + 1
        s = ref.make([1, 1, 1], [1, 1, 1], kv_heads=H, group=G, head_dim=D, block=P, seed=20 + step)
        p.ctx, p.rows, p.rb, p.max_rows = ctx, [1, 1, 1], s.rb, 1
        p.q, p.k_new, p.v_new = s.q, s.k_new, s.v_new
        want = ref.append(p)
        d = [d[0], d[1], d[2], d[3], p.bt.cuda(), p.ctx.cuda()]
        lib.pmqa_cache_append(p.k_new.cuda(), p.v_new.cuda(), *d, p.rb.cuda(), 1, ws=ws)
        p.kc, p.ks, p.vc, p.vs = want
        out, lse = attend(lib, p, d, ws)
        matches(p, out, lse)
        before = mass.cpu()
        lib.pmqa_cache_weigh(p.q.cuda(), d[0], d[2], d[4], d[5], p.rb.cuda(), 1, p.sm, lse, mass,
                             mass_out=mass, ws=ws)
        wm, tol = ref.weigh(p, lse.cpu(), before)
        held = ~torch.isnan(wm)
        check(mass.cpu()[held], wm[held], tol[held])
    status_is(lib, ws)


def test_rows_of_no_request_are_left_as_they_were(cuda_lib):
    p = ref.make([40, 1], [90, 7], kv_heads=2, group=2, head_dim=64, block=8, seed=3, lead=3, tail=4)
    q = p.q.cuda()
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    cuda_lib.pmqa_cache_attention(q, *cuda(p), p.rb.cuda(), p.max_rows, p.sm, out=out, lse=lse)
    for t in (out, lse):
        assert torch.all(t[:3] == 7.0) and torch.all(t[-4:] == 7.0)
    matches(p, out, lse)


@pytest.mark.parametrize("rows", [1, 60])
def test_bad_blocks_are_left_out(cuda_lib, rows):
    """A table entry outside the pool is reported and its tokens take no part."""
    p = ref.make([rows, 1], [150, 20], kv_heads=2, group=2, head_dim=128, block=32, seed=4)
    for bad in (-1, p.kc.shape[0], 2 ** 31 - 1):
        ws = cuda_lib.cache_workspace()
        d = cuda(p)
        d[4] = d[4].clone()
        d[4][0, 1] = bad
        out, lse = attend(cuda_lib, p, d, ws)
        status_is(cuda_lib, ws, cuda_lib.PMQA_DEV_BAD_BLOCK_ID)
        mass = cuda_lib.pmqa_cache_weigh(p.q.cuda(), d[0], d[2], d[4], d[5], p.rb.cuda(),
                                         p.max_rows, p.sm, lse, ws=ws)
        status_is(cuda_lib, ws, cuda_lib.PMQA_DEV_BAD_BLOCK_ID)
        assert torch.all(mass[0, :, 32:64] == 0.0) and torch.all(mass[0, :, :32] > 0.0)
        # the same request without those 32 tokens, its rows behind the last token
        s = ref.make([rows, 1], [150, 20], kv_heads=2, group=2, head_dim=128, block=32, seed=4)
        s.bt = torch.cat([s.bt[:, :1], s.bt[:, 2:], s.bt[:, 1:2]], 1).contiguous()
        s.bt[1] = p.bt[1]
        s.ctx = torch.tensor([118, 20], dtype=torch.int32)
        if rows == 1:
            matches(s, out, lse)
        # the second request is untouched by the first one's table
        want, _, tol, _ = ref.attention(p)
        check(out.cpu()[rows:], want[rows:], tol[rows:])


def test_append_and_evict_skip_bad_blocks(cuda_lib):
    p = ref.make([40], [70], kv_heads=2, group=1, head_dim=64, block=16, seed=5, spare=6)
    ws = cuda_lib.cache_workspace()
    d = cuda(p)
    want = ref.append(p)
    d[4][0, 3] = -5
    cuda_lib.pmqa_cache_append(p.k_new.cuda(), p.v_new.cuda(), *d, p.rb.cuda(), 40, ws=ws)
    status_is(cuda_lib, ws, cuda_lib.PMQA_DEV_BAD_BLOCK_ID)
    skipped = int(p.bt[0, 3])
    rest = [b for b in range(p.kc.shape[0]) if b != skipped]
    assert torch.equal(d[0].cpu()[rest], want[0][rest])
    assert torch.equal(d[0].cpu()[skipped], p.kc[skipped])
    # evict: a bad new block is not written, a bad old one moves zeros
    new = p.free[:2].reshape(1, 2).clone()
    mass = torch.rand((1, 2, 80), device="cuda")
    d = cuda(p)
    new[0, 1] = p.kc.shape[0] + 3
    cuda_lib.pmqa_cache_evict(*d, mass, 32, 0, 32, new.cuda(), ws=ws)
    status_is(cuda_lib, ws, cuda_lib.PMQA_DEV_BAD_BLOCK_ID)
    d = cuda(p)
    d[4][0, 4] = -1
    new[0, 1] = p.free[1]
    cuda_lib.pmqa_cache_evict(*d, mass, 32, 0, 32, new.cuda(), ws=ws)
    status_is(cuda_lib, ws, cuda_lib.PMQA_DEV_BAD_BLOCK_ID)
    assert torch.all(d[0].cpu()[int(new[0, 1]), :, 10:16] == 0)  # slots 64 .. 69


def test_contexts_and_rows_past_their_arrays_are_clamped(cuda_lib):
    p = ref.make([1, 1], [64, 30], kv_heads=1, group=2, head_dim=64, block=16, seed=6)
    d = cuda(p)
    cap = p.bt.shape[1] * 16
    for ctx in (cap + 1, 2 ** 31 - 1, -3):
        ws = cuda_lib.cache_workspace()
        d[5] = torch.tensor([ctx, 30], dtype=torch.int32, device="cuda")
        out, _ = attend(cuda_lib, p, d, ws)
        # the table's fifth entry is -1 where a context reaches it
        bits = cuda_lib.PMQA_DEV_BAD_CONTEXT | (cuda_lib.PMQA_DEV_BAD_BLOCK_ID if ctx > 0 else 0)
        status_is(cuda_lib, ws, bits)
        if ctx < 0:
            assert torch.all(out[0] == 0.0)
        want, _, tol, _ = ref.attention(p)
        check(out.cpu()[1:], want[1:], tol[1:])
    for rb in ([0, 5, 6], [-1, 1, 2], [0, 1, 100], [1, 0, 2]):
        ws = cuda_lib.cache_workspace()
        q = p.q.cuda()
        cuda_lib.pmqa_cache_attention(q, *cuda(p), torch.tensor(rb, dtype=torch.int32).cuda(), 1,
                                      p.sm, ws=ws)
        status_is(cuda_lib, ws, cuda_lib.PMQA_DEV_BAD_CONTEXT)


@pytest.mark.parametrize("rows,G", [(1, 4), (3, 8), (50, 2)])
@pytest.mark.parametrize("kind", ["zeros", "tiny", "spread", "negative", "odd"])
def test_block_scales(cuda_lib, rows, G, kind):
    """Blocks of zeros (scale 2^-100), scales far apart, negative ones: nothing
    overflows and nothing hangs."""
    p = ref.make([rows], [300], kv_heads=2, group=G, head_dim=128, block=16, seed=7, poison=False)
    used = p.bt[0, :19].long()
    if kind == "zeros":
        for b in used[::3]:
            p.vc[b], p.vs[b] = 0, 2.0 ** -100
            p.kc[b], p.ks[b] = 0, 2.0 ** -100
    elif kind == "tiny":
        p.vs[used] *= 2.0 ** -60
        p.ks[used] *= 2.0 ** -60
    elif kind == "spread":
        p.vs[used[::2]] *= 2.0 ** 9
        p.vs[used[1::4]] *= 2.0 ** -9
    elif kind == "negative":
        p.ks[used[::2]] *= -1.0
        p.vs[used[1::2]] *= -1.0
    else:
        p.vs[used] = torch.rand_like(p.vs[used]) + 0.01
        p.ks[used] = torch.rand_like(p.ks[used]) * 0.1 - 0.03
    ws = cuda_lib.cache_workspace()
    out, lse = attend(cuda_lib, p, ws=ws)
    status_is(cuda_lib, ws)
    matches(p, out, lse)


@pytest.mark.parametrize("rows", [1, 40])
def test_a_nan_scale_or_key_reaches_its_rows_only(cuda_lib, rows):
    p = ref.make([rows, 1], [200, 50], kv_heads=2, group=2, head_dim=128, block=32, seed=9)
    p.ks[p.bt[0, 2], 1] = math.nan
    p.kc[p.bt[0, 1], 0, 3, 5] = ref.NAN8
    ws = cuda_lib.cache_workspace()
    out, lse = attend(cuda_lib, p, ws=ws)
    status_is(cuda_lib, ws)
    assert torch.all(torch.isnan(out[:rows])) and torch.all(torch.isnan(lse[:rows]))
    want, _, tol, _ = ref.attention(p)
    check(out.cpu()[rows:], want[rows:], tol[rows:])


@pytest.mark.parametrize("rows", [2, 40])
def test_a_nan_key_behind_a_row_is_not_seen(cuda_lib, rows):
    """The last token's key is NaN: only the last row, which sees it, is NaN."""
    p = ref.make([rows], [100], kv_heads=1, group=2, head_dim=64, block=16, seed=10)
    p.kc[p.bt[0, 6], 0, 3] = ref.NAN8
    out, lse = attend(cuda_lib, p)
    assert torch.all(torch.isnan(out[-1])) and torch.all(torch.isnan(lse[-1]))
    assert torch.all(torch.isfinite(out[:-1])) and torch.all(torch.isfinite(lse[:-1]))


@pytest.mark.parametrize("rows", [1, 40])
@pytest.mark.parametrize("sm", [0.0, -0.3, 4.0])
def test_score_scales(cuda_lib, rows, sm):
    p = ref.make([rows], [170], kv_heads=2, group=3, head_dim=64, block=8, seed=11)
    p.sm = sm
    out, lse = attend(cuda_lib, p)
    matches(p, out, lse)
    mass = cuda_lib.pmqa_cache_weigh(p.q.cuda(), *[t.cuda() for t in (p.kc, p.ks, p.bt, p.ctx, p.rb)],
                                     p.max_rows, sm, lse)
    want, tol = ref.weigh(p, lse.cpu(), torch.zeros(mass.shape))
    check(mass.cpu(), want.nan_to_num(0.0), tol)


@pytest.mark.parametrize("rows", [1, 40])
def test_a_rising_score_moves_the_maximum(cuda_lib, rows):
    """Keys that grow along the context: the running maximum moves many times,
    by more than a weight's f16 range."""
    p = ref.make([rows], [1200], kv_heads=1, group=4, head_dim=128, block=64, seed=12, poison=False)
    for b in range(19):
        p.ks[p.bt[0, b]] *= 1.0 + 0.5 * b
    q = p.q.float()
    k, _ = ref.tokens(p.kc, p.ks, p.bt, 0, 1200, 64)
    p.q = (q * 0.2 + k[0, -1].float() * 0.3).to(torch.bfloat16)
    out, lse = attend(cuda_lib, p)
    matches(p, out, lse)


def test_offsets_past_32_bits(cuda_lib):
    """A pool of 5 GB, its used blocks at the end."""
    H, D, P = 8, 128, 64
    nb = 5 * (1 << 30) // (H * D * P)
    p = ref.make([1, 40], [130, 80], kv_heads=H, group=2, head_dim=D, block=P, seed=13, poison=False)
    n = p.kc.shape[0]
    pools = []
    for code, scale in ((p.kc, p.ks), (p.vc, p.vs)):
        big = torch.zeros((nb, H, P, D), dtype=torch.uint8, device="cuda")
        bs = torch.zeros((nb, H), device="cuda")
        big[nb - n:], bs[nb - n:] = code.cuda(), scale.cuda()
        pools.append((big, bs))
    bt = torch.where(p.bt >= 0, p.bt + (nb - n), p.bt).to(torch.int32).cuda()
    d = [pools[0][0], pools[1][0], pools[0][1], pools[1][1], bt, p.ctx.cuda()]
    out, lse = attend(cuda_lib, p, d)
    matches(p, out, lse)
    mass = cuda_lib.pmqa_cache_weigh(p.q.cuda(), d[0], d[2], bt, d[5], p.rb.cuda(), p.max_rows, p.sm,
                                     lse)
    want, tol = ref.weigh(p, lse.cpu(), torch.zeros(mass.shape))
    check(mass.cpu(), want.nan_to_num(0.0), tol)
    want = ref.append(p)
    cuda_lib.pmqa_cache_append(p.k_new.cuda(), p.v_new.cuda(), *d, p.rb.cuda(), p.max_rows)
    assert torch.equal(d[0][nb - n:].cpu(), want[0]) and torch.equal(d[3][nb - n:].cpu(), want[3])


def test_other_stream_and_graph(cuda_lib):
    """All four calls captured into one graph on a side stream, replayed with new
    inputs and lengths in the same tensors."""
    lib = cuda_lib
    shape = dict(kv_heads=2, group=4, head_dim=128, block=16, poison=False, spare=9)
    p = ref.make([3, 50], [90, 120], seed=14, **shape)
    r = ref.make([2, 40], [85, 113], seed=15, tail=11, **shape)
    ws = lib.cache_workspace()
    q, rb, kn, vn = (t.cuda() for t in (p.q, p.rb, p.k_new, p.v_new))
    d = cuda(p)
    mass_in = torch.rand((2, 2, 144), device="cuda")
    new = p.free[:8].reshape(2, 4).contiguous().cuda()
    stream = torch.cuda.Stream()

    def calls():
        lib.pmqa_cache_append(kn, vn, *d, rb, 50, ws=ws)
        out, lse = lib.pmqa_cache_attention(q, *d, rb, 50, p.sm, want_lse=True, ws=ws)
        mass = lib.pmqa_cache_weigh(q, d[0], d[2], d[4], d[5], rb, 50, p.sm, lse, mass_in, ws=ws)
        return (out, lse, mass) + tuple(lib.pmqa_cache_evict(*d, mass, 64, 2, 8, new, ws=ws))

    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        calls()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            got = calls()
    for s in (p, r):
        for t, x in zip(d + [q, rb, kn, vn], [s.kc, s.vc, s.ks, s.vs, s.bt, s.ctx, s.q, s.rb,
                                              s.k_new, s.v_new]):
            t.copy_(x)
        new.copy_(s.free[:8].reshape(2, 4))
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            graph.replay()
        torch.cuda.synchronize()
        s.kc, s.ks, s.vc, s.vs = ref.append(s)
        matches(s, got[0], got[1])
        wm, tol = ref.weigh(s, got[1].cpu(), mass_in.cpu())
        held = ~torch.isnan(wm)
        check(got[2].cpu()[held], wm[held], tol[held])
        gone = ref.evict(s, got[2].cpu(), 64, 2, 8, s.free[:8].reshape(2, 4))
        assert torch.equal(got[3].cpu(), gone[0]) and torch.equal(got[4].cpu(), gone[1])
    status_is(lib, ws)


def test_a_given_stream_also_allocates_and_fills(cuda_lib):
    """With stream=, zeros and copies made by the call are that stream's: work
    that is late on the current stream does not undo the result."""
    lib = cuda_lib
    p = ref.make([2, 40], [70, 60], kv_heads=2, group=2, head_dim=64, block=16, seed=16)
    d, q, rb = cuda(p), p.q.cuda(), p.rb.cuda()
    had = torch.rand((2, 2, 96), device="cuda")
    out, lse = attend(lib, p, d)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(50_000_000)  # about 25 ms on the current stream
    args = (q, d[0], d[2], d[4], d[5], rb, p.max_rows, p.sm, lse)
    a = lib.pmqa_cache_weigh(*args, mass_width=96, stream=side)
    b = lib.pmqa_cache_weigh(*args, had, stream=side)
    again = lib.pmqa_cache_attention(q, *d, rb, p.max_rows, p.sm, stream=side)
    torch.cuda.synchronize()
    for got, start in ((a, torch.zeros_like(had)), (b, had)):
        want, tol = ref.weigh(p, lse.cpu(), start.cpu())
        check(got.cpu(), torch.where(torch.isnan(want), start.cpu().double(), want), tol)
    assert torch.equal(again, out)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows", [1, 12, 40])
@pytest.mark.parametrize("power", [122, -112])
def test_queries_at_the_ends_of_the_range(cuda_lib, rows, D, power):
    """q of 2^122 (up to 2^125) or 2^-112 under a score scale that undoes it; a power
    of two in q is exact, so the tolerances are those of ordinary values."""
    p = ref.make([rows, 1], [rows + 90, 33], kv_heads=2, group=2, head_dim=D, block=16, seed=17)
    p.q = (p.q.float() * 2.0 ** power).to(torch.bfloat16)
    p.sm *= 2.0 ** -power
    out, lse = attend(cuda_lib, p)
    matches(p, out, lse)
    d = cuda(p)
    width = p.bt.shape[1] * 16
    mass = cuda_lib.pmqa_cache_weigh(p.q.cuda(), d[0], d[2], d[4], d[5], p.rb.cuda(), p.max_rows,
                                     p.sm, lse)
    want, tol = ref.weigh(p, lse.cpu(), torch.zeros((2, 2, width)))
    check(mass.cpu(), want.nan_to_num(0.0), tol)


def test_the_same_call_gives_the_same_bits(cuda_lib):
    p = ref.make([1, 4, 90], [3000, 900, 700], kv_heads=2, group=4, head_dim=128, block=32, seed=16)
    d = cuda(p)
    out, lse = attend(cuda_lib, p, d)
    mass = cuda_lib.pmqa_cache_weigh(p.q.cuda(), d[0], d[2], d[4], d[5], p.rb.cuda(), p.max_rows,
                                     p.sm, lse)
    for _ in range(3):
        o, l = attend(cuda_lib, p, d)
        assert torch.equal(o, out) and torch.equal(l, lse)
        m = cuda_lib.pmqa_cache_weigh(p.q.cuda(), d[0], d[2], d[4], d[5], p.rb.cuda(), p.max_rows,
                                      p.sm, lse)
        assert torch.equal(m, mass)


def test_long_contexts_are_cut_and_joined(cuda_lib):
    """One request over every SM, and lengths around the tile."""
    for ctx in ([20000], [63, 64, 65, 127, 128, 129, 1025], [1]):
        p = ref.make([2] * len(ctx) if ctx != [1] else [1], ctx, kv_heads=1, group=4, head_dim=64,
                     block=64, seed=17)
        out, lse = attend(cuda_lib, p)
        matches(p, out, lse)


@pytest.mark.parametrize("rows,ctx,H,G,D,P", [
    ([40], [5000], 1, 1, 128, 64),                       # one row block over many CTAs
    ([5, 1, 5], [3100, 700, 2049], 2, 8, 64, 48),        # beside a request of few rows
    ([300, 33], [300, 4000], 1, 2, 128, 16),             # blocks that see only the first pieces
    ([9, 12, 7, 11], [513, 1025, 9, 0], 3, 5, 128, 24),  # pieces of few tokens, an empty context
    ([2, 1], [1500, 900], 1, 40, 64, 32),                # more query heads than the few-row kernel takes
    ([70, 60], [60, 2000], 1, 1, 64, 8),                 # rows before slot 0
])
def test_many_rows_of_few_requests_are_cut_and_joined(cuda_lib, rows, ctx, H, G, D, P):
    p = ref.make(rows, ctx, kv_heads=H, group=G, head_dim=D, block=P, seed=21, lead=2, tail=1)
    ws = cuda_lib.cache_workspace()
    out, lse = attend(cuda_lib, p, ws=ws)
    matches(p, out, lse)
    again, lse2 = attend(cuda_lib, p, ws=ws)
    r0, r1 = int(p.rb[0]), int(p.rb[-1])
    assert torch.equal(out[r0:r1], again[r0:r1]) and torch.equal(lse[r0:r1], lse2[r0:r1])
    status_is(cuda_lib, ws)


@pytest.mark.parametrize("bs", [128, 140])
def test_many_requests_with_many_rows(cuda_lib, bs):
    """More row blocks than SMs, in order of length (up to 128 requests) or of rows."""
    rows = [40 if i % 3 else 1 for i in range(bs)]
    ctx = [max(n, (53 * i) % 400) for i, n in enumerate(rows)]
    p = ref.make(rows, ctx, kv_heads=2, group=2, head_dim=64, block=16, seed=23)
    ws = cuda_lib.cache_workspace()
    out, lse = attend(cuda_lib, p, ws=ws)
    matches(p, out, lse)
    status_is(cuda_lib, ws)


def test_cut_contexts_with_a_bad_block_and_a_nan_key(cuda_lib):
    """A key that is NaN reaches the rows that see it and no other piece's; a table
    entry outside the pool is left out of its piece."""
    p = ref.make([50, 40], [3000, 2500], kv_heads=1, group=1, head_dim=128, block=32, seed=22)
    p.kc[p.bt[0, 2980 // 32].long(), 0, 2980 % 32, 5] = ref.NAN8  # rows 30 and later see it
    ws = cuda_lib.cache_workspace()
    d = cuda(p)
    out, lse = attend(cuda_lib, p, d, ws)
    assert torch.all(torch.isnan(lse[30:50])) and torch.all(torch.isnan(out[30:50]))
    want, want_l, tol, ltol = ref.attention(p)
    for a, b in ((0, 30), (50, 90)):
        check(out.cpu()[a:b], want[a:b], tol[a:b])
        check(lse.cpu()[a:b], want_l[a:b], ltol[a:b])
    status_is(cuda_lib, ws)
    d[4] = d[4].clone()
    d[4][1, 40] = p.kc.shape[0]
    again, _ = attend(cuda_lib, p, d, ws)
    status_is(cuda_lib, ws, cuda_lib.PMQA_DEV_BAD_BLOCK_ID)
    assert torch.equal(again[:30], out[:30]) and torch.isfinite(again[50:].float()).all()


@pytest.mark.parametrize("bs", [40, 140])
def test_evict_of_many_requests(cuda_lib, bs):
    """More lists than SMs: taken in the order of their length (up to 128 requests) or
    of their number; equal lengths, empty requests and ones that keep everything."""
    keep, P, H = 20, 8, 4
    ctx = [(37 * i) % 90 if i % 5 else 70 for i in range(bs)]
    p = ref.make([0] * bs, ctx, kv_heads=H, group=1, head_dim=64, block=P, seed=24, poison=False,
                 spare=3 * bs)
    new = p.free[:3 * bs].reshape(bs, 3).contiguous()
    mass = torch.rand((bs, H, 96), generator=p.gen).mul(8).round()  # many ties
    want = ref.evict(p, mass, keep, 2, 5, new)
    d = cuda(p)
    ws = cuda_lib.cache_workspace()
    kept, lens, out = cuda_lib.pmqa_cache_evict(*d, mass.cuda(), keep, 2, 5, new.cuda(), ws=ws)
    assert torch.equal(kept.cpu(), want[0]) and torch.equal(lens.cpu(), want[1])
    assert torch.equal(out.cpu(), want[2])
    for got, w in zip((d[0], d[2], d[1], d[3]), want[3:]):
        assert torch.equal(got.cpu(), w)
    status_is(cuda_lib, ws)


def test_evict_longer_than_a_cluster_holds(cuda_lib):
    """More masses than eight CTAs keep in shared memory, ties across the border."""
    ctx, P, keep = 420000, 1024, 3000
    H, D = 1, 64
    nb = -(-ctx // P) + -(-keep // P)
    g = torch.Generator(device="cuda").manual_seed(3)
    code = torch.randint(0, 120, (nb, H, P, D), generator=g, device="cuda", dtype=torch.uint8)
    scale = torch.ones((nb, H), device="cuda")
    mass = torch.rand((1, H, ctx), generator=g, device="cuda")
    mass[0, 0, 390000:400000] = 0.995  # many equal ones around the threshold
    bt = torch.arange(-(-ctx // P), dtype=torch.int32, device="cuda")[None]
    new = torch.arange(-(-ctx // P), nb, dtype=torch.int32, device="cuda")[None]
    lens = torch.tensor([ctx], dtype=torch.int32, device="cuda")
    ws = cuda_lib.cache_workspace()
    kept, _, _ = cuda_lib.pmqa_cache_evict(code, code.clone(), scale, scale.clone(), bt, lens, mass,
                                           keep, 5, 11, new, ws=ws)
    status_is(cuda_lib, ws)
    rank = mass[0, 0].clone()
    rank[:5] = math.inf
    rank[-11:] = math.inf
    want = torch.sort(rank, descending=True, stable=True).indices[:keep].sort().values
    assert torch.equal(kept[0, 0].long(), want)


def test_no_device_memory_is_allocated(cuda_lib):
    """With outputs and workspace given, a call allocates nothing."""
    p = ref.make([1, 40], [90, 120], kv_heads=2, group=4, head_dim=128, block=16, seed=18)
    d, q, rb = cuda(p), p.q.cuda(), p.rb.cuda()
    ws = cuda_lib.cache_workspace()
    out, lse = attend(cuda_lib, p, d, ws)
    torch.cuda.synchronize()
    before = torch.cuda.mem_get_info()[0], torch.cuda.memory_allocated()
    for _ in range(3):
        cuda_lib.pmqa_cache_attention(q, *d, rb, p.max_rows, p.sm, out=out, lse=lse, ws=ws)
    torch.cuda.synchronize()
    assert (torch.cuda.mem_get_info()[0], torch.cuda.memory_allocated()) == before
