"""How the operators around the sparse-MLA step are used together and with what
was there, and the calls that their documentation allows at the edges: captured graphs,
other streams, offsets past 32 bits, long contexts, shared blocks, strided and
empty inputs."""

import math
from types import SimpleNamespace

import numpy as np
import pytest
import torch

import oracle
from synth.inputs import Problem
from tests import cache_ref, step_ref as ref
from tests.parity import check_logits, check_mla, check_topk_rows
from tests.test_gpu_latent_attention import check, run
from tests.test_gpu_step_rows import index_case

pytestmark = pytest.mark.gpu

F8 = torch.float8_e4m3fn
BF = torch.bfloat16


def bits(t):
    return t.contiguous().view(torch.uint8)


def same(a, b):
    return torch.equal(bits(a), bits(b))


def rotary(lib, dim=64, begin=0, interleaved=True):
    f, s = lib.rope_frequencies(dim, kind=lib.PMQA_ROPE_PARTS, factor=40.0)
    return lib.Rotary(f, begin, interleaved, s)


def cache(p, kv=None):
    return [t.cuda() for t in (p.kv if kv is None else kv, p.bt, p.ctx, p.rb)] + [p.max_rows]


def latent_case(rows, ctx, block, heads, seed=0, **kw):
    p = ref.layout(rows, ctx, block, seed, **kw)
    p.kv = torch.randint(0, 127, (p.nb, block, 576), generator=p.gen, dtype=torch.uint8)
    p.c, p.k_pe, p.q_c, p.q_pe = (torch.randn(s, generator=p.gen).to(BF) for s in (
        (p.total, 512), (p.total, 64), (p.total, heads, 512), (p.total, heads, 64)))
    p.heads, p.kv_scale, p.q_scale, p.sm = heads, 0.03, 0.02, 192 ** -0.5
    return p


# ------------------------------------------------------------- together

def test_index_rows_feed_the_logits_and_topk(cuda_lib):
    """Keys appended over a prompt and three steps; the logits and top-k calls over what lies in
    the cache then, against the oracle on the same bytes."""
    lib, bs, nn, heads, P = cuda_lib, 3, 2, 64, 16
    first, steps = [40, 200, 90], 3
    ctx = [c + nn * steps for c in first]
    lay = ref.layout(first, ctx, P, seed=4)
    kv = torch.zeros((lay.nb, P, 132), dtype=torch.uint8, device="cuda")
    bt, r, ws = lay.bt.cuda(), rotary(lib), lib.workspace(1, 1, 1, 0, lib.PMQA_OP_LOGITS)
    norm = lib.Norm(lib.PMQA_NORM_LAYER, torch.rand(128, device="cuda") + 0.5, torch.randn(128, device="cuda"))
    g = torch.Generator().manual_seed(5)

    def append(rows, ctx):
        rb = torch.tensor([0] + rows).cumsum(0).to(torch.int32).cuda()
        n = sum(rows)
        k = torch.randn((n, 128), generator=g).to(BF).cuda()
        q = torch.randn((n, heads, 128), generator=g).to(BF).cuda()
        w = torch.randn((n, heads), generator=g).cuda()
        lens = torch.tensor(ctx, dtype=torch.int32).cuda()
        return lens, lib.pmqa_index_append(k, kv, bt, lens, rb, max(rows), q=q, weights=w, weight_scale=0.1,
                                           norm=norm, rotary=r, ws=ws)

    append(first, first)
    for s in range(steps):
        lens, (q, w) = append([nn] * bs, [c + nn * (s + 1) for c in first])
    mml, k = bt.shape[1] * P, 64
    q = q.reshape(bs, nn, heads, 128)
    got = lib.pmqa_logits(q, kv, w, lens, bt, mml)
    idx, vals = lib.pmqa_logits_topk(q, kv, w, lens, bt, mml, k, want_vals=True)
    prob = Problem(q=q.view(torch.uint8).cpu().numpy(), kv=kv.cpu().numpy(), weights=w.cpu().numpy(),
                   context_lens=lens.cpu().numpy(), block_tables=lay.bt.numpy(), bs=bs, next_n=nn, heads=heads,
                   block_size=P, max_model_len=mml, k=k)
    want, w64, tol = oracle.logits(prob, want64=True, want_tol=True)
    check_logits(got.cpu().numpy(), want, tol)
    check_topk_rows(idx.cpu().numpy(), w64, tol, prob.context_lens, nn, k, vals=vals.cpu().numpy())
    assert lib.pmqa_read_device_status(ws) == 0


def test_index_rows_read_back_feed_the_prefill_logits(cuda_lib):
    """A chunk of prompts: keys into the cache, the contexts' keys back as contiguous rows, and
    the chunk's queries against them; against the oracle on the same bytes."""
    lib, heads = cuda_lib, 32
    p = index_case([50, 1, 120], [170, 1, 120], 16, heads, seed=8)
    kv, bt, ctx, rb, most = cache(p)
    q, w = lib.pmqa_index_append(p.k.cuda(), kv, bt, ctx, rb, most, q=p.q.cuda(), weights=p.w.cuda(),
                                 rotary=rotary(lib))
    # the slots before the chunk hold bytes of any value: let their keys be small ones
    flat = kv.reshape(-1, 132)
    old = torch.cat([ref.places(p, i, 0, int(p.ctx[i]) - n) for i, n in enumerate(p.rows)]).cuda()
    flat[old, :128] &= 0xBF
    flat[old, 128:] = torch.tensor([0.01], device="cuda").view(torch.uint8)
    starts = torch.tensor([0] + p.ctx.tolist()).cumsum(0).to(torch.int32)
    n = int(starts[-1])
    keys, scale = lib.pmqa_index_read(kv, bt, starts.cuda(), n)
    at = torch.cat([ref.places(p, i, 0, int(c)) for i, c in enumerate(p.ctx)])
    assert torch.equal(keys.view(torch.uint8).cpu(), kv.cpu().reshape(-1, 132)[at, :128])
    ks = torch.tensor([int(starts[i]) for _, i, _ in ref.slots(p)], dtype=torch.int32)
    ke = torch.tensor([int(starts[i]) + t + 1 for _, i, t in ref.slots(p)], dtype=torch.int32)
    got = lib.pmqa_mqa_logits(q, keys, scale, w, ks.cuda(), ke.cuda())
    prob = SimpleNamespace(q=q.view(torch.uint8).cpu().numpy(), k=keys.view(torch.uint8).cpu().numpy(),
                           k_scale=scale.cpu().numpy(), weights=w.cpu().numpy(), ks=ks.numpy(), ke=ke.numpy(),
                           m=p.total, n=n, heads=heads)
    want, _, tol = oracle.mqa_logits(prob, want_tol=True)
    check_logits(got.cpu().numpy(), want, tol)


def test_latent_rows_feed_both_attentions(cuda_lib):
    """A prompt's latent rows and two steps appended; the dense attention, and the sparse one
    over the list of all positions, on the same cache and queries, each within its own bound of
    64 bits."""
    lib, bs, heads, P = cuda_lib, 3, 16, 16
    first = [70, 33, 130]
    p = latent_case(first, first, P, heads, seed=21, spare=20)
    p.kv[:] = ref.NAN8
    p.bt[:] = torch.randperm(p.nb, generator=p.gen).to(torch.int32)[:p.bt.numel()].reshape(p.bt.shape)
    kv, bt, ctx, rb, most = cache(p)
    r, ws = rotary(lib), lib.latent_workspace()
    norm = lib.Norm(lib.PMQA_NORM_RMS, torch.rand(512, device="cuda") + 0.5, None)

    def append(c, k_pe, q_c, q_pe, lens, rb, most):
        return lib.pmqa_latent_append(c.cuda(), k_pe.cuda(), kv, bt, lens, rb, most, p.kv_scale, q_c=q_c.cuda(),
                                      q_pe=q_pe.cuda(), q_scale=p.q_scale, norm=norm, rotary=r, ws=ws)

    q = append(p.c, p.k_pe, p.q_c, p.q_pe, ctx, rb, most)

    def dense(q, lens, rb, most):
        return lib.pmqa_latent_attention(q, kv, bt, lens, rb, most, p.q_scale, p.kv_scale, p.sm, want_lse=True, ws=ws)

    got = dense(q, ctx, rb, most)
    p.kv, p.q = kv.cpu(), q.view(torch.uint8).cpu()
    assert check((got[0].cpu(), got[1].cpu(), lib.pmqa_read_device_status(ws)), ref.attention(p), p) == 0
    for s in range(2):
        nn = 2
        lens = torch.tensor([c + nn * (s + 1) for c in first], dtype=torch.int32)
        st = latent_case([nn] * bs, lens.tolist(), P, heads, seed=30 + s)
        st.bt, st.nb = p.bt, p.nb
        q = append(st.c, st.k_pe, st.q_c, st.q_pe, lens.cuda(), st.rb.cuda(), nn)
        got = dense(q, lens.cuda(), st.rb.cuda(), nn)
        st.kv, st.q = kv.cpu(), q.view(torch.uint8).cpu()
        want = ref.attention(st)
        assert check((got[0].cpu(), got[1].cpu(), lib.pmqa_read_device_status(ws)), want, st) == 0
        idx = torch.full((bs * nn, 256), -1, dtype=torch.int32)
        for row, i, t in ref.slots(st):
            idx[row, :t + 1] = torch.randperm(t + 1, generator=st.gen).to(torch.int32)
        out, lse = lib.pmqa_sparse_mla_decode(q, kv.view(F8), idx.cuda(), bt, nn, p.q_scale, p.kv_scale, p.sm,
                                              want_lse=True)
        prob = SimpleNamespace(q=st.q.numpy().reshape(bs, nn, heads, 576), kv=st.kv.numpy(), indices=idx.numpy(),
                               block_tables=st.bt.numpy(), q_scale=p.q_scale, kv_scale=p.kv_scale, sm_scale=p.sm,
                               bs=bs, next_n=nn, heads=heads)
        o, l, tol = oracle.sparse_mla(prob, want_tol=True)
        check_mla(out.float().cpu().numpy(), lse.cpu().numpy(), o, l, tol)
        assert np.allclose(o, want[0].numpy(), rtol=1e-9, atol=1e-9) and np.allclose(l, want[1].numpy(), rtol=1e-9)


def test_rope_feeds_the_kv_cache(cuda_lib):
    """Queries and keys of a fused projection rotated where they lie, then appended and attended
    to by the calls on the 8-bit K/V cache, against their own plain forms on the rotated values."""
    lib, H, G, D = cuda_lib, 2, 4, 128
    p = cache_ref.make([30, 2], [64, 90], kv_heads=H, group=G, head_dim=D, block=16, seed=3, poison=False)
    n = p.q.shape[0]
    fused = torch.cat([p.q, p.k_new, p.v_new], 1).cuda()
    q, k, v = fused.split([H * G, H, H], 1)
    pos = torch.tensor([int(p.ctx[i]) - m + j for i, m in enumerate(p.rows) for j in range(m)], dtype=torch.int32)
    r = rotary(lib, D, 0, False)
    lib.pmqa_rope(q, pos.cuda(), r, other=k, out=q, other_out=k)
    for x, y in ((p.q, q), (p.k_new, k)):
        want, e = ref.rotate(x.double(), pos, r.inv_freq.cpu(), 0, False, r.scale)
        assert bool(((y.cpu().double() - want).abs() <= e + (want.abs() + e) * 2.0 ** -8).all())
    assert torch.equal(v.cpu(), p.v_new)
    p.q, p.k_new = q.cpu().contiguous(), k.cpu().contiguous()
    d = [t.cuda() for t in (p.kc, p.vc, p.ks, p.vs, p.bt, p.ctx)]
    want = cache_ref.append(p)
    lib.pmqa_cache_append(k.contiguous(), v.contiguous(), *d, p.rb.cuda(), p.max_rows)
    assert torch.equal(d[0].cpu(), want[0]) and torch.equal(d[2].cpu(), want[1])
    p.kc, p.ks, p.vc, p.vs = want
    out, lse = lib.pmqa_cache_attention(q.contiguous(), *d, p.rb.cuda(), p.max_rows, p.sm, want_lse=True)
    o, l, tol, ltol = cache_ref.attention(p)
    assert n == o.shape[0] and bool(((out.cpu().double() - o).abs() <= tol).all())
    assert bool(((lse.cpu().double() - l).abs() <= ltol).all())


# ------------------------------------------------------------- graphs and streams

def test_a_step_captured_and_replayed(cuda_lib):
    """All calls of a step in one graph on a side stream, replayed with other inputs, lengths
    and tables in the same tensors: the bits of the same calls made one by one."""
    lib, heads, P = cuda_lib, 16, 16
    ws, r = lib.latent_workspace(), rotary(lib)
    stream = torch.cuda.Stream()

    def inputs(seed):
        g = torch.Generator().manual_seed(seed)
        lat = latent_case([3, 1, 2], [seed * 7 + 60, 600, 5], P, heads, seed=seed)
        idx = index_case([3, 1, 2], [seed * 7 + 60, 600, 5], P, 64, seed=seed)
        bt = torch.full((3, 40), -1, dtype=torch.int32)
        bt[:, :lat.bt.shape[1]] = lat.bt
        pool = [torch.zeros((64, P, w), dtype=torch.uint8) for w in (576, 132)]
        for t, x in zip(pool, (lat.kv, idx.kv)):
            t[:x.shape[0]] = x
        pool[1].view(torch.float32)[..., 32] = 0.01
        return [t.cuda() for t in (lat.c, lat.k_pe, lat.q_c, lat.q_pe, idx.k, idx.q, idx.w, bt, lat.ctx, lat.rb,
                                   *pool, torch.randint(0, 1 << 20, (6,), generator=g, dtype=torch.int32))]

    def step(c, k_pe, q_c, q_pe, k, q, w, bt, ctx, rb, kv, ikv, pos):
        turned = lib.pmqa_rope(q, pos, r)
        iq, iw = lib.pmqa_index_append(k, ikv, bt, ctx, rb, 3, q=turned, weights=w, rotary=r, ws=ws)
        keys, s = lib.pmqa_index_read(ikv, bt, rb, 6, ws=ws)
        lq = lib.pmqa_latent_append(c, k_pe, kv, bt, ctx, rb, 3, 0.03, q_c=q_c, q_pe=q_pe, q_scale=0.02, rotary=r,
                                    positions=pos, ws=ws)
        out, lse = lib.pmqa_latent_attention(lq, kv, bt, ctx, rb, 3, 0.02, 0.03, 0.07, want_lse=True, ws=ws)
        return turned, iq, iw, keys, s, lq, out, lse, kv, ikv

    args = inputs(1)
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step(*args)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            got = step(*args)
    for seed in (1, 2, 3):
        fresh = inputs(seed)
        want = [t.clone() for t in step(*[t.clone() for t in fresh])]
        for a, b in zip(args, fresh):
            a.copy_(b)
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            graph.replay()
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(got, want))
    assert lib.pmqa_read_device_status(ws) == 0


@pytest.mark.parametrize("heads", [16, 128])
def test_two_graphs_share_a_workspace(cuda_lib, heads):
    lib, ws, stream = cuda_lib, cuda_lib.latent_workspace(), torch.cuda.Stream()
    cases = [ref.attention_problem([1, 1], [3000, 700], heads, 16, seed=1),
             ref.attention_problem([2], [1900], heads, 64, seed=2)]
    graphs = []
    for p in cases:
        a = [t.cuda() for t in (p.q, p.kv, p.bt, p.ctx, p.rb)] + [p.max_rows, p.q_scale, p.kv_scale, p.sm]
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            want = lib.pmqa_latent_attention(*a, want_lse=True, ws=ws)
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                got = lib.pmqa_latent_attention(*a, want_lse=True, ws=ws)
        graphs.append((graph, got, want, a))
    with torch.cuda.stream(stream):
        for i in (0, 1, 0, 1, 1):
            for t in graphs[i][1]:
                t.zero_()
            graphs[i][0].replay()
    torch.cuda.synchronize()
    for _, got, want, _ in graphs:
        assert all(same(x, y) for x, y in zip(got, want))
    p = cases[0]
    got = graphs[0][1]
    assert check((got[0].cpu(), got[1].cpu(), lib.pmqa_read_device_status(ws)), ref.attention(p), p) == 0


def test_calls_at_once_on_two_streams(cuda_lib):
    """Each with its own workspace: the same bits as one after the other."""
    lib = cuda_lib
    work = []
    for heads, seed in ((128, 1), (16, 2)):
        p = ref.attention_problem([1] * 6, [5000, 300, 2000, 7, 900, 4100], heads, 64, seed=seed)
        a = [t.cuda() for t in (p.q, p.kv, p.bt, p.ctx, p.rb)] + [p.max_rows, p.q_scale, p.kv_scale, p.sm]
        work.append((a, lib.latent_workspace(), torch.cuda.Stream()))
    alone = [lib.pmqa_latent_attention(*a, want_lse=True, ws=ws) for a, ws, _ in work]
    torch.cuda.synchronize()
    both = [[lib.pmqa_latent_attention(*a, want_lse=True, ws=ws, stream=s) for a, ws, s in work] for _ in range(20)]
    torch.cuda.synchronize()
    for one in both:
        for (o, l), (x, y) in zip(one, alone):
            assert same(o, x) and same(l, y)


def test_a_given_stream_is_the_calls_own(cuda_lib):
    """Work that is late on the current stream holds nothing up and undoes nothing; the calls make
    their workspaces and results on the stream given."""
    lib = cuda_lib
    i, l = index_case([2, 1], [50, 9], 16, 64, seed=1), latent_case([2, 1], [50, 9], 16, 16, seed=2)
    ic, lc, r = cache(i), cache(l), rotary(lib)
    d = [t.cuda() for t in (i.k, i.q, i.w, l.c, l.k_pe, l.q_c, l.q_pe)]
    pos = torch.arange(3, dtype=torch.int32).cuda()

    def calls(kv, ikv, stream=None):
        q, w = lib.pmqa_index_append(d[0], ikv, *ic[1:], q=d[1], weights=d[2], rotary=r, stream=stream)
        k, s = lib.pmqa_index_read(ikv, ic[1], ic[3], 3, stream=stream)
        lq = lib.pmqa_latent_append(d[3], d[4], kv, *lc[1:], 0.03, q_c=d[5], q_pe=d[6], q_scale=0.02, rotary=r,
                                    stream=stream)
        o = lib.pmqa_latent_attention(lq, kv, *lc[1:], 0.02, 0.03, 0.07, want_lse=True, stream=stream)
        return [q, w, k, s, lq, *o, lib.pmqa_rope(d[1], pos, r, stream=stream), kv, ikv]

    want = calls(lc[0].clone(), ic[0].clone())
    kv, ikv, side = lc[0].clone(), ic[0].clone(), torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(200_000_000)  # about 100 ms on the current stream
    late = torch.cuda.Event()
    late.record()
    got = calls(kv, ikv, side)
    side.synchronize()
    assert not late.query()
    # copied out on the side stream, where they belong
    with torch.cuda.stream(side):
        got = [t.cpu() for t in got]
    torch.cuda.synchronize()
    assert all(same(a, b.cpu()) for a, b in zip(got, want))


# ------------------------------------------------------------- large ones

def test_index_pool_past_32_bits(cuda_lib):
    """The requests' blocks behind 4.4 GB of others."""
    lib = cuda_lib
    p = index_case([5, 1, 3], [200, 64, 3], 64, 16, seed=2)
    small, bt, ctx, rb, most = cache(p)
    before = 4_400_000_000 // (64 * 132)
    pool = torch.zeros((before + p.nb, 64, 132), dtype=torch.uint8, device="cuda")
    pool[before:] = small
    moved = torch.where(bt >= 0, bt + before, bt)
    r, ws = rotary(lib), lib.workspace(1, 1, 1, 0, lib.PMQA_OP_LOGITS)
    for kv, t in ((small, bt), (pool, moved)):
        lib.pmqa_index_append(p.k.cuda(), kv, t, ctx, rb, most, rotary=r, ws=ws)
    assert torch.equal(pool[before:], small) and int(pool[:before].count_nonzero()) == 0
    starts = torch.tensor([0] + p.ctx.tolist()).cumsum(0).to(torch.int32).cuda()
    a, b = (lib.pmqa_index_read(kv, t, starts, 267, ws=ws) for kv, t in ((small, bt), (pool, moved)))
    assert same(a[0], b[0]) and same(a[1], b[1])
    assert lib.pmqa_read_device_status(ws) == 0


@pytest.mark.parametrize("heads", [16, 64, 128])
def test_latent_pool_past_32_bits(cuda_lib, heads):
    lib = cuda_lib
    p = latent_case([5, 1, 3], [900, 64, 3], 64, heads, seed=2)
    small, bt, ctx, rb, most = cache(p)
    before = 4_400_000_000 // (64 * 576)
    pool = torch.full((before + p.nb, 64, 576), ref.NAN8, dtype=torch.uint8, device="cuda")
    pool[before:] = small
    moved = torch.where(bt >= 0, bt + before, bt)
    r, ws = rotary(lib), lib.latent_workspace()
    res = []
    for kv, t in ((small, bt), (pool, moved)):
        q = lib.pmqa_latent_append(p.c.cuda(), p.k_pe.cuda(), kv, t, ctx, rb, most, 0.03, q_c=p.q_c.cuda(),
                                   q_pe=p.q_pe.cuda(), q_scale=0.02, rotary=r, ws=ws)
        res.append((q, *lib.pmqa_latent_attention(q, kv, t, ctx, rb, most, 0.02, 0.03, 0.07, want_lse=True, ws=ws)))
    assert torch.equal(pool[before:], small)
    assert all(same(x, y) for x, y in zip(*res))
    assert lib.pmqa_read_device_status(ws) == 0


def test_rope_past_32_bits(cuda_lib):
    """2.3e9 elements: the last rows as in a call of their own."""
    lib, rows, heads, dim = cuda_lib, 36000, 128, 512
    x = torch.zeros((rows, heads, dim), dtype=BF, device="cuda")
    x[-7:] = torch.randn((7, heads, dim), device="cuda").to(BF)
    pos = torch.arange(rows, dtype=torch.int32, device="cuda")
    r = rotary(lib, 64, 128, False)
    y = lib.pmqa_rope(x, pos, r)
    assert same(y[-7:], lib.pmqa_rope(x[-7:].clone(), pos[-7:].clone(), r))
    assert int(y[:-7].count_nonzero()) == 0


def test_index_queries_past_32_bits(cuda_lib):
    """270,000 rows of 128 heads: 4.4 GB of codes."""
    lib, rows, heads = cuda_lib, 270000, 128
    q = torch.zeros((rows, heads, 128), dtype=BF, device="cuda")
    q[-5:] = torch.randn((5, heads, 128), device="cuda").to(BF)
    w = torch.ones((rows, heads), device="cuda")
    kv = torch.zeros((1, 16, 132), dtype=torch.uint8, device="cuda")
    bt = torch.zeros((1, rows // 16 + 1), dtype=torch.int32, device="cuda")
    r, i32 = rotary(lib), dict(dtype=torch.int32, device="cuda")
    ctx, rb = torch.tensor([rows], **i32), torch.tensor([0, rows], **i32)
    got = lib.pmqa_index_append(None, kv, bt, ctx, rb, rows, q=q, weights=w, rotary=r)
    want = lib.pmqa_index_append(None, kv, bt, ctx, torch.tensor([0, 5], **i32), 5, q=q[-5:].clone(), weights=w[:5],
                                 rotary=r)
    assert same(got[0][-5:], want[0]) and same(got[1][-5:], want[1])
    # zeros of either sign (0 cos - 0 sin is -0 where the cosine is negative and the sine not)
    assert int((got[0][:-5].view(torch.uint8) & 0x7F).count_nonzero()) == 0


def test_latent_queries_past_32_bits(cuda_lib):
    """60,000 requests of one row and 128 heads: 4.4 GB of query codes, 7.9 GB of output."""
    lib, n, heads, P = cuda_lib, 60000, 128, 64
    p = ref.attention_problem([1, 1, 1], [100, 7, 640], heads, P, seed=6, poison=False)
    small = p.bt.shape[1]
    bt = torch.zeros((n + 3, small), dtype=torch.int32)
    bt[n:] = p.bt
    i32 = dict(dtype=torch.int32, device="cuda")
    ctx = torch.full((n + 3,), 2, dtype=torch.int32)
    ctx[n:] = p.ctx
    rb = torch.arange(n + 4, **i32)
    q_c = torch.zeros((n + 3, heads, 512), dtype=BF, device="cuda")
    q_pe = torch.zeros((n + 3, heads, 64), dtype=BF, device="cuda")
    q_c[n:] = ref.value(p.q[..., :512]).to(BF).cuda()
    q_pe[n:] = ref.value(p.q[..., 512:]).to(BF).cuda()
    kv, bt, ctx = p.kv.cuda(), bt.cuda(), ctx.cuda()
    q = lib.pmqa_latent_append(None, None, kv, bt, ctx, rb, 1, 1.0, q_c=q_c, q_pe=q_pe, q_scale=1.0)
    assert same(q[n:], p.q.cuda()) and int(q[:n].view(torch.uint8).count_nonzero()) == 0
    del q_c, q_pe
    ws = lib.latent_workspace()
    out, lse = lib.pmqa_latent_attention(q, kv, bt, ctx, rb, 1, p.q_scale, p.kv_scale, p.sm, want_lse=True, ws=ws)
    assert check((out[n:].cpu(), lse[n:].cpu(), lib.pmqa_read_device_status(ws)), ref.attention(p), p) == 0
    # scores of 0: the mean of two tokens, e4m3 values summed exactly, one rounding
    v = (ref.value(p.kv[0, :2, :512]) * p.kv_scale).mean(0).cuda()
    assert bool(((out[:n].amax(0) - v).abs() <= v.abs() * (2.0 ** -8 + 2.0 ** -10) + 1e-6).all())
    assert bool(((out[:n].amin(0) - v).abs() <= v.abs() * (2.0 ** -8 + 2.0 ** -10) + 1e-6).all())
    assert bool(((lse[:n] - math.log(2)).abs() < 2.0 ** -18).all())


@pytest.mark.parametrize("heads,rows,ctx", [(16, 1, 300000), (16, 4, 100000), (128, 1, 100001)])
def test_long_contexts(cuda_lib, heads, rows, ctx):
    p = ref.attention_problem([rows], [ctx], heads, 64, seed=heads)
    assert check(run(cuda_lib, p), ref.attention(p), p) == 0


@pytest.mark.parametrize("heads", [16, 128])
def test_many_requests(cuda_lib, heads):
    n = 1500 if heads == 16 else 300
    g = torch.Generator().manual_seed(3)
    ctx = torch.randint(0, 300, (n,), generator=g)
    rows = torch.minimum(torch.randint(0, 4, (n,), generator=g), ctx)
    p = ref.attention_problem(rows.tolist(), ctx.tolist(), heads, 16, seed=4)
    assert check(run(cuda_lib, p), ref.attention(p), p) == 0


@pytest.mark.parametrize("heads", [16, 128])
def test_a_padded_batch(cuda_lib, heads):
    """Requests without rows before, between and behind the others, some of them with contexts."""
    rows, ctx = [0] * 4000, [0] * 4000
    for i, n, c in ((7, 1, 300), (8, 2, 40), (16, 1, 1000), (1500, 3, 3), (1501, 1, 129), (2700, 1, 700)):
        rows[i], ctx[i] = n, c
    for i in (0, 9, 15, 1499, 3999):
        ctx[i] = 100
    p = ref.attention_problem(rows, ctx, heads, 16, seed=14, tail=2)
    assert check(run(cuda_lib, p), ref.attention(p), p) == 0
    # the table wide enough for contexts to be cut
    p.bt = torch.cat([p.bt, torch.full((4000, 8), -1, dtype=torch.int32)], 1)
    assert check(run(cuda_lib, p), ref.attention(p), p) == 0


def test_rows_of_no_request_at_all(cuda_lib):
    p = ref.attention_problem([0, 0], [30, 0], 16, 16, seed=15, lead=3)
    assert check(run(cuda_lib, p), ref.attention(p), p) == 0


# ------------------------------------------------------------- shared, strided, empty

@pytest.mark.parametrize("heads", [16, 64, 128])
def test_shared_and_repeated_blocks(cuda_lib, heads):
    """A prefix that two requests share, and a block that a request lists twice."""
    p = ref.attention_problem([2, 3], [200, 260], heads, 16, seed=7, poison=False)
    p.bt[1, :6] = p.bt[0, :6]
    p.bt[1, 9] = p.bt[1, 3]
    assert check(run(cuda_lib, p), ref.attention(p), p) == 0


def test_index_rows_strided_and_in_place(cuda_lib):
    """Keys, queries and weights as slices of one projection, weights scaled where they lie, a key
    and a query that all rows share: the bits of contiguous tensors."""
    lib, heads = cuda_lib, 20
    p = index_case([3, 40], [30, 40], 16, heads, seed=9)
    n = p.total
    fused = torch.cat([p.q.reshape(n, -1), p.k, p.w.to(BF), torch.zeros((n, 4), dtype=BF)], 1).cuda()
    q = fused[:, :heads * 128].view(n, heads, 128)
    k, w = fused[:, heads * 128:heads * 128 + 128], fused[:, heads * 128 + 128:heads * 128 + 128 + heads]
    assert not q.is_contiguous() and not k.is_contiguous() and not w.is_contiguous()
    r, (kv, bt, ctx, rb, most) = rotary(lib), cache(p)
    kv2 = kv.clone()
    a = lib.pmqa_index_append(k, kv, bt, ctx, rb, most, q=q, weights=w, weight_scale=0.5, rotary=r)
    b = lib.pmqa_index_append(p.k.cuda(), kv2, bt, ctx, rb, most, q=p.q.cuda(), weights=w.contiguous(),
                              weight_scale=0.5, rotary=r)
    assert same(a[0], b[0]) and same(a[1], b[1]) and same(kv, kv2)
    w32 = w.float().contiguous()
    c = lib.pmqa_index_append(None, kv, bt, ctx, rb, most, q=p.q.cuda(), weights=w32, weight_scale=0.5, rotary=r,
                              weights_out=w32)
    assert c[1] is w32 and same(w32, a[1])
    one = lib.pmqa_index_append(p.k[:1].cuda().expand(n, 128), kv, bt, ctx, rb, most,
                                q=p.q[:1, :1].cuda().expand(n, heads, 128), weights=w, rotary=r)
    many = lib.pmqa_index_append(p.k[:1].cuda().repeat(n, 1), kv2, bt, ctx, rb, most,
                                 q=p.q[:1, :1].cuda().repeat(n, heads, 1), weights=w, rotary=r)
    assert same(one[0], many[0]) and same(one[1], many[1]) and same(kv, kv2)


def test_latent_rows_strided_or_alone(cuda_lib):
    """Latent and rotary values as slices of one projection, head-major queries, keys or queries
    alone, rows of no request: the bits of one call on contiguous tensors."""
    lib, heads = cuda_lib, 9
    p = latent_case([3, 40], [30, 40], 16, heads, seed=9, lead=2, tail=3)
    r, (kv, bt, ctx, rb, most) = rotary(lib, 32, 16), cache(p)
    kv2, kv3 = kv.clone(), kv.clone()
    qo, qo2 = (torch.full((p.total, heads, 576), 5, dtype=torch.uint8, device="cuda") for _ in range(2))
    args = dict(q_c=p.q_c.cuda(), q_pe=p.q_pe.cuda(), q_scale=p.q_scale, rotary=r)
    lib.pmqa_latent_append(p.c.cuda(), p.k_pe.cuda(), kv, bt, ctx, rb, most, 0.03, q_out=qo, **args)
    assert bool((qo[:2] == 5).all()) and bool((qo[-3:] == 5).all()) and not bool((qo[2:-3] == 5).all(-1).any())
    both = torch.cat([p.c, p.k_pe], 1).cuda()
    turned = p.q_c.transpose(0, 1).contiguous().cuda().transpose(0, 1)
    lib.pmqa_latent_append(both[:, :512], both[:, 512:], kv2, bt, ctx, rb, most, 0.03, q_out=qo2,
                           **{**args, "q_c": turned})
    assert same(qo, qo2) and same(kv, kv2)
    assert lib.pmqa_latent_append(p.c.cuda(), p.k_pe.cuda(), kv3, bt, ctx, rb, most, 0.03, rotary=r) is None
    assert same(kv, kv3)
    alone = lib.pmqa_latent_append(None, None, kv3, bt, ctx, rb, most, 0.03, **args)
    assert same(alone[2:-3], qo[2:-3]) and same(kv, kv3)


def test_latent_rows_saturate_and_keep_nan(cuda_lib):
    lib = cuda_lib
    p = latent_case([4], [4], 16, 1, seed=3)
    for t in (p.c, p.k_pe, p.q_c.view(4, 512), p.q_pe.view(4, 64)):
        t[0, 3], t[1, 5], t[2, 7], t[3, 9] = math.inf, -math.inf, math.nan, 3e38
    kv, bt, ctx, rb, most = cache(p)
    q = lib.pmqa_latent_append(p.c.cuda(), p.k_pe.cuda(), kv, bt, ctx, rb, most, 0.03, q_c=p.q_c.cuda(),
                               q_pe=p.q_pe.cuda(), q_scale=0.02)
    k = ref.value(kv.cpu().reshape(-1, 576)[ref.places(p, 0, 0, 4)])
    for got in (k, ref.value(q.cpu()[:, 0].view(torch.uint8))):
        for base in (0, 512):
            assert got[0, base + 3] == 448 and got[1, base + 5] == -448 and bool(got[2, base + 7].isnan())
            assert got[3, base + 9] == 448
        assert int(got.isnan().sum()) == 2


def test_latent_append_bad_places_are_reported(cuda_lib):
    lib, ws = cuda_lib, cuda_lib.latent_workspace()
    p = latent_case([3, 4], [70, 30], 16, 16, seed=6)
    p.bt[0, 4] = p.nb  # the block of the last rows
    kv, bt, ctx, rb, most = cache(p)
    lib.pmqa_latent_append(p.c.cuda(), p.k_pe.cuda(), kv, bt, ctx, rb, most, 0.03, ws=ws)
    assert lib.pmqa_read_device_status(ws) == lib.PMQA_DEV_BAD_BLOCK_ID
    changed = (kv.cpu() != p.kv).reshape(-1, 576).any(1)
    mine = torch.zeros_like(changed)
    mine[ref.places(p, 1, 26, 30)] = True
    assert torch.equal(changed, mine)
    # fewer tokens than rows, and a context behind the table
    for c, slots in ((1, [0]), (p.bt.shape[1] * 16 + 2, [p.bt.shape[1] * 16 - 1])):
        p = latent_case([3, 4], [70, 30], 16, 16, seed=6)
        p.bt[0] = torch.arange(p.bt.shape[1])
        p.ctx[0] = c
        kv, bt, ctx, rb, most = cache(p)
        rb[2] = 3
        lib.pmqa_latent_append(p.c.cuda(), p.k_pe.cuda(), kv, bt, ctx, rb, most, 0.03, ws=ws)
        assert lib.pmqa_read_device_status(ws) == lib.PMQA_DEV_BAD_CONTEXT
        changed = (kv.cpu() != p.kv).reshape(-1, 576).any(1)
        assert changed.nonzero().flatten().tolist() == slots


def test_rope_of_two_shapes_one_in_place(cuda_lib):
    """Wide heads rotated where they lie beside narrow ones into a new tensor, and the other way
    round; many heads of one row."""
    lib = cuda_lib
    g = torch.Generator().manual_seed(3)
    pos = torch.randint(0, 9000, (6,), generator=g, dtype=torch.int32)
    a, b = torch.randn((6, 5, 192), generator=g).to(BF), torch.randn((6, 2, 64), generator=g).to(BF)
    r = rotary(lib, 32, 16, False)
    want = [lib.pmqa_rope(t.cuda(), pos.cuda(), r) for t in (a, b)]
    x, y = a.cuda(), b.cuda()
    got = lib.pmqa_rope(x, pos.cuda(), r, other=y, out=x)
    assert got[0] is x and all(same(s, t) for s, t in zip(got, want)) and torch.equal(y.cpu(), b)
    x = a.cuda()
    got = lib.pmqa_rope(x, pos.cuda(), r, other=y, other_out=y)
    assert got[1] is y and all(same(s, t) for s, t in zip(got, want)) and torch.equal(x.cpu(), a)
    many = torch.randn((1, 5000, 64), generator=g).to(BF)
    got = lib.pmqa_rope(many.cuda(), pos[:1].cuda(), r)
    z, e = ref.rotate(many.double(), pos[:1], r.inv_freq.cpu(), 16, False, r.scale)
    assert bool(((got.cpu().double() - z).abs() <= e + (z.abs() + e) * 2.0 ** -8).all())


def test_no_rows(cuda_lib):
    lib = cuda_lib
    i, l = index_case([0, 0], [50, 9], 16, 64, seed=1), latent_case([0, 0], [50, 9], 16, 16, seed=2)
    ic, lc, r = cache(i), cache(l), rotary(lib)
    q, w = lib.pmqa_index_append(i.k.cuda(), *ic, q=i.q.cuda(), weights=i.w.cuda(), rotary=r)
    assert q.shape == (0, 64, 128) and w.shape == (0, 64) and torch.equal(ic[0].cpu(), i.kv)
    k, s = lib.pmqa_index_read(ic[0], ic[1], ic[3], 0)
    assert k.shape == (0, 128) and s.shape == (0,)
    lq = lib.pmqa_latent_append(l.c.cuda(), l.k_pe.cuda(), *lc, 0.03, q_c=l.q_c.cuda(), q_pe=l.q_pe.cuda(), rotary=r)
    out, lse = lib.pmqa_latent_attention(lq, *lc, 0.02, 0.03, 0.07, want_lse=True)
    assert out.shape == (0, 16, 512) and lse.shape == (0, 16) and torch.equal(lc[0].cpu(), l.kv)
    assert lib.pmqa_rope(i.q.cuda(), torch.zeros(0, dtype=torch.int32).cuda(), r).shape == (0, 64, 128)
