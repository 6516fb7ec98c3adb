"""Rope, index append and read, and latent append against their 64-bit forms."""

import math

import pytest
import torch

from tests import step_ref as ref

pytestmark = pytest.mark.gpu

PARTS = dict(kind=2, factor=40.0, trained=4096.0)


def frequencies(pmqa, dim, base=10000.0, **kw):
    f, scale = pmqa.rope_frequencies(dim, base, **kw)
    return f, scale


# ------------------------------------------------------------------ rope

@pytest.mark.parametrize("rows,heads,head_dim,dim,begin", [
    (1, 1, 16, 16, 0), (3, 2, 64, 64, 0), (5, 3, 192, 64, 128), (2, 40, 128, 128, 0), (7, 1, 80, 16, 24),
    (9, 2, 96, 32, 64), (1, 64, 576, 64, 512), (3, 2, 1024, 1024, 0), (2500, 2, 32, 32, 0), (4, 0, 64, 64, 0),
])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_against_the_64_bit_form(cuda_lib, rows, heads, head_dim, dim, begin, interleaved):
    g = torch.Generator().manual_seed(rows + heads)
    x = torch.randn((rows, heads, head_dim), generator=g).to(torch.bfloat16)
    k = torch.randn((rows, 2, head_dim), generator=g).to(torch.bfloat16)
    pos = torch.randint(0, 200000, (rows,), generator=g, dtype=torch.int32)
    f, scale = frequencies(cuda_lib, dim, **(PARTS if rows % 2 else {}))
    r = cuda_lib.Rotary(f, begin, interleaved, scale)
    got = cuda_lib.pmqa_rope(x.cuda(), pos.cuda(), r, other=k.cuda())
    for t, y in zip((x, k), got):
        want, e = ref.rotate(t.double(), pos, f.cpu(), begin, interleaved, scale)
        outside = torch.ones(head_dim, dtype=torch.bool)
        outside[begin:begin + dim] = False
        assert torch.equal(y.cpu()[..., outside], t[..., outside])
        assert bool(((y.cpu().double() - want).abs() <= e + (want.abs() + e) * 2.0 ** -8).all())


def test_rope_at_far_and_negative_positions(cuda_lib):
    """No accuracy is lost at 2^31 - 1, and turning back undoes a turn."""
    g = torch.Generator().manual_seed(1)
    pos = torch.tensor([2 ** 31 - 1, -2 ** 31, -1, 0, 1 << 30, 12345678], dtype=torch.int32)
    x = torch.randn((6, 4, 64), generator=g).to(torch.bfloat16)
    f, _ = frequencies(cuda_lib, 64)
    y = cuda_lib.pmqa_rope(x.cuda(), pos.cuda(), cuda_lib.Rotary(f))
    want, e = ref.rotate(x.double(), pos, f.cpu())
    # the frequency itself is known to 2^-53: 2^31 positions make that 2^-22 of a radian
    e = e + (want.abs().amax() * 2) * 2.0 ** -21
    assert bool(((y.cpu().double() - want).abs() <= e + (want.abs() + e) * 2.0 ** -8).all())
    back = cuda_lib.pmqa_rope(y, (-pos).cuda(), cuda_lib.Rotary(f))
    big = x.double().abs().amax() * 2
    off = (back.cpu().double() - x.double()).abs()
    there = pos != -2 ** 31  # whose negative is no int32
    assert bool((off[there] <= big * (2.0 ** -7 + 2.0 ** -18)).all())


def test_rope_in_place_and_strided(cuda_lib):
    """Queries and keys in one fused projection, rotated where they lie; a head-major result."""
    g = torch.Generator().manual_seed(2)
    fused = torch.randn((33, 7, 128), generator=g).to(torch.bfloat16)
    pos = torch.arange(33, dtype=torch.int32)
    f, _ = frequencies(cuda_lib, 64)
    r = cuda_lib.Rotary(f, 32)
    want, e = ref.rotate(fused.double(), pos, f.cpu(), 32)
    d = fused.cuda()
    q, k = d[:, :5], d[:, 5:6]
    out = cuda_lib.pmqa_rope(q, pos.cuda(), r, other=k, out=q, other_out=k)
    assert out[0].data_ptr() == d.data_ptr()
    y = d.cpu()
    assert torch.equal(y[:, 6], fused[:, 6])  # the values beside them
    ok = (y.double() - want).abs() <= e + (want.abs() + e) * 2.0 ** -8
    assert bool(ok[:, :6].all())
    o = torch.zeros((5, 33, 128), dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    cuda_lib.pmqa_rope(fused.cuda()[:, :5], pos.cuda(), r, out=o)
    assert torch.equal(o.cpu(), y[:, :5])


def test_rope_keeps_infinities_and_nan_in_their_pairs(cuda_lib):
    x = torch.ones((2, 1, 64), dtype=torch.bfloat16)
    x[0, 0, 3], x[0, 0, 50], x[1, 0, 9] = math.inf, math.inf, math.nan
    f, _ = frequencies(cuda_lib, 32)
    y = cuda_lib.pmqa_rope(x.cuda(), torch.tensor([5, 6], dtype=torch.int32).cuda(), cuda_lib.Rotary(f)).cpu()
    fine = torch.ones((2, 64), dtype=torch.bool)
    fine[0, [3, 19]] = fine[1, [9, 25]] = False
    fine[0, 50] = False
    assert y[0, 0, 50] == math.inf and bool(y[:, 0][fine].isfinite().all())
    assert not bool(y[0, 0, [3, 19]].isfinite().any()) and bool(y[1, 0, [9, 25]].isnan().all())


# ------------------------------------------------------------------ index

def index_case(rows, ctx, block, heads, seed=0, **kw):
    p = ref.layout(rows, ctx, block, seed, **kw)
    g = p.gen
    p.kv = torch.randint(0, 256, (p.nb, block, 132), generator=g, dtype=torch.uint8)
    p.k = torch.randn((p.total, 128), generator=g).to(torch.bfloat16)
    p.q = (torch.randn((p.total, heads, 128), generator=g) * 3).to(torch.bfloat16)
    p.w = torch.randn((p.total, heads), generator=g)
    p.weight, p.bias = 1 + 0.1 * torch.randn(128, generator=g), 0.1 * torch.randn(128, generator=g)
    return p


def check_codes(code, scale, y, e):
    """Codes and scales of rows y (64 bits, off by e in the kernel)."""
    top = y.abs().amax(-1).clamp(min=ref.TINY)
    et = e.amax(-1)
    assert bool(((scale - top / 448).abs() <= et / 448 + top * 2.0 ** -22).all())
    x, tol = ref.coded(y, e + (et + top * 2.0 ** -22)[..., None] * (y.abs() / top[..., None]), 448 / top[..., None])
    assert bool(((code - x).abs() <= tol).all()), float(((code - x).abs() / tol).max())


def index_check(pmqa, p, kind, interleaved, begin, dim, positions=None, bf16=False):
    f, scale = frequencies(pmqa, dim, **PARTS)
    r = pmqa.Rotary(f, begin, interleaved, scale)
    norm = pmqa.Norm(kind, p.weight.cuda(), p.bias.cuda() if kind == 1 else None)
    kv, ws = p.kv.cuda(), pmqa.workspace(1, 1, 1, 0, pmqa.PMQA_OP_LOGITS)
    w = p.w.to(torch.bfloat16) if bf16 else p.w
    heads = p.q.shape[1]
    qo = torch.full((p.total, heads, 128), 7, dtype=torch.uint8, device="cuda")
    wo = torch.full((p.total, heads), 7.0, device="cuda")
    pmqa.pmqa_index_append(p.k.cuda(), kv, p.bt.cuda(), p.ctx.cuda(), p.rb.cuda(), p.max_rows, q=p.q.cuda(),
                           weights=w.cuda(), weight_scale=0.25, norm=norm, rotary=r,
                           positions=None if positions is None else positions.cuda(), q_out=qo, weights_out=wo, ws=ws)
    assert pmqa.pmqa_read_device_status(ws) == 0
    rows = torch.tensor([r for r, _, _ in ref.slots(p)], dtype=torch.long)
    slot = torch.tensor([t for _, _, t in ref.slots(p)], dtype=torch.int32)
    pos = slot if positions is None else positions[rows]
    at = torch.cat([ref.places(p, i, t, t + 1) for _, i, t in ref.slots(p)])
    y, e0 = ref.norm(p.k[rows].double(), kind, p.weight, p.bias if kind == 1 else None, 1e-6)
    z, e = ref.rotate(y[:, None], pos, f.cpu(), begin, interleaved, scale)
    e = e[:, 0] + 2 * abs(scale) * e0.amax(-1, keepdim=True)
    got = kv.cpu().reshape(-1, 132)
    check_codes(ref.value(got[at, :128].contiguous()), got[at, 128:].contiguous().view(torch.float32)[:, 0].double(), z[:, 0], e)
    other = torch.ones(got.shape[0], dtype=torch.bool)
    other[at] = False
    assert torch.equal(got[other], p.kv.reshape(-1, 132)[other]), "slots without a new key"
    z, e = ref.rotate(p.q[rows].double(), pos, f.cpu(), begin, interleaved, scale)
    s = wo.cpu()[rows].double() / (w[rows].double() * 0.25)
    check_codes(ref.value(qo.cpu()[rows]), s, z, e)
    none = torch.ones(p.total, dtype=torch.bool)
    none[rows] = False
    assert bool((qo.cpu()[none] == 7).all()) and bool((wo.cpu()[none] == 7).all()), "rows of no request"


@pytest.mark.parametrize("kind", [0, 1, 2])
@pytest.mark.parametrize("interleaved,begin,dim", [(False, 0, 64), (True, 0, 64), (False, 64, 64), (True, 32, 16),
                                                   (False, 0, 128), (False, 8, 112)])
def test_index_append(cuda_lib, kind, interleaved, begin, dim):
    p = index_case([3, 1, 0, 5], [70, 1, 9, 300], 16, 64, seed=dim, lead=2, tail=1)
    index_check(cuda_lib, p, kind, interleaved, begin, dim)


@pytest.mark.parametrize("rows,ctx,block,heads", [([1], [1], 1, 16), ([4] * 9, [4 + 37 * i for i in range(9)], 1, 5),
                                                  ([600, 1, 1900], [700, 4, 1900], 64, 3), ([2], [200], 256, 128),
                                                  ([1] * 40, [1 + 3 * i for i in range(40)], 3, 32)])
def test_index_append_sizes(cuda_lib, rows, ctx, block, heads):
    p = index_case(rows, ctx, block, heads, seed=heads)
    index_check(cuda_lib, p, 1, True, 0, 64, bf16=heads == 5)


def test_index_append_positions(cuda_lib):
    """Positions that are not the slots (a cache that tokens were evicted from)."""
    p = index_case([3, 4], [70, 30], 16, 16, seed=3)
    index_check(cuda_lib, p, 1, False, 0, 64, positions=torch.randint(-5, 10 ** 6, (p.total,), dtype=torch.int32))


def test_index_append_keys_or_queries_alone(cuda_lib):
    p = index_case([3, 4], [70, 30], 16, 16, seed=4)
    d = [t.cuda() for t in (p.bt, p.ctx, p.rb)]
    both = p.kv.cuda()
    q, w = cuda_lib.pmqa_index_append(p.k.cuda(), both, *d, p.max_rows, q=p.q.cuda(), weights=p.w.cuda())
    one = p.kv.cuda()
    assert cuda_lib.pmqa_index_append(p.k.cuda(), one, *d, p.max_rows) is None
    assert torch.equal(one, both)
    q1, w1 = cuda_lib.pmqa_index_append(None, one, *d, p.max_rows, q=p.q.cuda(), weights=p.w.cuda())
    assert torch.equal(one, both) and torch.equal(q1.view(torch.uint8), q.view(torch.uint8)) and torch.equal(w1, w)
    # weights in place, strided rows
    wide = torch.zeros((p.total, 3, 128), dtype=torch.bfloat16)
    wide[:, 1] = p.k
    w2 = p.w.cuda()
    two = p.kv.cuda()
    cuda_lib.pmqa_index_append(wide.cuda()[:, 1], two, *d, p.max_rows, q=p.q.cuda(), weights=w2, weights_out=w2)
    assert torch.equal(two, both) and torch.equal(w2, w)


def test_index_append_infinities_nan_and_zeros(cuda_lib):
    p = index_case([4], [4], 4, 16, seed=5)
    p.k[0] = 0.0
    p.k[1, 7], p.k[1, 8] = math.inf, -math.inf
    p.k[2, 3] = math.nan
    p.k[3] = math.inf
    kv = p.kv.cuda()
    cuda_lib.pmqa_index_append(p.k.cuda(), kv, p.bt.cuda(), p.ctx.cuda(), p.rb.cuda(), 4)
    got = kv.cpu().reshape(-1, 132)[ref.places(p, 0, 0, 4)]
    code, s = ref.value(got[:, :128].contiguous()), got[:, 128:].contiguous().view(torch.float32)[:, 0]
    tiny = torch.tensor(2.0 ** -100 / 448).float()
    assert bool((code[0] == 0).all()) and bool(s[0] == tiny)
    assert code[1, 7] == 448 and code[1, 8] == -448
    fine = p.k[1].double()
    fine[[7, 8]] = 0.0
    assert bool(((code[1] * s[1] - fine).abs()[[i for i in range(128) if i not in (7, 8)]] <=
                 float(fine.abs().max()) * 2.0 ** -4).all())
    assert bool(code[2, 3].isnan()) and int(code[2].isnan().sum()) == 1 and math.isfinite(s[2])
    assert bool((code[3] == 448).all()) and bool(s[3] == tiny)


def test_index_append_at_the_ends_of_the_range(cuda_lib):
    """The largest finite bf16 values, whose quotient's factor is below 2^-119, and the least."""
    pmqa = cuda_lib
    p = index_case([6], [6], 16, 3, seed=8)
    for t in (p.k, p.q.view(-1, 128)):
        for r, a in enumerate((3.38e38, 1.2e38, 8.6e37, 1e37, 1e-38, 1e-29)):
            t[r] = (t[r].float() / t[r].float().abs().amax() * a).to(torch.bfloat16)
    kv, qo, wo = p.kv.cuda(), *(torch.empty(s, dtype=d, device="cuda") for s, d in (
        ((6, 3, 128), torch.uint8), ((6, 3), torch.float32)))
    pmqa.pmqa_index_append(p.k.cuda(), kv, p.bt.cuda(), p.ctx.cuda(), p.rb.cuda(), 6, q=p.q.cuda(),
                           weights=torch.ones((6, 3)).cuda(), q_out=qo, weights_out=wo)
    got = kv.cpu().reshape(-1, 132)[ref.places(p, 0, 0, 6)]
    y = p.k.double()
    check_codes(ref.value(got[:, :128].contiguous()), got[:, 128:].contiguous().view(torch.float32)[:, 0].double(), y,
                torch.zeros_like(y))
    y = p.q.double()
    check_codes(ref.value(qo.cpu()), wo.cpu().double(), y, torch.zeros_like(y))


def test_index_append_bad_places_are_reported(cuda_lib):
    pmqa = cuda_lib
    ws = pmqa.workspace(1, 1, 1, 0, pmqa.PMQA_OP_LOGITS)
    p = index_case([3, 4], [70, 30], 16, 16, seed=6)
    p.bt[0, 4] = p.nb  # the block of the last rows
    kv = p.kv.cuda()
    q, w = pmqa.pmqa_index_append(p.k.cuda(), kv, p.bt.cuda(), p.ctx.cuda(), p.rb.cuda(), 4, q=p.q.cuda(),
                                  weights=p.w.cuda(), ws=ws)
    assert pmqa.pmqa_read_device_status(ws) == pmqa.PMQA_DEV_BAD_BLOCK_ID
    changed = (kv.cpu() != p.kv).reshape(-1, 132).any(1)
    mine = torch.zeros_like(changed)
    mine[ref.places(p, 1, 26, 30)] = True
    assert torch.equal(changed, mine)
    # fewer tokens than rows: the rows before slot 0 write no key
    p = index_case([3], [3], 16, 16, seed=6)
    p.ctx = torch.tensor([1], dtype=torch.int32)
    kv = p.kv.cuda()
    pmqa.pmqa_index_append(p.k.cuda(), kv, p.bt.cuda(), p.ctx.cuda(), p.rb.cuda(), 3, ws=ws)
    assert pmqa.pmqa_read_device_status(ws) == pmqa.PMQA_DEV_BAD_CONTEXT
    changed = (kv.cpu() != p.kv).reshape(-1, 132).any(1)
    assert changed.nonzero().flatten().tolist() == ref.places(p, 0, 0, 1).tolist()
    # rows past max_rows
    p = index_case([5], [5], 16, 16, seed=7)
    kv = p.kv.cuda()
    pmqa.pmqa_index_append(p.k.cuda(), kv, p.bt.cuda(), p.ctx.cuda(), p.rb.cuda(), 2, ws=ws)
    assert pmqa.pmqa_read_device_status(ws) == pmqa.PMQA_DEV_BAD_CONTEXT
    changed = (kv.cpu() != p.kv).reshape(-1, 132).any(1)
    assert sorted(changed.nonzero().flatten().tolist()) == sorted(ref.places(p, 0, 0, 2).tolist())


# ------------------------------------------------------------------ read

@pytest.mark.parametrize("lens,block", [([1], 1), ([5, 0, 33, 1], 16), ([300, 1, 1, 700], 1), ([64, 65, 63], 64),
                                        ([1] * 70, 3), ([200000], 64)])
@pytest.mark.parametrize("offset", [0, 3])
def test_index_read(cuda_lib, lens, block, offset):
    p = ref.layout(lens, [n + offset for n in lens], block, seed=len(lens), lead=2, tail=3)
    p.kv = torch.randint(0, 256, (p.nb, block, 132), generator=p.gen, dtype=torch.uint8)
    ws = cuda_lib.workspace(1, 1, 1, 0, cuda_lib.PMQA_OP_LOGITS)
    k = torch.full((p.total, 128), 9, dtype=torch.uint8, device="cuda")
    s = torch.full((p.total,), 9.0, device="cuda")
    start = torch.full((p.bs,), offset, dtype=torch.int32).cuda() if offset else None
    cuda_lib.pmqa_index_read(p.kv.cuda(), p.bt.cuda(), p.rb.cuda(), p.total, start=start, k=k, k_scale=s, ws=ws)
    assert cuda_lib.pmqa_read_device_status(ws) == 0
    at = torch.cat([ref.places(p, i, offset, offset + n) for i, n in enumerate(lens)])
    want = p.kv.reshape(-1, 132)[at]
    k, s = k.cpu(), s.cpu()
    assert torch.equal(k[2:-3], want[:, :128]) and torch.equal(s.view(torch.int32)[2:-3], want[:, 128:].contiguous().view(torch.int32)[:, 0])
    assert bool((k[:2] == 9).all()) and bool((k[-3:] == 9).all()) and bool((s[-3:] == 9).all())


def test_index_read_bad_places_give_zeros(cuda_lib):
    p = ref.layout([40, 20], [40, 20], 8, seed=1)
    p.kv = torch.randint(1, 256, (p.nb, 8, 132), generator=p.gen, dtype=torch.uint8)
    want = [p.kv.reshape(-1, 132)[ref.places(p, i, 0, n), :128] for i, n in enumerate((40, 20))]
    want[0][8:16] = 0
    p.bt[0, 1] = -3
    ws = cuda_lib.workspace(1, 1, 1, 0, cuda_lib.PMQA_OP_LOGITS)
    k, s = cuda_lib.pmqa_index_read(p.kv.cuda(), p.bt.cuda(), p.rb.cuda(), 60, ws=ws)
    assert cuda_lib.pmqa_read_device_status(ws) == cuda_lib.PMQA_DEV_BAD_BLOCK_ID
    assert torch.equal(k.cpu().view(torch.uint8), torch.cat(want)) and bool((s.cpu()[8:16] == 0).all())
    start = torch.tensor([0, -2], dtype=torch.int32).cuda()
    k, s = cuda_lib.pmqa_index_read(p.kv.cuda(), p.bt.cuda(), p.rb.cuda(), 60, start=start, ws=ws)
    assert cuda_lib.pmqa_read_device_status(ws) == cuda_lib.PMQA_DEV_BAD_BLOCK_ID | cuda_lib.PMQA_DEV_BAD_CONTEXT
    assert bool((k.cpu().view(torch.uint8)[40:42] == 0).all()) and torch.equal(k.cpu().view(torch.uint8)[42:], want[1][:18])


# ------------------------------------------------------------------ latent

@pytest.mark.parametrize("rows,ctx,block,heads", [([1], [1], 1, 16), ([3, 1, 0, 5], [70, 1, 9, 300], 16, 5),
                                                  ([4] * 9, [4 + 37 * i for i in range(9)], 1, 128),
                                                  ([700, 1, 1900], [700, 4, 2000], 64, 2)])
@pytest.mark.parametrize("kind,interleaved,begin,dim", [(0, False, 0, 64), (1, True, 0, 64), (2, False, 0, 64),
                                                        (2, True, 16, 32), (2, False, 8, 48)])
def test_latent_append(cuda_lib, rows, ctx, block, heads, kind, interleaved, begin, dim):
    pmqa = cuda_lib
    p = ref.layout(rows, ctx, block, seed=heads, lead=1, tail=2)
    g = p.gen
    p.kv = torch.randint(0, 256, (p.nb, block, 576), generator=g, dtype=torch.uint8)
    new = torch.randn((p.total, 576), generator=g).to(torch.bfloat16)
    qc = (torch.randn((p.total, heads, 512), generator=g) * 8).to(torch.bfloat16)
    qp = (torch.randn((p.total, heads, 64), generator=g) * 8).to(torch.bfloat16)
    weight, bias = 1 + 0.1 * torch.randn(512, generator=g), 0.1 * torch.randn(512, generator=g)
    f, scale = frequencies(pmqa, dim, **PARTS)
    kv, ws, dnew = p.kv.cuda(), pmqa.latent_workspace(), new.cuda()
    qo = torch.full((p.total, heads, 576), 7, dtype=torch.uint8, device="cuda")
    ks, qs = 0.011, 0.05  # the largest queries saturate
    pmqa.pmqa_latent_append(dnew[:, :512], dnew[:, 512:], kv, p.bt.cuda(), p.ctx.cuda(), p.rb.cuda(), p.max_rows,
                            ks, q_c=qc.cuda(), q_pe=qp.cuda(), q_scale=qs,
                            norm=pmqa.Norm(kind, weight.cuda(), bias.cuda() if kind == 1 else None),
                            rotary=pmqa.Rotary(f, begin, interleaved, scale), q_out=qo, ws=ws)
    assert pmqa.pmqa_read_device_status(ws) == 0
    sl = ref.slots(p)
    r = torch.tensor([x for x, _, _ in sl], dtype=torch.long)
    pos = torch.tensor([t for _, _, t in sl], dtype=torch.int32)
    at = torch.cat([ref.places(p, i, t, t + 1) for _, i, t in sl])
    c, e = ref.norm(new[r, :512].double(), kind, weight, bias if kind == 1 else None, 1e-6)
    pe, e2 = ref.rotate(new[r, None, 512:].double(), pos, f.cpu(), begin, interleaved, scale)
    y, e = torch.cat((c, pe[:, 0]), 1), torch.cat((e, e2[:, 0]), 1)
    got = kv.cpu().reshape(-1, 576)
    want, tol = ref.coded(y, e, 1 / torch.tensor(ks).float().double())
    assert bool(((ref.value(got[at]) - want).abs() <= tol).all())
    other = torch.ones(got.shape[0], dtype=torch.bool)
    other[at] = False
    assert torch.equal(got[other], p.kv.reshape(-1, 576)[other])
    pe, e2 = ref.rotate(qp[r].double(), pos, f.cpu(), begin, interleaved, scale)
    y, e = torch.cat((qc[r].double(), pe), 2), torch.cat((torch.zeros(qc[r].shape, dtype=torch.float64), e2), 2)
    want, tol = ref.coded(y, e, 1 / torch.tensor(qs).float().double())
    assert bool(((ref.value(qo.cpu()[r]) - want).abs() <= tol).all())
    none = torch.ones(p.total, dtype=torch.bool)
    none[r] = False
    assert bool((qo.cpu()[none] == 7).all())
