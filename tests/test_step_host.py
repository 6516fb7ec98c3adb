"""Host-only checks of the operators around the sparse-MLA step: what the C ABI
refuses before it touches the device, what the binding refuses, and the rotary
frequencies against their formulas."""

import ctypes
import math

import pytest
import torch

from sparse_attention_indexer_pmqa_gb300 import build, pmqa

OK, INV, UNS, SPACE = (pmqa.PMQA_OK, pmqa.PMQA_ERR_INVALID_ARG, pmqa.PMQA_ERR_UNSUPPORTED,
                       pmqa.PMQA_ERR_WORKSPACE)
WS = 0x100000
INF, NAN = math.inf, math.nan


@pytest.fixture(scope="module")
def lib():
    build.build()
    return pmqa.load()


# fake, suitably aligned device addresses: argument checks run before any CUDA call

def fill(cls, base, kw):
    for k in kw:
        assert k in base, k
    return cls(**{**base, **kw})


def paged(**kw):
    return fill(pmqa.PagedRows, dict(block_tables=0xA0000, context_lens=0xB0000, row_begin=0xC0000, bs=2,
                                     block_size=16, max_blocks_per_seq=8, rows=4, max_rows=3, num_blocks=32), kw)


def rotary(**kw):
    return fill(pmqa.RotaryArgs, dict(inv_freq=0xD0000, positions=0xD8000, dim=64, begin=0, interleaved=0,
                                      scale=1.0), kw)


def norm(**kw):
    return fill(pmqa.NormArgs, dict(kind=1, eps=1e-6, weight=0xE0000, bias=0xE8000), kw)


def heads(**kw):
    return fill(pmqa.Heads, dict(x=0x1000000, out=0x2000000, x_row=512, x_head=128, out_row=512, out_head=128,
                                 heads=4, head_dim=128), kw)


def index_rows(**kw):
    return fill(pmqa.IndexRows, dict(k=0x1000000, q=0x2000000, weights=0x3000000, q_out=0x4000000,
                                     weights_out=0x5000000, k_row=128, q_row=512, q_head=128, weights_row=4,
                                     heads=4, weights_bf16=0, weight_scale=1.0), kw)


def latent_rows(**kw):
    return fill(pmqa.LatentRows, dict(c=0x1000000, k_pe=0x2000000, q_c=0x3000000, q_pe=0x4000000,
                                      q_out=0x5000000, c_row=512, pe_row=64, q_c_row=2048, q_c_head=512,
                                      q_pe_row=256, q_pe_head=64, heads=4, kv_scale=0.1, q_scale=0.1), kw)


def ref(x):
    return None if x is None else ctypes.byref(x)


def rope(lib, r=None, rows=4, a=None, b=None):
    return lib.pmqa_rope(ref(r or rotary()), rows, ref(a or heads()), ref(b), None)


def index_append(lib, p=None, x=None, kv=0x6000000, n=None, r=None, ws=WS, size=256):
    return lib.pmqa_index_append(ref(p or paged()), kv, ref(x or index_rows()), ref(n), ref(r), ws, size, None)


def index_read(lib, p=None, kv=0x6000000, start=None, k=0x7000000, s=0x8000000, ws=WS, size=256):
    return lib.pmqa_index_read(ref(p or paged()), kv, start, k, s, ws, size, None)


def latent_append(lib, p=None, x=None, kv=0x6000000, n=None, r=None, ws=WS, size=256):
    return lib.pmqa_latent_append(ref(p or paged()), kv, ref(x or latent_rows()), ref(n), ref(r), ws, size, None)


def attention(lib, p=None, q=0x1000000, kv=0x6000000, heads=8, qs=0.1, ks=0.1, sm=0.1, out=0x7000000, lse=None,
              ws=WS, size=None):
    return lib.pmqa_latent_attention(ref(p or paged()), q, kv, heads, qs, ks, sm, out, lse, ws,
                                     pmqa.pmqa_latent_workspace_bytes() if size is None else size, None)


APPENDS = [index_append, latent_append]
CALLS = APPENDS + [index_read, attention]


@pytest.mark.parametrize("call", CALLS)
def test_rows_and_workspace(lib, call):
    for kw, code in [(dict(bs=-1), INV), (dict(block_size=0), INV), (dict(max_blocks_per_seq=0), INV),
                     (dict(rows=-1), INV), (dict(num_blocks=0), INV), (dict(block_tables=None), INV),
                     (dict(block_tables=0xA0002), INV), (dict(row_begin=None), INV), (dict(row_begin=0xC0001), INV),
                     (dict(bs=1 << 20, max_blocks_per_seq=1 << 11), UNS), (dict(num_blocks=(1 << 32) // 16), UNS),
                     (dict(num_blocks=1 << 60), UNS)]:
        assert call(lib, paged(**kw)) == code, kw
    lens = [(dict(max_rows=0), INV), (dict(context_lens=None), INV), (dict(context_lens=0xB0002), INV)]
    if call is not index_read:  # which has no lengths
        for kw, code in lens:
            assert call(lib, paged(**kw)) == code, kw
    assert call(lib, ws=None) == INV and call(lib, ws=WS + 128) == INV
    assert call(lib, size=255) == SPACE and call(lib, size=0) == SPACE
    if call is attention:
        assert call(lib, size=pmqa.pmqa_latent_workspace_bytes() - 1) == SPACE
    # nothing to do: no device work, pointers not looked at
    for kw in (dict(bs=0), dict(rows=0)):
        assert call(lib, paged(block_tables=None, row_begin=None, context_lens=None, **kw)) == OK


@pytest.mark.parametrize("call", [rope, *APPENDS])
@pytest.mark.parametrize("kw,code", [
    (dict(dim=-16), INV), (dict(begin=-8), INV), (dict(begin=72), INV), (dict(dim=1040), INV),
    (dict(scale=INF), INV), (dict(scale=NAN), INV), (dict(interleaved=2), INV), (dict(inv_freq=None), INV),
    (dict(inv_freq=0xD0004), INV), (dict(positions=0xD8002), INV), (dict(dim=24), UNS), (dict(dim=8), UNS),
    (dict(dim=48, begin=4), UNS),
])
def test_rotary(lib, call, kw, code):
    assert call(lib, r=rotary(**kw)) == code


@pytest.mark.parametrize("call", APPENDS)
@pytest.mark.parametrize("kw", [dict(kind=3), dict(kind=-1), dict(eps=-1e-6), dict(eps=INF), dict(eps=NAN),
                                dict(weight=0xE0008), dict(bias=0xE0004)])
def test_norm(lib, call, kw):
    assert call(lib, n=norm(**kw)) == INV


def test_rope(lib):
    assert lib.pmqa_rope(None, 4, ref(heads()), None, None) == INV
    assert lib.pmqa_rope(ref(rotary()), 4, None, None, None) == INV
    assert rope(lib, rows=-1) == INV
    assert rope(lib, rotary(positions=None)) == INV
    assert rope(lib, rotary(dim=64, begin=72), b=heads(x=0x3000000, out=0x4000000)) == INV  # 136 > 128
    for kw, code in [
            (dict(heads=-1), INV), (dict(head_dim=0), INV), (dict(head_dim=132), UNS), (dict(head_dim=1032), UNS),
            (dict(heads=1 << 25, x_head=0, out_row=1 << 40), UNS),
            (dict(x=None), INV), (dict(x=0x1000008), INV), (dict(out=None), INV), (dict(out=0x2000008), INV),
            (dict(x_row=4), INV), (dict(x_row=-512), INV), (dict(x_head=12), INV), (dict(x_head=-128), INV),
            (dict(out_row=0), INV), (dict(out_head=64), INV), (dict(out_head=0), INV),
            (dict(out_row=136), INV),  # into the next row's second head
            (dict(out=0x1000000, out_row=1024), INV),  # in place with other strides
            (dict(out=0x1000100), INV), (dict(out=0x1000000 - 256), INV),  # overlapping in part
            (dict(x_row=1 << 62), INV), (dict(out_head=1 << 62), INV)]:
        assert rope(lib, a=heads(**kw)) == code, kw
        assert rope(lib, b=heads(**kw)) == code, kw
    # one tensor's result where the other's begins
    assert rope(lib, b=heads(x=0x3000000)) == INV
    assert rope(lib, b=heads(x=0x2000000, out=0x4000000)) == INV
    assert rope(lib, b=heads(x=0x3000000, out=0x1000000)) == INV
    # narrower heads beside wide ones: the rotated part has to fit both
    assert rope(lib, rotary(dim=128), b=heads(head_dim=64, x=0x3000000, out=0x4000000)) == INV
    # nothing to do
    assert rope(lib, rows=0, a=heads(x=None, out=None)) == OK
    assert rope(lib, a=heads(heads=0, x=None, out=None)) == OK
    assert rope(lib, rotary(dim=0, inv_freq=None, positions=None), a=heads(out=0x1000000)) == OK


def test_index_append(lib):
    p = paged()
    assert lib.pmqa_index_append(ref(p), 0x6000000, None, None, None, WS, 256, None) == INV
    assert lib.pmqa_index_append(None, 0x6000000, ref(index_rows()), None, None, WS, 256, None) == INV
    for kw, code in [
            (dict(k=0x1000008), INV), (dict(k_row=-128), INV), (dict(k_row=132), INV), (dict(q=0x2000008), INV),
            (dict(q_row=4), INV), (dict(q_head=-128), INV), (dict(q_out=None), INV), (dict(q_out=0x4000004), INV),
            (dict(weights=None), INV), (dict(weights=0x3000002), INV), (dict(weights_bf16=1, weights=0x3000001), INV),
            (dict(weights_out=None), INV), (dict(weights_out=0x5000002), INV), (dict(weights_row=-4), INV),
            (dict(heads=0), INV), (dict(heads=65536, weights_row=65536), UNS), (dict(weight_scale=INF), INV),
            (dict(weight_scale=NAN), INV),
            (dict(weights_out=0x3000000, weights_row=8), INV), (dict(weights_out=0x3000004), INV),
            (dict(weights_out=0x3000000, weights_bf16=1), INV)]:
        assert index_append(lib, x=index_rows(**kw)) == code, kw
    assert index_append(lib, kv=None) == INV and index_append(lib, kv=0x6000002) == INV
    assert index_append(lib, paged(rows=1 << 17), index_rows(heads=1 << 14)) == UNS  # 2^31 query heads
    # no keys and no queries
    assert index_append(lib, x=index_rows(k=None, q=None), kv=None) == OK
    # a bad rotary part is refused whatever there is to do
    assert index_append(lib, paged(rows=0), r=rotary(dim=-1)) == INV


def test_index_read(lib):
    assert index_read(lib, kv=None) == INV and index_read(lib, kv=0x6000002) == INV
    assert index_read(lib, start=0x9000002) == INV
    assert index_read(lib, k=None) == INV and index_read(lib, k=0x7000008) == INV
    assert index_read(lib, s=None) == INV and index_read(lib, s=0x8000002) == INV


def test_latent_append(lib):
    p = paged()
    assert lib.pmqa_latent_append(ref(p), 0x6000000, None, None, None, WS, 256, None) == INV
    tiny = 1e-39  # its fp32 reciprocal is infinite
    for kw, code in [
            (dict(c=0x1000008), INV), (dict(c_row=-512), INV), (dict(c_row=516), INV), (dict(k_pe=None), INV),
            (dict(pe_row=68), INV), (dict(q_c=0x3000008), INV), (dict(q_c_row=-8), INV), (dict(q_c_head=516), INV),
            (dict(q_pe=None), INV), (dict(q_pe_row=4), INV), (dict(q_pe_head=-64), INV), (dict(q_out=None), INV),
            (dict(q_out=0x5000004), INV), (dict(heads=0), INV), (dict(heads=65536, q_c_head=0, q_pe_head=0), UNS)]:
        assert latent_append(lib, x=latent_rows(**kw)) == code, kw
    for s in (0.0, tiny, INF, NAN):
        assert latent_append(lib, x=latent_rows(kv_scale=s)) == INV
        assert latent_append(lib, x=latent_rows(q_scale=s)) == INV
    assert latent_append(lib, kv=None) == INV and latent_append(lib, kv=0x6000004) == INV
    assert latent_append(lib, paged(rows=1 << 17), latent_rows(heads=1 << 14)) == UNS
    # scales of what is absent are not looked at
    assert latent_append(lib, x=latent_rows(c=None, q_c=None, kv_scale=0.0, q_scale=0.0), kv=None) == OK


def test_attention(lib):
    assert attention(lib, heads=0) == INV and attention(lib, heads=129) == UNS
    assert attention(lib, paged(rows=1 << 25), heads=128) == UNS
    for bad in (INF, NAN):
        assert attention(lib, qs=bad) == INV and attention(lib, ks=bad) == INV and attention(lib, sm=bad) == INV
    assert attention(lib, sm=1e10, qs=1e10, ks=10.0) == UNS  # the scores' factor past 1e20
    for name in ("q", "kv", "out"):
        assert attention(lib, **{name: None}) == INV
        assert attention(lib, **{name: 0x1000008}) == INV
    assert attention(lib, lse=0x9000002) == INV
    assert 40 << 20 < pmqa.pmqa_latent_workspace_bytes() < 48 << 20


# ------------------------------------------------------------- frequencies

@pytest.mark.parametrize("dim,base", [(2, 10000.0), (64, 10000.0), (128, 500000.0), (1024, 1.5)])
def test_frequencies_plain_and_linear(lib, dim, base):
    """The device's own, from the host's pow: a unit of 2^-52, and one more of the reference's."""
    want = [base ** (-2 * i / dim) for i in range(dim // 2)]
    f, s = pmqa.rope_frequencies(dim, base, device="cpu")
    assert f.dtype is torch.float64 and s == 1.0
    assert all(abs(a - b) <= b * 2.0 ** -50 for a, b in zip(f.tolist(), want))
    f, s = pmqa.rope_frequencies(dim, base, kind=pmqa.PMQA_ROPE_LINEAR, factor=8.0, device="cpu")
    assert s == 1.0 and all(abs(a - b / 8) <= b * 2.0 ** -50 for a, b in zip(f.tolist(), want))


@pytest.mark.parametrize("dim,base,factor,trained,slow,fast", [
    (64, 10000.0, 40.0, 4096.0, 1.0, 32.0), (128, 1e6, 4.0, 32768.0, 1.0, 32.0), (16, 10000.0, 1.0, 1.0, 0.5, 2.0)])
def test_frequencies_in_parts(lib, dim, base, factor, trained, slow, fast):
    f, s = pmqa.rope_frequencies(dim, base, kind=pmqa.PMQA_ROPE_PARTS, factor=factor, trained=trained,
                                 slow_turns=slow, fast_turns=fast, device="cpu")
    # as fp32: half a step of a value up to 1.4
    assert abs(s - (0.1 * math.log(factor) + 1)) <= 1.5 * 2.0 ** -24
    # a pair that turns more than `fast` times is kept, one that turns less than `slow` is divided
    plain = [base ** (-2 * i / dim) for i in range(dim // 2)]
    share = []
    for a, b in zip(f.tolist(), plain):
        t = trained * b / (2 * math.pi)
        if t > fast:
            # (rounded outwards: the first pair past the end may be weighted too)
            assert b / factor <= a * (1 + 2.0 ** -40) and a <= b * (1 + 2.0 ** -40)
        if t < slow / base ** (2 / dim):
            assert abs(a - b / factor) <= b * 2.0 ** -45
        if t > fast * base ** (2 / dim):
            assert abs(a - b) <= b * 2.0 ** -45
        share.append((b - a) / (b - b / factor) if factor > 1 else 0.0)
    # linear in between
    inside = [x for x in share if 1e-9 < x < 1 - 1e-9]
    steps = [y - x for x, y in zip(inside, inside[1:])]
    assert all(abs(x - steps[0]) <= 1e-9 for x in steps)


@pytest.mark.parametrize("kw", [
    dict(dim=0), dict(dim=-2), dict(dim=7), dict(base=1.0), dict(base=INF), dict(base=NAN), dict(kind=3), dict(kind=-1),
    dict(kind=1, factor=0.5), dict(kind=1, factor=INF), dict(kind=2, factor=NAN), dict(kind=2, trained=0.0),
    dict(kind=2, slow_turns=0.0), dict(kind=2, slow_turns=32.0), dict(kind=2, fast_turns=INF)])
def test_frequencies_refusals(lib, kw):
    with pytest.raises(pmqa.PmqaError):
        pmqa.rope_frequencies(**{**dict(dim=64, base=10000.0, factor=2.0, device="cpu"), **kw})


def test_frequencies_need_both_outputs(lib):
    out, s = (ctypes.c_double * 4)(), ctypes.c_float()
    assert lib.pmqa_rope_frequencies(8, 1e4, 0, 1.0, 1.0, 1.0, 32.0, None, ctypes.byref(s)) == INV
    assert lib.pmqa_rope_frequencies(8, 1e4, 0, 1.0, 1.0, 1.0, 32.0, out, None) == INV


# ------------------------------------------------------------- the binding

BF, F32 = torch.bfloat16, torch.float32


def zeros(*shape, dtype=BF):
    return torch.zeros(shape, dtype=dtype)


def step(width):
    """Pool, tables, lengths, row starts and max_rows of 2 requests with 5 rows."""
    return dict(kv_cache=zeros(8, 4, width, dtype=torch.uint8), block_tables=zeros(2, 3, dtype=torch.int32),
                context_lens=zeros(2, dtype=torch.int32), row_begin=zeros(3, dtype=torch.int32), max_rows=3)


INDEX = dict(k=zeros(5, 128), q=zeros(5, 4, 128), weights=zeros(5, 4, dtype=F32))
LATENT = dict(c=zeros(5, 512), k_pe=zeros(5, 64), kv_scale=0.1, q_c=zeros(5, 4, 512), q_pe=zeros(5, 4, 64))
QUERY = dict(q=zeros(5, 4, 576, dtype=torch.uint8), q_scale=0.1, kv_scale=0.1, sm_scale=0.1)
FREQ = zeros(32, dtype=torch.float64)


def refusal(fn, base, match, **kw):
    with pytest.raises(AssertionError, match=match):
        fn(**{**base, **kw})


@pytest.mark.parametrize("fn,base,width", [
    (pmqa.pmqa_index_append, {**step(132), **INDEX}, 132), (pmqa.pmqa_latent_append, {**step(576), **LATENT}, 576),
    (pmqa.pmqa_latent_attention, {**step(576), **QUERY}, 576),
    (pmqa.pmqa_index_read, {k: v for k, v in {**step(132), "rows": 5}.items() if k not in ("context_lens", "max_rows")}, 132)])
def test_binding_refuses_other_pools_and_tables(lib, fn, base, width):
    refusal(fn, base, "cuda")  # everything as documented, on the host
    kv, bt = base["kv_cache"], base["block_tables"]
    refusal(fn, base, "pool", kv_cache=zeros(8, 4, width - 4, dtype=torch.uint8))
    refusal(fn, base, "pool", kv_cache=kv.reshape(32, width))
    refusal(fn, base, "pool", kv_cache=kv.view(torch.int8))
    refusal(fn, base, "pool", kv_cache=kv[:, ::2])
    refusal(fn, base, "int32", block_tables=bt.long())
    refusal(fn, base, "contiguous", block_tables=zeros(2, 6, dtype=torch.int32)[:, ::2])
    refusal(fn, base, "shape", row_begin=zeros(2, dtype=torch.int32))
    refusal(fn, base, "int32", row_begin=zeros(3, dtype=torch.int64))
    if "context_lens" in base:
        refusal(fn, base, "shape", context_lens=zeros(3, dtype=torch.int32))
    refusal(fn, base, "cuda", kv_cache=kv.view(torch.float8_e4m3fn))


def test_binding_refuses_other_rows(lib):
    fn, base = pmqa.pmqa_index_append, {**step(132), **INDEX}
    refusal(fn, base, "keys, queries or both", k=None, q=None)
    refusal(fn, base, "weights", weights=None)
    refusal(fn, base, "bfloat16", k=INDEX["k"].half())
    refusal(fn, base, "shape", k=zeros(4, 128))
    refusal(fn, base, "last dimension", k=zeros(128, 5).T)
    refusal(fn, base, "bfloat16", q=INDEX["q"].float())
    refusal(fn, base, "shape", q=zeros(5, 4, 64))
    refusal(fn, base, "weights", weights=zeros(5, 3, dtype=F32))
    refusal(fn, base, "weights", weights=zeros(5, 4, dtype=torch.float16))
    refusal(fn, base, "weights", weights=zeros(4, 5, dtype=F32).T)
    refusal(fn, base, "float8", q_out=zeros(5, 4, 128, dtype=torch.int8))
    refusal(fn, base, "shape", weights_out=zeros(5, 5, dtype=F32))
    refusal(fn, base, "shape", norm=pmqa.Norm(1, zeros(64, dtype=F32), None))
    refusal(fn, base, "float32", norm=pmqa.Norm(1, None, zeros(128)))
    refusal(fn, base, "float64", rotary=pmqa.Rotary(FREQ.float()))
    refusal(fn, base, "shape", rotary=pmqa.Rotary(FREQ), positions=zeros(4, dtype=torch.int32))
    fn, base = pmqa.pmqa_latent_append, {**step(576), **LATENT}
    for kw in (dict(c=None, k_pe=None, q_c=None, q_pe=None), dict(k_pe=None), dict(q_pe=None), dict(c=None)):
        refusal(fn, base, "rotary part", **kw)
    refusal(fn, base, "shape", c=zeros(5, 576))
    refusal(fn, base, "bfloat16", k_pe=zeros(5, 64, dtype=F32))
    refusal(fn, base, "shape", q_c=zeros(5, 4, 64))
    refusal(fn, base, "shape", q_pe=zeros(5, 3, 64))
    refusal(fn, base, "float8", q_out=zeros(5, 4, 512, dtype=torch.uint8))
    refusal(fn, base, "shape", norm=pmqa.Norm(2, zeros(128, dtype=F32), None))
    fn, base = pmqa.pmqa_latent_attention, {**step(576), **QUERY}
    refusal(fn, base, "float8", q=zeros(5, 4, 576))
    refusal(fn, base, "float8", q=zeros(5, 4, 512, dtype=torch.uint8))
    refusal(fn, base, "shape", out=zeros(5, 4, 576))
    refusal(fn, base, "float32", lse=zeros(5, 4))
    fn = pmqa.pmqa_index_read
    base = {k: v for k, v in {**step(132), "rows": 5}.items() if k not in ("context_lens", "max_rows")}
    refusal(fn, base, "shape", start=zeros(3, dtype=torch.int32))
    refusal(fn, base, "float8", k=zeros(4, 128, dtype=torch.uint8))
    refusal(fn, base, "shape", k_scale=zeros(4, dtype=F32))


def test_binding_refuses_other_heads(lib):
    base = dict(x=zeros(5, 4, 128), positions=zeros(5, dtype=torch.int32), rotary=pmqa.Rotary(FREQ))
    refusal(pmqa.pmqa_rope, base, "cuda")
    refusal(pmqa.pmqa_rope, base, "bfloat16", x=base["x"].float())
    refusal(pmqa.pmqa_rope, base, "last dimension", x=zeros(5, 128, 4).transpose(1, 2))
    refusal(pmqa.pmqa_rope, base, "shape", positions=zeros(4, dtype=torch.int32))
    refusal(pmqa.pmqa_rope, base, "int32", positions=zeros(5, dtype=torch.int64))
    refusal(pmqa.pmqa_rope, base, "shape", out=zeros(5, 4, 64))
    refusal(pmqa.pmqa_rope, base, "shape", other=zeros(4, 2, 128))
    refusal(pmqa.pmqa_rope, base, "float64", rotary=pmqa.Rotary(FREQ.float()))
