"""What else the operators on the 8-bit K/V cache refuse before they touch the
device: outputs that overlap inputs in part, and tensors of another type or shape
than the binding documents."""

import ctypes

import pytest
import torch

from sparse_attention_indexer_pmqa_gb300 import build, pmqa
from tests import cache_ref as ref
from tests.test_cache_host import INV, evict, problem, weigh


@pytest.fixture(scope="module")
def lib():
    build.build()
    return pmqa.load()


def at(address):
    return ctypes.c_void_p(address)


def test_weigh_refuses_masses_that_overlap_in_part(lib):
    """mass_in may be mass_out; shifted against it, tokens' sums would be read as
    other tokens' earlier masses."""
    p = problem()  # 2 requests x 2 heads x 128
    size = 4 * 2 * 2 * 128
    for shift in (4, -4, size - 4, 4 - size):
        assert weigh(lib, p, had=at(0x30000 + shift), out=at(0x30000)) == INV


def test_evict_refuses_lengths_that_overlap_in_part(lib):
    """lens_out is written while context_lens is read: one word in common is refused
    as the whole is."""
    p = problem()  # 2 requests
    for shift in (0, 4, -4):
        assert evict(lib, p, lens=at(p.context_lens + shift)) == INV


# ------------------------------------------------------------- the binding

def cache(p):
    return dict(k_cache=p.kc, v_cache=p.vc, k_scale=p.ks, v_scale=p.vs, block_tables=p.bt,
                context_lens=p.ctx)


@pytest.mark.parametrize("call", ["append", "attention", "weigh", "evict"])
def test_binding_refuses_other_types_and_shapes(lib, call):
    """By type and shape first, so that the refusals are the same without a GPU."""
    p = ref.make([3, 2], [9, 5], kv_heads=2, group=2, head_dim=64, block=4, seed=1)
    lse, mass = torch.zeros((5, 4)), torch.zeros((2, 2, 16))
    new = torch.zeros((2, 1), dtype=torch.int32)

    def run(**kw):
        c = cache(p)
        c.update({k: v for k, v in kw.items() if k in c})
        o = {k: v for k, v in kw.items() if k not in c}
        if call == "append":
            pmqa.pmqa_cache_append(o.get("k", p.k_new), o.get("v", p.v_new), **c, row_begin=o.get("rb", p.rb),
                                   max_rows=3)
        elif call == "attention":
            pmqa.pmqa_cache_attention(o.get("q", p.q), **c, row_begin=o.get("rb", p.rb), max_rows=3,
                                      sm_scale=p.sm, out=o.get("out"), lse=o.get("lse"))
        elif call == "weigh":
            c.pop("v_cache"), c.pop("v_scale")
            pmqa.pmqa_cache_weigh(o.get("q", p.q), **c, row_begin=o.get("rb", p.rb), max_rows=3,
                                  sm_scale=p.sm, lse=o.get("lse", lse), mass_in=o.get("mass"),
                                  mass_out=o.get("mass_out"), mass_width=o.get("width"))
        else:
            pmqa.pmqa_cache_evict(**c, mass=o.get("mass", mass), keep=4, sinks=0, recent=0,
                                  new_tables=o.get("new", new), kept=o.get("kept"),
                                  lens_out=o.get("lens"), mass_out=o.get("mass_out"))

    def refuses(match, **kw):
        with pytest.raises(AssertionError, match=match):
            run(**kw)

    refuses("cuda")  # everything as documented, on the host
    values = call != "weigh"
    for t in (torch.float8_e5m2, torch.int8, torch.bool):
        refuses("float8_e4m3fn", k_cache=p.kc.view(t), **(dict(v_cache=p.vc.view(t)) if values else {}))
    refuses("contiguous", k_cache=p.kc.transpose(1, 2))
    refuses("shape", k_scale=p.ks.reshape(2, -1).contiguous())
    refuses("shape", block_tables=p.bt.reshape(1, -1))
    refuses("shape", context_lens=p.ctx[:1])
    refuses("int32", context_lens=p.ctx.long())
    refuses("contiguous", block_tables=p.bt[:, ::2])
    if values:
        refuses("uint8", v_cache=p.vc.view(torch.float8_e4m3fn))
        refuses("shape", v_cache=p.vc.transpose(1, 2).contiguous())
    if call != "evict":
        refuses("shape", rb=p.rb[:-1])
    if call == "append":
        for name in ("k", "v"):
            refuses("shape", **{name: p.k_new.transpose(0, 1).contiguous()})
            refuses("bfloat16", **{name: p.k_new.half()})
    if call in ("attention", "weigh"):
        refuses("shape", q=p.q[..., :32].contiguous())
        refuses("bfloat16", q=p.q.half())
        refuses("shape", lse=lse.reshape(4, 5))
    if call == "attention":
        refuses("shape", out=torch.zeros((4, 5, 64), dtype=torch.bfloat16))
    if call == "weigh":
        refuses("shape", mass=torch.zeros((2, 4, 8)))
        refuses("shape", mass=mass, mass_out=torch.zeros((2, 2, 20)))
        refuses("mass_width", mass=mass, width=20)
    if call == "evict":
        refuses("shape", mass=torch.zeros((4, 2, 8)))
        refuses("shape", new=new.reshape(1, 2))
        refuses("shape", kept=torch.zeros((2, 4, 2), dtype=torch.int32))
        refuses("shape", lens=torch.zeros(3, dtype=torch.int32))
        refuses("shape", mass_out=torch.zeros((2, 2, 17)))
