"""Host-only checks of the operators on the 8-bit K/V cache: the C ABI refuses
bad arguments before it touches the device, the binding refuses bad tensors, and
the plain forms that the GPU tests compare with agree with dense attention."""

import ctypes
import math

import pytest
import torch

from sparse_attention_indexer_pmqa_gb300 import build, pmqa
from tests import cache_ref as ref

INV, UNS, SPACE = pmqa.PMQA_ERR_INVALID_ARG, pmqa.PMQA_ERR_UNSUPPORTED, pmqa.PMQA_ERR_WORKSPACE
A, B, C, D, E = (ctypes.c_void_p(x) for x in (0x10000, 0x20000, 0x30000, 0x40000, 0x50000))
WS = ctypes.c_void_p(0x100000)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return pmqa.load()


def problem(**kw):
    # fake, suitably aligned device addresses: argument checks run before any CUDA call
    base = dict(k_cache=0x60000, v_cache=0x70000, k_scale=0x80000, v_scale=0x90000,
                block_tables=0xA0000, context_lens=0xB0000, row_begin=0xC0000, bs=2, kv_heads=2,
                head_dim=128, block_size=16, max_blocks_per_seq=8, rows=4, max_rows=3,
                num_blocks=32)
    base.update(kw)
    return pmqa.CacheProblem(**base)


def size():
    return pmqa.pmqa_cache_workspace_bytes()


def append(lib, p, k=A, v=B, ws=WS, n=None):
    return lib.pmqa_cache_append(ctypes.byref(p), k, v, ws, size() if n is None else n, None)


def attention(lib, p, q=A, heads=8, sm=0.1, out=B, lse=None, ws=WS, n=None):
    return lib.pmqa_cache_attention(ctypes.byref(p), q, heads, sm, out, lse, ws,
                                    size() if n is None else n, None)


def weigh(lib, p, q=A, heads=8, sm=0.1, lse=B, had=None, out=C, width=128, ws=WS, n=None):
    return lib.pmqa_cache_weigh(ctypes.byref(p), q, heads, sm, lse, had, out, width, ws,
                                size() if n is None else n, None)


def evict(lib, p, mass=A, width=128, keep=32, sinks=2, recent=4, new=B, new_w=2, kept=C, lens=D,
          out=E, ws=WS, n=None):
    return lib.pmqa_cache_evict(ctypes.byref(p), mass, width, keep, sinks, recent, new, new_w, kept,
                                lens, out, ws, size() if n is None else n, None)


CALLS = [append, attention, weigh, evict]


def test_workspace_is_one_size(lib):
    assert 1 << 20 < size() < 32 << 20


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("kw,code", [
    (dict(bs=-1), INV), (dict(kv_heads=0), INV), (dict(head_dim=0), INV), (dict(block_size=0), INV),
    (dict(max_blocks_per_seq=0), INV), (dict(num_blocks=0), INV),
    (dict(head_dim=96), UNS), (dict(head_dim=256), UNS), (dict(block_size=1025), UNS),
    (dict(kv_heads=65536), UNS), (dict(num_blocks=1 << 40), UNS),
    (dict(k_cache=None), INV), (dict(k_cache=0x60008), INV), (dict(k_scale=None), INV),
    (dict(block_tables=0xA0002), INV), (dict(context_lens=None), INV),
])
def test_problem_checks(lib, call, kw, code):
    assert call(lib, problem(**kw)) == code


@pytest.mark.parametrize("call", [append, attention, weigh])
@pytest.mark.parametrize("kw", [dict(rows=-1), dict(max_rows=0), dict(row_begin=None),
                                dict(row_begin=0xC0001)])
def test_row_checks(lib, call, kw):
    assert call(lib, problem(**kw)) == INV


@pytest.mark.parametrize("call", [append, attention, evict])
def test_value_pool_checks(lib, call):
    for kw in (dict(v_cache=None), dict(v_cache=0x70004), dict(v_scale=None)):
        assert call(lib, problem(**kw)) == INV


@pytest.mark.parametrize("call", CALLS)
def test_workspace_checks(lib, call):
    p = problem()
    assert call(lib, p, n=size() - 1) == SPACE
    assert call(lib, p, ws=None) == INV
    assert call(lib, p, ws=ctypes.c_void_p(0x100040)) == INV


@pytest.mark.parametrize("call", CALLS)
def test_empty_batch_is_a_no_op(lib, call):
    assert call(lib, problem(bs=0, k_cache=None, row_begin=None)) == pmqa.PMQA_OK


def test_no_rows_is_a_no_op(lib):
    assert append(lib, problem(rows=0), k=None, v=None) == pmqa.PMQA_OK
    assert attention(lib, problem(rows=0), q=None, out=None) == pmqa.PMQA_OK


def test_null_problem(lib):
    n = size()
    assert lib.pmqa_cache_append(None, A, B, WS, n, None) == INV
    assert lib.pmqa_cache_attention(None, A, 8, 0.1, B, None, WS, n, None) == INV
    assert lib.pmqa_cache_weigh(None, A, 8, 0.1, B, None, C, 128, WS, n, None) == INV
    assert lib.pmqa_cache_evict(None, A, 128, 32, 2, 4, B, 2, C, D, E, WS, n, None) == INV


def test_operand_checks(lib):
    p, odd = problem(), ctypes.c_void_p(0x10008)
    for bad in (None, odd):
        assert append(lib, p, k=bad) == INV
        assert append(lib, p, v=bad) == INV
        assert attention(lib, p, q=bad) == INV
        assert attention(lib, p, out=bad) == INV
        assert weigh(lib, p, q=bad) == INV
    assert attention(lib, p, lse=ctypes.c_void_p(0x10002)) == INV
    assert weigh(lib, p, lse=None) == INV
    assert weigh(lib, p, out=None) == INV
    assert weigh(lib, p, width=0) == INV
    for name in ("mass", "new", "kept", "lens"):
        assert evict(lib, p, **{name: None}) == INV


@pytest.mark.parametrize("call", [attention, weigh])
def test_head_checks(lib, call):
    p = problem()
    assert call(lib, p, heads=0) == INV
    assert call(lib, p, heads=7) == INV
    assert call(lib, p, heads=2 * 129) == UNS
    assert call(lib, p, sm=math.inf) == INV
    assert call(lib, p, sm=math.nan) == INV
    assert call(lib, p, sm=3.0e38) == INV  # infinite in base 2
    assert call(lib, problem(rows=1 << 28, max_rows=1 << 28), heads=8) == UNS


def test_evict_checks(lib):
    p = problem()
    for kw in (dict(width=0), dict(keep=0), dict(sinks=-1), dict(recent=-1),
               dict(sinks=20, recent=13), dict(new_w=0), dict(new_w=1),  # 1 block of 16 < 32
               dict(lens=ctypes.c_void_p(p.context_lens)), dict(out=A),
               dict(out=ctypes.c_void_p(0x10000 + 4 * (2 * 2 * 128 - 1)))):
        assert evict(lib, p, **kw) == INV, kw


def test_binding_refuses_host_tensors(lib):
    p = ref.make([1], [5], kv_heads=2, group=2, head_dim=64, block=4)
    cache = (p.kc, p.vc, p.ks, p.vs, p.bt, p.ctx)
    with pytest.raises(AssertionError):
        pmqa.pmqa_cache_attention(p.q, *cache, p.rb, 1, p.sm)
    with pytest.raises(AssertionError):
        pmqa.pmqa_cache_append(p.k_new, p.v_new, *cache, p.rb, 1)


# ------------------------------------------------- the plain forms themselves

def test_plain_attention_is_dense_attention():
    p = ref.make([3, 1], [9, 4], kv_heads=2, group=3, head_dim=64, block=4, seed=1)
    out, lse, _, _ = ref.attention(p)
    for i, (n, c) in enumerate(zip(p.rows, p.ctx.tolist())):
        r0 = int(p.rb[i])
        k, _ = ref.tokens(p.kc, p.ks, p.bt, i, c, p.P)
        v, _ = ref.tokens(p.vc, p.vs, p.bt, i, c, p.P)
        for j in range(n):
            for hq in range(6):
                q = p.q[r0 + j, hq].double()
                seen = c - n + j + 1
                s = (k[hq // 3, :seen] @ q) * p.sm
                torch.testing.assert_close(out[r0 + j, hq], torch.softmax(s, 0) @ v[hq // 3, :seen])
                torch.testing.assert_close(lse[r0 + j, hq], torch.logsumexp(s, 0))


def test_plain_weights_of_a_row_sum_to_one():
    p = ref.make([2, 5], [7, 5], kv_heads=1, group=2, head_dim=64, block=3, seed=2)
    _, lse, _, _ = ref.attention(p)
    mass, _ = ref.weigh(p, lse, torch.zeros((2, 1, 12)))
    want = torch.tensor([2 * 2.0, 5 * 2.0], dtype=torch.float64)  # rows x group
    torch.testing.assert_close(mass.nan_to_num(0.0).sum((1, 2)), want)


def test_plain_scale_is_the_smallest_power_of_two():
    a = torch.tensor([0.0, 448.0, 448.0001, 1.0, 3.5, 3.5000002, 1e-40], dtype=torch.float64)
    s = ref.scale_of(a)
    assert s[0] == 2.0 ** -100 and s[-1] == 2.0 ** -100
    for x, y in zip(a[1:-1], s[1:-1]):
        assert x / y <= 448.0 < 2 * x / y and math.log2(float(y)) % 1 == 0
