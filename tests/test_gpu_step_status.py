"""What the calls around the sparse-MLA step record in the status word: rows without a slot, and
scores out of range where they are a row's largest."""

import math

import pytest
import torch

from tests import step_ref as ref
from tests.test_gpu_latent_attention import run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads", [1, 16, 24, 64, 128])
@pytest.mark.parametrize("rows,ctx", [(3, 2), (1, 0), (70, 69)])
def test_attention_reports_rows_before_slot_0(cuda_lib, heads, rows, ctx):
    """Also behind a request that has all of its rows; those rows see nothing."""
    p = ref.attention_problem([2, rows], [40, rows], heads, 16, seed=2)
    p.ctx[1] = ctx
    out, lse, status = run(cuda_lib, p)
    assert status == cuda_lib.PMQA_DEV_BAD_CONTEXT
    none = 2 + rows - ctx
    assert bool((out[2:none] == 0).all()) and bool((lse[2:none] == -math.inf).all())
    assert bool(lse[:2].isfinite().all()) and bool(lse[none:].isfinite().all())
    p.ctx[1] = rows
    assert run(cuda_lib, p)[2] == 0


@pytest.mark.parametrize("rows,ctx", [(3, 2), (1, 0), (2, 49), (4000, 3999)])
def test_appends_without_keys_report_rows_without_a_slot(cuda_lib, rows, ctx):
    """The queries are written all the same."""
    lib, ws = cuda_lib, cuda_lib.latent_workspace()
    p = ref.layout([rows], [rows if rows > 4 else 48], 16, tail=1)
    p.bt[0] = torch.arange(p.bt.shape[1])
    full = p.bt.shape[1] * 16
    g = torch.Generator().manual_seed(1)
    q = torch.randn((p.total, 4, 128), generator=g).to(torch.bfloat16).cuda()
    w = torch.randn((p.total, 4), generator=g).cuda()
    c, pe = (torch.randn((p.total, 4, n), generator=g).to(torch.bfloat16).cuda() for n in (512, 64))
    kv, lat = (torch.zeros((p.nb, 16, n), dtype=torch.uint8, device="cuda") for n in (132, 576))
    bt, rb = p.bt.cuda(), p.rb.cuda()
    for context in (min(full, max(rows, ctx)) if ctx < 49 or rows > 4 else 48, ctx if ctx != 49 else full + 1):
        at = (bt, torch.tensor([context], dtype=torch.int32, device="cuda"), rb, rows)
        want = 0 if rows <= context <= full else lib.PMQA_DEV_BAD_CONTEXT
        q8 = torch.full((p.total, 4, 128), 7, dtype=torch.uint8, device="cuda")
        lib.pmqa_index_append(None, kv, *at, q=q, weights=w, q_out=q8, ws=ws)
        assert lib.pmqa_read_device_status(ws) == want
        q16 = torch.full((p.total, 4, 576), 7, dtype=torch.uint8, device="cuda")
        lib.pmqa_latent_append(None, None, lat, *at, 0.03, q_c=c, q_pe=pe, q_scale=0.03, q_out=q16, ws=ws)
        assert lib.pmqa_read_device_status(ws) == want
        for x in (q8, q16):
            assert bool((x[:rows] != 7).flatten(1).any(1).all()) and bool((x[rows:] == 7).all())
    assert not bool(kv.any()) and not bool(lat.any())


@pytest.mark.parametrize("heads", [1, 16, 24, 64, 128])
@pytest.mark.parametrize("ctx,block", [(500, 4), (3000, 64)])
@pytest.mark.parametrize("factor", [10.0, 1e6, -1e12])
@pytest.mark.parametrize("where", ["first", "last", "some", "but one", "none", "all"])
def test_far_scores_are_reported_where_they_are_the_largest(cuda_lib, heads, ctx, block, factor, where):
    """Scores from -3.2e6 factor to -2.3e6 factor (in powers of two) beside scores of 0: these alone have
    weight, all the same. With one range for a context and many."""
    lib = cuda_lib
    p = ref.attention_problem([2], [ctx], heads, block, seed=6)
    t = torch.arange(ctx)
    far = dict(first=t < 256, last=t >= ctx - 200, some=t % 37 < 5, none=t < 0, all=t >= 0)
    far["but one"] = t != 131
    far = far[where]
    p.q[:] = 0
    p.q.view(ref.F8)[..., 512:528] = 448.0
    k = ref.value(p.kv.reshape(-1, 576)).float().clamp(-2, 2)
    k[:, 512:] = 0.0
    at = ref.places(p, 0, 0, ctx)
    k[at[far], 512:528] = (-math.copysign(1.0, factor) * (448.0 - 32.0 * (t[far] % 5).float()))[:, None]
    p.kv = k.to(ref.F8).view(torch.uint8).reshape(p.kv.shape)
    p.q_scale, p.kv_scale, p.sm = 1.0, 1.0, factor / math.log2(math.e)
    out, lse, status = run(lib, p)
    if where == "all":
        assert status == lib.PMQA_DEV_SCORE_RANGE
        return
    assert status == 0
    for j in range(2):
        light = ~far & (t <= ctx - 2 + j)
        v = ref.value(p.kv.reshape(-1, 576))[at[light], :512]
        mean, size = v.mean(0), v.abs().mean(0)
        # a weight's two terms and f16, sums in fp32; one rounding
        tol = size * (2.0 ** -7 + 2.0 ** -11 + 2.0 ** -17)
        tol = tol + (mean.abs() + tol) * 2.0 ** -8
        assert bool(((out[j].double() - mean).abs() <= tol).all())
        assert bool(((lse[j].double() - math.log(int(light.sum()))).abs() <= 2.0 ** -17).all())
