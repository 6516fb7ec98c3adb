"""Attention to all latent tokens against its 64-bit form: head counts, rows,
contexts and block sizes at which the tiles, packed rows and cuts change, masked and
missing tokens, NaN, rows of no request."""

import math

import pytest
import torch

from tests import step_ref as ref

pytestmark = pytest.mark.gpu


def run(pmqa, p, ws=None, **kw):
    ws = pmqa.latent_workspace() if ws is None else ws
    out = torch.full((p.total, p.heads, 512), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((p.total, p.heads), 7.0, device="cuda")
    args = [t.cuda() for t in (p.q, p.kv, p.bt, p.ctx, p.rb)]
    pmqa.pmqa_latent_attention(*args, kw.pop("max_rows", p.max_rows), p.q_scale, p.kv_scale, p.sm, out=out,
                               lse=lse, ws=ws, **kw)
    return out.cpu(), lse.cpu(), pmqa.pmqa_read_device_status(ws)


def check(got, want, p):
    out, lse, status = got
    o, l, tol, ltol = want
    mine = torch.zeros(p.total, dtype=torch.bool)
    for r, _, _ in ref.slots(p):
        mine[r] = True
    assert bool((out[~mine] == 7.0).all()) and bool((lse[~mine] == 7.0).all()), "rows of no request"
    out, lse, o, l = out[mine].double(), lse[mine].double(), o[mine], l[mine]
    assert torch.equal(out.isnan(), o.isnan()) and torch.equal(lse.isnan(), l.isnan())
    assert torch.equal(lse == -math.inf, l == -math.inf)
    bad = ((out - o).abs() > tol[mine]) & ~o.isnan()
    assert not bool(bad.any()), (int(bad.sum()), float(((out - o).abs() / tol[mine]).nan_to_num(0.0).max()))
    far = ((lse - l).abs() > ltol[mine]) & l.isfinite()
    assert not bool(far.any()), float(((lse - l).abs() / ltol[mine])[l.isfinite()].max())
    return status


@pytest.mark.parametrize("heads,rows,ctx,block", [
    (16, [1], [1], 1), (16, [1], [500], 16), (1, [1], [129], 64), (16, [1] * 5, [127, 128, 129, 1, 1000], 1),
    (8, [2, 1], [300, 77], 24), (5, [4, 3], [513, 200], 8), (32, [1, 1], [640, 641], 64),
    (16, [4] * 3, [1500, 4, 900], 1), (16, [2] * 4, [700] * 4, 48), (64, [1, 1, 1], [257, 2000, 1], 64),
    (40, [3, 1], [400, 1300], 16), (128, [1], [3000], 64), (128, [2, 1], [130, 700], 1),
    (96, [1, 2], [257, 129], 64), (65, [1], [385], 7), (127, [3], [260], 1), (128, [70], [200], 64),
    (16, [200, 1, 33], [260, 900, 33], 64), (24, [150], [150], 1), (3, [260], [300], 128), (1, [400], [401], 5),
])
def test_against_the_64_bit_form(cuda_lib, heads, rows, ctx, block):
    p = ref.attention_problem(rows, ctx, heads, block, seed=heads + len(rows))
    assert check(run(cuda_lib, p), ref.attention(p), p) == 0


@pytest.mark.parametrize("heads", [16, 20, 64, 128])
def test_rows_of_no_request_and_empty_requests(cuda_lib, heads):
    p = ref.attention_problem([2, 0, 1, 0], [300, 50, 129, 0], heads, 16, seed=3, lead=3, tail=2)
    assert check(run(cuda_lib, p), ref.attention(p), p) == 0


@pytest.mark.parametrize("heads", [8, 16, 64, 128])
def test_a_bad_table_entry_is_left_out(cuda_lib, heads):
    p = ref.attention_problem([2, 3], [400, 260], heads, 16, seed=5)
    leave = [(0, t) for t in range(32, 48)] + [(1, t) for t in range(128, 144)]
    want = ref.attention(p, leave)
    p.bt[0, 2], p.bt[1, 8] = p.nb, -5
    assert check(run(cuda_lib, p), want, p) == cuda_lib.PMQA_DEV_BAD_BLOCK_ID


def test_all_tokens_behind_bad_entries(cuda_lib):
    p = ref.attention_problem([1, 1], [200, 30], 16, 32, seed=5)
    want = ref.attention(p, [(0, t) for t in range(200)])
    p.bt[0] = -1
    assert check(run(cuda_lib, p), want, p) == cuda_lib.PMQA_DEV_BAD_BLOCK_ID


@pytest.mark.parametrize("heads", [8, 16, 64, 128])
@pytest.mark.parametrize("at", [5, 520, 575])
def test_a_nan_token_reaches_the_rows_that_see_it(cuda_lib, heads, at):
    """In the values or in the rotary part, of a token that the last rows alone see, of one that
    all see, and in a query."""
    p = ref.attention_problem([6, 4], [140, 300], heads, 8, seed=9)
    p.kv.reshape(-1, 576)[ref.places(p, 0, 137, 138), at] = 0xFF
    p.kv.reshape(-1, 576)[ref.places(p, 1, 20, 21), at] = 0x7F
    want = ref.attention(p)
    got = run(cuda_lib, p)
    assert check(got, want, p) == 0
    assert not bool(got[0][:3].isnan().any()) and bool(got[0][3:].isnan().all())
    p = ref.attention_problem([6, 4], [140, 300], heads, 8, seed=9)
    p.q[1, heads // 2, at] = 0x7F
    p.q[8, :, at] = 0x7F
    got = run(cuda_lib, p)
    assert check(got, ref.attention(p), p) == 0


def test_tokens_that_no_row_sees_are_not_read(cuda_lib):
    """Slots behind a context (the test's poison) and blocks of other requests."""
    p = ref.attention_problem([3], [130], 16, 64, seed=1)
    assert check(run(cuda_lib, p), ref.attention(p), p) == 0


@pytest.mark.parametrize("sm", [0.0, -0.1, 3.0])
def test_score_scales(cuda_lib, sm):
    """Equal weights, reversed order, and one token that takes nearly all of the weight."""
    p = ref.attention_problem([1, 2], [1300, 400], 16, 64, seed=11)
    p.sm = sm
    assert check(run(cuda_lib, p), ref.attention(p), p) == 0


@pytest.mark.parametrize("heads,rows", [(16, 1), (16, 2), (64, 1), (128, 1)])
def test_scores_that_rise_along_the_context(cuda_lib, heads, rows):
    """The maximum moves again and again, by more than the slack each time."""
    p = ref.attention_problem([rows], [2000], heads, 64, seed=13)
    q = torch.zeros((p.total, heads, 576))
    q[..., 0], q[..., 1] = 8.0, 1.0
    p.q = (q / p.q_scale).clamp(-448, 448).to(ref.F8).view(torch.uint8)
    k = ref.value(p.kv.reshape(-1, 576)).float()
    k[ref.places(p, 0, 0, 2000), 0] = torch.linspace(-400, 400, 2000)
    p.kv = k.to(ref.F8).view(torch.uint8).reshape(p.kv.shape)
    p.sm = 0.5
    assert check(run(cuda_lib, p), ref.attention(p), p) == 0


@pytest.mark.parametrize("heads", [8, 16, 64, 128])
@pytest.mark.parametrize("sm,far", [(60.0, True), (-60.0, True), (0.06, False), (-0.06, False)])
def test_scores_out_of_range_are_reported(cuda_lib, heads, sm, far):
    """Equal tokens of the largest values, with unit scales: each score is 0.7 or 700 times the
    largest of the range; within it all weights are equal."""
    p = ref.attention_problem([1, 1], [300, 7], heads, 16, seed=4)
    p.kv[:], p.q[:] = 0x7E, 0x7E
    p.q_scale, p.kv_scale, p.sm = 1.0, 1.0, sm / 1.44269504 / 1.1561
    out, _, status = run(cuda_lib, p)
    if far:
        assert status == cuda_lib.PMQA_DEV_SCORE_RANGE
    else:
        # equal weights: off by a weight's two terms, and one rounding
        assert status == 0
        assert bool(((out.double() - 448.0).abs() <= 448.0 * (2.0 ** -7 + 2.0 ** -8 + 2.0 ** -11)).all())


def test_without_a_log_sum_exp(cuda_lib):
    p = ref.attention_problem([1, 2], [700, 90], 16, 16, seed=12)
    args = [t.cuda() for t in (p.q, p.kv, p.bt, p.ctx, p.rb)] + [p.max_rows, p.q_scale, p.kv_scale, p.sm]
    assert torch.equal(cuda_lib.pmqa_latent_attention(*args).cpu(), run(cuda_lib, p)[0])


def test_lengths_that_break_the_rules_are_clamped(cuda_lib):
    p = ref.attention_problem([2, 2], [40, 64], 16, 16, seed=2)
    want = ref.attention(p)
    cap = p.bt.shape[1] * 16
    p.bt[1] = torch.arange(p.bt.shape[1])  # every entry is a block
    q = ref.attention_problem([2, 2], [40, 64], 16, 16, seed=2)
    q.bt, q.ctx = p.bt, torch.tensor([40, cap + 9], dtype=torch.int32)
    got = run(cuda_lib, q)
    assert got[2] == cuda_lib.PMQA_DEV_BAD_CONTEXT
    assert bool(((got[0][:2].double() - want[0][:2]).abs() <= want[2][:2]).all())
    # fewer tokens than rows: the first row sees none
    q = ref.attention_problem([3], [3], 16, 16, seed=2)
    q.ctx = torch.tensor([2], dtype=torch.int32)
    out, lse, _ = run(cuda_lib, q)
    assert bool((out[0] == 0).all()) and bool((lse[0] == -math.inf).all()) and bool(lse[1:].isfinite().all())


def test_equal_calls_give_equal_bits_and_leave_the_workspace_ready(cuda_lib):
    ws = cuda_lib.latent_workspace()
    p = ref.attention_problem([1] * 7, [3000, 5, 700, 1300, 2, 900, 128], 128, 64, seed=17)
    a = run(cuda_lib, p, ws)
    q = ref.attention_problem([4] * 3, [600, 900, 1300], 16, 1, seed=18)
    assert check(run(cuda_lib, q, ws), ref.attention(q), q) == 0
    b = run(cuda_lib, p, ws)
    assert torch.equal(a[0].view(torch.int16), b[0].view(torch.int16)) and torch.equal(a[1], b[1])
    assert check(b, ref.attention(p), p) == 0
