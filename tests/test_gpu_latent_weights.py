"""Small weights in the attention to all latent tokens: heavy tokens before, among and behind many
light ones, whose weights add up to as much as anyone's.

Every SM (every two with more than 64 packed rows) gets one request, all of the same tokens, so
that none is cut and one running maximum holds for a whole context. The bound of each
output is the sum over the tokens of |v| times the bound of the weight's error:
  * of itself a weight loses 2^-8 (up to 32 packed rows) or 2^-7 (more), 2^-11 as f16, and what
    its score's error makes of it (step_ref.attention);
  * or at most half a step of its terms, 2^-14 or 2^-13 in the unit of its tile, or itself if it is
    less. The unit is what the kernel's rule gives (`units`), in 64 bits."""

import math
from types import SimpleNamespace

import pytest
import torch

from tests import step_ref as ref

pytestmark = pytest.mark.gpu

SM, QS, KS = 192 ** -0.5, 0.05, 0.03
LIFT = 16       # rotary values that lift a token's scores
Q_LIFT = 64.0   # the queries' there


def problem(heads, rows, ctx, lift, sigma=1.0, seed=0, q_lift=Q_LIFT, zero=True):
    """lift: float [ctx], nats that the tokens' scores lie above the others'; light scores have a
    standard deviation of about sigma, and values a mean of 1: what is lost does not cancel. zero: the
    heavy tokens' values are 0."""
    nats = SM * QS * KS * LIFT * q_lift  # of a token's score for a code of 1
    g = torch.Generator(device="cuda").manual_seed(seed)
    k = torch.randn((ctx, 576), generator=g, device="cuda") + 1.0
    k[:, 512:512 + LIFT] = (lift.cuda() / nats * KS)[:, None]
    if zero:
        k[(lift > 0).cuda(), :512] = 0.0
    q = torch.randn((rows, heads, 576), generator=g, device="cuda") * (sigma * 13.86 / 560 ** 0.5)
    q[..., 512:512 + LIFT] = q_lift * QS
    code = [(x / s).clamp(-448, 448).to(ref.F8) for x, s in ((k, KS), (q, QS))]
    return SimpleNamespace(k=code[0], q=code[1], heads=heads, rows=rows, ctx=ctx)


def run(pmqa, p, block=64):
    """The problem once for each SM (or two), in one call: [copies, rows, heads, 512]."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    n = sms if p.rows * p.heads <= 64 else sms // 2
    pages = -(-p.ctx // block)
    pool = torch.zeros((pages * block, 576), dtype=torch.uint8, device="cuda")
    g = torch.Generator().manual_seed(1)
    perm = torch.randperm(pages, generator=g)
    t = torch.arange(p.ctx)
    pool[(perm[t // block] * block + t % block).cuda()] = p.k.view(torch.uint8)
    i32 = dict(dtype=torch.int32, device="cuda")
    ws = pmqa.latent_workspace()
    out, lse = pmqa.pmqa_latent_attention(
        p.q.view(torch.uint8).repeat(n, 1, 1), pool.reshape(pages, block, 576), perm.to(**i32).repeat(n, 1),
        torch.full((n,), p.ctx, **i32), torch.arange(n + 1, **i32) * p.rows, p.rows, QS, KS, SM,
        want_lse=True, ws=ws)
    assert pmqa.pmqa_read_device_status(ws) == 0
    return out.reshape(n, p.rows, p.heads, 512).double(), lse.reshape(n, p.rows, p.heads).double()


def units(s, wide, edge):
    """Per row and tile the unit of the weights, as the power of two of its score, by the rule: a
    row's unit moves up where a weight would pass 2^8; the sum of the weights of the n tiles so far is
    to be at least 1.5 n (of 128 tokens), and where it is not the unit moves down until it is twice
    that and the tile's largest weight 1, as far as that stays below 2^8 and the sum below 2^30. Up to 64
    packed rows this is looked at before tiles 2, 4, 8, ..., for all up to the next of them, and where a
    row's unit moves up; with more for every tile, the sums are those of every second one, and the unit stays
    within 2^30 of the largest it was. s: scores in powers of two [rows, tiles, tokens]; edge: a
    factor of the sums near 1."""
    rows, tiles, tokens = s.shape
    x, sums, l2 = s.amax(-1), s.exp2().sum(-1), [torch.zeros(rows, dtype=torch.float64) for _ in range(2)]
    m, out, look, aim = torch.full((rows,), -1e30, dtype=torch.float64), torch.zeros_like(x), 2, 0.0 if wide else 1.0
    each = 1.5 * tokens / 128 * edge
    for t in range(tiles):
        g = t % 2 if wide else 0
        n = t // 2 + 1 if wide else t + 1
        up = x[:, t] - m > 8
        at = t + 1 == look
        if wide or at or bool(up.any()):
            nxt = n + 1 if wide else 2 * n if at else look
            m = torch.where(up, x[:, t] - aim, m)
            have = l2[g] * (-m).exp2() + (x[:, t] - m).exp2()
            need = each * (nxt - 1)
            bits, room = (need / have).log2(), 8 - (x[:, t] - m)
            down = torch.minimum(torch.maximum(bits + 1, m - x[:, t]), 30 - have.log2()).minimum(room)
            if wide and t > 0:
                down = torch.minimum(down, m - out[:, :t].amax(-1) + 30)
            short = (have < need) & (have > 0)
            look = t + 2 if bool((short & (room < bits)).any()) else nxt
            m = torch.where(short, m - down, m)
        l2[g] += sums[:, t]
        out[:, t] = m
    return out


def check(pmqa, p):
    few, tile = p.rows * p.heads <= 32, 128 if p.rows * p.heads <= 64 else 64
    part, step = (2.0 ** -8, 2.0 ** -14) if few else (2.0 ** -7, 2.0 ** -13)
    out, lse = run(pmqa, p)
    k, v = p.k.double() * KS, p.k[:, :512].double() * KS
    pad = -p.ctx % tile
    scores = torch.full((p.rows, p.heads, p.ctx + pad), -math.inf, dtype=torch.float64)
    for j in range(p.rows):
        scores[j, :, :p.ctx - p.rows + j + 1] = ((p.q[j].double() * QS) @ k.T * SM).cpu()[:, :p.ctx - p.rows + j + 1]
    # a block of packed rows looks together; up to 64 rows in groups of 16 or 32
    flat = scores.reshape(p.rows * p.heads, -1, tile) * math.log2(math.e)
    group = 16 if p.rows * p.heads <= 32 else 32
    unit = torch.cat([torch.maximum(*[units(x, tile == 64, e) for e in (0.999, 1.001)]) for x in flat.split(group)])
    unit = (unit * math.log(2)).reshape(p.rows, p.heads, -1).cuda()
    for j in range(p.rows):
        x = p.q[j].double() * QS
        s = x @ k.T * SM
        seen = torch.arange(p.ctx, device="cuda") <= p.ctx - p.rows + j
        s = s.masked_fill(~seen, -math.inf)
        d = (x.abs() @ k.abs().T * (SM * 580 * 2.0 ** -23) + s.abs() * 2.0 ** -20 + 2.0 ** -18).masked_fill(~seen, 0.0)
        l = torch.logsumexp(s, -1, keepdim=True)
        w = (s - l).exp()
        lost = torch.minimum(w, step * 1.01 * (unit[j] - l).exp().repeat_interleave(tile, -1)[:, :p.ctx])
        dtop = d.amax(-1, keepdim=True)
        e = (w * (part + 2.0 ** -11 + d + dtop) + lost) @ v.abs()
        o = w @ v
        tol = e + (o.abs() + e) * 2.0 ** -8
        worst = ((out[:, j] - o).abs() / tol).amax()
        assert worst <= 1.0, (j, float(worst))
        far = (lse[:, j] - l[:, 0]).abs() - (dtop[:, 0] + l[:, 0].abs() * 2.0 ** -21 + 2.0 ** -18)
        assert far.max() <= 0.0, (j, float(far.max()))


def one(ctx, at, nats):
    lift = torch.zeros(ctx)
    lift[at] = nats
    return lift


SHAPES = [(1, 1), (16, 1), (32, 1), (8, 4), (64, 1), (16, 4), (128, 1), (40, 2)]


@pytest.mark.parametrize("heads,rows", SHAPES)
@pytest.mark.parametrize("ctx", [8192, 32768, 131072])
@pytest.mark.parametrize("where", ["start", "middle", "end"])
def test_one_heavy_token_among_light_ones(cuda_lib, heads, rows, ctx, where):
    """80 % of the weight, with a value of zero: the output is what the light tokens give."""
    at = dict(start=0, middle=ctx // 2 + 5, end=ctx - rows - 2)[where]
    check(cuda_lib, problem(heads, rows, ctx, one(ctx, at, math.log(4 * ctx) + 0.5)))


@pytest.mark.parametrize("heads,rows", SHAPES)
@pytest.mark.parametrize("nats", [3.0, 6.0, 14.0, 20.0, 28.0, 45.0])
def test_light_tokens_of_equal_scores(cuda_lib, heads, rows, nats):
    """Equal weights are all rounded the same way."""
    ctx = 16384
    lift = torch.zeros(ctx)
    lift[[0, 5000]] = nats
    check(cuda_lib, problem(heads, rows, ctx, lift, sigma=0.0))


@pytest.mark.parametrize("heads,rows", SHAPES)
@pytest.mark.parametrize("kind", ["falling", "rising", "turns", "peaks", "wide"])
def test_scores_that_move_along_the_context(cuda_lib, heads, rows, kind):
    """Down and up by many powers of two, a tile at a time, and scores spread over many."""
    ctx = 10007
    t = torch.arange(ctx)
    lift = dict(falling=50.0 * (1 - t / ctx), rising=50.0 * t / ctx, turns=40.0 * (t // 128 % 2),
                peaks=30.0 * (t % 640 == 77) + 8.0 * (t % 128 == 3), wide=torch.zeros(ctx))[kind]
    p = problem(heads, rows, ctx, lift, sigma=6.0 if kind == "wide" else 1.0, seed=2)
    g = torch.Generator(device="cuda").manual_seed(3)
    p.k[:, :512] = (torch.randn((ctx, 512), generator=g, device="cuda") + 1.0).div(KS).clamp(-448, 448).to(ref.F8)
    check(cuda_lib, p)


@pytest.mark.parametrize("heads,rows", SHAPES)
@pytest.mark.parametrize("nats", [70.0, 100.0, 200.0, 330.0])
@pytest.mark.parametrize("at", [[0], [64], [70, 2000], [0, 64, 128, 1999, 2500]])
def test_tokens_that_outweigh_the_others_by_far(cuda_lib, heads, rows, nats, at):
    """By more than fp32's range; all weights but theirs are next to nothing."""
    lift = torch.zeros(3000)
    lift[at] = nats
    check(cuda_lib, problem(heads, rows, 3000, lift, q_lift=448.0, zero=False))


@pytest.mark.parametrize("heads,rows", [(16, 4), (8, 4), (40, 2), (128, 3)])
def test_a_heavy_token_that_the_last_row_alone_sees(cuda_lib, heads, rows):
    ctx = 20000
    check(cuda_lib, problem(heads, rows, ctx, one(ctx, ctx - 1, 14.0)))
