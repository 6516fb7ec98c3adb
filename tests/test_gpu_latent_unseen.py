"""Tokens that no row sees: they have no effect, and nothing behind a context is looked up."""

import pytest
import torch

from tests import step_ref as ref
from tests.test_gpu_latent_attention import check, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads", [1, 16, 24, 64, 128])
@pytest.mark.parametrize("rows,ctx", [([1, 1], [127, 130]), ([3, 2], [128, 64]), ([2, 5], [61, 193]), ([1, 40], [700, 257])])
def test_entries_behind_a_context_are_not_looked_up(cuda_lib, heads, rows, ctx):
    """Bad table entries from the first one behind each context on, with pages of one token and of
    several: nothing is reported. The last page's unused slots hold NaN."""
    for block in (1, 8):
        p = ref.attention_problem(rows, ctx, heads, block, seed=heads + block)
        for i, c in enumerate(ctx):
            p.bt[i, -(-c // block):] = p.nb + 7 if i else -3
        assert check(run(cuda_lib, p), ref.attention(p), p) == 0


@pytest.mark.parametrize("heads", [1, 16, 24, 64, 128])
def test_nan_that_only_other_requests_see(cuda_lib, heads):
    """A request whose tokens are all NaN between two others: its rows are NaN, theirs are not."""
    p = ref.attention_problem([2, 3, 1], [130, 70, 200], heads, 16, seed=heads)
    p.kv.reshape(-1, 576)[ref.places(p, 1, 0, 70)] = ref.NAN8
    got = run(cuda_lib, p)
    assert check(got, ref.attention(p), p) == 0
    assert bool(got[0][2:5].isnan().all()) and not bool(got[0][:2].isnan().any()) and not bool(got[0][5:].isnan().any())
