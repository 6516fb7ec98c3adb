"""Values of the cache operators inside bounds that stay a small part of them."""

import pytest

from tests import cache_bounds as cb
from tests import cache_ref as ref
from tests.test_gpu_cache import status_is
from tests.test_gpu_cache_paths import attend

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------- long contexts

LONG = [
    # rows, ctx, kv_heads, group, head_dim, block
    ([2], [20000], 1, 4, 64, 64),
    ([1], [60000], 1, 8, 128, 64),
    ([1, 2], [30000, 9000], 2, 12, 128, 48),
    ([40], [5000], 1, 1, 128, 64),
    ([5, 1, 5], [3100, 700, 2049], 2, 8, 64, 48),
    ([9, 12], [9000, 12345], 1, 6, 128, 24),
]


@pytest.mark.parametrize("flat", [False, True])
@pytest.mark.parametrize("case", LONG)
def test_values_of_long_contexts(cuda_lib, case, flat):
    rows, ctx, H, G, D, P = case
    p = ref.make(rows, ctx, kv_heads=H, group=G, head_dim=D, block=P, seed=41)
    if flat:
        p.q *= 0.125  # every token has some of the weight: a lost part shows
    ws = cuda_lib.cache_workspace()
    out, lse = attend(cuda_lib, p, ws=ws)
    status_is(cuda_lib, ws)
    cb.matches(p, out, lse)
