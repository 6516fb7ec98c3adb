"""What else the operators on the 8-bit K/V cache refuse before they touch the
device: outputs that overlap inputs in part."""

import ctypes

import pytest

from sparse_attention_indexer_pmqa_gb300 import build, pmqa
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
