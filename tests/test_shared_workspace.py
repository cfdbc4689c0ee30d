"""The workspace of attention over shared prefixes, as its query gives it: one that is sized for the largest batch serves every
smaller one, whatever the lengths of the prefixes."""

import ctypes
import random

import pytest

from speculative_decoding_verify_qmm_gb300 import binding, build
from tests.test_attention_refusals import _cache, _offs


@pytest.fixture(scope="module")
def raw():
    build.build()
    return binding.load_library()


def size(raw, counts, groups, pages, hq, hk, dim, page=64):
    """Of requests with these rows in groups of these many requests."""
    offs, goffs = [0], [0]
    for n in counts:
        offs.append(offs[-1] + n)
    for n in groups:
        goffs.append(goffs[-1] + n)
    cache = _cache(n_kv_heads=hk, head_dim=dim, page_size=page, n_pages=1000)
    got = raw.sv_tree_attention_shared_workspace_bytes(ctypes.byref(cache), len(groups), _offs(*goffs), _offs(*pages), len(counts), _offs(*offs), hq)
    assert got > 0, raw.sv_last_error()
    return got


@pytest.mark.parametrize("rows,tokens,fewer,shorter", [(16, 16384, 12, 16384), (8, 24384, 8, 24320), (32, 20000, 32, 16384), (33, 16384, 32, 16384)])
def test_fewer_rows_and_other_prefixes_need_no_more(raw, rows, tokens, fewer, shorter):
    most = size(raw, [rows] * 16, [16], [tokens // 16], 32, 8, 128, page=16)
    for n in (fewer, 1):
        for t in (shorter, tokens, 16, 0):
            assert size(raw, [n] * 16, [16], [t // 16], 32, 8, 128, page=16) <= most


@pytest.mark.parametrize("seed", range(60))
def test_less_of_a_batch_never_needs_more(raw, seed):
    r = random.Random(seed)
    hk = r.choice([1, 2, 8])
    hq, dim = hk * r.randint(1, 16), r.choice([64, 128])
    groups = [r.randint(0, 12) for _ in range(r.randint(1, 6))] + [1]
    widest = r.choice([2, 4, 9, 32, 64])
    counts = [r.randint(0, widest) for _ in range(sum(groups))]
    pages = [r.randint(0, 2000) for _ in groups]
    most = size(raw, counts, groups, pages, hq, hk, dim)
    for _ in range(20):
        assert size(raw, counts, groups, [r.randint(0, 2000) for _ in groups], hq, hk, dim) == most
    # rows go, then requests, then groups
    while len(counts) > 1:
        kind = r.randrange(3)
        b = r.randrange(len(counts))
        if kind == 0:
            counts[b] = r.randint(0, counts[b])
        elif kind == 1:
            g = next(g for g in range(len(groups)) if sum(groups[:g + 1]) > b)
            groups[g] -= 1
            del counts[b]
        elif len(groups) > 1:
            g = r.randrange(len(groups))
            if sum(groups) == groups[g]:
                continue
            first = sum(groups[:g])
            del counts[first:first + groups[g]]
            del groups[g], pages[g]
        now = size(raw, counts, groups, [r.randint(0, 2000) for _ in groups], hq, hk, dim)
        assert now <= most
        most = now
