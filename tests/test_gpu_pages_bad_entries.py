"""Entries of the block tables that name no page of the cache, or none in use: reported, and what they belong to is left alone."""

import pytest
import torch

from tests.test_gpu_attention import i32
from tests.test_gpu_pages import World

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page", [-1, 12, 2 ** 31 - 1, -2 ** 31])
@pytest.mark.parametrize("keep,need,entry", [(0, 0, 0), (0, 0, 3), (0, 0, 1), (20, 20, 2), (20, 20, 3), (16, 16, 1), (20, 30, 2), (5, 20, 3), (48, 48, 3)])
def test_a_free_or_trim_with_a_bad_entry_leaves_the_slot_alone(lib, keep, need, entry, page):
    w = World(lib, 20, 12, 16, 4, 5)
    w.reserve([0] * 4, [60, 5, 40, -1])
    w.fork([0], [3], [25])                                       # (its half-filled page is shared)
    good = w.model.table[0][entry]
    w.pages.block_table[0, entry] = page
    counts, _ = lib.kv_reserve(w.pages, w.caches, i32([keep, 5, 0, 25]), i32([need, 20, 0, -1]), workspace=w.ws)
    assert lib.device_error() == 4 and counts.tolist() == [0, 0, 1] and not w.ws.any()
    assert w.pages.block_table[0, entry].item() == page
    w.pages.block_table[0, entry] = good
    w.model.reserve([0, 5, 0, 25], [-1, 20, 0, -1])
    w.check()
    w.reserve([keep, 0, 0, 0], [need, 0, -1, 0])                 # put right, the same call works
    w.check()


def test_a_bad_entry_far_behind(lib):
    """Longer tables than a warp looks at in one step; entries that are kept are not looked at."""
    w = World(lib, 21, 1000, 16, 2, 900)
    w.reserve([0, 0], [900 * 16, 16])
    good = w.model.table[0][700]
    w.pages.block_table[0, 700] = 1000
    for keep in (0, 16, 699 * 16, 700 * 16):
        lib.kv_reserve(w.pages, w.caches, i32([keep, 0]), i32([keep, -1]), workspace=w.ws)
        assert lib.device_error() == 4 and w.pages.held.tolist() == [900, 1]
    counts, _ = lib.kv_reserve(w.pages, w.caches, i32([701 * 16, 0]), i32([701 * 16, -1]), workspace=w.ws)
    assert lib.device_error() == 0 and counts.tolist() == [0, 0, 0]
    w.pages.block_table[0, 700] = good
    w.model.reserve([701 * 16, 0], [701 * 16, -1])
    w.check()


def test_bad_entries_among_many_slots(lib):
    """Every third slot has one; the others are freed as if those were not there."""
    w = World(lib, 22, 600, 16, 100, 6)
    need = [1 + (7 * s) % 90 for s in range(100)]
    w.reserve([0] * 100, need)
    good = w.pages.block_table.clone()
    for s in range(0, 100, 3):
        w.pages.block_table[s, (s // 3) % w.model.held[s]] = -1 - s
    lib.kv_reserve(w.pages, w.caches, i32([0] * 100), i32([0] * 100), workspace=w.ws)
    assert lib.device_error() == 4 and not w.ws.any()
    w.pages.block_table.copy_(good)
    w.model.reserve([0] * 100, [-1 if s % 3 == 0 else 0 for s in range(100)])
    w.check()
    assert torch.equal(w.pages.block_table, good)


def test_compact_reports_entries_that_name_no_page_in_use(lib):
    """A stale entry of each kind: a hole that is filled, a page behind the last in use, one outside the cache."""
    def world():
        w = World(lib, 23, 20, 16, 5, 6)
        w.reserve([0] * 5, [40, 30, 60, 20, 33])
        w.reserve([0] * 5, [-1, 0, -1, 0, -1])                   # pages 3, 4 and 9, 10 are free now
        return w
    w = world()
    assert [i for i, r in enumerate(w.model.refs) if not r] == [3, 4, 9, 10] + list(range(14, 20))
    for slot, entry, stale in ((0, 1, 3), (0, 0, 4), (2, 3, 9), (4, 2, 10), (4, 0, 14), (2, 1, 19), (0, 2, 20), (2, 0, -1), (4, 1, 2 ** 31 - 1)):
        w = world()
        live, moves = w.model.compact()
        assert live == 10 and moves == [(11, 3), (12, 4), (13, 9)]
        w.pages.block_table[slot, entry] = stale
        counts, out = lib.kv_compact(w.pages, w.caches)
        low = stale in (3, 4, 9)
        assert lib.device_error() == 4, (slot, entry, stale)
        assert counts.tolist() == [live, 3] and out[:3].tolist() == [list(m) for m in moves] and low == (stale in [d for _, d in moves])
        assert w.pages.block_table[slot, entry].item() == stale
        w.pages.block_table[slot, entry] = w.model.table[slot][entry]
        w.check()


def test_compact_of_what_is_dense_already(lib):
    """Nothing moves: every entry in use stands, the others are reported."""
    w = World(lib, 24, 9, 16, 3, 4)
    w.reserve([0] * 3, [40, 30, -1])
    w.fork([0], [2], [40])
    w.compact()
    w.check()
    for stale in (5, 8, 9, -1):
        w.pages.block_table[1, 1] = stale
        counts, _ = lib.kv_compact(w.pages, w.caches)
        assert lib.device_error() == 4 and counts.tolist() == [5, 0] and w.pages.block_table[1, 1].item() == stale
