"""Sizes of a page state at the limits of what its calls count in: refused on the host, before any launch."""

import ctypes

import pytest

from speculative_decoding_verify_qmm_gb300 import binding, build
from speculative_decoding_verify_qmm_gb300.binding import SV_EUNSUPPORTED, SV_OK
from tests.test_shared_refusals import _pool


@pytest.fixture(scope="module")
def raw():
    build.build()
    return binding.load_library()


@pytest.mark.parametrize("slots,width,page", [(256, (1 << 22) + 1, 16), (256, 1 << 23, 128), (17, 1 << 26, 16), (256, 1 << 26, 16), (255, 4210753, 16)])
def test_tables_of_more_entries_than_a_call_counts_are_refused(raw, slots, width, page):
    """reserve adds the entries that 256 slots will write in 32 bits: from 2^31 on it would have seen none of them."""
    pool = _pool(slots=slots, table_pages=width, page_size=page)
    ref = ctypes.byref(pool)
    assert raw.sv_kv_reserve_workspace_bytes(ref) == 0
    assert raw.sv_kv_fork(ref, 1, 16, 16, 16, None) == SV_EUNSUPPORTED and b"table_pages" in raw.sv_last_error()
    assert raw.sv_kv_reserve(ref, None, 0, 16, 16, 16, 16, 256, 1 << 20, None) == SV_EUNSUPPORTED
    assert raw.sv_kv_compact(ref, None, 0, 16, 16, None) == SV_EUNSUPPORTED


@pytest.mark.parametrize("slots,width,page", [(256, 1 << 22, 16), (16, 1 << 26, 16), (1, 1 << 26, 16), (256, 1 << 14, 65536)])
def test_the_largest_tables_are_accepted(raw, slots, width, page):
    ref = ctypes.byref(_pool(slots=slots, table_pages=width, page_size=page))
    assert raw.sv_kv_reserve_workspace_bytes(ref) > 0
    assert raw.sv_kv_fork(ref, 0, None, None, None, None) == SV_OK
