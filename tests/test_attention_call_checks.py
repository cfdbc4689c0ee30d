"""Refusals of the attention-side calls that need no GPU: limits of their arguments and what the binding hands over."""

import ctypes

import pytest

from speculative_decoding_verify_qmm_gb300 import binding, build
from speculative_decoding_verify_qmm_gb300.binding import SV_EINVAL
from tests.test_attention_refusals import _attend, _cache


@pytest.fixture(scope="module")
def raw():
    build.build()
    return binding.load_library()


@pytest.mark.parametrize("scale", [1.8e38, -1.8e38, 3.4e38])
def test_tree_attention_refuses_a_scale_out_of_range(raw, scale):
    assert _attend(raw, _cache(), scale=scale) == SV_EINVAL
    assert _attend(raw, _cache(), scale=scale / 2, offs=(ctypes.c_int32 * 2)(0, 0)) == binding.SV_OK


def test_tree_attention_in_place_needs_equal_strides(raw):
    """Some blocks would write rows that others still read.  One row has no stride."""
    assert _attend(raw, _cache(), q=4096, out=4096, ldq=256, ldo=264) == SV_EINVAL
    assert _attend(raw, _cache(), q=4096, out=4096, ldq=264, ldo=256) == SV_EINVAL
    assert b"equal strides" in raw.sv_last_error()
    status = _attend(raw, _cache(), q=4096, out=4096, ldq=264, ldo=256, offs=(ctypes.c_int32 * 2)(0, 1), ws=None)
    assert status == SV_EINVAL and b"workspace" in raw.sv_last_error()        # passed that check and stopped at a later one
