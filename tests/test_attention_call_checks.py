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
