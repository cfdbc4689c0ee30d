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


def _host(lib):
    """A cache of host tensors: what the binding checks before it asks for their device."""
    import torch
    k, v = torch.zeros((2, 2, 16, 64), dtype=torch.bfloat16), torch.zeros((2, 2, 16, 64), dtype=torch.bfloat16)
    cache = binding.KVCache(binding.KVCacheView(k.data_ptr(), v.data_ptr(), None, None, None, None, 2, 16, 2, 64, 16), [k, v])
    ints = lambda *s: torch.zeros(s, dtype=torch.int32)                       # noqa: E731
    return cache, ints, torch.zeros((4, 128), dtype=torch.bfloat16)


@pytest.mark.parametrize("offs", [[0, 2 ** 32 + 2], [0, 2 ** 32], [2 ** 32, 2], [0, -2 ** 32], [0, 3, 0], [3, 0], [], [0, -1],
                                  (ctypes.c_int32 * 3)(0, 3, 0), (ctypes.c_int64 * 2)(0, 2 ** 32 + 1)])
def test_binding_refuses_row_offsets(offs):
    """Numbers that a C int would take for others, and offsets that go down to no rows at all."""
    build.build()
    lib = binding.load()
    cache, ints, x = _host(lib)
    args = (ints(4), ints(4, 2))
    for call in (lambda: lib.kv_append(cache, offs, *args, x, x), lambda: lib.kv_read(cache, offs, *args, x, x),
                 lambda: lib.kv_read(cache, offs, *args), lambda: lib.tree_attention(cache, offs, *args, x, 2)):
        with pytest.raises(binding.SVError, match="row_offsets"):
            call()


def test_binding_refuses_strides_past_a_c_int():
    import torch
    far = torch.empty_strided((2, 128), (2 ** 32 + 128, 1), dtype=torch.bfloat16, device="meta")
    with pytest.raises(binding.SVError, match="row stride"):
        binding._matrix("q", far, torch.bfloat16, -1, 2, 128)
    assert binding._matrix("q", far[:1], torch.bfloat16, -1, 1, 128) >= 128   # one row: no stride is used
    near = torch.empty_strided((2, 128), (2 ** 31 - 8, 1), dtype=torch.bfloat16, device="meta")
    assert binding._matrix("q", near, torch.bfloat16, -1, 2, 128) == 2 ** 31 - 8


def test_workspace_query_of_bad_offsets_is_zero():
    build.build()
    lib = binding.load()
    cache, _, _ = _host(lib)
    assert lib.tree_attention_workspace_bytes(cache, [0, 2], 2) > 0
    for offs in ([0, -1], [], [0], [1, 2], [0, 65]):
        assert lib.tree_attention_workspace_bytes(cache, offs, 2) == 0
