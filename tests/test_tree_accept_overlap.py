"""Tree accept refuses outputs that lie in its inputs or in each other, before any launch: the CTAs of a request read the tree one by one
and have to see the same."""

import pytest

from speculative_decoding_verify_qmm_gb300 import binding, build
from speculative_decoding_verify_qmm_gb300.binding import SV_EINVAL
from tests.test_attention_refusals import _offs

ROWS, V, MOST = 5, 100, 3
MB = 1 << 20
# each array a megabyte on
INPUTS = ["logits", "row_max", "row_sumexp", "row_argmax", "parent", "token", "q", "u"]
OUTPUTS = {"out_len": 2, "out_tokens": ROWS, "path": 2 * MOST}
SIZES = dict(OUTPUTS, logits=ROWS * V, q=ROWS * V, row_max=ROWS, row_sumexp=ROWS, row_argmax=ROWS, parent=ROWS, token=ROWS, u=ROWS)


@pytest.fixture(scope="module")
def raw():
    build.build()
    return binding.load_library()


def call(raw, at, T=0.5):
    return raw.sv_tree_accept(2, _offs(0, 3, 5), at["logits"], V, at["row_max"], at["row_sumexp"], at["row_argmax"], at["parent"], at["token"],
                              at["q"], V, 0, V, T, at["u"], 0, 1.0, at["out_len"], at["out_tokens"], at["path"], MOST, None, 0, None)


@pytest.mark.parametrize("out", OUTPUTS)
@pytest.mark.parametrize("other", INPUTS + list(OUTPUTS))
def test_overlaps_are_refused(raw, out, other):
    if out == other:
        return
    base = {name: (i + 1) * MB for i, name in enumerate(INPUTS + list(OUTPUTS))}
    for shift in (0, SIZES[other] - 1, 1 - SIZES[out]):          # at its beginning, in its last element, its own last element there
        at = dict(base)
        at[out] = base[other] + 4 * shift
        assert call(raw, at) == SV_EINVAL, shift
        assert b"overlap" in raw.sv_last_error()


@pytest.mark.parametrize("T", [0.0, 0.5])
def test_the_tree_s_own_arrays_are_no_place_for_results(raw, T):
    base = {name: (i + 1) * MB for i, name in enumerate(INPUTS + list(OUTPUTS))}
    assert call(raw, dict(base, out_tokens=base["token"]), T) == SV_EINVAL
    assert call(raw, dict(base, path=base["parent"]), T) == SV_EINVAL
