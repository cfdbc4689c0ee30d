"""Tree accept with everything in one buffer, side by side: the same results; one element nearer, and the call is refused."""

import pytest
import torch

from speculative_decoding_verify_qmm_gb300.binding import SVError
from tests.test_gpu_tree_accept import Case, dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("mode", ["greedy", "independent"])
def test_adjacent_arrays(lib, mode):
    c = Case(60, [9, 4], 301, 0.0 if mode == "greedy" else 0.7, mode)
    rows, most = 13, 9
    ints = torch.full((2 * rows + 2 + rows + 2 * most,), -1, dtype=torch.int32, device="cuda")
    parent, token = ints[:rows], ints[rows:2 * rows]
    parent.copy_(dev(c.parent)), token.copy_(dev(c.token))
    out = (ints[2 * rows:2 * rows + 2], ints[2 * rows + 2:3 * rows + 2], ints[3 * rows + 2:].view(2, most))
    args = dict(q=None if c.q is None else dev(c.q), u=dev(c.u))
    lib.tree_accept(c.offs, dev(c.z), parent, token, c.T, out=out, **args)
    c.check(out)
    assert lib.device_error() == 0
    for bad in ((ints[2 * rows - 1:2 * rows + 1], out[1], out[2]), (out[0], ints[2 * rows + 1:3 * rows + 1], out[2]),
                (out[0], out[1], ints[3 * rows + 1:3 * rows + 1 + 2 * most].view(2, most)), (out[0], token, out[2])):
        with pytest.raises(SVError, match="overlap"):
            lib.tree_accept(c.offs, dev(c.z), parent, token, c.T, out=bad, **args)
