"""Blocks of rows that end inside a warp: lanes with a row beside lanes without one, at every place of a block of the tensor-core kernels."""

import numpy as np
import pytest

from tests.test_gpu_attention import attend_case, i32
from tests.test_gpu_attention_limits import check
from tests.test_gpu_attention_shared import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("requests", [2, 31, 33, 50, 95, 97, 127, 129, 150, 161, 223, 255])
def test_blocks_of_a_shared_prefix(lib, bits, requests):
    """A row each behind one prefix: as many rows a key head as there are requests."""
    pages = -(-500000 // ((requests - 1) * 8 * 64))
    b = Batch(lib, requests + bits, bits, [[(1, i % 7) for i in range(requests)]], [pages], 8, 8, 128 if requests % 4 else 64, 64)
    assert b.shares()
    out = b.call()
    assert lib.device_error() == 0
    b.check(out, requests=sorted({0, 1, 30 % requests, requests // 2, requests - 2, requests - 1}))


@pytest.mark.parametrize("bits", [16, 8, 4])
@pytest.mark.parametrize("rows,hq", [(1, 33), (3, 15), (5, 13), (3, 27), (2, 49), (3, 37), (1, 64), (7, 21), (3, 50)])
def test_blocks_of_a_request(lib, bits, rows, hq):
    """33 to 150 rows over one key head, in one tile and in several CTAs' shares of many."""
    for length in (40, 3000):
        cache, offs, table, q, _ = attend_case(lib, np.random.default_rng(rows + hq), bits, [rows], [length], hq, 1, 128, 64, qscale=1.0)
        out = lib.tree_attention(cache, offs, i32([length]), i32(table.tolist()), q.cuda(), hq)
        assert lib.device_error() == 0
        check(out, cache, bits, offs, [length], table, 64, q, hq, 128 ** -0.5)
