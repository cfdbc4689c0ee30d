"""Where the rule of a draft tree and that of a chain part, and what the tree's call does not read."""

import numpy as np
import pytest
import torch

from oracle import tree as ot
from tests.test_gpu_tree_accept import Case, dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("stats", [False, True])
def test_a_draft_that_neither_distribution_holds(lib, stats):
    """q(x) = p(x) = 0: 0 < 0 rejects it in a tree; the chain's ratio is infinite and accepts it."""
    c = Case(70, [2], 50, 0.9, "independent")
    c.token[1] = 7
    c.z[0, 7], c.q[0, 7] = -np.inf, 0.0
    c.u[:] = [0.3, 0.5]
    length, tokens, _ = c.call(lib, stats)
    assert length.item() == 1 and tokens[0].item() != 7
    want = ot.accept(c.z, c.parent.tolist(), c.token.tolist(), c.T, c.q, c.u)   # (its margin is 0: it says which side is the rule's)
    assert want[0] == [0] and tokens[0].item() == want[1][0]
    n, chain = lib.spec_accept_batched(c.offs, dev(c.z), dev(c.token[1:]), c.T, q=dev(c.q[:1]), u=dev(c.u[::-1].copy()))
    assert n.item() == 2 and chain[0].item() == 7


@pytest.mark.parametrize("mode", ["independent", "distinct"])
def test_what_is_not_read(lib, mode):
    """q of nodes without children, the anchor's token and parent, rows behind the last request's: NaN and nonsense there change nothing."""
    c = Case(71, [12, 5, 1], 400, 0.8, mode)
    want = c.call(lib)
    leaf = [i for b, n in enumerate(c.counts) for i in range(c.offs[b], c.offs[b] + n) if i - c.offs[b] not in c.parent[c.offs[b] + 1:c.offs[b] + n]]
    assert 17 in leaf and len(leaf) > 4
    c.q[leaf] = np.nan
    c.parent[c.offs[:-1]], c.token[c.offs[:-1]] = 10 ** 6, -10 ** 6
    z, q, u = (np.concatenate([x, np.full((3,) + x.shape[1:], np.nan, np.float32)]) for x in (c.z, c.q, c.u))
    p, t = (np.concatenate([x, np.full(3, -5, np.int32)]) for x in (c.parent, c.token))
    got = lib.tree_accept(c.offs, dev(z), dev(p), dev(t), c.T, q=dev(q), u=dev(u), distinct=mode == "distinct")
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and lib.device_error() == 0
