"""Drafts that neither distribution holds, and what the call does not read."""

import numpy as np
import pytest
import torch

from oracle import tree as ot
from tests.test_gpu_tree_accept import Case, dev

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("stats", [False, True])
@pytest.mark.parametrize("z,accepted", [(-np.inf, False), (-30.0, True), (0.0, True), (-300.0, True)])
def test_a_draft_that_came_with_probability_0(lib, stats, z, accepted):
    """q(x) = 0: taken where p(x) > 0, however small, and not where p(x) = 0; a chain and a tree of one child alike."""
    c = Case(70, [2], 50, 0.9, "independent")
    c.token[1] = 7
    c.z[0, 7], c.q[0, 7] = z, 0.0
    c.u[:] = [0.3, 0.5]
    length, tokens, _ = c.call(lib, stats)
    assert length.item() == 1 + accepted and (tokens[0].item() == 7) == accepted
    want = ot.accept(c.z, c.parent.tolist(), c.token.tolist(), c.T, c.q, c.u)[1]   # (its margin is 0 here: it says which side is the rule's)
    assert tokens[0].item() == want[0]
    n, chain = lib.spec_accept_batched(c.offs, dev(c.z), dev(c.token[1:]), c.T, q=dev(c.q[:1]), u=dev(c.u[::-1].copy()))
    assert n.item() == length.item() and chain[0].item() == tokens[0].item()


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
