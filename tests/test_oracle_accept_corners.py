"""The oracle's chain and tree where a draft came with probability 0."""

import numpy as np
import pytest

from oracle import accept, tree


@pytest.mark.parametrize("z,accepted", [(-np.inf, False), (-300.0, True), (0.0, True)])
def test_a_draft_that_came_with_probability_0(z, accepted):
    logits = np.zeros((2, 6), np.float32)
    logits[0, 4] = z
    q = np.full((1, 6), 0.2, np.float32)
    q[0, 4] = 0.0
    chain = accept.sampled_accept_detail(logits, q, [4], 1.0, np.array([0.5, 0.3], np.float32))
    path, tokens, _ = tree.accept(logits, [-1, 0], [0, 4], 1.0, q=np.concatenate([q, q]), u=np.array([0.3, 0.5], np.float32))
    assert (path == [0, 1]) == accepted and (tokens[0] == 4) == accepted
    assert chain["out_len"] == len(path) and chain["tokens"] == tokens and (chain["reject"] == -1) == accepted
