"""One workspace, sized for the largest batch, under smaller ones and other prefixes: attention over shared prefixes gives what it gives in a
workspace of its own, and leaves zeros."""

import pytest
import torch

from tests.test_gpu_attention_shared import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [16, 4])
def test_the_largest_batch_s_workspace_serves_all(lib, bits):
    hq, hk, d, page = 32, 8, 128, 16
    sizes = [([[(12, 20)] * 8], [600]), ([[(12, 3)] * 8], [603]), ([[(9, 40)] * 8], [1040]), ([[(1, 30)] * 8], [2100]), ([[(12, 9)] * 3], [2000]),
             ([[(8, 20)] * 6], [800]), ([[(3, 0), (12, 5), (0, 9), (7, 11)]], [2000]), ([[(12, 20)] * 8], [0])]
    batches = [Batch(lib, 80 + i, bits, groups, shared, hq, hk, d, page) for i, (groups, shared) in enumerate(sizes)]
    need = [lib.tree_attention_shared_workspace_bytes(b.cache, b.groups, b.offs, hq) for b in batches]
    assert max(need) == need[0] and [b.shares() for b in batches] == [True] * 7 + [False]
    ws = torch.zeros(need[0] + 4096, dtype=torch.uint8, device="cuda")
    ws[need[0]:] = 77
    for _ in range(2):
        for b in batches:
            got = b.call(workspace=ws[:need[0]])
            assert torch.equal(got, b.call()) and not ws[:need[0]].any() and (ws[need[0]:] == 77).all()
    for b in batches:
        b.check(b.call(workspace=ws[:need[0]]), requests=[0, len(b.counts) - 1])
    assert lib.device_error() == 0
