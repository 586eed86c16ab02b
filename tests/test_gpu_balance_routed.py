"""num_routed where a warp's lanes go different ways: ragged chunks, slots of every kind, ids that collide."""

import pytest
import torch

import combine_get_layout_02_b200 as cgl

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("k", [1, 3, 4, 8, 13, 32])
@pytest.mark.parametrize("n,S", [(1, 1), (31, 1), (33, 1), (511, 1), (513, 1), (1025, 5), (4097, 1), (16411, 1), (9999, 3), (70001, 1)])
def test_routed_tokens_of_ragged_batches(n, S, k):
    g = torch.Generator().manual_seed(n + k)
    e = 24
    idx = torch.randint(0, e, (n, k), generator=g, dtype=torch.int32)
    idx[torch.rand(n, generator=g) < 0.5] = -1                        # padding, half of the lanes
    idx[torch.rand(n, k, generator=g) < 0.3] = -1
    one = torch.rand(n, generator=g) < 0.2                            # every lane the same expert
    idx[one, 0] = 5
    bad = torch.rand(n, k, generator=g) < 0.02                        # out of range: not counted
    idx[bad] = torch.where(torch.rand(n, k, generator=g)[bad] < 0.5, e, -7).int()
    ok = (idx >= 0) & (idx < e)
    routed = ok.any(1).view(S, -1).sum(1).int()
    counts = torch.stack([torch.bincount(i[o].long(), minlength=e) for i, o in zip(idx.view(S, -1), ok.view(S, -1))]).int()
    logits = torch.zeros(n, e, device="cuda")
    for _ in range(3):
        b = cgl.balance_loss(logits, idx.cuda(), num_sequences=S)
        assert torch.equal(b.num_routed.cpu(), routed) and torch.equal(b.counts.cpu(), counts)
