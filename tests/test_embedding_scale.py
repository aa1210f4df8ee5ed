"""The embedding's gradient with scales that are negative or not finite: rows
without a token become zeros all the same."""
import numpy as np
import pytest

import block_quantized_communication_amd as zpq

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [float("inf"), float("nan"), -2.0, 0.0])
@pytest.mark.parametrize("tokens,rows,dim", [(5, 9, 3), (40, 300, 24), (700, 1000, 600), (5000, 70000, 7),
                                             (30000, 900, 16)])
def test_rows_without_a_token_are_zeros(tokens, rows, dim, scale):
    import torch
    ids = np.random.default_rng(tokens).integers(0, rows // 3, tokens) * 3          # two rows of three get none
    t = torch.from_numpy(ids).cuda()
    y = torch.ones(tokens, dim, device="cuda")
    n = torch.from_numpy(np.bincount(ids, minlength=rows)).cuda()
    want = (n.float() * scale)[:, None].expand(rows, dim).clone()                   # exact: counts below 2^24
    want[n == 0] = 0.0
    g = zpq.embedding_grad(t, y, rows, scale=scale)
    assert torch.equal(g.nan_to_num(7.0, 8.0, 9.0), want.nan_to_num(7.0, 8.0, 9.0))
    assert not bool(torch.signbit(g[n == 0]).any())
    old = torch.full((rows, dim), 3.0, device="cuda")
    zpq.embedding_grad(t, y, rows, scale=scale, out=old, accumulate=True)
    assert bool((old[n == 0] == 3.0).all())
