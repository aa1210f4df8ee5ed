"""The smallest eps that the step accepts: the root of a second moment below
binary32's normal range counts there."""
import numpy as np
import pytest

import block_quantized_communication_amd as zpq
import step_ref as ref

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("eps", [1e-30, 1e-20, 1e-15, 1e-8])
@pytest.mark.parametrize("first_step", [1, 1000])
def test_small_gradients_and_small_eps(eps, bits, first_step):
    """Gradients from 1e-21 (squares of few bits) to 1, steps of the order of lr each.
    The new moments are those of binary32, operation by operation; from them the update
    in 64 bits, which binary32 gives within the roundings counted below."""
    import torch
    gen = np.random.default_rng(1)
    rows = [gen.standard_normal(256) * 10.0 ** e for e in (-21, -20, -19, -18.5, -18, -17, -12, -6, 0)]
    g0 = np.concatenate(rows).astype(np.float32)
    n = g0.size
    p, g = torch.zeros(n, device="cuda"), torch.from_numpy(g0).cuda()
    lr, betas = 1e-2, (0.9, 0.99)
    opt = zpq.AdamW([p], [g], lr=lr, betas=betas, eps=eps, weight_decay=0.0, state_bits=bits, seed=7)
    opt.step(first_step)
    m, v = ref.adamw32_moments(g0, np.zeros(n), np.zeros(n), 1.0, betas)
    if bits == 32:
        assert np.array_equal(opt.exp_avg[0].cpu().numpy(), m) and np.array_equal(opt.exp_avg_sq[0].cpu().numpy(), v)
    m, v = m.astype(np.float64), v.astype(np.float64)
    den = np.sqrt(v) / np.sqrt(1 - betas[1] ** first_step) + eps
    want = -lr / (1 - betas[0] ** first_step) * m / den
    assert np.any((v > 0) & (v < 2.0 ** -126)) and np.any(v > 1e-6)
    # in U: root 2, its constant and product 2, eps and sum 2, reciprocal 2, product 1, rate and its product 2: 11,
    # and what they do to one another
    off = 12 * ref.U * np.abs(want) + 2e-45
    got = p.double().cpu().numpy()
    assert np.all(np.abs(got - want) <= off), np.max(np.abs(got - want) / off)
