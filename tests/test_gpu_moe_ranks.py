"""Order of the chosen experts where logits are infinite or NaN."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("t", [1, 6, 70])
@pytest.mark.parametrize("e", [5, 100, 300])
def test_nan_ranks_below_minus_infinity(t, e):
    """An infinite activation: logits are +-infinity by the sign of the
    router's value, NaN where it is 0.  Numbers come first, the largest first,
    then NaN; ties go to the lowest index."""
    import fp8_tensor_scaled_amd as f
    d, h, k = 64, 16, 5
    rng = np.random.default_rng(t + e)
    r = np.zeros((e, d), np.float32)
    r[:, 0] = rng.choice([-1.0, 0.0], e)
    r[rng.integers(0, e, 2), 0] = 1.0
    r[0, 0], r[1, 0] = 0.0, -1.0
    x = np.ones((t, d), np.float32)
    x[:, 0] = np.inf
    logit = np.where(r[:, 0] > 0, np.inf, np.where(r[:, 0] < 0, -np.inf, np.nan))
    want = sorted(range(e), key=lambda i: (np.isnan(logit[i]), -np.nan_to_num(logit[i]), i))[:k]
    dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    zeros = lambda *s, dt=torch.uint8: torch.zeros(*s, dtype=dt, device="cuda")  # noqa: E731
    ids, out = zeros(t, k, dt=torch.int32), zeros(t, d, dt=torch.bfloat16)
    f.fp8_moe(dev(x).bfloat16(), dev(r).bfloat16(), zeros(e, 2 * h, d),
              zeros(e, 1, 1, dt=torch.float32), zeros(e, d, h), zeros(e, 1, 1, dt=torch.float32),
              t, e, k, d, h, f.E4M3, True, zeros(f.fp8_moe_workspace(t, e, k, d, h)), out, ids=ids)
    torch.cuda.synchronize()
    assert (ids.cpu().numpy() == want).all()
    assert torch.isnan(out).all()
