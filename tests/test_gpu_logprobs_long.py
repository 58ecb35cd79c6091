"""Log probabilities of rows above 48 KB, whose CTA goes through several spans of them: signs where one token has all of the
probability, rows that are hard on the picking of the best keys in spans after the first, many rows (a CTA each) and few (several each).
Values against the formulas in 64 bits, as in test_gpu_logprobs.py."""
import numpy as np
import pytest
import torch

import kv8_ref as K
from test_gpu_logprobs import check, ids_for

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    import quantized_routed_expert_grouped_gb300 as mod
    mod.lib()
    return mod


@pytest.mark.parametrize("dtype", list(K.TYPES))
@pytest.mark.parametrize("V", [300, 20001, 70001])
@pytest.mark.parametrize("R_", [40, 320])
def test_signs(m, R_, V, dtype):
    """Where one token has nearly all of the probability, its log is at most 0, and the entropy at least 0."""
    rng = np.random.default_rng(V)
    at = rng.integers(0, V, R_)
    best = 7.3 + 0.37 * np.arange(R_) % 9 - 4
    x = best[:, None] - 30 - 10 * rng.random((R_, V))
    x[np.arange(R_), at] = best
    x[::3] = np.where(x[::3] < best[::3, None] - 1, -60000.0, x[::3])
    x[1::6] = np.where(x[1::6] < best[1::6, None] - 1, -np.inf, x[1::6])
    dev = torch.from_numpy(x).to(K.TYPES[dtype]).cuda()
    ids = torch.from_numpy(at.astype(np.int32)).cuda().view(-1, 1)
    for scale in (1.0, 1 / 0.7, 3.0, 1000.0):
        lp, tl, ti, ent, _ = m.token_logprobs(dev, ids, top=3, scale=scale)
        assert torch.equal(ti[:, :1], ids)
        assert bool((lp <= 0).all() and (tl <= 0).all() and (ent >= 0).all()), (float(lp.max()), float(tl.max()), float(ent.min()))
        check(m, dev[:12], at[:12, None], 3, scale)
