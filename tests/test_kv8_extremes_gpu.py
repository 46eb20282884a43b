"""The 8-bit KV cache where magnitudes, scales or counts lie near the ends of their types."""

import numpy as np
import pytest
import torch

from test_kv8_gpu import B, DT, Dev, check  # noqa: F401  (B: the fixture)
from test_kv8_scales_gpu import stored

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("qpow,kpow", [(120, -60), (-60, 120), (100, -90), (-90, 100), (0, 0)])
def test_select_with_loud_queries_and_quiet_keys(B, D, qpow, kpow):  # noqa: F811
    """Scores inside fp32's range whose factors are not near 1: the order is the scores'."""
    rng = np.random.default_rng(abs(D + qpow))
    n, PT, R = 900, 32, 5
    k, v = rng.normal(size=(2, n, 2, D))
    c, d = stored(B, rng, "int8", PT, k * 2.0 ** kpow, v)
    q = torch.from_numpy(rng.normal(size=(R, 4, D)) * 2.0 ** qpow).to(torch.float32).cuda()
    lim = [n, n - 1, 600, 333, 40]
    sp, sc = d.select(q, [0, R], lim, R, 6, 1, 1)
    for r in range(R):
        want = c.select(0, q[r].double().cpu().numpy(), lim[r], 6, 1, 1)
        for h in range(2):
            assert sp[r, h, :int(sc[r, h])].tolist() == want[h], (r, h)
