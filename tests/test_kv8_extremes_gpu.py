"""The 8-bit KV cache where magnitudes, scales or counts lie near the ends of their types."""

import numpy as np
import pytest
import torch

from test_kv8_gpu import B, DT, Dev, check  # noqa: F401  (B: the fixture)
from test_kv8_scales_gpu import KEYS, stored

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


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("power", [60, 80, 100])
@pytest.mark.parametrize("rows_", [3, 130])
def test_scores_of_zero_between_loud_queries_and_keys(B, dt, power, rows_):  # noqa: F811
    """Query and keys of 2^power in different channels: every score is 0, and a row gives the mean of what it sees."""
    rng = np.random.default_rng(power)
    n, D = 100, 64
    k, v = np.zeros((n, 1, D)), rng.normal(size=(n, 1, D))
    k[..., 1] = 2.0 ** power
    c, d = stored(B, rng, "int8", 32, k, v)
    q = torch.zeros(rows_, 1, D, dtype=DT[dt], device="cuda")
    q[..., 0] = 2.0 ** power
    lim = [1 + (7 * i) % n for i in range(rows_)]
    values = c.keys(0, range(4))[1][0]
    for keys in KEYS:
        out, lse = d.attend(q, [0, rows_], lim, rows_, 0.125, max_keys=keys)
        for r in range(rows_):
            seen = values[:lim[r]]
            # weights are equal and exact; n + 64 roundings of sums of |v| / n, and the output's
            tol = np.abs(seen).mean(0) * (n + 64) * 2.0 ** -23
            want = seen.mean(0)
            assert (np.abs(out[r, 0].double().cpu().numpy() - want) <= tol + (np.abs(want) + tol) * torch.finfo(DT[dt]).eps / 2).all()
            assert abs(float(lse[r, 0]) - np.log(lim[r])) <= 2.0 ** -20


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("top", [64.0, 96.0])
@pytest.mark.parametrize("rows_", [3, 130])
def test_zero_keys_beside_loud_ones_keep_their_weight(B, dt, top, rows_):  # noqa: F811
    """A block of zero keys, one of keys of 2^20 that the query is orthogonal to, one with scores of 8 or 12: the zero keys
    have weights of e^-8 or e^-12 beside them."""
    rng = np.random.default_rng(3)
    n, D = 64, 64
    k, v = np.zeros((n, 1, D)), rng.normal(size=(n, 1, D))
    k[16:32, :, 0] = 2.0 ** 20
    k[32:48, :, 1] = top
    k[48:, :, 1] = 1.0
    v[:16] *= 2000.0
    c, d = stored(B, rng, "int8", 32, k, v)
    q = torch.zeros(rows_, 1, D, dtype=DT[dt], device="cuda")
    q[..., 1] = 1.0
    lim = [48 + i % 17 for i in range(rows_)]
    for keys in KEYS:
        out, lse = d.attend(q, [0, rows_], lim, rows_, 0.125, max_keys=keys)
        check(c, q, out, lse, [0, rows_], lim, 0.125, dt)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("rows_", [3, 130])
@pytest.mark.parametrize("scale", [3e38, -3.4e38, 2e38])
def test_scales_near_the_end_of_fp32(B, dt, rows_, scale):  # noqa: F811
    rng = np.random.default_rng(5)
    n, D = 130, 64
    k, v = rng.normal(size=(2, n, 1, D))
    c, d = stored(B, rng, "int8", 32, k * 1e-8, v)
    q = torch.from_numpy(rng.normal(size=(rows_, 1, D)) * 1e-31).to(torch.float32).to(DT[dt]).cuda()
    lim = [1 + (7 * i) % n for i in range(rows_)]
    for keys in KEYS:
        out, lse = d.attend(q, [0, rows_], lim, rows_, scale, max_keys=keys)
        check(c, q, out, lse, [0, rows_], lim, float(np.float32(scale)), dt)


def test_append_from_the_end_of_a_long_array(B):  # noqa: F811
    """Rows whose numbers are near 2^31: one row expanded over the array, so that it takes no memory."""
    from _kv8_ref import Cache

    n, rng = 2 ** 31 - 1, np.random.default_rng(6)
    c = Cache("int8", 4, 1, 16, 32, [[2, 0], [3, 1]], rng)
    d = Dev(B, c)
    x = torch.from_numpy(rng.normal(size=(2, 1, 1, 32))).to(torch.float32).cuda()
    k, v = (y.expand(n, 1, 32) for y in x)
    # as many rows of a sequence as the array has are allowed for; there are 20 and 9
    d.append(k, v, [n - 29, n - 9, n], [3, 5], n)
    for s, (start, m) in enumerate(((3, 20), (5, 9))):
        c.append(s, start, *(y[0].expand(m, 1, 32).double().cpu().numpy() for y in x))
    d.same()
    assert int(d.status) == 0
