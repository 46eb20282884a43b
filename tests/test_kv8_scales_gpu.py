"""Attention over the 8-bit KV cache where queries, keys or values are zero, tiny, or blocks of very different scale.

Both kernels (few rows, many rows: chosen by max_keys) against the definition, within the bounds of Cache.attend, which are
made of what a row sees.
"""

import numpy as np
import pytest
import torch

from _kv8_ref import Cache
from test_kv8_gpu import B, DT, Dev, check, table  # noqa: F401  (B: the fixture)

pytestmark = pytest.mark.gpu

KEYS = (0, 1 << 20)  # expected keys: few-row tiles, many-row tiles (from 64 queries on)


def stored(B, rng, fmt, PT, k, v):  # noqa: F811
    """A cache that holds one sequence's fp32 rows k, v [n, H, D]."""
    n, H, D = k.shape
    tab, n_pages = table(rng, 1, -(-n // PT))
    c = Cache(fmt, n_pages, H, PT, D, tab, rng)
    d = Dev(B, c)
    d.append(*(torch.from_numpy(x).to(torch.float32).cuda() for x in (k, v)), [0, n], [0], n)
    for name, t in d.t.items():
        setattr(c, name, t.cpu().numpy())
    return c, d


@pytest.mark.parametrize("dt,D,PT", [("f32", 64, 64), ("bf16", 64, 16), ("f16", 128, 64), ("bf16", 96, 32), ("f32", 32, 64), ("f32", 128, 16)])
@pytest.mark.parametrize("quiet", ["zero", "start", "tiny"])
@pytest.mark.parametrize("mask", ["causal", "ragged"])
def test_zero_and_tiny_queries_and_keys(B, dt, D, PT, quiet, mask):  # noqa: F811
    """Padding in front of a prompt and zeroed buffers: scores of 0 give the mean of the values, hidden keys nothing."""
    rng = np.random.default_rng(D + PT)
    n, R = 200, 130
    k, v = rng.normal(size=(2, n, 2, D))
    if quiet == "zero":
        k[:] = 0.0
    elif quiet == "start":
        k[:70] = 0.0
        v[:30] = 0.0
        k[70:130] *= 1e-9
    else:
        k *= 1e-30
    c, d = stored(B, rng, "int8" if D != 96 else "e4m3", PT, k, v)
    q = rng.normal(size=(R + 1, 2, D)) * np.array([0.0, 1e-9, 1.0, 1e-30, 0.0])[np.arange(R + 1) % 5][:, None, None]
    q = torch.from_numpy(q).to(torch.float32).to(DT[dt]).cuda()
    lim = list(range(n - R + 1, n + 1)) if mask == "causal" else [int(x) for x in rng.integers(0, n + 1, R)]
    if mask == "ragged":
        lim[:7] = [0, 0, 1, 33, 63, 64, 65]
    lim.append(9)
    for keys in KEYS:
        out, lse = d.attend(q, [0, R], lim, R, D ** -0.5, max_keys=keys)
        assert bool(torch.isfinite(out).all()) and not bool(torch.isnan(lse).any())
        check(c, q, out, lse, [0, R], lim, D ** -0.5, dt)
    assert int(d.status) == 0


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("D,power", [(64, 18), (64, 26), (128, 30), (32, 26), (96, 60)])
@pytest.mark.parametrize("rows_", [3, 130])
def test_a_loud_key_without_weight_changes_no_other(B, dt, fmt, D, power, rows_):  # noqa: F811
    """A block of keys far louder than its neighbours whose scores are far below theirs: the result is the others'."""
    rng = np.random.default_rng(D + power)
    n = 100
    k, v = rng.normal(size=(2, n, 1, D))
    k[..., 0] = 0.0
    k[32:48] = 0.0
    k[32:48, :, 0] = -2.0 ** power
    c, d = stored(B, rng, fmt, 16, k, v)
    qn = rng.normal(size=(rows_, 1, D))
    qn[..., 0] = 1.0 + np.abs(qn[..., 0])
    q = torch.from_numpy(qn).to(DT[dt]).cuda()
    lim = [int(x) for x in rng.integers(49, n + 1, rows_)]
    others = [[[0, 1, 3, 4, 5, 6]]] * rows_
    for keys in KEYS:
        out, lse = d.attend(q, [0, rows_], lim, rows_, 0.125, max_keys=keys)
        assert bool(torch.isfinite(out).all()) and not bool(torch.isnan(lse).any())
        check(c, q, out, lse, [0, rows_], lim, 0.125, dt, others)
    assert int(d.status) == 0


def unseen(B, dt, fmt, D, step, loud, rows_, keys):  # noqa: F811
    """Each block of 16 positions is 2^step louder than the one before: a row's result is as exact as what it sees."""
    rng = np.random.default_rng(D + step)
    nb = min(6, 110 // step + 1)
    n = 16 * nb
    k, v = rng.normal(size=(2, n, 1, D))
    x = k if loud == "k" else v
    x *= 2.0 ** (step * (np.arange(n) // 16))[:, None, None]
    c, d = stored(B, rng, fmt, 32, k, v)
    q = torch.from_numpy(rng.normal(size=(rows_, 1, D))).to(DT[dt]).cuda()
    lim = [int(x) for x in rng.integers(1, n + 1, rows_)]
    lim[:6] = [16, n, 5, 17, 32, 0]
    out, lse = d.attend(q, [0, rows_], lim, rows_, 0.125, max_keys=keys)
    assert bool(torch.isfinite(out).all()) and not bool(torch.isnan(lse).any())
    check(c, q, out, lse, [0, rows_], lim, 0.125, dt)
    assert int(d.status) == 0


SCALES = pytest.mark.parametrize("dt,fmt,D,step", [(dt, fmt, D, step) for dt in ("f32", "bf16") for fmt in ("int8", "e4m3")
                                                   for D, step in ((64, 17), (64, 26), (64, 34), (128, 26), (32, 34), (96, 17))])


@SCALES
@pytest.mark.parametrize("rows_", [6, 12])
def test_values_that_a_row_does_not_see_few_rows(B, dt, fmt, D, step, rows_):  # noqa: F811
    unseen(B, dt, fmt, D, step, "v", rows_, 0)


@SCALES
def test_values_that_a_row_does_not_see_many_rows(B, dt, fmt, D, step):  # noqa: F811
    unseen(B, dt, fmt, D, step, "v", 130, 1 << 20)
