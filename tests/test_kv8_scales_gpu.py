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


@SCALES
@pytest.mark.parametrize("rows_,keys", [(12, 0), (130, 1 << 20)])
def test_keys_that_a_row_does_not_see(B, dt, fmt, D, step, rows_, keys):  # noqa: F811
    unseen(B, dt, fmt, D, step, "k", rows_, keys)


@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("D,power", [(64, 17), (64, 20), (96, 23), (64, 26), (64, 40), (128, 60), (32, 90), (96, 29)])
@pytest.mark.parametrize("rows_", [3, 130])
def test_scores_beyond_whole_numbers_of_fp32(B, dt, D, power, rows_):  # noqa: F811
    """Scores around 2^power: where the largest leads by more than fp32's rounding of it, the row takes that key's value."""
    rng = np.random.default_rng(D + power)
    n = 180
    k, v = rng.normal(size=(2, n, 1, D))
    v[::3] *= 64.0
    c, d = stored(B, rng, "int8", 32, k * 2.0 ** power, v)
    q = torch.from_numpy(rng.normal(size=(rows_, 1, D))).to(DT[dt]).cuda()
    lim = [int(x) for x in rng.integers(1, n + 1, rows_)]
    keys_, values = (x[0] for x in c.keys(0, range(6)))
    for keys in KEYS:
        out, lse = d.attend(q, [0, rows_], lim, rows_, 0.125, max_keys=keys)
        for r in range(rows_):
            qr = q[r, 0].double().cpu().numpy()
            z = 0.125 * keys_[:lim[r]] @ qr
            # a score's rounding: D + 4 steps of 2^-23 of the sum of magnitudes, and 2^-22 of q
            err = 0.125 * (np.abs(keys_[:lim[r]]) @ np.abs(qr)).max() * ((D + 4) * 2.0 ** -23 + 2.0 ** -22)
            first, second = np.sort(z)[::-1][:2] if lim[r] > 1 else (z[0], -np.inf)
            assert abs(float(lse[r, 0]) - first) <= err + 2.0 ** -22 * abs(first) + np.log(n)
            want = values[int(z.argmax())]
            got = out[r, 0].double().cpu().numpy()
            assert np.isfinite(got).all() and (np.abs(got) <= np.abs(values).max() * (1 + 2.0 ** -7)).all()
            if first - second > 2 * err + 200:
                assert (np.abs(got - want) <= np.abs(want) * torch.finfo(DT[dt]).eps / 2 + 2.0 ** -25).all()


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("power", [0, 22, 27, 60])
@pytest.mark.parametrize("rows_", [3, 130])
def test_equal_scores_of_any_size_give_the_mean(B, dt, power, rows_):  # noqa: F811
    """The same key everywhere, values whose blocks differ in scale: the mean of what a row sees, whatever the score."""
    rng = np.random.default_rng(power)
    n, D = 100, 64
    k, v = np.ones((n, 1, D)) * 2.0 ** power, rng.normal(size=(n, 1, D)) * 2.0 ** (np.arange(n) // 16)[:, None, None]
    c, d = stored(B, rng, "int8", 32, k, v)
    q = torch.full((rows_, 1, D), 1.25, dtype=DT[dt], device="cuda")
    lim = [1 + (7 * i) % n for i in range(rows_)]
    values = c.keys(0, range(4))[1][0]
    for keys in KEYS:
        out, _ = d.attend(q, [0, rows_], lim, rows_, 0.125, max_keys=keys)
        for r in range(rows_):
            seen = values[:lim[r]]
            # weights are equal and exact; n + 64 roundings of sums of |v| / n, and the output's
            tol = np.abs(seen).mean(0) * (n + 64) * 2.0 ** -23
            want = seen.mean(0)
            assert (np.abs(out[r, 0].double().cpu().numpy() - want) <= tol + (np.abs(want) + tol) * torch.finfo(DT[dt]).eps / 2).all()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("top", [float(np.finfo(np.float32).max), 3.39e38, 1e38, 1e-38])
def test_kept_rows_near_the_ends_of_fp32(B, fmt, top):  # noqa: F811
    """Rows stored one by one behind rows of magnitudes whose codes' values lie beyond fp32: the kept codes stay."""
    c = Cache(fmt, 1, 1, 16, 32, [[0]], np.random.default_rng(0))
    d = Dev(B, c)
    x = torch.tensor([top, -top, top / 2, 1.0], device="cuda")[:, None, None].expand(4, 1, 32).contiguous()
    loudest = 0
    for i in range(4):
        d.append(x[i:i + 1], x[i:i + 1], [0, 1], [i], 1)
        e = int(d.t["k_exp"])
        assert int(d.t["v_exp"]) == e and torch.equal(d.t["k"][0, 0, :i + 1], d.t["v"][0, 0, :i + 1])
        loudest = max(loudest, e)
        assert e == loudest  # the least exponent whose range holds every row: it does not fall
        setattr(c, "k", d.t["k"].cpu().numpy())
        setattr(c, "k_exp", d.t["k_exp"].cpu().numpy())
        got = c.keys(0, [0])[0][0, :i + 1, 0]
        want = x[:i + 1, 0, 0].double().cpu().numpy()
        # off by at most one step of the largest exponent: 1 code, or 2^-3 of an e4m3 value (its subnormals: 2^-9)
        step = 2.0 ** (loudest - 127) * (np.ones(i + 1) if fmt == "int8" else np.maximum(np.abs(want) / 2.0 ** (loudest - 127) * 2.0 ** -3, 2.0 ** -9))
        assert (np.abs(got - want) <= step).all(), (i, got, want)
