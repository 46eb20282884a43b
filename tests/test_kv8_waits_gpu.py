"""Attention of many rows over the 8-bit KV cache when a wait inside the kernel runs out (BLT_KV8_TEST_STALL: one CTA's keys
never come): the rows concerned keep what they held, the status word says so, and the rest of the call is done."""

import numpy as np
import pytest
import torch

from test_kv8_gpu import B, DT, filled, i32  # noqa: F401  (B: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dt,D", [("bf16", 64), ("f32", 64), ("f16", 128)])
@pytest.mark.parametrize("keys", [1024, 1 << 14])  # one CTA a tile; the keys of a tile split over a cluster
@pytest.mark.parametrize("status", [True, False])
def test_a_wait_that_runs_out_leaves_its_rows(B, dt, D, keys, status):  # noqa: F811
    rng = np.random.default_rng(41)
    R, G = 300, 2
    c, d = filled(B, rng, "int8", 2, 64, D, [1500, 1500])
    desc = B.kv8_cache("int8", d.t["k"], d.t["v"], d.t["k_exp"], d.t["v_exp"], d.table, status=d.status if status else None)
    q = torch.from_numpy(rng.normal(size=(2 * R, 2 * G, D))).to(DT[dt]).cuda()
    off, lim = i32([0, R, 2 * R]), i32([1500 - i for i in range(R)] * 2)
    want, wl = d.attend(q, [0, R, 2 * R], lim.tolist(), R, 0.125, max_keys=keys)
    out = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    a = B.kv8_attention(q, out, off, lim, R, keys, 0.125, lse)
    a.flags = B.BLT_KV8_TEST_STALL
    B.blt_kv8_attend(desc, a, torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert int(d.status) == (B.BLT_ERR_DEVICE if status else 0)
    first = (R * G - 1) // 128 * 128  # of the last tile's (row, head of the group) pairs
    held = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    for n in range(first, R * G):
        held[n // G, n % G] = True
    assert bool((out[held] == 7.0).all()) and bool((lse[held] == 7.0).all())
    assert torch.equal(out[~held], want[~held]) and torch.equal(lse[~held], wl[~held])
    d.status.zero_()
    a.flags = 0
    B.blt_kv8_attend(desc, a, torch.cuda.current_stream().cuda_stream)
    assert torch.equal(out, want) and torch.equal(lse, wl) and int(d.status) == 0
