"""The 8-bit KV cache's calls beside others of the same thread: what an earlier call left changes nothing."""

import pytest
import torch

from test_kv8_gpu import B, i32  # noqa: F401  (B: the fixture)

pytestmark = pytest.mark.gpu


def test_an_earlier_call_that_failed_is_not_reported(B):  # noqa: F811
    """A decoder handle that does not fit into memory fails; the cache's calls behind it queue their work and say so."""
    from block_diffusion_byte_b200.driver import Engine
    from workload import CONFIGS, WeightSet

    shape = CONFIGS["tiny_d4"].shape
    ws = WeightSet(shape, gain_std=0.1).materialize()
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
    i8 = lambda *s: torch.zeros(*s, dtype=torch.int8, device="cuda")  # noqa: E731
    cache = B.kv8_cache("int8", u8(2, 1, 16, 64), u8(2, 1, 16, 64), u8(2, 1, 1), u8(2, 1, 1), i32([0, 1]).view(1, 2), i8(2, 1, 64),
                        i8(2, 1, 64), u8(2, 1))
    x = torch.ones(20, 1, 64, device="cuda")
    back = [torch.zeros_like(x) for _ in range(2)]
    out = torch.zeros_like(x)
    off, start, lim = i32([0, 20]), i32([0]), i32([20] * 20)
    sp, sc = i32([7] * 20).view(20, 1, 1), i32([7] * 20).view(20, 1)
    calls = [(B.blt_kv8_append, B.kv8_rows(x, x, off, start, 20)), (B.blt_kv8_read, B.kv8_rows(*back, off, start, 20)),
             (B.blt_kv8_attend, B.kv8_attention(x, out, off, lim, 20, 20, 0.125)),
             (B.blt_kv8_select, B.kv8_selection(x, off, lim, 20, 20, sp, sc))]
    for call, args in calls:
        with pytest.raises(B.BltError, match="blt_dec_init"):
            Engine(shape, ws, max_batch=4, max_ctx=128, max_block=8, max_rows=64, max_latents=1 << 30)
        call(cache, args, torch.cuda.current_stream().cuda_stream)
    assert torch.equal(back[0], x) and torch.equal(back[1], x) and torch.equal(out, x)
    assert sp.view(-1).tolist() == [0] * 20  # equal scores: the lower page
