"""The engine with an 8-bit KV cache against the fp64 oracle whose K/V pass through the same 8 bits.

Tolerance: the workload definition's logits max-abs 2e-2.  A key or value that lies next to the border of two
codes may be stored as either (the engine computes it in fp32): one element off by one step, far inside it.
"""

from dataclasses import replace

import numpy as np
import pytest
import torch

from _kv8_ref import decode, quantise
from oracle.model import BLOCK, CAUSAL, OracleModel, Row, SeqState, decoder_pass
from oracle.policies import OracleSequence
from workload import CONFIGS, Patcher, WeightSet, prefix_bytes

pytestmark = pytest.mark.gpu

LOGIT_TOL = 2e-2


class Kept:
    """K or V by position, held in blocks of 16 positions as the 8-bit cache holds them."""

    def __init__(self, a, fmt):
        self.a, self.fmt = a, fmt
        self.shape = a.shape

    def __getitem__(self, i):
        return self.a[i]

    def __setitem__(self, i, x):
        l, pos = i
        start, end = int(pos[0]), int(pos[-1]) + 1
        assert np.array_equal(pos, np.arange(start, end))
        a = self.a[l]
        a[start:end] = x
        for b in range(start // 16 * 16, end, 16):
            e = min(b + 16, end)
            for h in range(a.shape[1]):
                blk = np.zeros((16, a.shape[2]))
                blk[:e - b] = a[b:e, h]
                q, ex = quantise(blk, self.fmt)
                a[b:e, h] = decode(q[None], np.array([[ex]], np.uint8), self.fmt)[0, :e - b]


class State8(SeqState):
    def __init__(self, shape, capacity, fmt):
        super().__init__(shape, capacity)
        self.K, self.V = Kept(self.K, fmt), Kept(self.V, fmt)

    def ensure(self, n):
        assert n <= self.K.shape[1]


def _setup(weight_dtype, d_model, prefix):
    from block_diffusion_byte_b200 import _build

    _build.build()
    wl = CONFIGS["tiny_d4"]
    wl = replace(wl, shape=replace(wl.shape, weight_dtype=weight_dtype, d_model=d_model), prefix_len=prefix)
    ws = WeightSet(wl.shape, gain_std=0.1).materialize()
    return wl, ws, OracleModel(wl.shape, ws)


@pytest.mark.parametrize("fmt,weight_dtype,d_model,prefix", [("int8", "f32", 128, 64), ("e4m3", "f32", 256, 75), ("int8", "bf16", 256, 300),
                                                             ("e4m3", "bf16", 512, 141)])
def test_prefill_block_and_verification_logits(fmt, weight_dtype, d_model, prefix):
    """A prompt (chunked; through the tcgen05 projections where it has rows enough), a masked block, then a drafted
    run and its verification, whose rows share their 16 positions with committed ones."""
    from block_diffusion_byte_b200 import binding as B
    from block_diffusion_byte_b200.driver import Engine, SeqHost

    wl, ws, om = _setup(weight_dtype, d_model, prefix)
    pre = [int(b) for b in prefix_bytes(wl.seed, wl.cfg_index, 0, wl.prefix_len)]
    N, k = len(pre), 4
    eng = Engine(wl.shape, ws, max_batch=2, max_ctx=N + 64, max_block=16, max_rows=160, kv8=fmt, persistent=True)
    try:
        s = SeqHost(Patcher(wl.patch_kind, wl.seed, wl.cfg_index, 0), wl.seed, wl.cfg_index, 0, wl.shape.d_global)
        s.commit(pre)
        b, sl, lat = s.take_pending()
        r, keep = eng.rows([b[:-1]], [sl[:-1]], [lat])
        got = torch.zeros((N - 1, 256), dtype=torch.float32, device="cuda")
        torch.cuda.synchronize()
        B.blt_dec_prefill(eng.h, 1, r, got)
        r, keep = eng.rows([b[-1:]], [sl[-1:]], [[]])
        blk = torch.zeros((1, 1, k, 256), dtype=torch.float32, device="cuda")
        torch.cuda.synchronize()
        B.blt_dec_diffuse_block(eng.h, 1, r, k, 0.0, 1, eng.d_out, eng.d_steps, blk)
        ver = torch.zeros((1, k, 256), dtype=torch.float32, device="cuda")
        y = int(pre[0])
        r, keep = eng.rows([[y]], [sl[-1:]], [[]])
        torch.cuda.synchronize()
        B.blt_dec_draft(eng.h, 1, r, B.BLT_DRAFT_AR, k, 0.0, 0, eng.d_out, None)
        assert B.blt_dec_sync(eng.h) == 0
        draft = eng._get(eng.out_view(1, k))[0].tolist()
        B.blt_dec_verify_accept(eng.h, eng._put(eng.d_vslots.view(-1), np.full(k, sl[-1], np.int32)), None, None, eng.d_acc, eng.d_next, ver)
        assert B.blt_dec_sync(eng.h) == 0
        st = B.blt_dec_stats(eng.h)
        assert st["persistent_calls"] == 0
        if weight_dtype == "bf16":
            assert st["tc_gemms"] > 0
        got, blk, ver = got.cpu().numpy(), blk.cpu().numpy()[0, 0], ver.cpu().numpy()[0]
    finally:
        eng.close()
    o = OracleSequence(om, wl, 0, pre)
    st8 = State8(wl.shape, N + 64, fmt)
    st8.latents = o.st.latents
    chunk = 160
    want = np.concatenate([decoder_pass(om, st8, [Row(pre[p], p, o.lat[p], CAUSAL) for p in range(a, min(a + chunk, N - 1))])
                           for a in range(0, N - 1, chunk)])
    assert np.abs(got - want).max() < LOGIT_TOL
    mask = wl.shape.vocab - 1
    last = len(st8.latents) - 1
    rows = [Row(pre[-1], N - 1, o.lat[N - 1], CAUSAL)] + [Row(mask, N + i, last, BLOCK, N + k) for i in range(k)]
    want = decoder_pass(om, st8, rows)[1:]
    assert np.abs(blk - want).max() < LOGIT_TOL
    # the draft's passes: the pending byte, then draft bytes one by one; then the verification of all of them
    decoder_pass(om, st8, [Row(y, N, sl[-1], CAUSAL)])
    for i in range(k - 1):
        decoder_pass(om, st8, [Row(draft[i], N + 1 + i, last, CAUSAL)])
    want = decoder_pass(om, st8, [Row(draft[i], N + 1 + i, sl[-1], CAUSAL) for i in range(k)])
    assert np.abs(ver - want).max() < LOGIT_TOL


@pytest.mark.parametrize("mode,kind", [("D", "int8"), ("DV", "e4m3"), ("S", "int8"), ("D", "e4m3")])
def test_generation_runs_and_repeats(mode, kind):
    """Whole generations of two sequences: the same bytes on a second handle."""
    from block_diffusion_byte_b200.driver import Engine, generate

    wl, ws, _ = _setup("f32", 128, 64)
    wl = replace(wl, mode=mode, block=8 if mode != "D" else 4, alpha=0.0 if mode == "DV" else wl.alpha)
    pres = [[int(b) for b in prefix_bytes(wl.seed, wl.cfg_index, i, wl.prefix_len)] for i in range(2)]
    outs = []
    for kv8 in (kind, kind):
        eng = Engine(wl.shape, ws, max_batch=2, max_ctx=wl.prefix_len + 64, max_block=16, max_rows=256, kv8=kv8)
        try:
            res = generate(eng, wl, pres, 24)
            assert [len(o) for o in res.out] == [24, 24]
            outs.append(res.out)
        finally:
            eng.close()
    assert outs[0] == outs[1]


def test_the_8_bit_cache_takes_half_the_bytes_and_its_limits_are_refused():
    from block_diffusion_byte_b200 import binding as B
    from block_diffusion_byte_b200.driver import Engine, SeqHost

    wl, ws, _ = _setup("bf16", 256, 64)
    pre = [int(b) for b in prefix_bytes(wl.seed, wl.cfg_index, 0, 64)]
    read = []
    for kv8 in (None, "int8"):
        eng = Engine(wl.shape, ws, max_batch=1, max_ctx=128, max_block=16, max_rows=256, kv8=kv8)
        try:
            s = SeqHost(Patcher(wl.patch_kind, wl.seed, wl.cfg_index, 0), wl.seed, wl.cfg_index, 0, wl.shape.d_global)
            s.commit(pre)
            b, sl, lat = s.take_pending()
            r, keep = eng.rows([b], [sl], [lat])
            if kv8:
                with pytest.raises(B.BltError):
                    B.blt_dec_prefill_noalloc(eng.h, 1, r, None)
            B.blt_dec_prefill(eng.h, 1, r, None)
            assert B.blt_dec_sync(eng.h) == 0
            read.append(B.blt_dec_stats(eng.h)["prefill_kv_read_bytes"])
        finally:
            eng.close()
    L, H, d = wl.shape.n_layers, wl.shape.n_heads, wl.shape.d_model
    assert read == [64 * L * 2 * d * 2, 64 * (L * 2 * d + L * 2 * H // 16)]
    for kw in (dict(extra_flags=B.BLT_FLAG_KV8_INT8 | B.BLT_FLAG_KV8_E4M3), dict(kv8="int8", page_tokens=512)):
        with pytest.raises(B.BltError):
            Engine(wl.shape, ws, max_batch=1, max_ctx=1024, max_block=16, **kw)
    narrow = replace(wl.shape, n_heads=16)  # head dim 16
    with pytest.raises(B.BltError):
        Engine(narrow, WeightSet(narrow).materialize(), max_batch=1, max_ctx=128, max_block=16, kv8="int8")
