"""The 8-bit KV cache's C ABI without a GPU: struct layouts, refusals, and the reference the GPU tests use."""

import ctypes as C
import os
import subprocess

import numpy as np
import pytest

from _kv8_ref import E4M3, Cache, decode, exponent, quantise

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def B():
    from block_diffusion_byte_b200 import _build, binding

    _build.build()
    binding.load_library()
    return binding


def test_struct_layouts_match_header(B, tmp_path):
    structs = {n: getattr(B, n) for n in ("blt_kv8_cache", "blt_kv8_rows", "blt_kv8_attention", "blt_kv8_selection")}
    lines = ["#include <stddef.h>", "#include <stdio.h>", '#include "bltkv8.h"', "int main(void) {"]
    for name, cls in structs.items():
        lines.append(f'  printf("{name} %zu\\n", sizeof({name}));')
        lines += [f'  printf("{name}.{f} %zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    src = tmp_path / "layout.c"
    src.write_text("\n".join(lines + ["  return 0; }"]))
    exe = tmp_path / "layout"
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), "-o", str(exe), str(src)], check=True)
    got = dict(line.split() for line in subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.splitlines())
    for name, cls in structs.items():
        assert int(got[name]) == C.sizeof(cls), name
        for f, _ in cls._fields_:
            assert int(got[f"{name}.{f}"]) == getattr(cls, f).offset, (name, f)


def _cache(B, **kw):
    base = dict(format=0, n_heads=2, head_dim=64, page_tokens=64, n_pages=8, batch=2, max_pages=4, k=4096, v=8192, k_exp=64, v_exp=128,
                page_table=256, k_min=512, k_max=1024, k_sexp=2048)
    return B.blt_kv8_cache(**{**base, **kw})


def _rows(B, **kw):
    base = dict(k=4096, v=8192, dtype=0, n_rows=4, max_rows=2, row_stride=128, head_stride=64, row_offsets=64, start=128)
    return B.blt_kv8_rows(**{**base, **kw})


def _attn(B, **kw):
    base = dict(q=4096, out=8192, dtype=1, n_q_heads=4, n_rows=4, max_rows=2, max_keys=64, scale=0.125, q_row_stride=256, q_head_stride=64,
                out_row_stride=256, out_head_stride=64, row_offsets=64, row_limit=128)
    return B.blt_kv8_attention(**{**base, **kw})


def _sel(B, **kw):
    base = dict(q=4096, dtype=1, n_q_heads=4, n_rows=4, max_rows=2, max_keys=64, n_select=4, n_sink=1, n_local=1, q_row_stride=256,
                q_head_stride=64, row_offsets=64, row_limit=128, sel_pages=256, sel_count=512)
    return B.blt_kv8_selection(**{**base, **kw})


BAD_CACHE = [dict(format=2), dict(format=-1), dict(n_heads=0), dict(head_dim=48), dict(head_dim=256), dict(page_tokens=8),
             dict(page_tokens=24), dict(page_tokens=272), dict(n_pages=0), dict(batch=0), dict(batch=65536), dict(max_pages=0),
             dict(max_pages=1 << 24), dict(k=None), dict(v=None), dict(k_exp=None), dict(v_exp=None), dict(page_table=None),
             dict(k=4097), dict(v=8200), dict(page_stride=100), dict(page_stride=8200), dict(exp_stride=1), dict(sum_stride=8),
             dict(sum_stride=130), dict(sexp_stride=1), dict(k_min=None), dict(k_sexp=None), dict(page_table=258), dict(status=3),
             dict(k_max=1025)]


@pytest.mark.parametrize("kw", BAD_CACHE, ids=lambda kw: ",".join(f"{k}={v}" for k, v in kw.items()))
def test_bad_caches_are_refused(B, kw):
    lib = B.load_library()
    for fn, arg in (("blt_kv8_append", _rows(B)), ("blt_kv8_read", _rows(B)), ("blt_kv8_attend", _attn(B)), ("blt_kv8_select", _sel(B))):
        assert getattr(lib, fn)(_cache(B, **kw), arg, None) == B.BLT_ERR_INVALID_ARG, fn
        assert lib.blt_kv8_last_error() != b""


@pytest.mark.parametrize("kw", [dict(dtype=3), dict(n_rows=-1), dict(max_rows=-1), dict(k=None), dict(v=None), dict(row_offsets=None),
                                dict(start=None), dict(k=4097), dict(v=8194), dict(row_stride=-1), dict(head_stride=-64), dict(start=130)],
                         ids=lambda kw: ",".join(f"{k}={v}" for k, v in kw.items()))
def test_bad_rows_are_refused(B, kw):
    lib = B.load_library()
    for fn in ("blt_kv8_append", "blt_kv8_read"):
        assert getattr(lib, fn)(_cache(B), _rows(B, **kw), None) == B.BLT_ERR_INVALID_ARG, fn


@pytest.mark.parametrize("kw", [dict(dtype=-1), dict(n_q_heads=0), dict(n_q_heads=3), dict(n_rows=-1), dict(max_rows=-2), dict(max_keys=-1),
                                dict(scale=float("nan")), dict(scale=float("inf")), dict(q=None), dict(out=None), dict(row_offsets=None),
                                dict(row_limit=None), dict(q=4097), dict(out=8193), dict(lse=6), dict(q_row_stride=-1), dict(out_head_stride=-1),
                                dict(sel_pages=256), dict(sel_count=256), dict(sel_pages=256, sel_count=512, n_select=0),
                                dict(n_rows=1 << 25, max_rows=1 << 25)],
                         ids=lambda kw: ",".join(f"{k}={v}" for k, v in kw.items()))
def test_bad_attentions_are_refused(B, kw):
    assert B.load_library().blt_kv8_attend(_cache(B), _attn(B, **kw), None) == B.BLT_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [dict(dtype=9), dict(n_q_heads=5), dict(n_q_heads=256), dict(n_rows=-1), dict(n_select=0), dict(n_sink=-1),
                                dict(n_local=-1), dict(n_sink=3, n_local=2), dict(q=None), dict(sel_pages=None), dict(sel_count=None),
                                dict(row_limit=None), dict(q=4097), dict(sel_pages=258), dict(q_head_stride=-1)],
                         ids=lambda kw: ",".join(f"{k}={v}" for k, v in kw.items()))
def test_bad_selections_are_refused(B, kw):
    assert B.load_library().blt_kv8_select(_cache(B), _sel(B, **kw), None) == B.BLT_ERR_INVALID_ARG


def test_selection_needs_summaries_and_few_enough_pages(B):
    lib = B.load_library()
    assert lib.blt_kv8_select(_cache(B, k_min=None, k_max=None, k_sexp=None), _sel(B), None) == B.BLT_ERR_INVALID_ARG
    assert b"summaries" in lib.blt_kv8_last_error()
    assert lib.blt_kv8_select(_cache(B, max_pages=49153, page_tokens=16), _sel(B), None) == B.BLT_ERR_INVALID_ARG


def test_null_descriptors_are_refused_and_no_rows_is_no_work(B):
    lib = B.load_library()
    for fn, make in (("blt_kv8_append", _rows), ("blt_kv8_read", _rows), ("blt_kv8_attend", _attn), ("blt_kv8_select", _sel)):
        f = getattr(lib, fn)
        assert f(None, make(B), None) == B.BLT_ERR_INVALID_ARG
        assert f(_cache(B), None, None) == B.BLT_ERR_INVALID_ARG
        for kw in (dict(n_rows=0), dict(max_rows=0)):
            assert f(_cache(B), make(B, **kw), None) == B.BLT_OK, (fn, kw)
        assert lib.blt_kv8_last_error() == b""


def test_binding_refuses_wrong_tensors(B):
    import torch

    z = lambda *s, dt=torch.uint8: torch.zeros(*s, dtype=dt)  # noqa: E731
    with pytest.raises(ValueError, match="CUDA"):
        B.kv8_cache("int8", z(4, 2, 64, 64), z(4, 2, 64, 64), z(4, 2, 4), z(4, 2, 4), z(1, 4, dt=torch.int32))
    with pytest.raises(ValueError, match="format"):
        B.kv8_cache("int4", z(4, 2, 64, 64), z(4, 2, 64, 64), z(4, 2, 4), z(4, 2, 4), z(1, 4, dt=torch.int32))
    with pytest.raises(ValueError, match="k:"):
        B.kv8_cache("int8", z(4, 2, 64, 64, dt=torch.int8), z(4, 2, 64, 64), z(4, 2, 4), z(4, 2, 4), z(1, 4, dt=torch.int32))
    with pytest.raises(ValueError):
        B.kv8_rows(z(4, 2, 64, dt=torch.float64), z(4, 2, 64, dt=torch.float64), z(2, dt=torch.int32), z(1, dt=torch.int32), 4)


# ------------------------------------------------------------------ the reference against torch and brute force
def test_reference_e4m3_matches_torch():
    import torch

    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    ok = ~np.isnan(want)
    assert ok.sum() == 254 and np.array_equal(E4M3[ok], want[ok])
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.normal(size=3000) * 10.0 ** rng.integers(-4, 3, 3000), E4M3[:127], (E4M3[:126] + E4M3[1:127]) / 2])
    x = np.clip(x, -448, 448)[: 16 * 203].reshape(-1, 16, 1)
    for blk in x:
        blk[0] = 448.0  # exponent 127
        q, e = quantise(blk, "e4m3")
        assert e == 127
        t = torch.from_numpy(blk).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
        same = torch.from_numpy(blk).float().double().numpy() == blk
        assert np.array_equal(q[same], t[same])


def test_reference_exponent_is_least():
    rng = np.random.default_rng(1)
    for top in (127.0, 448.0):
        for a in list(2.0 ** rng.uniform(-100, 127, 200)) + [top, top * 2, top * (1 + 1e-7), 1.0, 63.5, 64.0]:
            e = exponent(a, top)
            assert a <= top * 2.0 ** (e - 127) and (e == 16 or a > top * 2.0 ** (e - 128))
    assert exponent(0.0, 127.0) == 16 and exponent(1e-40, 127.0) == 16


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_reference_quantisation_error(fmt):
    """Half a step: 2^(e - 128) for int8; half a unit in the last of 4 bits (2^-4) or half of 2^(e - 136) for e4m3."""
    rng = np.random.default_rng(2)
    x = rng.normal(size=(16, 64)) * np.exp(rng.normal(size=(16, 64)))
    q, e = quantise(x, fmt)
    y = decode(q[None], np.array([[e]], np.uint8), fmt)[0]
    bound = 2.0 ** (e - 128) if fmt == "int8" else np.maximum(np.abs(x) * 2.0 ** -4, 2.0 ** (e - 137))
    assert (np.abs(y - x) <= bound).all()


def test_reference_attention_matches_dense_softmax():
    import torch

    rng = np.random.default_rng(3)
    c = Cache("int8", 6, 2, 16, 32, [[3, 0, 5, -1]], rng)
    k, v = rng.normal(size=(2, 40, 2, 32))
    c.append(0, 0, k, v)
    q = rng.normal(size=(4, 32))
    out, lse, _, _ = c.attend(0, q, 37, 0.2)
    kk, vv = c.keys(0, [0, 1, 2])
    for h in range(4):
        z = torch.from_numpy(0.2 * kk[h // 2, :37] @ q[h])
        assert np.allclose(out[h], (torch.softmax(z, 0).numpy() @ vv[h // 2, :37]), rtol=1e-12, atol=1e-12)
        assert np.isclose(lse[h], float(torch.logsumexp(z, 0)))
    only = c.attend(0, q, 37, 0.2, pages=[[0, 2], [1]])[0]
    kk2, vv2 = c.keys(0, [0, 2])
    z = torch.from_numpy(0.2 * kk2[0, :21] @ q[1])
    assert np.allclose(only[1], torch.softmax(z, 0).numpy() @ vv2[0, :21])
    assert c.select(0, q, 37, 3, 0, 0) == [[0, 1, 2]] * 2
    bound = c.select(0, q, 37, 2, 0, 1)
    assert all(x[-1] == 2 and len(x) == 2 for x in bound)
