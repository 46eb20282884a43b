"""The 8-bit KV cache on the GPU against its definitions in 64 bits.

Stored codes, exponents, summaries and chosen pages are whole numbers and have to be equal.  Attention is
compared within the bounds that Cache.attend derives from the kernels' formats (fp32 sums, queries and weights
in f16 planes), plus half a step of the output's type.
"""

import numpy as np
import pytest
import torch

from _kv8_ref import Cache, decode

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
PLANES = {"f32": 22, "bf16": 11, "f16": 22}  # weights in two f16 planes (relative error 2^-11 each), for bf16 in one


@pytest.fixture(scope="module")
def B():
    from block_diffusion_byte_b200 import _build, binding

    _build.build()
    return binding


def dev(x, dt=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dt is None else t.to(dt)


def i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def table(rng, batch, pages, spare=2):
    """Page table with pages in no order, and the pool's size."""
    n = batch * pages + spare
    return rng.permutation(n)[:batch * pages].reshape(batch, pages).astype(np.int32), n


class Dev:
    """A Cache's arrays on the GPU."""

    def __init__(self, B, c, device="cuda"):
        self.B, self.c = B, c
        self.t = {n: dev(getattr(c, n)) for n in ("k", "v", "k_exp", "v_exp", "k_min", "k_max", "k_sexp") if getattr(c, n) is not None}
        self.table, self.status = dev(c.table), i32([0])
        self.desc = B.kv8_cache(c.fmt, self.t["k"], self.t["v"], self.t["k_exp"], self.t["v_exp"], self.table, self.t.get("k_min"),
                                self.t.get("k_max"), self.t.get("k_sexp"), self.status)

    def append(self, k, v, off, start, max_rows):
        self.B.blt_kv8_append(self.desc, self.B.kv8_rows(k, v, i32(off), i32(start), max_rows), torch.cuda.current_stream().cuda_stream)

    def read(self, off, start, dt, most):
        k, v = (torch.full((off[-1], self.c.H, self.c.D), 7.0, dtype=dt, device="cuda") for _ in range(2))
        self.B.blt_kv8_read(self.desc, self.B.kv8_rows(k, v, i32(off), i32(start), most), torch.cuda.current_stream().cuda_stream)
        return k, v

    def attend(self, q, off, lim, max_rows, scale, max_keys=None, out=None, lse=True, sel=None):
        out = torch.full_like(q, 7.0) if out is None else out
        ls = torch.full(q.shape[:2], 7.0, dtype=torch.float32, device="cuda") if lse else None
        sel = sel or (None, None)
        a = self.B.kv8_attention(q, out, i32(off), i32(lim), max_rows, max(lim, default=0) if max_keys is None else max_keys, scale, ls, *sel)
        self.B.blt_kv8_attend(self.desc, a, torch.cuda.current_stream().cuda_stream)
        return out, ls

    def select(self, q, off, lim, max_rows, n, sink, local):
        sp = torch.full((q.shape[0], self.c.H, n), 77, dtype=torch.int32, device="cuda")
        sc = torch.full((q.shape[0], self.c.H), 77, dtype=torch.int32, device="cuda")
        s = self.B.kv8_selection(q, i32(off), i32(lim), max_rows, max(lim, default=0), sp, sc, sink, local)
        self.B.blt_kv8_select(self.desc, s, torch.cuda.current_stream().cuda_stream)
        return sp, sc

    def same(self):
        for n, t in self.t.items():
            assert np.array_equal(t.cpu().numpy(), getattr(self.c, n)), n


def rows(rng, n, H, D, dt, wild=False):
    x = rng.normal(size=(n, H, D)) * np.exp(rng.normal(size=(n, 1, 1)) * 1.5)
    if wild and x.size:
        flat = x.reshape(-1)
        for val in (np.nan, np.inf, -np.inf, 0.0, -0.0, 1e-42, 3e38, -3e-38, 1.5e-34):
            flat[rng.integers(0, flat.size, 2)] = val
        x[rng.integers(0, n)] = 0.0
    with np.errstate(over="ignore"):
        t = torch.from_numpy(x).to(torch.float32).to(dt).cuda()
    return t, t.double().cpu().numpy()


def filled(B, rng, fmt, H, PT, D, lens, dt=torch.float32, max_pages=None, summaries=True):
    """A cache with lens[s] rows in each sequence, stored by the library and by the reference."""
    mp = max_pages or max(1, max(-(-n // PT) for n in lens))
    tab, n_pages = table(rng, len(lens), mp)
    c = Cache(fmt, n_pages, H, PT, D, tab, rng, summaries)
    d = Dev(B, c)
    off = [0] + list(np.cumsum(lens))
    chan = np.where(rng.random((1, H, D)) < 0.05, 4.0, 1.0)
    k = torch.from_numpy(rng.normal(size=(off[-1], H, D)) * chan).to(dt).cuda()
    v = torch.from_numpy(rng.normal(size=(off[-1], H, D))).to(dt).cuda()
    if off[-1]:
        d.append(k, v, off, [0] * len(lens), max(lens))
    for n, t in d.t.items():  # checked against the reference by the tests of append
        setattr(c, n, t.cpu().numpy())
    return c, d


# ------------------------------------------------------------------------------- append, read
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dt,D,PT,H", [("f32", 64, 64, 2), ("bf16", 64, 16, 3), ("f16", 128, 32, 1), ("bf16", 96, 48, 2), ("f32", 32, 256, 1),
                                       ("bf16", 128, 128, 4)])
def test_append_stores_what_the_definition_says(B, fmt, dt, D, PT, H):
    """Three appends in turn: from zero, behind odd ends, and over positions that were stored before."""
    rng = np.random.default_rng(D + PT)
    tab, n_pages = table(rng, 5, 3 if PT < 256 else 2)
    c = Cache(fmt, n_pages, H, PT, D, tab, rng)
    d = Dev(B, c)
    cap = tab.shape[1] * PT
    held = [0] * 5
    for turn in range(3):
        n = [int(rng.integers(0, min(40, cap - 45))), 1, 0, int(rng.integers(1, 17)), 16]
        start = list(held) if turn < 2 else [max(0, h - 5) for h in held]
        off = [0] + list(np.cumsum(n))
        (k, kn), (v, vn) = (rows(rng, off[-1], H, D, DT[dt], wild=turn > 0) for _ in range(2))
        d.append(k, v, off, start, max(n))
        for s in range(5):
            c.append(s, start[s], kn[off[s]:off[s + 1]], vn[off[s]:off[s + 1]])
            held[s] = start[s] + n[s]
        d.same()
    assert int(d.status) == 0


def test_append_long_prompt_without_summaries_and_strided_rows(B):
    rng = np.random.default_rng(5)
    H, D, PT, n = 2, 64, 64, 500
    tab, n_pages = table(rng, 1, 9)
    c = Cache("int8", n_pages, H, PT, D, tab, rng, summaries=False)
    d = Dev(B, c)
    buf = torch.from_numpy(rng.normal(size=(n, 3, H, D + 1))).to(torch.bfloat16).cuda()  # rows of a wider, oddly strided buffer
    k, v = buf[:, 0, :, :D], buf[:, 1, :, :D]
    for start, r in ((0, slice(0, 13)), (13, slice(13, n))):
        d.append(k[r], v[r], [0, len(k[r])], [start], n)
        c.append(0, start, k[r].double().cpu().numpy(), v[r].double().cpu().numpy())
    d.same()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dt", ["f32", "bf16", "f16"])
def test_read_gives_the_stored_values(B, fmt, dt):
    rng = np.random.default_rng(7)
    c, d = filled(B, rng, fmt, 2, 32, 96, [70, 0, 33])
    off, start = [0, 50, 50, 70], [20, 0, 13]
    k, v = d.read(off, start, DT[dt], 50)
    for name, got in (("k", k), ("v", v)):
        for s in range(3):
            pos = np.arange(start[s], start[s] + off[s + 1] - off[s])
            want = decode(getattr(c, name), getattr(c, name + "_exp"), fmt)[c.table[s, pos // 32], :, pos % 32]
            assert torch.equal(got[off[s]:off[s + 1]].cpu(), torch.from_numpy(want).to(torch.float32).to(DT[dt]))


def test_missing_pages_and_bad_offsets_are_reported_and_skipped(B):
    """Page numbers outside the pool, offsets beyond the arrays and rows beyond the table: checked by the kernels."""
    rng = np.random.default_rng(8)
    H, D, PT = 1, 32, 16
    c, d = filled(B, rng, "int8", H, PT, D, [40, 40])
    before = {n: t.clone() for n, t in d.t.items()}
    d.table[1, 1] = c.k.shape[0]
    d.table[1, 2] = -5
    k, v = d.read([0, 40, 80], [0, 0], torch.float32, 40)
    assert int(d.status) == B.BLT_ERR_DEVICE
    assert (k[56:] == 0).all() and (v[56:] == 0).all() and (k[:56] != 7.0).all()
    d.status.zero_()
    x = torch.randn(24, H, D, device="cuda")
    d.append(x, x, [0, 0, 24], [0, 16], 24)  # both pages are missing
    assert int(d.status) == B.BLT_ERR_DEVICE
    assert all(torch.equal(t, before[n]) for n, t in d.t.items())
    d.status.zero_()
    q = torch.randn(2, 1, D, device="cuda")
    out, lse = d.attend(q, [0, 1, 2], [40, 40], 1, 0.2)
    assert int(d.status) == B.BLT_ERR_DEVICE
    c.table[1, 1:] = c.table[1, 0]
    want = c.attend(1, q[1].double().cpu().numpy(), 16, 0.2)[0]  # the keys whose page is there
    assert np.abs(out[1].cpu().numpy() - want).max() < 1e-4
    d.status.zero_()
    big = q.repeat(100, 1, 1)
    out, _ = d.attend(big, [0, 100, 200], [40] * 200, 100, 0.2, max_keys=1 << 14)  # many-row tiles
    assert int(d.status) == B.BLT_ERR_DEVICE
    assert np.abs(out[101::2].cpu().numpy() - want).max() < 1e-4
    d.status.zero_()
    out, _ = d.attend(q, [0, 1, 99], [40, 16], 5, 0.2)  # the second sequence's end is cut to the array
    assert int(d.status) == B.BLT_ERR_DEVICE and bool((out != 7.0).all())
    d.status.zero_()
    d.append(x, x, [0, 24, 24], [30, 0], 24)  # 54 positions in 48
    assert int(d.status) == B.BLT_ERR_DEVICE
    assert all(torch.equal(t, before[n]) for n, t in d.t.items())


# ------------------------------------------------------------------------------- attend
def check(c, q, out, lse, off, lim, scale, dt, pages=None):
    """Rows of every sequence against the definition, rows outside left as they were."""
    eps = torch.finfo(DT[dt]).eps / 2
    qn, on, ln = q.double().cpu().numpy(), out.double().cpu().numpy(), lse.cpu().numpy()
    for s in range(len(off) - 1):
        for r in range(off[s], off[s + 1]):
            want, wl, eo, el = c.attend(s, qn[r], lim[r], scale, None if pages is None else pages[r], planes=PLANES[dt])
            tol = eo + (np.abs(want) + eo) * eps + 2.0 ** -25 * (dt == "f16")  # fp16 results may be subnormal
            bad = np.abs(on[r] - want) > tol
            assert not bad.any(), (s, r, np.abs(on[r] - want).max(), tol[bad].min())
            seen = np.isfinite(wl)
            assert np.array_equal(np.isneginf(ln[r]), ~seen)
            assert (np.abs(ln[r][seen] - wl[seen]) <= el[seen]).all()
    assert (on[off[-1]:] == 7.0).all() and (ln[off[-1]:] == 7.0).all()


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dt,D,PT,H,G", [("f32", 64, 64, 2, 1), ("bf16", 64, 16, 1, 4), ("f16", 128, 64, 1, 4), ("bf16", 96, 48, 2, 3),
                                         ("f32", 128, 32, 1, 8), ("f32", 32, 16, 3, 1), ("f16", 32, 128, 1, 16), ("bf16", 128, 256, 2, 2),
                                         ("f16", 96, 16, 1, 1), ("f32", 96, 80, 1, 2)])
def test_attend_few_rows(B, fmt, dt, D, PT, H, G):
    """Single tokens, blocks and drafts; rows that see nothing; a sequence without rows; rows behind the last."""
    rng = np.random.default_rng(D + PT + G)
    lens = [1, 300, 17, 0, 161, 64]
    c, d = filled(B, rng, fmt, H, PT, D, lens)
    off = [0, 1, 6, 6, 7, 23, 24]
    lim = [1] + [296, 297, 0, 299, 300] + [0] + [161] * 8 + list(range(1, 9)) + [63] + [5, 5]
    q = torch.from_numpy(rng.normal(size=(26, H * G, D)) * 1.5).to(DT[dt]).cuda()
    scale = D ** -0.5
    out, lse = d.attend(q, off, lim, 16, scale)
    check(c, q, out, lse, off, lim, scale, dt)
    assert int(d.status) == 0


@pytest.mark.parametrize("dt,D,H,G,rows_,ctx", [("bf16", 64, 1, 1, 130, 130), ("f32", 64, 1, 1, 129, 400), ("f16", 128, 1, 2, 65, 257),
                                                ("bf16", 96, 1, 1, 140, 300), ("bf16", 32, 2, 1, 200, 203), ("f32", 128, 1, 1, 160, 170),
                                                ("bf16", 128, 1, 3, 97, 500), ("f32", 96, 1, 1, 150, 151), ("f16", 64, 1, 5, 61, 700),
                                                ("f32", 32, 1, 1, 257, 300), ("f16", 96, 1, 1, 128, 129), ("f16", 32, 1, 4, 96, 97)])
@pytest.mark.parametrize("mask", ["causal", "block", "ragged"])
def test_attend_many_rows(B, dt, D, H, G, rows_, ctx, mask):
    """Prompts: causal rows, rows that see each other, and limits in no order with empty rows among them."""
    rng = np.random.default_rng(rows_ + ctx)
    c, d = filled(B, rng, "int8" if rows_ % 2 else "e4m3", H, 64, D, [ctx, ctx // 3, 40])
    n2 = min(rows_, ctx // 3)
    off = [0, rows_, rows_ + n2, rows_ + n2]
    if mask == "causal":
        lim = list(range(ctx - rows_ + 1, ctx + 1)) + list(range(1, n2 + 1))
    elif mask == "block":
        lim = [ctx] * rows_ + [ctx // 3] * n2
    else:
        lim = [int(x) for x in rng.integers(0, ctx + 1, rows_)] + [0] * n2
        lim[0:5] = [0, ctx, 1, 0, 2]
    lim += [9, 9]  # rows of no sequence
    q = torch.from_numpy(rng.normal(size=(off[-1] + 2, H * G, D))).to(DT[dt]).cuda()
    scale = D ** -0.5
    for keys in (None, 4096, 1 << 20):  # the expected keys choose between few-row and many-row tiles, and how the keys are split
        out, lse = d.attend(q, off, lim, rows_, scale, max_keys=keys)
        check(c, q, out, lse, off, lim, scale, dt)


def dense(c, d, q, off, lim, scale, planes):
    """Cache.attend and its bounds for all rows at once, in 64 bits on the GPU."""
    kv = []
    for name in ("k", "v"):
        x = torch.from_numpy(decode(d.t[name].cpu().numpy(), d.t[name + "_exp"].cpu().numpy(), c.fmt)).cuda()
        kv.append(x[torch.from_numpy(c.table).cuda().long()].transpose(1, 2).flatten(2, 3))  # [B, H, n, D]
    outs, errs = [], []
    for s in range(len(off) - 1):
        n = max(lim[off[s]:off[s + 1]])
        k, v = (x[s, :, :n] for x in kv)
        qs = q[off[s]:off[s + 1]].double().unflatten(1, (c.H, -1))  # [R, H, G, D]
        z = torch.einsum("rhgd,hnd->rhgn", qs, k) * scale
        z = z.masked_fill(torch.arange(n, device="cuda") >= i32(lim[off[s]:off[s + 1]])[:, None, None, None], float("-inf"))
        mag = abs(scale) * torch.einsum("rhgd,hnd->rhgn", qs.abs(), k.abs()).amax(-1)
        zmax = z.masked_fill(z == float("-inf"), 0).abs().amax(-1)
        dd = mag * ((c.D + 4) * 2.0 ** -23 + 2.0 ** -22) + 2.0 ** -22 * (1 + zmax)
        dd = dd + 2.0 ** -39 * abs(scale) * qs.abs().amax(-1) * k.abs().sum(-1).amax(-1)[None, :, None]
        w = torch.softmax(z, -1)
        outs.append(torch.einsum("rhgn,hnd->rhgd", w, v).flatten(1, 2))
        e = torch.einsum("rhgn,hnd->rhgd", w, v.abs()) * (2 * dd + (n / 4 + 64) * 2.0 ** -23 + 2.0 ** -planes)[..., None]
        # the largest value scale: at most twice the largest magnitude over top, as a block's exponent is the least
        errs.append((e + 2.0 ** -33 * n * 2 * v.abs().amax()).flatten(1, 2))
    return torch.cat(outs), torch.cat(errs)


@pytest.mark.parametrize("dt,D,H,G,rows_,ctx,batch", [("bf16", 64, 8, 1, 1024, 1024, 4), ("f32", 64, 4, 1, 512, 2100, 1), ("f16", 128, 2, 2, 640, 1500, 2),
                                                      ("f32", 128, 2, 1, 300, 3000, 1), ("bf16", 96, 4, 2, 777, 1001, 2), ("bf16", 32, 16, 1, 900, 900, 2),
                                                      ("f32", 64, 16, 1, 1024, 4096, 1), ("bf16", 128, 8, 1, 700, 700, 4)])
def test_attend_prompts_that_fill_the_gpu(B, dt, D, H, G, rows_, ctx, batch):
    """Many tiles of keys and many CTAs at once, twice: every row in its bounds, and the same bits again."""
    rng = np.random.default_rng(D + rows_)
    lens = [ctx - 37 * s for s in range(batch)]
    n = [rows_ - 37 * s for s in range(batch)]
    c, d = filled(B, rng, "int8" if D != 96 else "e4m3", H, 64, D, lens)
    off = [0] + [int(x) for x in np.cumsum(n)]
    lim = [int(x) for s in range(batch) for x in range(lens[s] - n[s] + 1, lens[s] + 1)]
    q = torch.from_numpy(rng.normal(size=(off[-1], H * G, D)) * 2).to(DT[dt]).cuda()
    want, err = dense(c, d, q, off, lim, D ** -0.5, PLANES[dt])
    first = None
    for _ in range(3):
        out, _ = d.attend(q, off, lim, max(n), D ** -0.5)
        assert bool((((out.double() - want).abs() <= err + (want.abs() + err) * torch.finfo(DT[dt]).eps / 2 + 2.0 ** -25)).all())
        first = out if first is None else first
        assert torch.equal(out, first)
    assert int(d.status) == 0


@pytest.mark.parametrize("dt,rows_", [("bf16", 1), ("f32", 3), ("f16", 140), ("f32", 140)])
def test_attend_loud_keys_and_scales(B, dt, rows_):
    """Scores far apart (one key takes all the weight), a negative scale and scale 0 (all keys alike)."""
    rng = np.random.default_rng(11)
    c, d = filled(B, rng, "int8", 1, 64, 64, [350])
    q = torch.from_numpy(rng.normal(size=(rows_, 2, 64)) * 30).to(DT[dt]).cuda()
    lim = [350 - i for i in range(rows_)]
    for scale in (1.0, -0.7, 0.0):
        for keys in (350, 1 << 20):
            out, lse = d.attend(q, [0, rows_], lim, rows_, scale, max_keys=keys)
            check(c, q, out, lse, [0, rows_], lim, scale, dt)


@pytest.mark.parametrize("dt,rows_", [("bf16", 2), ("f32", 2), ("f16", 150), ("f32", 150)])
def test_attend_ignores_what_lies_behind_the_limit(B, dt, rows_):
    """Codes behind the limit (NaN patterns among them) and whole pages of them change no bit."""
    rng = np.random.default_rng(12)
    c, d = filled(B, rng, "e4m3", 1, 32, 64, [200], max_pages=9)
    q = torch.from_numpy(rng.normal(size=(rows_, 1, 64))).to(DT[dt]).cuda()
    lim = [171 + i % 30 for i in range(rows_)]
    a, la = d.attend(q, [0, rows_], lim, rows_, 0.125, max_keys=1 << 14)
    for name in ("k", "v"):
        d.t[name][d.table[0, 6].long(), :, 8:] = 255
        d.t[name][d.table[0, 7:].long()] = 127
        d.t[name + "_exp"][d.table[0, 7:].long()] = 255
    b, lb = d.attend(q, [0, rows_], lim, rows_, 0.125, max_keys=1 << 14)
    assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("dt,rows_", [("bf16", 1), ("f16", 9), ("f32", 9), ("bf16", 130), ("f32", 130)])
def test_attend_strides_and_max_keys(B, dt, rows_):
    """Rows inside wider, oddly aligned buffers; max_keys only shapes the launch."""
    rng = np.random.default_rng(13)
    c, d = filled(B, rng, "int8", 2, 64, 64, [600])
    base = torch.from_numpy(rng.normal(size=(rows_, 3, 4, 65))).to(DT[dt]).cuda()
    q = base[:, 1, :, 1:]
    out = torch.full((4, rows_, 67), 7.0, dtype=DT[dt], device="cuda").transpose(0, 1)[..., 2:66]
    lim = [600 - 3 * i for i in range(rows_)]
    for keys in (0, 1, 600, 1 << 20):
        out, lse = d.attend(q, [0, rows_], lim, rows_, 0.125, max_keys=keys, out=out)
        check(c, q, out, lse, [0, rows_], lim, 0.125, dt)
    dense, _ = d.attend(q.contiguous(), [0, rows_], lim, rows_, 0.125)
    again, _ = d.attend(q.contiguous(), [0, rows_], lim, rows_, 0.125)
    assert torch.equal(dense, again)


@pytest.mark.parametrize("rows_", [1, 140])
def test_offsets_beyond_32_bits(B, rows_):
    """Pages of a layer inside a pool whose pages lie 96 MiB apart: 5 GB from the first to the last."""
    rng = np.random.default_rng(14)
    n, H, PT, D, stride = 54, 1, 16, 32, 96 << 20
    lens = [PT * 50 + 3]
    tab = rng.permutation(n)[:51].reshape(1, 51).astype(np.int32)
    c = Cache("int8", n, H, PT, D, tab, rng, summaries=False)
    pools = [torch.zeros(stride * (n - 1) + H * PT * D, dtype=torch.uint8, device="cuda") for _ in range(2)]
    k, v = (p.as_strided((n, H, PT, D), (stride, PT * D, D, 1)) for p in pools)
    ke, ve = (torch.zeros(n, H, 1, dtype=torch.uint8, device="cuda") for _ in range(2))
    d = Dev(B, c)
    d.t = dict(k=k, v=v, k_exp=ke, v_exp=ve)
    d.desc = B.kv8_cache("int8", k, v, ke, ve, d.table, status=d.status)
    x, xn = rows(rng, lens[0], H, D, torch.float32)
    y, yn = rows(rng, lens[0], H, D, torch.float32)
    d.append(x, y, [0, lens[0]], [0], lens[0])
    c.append(0, 0, xn, yn)
    used = torch.from_numpy(tab[0].astype(np.int64)).cuda()
    assert np.array_equal(ke[used].cpu().numpy(), c.k_exp[tab[0]])
    assert np.array_equal(k[used[:50]].cpu().numpy(), c.k[tab[0, :50]])
    q = torch.randn(rows_, 1, D, device="cuda")
    lim = [lens[0]] * rows_
    out, lse = d.attend(q, [0, rows_], lim, rows_, 0.2, max_keys=1 << 14)
    check(c, q, out, lse, [0, rows_], lim, 0.2, "f32")


# ------------------------------------------------------------------------------- select, and all together
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dt,D,PT,H,G,n,sink,local", [("f32", 64, 16, 2, 1, 5, 1, 2), ("bf16", 128, 16, 1, 4, 8, 0, 1), ("f16", 96, 32, 2, 2, 1, 0, 0),
                                                      ("f16", 32, 16, 1, 8, 12, 2, 0), ("bf16", 64, 64, 1, 2, 40, 1, 1), ("f32", 64, 16, 1, 3, 3, 1, 2)])
def test_select_chooses_the_highest_bounds(B, fmt, dt, D, PT, H, G, n, sink, local):
    rng = np.random.default_rng(D + n)
    c, d = filled(B, rng, fmt, H, PT, D, [900, 1, 333, 0])
    q = torch.from_numpy(rng.normal(size=(8, H * G, D))).to(DT[dt]).cuda()
    off, lim = [0, 3, 4, 6, 7], [900, 850, 0, 1, 333, 20, 0, 5]
    sp, sc = d.select(q, off, lim, 3, n, sink, local)
    qn = q.double().cpu().numpy()
    for s in range(4):
        for r in range(off[s], off[s + 1]):
            want = c.select(s, qn[r], lim[r], n, sink, local)
            for h in range(H):
                assert int(sc[r, h]) == len(want[h])
                assert sp[r, h].tolist() == want[h] + [-1] * (n - len(want[h])), (s, r, h)
    assert bool((sp[7] == 77).all()) and bool((sc[7] == 77).all())


def test_select_ties_extremes_and_odd_queries(B):
    """Equal scores go to the lowest pages; zero, NaN and infinite query channels; scores that leave fp32's range."""
    rng = np.random.default_rng(21)
    c, d = filled(B, rng, "int8", 1, 16, 32, [16 * 700])
    one = d.table[0].long()
    for name in ("k_min", "k_max", "k_sexp"):  # every page alike but a few
        d.t[name][one] = d.t[name][one[5]].clone()
    for p in (100, 101, 650):
        d.t["k_max"][one[p]] = 127
        d.t["k_min"][one[p]] = -127
    for n, t in d.t.items():
        setattr(c, n, t.cpu().numpy())
    q = torch.randn(4, 1, 32, device="cuda")
    q[1] = 0
    q[2, 0, 3], q[2, 0, 4] = float("nan"), float("inf")
    off, lim = [0, 4], [16 * 700] * 4
    sp, sc = d.select(q, off, lim, 4, 40, 2, 3)
    qn = q.double().cpu().numpy()
    for r in range(4):
        assert sp[r, 0].tolist() == c.select(0, qn[r], lim[r], 40, 2, 3)[0]
    d.t["k_sexp"][one] = 249  # with a loud query: every score beyond fp32
    sp, _ = d.select(torch.full((1, 1, 32), 3e38, device="cuda"), [0, 1], [16 * 700], 1, 9, 1, 4)
    assert sp[0, 0].tolist()[:1] == [0] and sp[0, 0].tolist()[-4:] == [696, 697, 698, 699]


@pytest.mark.parametrize("fmt,dt,D,H,G", [("int8", "bf16", 64, 2, 1), ("e4m3", "f16", 128, 1, 4), ("int8", "f32", 64, 1, 12), ("e4m3", "bf16", 96, 1, 20)])
def test_sparse_decoding_run(B, fmt, dt, D, H, G):
    """A prompt stored, then tokens one by one: stored, pages chosen, attended, as a serving loop does."""
    rng = np.random.default_rng(31)
    PT, n = 32, 6
    tab, n_pages = table(rng, 2, 16)
    c = Cache(fmt, n_pages, H, PT, D, tab, rng)
    d = Dev(B, c)
    held = [300, 411]
    off = [0, 300, 711]
    (k, kn), (v, vn) = (rows(rng, 711, H, D, DT[dt]) for _ in range(2))
    d.append(k, v, off, [0, 0], 411)
    for s in range(2):
        c.append(s, 0, kn[off[s]:off[s + 1]], vn[off[s]:off[s + 1]])
    for _ in range(4):
        (k, kn), (v, vn) = (rows(rng, 2, H, D, DT[dt]) for _ in range(2))
        q = torch.from_numpy(rng.normal(size=(2, H * G, D))).to(DT[dt]).cuda()
        d.append(k, v, [0, 1, 2], held, 1)
        for s in range(2):
            c.append(s, held[s], kn[s:s + 1], vn[s:s + 1])
            held[s] += 1
        sel = d.select(q, [0, 1, 2], held, 1, n, 1, 1)
        out, lse = d.attend(q, [0, 1, 2], held, 1, D ** -0.5, sel=sel)
        pages = [c.select(s, q[s].double().cpu().numpy(), held[s], n, 1, 1) for s in range(2)]
        assert sel[0].cpu().tolist() == pages
        check(c, q, out, lse, [0, 1, 2], held, D ** -0.5, dt, pages)
    d.same()


def test_selected_pages_out_of_order_or_range_are_ignored(B):
    rng = np.random.default_rng(32)
    c, d = filled(B, rng, "int8", 1, 16, 64, [200])
    q = torch.randn(3, 2, 64, device="cuda")
    sp = torch.tensor([[[2, 2, 1, 5, 7]], [[-1, 3, 99, 100, 12]], [[0, 4, 12, -1, -1]]], dtype=torch.int32, device="cuda")
    sc = torch.tensor([[5], [9], [3]], dtype=torch.int32, device="cuda")
    lim = [200, 200, 0]
    out, lse = d.attend(q, [0, 3], lim, 3, 0.125, sel=(sp, sc))
    # an entry not greater than the one before it is not read; one behind the table or the limit sees nothing
    check(c, q, out, lse, [0, 3], lim, 0.125, "f32", [[[2, 5, 7]], [[3]], [[]]])


def test_captured_calls_replay_beside_each_other(B):
    """The three calls of a step in two graphs that share the cache, replayed on two streams with new data."""
    rng = np.random.default_rng(33)
    c, d = filled(B, rng, "int8", 2, 32, 64, [400, 257], max_pages=20)
    lim = [400, 257]
    qs = [torch.randn(2, 4, 64, device="cuda") for _ in range(2)]
    outs, graphs = [], []
    streams = [torch.cuda.Stream() for _ in range(2)]
    off, lims = i32([0, 1, 2]), i32(lim)
    for q, st in zip(qs, streams):
        sp = torch.empty(2, 2, 5, dtype=torch.int32, device="cuda")
        sc = torch.empty(2, 2, dtype=torch.int32, device="cuda")
        full, part = torch.empty_like(q), torch.empty_like(q)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            h = torch.cuda.current_stream().cuda_stream
            B.blt_kv8_attend(d.desc, B.kv8_attention(q, full, off, lims, 1, 400, 0.125), h)
            B.blt_kv8_select(d.desc, B.kv8_selection(q, off, lims, 1, 400, sp, sc, 1, 1), h)
            B.blt_kv8_attend(d.desc, B.kv8_attention(q, part, off, lims, 1, 400, 0.125, sel_pages=sp, sel_count=sc), h)
        graphs.append(g)
        outs.append((full, part, sp, sc))
    for _ in range(3):
        for q in qs:
            q.copy_(torch.randn_like(q))
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for q, (full, part, sp, sc) in zip(qs, outs):
            want, _ = d.attend(q, [0, 1, 2], lim, 1, 0.125, max_keys=400)
            sel = d.select(q, [0, 1, 2], lim, 1, 5, 1, 1)
            wpart, _ = d.attend(q, [0, 1, 2], lim, 1, 0.125, max_keys=400, sel=sel)
            torch.cuda.synchronize()
            assert torch.equal(full, want) and torch.equal(sp, sel[0]) and torch.equal(part, wpart)


@pytest.mark.parametrize("dt,D", [("bf16", 64), ("f32", 64), ("f16", 128)])
def test_prompts_on_two_streams_and_in_graphs(B, dt, D):
    """Many-row calls that share the cache run beside each other (and share SMs' tensor memory), eager and replayed."""
    rng = np.random.default_rng(34)
    c, d = filled(B, rng, "int8", 4, 64, D, [700, 513])
    off, lim = [0, 300, 500], [401 + i for i in range(300)] + [314 + i for i in range(200)]
    qs = [torch.randn(500, 8, D, device="cuda").to(DT[dt]) for _ in range(2)]
    want = [d.attend(q, off, lim, 300, 0.1, max_keys=4096)[0] for q in qs]
    offs, lims = i32(off), i32(lim)
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [torch.empty_like(q) for q in qs]
    torch.cuda.synchronize()
    for _ in range(4):
        for q, out, st in zip(qs, outs, streams):
            B.blt_kv8_attend(d.desc, B.kv8_attention(q, out, offs, lims, 300, 4096, 0.1), st.cuda_stream)
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    graphs = []
    for q, out, st in zip(qs, outs, streams):
        out.zero_()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            B.blt_kv8_attend(d.desc, B.kv8_attention(q, out, offs, lims, 300, 4096, 0.1), torch.cuda.current_stream().cuda_stream)
        graphs.append(g)
    for _ in range(3):
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for o, w in zip(outs, want))
    assert int(d.status) == 0


def test_smallest_calls(B):
    """One row, one key, one head; a page of 16; rows and keys at a page's and a block's border; no rows in any sequence."""
    rng = np.random.default_rng(35)
    for n in (1, 15, 16, 17, 32, 33):
        c, d = filled(B, rng, "e4m3", 1, 16, 32, [n])
        q = torch.randn(1, 1, 32, device="cuda")
        out, lse = d.attend(q, [0, 1], [n], 1, 1.0)
        check(c, q, out, lse, [0, 1], [n], 1.0, "f32")
        sel = d.select(q, [0, 1], [n], 1, 1, 0, 1)
        assert sel[0][0, 0].tolist() == [(n - 1) // 16] and int(sel[1][0, 0]) == 1
        out, lse = d.attend(q, [0, 1], [n], 1, 1.0, sel=sel)
        check(c, q, out, lse, [0, 1], [n], 1.0, "f32", [[[(n - 1) // 16]]])
        out, lse = d.attend(q, [0, 0], [n], 1, 1.0)
        assert bool((out == 7.0).all()) and bool((lse == 7.0).all())
        before = {name: t.clone() for name, t in d.t.items()}
        d.append(q, q, [0, 0], [0], 1)
        assert all(torch.equal(t, before[name]) for name, t in d.t.items())
