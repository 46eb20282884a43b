"""The 8-bit KV cache's operators: what is timed, their plain forms and their values in 64 bits.

Three operators over a paged cache whose keys and values are 8-bit codes with one power-of-two
scale per 16 tokens and head (value = code * 2^(exponent - 127)):

append  rows of keys and values quantised into the pages (a block that already holds rows is
        quantised again together with the new ones) and read back as the values the cache holds;
attend  softmax(scale q k^T) v over the first row_limit keys of each row's sequence;
sparse  the pages that score highest for a row by their keys' per-channel minima and maxima
        (a bound on q.k in whole numbers), then attention over those pages alone.

A page table gives each sequence's pages; pages lie in the pool in no order.
"""

import math

import torch

own = False

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
TOP = {"int8": 127.0, "e4m3": 448.0}
LOW = 16  # least stored exponent: 2^-111


# ------------------------------------------------------------------------------- cases
def _append(name, **k):
    return dict(name=name, op="append", **k)


def _attend(name, **k):
    return dict(dict(name=name, op="attend", lse=False, empty=False), **k)


def _sparse(name, **k):
    return dict(name=name, op="sparse", **k)


def listed():
    h16 = dict(kv_heads=16, dim=64, page=64)
    return [
        # one decoded byte of one sequence goes into the cache (fp32 rows, as the decoder computes them)
        _append("append_byte_b1", batch=1, rows=1, ctx=1024, format="int8", dtype="f32", **h16),
        # the accepted 16-byte drafts of 64 sequences, each ending at its own odd position
        _append("append_block16_b64", batch=64, rows=16, ctx=2048, format="e4m3", dtype="bf16", **h16),
        # four prompts of 8192 bytes
        _append("append_prompt8k_b4", batch=4, rows=8192, ctx=8192, format="int8", dtype="bf16", **h16),
        # a masked block of 4 bytes that sees itself and a prefix of 1024: one step of block diffusion at batch 1
        _attend("attend_block4_b1_1k", batch=1, rows=4, ctx=1028, mask="block", q_heads=16, format="int8", dtype="f32", **h16),
        # one byte at the end of 8192
        _attend("attend_byte_b1_8k", batch=1, rows=1, ctx=8192, mask="causal", q_heads=16, format="int8", dtype="bf16", **h16),
        # verification of 8-byte drafts of 16 sequences near 4096 bytes
        _attend("attend_verify8_b16_4k", batch=16, rows=8, ctx=4096, mask="causal", q_heads=16, format="int8", dtype="bf16", **h16),
        # one token each of 64 sequences of 4096 to 8192, four query heads to a key head
        _attend("attend_token_b64_gqa_8k", batch=64, rows=1, ctx=8192, mask="causal", q_heads=32, kv_heads=8, dim=128, page=64,
                format="e4m3", dtype="f16"),
        # four prompts of 2048 bytes, log-sum-exp kept to join them with another part
        _attend("attend_prompt2k_b4", batch=4, rows=2048, ctx=2048, mask="causal", q_heads=16, format="int8", dtype="bf16",
                **h16) | {"lse": True},
        # the last 1024 rows of a prompt of 8192 bytes (fp32 rows, as the decoder computes them)
        _attend("attend_chunk1k_b1_8k", batch=1, rows=1024, ctx=8192, mask="causal", q_heads=16, format="int8", dtype="f32", **h16),
        # one byte at the end of 32768, 2048 of them read
        _sparse("sparse_byte_b1_32k", batch=1, rows=1, ctx=32768, mask="causal", q_heads=16, format="int8", dtype="bf16",
                select=32, sink=1, local=2, **h16),
        # blocks of 4 masked bytes of 16 sequences of 8192, each row with pages of its own
        _sparse("sparse_block4_b16_8k", batch=16, rows=4, ctx=8192, mask="block", q_heads=16, format="int8", dtype="f32",
                select=16, sink=1, local=2, **h16),
        # one token each of 8 sequences of 32768, four query heads to a key head
        _sparse("sparse_token_b8_gqa_32k", batch=8, rows=1, ctx=32768, mask="causal", q_heads=32, kv_heads=8, dim=128, page=64,
                format="e4m3", dtype="f16", select=64, sink=1, local=4),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "sparse"])
    c = dict(op=op, page=rng.choice([16, 32, 64, 64, 128]), format=rng.choice(["int8", "e4m3"]),
             dtype=rng.choice(["f32", "bf16", "bf16", "f16"]), dim=rng.choice([32, 64, 64, 96, 128]))
    kv = rng.choice([1, 2, 4, 8, 16, 16])
    c["kv_heads"] = kv
    c["batch"] = _log(rng, 1, 64)
    if op == "append":
        c["rows"] = _log(rng, 1, 8192)
        while c["batch"] * c["rows"] > 32768:
            c["batch"] = max(1, c["batch"] // 2)
        c["rows"] = max(1, min(c["rows"], 32768 // c["batch"]))
        c["ctx"] = c["rows"] + rng.choice([0, rng.randrange(1, 100), rng.randrange(100, 1000)])
        while c["kv_heads"] * c["dim"] > 1024:
            c["kv_heads"] //= 2
        return c
    c["q_heads"] = kv * rng.choice([1, 1, 2, 3, 4, 8])
    while c["q_heads"] > 32:
        c["q_heads"] -= kv
    c["mask"] = rng.choice(["causal", "block"])
    if op == "attend":
        c["lse"] = rng.random() < 0.5
        c["empty"] = rng.random() < 0.3
        c["rows"] = rng.choice([1, rng.randrange(2, 33), _log(rng, 33, 2048)])
        c["ctx"] = c["rows"] + _log(rng, 1, 8192)
        while c["batch"] > 1 and (c["batch"] * c["ctx"] * kv * c["dim"] > 1 << 28 or work(c)["flops"] > 3e10):
            c["batch"] //= 2
        while work(c)["flops"] > 3e10:
            c["rows"] = c["rows"] // 2 + 1
        return c
    c["rows"] = rng.choice([1, 1, rng.randrange(2, 9)])
    c["ctx"] = c["rows"] + _log(rng, 256, 32768)
    c["select"] = _log(rng, 4, max(4, 4096 // c["page"]))
    c["sink"] = rng.randrange(0, 3)
    c["local"] = rng.randrange(1, 3)
    while c["batch"] > 1 and (c["batch"] * c["ctx"] * kv * c["dim"] > 1 << 28 or
                              c["batch"] * c["rows"] * c["select"] * c["page"] * kv * c["dim"] > 1 << 26):
        c["batch"] //= 2
    return c


# ------------------------------------------------------------------------------- inputs
def _pow2(n):
    """2^n in fp32 for whole n in -126 .. 127."""
    return ((n.to(torch.int32) + 127) << 23).view(torch.float32)


def _exponent(amax, top):
    """Least e with amax <= top * 2^(e - 127), not below LOW."""
    m, x = torch.frexp(amax)  # amax = m 2^x, m in [1/2, 1)
    tm, tx = math.frexp(top)
    e = x - tx + (m > tm).to(x.dtype) + 127
    return torch.where(amax > 0, e, torch.full_like(e, LOW)).clamp_min(LOW)


def _codes(x, e, fmt):
    """Codes (bytes) of x at exponent e (broadcast), to nearest even."""
    y = x * _pow2(127 - e)
    if fmt == "int8":
        return y.round().clamp(-127, 127).to(torch.int8).view(torch.uint8)
    return y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)


def _fill(c, g, lens, pool_pages, table, dev):
    """Pages holding lens[s] quantised rows of each sequence; bytes behind them are arbitrary."""
    H, D, PT = c["kv_heads"], c["dim"], c["page"]
    out = {}
    for name in ("k", "v"):
        codes = torch.randint(0, 255 if c["format"] == "int8" else 126, (pool_pages, H, PT, D), generator=g, device=dev, dtype=torch.uint8)
        exps = torch.randint(100, 120, (pool_pages, H, PT // 16), generator=g, device=dev, dtype=torch.uint8)
        chan = 0.5 + torch.rand(H, 1, D, generator=g, device=dev) * (1.0 if name == "v" else 1.5)
        if name == "k":
            chan = chan * torch.where(torch.rand(H, 1, D, generator=g, device=dev) < 0.04, 4.0, 1.0)  # a few loud channels
        for s, n in enumerate(lens):
            np_ = -(-n // PT)
            if np_ == 0:
                continue
            x = torch.randn(np_, H, PT, D, generator=g, device=dev) * chan
            if name == "k":  # pages differ, as stretches of a text do
                x += torch.randn(np_, H, 1, D, generator=g, device=dev) * chan * 0.7
            pos = torch.arange(np_ * PT, device=dev).view(np_, 1, PT, 1)
            x = torch.where(pos < n, x, torch.zeros_like(x))
            e = _exponent(x.abs().view(np_, H, PT // 16, 16 * D).amax(-1), TOP[c["format"]])
            q = _codes(x.view(np_, H, PT // 16, 16, D), e[..., None, None], c["format"]).view(np_, H, PT, D)
            at = table[s, :np_].long()
            codes[at] = torch.where(pos < n, q, codes[at])
            exps[at] = e.to(torch.uint8)
        out[name], out[name + "_exp"] = codes, exps
    return out


def prepare(case, seed):
    c, dev = case, "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    B, R, H, D, PT = c["batch"], c["rows"], c["kv_heads"], c["dim"], c["page"]
    if c["op"] == "append":
        # room for ctx rows; each sequence holds `start` rows when its new ones come
        slack = c["ctx"] - R
        start = [slack - (7 * s + 3) % (min(slack, 61) + 1) for s in range(B)]
        ends = [a + R for a in start]
        held = start
    else:
        spread = 0 if B == 1 else (c["ctx"] - R) // 2  # sequences of a batch have lengths of their own
        r = torch.rand(B, generator=g, device=dev).cpu()
        held = [c["ctx"] - int(spread * float(r[s])) for s in range(B)]
        ends = held
    max_pages = -(-c["ctx"] // PT) + 1
    need = [-(-e // PT) for e in ends]
    pool = sum(need) + 3
    perm = torch.randperm(pool, generator=g, device=dev).to(torch.int32)
    table = torch.full((B, max_pages), -1, dtype=torch.int32, device=dev)
    at = 0
    for s in range(B):
        table[s, :need[s]] = perm[at:at + need[s]]
        at += need[s]
    st = dict(case=c, table=table, **_fill(c, g, held, pool, table, dev))
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    st["row_offsets"] = i32([s * R for s in range(B + 1)])
    if c["op"] == "append":
        st["start"] = i32(start)
        for name in ("new_k", "new_v"):
            x = torch.randn(B * R, H, D, generator=g, device=dev)
            st[name] = (x * torch.where(torch.rand(B * R, 1, 1, generator=g, device=dev) < 0.02, 3.0, 1.0)).to(DT[c["dtype"]])
        first = [a // 16 * 16 for a in start]  # rows read back: from the first block that changed
        st["first"] = i32(first)
        off = [0]
        for s in range(B):
            off.append(off[-1] + ends[s] - first[s])
        st["read_offsets"], st["n_read"] = i32(off), off[-1]
        st["most_read"] = max(off[s + 1] - off[s] for s in range(B))
        st["read_k"], st["read_v"] = (torch.empty(off[-1], H, D, dtype=torch.bfloat16, device=dev) for _ in range(2))
        return st
    q = torch.randn(B * R, c["q_heads"], D, generator=g, device=dev)
    st["q"] = q.to(DT[c["dtype"]])
    row = torch.arange(R)
    lim = []
    for s in range(B):
        n = torch.full((R,), ends[s]) if c["mask"] == "block" else ends[s] - R + 1 + row
        lim.append(torch.zeros_like(n) if c.get("empty") and s == 0 else n)  # a slot without a sequence sees nothing
    st["row_limit"] = torch.cat(lim).to(torch.int32).to(dev)
    st["max_keys"] = max(ends)
    st["scale"] = 1.0 / math.sqrt(D)
    st["out"] = torch.empty(B * R, c["q_heads"], D, dtype=DT[c["dtype"]], device=dev)
    st["lse"] = torch.empty(B * R, c["q_heads"], dtype=torch.float32, device=dev) if c.get("lse") else None
    if c["op"] == "sparse":
        # what the cache keeps beside its keys: each page's least and greatest key value per channel, in 8 bits
        kmin = torch.zeros(pool, H, D, dtype=torch.int8, device=dev)
        kmax, ksexp = torch.zeros_like(kmin), torch.full((pool, H), LOW, dtype=torch.uint8, device=dev)
        for s in range(B):
            ids = table[s, :need[s]].long()
            x = _values(st["k"][ids], st["k_exp"][ids], c["format"])
            seen = (torch.arange(need[s] * PT, device=dev) < ends[s]).view(need[s], 1, PT, 1)
            lo = torch.where(seen, x, torch.full_like(x, float("inf"))).amin(2)
            hi = torch.where(seen, x, torch.full_like(x, float("-inf"))).amax(2)
            e = _exponent(torch.maximum(lo.abs(), hi.abs()).amax(-1), 127.0)
            kmin[ids] = (lo * _pow2(127 - e[..., None])).round().to(torch.int8)
            kmax[ids] = (hi * _pow2(127 - e[..., None])).round().to(torch.int8)
            ksexp[ids] = e.to(torch.uint8)
        st.update(k_min=kmin, k_max=kmax, k_sexp=ksexp)
        st["sel_pages"] = torch.empty(B * R, H, c["select"], dtype=torch.int32, device=dev)
        st["sel_count"] = torch.empty(B * R, H, dtype=torch.int32, device=dev)
    return st


# ------------------------------------------------------------------------------- plain forms
def _values(codes, exps, fmt):
    """[pages, H, PT, D] codes and [pages, H, PT / 16] exponents as fp32 values."""
    x = codes.view(torch.int8).float() if fmt == "int8" else codes.view(torch.float8_e4m3fn).float()
    return x * _pow2((exps.to(torch.int32) - 127).repeat_interleave(16, dim=-1)[..., None])


def _plain_append(s):
    c = s["case"]
    B, R, H, D, PT = c["batch"], c["rows"], c["kv_heads"], c["dim"], c["page"]
    dev, start = s["start"].device, s["start"].long()
    nb = (R + 30) // 16  # blocks of 16 tokens that R rows can touch
    blk = start[:, None] // 16 + torch.arange(nb, device=dev)  # [B, nb]
    pos = blk[..., None] * 16 + torch.arange(16, device=dev)  # [B, nb, 16]
    touched = blk * 16 < start[:, None] + R
    page = s["table"].long().gather(1, (blk * 16 // PT).clamp_max(s["table"].shape[1] - 1))
    page = torch.where(touched, page, torch.zeros_like(page))
    sub = blk * 16 % PT // 16
    old, new = pos < start[:, None, None], pos < start[:, None, None] + R
    src = (pos - start[:, None, None]).clamp(0, R - 1) + torch.arange(B, device=dev)[:, None, None] * R
    outs = []
    for name in ("k", "v"):
        codes = s[name].view(-1, H, PT // 16, 16, D)
        exps = s[name + "_exp"]
        had = codes[page, :, sub]  # [B, nb, H, 16, D]
        e0 = exps[page, :, sub]  # [B, nb, H]
        had_v = had.view(torch.int8).float() if c["format"] == "int8" else had.view(torch.float8_e4m3fn).float()
        had_v = had_v * _pow2(e0.to(torch.int32)[..., None, None] - 127)
        x = s["new_" + name][src].float().transpose(2, 3)  # [B, nb, H, 16, D]
        o, n = old[:, :, None, :, None], new[:, :, None, :, None]
        x = torch.where(o, had_v, torch.where(n, x, torch.zeros_like(x)))
        e = _exponent(x.abs().amax((-1, -2)), TOP[c["format"]])
        q = _codes(x, e[..., None, None], c["format"])
        t = touched.nonzero(as_tuple=True)
        codes[page[t], :, sub[t]] = torch.where(n.expand_as(q), q, had)[t]
        exps[page[t], :, sub[t]] = e.to(torch.uint8)[t]
        v = q.view(torch.int8).float() if c["format"] == "int8" else q.view(torch.float8_e4m3fn).float()
        v = (v * _pow2(e[..., None, None] - 127)).transpose(2, 3)  # [B, nb, 16, H, D]
        outs.append(v[new].to(torch.bfloat16))
    return outs


def _softmax(sc, seen):
    """Weights and log-sum-exp over the last axis; rows that see nothing get zeros and -inf."""
    sc = torch.where(seen, sc, torch.full_like(sc, float("-inf")))
    m = sc.amax(-1, keepdim=True)
    m0 = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    p = (sc - m0).exp()
    l = p.sum(-1, keepdim=True)
    lse = (m0 + l.log()).squeeze(-1)
    return p / torch.where(l > 0, l, torch.ones_like(l)), lse


def _plain_attend(s):
    c = s["case"]
    B, R, H, D, PT = c["batch"], c["rows"], c["kv_heads"], c["dim"], c["page"]
    G, n = c["q_heads"] // H, -(-s["max_keys"] // PT)
    ids = s["table"][:, :n].long().clamp_min(0)
    k, v = (_values(s[x][ids].flatten(0, 1), s[x + "_exp"][ids].flatten(0, 1), c["format"])
            .view(B, n, H, PT, D).transpose(1, 2).reshape(B, H, n * PT, D) for x in ("k", "v"))
    q = s["q"].float().view(B, R, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * R, D)
    sc = (q @ k.transpose(-1, -2)).view(B, H, G, R, n * PT) * s["scale"]
    seen = torch.arange(n * PT, device=q.device) < s["row_limit"].view(B, 1, 1, R, 1)
    p, lse = _softmax(sc, seen)
    o = (p.view(B, H, G * R, n * PT) @ v).view(B, H, G, R, D).permute(0, 3, 1, 2, 4).reshape(B * R, H * G, D)
    out = [o.to(DT[c["dtype"]])]
    if c["lse"]:
        out.append(lse.permute(0, 3, 1, 2).reshape(B * R, H * G))
    return out


def _plain_sparse(s):
    c = s["case"]
    B, R, H, D, PT = c["batch"], c["rows"], c["kv_heads"], c["dim"], c["page"]
    G, NS, n, N = c["q_heads"] // H, c["select"], -(-s["max_keys"] // PT), B * R
    dev, lim = s["q"].device, s["row_limit"].long()
    table = s["table"][:, :n].long().clamp_min(0)
    # scores: q in 8 bits with a power-of-two scale; sums of whole numbers below 2^24, so fp32 holds them
    q = s["q"].float()
    eq = _exponent(q.abs().amax(-1), 127.0)
    qi = (q * _pow2(127 - eq[..., None])).round().view(B, R, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, R * G, D)
    lo, hi = (s[x][table].float().transpose(1, 2) for x in ("k_min", "k_max"))  # [B, H, n, D]
    dot = qi.clamp_min(0) @ hi.transpose(-1, -2) + qi.clamp_max(0) @ lo.transpose(-1, -2)  # [B, H, R G, n]
    sc = dot.view(B, H, R, G, n).permute(0, 2, 1, 3, 4)  # [B, R, H, G, n]
    es = s["k_sexp"][table].to(torch.int32).transpose(1, 2)  # [B, H, n]
    sc = sc * _pow2(eq.view(B, R, H, G, 1) - 127) * _pow2(es[:, None, :, None, :] - 127)
    sc = sc.amax(3).view(N, H, n)
    # the first and the last pages always, then the highest scores, the lowest page first among equals
    pg = torch.arange(n, device=dev)
    nb = ((lim + PT - 1) // PT).view(N, 1, 1)
    sc = torch.where((pg < c["sink"]) | (pg >= nb - c["local"]), torch.full_like(sc, float("inf")), sc)
    sc = torch.where(pg < nb, sc, torch.full_like(sc, float("-inf")))
    order = torch.sort(sc, dim=-1, descending=True, stable=True)[1][..., :NS]
    if n < NS:
        order = torch.cat([order, order.new_full((N, H, NS - n), n)], -1)
    order = torch.where(order < nb, order, torch.full_like(order, 1 << 30)).sort(-1)[0]
    ok = order < (1 << 30)
    pages, count = torch.where(ok, order, torch.full_like(order, -1)), ok.sum(-1)
    # attention over them
    seq = torch.arange(N, device=dev)[:, None, None] // R
    ids = table[seq, pages.clamp_min(0)]  # [N, H, NS]
    hd = torch.arange(H, device=dev)[None, :, None]
    k, v = (_values(s[x][ids, hd].flatten(0, 1), s[x + "_exp"][ids, hd].flatten(0, 1), c["format"]).view(N, H, NS * PT, D)
            for x in ("k", "v"))
    at = (pages[..., None] * PT + torch.arange(PT, device=dev)).view(N, H, NS * PT)
    seen = ok.repeat_interleave(PT, -1) & (at < lim.view(N, 1, 1))
    p, _ = _softmax(q.view(N, H, G, D) @ k.transpose(-1, -2) * s["scale"], seen[:, :, None])
    return [(p @ v).view(N, H * G, D).to(DT[c["dtype"]]), pages.to(torch.int32), count.to(torch.int32)]


# ------------------------------------------------------------------------------- the framework's calls
def _plan(s):
    """The descriptors a user's program builds once for its buffers."""
    from block_diffusion_byte_b200 import binding as B

    c = s["case"]
    cache = B.kv8_cache(c["format"], s["k"], s["v"], s["k_exp"], s["v_exp"], s["table"], k_min=s.get("k_min"),
                        k_max=s.get("k_max"), k_sexp=s.get("k_sexp"))
    if c["op"] == "append":
        rows = B.kv8_rows(s["new_k"], s["new_v"], s["row_offsets"], s["start"], c["rows"])
        back = B.kv8_rows(s["read_k"], s["read_v"], s["read_offsets"], s["first"], s["most_read"])
        return [(B.blt_kv8_append, cache, rows), (B.blt_kv8_read, cache, back)], [s["read_k"], s["read_v"]]
    calls, outs, sel = [], [s["out"]], {}
    if c["op"] == "sparse":
        calls.append((B.blt_kv8_select, cache, B.kv8_selection(s["q"], s["row_offsets"], s["row_limit"], c["rows"], s["max_keys"],
                                                               s["sel_pages"], s["sel_count"], c["sink"], c["local"])))
        outs += [s["sel_pages"], s["sel_count"]]
        sel = dict(sel_pages=s["sel_pages"], sel_count=s["sel_count"])
    elif c["lse"]:
        outs.append(s["lse"])
    calls.append((B.blt_kv8_attend, cache, B.kv8_attention(s["q"], s["out"], s["row_offsets"], s["row_limit"], c["rows"],
                                                           s["max_keys"], s["scale"], lse=s["lse"], **sel)))
    return calls, outs


def run(state):
    if own:
        if "plan" not in state:
            state["plan"] = _plan(state)
        calls, outs = state["plan"]
        stream = torch.cuda.current_stream().cuda_stream
        for call, cache, args in calls:
            call(cache, args, stream)
        return outs
    return {"append": _plain_append, "attend": _plain_attend, "sparse": _plain_sparse}[state["case"]["op"]](state)


# ------------------------------------------------------------------------------- work
def work(case):
    """Codes, exponents and rows read and written once."""
    c, size = case, {"f32": 4, "bf16": 2, "f16": 2}[case["dtype"]]
    B, R, H, D = c["batch"], c["rows"], c["kv_heads"], c["dim"]
    key = 2 * H * (D + 1 / 16)  # a key's and a value's codes and exponents, all heads
    if c["op"] == "append":
        kept = 8 if c["ctx"] > R else 0  # rows of the first block that are already there, on average
        return {"bytes": B * (2 * R * H * D * size + (2 * kept + 2 * R) * key + 2 * (R + kept) * H * D * 2), "flops": 4 * B * R * H * D}
    held = c["ctx"] if B == 1 else c["ctx"] - (c["ctx"] - R) / 4
    io = B * R * c["q_heads"] * D * size * 2
    if c["op"] == "attend":
        keys = held if c["mask"] == "block" else held - (R - 1) / 2
        live = B - 1 if c["empty"] and B > 1 else B
        return {"bytes": live * held * key + io + (B * R * c["q_heads"] * 4 if c["lse"] else 0),
                "flops": 4.0 * live * R * keys * c["q_heads"] * D}
    pages = min(c["select"], held / c["page"])
    return {"bytes": B * (held / c["page"] * H * (2 * D + 1) + min(R * pages * c["page"], held) * key) + io + B * R * H * (c["select"] + 1) * 4,
            "flops": 4.0 * B * R * c["q_heads"] * D * (pages * c["page"] + held / c["page"])}


# ------------------------------------------------------------------------------- 64 bits
_E4M3 = [(-1.0 if b >> 7 else 1.0) * ((b & 7) / 8 * 2.0 ** -6 if (b >> 3 & 15) == 0 else (1 + (b & 7) / 8) * 2.0 ** ((b >> 3 & 15) - 7))
         for b in range(256)]


def _decode(codes, exps, fmt):
    """fp64 values of codes [..., 16 or PT, D] with exponents that broadcast to [...]."""
    if fmt == "int8":
        b = codes.double()
        x = torch.where(b > 127, b - 256, b)
    else:
        x = torch.tensor(_E4M3, dtype=torch.float64, device=codes.device)[codes.long()]
    return x * (exps.double() - 127).exp2()


def _sequence(st, name, s, n):
    """fp64 keys or values 0 .. n-1 of sequence s: [H, n, D]."""
    c = st["case"]
    np_ = -(-n // c["page"])
    ids = st["table"][s, :np_].long()
    x = _decode(st[name][ids], st[name + "_exp"][ids].repeat_interleave(16, -1)[..., None], c["format"])
    return x.transpose(0, 1).reshape(c["kv_heads"], np_ * c["page"], c["dim"])[:, :n]


def _quantised(x, fmt):
    """The fp64 values that 8 bits and a power-of-two scale hold of one block x [..., 16, D] (its own amax)."""
    top = TOP[fmt]
    a = x.abs().amax((-1, -2), keepdim=True)
    e = torch.ceil(torch.log2(torch.where(a > 0, a, torch.ones_like(a)) / top))
    e = torch.where(a > top * e.exp2(), e + 1, e)  # the logarithm's rounding
    e = torch.where(a <= top * (e - 1).exp2(), e - 1, e)
    e = torch.where(a > 0, e, torch.full_like(e, LOW - 127.0)).clamp_min(LOW - 127.0)
    y = x / e.exp2()
    if fmt == "int8":
        return y.round() * e.exp2()
    step = torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -6))).clamp_min(-6.0) - 3  # spacing of e4m3 around y
    return (y / step.exp2()).round() * step.exp2() * e.exp2()


def exact(case, seed):
    st = prepare(case, seed)
    c = case
    B, R, H, D, PT = c["batch"], c["rows"], c["kv_heads"], c["dim"], c["page"]
    if c["op"] == "append":
        outs = []
        for name in ("k", "v"):
            parts = []
            for s in range(B):
                a = int(st["start"][s])
                f = a // 16 * 16
                old = _sequence(st, name, s, a)[:, f:] if a > f else torch.zeros(H, 0, D, dtype=torch.float64, device="cuda")
                x = torch.cat([old, st["new_" + name][s * R:(s + 1) * R].double().transpose(0, 1)], 1)
                n = x.shape[1]
                x = torch.cat([x, x.new_zeros(H, -n % 16, D)], 1).view(H, -1, 16, D)
                parts.append(_quantised(x, c["format"]).reshape(H, -1, D)[:, :n].transpose(0, 1))
            outs.append(torch.cat(parts))
        return outs
    G = c["q_heads"] // H
    q = st["q"].double().view(B, R, H, G, D)
    lim = st["row_limit"].view(B, R)
    out, lse, pages, count = [], [], [], []
    for s in range(B):
        n = int(lim[s].max())
        if n == 0:
            out.append(torch.zeros(R, H * G, D, dtype=torch.float64, device="cuda"))
            lse.append(torch.full((R, H * G), float("-inf"), dtype=torch.float64, device="cuda"))
            continue
        k, v = _sequence(st, "k", s, n), _sequence(st, "v", s, n)
        see = (torch.arange(n, device="cuda") < lim[s][:, None])[:, None].expand(R, H, n)
        if c["op"] == "sparse":
            np_ = -(-n // PT)
            ids = st["table"][s, :np_].long()
            lo, hi = (st[x][ids].double() for x in ("k_min", "k_max"))  # [np, H, D]
            a = q[s].abs().amax(-1, keepdim=True)
            e = torch.ceil(torch.log2(a / 127.0))
            e = torch.where(a > 127.0 * e.exp2(), e + 1, e)
            e = torch.where(a <= 127.0 * (e - 1).exp2(), e - 1, e)
            qi = (q[s] / e.exp2()).round()  # [R, H, G, D]
            sc = torch.einsum("rhgd,phd->rhgp", qi.clamp_min(0), hi) + torch.einsum("rhgd,phd->rhgp", qi.clamp_max(0), lo)
            sc = (sc * e.exp2()).amax(2) * (st["k_sexp"][ids].double().T - 127).exp2()  # [R, H, np]
            for r in range(R):
                nb = -(-int(lim[s, r]) // PT)
                must = [p for p in range(nb) if p < c["sink"] or p >= nb - c["local"]]
                rest = sc[r, :, :nb].cpu().numpy()
                row = []
                for h in range(H):
                    order = must + [p for p in sorted(range(nb), key=lambda p: (-rest[h, p], p)) if p not in must]  # noqa: B023
                    row.append(sorted(order[:c["select"]]))
                count.append([len(x) for x in row])
                pages.append([x + [-1] * (c["select"] - len(x)) for x in row])
            pk = torch.zeros(R, H, np_ + 1, dtype=torch.bool, device="cuda")
            mine = torch.tensor(pages[-R:], device="cuda")
            pk.scatter_(2, torch.where(mine < 0, torch.full_like(mine, np_), mine), True)
            see = see & pk[..., :np_].repeat_interleave(PT, -1)[..., :n]
        for r0 in range(0, R, 256):  # a few rows at a time
            z = torch.einsum("rhgd,hnd->rhgn", q[s, r0:r0 + 256], k) * st["scale"]
            z = z.masked_fill(~see[r0:r0 + 256, :, None], float("-inf"))
            m = torch.logsumexp(z, -1)
            w = (z - torch.where(m == float("-inf"), torch.zeros_like(m), m)[..., None]).exp()
            out.append(torch.einsum("rhgn,hnd->rhgd", w, v).flatten(1, 2))
            lse.append(m.flatten(1))
    out = torch.cat(out)
    if c["op"] == "sparse":
        i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        return [out, i32(pages), i32(count)]
    return [out, torch.cat(lse)] if c["lse"] else [out]
