"""Calls of the 8-bit KV cache that are refused, without a GPU: flags that mean nothing, tensors that do not fit."""

import pytest
import torch

from test_kv8 import B, _attn, _cache, _rows  # noqa: F401  (B: the fixture)


@pytest.mark.parametrize("flags", [2, 3, -1, 1 << 30])
def test_unknown_flags_are_refused(B, flags):  # noqa: F811
    assert B.load_library().blt_kv8_attend(_cache(B), _attn(B, flags=flags), None) == B.BLT_ERR_INVALID_ARG
    assert b"flags" in B.load_library().blt_kv8_last_error()


class OnGpu(torch.Tensor):
    """A CPU tensor that says it lies on a GPU: the binding looks at tensors, it does not touch them."""

    gpu = 0
    is_cuda = True

    @property
    def device(self):
        return torch.device("cuda", self.gpu)


class OnOtherGpu(OnGpu):
    gpu = 1


def gpu(*shape, dt=torch.uint8, on=OnGpu):
    return torch.zeros(*shape, dtype=dt).as_subclass(on)


def arrays(on=OnGpu, **kw):
    i8 = torch.int8
    return {**dict(k=gpu(4, 2, 32, 64, on=on), v=gpu(4, 2, 32, 64, on=on), k_exp=gpu(4, 2, 2, on=on), v_exp=gpu(4, 2, 2, on=on),
                   page_table=gpu(1, 4, dt=torch.int32, on=on), k_min=gpu(4, 2, 64, dt=i8, on=on), k_max=gpu(4, 2, 64, dt=i8, on=on),
                   k_sexp=gpu(4, 2, on=on)), **kw}


@pytest.mark.parametrize("names", [("k", "v"), ("k_exp", "v_exp"), ("k_min", "k_max"), ("k_sexp",)])
def test_one_page_expanded_over_the_pool_is_refused(B, names):  # noqa: F811
    """A page stride of 0 means dense in the C struct: the kernels would go past the one page there is."""
    a = arrays()
    B.kv8_cache("int8", **a)
    wrong = {n: a[n][:1].expand(a[n].shape) for n in names}
    with pytest.raises(ValueError, match="expanded"):
        B.kv8_cache("int8", **{**a, **wrong})
    one = {n: t[:1] for n, t in arrays().items()}
    one["page_table"] = gpu(1, 4, dt=torch.int32)
    B.kv8_cache("int8", **one)  # a pool of one page


def descriptors(B, on):  # noqa: F811
    i32 = torch.int32
    off, one, lim = gpu(2, dt=i32, on=on), gpu(1, dt=i32, on=on), gpu(3, dt=i32, on=on)
    x, q = gpu(3, 2, 64, dt=torch.float32, on=on), gpu(3, 4, 64, dt=torch.float32, on=on)
    sp, sc = gpu(3, 2, 4, dt=i32, on=on), gpu(3, 2, dt=i32, on=on)
    rows = B.kv8_rows(x, x.clone(), off, one, 3)
    return [("append", rows), ("read", rows), ("attend", B.kv8_attention(q, q.clone(), off, lim, 3, 64, 0.125)),
            ("select", B.kv8_selection(q, off, lim, 3, 64, sp, sc))]


@pytest.mark.parametrize("i", range(4))
def test_arguments_on_another_device_than_the_cache_are_refused(B, i):  # noqa: F811
    cache = B.kv8_cache("int8", **arrays())
    name, args = descriptors(B, OnOtherGpu)[i]
    with pytest.raises(ValueError, match="cuda:1"):
        getattr(B, "blt_kv8_" + name)(cache, args)


@pytest.mark.skipif(torch.cuda.is_available(), reason="the tensors only say that they lie on a GPU")
@pytest.mark.parametrize("i", range(4))
def test_arguments_on_the_same_device_reach_the_library(B, i):  # noqa: F811
    cache = B.kv8_cache("int8", **arrays())
    name, args = descriptors(B, OnGpu)[i]
    with pytest.raises(B.BltError):  # no GPU here
        getattr(B, "blt_kv8_" + name)(cache, args)


def test_threads_have_messages_of_their_own(B):  # noqa: F811
    import threading

    lib, seen = B.load_library(), {}

    def work(i):
        for _ in range(200):
            assert lib.blt_kv8_attend(_cache(B), _attn(B, dtype=10 + i), None) == B.BLT_ERR_INVALID_ARG
            seen.setdefault(i, set()).add(lib.blt_kv8_last_error())

    threads = [threading.Thread(target=work, args=(i,)) for i in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert seen == {i: {b"dtype %d" % (10 + i)} for i in range(8)}


@pytest.mark.parametrize("kw", [dict(out_row_stride=0), dict(out_row_stride=32), dict(out_head_stride=0), dict(out_head_stride=63)],
                         ids=lambda kw: ",".join(f"{k}={v}" for k, v in kw.items()))
def test_rows_of_out_that_share_elements_are_refused(B, kw):  # noqa: F811
    """An expanded out: every row would be written to one place, in no order."""
    lib = B.load_library()
    assert lib.blt_kv8_attend(_cache(B), _attn(B, **kw), None) == B.BLT_ERR_INVALID_ARG
    assert b"overlap" in lib.blt_kv8_last_error()


def test_rows_to_be_read_into_that_share_elements_are_refused(B):  # noqa: F811
    lib = B.load_library()
    for kw in (dict(row_stride=0), dict(head_stride=0), dict(head_stride=63), dict(row_stride=63)):
        assert lib.blt_kv8_read(_cache(B), _rows(B, **kw), None) == B.BLT_ERR_INVALID_ARG, kw
        assert b"overlap" in lib.blt_kv8_last_error()


def share(rows, rs, heads, hs, dim):
    at = sorted(i * rs + j * hs for i in range(rows) for j in range(heads))
    return any(b - a < dim for a, b in zip(at, at[1:]))


def test_rows_and_heads_that_share_elements_are_refused_and_no_others(B):  # noqa: F811
    """Strides that are each wide enough, and rows that meet other rows' heads all the same; interleaved ones that do not."""
    lib = B.load_library()
    seen = {True: 0, False: 0}
    for rows, heads in ((1, 2), (2, 2), (3, 2), (5, 4), (4, 8), (7, 6)):
        for rs in (64, 96, 128, 160, 191, 192, 193, 256, 320, 384, 448, 512):
            for hs in (64, 65, 96, 127, 128, 192, 200, 256, 448, 512):
                want = share(rows, rs, heads, hs, 64)
                lib.blt_kv8_attend(_cache(B), _attn(B, n_rows=rows, max_rows=rows, n_q_heads=heads, out_row_stride=rs, out_head_stride=hs), None)
                assert (b"overlap" in lib.blt_kv8_last_error()) == want, (rows, rs, heads, hs)
                seen[want] += 1
    assert min(seen.values()) > 50
