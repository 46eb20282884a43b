"""ctypes binding of the bltdec C ABI (include/bltdec.h, include/bltkv8.h): argument marshalling only.

Every function keeps the C name and signature; device pointers are passed as
torch CUDA tensors (or raw integers), host arrays as sequences of ints.  No
decoder arithmetic happens here.  The library must exist: there is no
fallback, and loading fails loudly when it is missing.
"""

from __future__ import annotations

import ctypes as C
import os
from typing import Optional, Sequence

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libbltdec.so")

BLT_OK = 0
BLT_ERR_INVALID_ARG = -1
BLT_ERR_NO_SPACE = -2
BLT_ERR_STATE = -3
BLT_ERR_CUDA = -4
BLT_ERR_STEP_LIMIT = -5
BLT_ERR_DEVICE = -6
BLT_W_F32 = 0
BLT_W_BF16 = 1
BLT_DRAFT_AR = 0
BLT_DRAFT_DIFFUSION = 1
BLT_FLAG_TIME_PASSES = 1
BLT_FLAG_PERSISTENT = 2
BLT_FLAG_TEST_STALL = 4  # test only: the persistent kernel's bounded waits must run out
BLT_FLAG_TENSOR_CORES = 8  # passes of >= 128 rows: projections on the tcgen05 GEMM
BLT_FLAG_KV8_INT8 = 16  # KV cache in 8 bits: int8 codes,
BLT_FLAG_KV8_E4M3 = 32  # or e4m3 codes
BLT_UNMASK_CONFIDENCE = 0
BLT_UNMASK_EB = 1
BLT_KV8_INT8 = 0
BLT_KV8_E4M3 = 1
BLT_KV8_TEST_STALL = 1  # test only: waits of blt_kv8_attend run out
BLT_T_F32 = 0
BLT_T_BF16 = 1
BLT_T_F16 = 2
BLT_LAYER_NT = 12
LAYER_ORDER = ("wq_c", "wk_c", "wv_c", "wo_c", "norm_c", "attn_norm", "wqkv", "wo", "ffn_norm", "w1", "w3", "w2")

EXPORTS = (
    "blt_dec_init",
    "blt_dec_prefill",
    "blt_dec_prefill_noalloc",
    "blt_dec_diffuse_block",
    "blt_dec_diffuse_block_eb",
    "blt_dec_draft",
    "blt_dec_verify_accept",
    "blt_dec_diffuse_block_sampled",
    "blt_dec_draft_sampled",
    "blt_dec_verify_sampled",
    "blt_dec_rewind",
    "blt_dec_stats",
    "blt_dec_upload",
    "blt_dec_download",
    "blt_dec_sync",
    "blt_dec_last_error",
    "blt_dec_free",
    "blt_kv8_append",
    "blt_kv8_read",
    "blt_kv8_attend",
    "blt_kv8_select",
    "blt_kv8_last_error",
)


class blt_dec_config(C.Structure):
    _fields_ = [
        ("n_layers", C.c_int32),
        ("d_model", C.c_int32),
        ("n_heads", C.c_int32),
        ("d_ffn", C.c_int32),
        ("d_global", C.c_int32),
        ("vocab", C.c_int32),
        ("weight_dtype", C.c_int32),
        ("rope_theta", C.c_float),
        ("norm_eps", C.c_float),
        ("max_batch", C.c_int32),
        ("max_ctx", C.c_int32),
        ("max_latents", C.c_int32),
        ("max_rows", C.c_int32),
        ("max_block", C.c_int32),
        ("page_tokens", C.c_int32),
        ("kv_pages", C.c_int32),
        ("attn_chunk", C.c_int32),
        ("flags", C.c_int32),
    ]


class blt_dec_weights(C.Structure):
    _fields_ = [
        ("embed", C.c_void_p),
        ("head", C.c_void_p),
        ("final_norm", C.c_void_p),
        ("layer", C.POINTER(C.c_void_p)),
    ]


class blt_rows_in(C.Structure):
    _fields_ = [
        ("bytes", C.c_void_p),
        ("row_latent", C.c_void_p),
        ("row_offsets", C.POINTER(C.c_int32)),
        ("new_latents", C.c_void_p),
        ("latent_offsets", C.POINTER(C.c_int32)),
    ]


class blt_sampling(C.Structure):
    _fields_ = [("temperature", C.c_float), ("top_p", C.c_float), ("uniforms", C.c_void_p)]


class blt_dec_counters(C.Structure):
    _fields_ = [
        ("passes", C.c_uint64),
        ("rows", C.c_uint64),
        ("prefill_rows", C.c_uint64),
        ("latents", C.c_uint64),
        ("calls", C.c_uint64),
        ("weight_bytes", C.c_uint64),
        ("kv_read_bytes", C.c_uint64),
        ("kernel_launches", C.c_uint64),
        ("timed_passes", C.c_uint64),
        ("pass_ns", C.c_uint64),
        ("persistent_calls", C.c_uint64),
        ("prefill_kv_read_bytes", C.c_uint64),
        ("tc_gemms", C.c_uint64),
    ]

    def as_dict(self):
        return {k: int(getattr(self, k)) for k, _ in self._fields_}


class blt_kv8_cache(C.Structure):
    _fields_ = [
        ("format", C.c_int32),
        ("n_heads", C.c_int32),
        ("head_dim", C.c_int32),
        ("page_tokens", C.c_int32),
        ("n_pages", C.c_int32),
        ("batch", C.c_int32),
        ("max_pages", C.c_int32),
        ("reserved", C.c_int32),
        ("k", C.c_void_p),
        ("v", C.c_void_p),
        ("k_exp", C.c_void_p),
        ("v_exp", C.c_void_p),
        ("page_stride", C.c_int64),
        ("exp_stride", C.c_int64),
        ("k_min", C.c_void_p),
        ("k_max", C.c_void_p),
        ("k_sexp", C.c_void_p),
        ("sum_stride", C.c_int64),
        ("sexp_stride", C.c_int64),
        ("page_table", C.c_void_p),
        ("status", C.c_void_p),
    ]


class blt_kv8_rows(C.Structure):
    fits = None  # the cache these arguments were found to fit
    _fields_ = [
        ("k", C.c_void_p),
        ("v", C.c_void_p),
        ("dtype", C.c_int32),
        ("n_rows", C.c_int32),
        ("max_rows", C.c_int32),
        ("reserved", C.c_int32),
        ("row_stride", C.c_int64),
        ("head_stride", C.c_int64),
        ("row_offsets", C.c_void_p),
        ("start", C.c_void_p),
    ]


class blt_kv8_attention(C.Structure):
    fits = None  # the cache these arguments were found to fit
    _fields_ = [
        ("q", C.c_void_p),
        ("out", C.c_void_p),
        ("lse", C.c_void_p),
        ("dtype", C.c_int32),
        ("n_q_heads", C.c_int32),
        ("n_rows", C.c_int32),
        ("max_rows", C.c_int32),
        ("max_keys", C.c_int32),
        ("scale", C.c_float),
        ("q_row_stride", C.c_int64),
        ("q_head_stride", C.c_int64),
        ("out_row_stride", C.c_int64),
        ("out_head_stride", C.c_int64),
        ("row_offsets", C.c_void_p),
        ("row_limit", C.c_void_p),
        ("sel_pages", C.c_void_p),
        ("sel_count", C.c_void_p),
        ("n_select", C.c_int32),
        ("flags", C.c_int32),
    ]


class blt_kv8_selection(C.Structure):
    fits = None  # the cache these arguments were found to fit
    _fields_ = [
        ("q", C.c_void_p),
        ("dtype", C.c_int32),
        ("n_q_heads", C.c_int32),
        ("n_rows", C.c_int32),
        ("max_rows", C.c_int32),
        ("max_keys", C.c_int32),
        ("n_select", C.c_int32),
        ("n_sink", C.c_int32),
        ("n_local", C.c_int32),
        ("q_row_stride", C.c_int64),
        ("q_head_stride", C.c_int64),
        ("row_offsets", C.c_void_p),
        ("row_limit", C.c_void_p),
        ("sel_pages", C.c_void_p),
        ("sel_count", C.c_void_p),
    ]


_lib = None


def load_library(path: str = LIB_PATH) -> C.CDLL:
    """Load libbltdec.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"bltdec engine library not built: {path} (run block_diffusion_byte_b200._build.build())")
    lib = C.CDLL(path)
    P, I, F, V = C.c_void_p, C.c_int, C.c_float, None
    lib.blt_dec_init.argtypes = [C.POINTER(blt_dec_config), C.POINTER(blt_dec_weights), P, C.POINTER(P)]
    lib.blt_dec_prefill.argtypes = [P, I, C.POINTER(blt_rows_in), P]
    lib.blt_dec_prefill_noalloc.argtypes = [P, I, C.POINTER(blt_rows_in), P]
    lib.blt_dec_diffuse_block.argtypes = [P, I, C.POINTER(blt_rows_in), I, F, I, P, P, P]
    lib.blt_dec_diffuse_block_eb.argtypes = [P, I, C.POINTER(blt_rows_in), I, F, I, P, P, P]
    lib.blt_dec_draft.argtypes = [P, I, C.POINTER(blt_rows_in), I, I, F, I, P, P]
    lib.blt_dec_verify_accept.argtypes = [P, P, P, C.POINTER(C.c_int32), P, P, P]
    SP = C.POINTER(blt_sampling)
    lib.blt_dec_diffuse_block_sampled.argtypes = [P, I, C.POINTER(blt_rows_in), I, F, I, I, SP, P, P, P]
    lib.blt_dec_draft_sampled.argtypes = [P, I, C.POINTER(blt_rows_in), I, I, F, I, SP, P, P]
    lib.blt_dec_verify_sampled.argtypes = [P, P, P, C.POINTER(C.c_int32), SP, P, P, P]
    lib.blt_dec_rewind.argtypes = [P, I, C.POINTER(C.c_int32), C.POINTER(C.c_int32)]
    lib.blt_dec_stats.argtypes = [P, C.POINTER(blt_dec_counters)]
    lib.blt_dec_upload.argtypes = [P, P, P, C.c_size_t]
    lib.blt_dec_download.argtypes = [P, P, P, C.c_size_t]
    lib.blt_dec_sync.argtypes = [P]
    lib.blt_dec_last_error.argtypes = [P]
    lib.blt_dec_last_error.restype = C.c_char_p
    lib.blt_dec_free.argtypes = [P]
    lib.blt_dec_free.restype = V
    KP = C.POINTER(blt_kv8_cache)
    lib.blt_kv8_append.argtypes = [KP, C.POINTER(blt_kv8_rows), P]
    lib.blt_kv8_read.argtypes = [KP, C.POINTER(blt_kv8_rows), P]
    lib.blt_kv8_attend.argtypes = [KP, C.POINTER(blt_kv8_attention), P]
    lib.blt_kv8_select.argtypes = [KP, C.POINTER(blt_kv8_selection), P]
    lib.blt_kv8_last_error.argtypes = []
    lib.blt_kv8_last_error.restype = C.c_char_p
    for name in EXPORTS:
        if name not in ("blt_dec_last_error", "blt_dec_free", "blt_kv8_last_error"):
            getattr(lib, name).restype = C.c_int
    _lib = lib
    return lib


class BltError(RuntimeError):
    def __init__(self, code: int, where: str, msg: str):
        super().__init__(f"{where} -> {code}: {msg}")
        self.code = code


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


def _i32(seq: Optional[Sequence[int]]):
    if seq is None:
        return None
    arr = (C.c_int32 * len(seq))(*[int(v) for v in seq])
    return arr


def _check(h, rc: int, where: str) -> None:
    if rc != BLT_OK:
        msg = load_library().blt_dec_last_error(h).decode() if h else ""
        raise BltError(rc, where, msg)


def rows_in(bytes_dev=None, row_latent_dev=None, row_offsets=None, new_latents_dev=None, latent_offsets=None):
    """Build a blt_rows_in; returns (struct, keepalive)."""
    ro = _i32(row_offsets)
    lo = _i32(latent_offsets)
    r = blt_rows_in(_ptr(bytes_dev), _ptr(row_latent_dev), ro, _ptr(new_latents_dev), lo)
    return r, (ro, lo, bytes_dev, row_latent_dev, new_latents_dev)


# ----------------------------------------------------------------------------- thin wrappers, C names
def blt_dec_init(cfg: blt_dec_config, embed, head, final_norm, layers, stream: Optional[int] = None) -> int:
    """``embed``, ``head``, ``final_norm``: float32 C-contiguous numpy arrays;
    ``layers``: per layer a list of BLT_LAYER_NT arrays (or None for unused ones)."""
    lib = load_library()
    keep = [embed, head, final_norm]
    ptrs = (C.c_void_p * (len(layers) * BLT_LAYER_NT))()
    for l, tensors in enumerate(layers):
        for t, arr in enumerate(tensors):
            if arr is not None:
                keep.append(arr)
                ptrs[l * BLT_LAYER_NT + t] = arr.ctypes.data
    w = blt_dec_weights(embed.ctypes.data, head.ctypes.data, final_norm.ctypes.data, ptrs)
    out = C.c_void_p()
    rc = lib.blt_dec_init(C.byref(cfg), C.byref(w), stream, C.byref(out))
    if rc != BLT_OK:
        raise BltError(rc, "blt_dec_init", "see stderr")
    return out.value


def blt_dec_prefill(h: int, batch: int, rows: blt_rows_in, out_logits=None) -> None:
    _check(h, load_library().blt_dec_prefill(h, batch, C.byref(rows), _ptr(out_logits)), "blt_dec_prefill")


def blt_dec_prefill_noalloc(h: int, batch: int, rows: blt_rows_in, out_logits=None) -> None:
    _check(h, load_library().blt_dec_prefill_noalloc(h, batch, C.byref(rows), _ptr(out_logits)), "blt_dec_prefill_noalloc")


def blt_dec_diffuse_block(h, batch, pending, k, alpha, max_steps, out_block, out_steps=None, out_logits=None) -> None:
    rc = load_library().blt_dec_diffuse_block(
        h, batch, C.byref(pending), k, float(alpha), max_steps, _ptr(out_block), _ptr(out_steps), _ptr(out_logits)
    )
    _check(h, rc, "blt_dec_diffuse_block")


def blt_dec_diffuse_block_eb(h, batch, pending, k, gamma, max_steps, out_block, out_steps=None, out_logits=None) -> None:
    rc = load_library().blt_dec_diffuse_block_eb(
        h, batch, C.byref(pending), k, float(gamma), max_steps, _ptr(out_block), _ptr(out_steps), _ptr(out_logits)
    )
    _check(h, rc, "blt_dec_diffuse_block_eb")


def blt_dec_draft(h, batch, pending, mode, k, alpha, max_steps, out_draft, out_logits=None) -> None:
    rc = load_library().blt_dec_draft(h, batch, C.byref(pending), mode, k, float(alpha), max_steps, _ptr(out_draft), _ptr(out_logits))
    _check(h, rc, "blt_dec_draft")


def blt_dec_verify_accept(h, draft_row_latent, new_latents, latent_offsets, out_accepted, out_next, out_logits=None) -> None:
    lo = _i32(latent_offsets)
    rc = load_library().blt_dec_verify_accept(
        h, _ptr(draft_row_latent), _ptr(new_latents), lo, _ptr(out_accepted), _ptr(out_next), _ptr(out_logits)
    )
    _check(h, rc, "blt_dec_verify_accept")


def sampling(temperature: float, top_p: float, uniforms_dev) -> blt_sampling:
    """Sampling parameters; uniforms_dev: device float32 [batch][2 k + 1] in [0, 1)."""
    return blt_sampling(float(temperature), float(top_p), _ptr(uniforms_dev))


def blt_dec_diffuse_block_sampled(h, batch, pending, k, threshold, unmask, max_steps, samp, out_block, out_steps=None,
                                  out_logits=None) -> None:
    rc = load_library().blt_dec_diffuse_block_sampled(h, batch, C.byref(pending), k, float(threshold), unmask, max_steps,
                                                      C.byref(samp), _ptr(out_block), _ptr(out_steps), _ptr(out_logits))
    _check(h, rc, "blt_dec_diffuse_block_sampled")


def blt_dec_draft_sampled(h, batch, pending, mode, k, alpha, max_steps, samp, out_draft, out_logits=None) -> None:
    rc = load_library().blt_dec_draft_sampled(h, batch, C.byref(pending), mode, k, float(alpha), max_steps, C.byref(samp),
                                              _ptr(out_draft), _ptr(out_logits))
    _check(h, rc, "blt_dec_draft_sampled")


def blt_dec_verify_sampled(h, draft_row_latent, new_latents, latent_offsets, samp, out_accepted, out_next, out_logits=None) -> None:
    lo = _i32(latent_offsets)
    rc = load_library().blt_dec_verify_sampled(h, _ptr(draft_row_latent), _ptr(new_latents), lo, C.byref(samp),
                                               _ptr(out_accepted), _ptr(out_next), _ptr(out_logits))
    _check(h, rc, "blt_dec_verify_sampled")


def blt_dec_rewind(h, batch, kv_len=None, n_latents=None) -> None:
    _check(h, load_library().blt_dec_rewind(h, batch, _i32(kv_len), _i32(n_latents)), "blt_dec_rewind")


def blt_dec_stats(h) -> dict:
    c = blt_dec_counters()
    _check(h, load_library().blt_dec_stats(h, C.byref(c)), "blt_dec_stats")
    return c.as_dict()


def blt_dec_upload(h, dst_device, src_host: int, n: int) -> None:
    """Host -> device copy of n bytes on the handle's stream (src_host: an address; reusable at once)."""
    _check(h, load_library().blt_dec_upload(h, _ptr(dst_device), src_host, n), "blt_dec_upload")


def blt_dec_download(h, dst_host: int, src_device, n: int) -> None:
    """Device -> host copy of n bytes after the handle's queued work (dst_host: an address)."""
    _check(h, load_library().blt_dec_download(h, dst_host, _ptr(src_device), n), "blt_dec_download")


def blt_dec_sync(h) -> int:
    """Returns the device status (0, BLT_ERR_STEP_LIMIT or BLT_ERR_DEVICE)."""
    rc = load_library().blt_dec_sync(h)
    if rc == BLT_ERR_CUDA:
        _check(h, rc, "blt_dec_sync")
    return rc


def blt_dec_last_error(h) -> str:
    return load_library().blt_dec_last_error(h).decode()


def blt_dec_free(h) -> None:
    if h:
        load_library().blt_dec_free(h)


# ----------------------------------------------------------------------------- 8-bit KV cache (bltkv8.h)
_KV8_FORMAT = {"int8": BLT_KV8_INT8, "e4m3": BLT_KV8_E4M3, BLT_KV8_INT8: BLT_KV8_INT8, BLT_KV8_E4M3: BLT_KV8_E4M3}
_TYPES = {"torch.float32": BLT_T_F32, "torch.bfloat16": BLT_T_BF16, "torch.float16": BLT_T_F16}


def _kv8_type(t) -> int:
    try:
        return _TYPES[str(t.dtype)]
    except KeyError:
        raise ValueError(f"dtype {t.dtype}: float32, bfloat16 or float16 is wanted") from None


def _want(t, name: str, dtype: str, ndim: int, device=None):
    """`t` as an argument: a CUDA tensor of the type and rank, dense in its last axis."""
    if t.dim() != ndim or str(t.dtype) not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise ValueError(f"{name}: {ndim} axes of {dtype} are wanted, got {t.dim()} of {t.dtype}")
    if not t.is_cuda or (device is not None and t.device != device):
        raise ValueError(f"{name}: a tensor on {device or 'a CUDA device'} is wanted, got {t.device}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name}: the last axis has stride {t.stride(-1)}")
    return t


def _dense_from(t, name: str, axis: int):
    """Raises unless the axes from `axis` on are contiguous."""
    n = 1
    for i in reversed(range(axis, t.dim())):
        if t.shape[i] > 1 and t.stride(i) != n:
            raise ValueError(f"{name}: axes from {axis} on have to be contiguous, strides are {tuple(t.stride())}")
        n *= t.shape[i]
    return t


def kv8_cache(format, k, v, k_exp, v_exp, page_table, k_min=None, k_max=None, k_sexp=None, status=None) -> blt_kv8_cache:
    """Describe an 8-bit paged KV cache held in torch tensors.

    format ``"int8"`` or ``"e4m3"``; ``k``, ``v`` uint8 [n_pages, n_heads, page_tokens, head_dim]; ``k_exp``, ``v_exp`` uint8
    [n_pages, n_heads, page_tokens / 16]; ``page_table`` int32 [batch, max_pages], contiguous; for
    :func:`blt_kv8_select` also ``k_min``, ``k_max`` int8 [n_pages, n_heads, head_dim] and ``k_sexp`` uint8
    [n_pages, n_heads]; ``status`` int32 [1].  The first axis may be strided (a layer's part of a larger
    pool).  The struct keeps the tensors alive."""
    if format not in _KV8_FORMAT:
        raise ValueError(f"format {format!r}: 'int8' or 'e4m3' is wanted")
    dev = k.device
    _want(k, "k", "torch.uint8", 4)
    n, h, pt, d = k.shape
    for t, name, dtype, shape in ((v, "v", "torch.uint8", (n, h, pt, d)), (k_exp, "k_exp", "torch.uint8", (n, h, pt // 16)),
                                  (v_exp, "v_exp", "torch.uint8", (n, h, pt // 16)), (k_min, "k_min", "torch.int8", (n, h, d)),
                                  (k_max, "k_max", "torch.int8", (n, h, d)), (k_sexp, "k_sexp", "torch.uint8", (n, h))):
        if t is not None and tuple(_want(t, name, dtype, len(shape), dev).shape) != shape:
            raise ValueError(f"{name}: shape {shape} is wanted, got {tuple(t.shape)}")
    for t, name in ((k, "k"), (v, "v"), (k_exp, "k_exp"), (v_exp, "v_exp"), (k_min, "k_min"), (k_max, "k_max"), (k_sexp, "k_sexp")):
        if t is not None:
            _dense_from(t, name, 1)
            if n > 1 and t.stride(0) == 0:  # 0 means dense to the library
                raise ValueError(f"{name}: one page expanded over {n} (a page stride of 0)")
    for a, b, name in ((k, v, "k and v"), (k_exp, v_exp, "k_exp and v_exp"), (k_min, k_max, "k_min and k_max")):
        if a is not None and b is not None and n > 1 and a.stride(0) != b.stride(0):
            raise ValueError(f"{name}: page strides differ")
    _dense_from(_want(page_table, "page_table", "torch.int32", 2, dev), "page_table", 0)
    if status is not None:
        _want(status, "status", "torch.int32", 1, dev)
    stride = lambda t: 0 if t is None or n == 1 else t.stride(0)  # noqa: E731
    c = blt_kv8_cache(_KV8_FORMAT[format], h, d, pt, n, page_table.shape[0], page_table.shape[1], 0, _ptr(k), _ptr(v), _ptr(k_exp),
                      _ptr(v_exp), stride(k), stride(k_exp), _ptr(k_min), _ptr(k_max), _ptr(k_sexp), stride(k_min), stride(k_sexp),
                      _ptr(page_table), _ptr(status))
    c.keep = (k, v, k_exp, v_exp, page_table, k_min, k_max, k_sexp, status)
    c.device = dev
    return c


def kv8_rows(k, v, row_offsets, start, max_rows: int) -> blt_kv8_rows:
    """Rows of keys and values: ``k``, ``v`` [n_rows, n_heads, head_dim] float32, bfloat16 or float16 with equal
    strides; ``row_offsets`` int32 [batch + 1]; ``start`` int32 [batch]; ``max_rows``: most rows of one sequence."""
    types = tuple(_TYPES)
    _want(k, "k", types, 3)
    _want(v, "v", types, 3, k.device)
    if v.dtype != k.dtype or v.shape != k.shape or v.stride() != k.stride():
        raise ValueError("k and v differ in type, shape or strides")
    _want(row_offsets, "row_offsets", "torch.int32", 1, k.device)
    _want(start, "start", "torch.int32", 1, k.device)
    if row_offsets.shape[0] != start.shape[0] + 1:
        raise ValueError(f"row_offsets has {row_offsets.shape[0]} entries for {start.shape[0]} sequences")
    r = blt_kv8_rows(_ptr(k), _ptr(v), _kv8_type(k), k.shape[0], int(max_rows), 0, k.stride(0), k.stride(1), _ptr(row_offsets), _ptr(start))
    r.keep = (k, v, row_offsets, start)
    r.shape, r.device = (start.shape[0], k.shape[1], k.shape[2]), k.device
    return r


def _kv8_q(q, row_offsets, row_limit):
    _want(q, "q", tuple(_TYPES), 3)
    _want(row_offsets, "row_offsets", "torch.int32", 1, q.device)
    _want(row_limit, "row_limit", "torch.int32", 1, q.device)
    if row_limit.shape[0] != q.shape[0]:
        raise ValueError(f"row_limit has {row_limit.shape[0]} entries for {q.shape[0]} rows")


def _kv8_sel(sel_pages, sel_count, q):
    _dense_from(_want(sel_pages, "sel_pages", "torch.int32", 3, q.device), "sel_pages", 0)
    _dense_from(_want(sel_count, "sel_count", "torch.int32", 2, q.device), "sel_count", 0)
    if sel_pages.shape[:2] != sel_count.shape or sel_count.shape[0] != q.shape[0]:
        raise ValueError(f"sel_pages {tuple(sel_pages.shape)} and sel_count {tuple(sel_count.shape)} for {q.shape[0]} rows")


def kv8_attention(q, out, row_offsets, row_limit, max_rows: int, max_keys: int, scale: float, lse=None, sel_pages=None,
                  sel_count=None) -> blt_kv8_attention:
    """Attention of rows ``q`` [n_rows, n_q_heads, head_dim] into ``out`` (same type and shape): ``row_offsets`` int32
    [batch + 1], ``row_limit`` int32 [n_rows]; ``max_rows``: most rows of one sequence, ``max_keys``: expected largest limit;
    ``lse`` float32 [n_rows, n_q_heads]; ``sel_pages`` int32 [n_rows, n_heads, n_select] and ``sel_count`` int32
    [n_rows, n_heads] limit the rows to pages (see :func:`blt_kv8_select`)."""
    _kv8_q(q, row_offsets, row_limit)
    _want(out, "out", str(q.dtype), 3, q.device)
    if out.shape != q.shape:
        raise ValueError(f"out has shape {tuple(out.shape)}, q {tuple(q.shape)}")
    if lse is not None and tuple(_dense_from(_want(lse, "lse", "torch.float32", 2, q.device), "lse", 0).shape) != tuple(q.shape[:2]):
        raise ValueError(f"lse has shape {tuple(lse.shape)}")
    if (sel_pages is None) != (sel_count is None):
        raise ValueError("sel_pages and sel_count come together")
    n_select = 0
    if sel_pages is not None:
        _kv8_sel(sel_pages, sel_count, q)
        n_select = sel_pages.shape[2]
    a = blt_kv8_attention(_ptr(q), _ptr(out), _ptr(lse), _kv8_type(q), q.shape[1], q.shape[0], int(max_rows), int(max_keys), float(scale),
                          q.stride(0), q.stride(1), out.stride(0), out.stride(1), _ptr(row_offsets), _ptr(row_limit), _ptr(sel_pages),
                          _ptr(sel_count), n_select, 0)
    a.keep = (q, out, row_offsets, row_limit, lse, sel_pages, sel_count)
    a.shape, a.device = (row_offsets.shape[0] - 1, None if sel_pages is None else sel_pages.shape[1], q.shape[2]), q.device
    return a


def kv8_selection(q, row_offsets, row_limit, max_rows: int, max_keys: int, sel_pages, sel_count, n_sink: int = 0,
                  n_local: int = 0) -> blt_kv8_selection:
    """Choice of pages for rows ``q`` into ``sel_pages`` int32 [n_rows, n_heads, n_select] and ``sel_count`` int32 [n_rows, n_heads]."""
    _kv8_q(q, row_offsets, row_limit)
    _kv8_sel(sel_pages, sel_count, q)
    s = blt_kv8_selection(_ptr(q), _kv8_type(q), q.shape[1], q.shape[0], int(max_rows), int(max_keys), sel_pages.shape[2], int(n_sink),
                          int(n_local), q.stride(0), q.stride(1), _ptr(row_offsets), _ptr(row_limit), _ptr(sel_pages), _ptr(sel_count))
    s.keep = (q, row_offsets, row_limit, sel_pages, sel_count)
    s.shape, s.device = (row_offsets.shape[0] - 1, sel_pages.shape[1], q.shape[2]), q.device
    return s


def _kv8_call(name: str, cache: blt_kv8_cache, args, stream) -> None:
    if args.fits is not cache:  # looked at once for each pair of descriptors
        batch, heads, dim = args.shape
        if batch != cache.batch or dim != cache.head_dim or heads not in (None, cache.n_heads):
            raise ValueError(f"{name}: arguments for {batch} sequences, {heads} heads of {dim}; the cache has {cache.batch}, {cache.n_heads} of {cache.head_dim}")
        if args.device != cache.device:
            raise ValueError(f"{name}: arguments on {args.device}, the cache on {cache.device}")
        args.fits = cache
    rc = getattr(_lib or load_library(), name)(cache, args, stream)
    if rc != BLT_OK:
        raise BltError(rc, name, _lib.blt_kv8_last_error().decode())


def blt_kv8_append(cache: blt_kv8_cache, rows: blt_kv8_rows, stream: Optional[int] = None) -> None:
    """``stream``: a cudaStream_t as an integer (``torch.cuda.current_stream().cuda_stream``); None or 0: the default stream."""
    _kv8_call("blt_kv8_append", cache, rows, stream)


def blt_kv8_read(cache: blt_kv8_cache, rows: blt_kv8_rows, stream: Optional[int] = None) -> None:
    _kv8_call("blt_kv8_read", cache, rows, stream)


def blt_kv8_attend(cache: blt_kv8_cache, attention: blt_kv8_attention, stream: Optional[int] = None) -> None:
    _kv8_call("blt_kv8_attend", cache, attention, stream)


def blt_kv8_select(cache: blt_kv8_cache, selection: blt_kv8_selection, stream: Optional[int] = None) -> None:
    _kv8_call("blt_kv8_select", cache, selection, stream)
