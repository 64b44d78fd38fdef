"""Python binding of libtq_gb300 (the sm_103a rotated Lloyd-Max KV-cache codec
and fused decode attention).

Argument marshalling only: every step of the codec and the attention runs in
the library's CUDA kernels.  Torch tensors supply device memory and the
current CUDA stream.  The functions carry the C names of ``include/tq.h``.
There is no CPU fallback: if the library is missing or a call fails, an
exception is raised.
"""
from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libtq_gb300.so")
CHUNK = 128

TQ_OK, TQ_ERR_INVALID_ARG, TQ_ERR_UNSUPPORTED, TQ_ERR_WORKSPACE, TQ_ERR_CUDA = range(5)

c_i32, c_i64, c_u64, c_f32, c_p = ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64, ctypes.c_float, ctypes.c_void_p


class tq_codec(ctypes.Structure):
    _fields_ = [("head_dim", c_i32), ("bits", c_i32), ("sign_seed", c_u64), ("outlier_T", c_f32),
                ("outlier_cap", c_i32), ("centroids", c_f32 * 16), ("boundaries", c_f32 * 15),
                ("sign_bits", ctypes.c_uint32 * 16), ("scale_mode", c_i32)]


class tq_evict_args(ctypes.Structure):
    _fields_ = [("n_layers", c_i32), ("batch", c_i32), ("n_kv_heads", c_i32),
                ("k_rec", c_p), ("v_rec", c_p), ("k_rec_layer_stride", c_i64),
                ("v_rec_layer_stride", c_i64), ("rec_cap", c_i32),
                ("k_tail", c_p), ("v_tail", c_p), ("tail_layer_stride", c_i64), ("tail_cap", c_i32),
                ("n_chunks", c_p), ("tail_start", c_p), ("tail_len", c_p),
                ("window", c_i32), ("margin", c_i32), ("t_q", c_i32), ("max_evict", c_i32),
                ("block_table", c_p), ("table_stride", c_i32)]


class tq_attn_args(ctypes.Structure):
    _fields_ = [("n_layers", c_i32), ("batch", c_i32), ("n_q_heads", c_i32), ("n_kv_heads", c_i32),
                ("head_dim", c_i32), ("scale", c_f32),
                ("q", c_p), ("q_layer_stride", c_i64), ("q_batch_stride", c_i64),
                ("out", c_p),
                ("k_rec", c_p), ("v_rec", c_p), ("k_rec_layer_stride", c_i64),
                ("v_rec_layer_stride", c_i64), ("rec_cap", c_i32),
                ("k_tail", c_p), ("v_tail", c_p), ("tail_layer_stride", c_i64), ("tail_cap", c_i32),
                ("n_chunks", c_p), ("tail_start", c_p), ("tail_len", c_p),
                ("max_chunks", c_i32), ("max_tail", c_i32), ("splits", c_i32), ("cuda_core_path", c_i32),
                ("softcap", c_f32), ("block_table", c_p), ("table_stride", c_i32), ("sparse_v_eps", c_f32)]


class tq_attn_plan(ctypes.Structure):
    _fields_ = [("compressed_kernel", c_i32), ("dense_kernel", c_i32), ("compressed_splits", c_i32),
                ("dense_splits", c_i32), ("records_per_split", c_i32), ("dense_tokens_per_split", c_i32),
                ("heads_per_cta", c_i32), ("dense_heads_per_cta", c_i32), ("launches", c_i32),
                ("warps_per_cta", c_i32), ("workspace_bytes", c_u64)]


class tq_append_args(ctypes.Structure):
    _fields_ = [("n_layers", c_i32), ("batch", c_i32), ("t_q", c_i32), ("n_q_heads", c_i32), ("n_kv_heads", c_i32),
                ("head_dim", c_i32), ("q", c_p), ("k", c_p), ("v", c_p),
                ("q_layer_stride", c_i64), ("q_batch_stride", c_i64), ("q_token_stride", c_i64),
                ("kv_layer_stride", c_i64), ("kv_batch_stride", c_i64), ("kv_token_stride", c_i64),
                ("q_out", c_p), ("q_out_layer_stride", c_i64), ("q_out_batch_stride", c_i64),
                ("q_out_token_stride", c_i64),
                ("q_lens", c_p), ("positions", c_p), ("n_axes", c_i32), ("rot_start", c_i32), ("rot_dim", c_i32),
                ("pair_adjacent", c_i32), ("inv_freq", c_p), ("pair_axis", ctypes.c_uint8 * 256),
                ("rot_scale", c_f32),
                ("k_tail", c_p), ("v_tail", c_p), ("tail_layer_stride", c_i64), ("tail_cap", c_i32),
                ("tail_start", c_p), ("tail_len", c_p), ("tail_len_out", c_p),
                ("mass", c_p), ("mass_layer_stride", c_i64), ("mass_cap", c_i32), ("n_chunks", c_p)]


class tq_query_args(ctypes.Structure):
    _fields_ = [("n_layers", c_i32), ("batch", c_i32), ("t_q", c_i32), ("n_q_heads", c_i32), ("n_kv_heads", c_i32),
                ("head_dim", c_i32), ("scale", c_f32), ("softcap", c_f32), ("causal", c_i32),
                ("q", c_p), ("q_layer_stride", c_i64), ("q_batch_stride", c_i64), ("q_token_stride", c_i64),
                ("out", c_p), ("out_layer_stride", c_i64), ("out_batch_stride", c_i64), ("out_token_stride", c_i64),
                ("q_lens", c_p),
                ("k_rec", c_p), ("v_rec", c_p), ("k_rec_layer_stride", c_i64), ("v_rec_layer_stride", c_i64),
                ("rec_cap", c_i32),
                ("k_tail", c_p), ("v_tail", c_p), ("tail_layer_stride", c_i64), ("tail_cap", c_i32),
                ("n_chunks", c_p), ("tail_start", c_p), ("tail_len", c_p),
                ("max_chunks", c_i32), ("max_tail", c_i32), ("block_table", c_p), ("table_stride", c_i32),
                ("splits", c_i32)]


class tq_evict_mass_args(ctypes.Structure):
    _fields_ = [("n_layers", c_i32), ("batch", c_i32), ("n_kv_heads", c_i32),
                ("k_rec", c_p), ("v_rec", c_p), ("k_rec_layer_stride", c_i64), ("v_rec_layer_stride", c_i64),
                ("rec_cap", c_i32), ("block_table", c_p), ("table_stride", c_i32),
                ("k_dst", c_p), ("v_dst", c_p), ("k_dst_layer_stride", c_i64), ("v_dst_layer_stride", c_i64),
                ("dst_cap", c_i32), ("dst_table", c_p), ("dst_table_stride", c_i32),
                ("mass", c_p), ("mass_dst", c_p), ("mass_layer_stride", c_i64), ("mass_dst_layer_stride", c_i64),
                ("mass_cap", c_i32), ("mass_dst_cap", c_i32),
                ("n_chunks", c_p), ("n_chunks_dst", c_p), ("tail_len", c_p),
                ("max_chunks", c_i32), ("max_tail", c_i32), ("keep_chunks", c_i32), ("sink", c_i32),
                ("recent", c_i32), ("kept", c_p)]


class tq_head_norm(ctypes.Structure):
    _fields_ = [("q_weight", c_p), ("k_weight", c_p), ("q_head_stride", c_i64), ("k_head_stride", c_i64), ("eps", c_f32)]


class tq_bounds_args(ctypes.Structure):
    _fields_ = [("n_layers", c_i32), ("batch", c_i32), ("n_kv_heads", c_i32),
                ("k_rec", c_p), ("k_rec_layer_stride", c_i64), ("rec_cap", c_i32),
                ("block_table", c_p), ("table_stride", c_i32), ("n_chunks", c_p), ("first", c_p),
                ("max_chunks", c_i32), ("max_new", c_i32), ("bounds", c_p), ("bounds_layer_stride", c_i64)]


class tq_select_args(ctypes.Structure):
    _fields_ = [("n_layers", c_i32), ("batch", c_i32), ("t_q", c_i32), ("n_q_heads", c_i32), ("n_kv_heads", c_i32),
                ("head_dim", c_i32), ("causal", c_i32), ("q", c_p), ("q_layer_stride", c_i64),
                ("q_batch_stride", c_i64), ("q_token_stride", c_i64), ("q_lens", c_p), ("bounds", c_p),
                ("bounds_layer_stride", c_i64), ("rec_cap", c_i32), ("block_table", c_p), ("table_stride", c_i32),
                ("n_chunks", c_p), ("tail_len", c_p), ("max_chunks", c_i32), ("max_tail", c_i32), ("q_block", c_i32),
                ("keep", c_i32), ("sink", c_i32), ("recent", c_i32), ("list", c_p), ("count", c_p)]


class tq_record_lists(ctypes.Structure):
    _fields_ = [("list", c_p), ("count", c_p), ("list_stride", c_i32), ("q_block", c_i32)]


ATTN_KERNELS = {0: "none", 1: "cuda_core", 2: "cuda_core_warp", 3: "mma", 4: "mma512", 5: "tcgen05"}

_SIGS = {
    "tq_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "tq_version": (ctypes.c_int, []),
    "tq_codebook_scratch_bytes": (ctypes.c_size_t, []),
    "tq_make_codebook": (ctypes.c_int, [ctypes.c_int, ctypes.c_int, c_u64, c_f32, ctypes.c_int, c_p,
                                        ctypes.c_size_t, ctypes.POINTER(tq_codec),
                                        ctypes.POINTER(ctypes.c_double), c_p]),
    "tq_record_bytes": (ctypes.c_size_t, [ctypes.POINTER(tq_codec)]),
    "tq_codec_set_centroids": (ctypes.c_int, [ctypes.POINTER(tq_codec), ctypes.POINTER(c_f32), ctypes.c_int]),
    "tq_encode": (ctypes.c_int, [ctypes.POINTER(tq_codec), c_p, c_i64, c_i64, c_i64, c_i64, c_p, c_i64,
                                 c_i64, c_p]),
    "tq_decode": (ctypes.c_int, [ctypes.POINTER(tq_codec), c_p, c_i64, c_i64, c_i64, c_i64, c_p, c_i64,
                                 c_i64, c_p]),
    "tq_evict": (ctypes.c_int, [ctypes.POINTER(tq_codec), ctypes.POINTER(tq_codec),
                                ctypes.POINTER(tq_evict_args), c_p]),
    "tq_rollback": (ctypes.c_int, [ctypes.POINTER(tq_codec), ctypes.POINTER(tq_codec),
                                   ctypes.POINTER(tq_evict_args), c_p, c_p]),
    "tq_decode_attn_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(tq_attn_args),
                                                        ctypes.POINTER(tq_codec),
                                                        ctypes.POINTER(tq_codec)]),
    "tq_decode_attn": (ctypes.c_int, [ctypes.POINTER(tq_attn_args), ctypes.POINTER(tq_codec),
                                      ctypes.POINTER(tq_codec), c_p, ctypes.c_size_t, c_p]),
    "tq_decode_attn_noalloc": (ctypes.c_int, [ctypes.POINTER(tq_attn_args), ctypes.POINTER(tq_codec),
                                              ctypes.POINTER(tq_codec), c_p]),
    "tq_decode_attn_plan": (ctypes.c_int, [ctypes.POINTER(tq_attn_args), ctypes.POINTER(tq_codec),
                                           ctypes.POINTER(tq_codec), ctypes.POINTER(tq_attn_plan)]),
    "tq_append": (ctypes.c_int, [ctypes.POINTER(tq_append_args), c_p]),
    "tq_prefill_attn_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(tq_query_args), ctypes.POINTER(tq_codec),
                                                         ctypes.POINTER(tq_codec)]),
    "tq_prefill_attn": (ctypes.c_int, [ctypes.POINTER(tq_query_args), ctypes.POINTER(tq_codec),
                                       ctypes.POINTER(tq_codec), c_p, ctypes.c_size_t, c_p]),
    "tq_attn_mass_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(tq_query_args), ctypes.POINTER(tq_codec)]),
    "tq_attn_mass": (ctypes.c_int, [ctypes.POINTER(tq_query_args), ctypes.POINTER(tq_codec), c_p, c_i64, c_i32,
                                    c_f32, c_p, ctypes.c_size_t, c_p]),
    "tq_evict_mass_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(tq_evict_mass_args), ctypes.POINTER(tq_codec),
                                                       ctypes.POINTER(tq_codec)]),
    "tq_evict_mass": (ctypes.c_int, [ctypes.POINTER(tq_evict_mass_args), ctypes.POINTER(tq_codec),
                                     ctypes.POINTER(tq_codec), c_p, ctypes.c_size_t, c_p]),
    "tq_norm_append": (ctypes.c_int, [ctypes.POINTER(tq_append_args), ctypes.POINTER(tq_head_norm), c_p]),
    "tq_key_bounds": (ctypes.c_int, [ctypes.POINTER(tq_codec), ctypes.POINTER(tq_bounds_args), c_p]),
    "tq_select_records_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(tq_select_args)]),
    "tq_select_records": (ctypes.c_int, [ctypes.POINTER(tq_select_args), c_p, ctypes.c_size_t, c_p]),
    "tq_sparse_attn_workspace_size": (ctypes.c_size_t, [ctypes.POINTER(tq_query_args), ctypes.POINTER(tq_record_lists),
                                                        ctypes.POINTER(tq_codec), ctypes.POINTER(tq_codec)]),
    "tq_sparse_attn": (ctypes.c_int, [ctypes.POINTER(tq_query_args), ctypes.POINTER(tq_record_lists),
                                      ctypes.POINTER(tq_codec), ctypes.POINTER(tq_codec), c_p, ctypes.c_size_t, c_p]),
}

NOALLOC_WORKSPACE_BYTES = 8 << 20

_lib = None


class TqError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn} failed: {status_string(status)}")


def load(path: str | None = None):
    """Load libtq_gb300.so (built by ``rotated_lloyd_max_gb300.build``)."""
    global _lib
    if _lib is None:
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise ImportError(f"{p} is missing: build it with `python -m rotated_lloyd_max_gb300.build` "
                              "(there is no CPU fallback)")
        lib = ctypes.CDLL(p)
        for name, (res, args) in _SIGS.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
    return _lib


def status_string(status: int) -> str:
    return load().tq_status_string(status).decode()


def _check(fn: str, status: int):
    if status != TQ_OK:
        raise TqError(fn, status)


_raw_stream = None  # torch's handle of the current stream by device (a Stream object costs microseconds)
_raw_device = None  # the current device's index (torch.cuda.current_device looks at torch's state first)


def _current_device() -> int:
    global _raw_device
    if _raw_device is None:
        import torch
        torch.cuda.current_device()  # CUDA is up from here on
        _raw_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    return _raw_device()


def _stream(stream):
    global _raw_stream
    if stream is None:
        if _raw_stream is None:
            import torch
            _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                                  lambda dev: torch.cuda.current_stream(dev).cuda_stream)
        return _raw_stream(_current_device())
    return stream if isinstance(stream, int) else stream.cuda_stream


def _ptr(t):
    return None if t is None else c_p(t.data_ptr())


# ---------------------------------------------------------------------------
# codec
# ---------------------------------------------------------------------------
@dataclass
class Codec:
    """A tq_codec filled by the device-side Lloyd-Max kernel."""
    c: tq_codec
    mse: float

    @property
    def head_dim(self):
        return self.c.head_dim

    @property
    def bits(self):
        return self.c.bits

    @property
    def record_bytes(self) -> int:
        return tq_record_bytes(self)

    def centroids(self):
        return list(self.c.centroids)[: 1 << self.c.bits]

    def boundaries(self):
        return list(self.c.boundaries)[: (1 << self.c.bits) - 1]

    def sign_words(self):
        return list(self.c.sign_bits)[: self.c.head_dim // 32]


def tq_make_codebook(bits: int, head_dim: int, sign_seed: int = 1, outlier_T: float = 0.0,
                     outlier_cap: int = 0, device=None, stream=None) -> Codec:
    import torch
    lib = load()
    dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    scratch = torch.empty(int(lib.tq_codebook_scratch_bytes()), dtype=torch.uint8, device=dev)
    out = tq_codec()
    mse = ctypes.c_double()
    _check("tq_make_codebook", lib.tq_make_codebook(bits, head_dim, sign_seed, float(outlier_T), outlier_cap,
                                                    _ptr(scratch), scratch.numel(), ctypes.byref(out),
                                                    ctypes.byref(mse), _stream(stream)))
    return Codec(out, mse.value)


SCALE_MODES = {"norm": 0, "matched_norm": 1, "inner_product": 2, "least_squares": 3}


def tq_codec_set_centroids(codec: Codec, centroids) -> Codec:
    """A copy of `codec` using the caller's ascending f32 table (2^bits values)."""
    vals = [float(v) for v in centroids]
    out = Codec(tq_codec.from_buffer_copy(codec.c), codec.mse)
    arr = (c_f32 * len(vals))(*vals)
    _check("tq_codec_set_centroids", load().tq_codec_set_centroids(ctypes.byref(out.c), arr, len(vals)))
    return out


def with_scale(codec: Codec, mode: str) -> Codec:
    """A copy of `codec` storing the per-vector scale `mode` (see SCALE_MODES)."""
    out = Codec(tq_codec.from_buffer_copy(codec.c), codec.mse)
    out.c.scale_mode = SCALE_MODES[mode]
    return out


def tq_record_bytes(codec: Codec) -> int:
    n = load().tq_record_bytes(ctypes.byref(codec.c))
    if n == 0:
        raise TqError("tq_record_bytes", TQ_ERR_INVALID_ARG)
    return int(n)


def _groups(t, inner: int):
    """(n_groups, n_rows, row_stride, group_stride) of a [.., rows, inner] view."""
    if t.dim() == 2:
        return 1, t.shape[0], t.stride(0), 0
    if t.dim() == 3:
        return t.shape[0], t.shape[1], t.stride(1), t.stride(0)
    raise ValueError("expected a 2-D [rows, inner] or 3-D [groups, rows, inner] tensor")


def tq_encode(codec: Codec, src, dst, first_vec: int = 0, stream=None):
    """Encode bf16 vectors src [n_vec, d] or [groups, n_vec, d] (last dim contiguous) into the
    record array dst (uint8 [n_rec, record_bytes] or [groups, n_rec, record_bytes])."""
    import torch
    assert src.dtype == torch.bfloat16 and src.stride(-1) == 1 and src.shape[-1] == codec.head_dim
    assert dst.dtype == torch.uint8 and dst.stride(-1) == 1
    g, n, vs, gs = _groups(src, codec.head_dim)
    dg = dst.stride(0) if dst.dim() == 3 else 0
    _check("tq_encode", load().tq_encode(ctypes.byref(codec.c), _ptr(src), g, n, vs, gs, _ptr(dst), dg,
                                         first_vec, _stream(stream)))


def tq_decode(codec: Codec, src, dst, first_vec: int = 0, stream=None):
    """Decode tokens [first_vec, first_vec + n) of record arrays src into f32 dst [.., n, d]."""
    import torch
    assert dst.dtype == torch.float32 and dst.stride(-1) == 1 and dst.shape[-1] == codec.head_dim
    assert src.dtype == torch.uint8
    g, n, vs, gs = _groups(dst, codec.head_dim)
    sg = src.stride(0) if src.dim() == 3 else 0
    _check("tq_decode", load().tq_decode(ctypes.byref(codec.c), _ptr(src), g, n, sg, first_vec, _ptr(dst),
                                         vs, gs, _stream(stream)))


def make_evict_args(*, k_rec, v_rec, k_tail, v_tail, n_chunks, tail_start, tail_len, window: int, margin: int,
                    t_q: int = 1, max_evict: int = 1, block_table=None) -> tq_evict_args:
    """tq_evict_args from tensors.  k_rec/v_rec: uint8 [L, B, Hkv, rec_cap, record_bytes]
    (v_rec may be k_rec for shared keys/values) or, with block_table (int32
    [B, table_stride]), per-layer pools uint8 [L, n_blocks, Hkv, record_bytes];
    k_tail/v_tail: bf16 [L, B, Hkv, tail_cap, d]; counters: int32 [L, B]."""
    if block_table is None:
        L, B, Hkv, rec_cap = k_rec.shape[:4]
        table, stride = None, 0
    else:
        L, rec_cap, Hkv = k_rec.shape[:3]
        B, stride = block_table.shape
        table = block_table.data_ptr()
    a = tq_evict_args(L, B, Hkv, k_rec.data_ptr(), v_rec.data_ptr(), k_rec.stride(0), v_rec.stride(0),
                      rec_cap, k_tail.data_ptr(), v_tail.data_ptr(), k_tail.stride(0), k_tail.shape[3],
                      n_chunks.data_ptr(), tail_start.data_ptr(), tail_len.data_ptr(), window, margin,
                      t_q, max_evict, table, stride)
    a._tensors = (k_rec, v_rec, k_tail, v_tail, n_chunks, tail_start, tail_len, block_table)
    return a


def tq_evict(k_codec: Codec, v_codec: Codec | None, *, stream=None, **kw):
    """Chunked eviction (arguments as make_evict_args; counters updated on the device)."""
    a = make_evict_args(**kw)
    vc = ctypes.byref(v_codec.c) if v_codec is not None else None
    _check("tq_evict", load().tq_evict(ctypes.byref(k_codec.c), vc, ctypes.byref(a), _stream(stream)))


def tq_rollback(k_codec: Codec, v_codec: Codec | None, new_len, *, stream=None, **kw):
    """Truncate every (layer, batch) stream to new_len (int32 [L, B], device) tokens; the
    cache as for tq_evict (window/margin/t_q are not used).  Counters and rings are
    updated on the device."""
    kw.setdefault("window", 0)
    kw.setdefault("margin", 0)
    a = make_evict_args(**kw)
    vc = ctypes.byref(v_codec.c) if v_codec is not None else None
    _check("tq_rollback", load().tq_rollback(ctypes.byref(k_codec.c), vc, ctypes.byref(a), _ptr(new_len),
                                             _stream(stream)))


def make_attn_args(*, q, out, scale: float, k_rec=None, v_rec=None, k_tail=None, v_tail=None,
                   n_chunks=None, tail_start=None, tail_len=None, max_chunks: int = 0,
                   max_tail: int = 0, splits: int = 0, n_kv_heads: int | None = None,
                   cuda_core_path: bool | int = False, softcap: float = 0.0, block_table=None,
                   sparse_v_eps: float = 0.0) -> tq_attn_args:
    """Build tq_attn_args from tensors.
    q: bf16 [L, B, Hq, d] (head and dim axes packed); out: f32 [L, B, Hq, d] contiguous;
    k_rec/v_rec: uint8 [L, B, Hkv, rec_cap, bytes], or with block_table (int32 [B, table_stride])
    per-layer pools uint8 [L, n_blocks, Hkv, bytes]; k_tail/v_tail: bf16 [L, B, Hkv, cap, d];
    counters int32 [L, B]; softcap > 0 caps each logit to softcap * tanh(logit / softcap)."""
    L, B, Hq, d = q.shape
    assert q.stride(3) == 1 and q.stride(2) == d, "query heads and dims must be packed"
    assert out.is_contiguous() and tuple(out.shape) == (L, B, Hq, d)
    src = k_rec if k_rec is not None else k_tail
    paged = block_table is not None
    Hkv = n_kv_heads if n_kv_heads is not None else (src.shape[2] if not (paged and k_rec is not None)
                                                     else k_rec.shape[2])
    a = tq_attn_args()
    a.n_layers, a.batch, a.n_q_heads, a.n_kv_heads, a.head_dim, a.scale = L, B, Hq, Hkv, d, scale
    a.q, a.q_layer_stride, a.q_batch_stride = q.data_ptr(), q.stride(0), q.stride(1)
    a.out = out.data_ptr()
    if k_rec is not None:
        a.k_rec, a.v_rec = k_rec.data_ptr(), v_rec.data_ptr()
        a.k_rec_layer_stride, a.v_rec_layer_stride = k_rec.stride(0), v_rec.stride(0)
        a.rec_cap = k_rec.shape[1] if paged else k_rec.shape[3]
    if paged:
        a.block_table, a.table_stride = block_table.data_ptr(), block_table.shape[1]
    if k_tail is not None:
        a.k_tail, a.v_tail = k_tail.data_ptr(), v_tail.data_ptr()
        a.tail_layer_stride, a.tail_cap = k_tail.stride(0), k_tail.shape[3]
    a.n_chunks = _ptr(n_chunks)
    a.tail_start = _ptr(tail_start)
    a.tail_len = _ptr(tail_len)
    a.max_chunks, a.max_tail, a.splits = max_chunks, max_tail, splits
    a.cuda_core_path = int(cuda_core_path)  # 0 automatic, 1 CUDA cores, 2 no tcgen05
    a.softcap = softcap
    a.sparse_v_eps = sparse_v_eps
    # the struct holds raw device pointers: keep the tensors alive with it
    a._tensors = (q, out, k_rec, v_rec, k_tail, v_tail, n_chunks, tail_start, tail_len, block_table)
    return a


def tq_decode_attn_plan(args: tq_attn_args, k_codec, v_codec) -> dict:
    """The kernels, split counts and launches tq_decode_attn would use (host
    only).  Codecs are Codec objects or raw tq_codec structs."""
    raw = lambda c: None if c is None else ctypes.byref(c.c if isinstance(c, Codec) else c)
    p = tq_attn_plan()
    _check("tq_decode_attn_plan", load().tq_decode_attn_plan(ctypes.byref(args), raw(k_codec), raw(v_codec),
                                                             ctypes.byref(p)))
    d = {f: getattr(p, f) for f, _ in tq_attn_plan._fields_}
    d["compressed_kernel"] = ATTN_KERNELS[d["compressed_kernel"]]
    d["dense_kernel"] = ATTN_KERNELS[d["dense_kernel"]]
    return d


def tq_decode_attn_workspace_size(args: tq_attn_args, k_codec: Codec | None, v_codec: Codec | None) -> int:
    kc = ctypes.byref(k_codec.c) if k_codec is not None else None
    vc = ctypes.byref(v_codec.c) if v_codec is not None else None
    n = load().tq_decode_attn_workspace_size(ctypes.byref(args), kc, vc)
    if n == 0:
        raise TqError("tq_decode_attn_workspace_size", TQ_ERR_INVALID_ARG)
    return int(n)


def tq_decode_attn(args: tq_attn_args, k_codec: Codec | None, v_codec: Codec | None, workspace,
                   stream=None):
    kc = ctypes.byref(k_codec.c) if k_codec is not None else None
    vc = ctypes.byref(v_codec.c) if v_codec is not None else None
    _check("tq_decode_attn", load().tq_decode_attn(ctypes.byref(args), kc, vc, _ptr(workspace),
                                                   workspace.numel() * workspace.element_size(),
                                                   _stream(stream)))


def tq_decode_attn_noalloc(args: tq_attn_args, k_codec: Codec | None, v_codec: Codec | None,
                           stream=None):
    """tq_decode_attn with the library's own fixed workspace (no allocation by
    caller or library).  Calls that overlap on the GPU share that workspace and
    race."""
    kc = ctypes.byref(k_codec.c) if k_codec is not None else None
    vc = ctypes.byref(v_codec.c) if v_codec is not None else None
    _check("tq_decode_attn_noalloc", load().tq_decode_attn_noalloc(ctypes.byref(args), kc, vc,
                                                                   _stream(stream)))


def decode_attn(*, k_codec=None, v_codec=None, workspace=None, stream=None, **kw):
    """Convenience: build the arguments, size/allocate the workspace if not given, run."""
    import torch
    a = make_attn_args(**kw)
    need = tq_decode_attn_workspace_size(a, k_codec, v_codec)
    if workspace is None or workspace.numel() < need:
        workspace = torch.empty(need, dtype=torch.uint8, device=kw["q"].device)
    tq_decode_attn(a, k_codec, v_codec, workspace, stream)
    return workspace


# ---------------------------------------------------------------------------
# several new tokens: append, prefill attention, accumulated weights, eviction
# ---------------------------------------------------------------------------
def _need(ok, why: str):
    if not ok:
        raise ValueError(why)


def _check_tensors(dtype_of: dict):
    """Every tensor given is of its dtype, on one CUDA device, which is the current one."""
    import torch
    dev = torch.device("cuda", torch.cuda.current_device()) if torch.cuda.is_available() else None
    for name, (t, dtype) in dtype_of.items():
        if t is not None:
            _need(t.dtype == dtype, f"{name}: expected {dtype}, got {t.dtype}")
            _need(dev is None or t.device == dev, f"{name} is on {t.device}, not on the current device {dev}")


def _ready(args, workspace=None):
    """The call runs where its tensors are (they may have been checked under another current device)."""
    dev = args._tensors[args._lead].get_device()
    if dev != _current_device():
        raise ValueError(f"the tensors are on device {dev}, not on the current one")
    if workspace is not None and not (workspace.get_device() == dev and workspace.is_contiguous()):
        raise ValueError("the workspace is on another device, or not contiguous")


def _fits(args, k_codec, v_codec):
    """The records are of the codecs' size (looked at once for an argument block and its codecs)."""
    if args._fit is None or args._fit[0] is not k_codec or args._fit[1] is not v_codec:
        for codec, rec, name in ((k_codec, args._records[0], "k_rec"), (v_codec, args._records[1], "v_rec")):
            _check_records(codec, rec, name)
        args._fit = (k_codec, v_codec)


def _scratch(size: int, device, stream):
    """A workspace that belongs to the stream the call runs on: freed, it serves that stream only."""
    import torch
    if stream is None:
        return torch.empty(size, dtype=torch.uint8, device=device)
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream, device) if stream else torch.cuda.default_stream(device)
    with torch.cuda.stream(stream):
        return torch.empty(size, dtype=torch.uint8, device=device)


def _heads_packed(t, name: str, d: int):
    """(layer, batch, token) strides of a [L, B, T, heads, d] view whose heads and dims are packed."""
    _need(t.dim() == 5 and t.shape[4] == d and t.stride(4) == 1 and (t.shape[3] == 1 or t.stride(3) == d),
          f"{name}: expected [L, B, T, heads, d] with heads and dims packed")
    return tuple(t.stride(i) if t.shape[i] > 1 else 0 for i in range(3))


def _ring_cap(t, name: str):
    L, B, H, cap, d = t.shape
    _need(t.stride(4) == 1 and t.stride(3) == d and (H == 1 or t.stride(2) == cap * d) and
          (B == 1 or t.stride(1) == H * cap * d), f"{name}: a layer's ring [B, Hkv, cap, d] must be contiguous")
    return cap


def _counts(t, name: str, L: int, B: int):
    _need(t is None or (t.is_contiguous() and tuple(t.shape) == (L, B)), f"{name}: expected contiguous int32 [{L}, {B}]")


def rope_pair_axis(sections, interleaved: bool = False):
    """Axis of every frequency pair for `sections` (pairs per axis): each axis turns its own run of
    frequencies, or, interleaved, the axes take turns (0, 1, 2, 0, 1, 2, ...) until a section is used up."""
    if not interleaved:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    left, out = list(sections), []
    while any(left):
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                out.append(a)
    return out


def make_append_args(*, k, k_tail, tail_len, tail_len_out=None, v=None, v_tail=None, q=None, q_out=None,
                     positions=None, inv_freq=None, pair_axis=None, rot_start: int = 0, pair_adjacent: bool = False,
                     rot_scale: float = 1.0, tail_start=None, q_lens=None, mass=None, n_chunks=None) -> tq_append_args:
    """tq_append_args from tensors.  q, k, v, q_out: bf16 views [L, B, T, heads, d] (heads and dims packed;
    k and v with equal strides); k_tail, v_tail: bf16 [L, B, Hkv, cap, d] (v and v_tail None where keys and
    values share a ring); positions: int32 [axes, B, T]; inv_freq: f32 [pairs], 2 * pairs coordinates from
    rot_start on turn; pair_axis: axis of each pair (default 0; rope_pair_axis); counters int32 [L, B]
    (tail_len_out defaults to tail_len); mass: f32 [L, B, Hkv, cap]."""
    import torch
    i32, f32, bf = torch.int32, torch.float32, torch.bfloat16
    _check_tensors(dict(q=(q, bf), k=(k, bf), v=(v, bf), q_out=(q_out, bf), k_tail=(k_tail, bf), v_tail=(v_tail, bf),
                        positions=(positions, i32), inv_freq=(inv_freq, f32), tail_start=(tail_start, i32),
                        tail_len=(tail_len, i32), tail_len_out=(tail_len_out, i32), q_lens=(q_lens, i32),
                        mass=(mass, f32), n_chunks=(n_chunks, i32)))
    L, B, T, Hkv, d = k.shape
    a = tq_append_args()
    a.n_layers, a.batch, a.t_q, a.n_kv_heads, a.head_dim = L, B, T, Hkv, d
    a.k, (a.kv_layer_stride, a.kv_batch_stride, a.kv_token_stride) = k.data_ptr(), _heads_packed(k, "k", d)
    if v is not None:
        _need(v.shape == k.shape and _heads_packed(v, "v", d) == _heads_packed(k, "k", d),
              "v: expected k's shape and strides")
        a.v = v.data_ptr()
    if q is not None:
        _need(q_out is not None and q_out.shape == q.shape and q.shape[:3] == k.shape[:3] and q.shape[4] == d,
              "q, q_out: expected [L, B, T, Hq, d] like k")
        a.n_q_heads = q.shape[3]
        a.q, (a.q_layer_stride, a.q_batch_stride, a.q_token_stride) = q.data_ptr(), _heads_packed(q, "q", d)
        a.q_out = q_out.data_ptr()
        a.q_out_layer_stride, a.q_out_batch_stride, a.q_out_token_stride = _heads_packed(q_out, "q_out", d)
    _need(tuple(k_tail.shape[:3]) == (L, B, Hkv) and k_tail.shape[4] == d, "k_tail: expected [L, B, Hkv, cap, d]")
    a.tail_cap = _ring_cap(k_tail, "k_tail")
    a.k_tail, a.tail_layer_stride = k_tail.data_ptr(), _layer_stride(k_tail)
    if v_tail is not None:
        _need(v_tail.shape == k_tail.shape and v_tail.stride() == k_tail.stride(), "v_tail: expected k_tail's layout")
        a.v_tail = v_tail.data_ptr()
    if inv_freq is not None:
        n = inv_freq.numel()
        _need(inv_freq.is_contiguous() and 0 < 2 * n <= d, "inv_freq: expected contiguous f32 [pairs], 2 * pairs <= d")
        _need(positions is not None and positions.is_contiguous() and positions.dim() == 3 and
              tuple(positions.shape[1:]) == (B, T), "positions: expected contiguous int32 [axes, B, T]")
        axis = [0] * n if pair_axis is None else [int(x) for x in pair_axis]
        _need(len(axis) == n and all(0 <= x < 256 for x in axis), "pair_axis: expected one axis for each pair")
        a.n_axes, a.rot_dim, a.rot_start = positions.shape[0], 2 * n, rot_start
        a.positions, a.inv_freq = positions.data_ptr(), inv_freq.data_ptr()
        a.pair_axis[:n] = axis
    a.pair_adjacent, a.rot_scale = int(pair_adjacent), rot_scale
    out = tail_len if tail_len_out is None else tail_len_out
    for name, t in (("tail_start", tail_start), ("tail_len", tail_len), ("tail_len_out", out), ("n_chunks", n_chunks)):
        _counts(t, name, L, B)
    _need(q_lens is None or (q_lens.is_contiguous() and tuple(q_lens.shape) == (B,)), "q_lens: expected int32 [B]")
    a.tail_start, a.tail_len, a.tail_len_out = _ptr(tail_start), tail_len.data_ptr(), out.data_ptr()
    a.q_lens, a.n_chunks = _ptr(q_lens), _ptr(n_chunks)
    if mass is not None:
        a.mass, a.mass_layer_stride, a.mass_cap = mass.data_ptr(), *_mass_layout(mass, L, B, Hkv)
    a._lead = 1
    a._tensors = (q, k, v, q_out, positions, inv_freq, k_tail, v_tail, tail_start, tail_len, out, q_lens, mass,
                  n_chunks)
    return a


def _layer_stride(t) -> int:
    return t.stride(0) if t.shape[0] > 1 else 0


def _mass_layout(mass, L: int, B: int, Hkv: int):
    cap = mass.shape[-1]
    _need(tuple(mass.shape[:3]) == (L, B, Hkv) and mass.dim() == 4 and mass.stride(3) == 1 and
          (Hkv == 1 or mass.stride(2) == cap) and (B == 1 or mass.stride(1) == Hkv * cap),
          "mass: expected f32 [L, B, Hkv, cap], contiguous within a layer")
    return _layer_stride(mass), cap


def tq_append(args: tq_append_args, stream=None):
    """Rotate queries and keys and append keys and values to the ring (include/tq.h)."""
    _ready(args)
    _check("tq_append", load().tq_append(ctypes.byref(args), _stream(stream)))


def make_query_args(*, q, scale: float, out=None, softcap: float = 0.0, causal: bool = True, q_lens=None, k_rec=None,
                    v_rec=None, k_tail=None, v_tail=None, n_chunks=None, tail_start=None, tail_len=None,
                    max_chunks: int = 0, max_tail: int = 0, block_table=None, splits: int = 0,
                    n_kv_heads: int | None = None) -> tq_query_args:
    """tq_query_args from tensors.  q, out: bf16 views [L, B, T, Hq, d] (heads and dims packed; out for
    tq_prefill_attn); the cache as for make_attn_args; q_lens: int32 [B]."""
    import torch
    i32, bf = torch.int32, torch.bfloat16
    _check_tensors(dict(q=(q, bf), out=(out, bf), k_rec=(k_rec, torch.uint8), v_rec=(v_rec, torch.uint8),
                        k_tail=(k_tail, bf), v_tail=(v_tail, bf), n_chunks=(n_chunks, i32),
                        tail_start=(tail_start, i32), tail_len=(tail_len, i32), q_lens=(q_lens, i32),
                        block_table=(block_table, i32)))
    L, B, T, Hq, d = q.shape
    a = tq_query_args()
    a.n_layers, a.batch, a.t_q, a.n_q_heads, a.head_dim = L, B, T, Hq, d
    a.scale, a.softcap, a.causal, a.splits = scale, softcap, int(causal), splits
    a.q, (a.q_layer_stride, a.q_batch_stride, a.q_token_stride) = q.data_ptr(), _heads_packed(q, "q", d)
    if out is not None:
        _need(out.shape == q.shape, "out: expected q's shape")
        a.out, (a.out_layer_stride, a.out_batch_stride, a.out_token_stride) = (out.data_ptr(),
                                                                              _heads_packed(out, "out", d))
    paged = block_table is not None
    src = k_rec if k_rec is not None else k_tail
    Hkv = n_kv_heads if n_kv_heads is not None else (src.shape[2] if src is not None else Hq)
    a.n_kv_heads = Hkv
    for r, name in ((k_rec, "k_rec"), (v_rec, "v_rec")):
        if r is not None:
            lead = (r.shape[0], r.shape[2]) if paged else tuple(r.shape[:3])
            _need(r.dim() == (4 if paged else 5) and lead == ((L, Hkv) if paged else (L, B, Hkv)) and
                  r[0].is_contiguous(),
                  f"{name}: expected records [L, B, Hkv, cap, bytes] or a pool [L, blocks, Hkv, bytes], "
                  "contiguous within a layer")
    if k_rec is not None:
        a.k_rec, a.k_rec_layer_stride = k_rec.data_ptr(), _layer_stride(k_rec)
        a.rec_cap = k_rec.shape[1] if paged else k_rec.shape[3]
    if v_rec is not None:
        _need(k_rec is not None and v_rec.shape[:-1] == k_rec.shape[:-1], "v_rec: expected k_rec's layout")
        a.v_rec, a.v_rec_layer_stride = v_rec.data_ptr(), _layer_stride(v_rec)
    if paged:
        _need(block_table.is_contiguous() and block_table.dim() == 2 and block_table.shape[0] == B,
              "block_table: expected contiguous int32 [B, stride]")
        a.block_table, a.table_stride = block_table.data_ptr(), block_table.shape[1]
    if k_tail is not None:
        _need(tuple(k_tail.shape[:3]) == (L, B, Hkv) and k_tail.shape[4] == d, "k_tail: expected [L, B, Hkv, cap, d]")
        a.k_tail, a.tail_layer_stride, a.tail_cap = k_tail.data_ptr(), _layer_stride(k_tail), _ring_cap(k_tail, "k_tail")
    if v_tail is not None:
        _need(k_tail is not None and v_tail.shape == k_tail.shape and v_tail.stride() == k_tail.stride(),
              "v_tail: expected k_tail's layout")
        a.v_tail = v_tail.data_ptr()
    for name, t in (("n_chunks", n_chunks), ("tail_start", tail_start), ("tail_len", tail_len)):
        _counts(t, name, L, B)
    _need(q_lens is None or (q_lens.is_contiguous() and tuple(q_lens.shape) == (B,)), "q_lens: expected int32 [B]")
    a.n_chunks, a.tail_start, a.tail_len, a.q_lens = _ptr(n_chunks), _ptr(tail_start), _ptr(tail_len), _ptr(q_lens)
    a.max_chunks, a.max_tail = max_chunks, max_tail
    a._lead, a._records, a._fit = 0, (k_rec, v_rec), None
    a._tensors = (q, out, k_rec, v_rec, k_tail, v_tail, n_chunks, tail_start, tail_len, q_lens, block_table)
    return a


def _raw(codec):
    return None if codec is None else ctypes.byref(codec.c)


def _check_records(codec, rec, name: str):
    _need(codec is None or rec is None or rec.shape[-1] == codec.record_bytes,
          f"{name}: records are not of the codec's {codec.record_bytes if codec else 0} bytes")


def tq_prefill_attn_workspace_size(args: tq_query_args, k_codec: Codec | None, v_codec: Codec | None) -> int:
    n = load().tq_prefill_attn_workspace_size(ctypes.byref(args), _raw(k_codec), _raw(v_codec))
    if n == 0:
        raise TqError("tq_prefill_attn_workspace_size", TQ_ERR_INVALID_ARG)
    return int(n)


def tq_prefill_attn(args: tq_query_args, k_codec: Codec | None, v_codec: Codec | None, workspace, stream=None):
    """Attention of several query tokens per sequence over records and ring, bf16 out (include/tq.h)."""
    _ready(args, workspace)
    _fits(args, k_codec, v_codec)
    _check("tq_prefill_attn", load().tq_prefill_attn(ctypes.byref(args), _raw(k_codec), _raw(v_codec), _ptr(workspace),
                                                     workspace.numel() * workspace.element_size(), _stream(stream)))


def prefill_attn(*, k_codec=None, v_codec=None, workspace=None, stream=None, **kw):
    """Convenience: build the arguments, size/allocate the workspace if not given, run."""
    a = make_query_args(**kw)
    need = tq_prefill_attn_workspace_size(a, k_codec, v_codec)
    if workspace is None or workspace.numel() < need:
        workspace = _scratch(need, kw["q"].device, stream)
    tq_prefill_attn(a, k_codec, v_codec, workspace, stream)
    return workspace


def tq_attn_mass_workspace_size(args: tq_query_args, k_codec: Codec | None) -> int:
    n = load().tq_attn_mass_workspace_size(ctypes.byref(args), _raw(k_codec))
    if n == 0:
        raise TqError("tq_attn_mass_workspace_size", TQ_ERR_INVALID_ARG)
    return int(n)


def tq_attn_mass(args: tq_query_args, k_codec: Codec | None, mass, workspace, decay: float = 1.0, stream=None):
    """mass (f32 [L, B, Hkv, cap]) = decay * mass + the attention weight each cached token receives
    from the queries (include/tq.h)."""
    _ready(args, workspace)
    _fits(args, k_codec, None)
    import torch
    _need(mass.dtype == torch.float32 and mass.device == args._tensors[0].device,
          "mass: expected f32 on the queries' device")
    stride, cap = _mass_layout(mass, args.n_layers, args.batch, args.n_kv_heads)
    _check("tq_attn_mass", load().tq_attn_mass(ctypes.byref(args), _raw(k_codec), _ptr(mass), stride, cap, decay,
                                               _ptr(workspace), workspace.numel() * workspace.element_size(),
                                               _stream(stream)))


def attn_mass(*, mass, k_codec=None, decay: float = 1.0, workspace=None, stream=None, **kw):
    """Convenience: build the arguments, size/allocate the workspace if not given, run."""
    import torch
    _check_tensors(dict(mass=(mass, torch.float32)))
    a = make_query_args(**kw)
    need = tq_attn_mass_workspace_size(a, k_codec)
    if workspace is None or workspace.numel() < need:
        workspace = _scratch(need, kw["q"].device, stream)
    tq_attn_mass(a, k_codec, mass, workspace, decay, stream)
    return workspace


def make_evict_mass_args(*, k_rec, v_rec, mass, n_chunks, max_chunks: int, keep_chunks: int, k_dst=None, v_dst=None,
                         mass_dst=None, n_chunks_dst=None, tail_len=None, max_tail: int = 0, sink: int = 0,
                         recent: int = 0, kept=None, block_table=None, dst_table=None) -> tq_evict_mass_args:
    """tq_evict_mass_args from tensors: records as for make_evict_args (v_rec may be k_rec), mass f32
    [L, B, Hkv, cap]; without k_dst, v_dst, mass_dst, n_chunks_dst the cache is compacted in place;
    kept: optional int32 [L, B, Hkv, 128 * keep_chunks]."""
    import torch
    i32, f32, u8 = torch.int32, torch.float32, torch.uint8
    dst = (k_dst, v_dst, mass_dst, n_chunks_dst)
    _need(all(t is None for t in dst) or all(t is not None for t in dst),
          "k_dst, v_dst, mass_dst and n_chunks_dst go together")
    in_place = k_dst is None
    _need(not in_place or dst_table is None, "dst_table: only out of place")
    if in_place:
        k_dst, v_dst, mass_dst, n_chunks_dst, dst_table = k_rec, v_rec, mass, n_chunks, block_table
    _check_tensors(dict(k_rec=(k_rec, u8), v_rec=(v_rec, u8), k_dst=(k_dst, u8), v_dst=(v_dst, u8), mass=(mass, f32),
                        mass_dst=(mass_dst, f32), n_chunks=(n_chunks, i32), n_chunks_dst=(n_chunks_dst, i32),
                        tail_len=(tail_len, i32), kept=(kept, i32), block_table=(block_table, i32),
                        dst_table=(dst_table, i32)))
    L, B, Hkv = mass.shape[:3]
    a = tq_evict_mass_args()
    a.n_layers, a.batch, a.n_kv_heads = L, B, Hkv
    for rec, table, name in ((k_rec, block_table, "k_rec"), (v_rec, block_table, "v_rec"), (k_dst, dst_table, "k_dst"),
                             (v_dst, dst_table, "v_dst")):
        lead = (rec.shape[0], rec.shape[2]) if table is not None else tuple(rec.shape[:3])
        _need(rec.dim() == (5 if table is None else 4) and
              lead == ((L, Hkv) if table is not None else (L, B, Hkv)) and rec[0].is_contiguous(),
              f"{name}: expected records [L, B, Hkv, cap, bytes] or a pool [L, blocks, Hkv, bytes], "
              "contiguous within a layer")
    _need(v_rec.shape[:-1] == k_rec.shape[:-1] and v_dst.shape[:-1] == k_dst.shape[:-1],
          "key and value records: expected one layout")
    _need(k_dst.shape[-1] == k_rec.shape[-1] and v_dst.shape[-1] == v_rec.shape[-1],
          "destination records: expected the source's size")
    a.k_rec, a.v_rec, a.k_dst, a.v_dst = (t.data_ptr() for t in (k_rec, v_rec, k_dst, v_dst))
    a.k_rec_layer_stride, a.v_rec_layer_stride = _layer_stride(k_rec), _layer_stride(v_rec)
    a.k_dst_layer_stride, a.v_dst_layer_stride = _layer_stride(k_dst), _layer_stride(v_dst)
    a.rec_cap = k_rec.shape[1] if block_table is not None else k_rec.shape[3]
    a.dst_cap = k_dst.shape[1] if dst_table is not None else k_dst.shape[3]
    for table, name in ((block_table, "block_table"), (dst_table, "dst_table")):
        _need(table is None or (table.is_contiguous() and table.dim() == 2 and table.shape[0] == B),
              f"{name}: expected contiguous int32 [B, stride]")
    if block_table is not None:
        a.block_table, a.table_stride = block_table.data_ptr(), block_table.shape[1]
    if dst_table is not None:
        a.dst_table, a.dst_table_stride = dst_table.data_ptr(), dst_table.shape[1]
    a.mass, a.mass_layer_stride, a.mass_cap = mass.data_ptr(), *_mass_layout(mass, L, B, Hkv)
    a.mass_dst, a.mass_dst_layer_stride, a.mass_dst_cap = mass_dst.data_ptr(), *_mass_layout(mass_dst, L, B, Hkv)
    for name, t in (("n_chunks", n_chunks), ("n_chunks_dst", n_chunks_dst), ("tail_len", tail_len)):
        _counts(t, name, L, B)
    a.n_chunks, a.n_chunks_dst, a.tail_len = n_chunks.data_ptr(), n_chunks_dst.data_ptr(), _ptr(tail_len)
    _need(kept is None or (kept.is_contiguous() and tuple(kept.shape) == (L, B, Hkv, CHUNK * keep_chunks)),
          "kept: expected contiguous int32 [L, B, Hkv, 128 * keep_chunks]")
    a.kept = _ptr(kept)
    a.max_chunks, a.max_tail, a.keep_chunks, a.sink, a.recent = max_chunks, max_tail, keep_chunks, sink, recent
    a._lead, a._records, a._fit = 0, (k_rec, v_rec), None
    a._tensors = (k_rec, v_rec, k_dst, v_dst, mass, mass_dst, n_chunks, n_chunks_dst, tail_len, kept, block_table,
                  dst_table)
    return a


def tq_evict_mass_workspace_size(args: tq_evict_mass_args, k_codec: Codec, v_codec: Codec | None) -> int:
    n = load().tq_evict_mass_workspace_size(ctypes.byref(args), _raw(k_codec), _raw(v_codec))
    if n == 0:
        raise TqError("tq_evict_mass_workspace_size", TQ_ERR_INVALID_ARG)
    return int(n)


def tq_evict_mass(args: tq_evict_mass_args, k_codec: Codec, v_codec: Codec | None, workspace, stream=None):
    """Keep the tokens of the largest accumulated weight and compact the records (include/tq.h)."""
    _ready(args, workspace)
    _fits(args, k_codec, v_codec)
    _check("tq_evict_mass", load().tq_evict_mass(ctypes.byref(args), _raw(k_codec), _raw(v_codec), _ptr(workspace),
                                                 workspace.numel() * workspace.element_size(), _stream(stream)))


def evict_mass(*, k_codec, v_codec=None, workspace=None, stream=None, **kw):
    """Convenience: build the arguments, size/allocate the workspace if not given, run."""
    a = make_evict_mass_args(**kw)
    need = tq_evict_mass_workspace_size(a, k_codec, v_codec)
    if workspace is None or workspace.numel() < need:
        workspace = _scratch(need, kw["k_rec"].device, stream)
    tq_evict_mass(a, k_codec, v_codec, workspace, stream)
    return workspace


# ---------------------------------------------------------------------------
# attention to a part of a long cache: head norms, key bounds, selection, listed records
# ---------------------------------------------------------------------------
def _bounds_layout(bounds, rec_cap: int, L: int, B: int, Hkv: int, d: int, paged: bool) -> int:
    """Layer stride of bounds that lie as the records do."""
    import torch
    want = (L, rec_cap, Hkv, 2, d) if paged else (L, B, Hkv, rec_cap, 2, d)
    _need(tuple(bounds.shape) == want and bounds[0].is_contiguous(),
          f"bounds: expected {torch.bfloat16} {list(want)}, contiguous within a layer")
    return _layer_stride(bounds)


def _table(a, block_table, B: int):
    if block_table is not None:
        _need(block_table.is_contiguous() and block_table.dim() == 2 and block_table.shape[0] == B,
              "block_table: expected contiguous int32 [B, stride]")
        a.block_table, a.table_stride = block_table.data_ptr(), block_table.shape[1]


def make_head_norm(*, q_weight=None, k_weight=None, eps: float = 1e-6) -> tq_head_norm:
    """tq_head_norm from tensors: f32 [d] for all heads or [heads, d] (rows packed within a head); None: that side
    is not normalised."""
    import torch
    _check_tensors(dict(q_weight=(q_weight, torch.float32), k_weight=(k_weight, torch.float32)))
    n = tq_head_norm()
    for name, w in (("q", q_weight), ("k", k_weight)):
        if w is not None:
            _need(w.dim() in (1, 2) and w.stride(-1) == 1, f"{name}_weight: expected f32 [d] or [heads, d]")
            setattr(n, name + "_weight", w.data_ptr())
            setattr(n, name + "_head_stride", w.stride(0) if w.dim() == 2 and w.shape[0] > 1 else 0)
    n.eps = eps
    n._tensors = (q_weight, k_weight)
    n._fit = None
    return n


def tq_norm_append(args: tq_append_args, norm: tq_head_norm, stream=None):
    """tq_append with the queries' and keys' heads normalised before the rotation (include/tq.h)."""
    _ready(args)
    if norm._fit is not args:  # looked at once for two argument blocks
        for w, heads in zip(norm._tensors, (args.n_q_heads, args.n_kv_heads)):
            _need(w is None or (w.shape[-1] == args.head_dim and (w.dim() == 1 or w.shape[0] == heads) and
                                w.device == args._tensors[args._lead].device),
                  "norm weights: expected [d] or [heads, d] on the tensors' device")
        norm._fit = args
    _check("tq_norm_append", load().tq_norm_append(ctypes.byref(args), ctypes.byref(norm), _stream(stream)))


def make_bounds_args(*, k_rec, bounds, n_chunks, max_chunks: int, first=None, max_new: int | None = None,
                     block_table=None) -> tq_bounds_args:
    """tq_bounds_args from tensors.  k_rec: uint8 [L, B, Hkv, cap, bytes], or with block_table (int32 [B, stride])
    pools [L, blocks, Hkv, bytes]; bounds: bf16 [L, B, Hkv, cap, 2, d] or [L, blocks, Hkv, 2, d]; n_chunks, first:
    int32 [L, B] (records from first on are bounded, max_new at most; default: all up to max_chunks)."""
    import torch
    i32 = torch.int32
    _check_tensors(dict(k_rec=(k_rec, torch.uint8), bounds=(bounds, torch.bfloat16), n_chunks=(n_chunks, i32),
                        first=(first, i32), block_table=(block_table, i32)))
    paged = block_table is not None
    _need(k_rec.dim() == (4 if paged else 5) and k_rec[0].is_contiguous(),
          "k_rec: expected records [L, B, Hkv, cap, bytes] or a pool [L, blocks, Hkv, bytes], contiguous within a layer")
    a = tq_bounds_args()
    if paged:
        (L, cap, Hkv), B = k_rec.shape[:3], block_table.shape[0]
    else:
        L, B, Hkv, cap = k_rec.shape[:4]
    _table(a, block_table, B)
    a.n_layers, a.batch, a.n_kv_heads, a.rec_cap = L, B, Hkv, cap
    a.k_rec, a.k_rec_layer_stride = k_rec.data_ptr(), _layer_stride(k_rec)
    a.bounds, a.bounds_layer_stride = bounds.data_ptr(), _bounds_layout(bounds, cap, L, B, Hkv, bounds.shape[-1], paged)
    _counts(n_chunks, "n_chunks", L, B)
    _counts(first, "first", L, B)
    a.n_chunks, a.first = n_chunks.data_ptr(), _ptr(first)
    a.max_chunks, a.max_new = max_chunks, max(max_chunks, 1) if max_new is None else max_new
    a._lead, a._records, a._fit = 0, (k_rec, None), None
    a._tensors = (k_rec, bounds, n_chunks, first, block_table)
    return a


def tq_key_bounds(args: tq_bounds_args, k_codec: Codec, stream=None):
    """Smallest and largest value of each coordinate of every record's keys; to be formed again where records have
    changed, as tq_evict_mass and evictions after tq_rollback change them (include/tq.h)."""
    _ready(args)
    _fits(args, k_codec, None)
    _need(args._tensors[1].shape[-1] == k_codec.head_dim, "bounds: expected the codec's head dim")
    _check("tq_key_bounds", load().tq_key_bounds(_raw(k_codec), ctypes.byref(args), _stream(stream)))


def key_bounds(*, k_codec, stream=None, **kw):
    """Convenience: build the arguments, run."""
    tq_key_bounds(make_bounds_args(**kw), k_codec, stream)


def make_select_args(*, q, bounds, n_chunks, max_chunks: int, list, count, keep: int, q_block: int = 1, sink: int = 1,
                     recent: int = 1, causal: bool = True, q_lens=None, tail_len=None, max_tail: int = 0,
                     block_table=None) -> tq_select_args:
    """tq_select_args from tensors.  q: bf16 view [L, B, T, Hq, d]; bounds as for make_bounds_args; list: int32
    [L, B, blocks, Hkv, keep], count: int32 [L, B, blocks, Hkv], blocks = ceil(T / q_block); counters int32 [L, B]."""
    import torch
    i32, bf = torch.int32, torch.bfloat16
    _check_tensors(dict(q=(q, bf), bounds=(bounds, bf), n_chunks=(n_chunks, i32), tail_len=(tail_len, i32),
                        q_lens=(q_lens, i32), block_table=(block_table, i32), list=(list, i32), count=(count, i32)))
    L, B, T, Hq, d = q.shape
    paged = block_table is not None
    _need(bounds.dim() == (5 if paged else 6), "bounds: expected [L, B, Hkv, cap, 2, d] or a pool [L, blocks, Hkv, 2, d]")
    Hkv, cap = bounds.shape[2], bounds.shape[1] if paged else bounds.shape[3]
    a = tq_select_args()
    a.n_layers, a.batch, a.t_q, a.n_q_heads, a.n_kv_heads, a.head_dim, a.causal = L, B, T, Hq, Hkv, d, int(causal)
    a.q, (a.q_layer_stride, a.q_batch_stride, a.q_token_stride) = q.data_ptr(), _heads_packed(q, "q", d)
    a.bounds, a.bounds_layer_stride = bounds.data_ptr(), _bounds_layout(bounds, cap, L, B, Hkv, d, paged)
    a.rec_cap = cap
    _table(a, block_table, B)
    for name, t in (("n_chunks", n_chunks), ("tail_len", tail_len)):
        _counts(t, name, L, B)
    _need(q_lens is None or (q_lens.is_contiguous() and tuple(q_lens.shape) == (B,)), "q_lens: expected int32 [B]")
    _need(q_block >= 1 and keep >= 1, "q_block, keep: expected at least 1")
    blocks = -(-T // q_block)
    _need(tuple(list.shape) == (L, B, blocks, Hkv, keep) and list.is_contiguous() and
          tuple(count.shape) == (L, B, blocks, Hkv) and count.is_contiguous(),
          f"list, count: expected contiguous int32 {[L, B, blocks, Hkv, keep]} and {[L, B, blocks, Hkv]}")
    a.q_lens, a.n_chunks, a.tail_len = _ptr(q_lens), n_chunks.data_ptr(), _ptr(tail_len)
    a.max_chunks, a.max_tail, a.q_block, a.keep, a.sink, a.recent = max_chunks, max_tail, q_block, keep, sink, recent
    a.list, a.count = list.data_ptr(), count.data_ptr()
    a._lead = 0
    a._tensors = (q, bounds, n_chunks, tail_len, q_lens, block_table, list, count)
    return a


def tq_select_records_workspace_size(args: tq_select_args) -> int:
    n = load().tq_select_records_workspace_size(ctypes.byref(args))
    if n == 0:
        raise TqError("tq_select_records_workspace_size", TQ_ERR_INVALID_ARG)
    return int(n)


def tq_select_records(args: tq_select_args, workspace, stream=None):
    """Records chosen for blocks of queries by an upper bound of their logits (include/tq.h)."""
    _ready(args, workspace)
    _check("tq_select_records", load().tq_select_records(ctypes.byref(args), _ptr(workspace),
                                                         workspace.numel() * workspace.element_size(), _stream(stream)))


def select_records(*, workspace=None, stream=None, **kw):
    """Convenience: build the arguments, size/allocate the workspace if not given, run."""
    a = make_select_args(**kw)
    need = tq_select_records_workspace_size(a)
    if workspace is None or workspace.numel() < need:
        workspace = _scratch(need, kw["q"].device, stream)
    tq_select_records(a, workspace, stream)
    return workspace


def make_record_lists(*, list, count, q_block: int = 1) -> tq_record_lists:
    """tq_record_lists from tensors: int32 [L, B, blocks, Hkv, entries] and [L, B, blocks, Hkv]."""
    import torch
    _check_tensors(dict(list=(list, torch.int32), count=(count, torch.int32)))
    _need(list.dim() == 5 and list.is_contiguous() and count.is_contiguous() and tuple(count.shape) == tuple(list.shape[:4]),
          "list, count: expected contiguous int32 [L, B, blocks, Hkv, entries] and [L, B, blocks, Hkv]")
    r = tq_record_lists(list.data_ptr(), count.data_ptr(), list.shape[4], q_block)
    r._tensors = (list, count)
    r._fit = None
    return r


def _lists_fit(args: tq_query_args, lists: tq_record_lists):
    """The lists are those of the queries (looked at once for two argument blocks)."""
    if lists._fit is args:
        return
    _need(lists.q_block >= 1, "q_block: expected at least 1")
    want = (args.n_layers, args.batch, -(-args.t_q // lists.q_block), args.n_kv_heads)
    _need(tuple(lists._tensors[1].shape) == want and lists._tensors[0].device == args._tensors[0].device,
          f"list, count: expected {list(want)} lists on the queries' device")
    lists._fit = args


def tq_sparse_attn_workspace_size(args: tq_query_args, lists: tq_record_lists, k_codec: Codec,
                                  v_codec: Codec | None) -> int:
    n = load().tq_sparse_attn_workspace_size(ctypes.byref(args), ctypes.byref(lists), _raw(k_codec), _raw(v_codec))
    if n == 0:
        raise TqError("tq_sparse_attn_workspace_size", TQ_ERR_INVALID_ARG)
    return int(n)


def tq_sparse_attn(args: tq_query_args, lists: tq_record_lists, k_codec: Codec, v_codec: Codec | None, workspace,
                   stream=None):
    """Attention over listed records and the ring, bf16 out (include/tq.h)."""
    _ready(args, workspace)
    _fits(args, k_codec, v_codec)
    _lists_fit(args, lists)
    _check("tq_sparse_attn", load().tq_sparse_attn(ctypes.byref(args), ctypes.byref(lists), _raw(k_codec), _raw(v_codec),
                                                   _ptr(workspace), workspace.numel() * workspace.element_size(),
                                                   _stream(stream)))


def sparse_attn(*, list, count, q_block: int = 1, k_codec=None, v_codec=None, workspace=None, stream=None, **kw):
    """Convenience: build the arguments, size/allocate the workspace if not given, run."""
    a = make_query_args(**kw)
    lists = make_record_lists(list=list, count=count, q_block=q_block)
    need = tq_sparse_attn_workspace_size(a, lists, k_codec, v_codec)
    if workspace is None or workspace.numel() < need:
        workspace = _scratch(need, kw["q"].device, stream)
    tq_sparse_attn(a, lists, k_codec, v_codec, workspace, stream)
    return workspace
