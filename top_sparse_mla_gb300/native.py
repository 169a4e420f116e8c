"""ctypes binding of the C ABI in include/*.h (argument marshalling only).

Every entry point keeps the C name.  Tensors are passed as raw device pointers
(``tensor.data_ptr()``); the stream is the caller's current CUDA stream.  All of the
computation happens in the CUDA library; when the library is missing this module raises
instead of falling back to anything else.
"""

from __future__ import annotations

import ctypes
import os

from .build import LIB_PATH

DSA_OK = 0
DSA_ERR_INVALID_ARG = -1
DSA_ERR_UNSUPPORTED_SHAPE = -2
DSA_ERR_WORKSPACE_TOO_SMALL = -3
DSA_ERR_CUDA = -4
DSA_ERR_UNSUPPORTED_DEVICE = -5
DSA_ERR_SCRATCH_LIMIT = -6
DSA_FLAG_CHECK_INDICES = 1
DSA_FLAG_TEST_WAIT_TIMEOUT = 2
DSA_STATUS_INDEX_OUT_OF_RANGE = 1
DSA_STATUS_WAIT_TIMEOUT = 2
DSA_MAX_HEADS = 64
DSA_MAX_DEVICES = 64
DSA_MAX_TOPK = 2048
DSA_ORDER_MAX_TOKENS = 65536
DSA_TOPK_MAX_COLS = 65536
DSA_TOPK_MAX_K = 2048
DSA_ROW_BYTES = 656
DSA_NOALLOC_SCRATCH_BYTES = 24 << 20
DSA_KV_FLAG_CHECK_SLOTS = 1
DSA_FLAG_AFTER_PRODUCER = 4
DSA_FLAG_SF_SWIZZLED = 8
DSA_FLAG_FP8_Q = 16
DSA_KV_FP8_DS_MLA = 0
DSA_KV_NVFP4_DS_MLA = 1
DSA_NVFP4_QK_DIMS = 512
DSA_NVFP4_SWA_ROW_BYTES = 528
DSA_NVFP4_CMP_ROW_BYTES = 288
DSA_STATUS_SLOT_OUT_OF_RANGE = 4
DSA_PAGE_MAP_MAX_REQ = 8192
DSA_STATUS_OUT_OF_PAGES = 8
DSA_STATUS_TABLE_FULL = 16
DSA_STATUS_TOKENS_FULL = 32
DSA_KV8_BF16 = 0
DSA_KV8_FP16 = 1
DSA_KV8_MAX_HEADS = 1024
DSA_KV8_MAX_GROUP = 128
DSA_KV8_MAX_REQ = 8192
DSA_KV8_MAX_GROUPS = 4096
DSA_KV8_FLAG_TEST_WAIT_TIMEOUT = 2
DSA_STATUS_QUERY_TOO_LONG = 64
DSA_QK_BF16 = 0
DSA_QK_FP16 = 1
DSA_QK_FLAG_INTERLEAVED = 1
DSA_QK_MAX_HEADS = 4096
DSA_MLA_BF16 = 0
DSA_MLA_FP16 = 1
DSA_MLA_MAX_HEADS = 1024
DSA_MLA_MAX_REQ = 8192
DSA_MLA_FLAG_TEST_WAIT_TIMEOUT = 2

EXPORTED = (
    "dsa_params_init",
    "dsa_sparse_attn_workspace_size",
    "dsa_sparse_attn_fwd",
    "dsa_sparse_attn_fwd_debug",
    "dsa_sparse_attn_fwd_noalloc",
    "dsa_sparse_attn_read_status",
    "dsa_sparse_attn_num_splits",
    "dsa_error_string",
    "dsa_topk_select",
    "dsa_kv_insert",
    "dsa_page_map",
    "dsa_kv8_insert",
    "dsa_kv8_params_init",
    "dsa_kv8_attn_workspace_size",
    "dsa_kv8_attn_fwd",
    "dsa_qk_params_init",
    "dsa_qk_norm_rope",
    "dsa_kv_gather",
    "dsa_mla_params_init",
    "dsa_mla_prefill_workspace_size",
    "dsa_mla_prefill_fwd",
    "dsa_kv8_prefix_workspace_size",
    "dsa_kv8_prefix_attn_fwd",
)


class DsaParams(ctypes.Structure):
    _fields_ = [
        ("s_q", ctypes.c_int32),
        ("h_q", ctypes.c_int32),
        ("topk", ctypes.c_int32),
        ("n_swa_cols", ctypes.c_int32),
        ("n_swa_rows", ctypes.c_int64),
        ("n_cmp_rows", ctypes.c_int64),
        ("softmax_scale", ctypes.c_float),
        ("rope_base", ctypes.c_float),
        ("rms_eps", ctypes.c_float),
        ("flags", ctypes.c_uint32),
        ("kv_format", ctypes.c_int32),
        ("cmp_scale", ctypes.c_float),
    ]


class DsaKv8Params(ctypes.Structure):
    _fields_ = [
        ("n_tokens", ctypes.c_int32),
        ("n_req", ctypes.c_int32),
        ("h_q", ctypes.c_int32),
        ("h_kv", ctypes.c_int32),
        ("d", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("n_pages", ctypes.c_int32),
        ("table_cols", ctypes.c_int32),
        ("max_q_len", ctypes.c_int32),
        ("window", ctypes.c_int32),
        ("type", ctypes.c_int32),
        ("softmax_scale", ctypes.c_float),
        ("flags", ctypes.c_uint32),
    ]


class DsaQkParams(ctypes.Structure):
    _fields_ = [
        ("n_tokens", ctypes.c_int32),
        ("h_q", ctypes.c_int32),
        ("h_k", ctypes.c_int32),
        ("d", ctypes.c_int32),
        ("rotary_dim", ctypes.c_int32),
        ("rotary_start", ctypes.c_int32),
        ("type", ctypes.c_int32),
        ("flags", ctypes.c_uint32),
        ("rms_eps", ctypes.c_float),
        ("rope_base", ctypes.c_float),
    ]


class DsaMlaParams(ctypes.Structure):
    _fields_ = [
        ("n_tokens", ctypes.c_int32),
        ("n_keys", ctypes.c_int32),
        ("n_req", ctypes.c_int32),
        ("h", ctypes.c_int32),
        ("max_q_len", ctypes.c_int32),
        ("max_kv_len", ctypes.c_int32),
        ("type", ctypes.c_int32),
        ("softmax_scale", ctypes.c_float),
        ("flags", ctypes.c_uint32),
    ]


class DsaError(RuntimeError):
    def __init__(self, code: int, where: str):
        super().__init__(f"{where}: {dsa_error_string(code)} (code {code})")
        self.code = code


_lib = None


def library(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the CUDA library once; raise if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise ImportError(f"{path} is missing: build it with top_sparse_mla_gb300.build.build()")
    lib = ctypes.CDLL(path)
    vp, sz = ctypes.c_void_p, ctypes.c_size_t
    pp = ctypes.POINTER(DsaParams)
    lib.dsa_params_init.argtypes = [pp, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32,
                                    ctypes.c_int64, ctypes.c_int64]
    lib.dsa_params_init.restype = ctypes.c_int
    lib.dsa_sparse_attn_workspace_size.argtypes = [pp, ctypes.c_int]
    lib.dsa_sparse_attn_workspace_size.restype = sz
    lib.dsa_sparse_attn_num_splits.argtypes = [pp, ctypes.c_int]
    lib.dsa_sparse_attn_num_splits.restype = ctypes.c_int
    lib.dsa_sparse_attn_fwd.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, pp, vp, sz, vp]
    lib.dsa_sparse_attn_fwd.restype = ctypes.c_int
    lib.dsa_sparse_attn_fwd_debug.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, vp, pp, vp, sz, vp]
    lib.dsa_sparse_attn_fwd_debug.restype = ctypes.c_int
    lib.dsa_sparse_attn_fwd_noalloc.argtypes = [vp, vp, vp, vp, vp, vp, vp, vp, vp, pp, vp, vp]
    lib.dsa_sparse_attn_fwd_noalloc.restype = ctypes.c_int
    lib.dsa_sparse_attn_read_status.argtypes = [vp, ctypes.POINTER(ctypes.c_uint32), vp]
    lib.dsa_sparse_attn_read_status.restype = ctypes.c_int
    lib.dsa_error_string.argtypes = [ctypes.c_int]
    lib.dsa_error_string.restype = ctypes.c_char_p
    lib.dsa_topk_select.argtypes = [vp, ctypes.c_int64, vp, ctypes.c_int32, ctypes.c_int32, ctypes.c_int32, vp, vp, vp]
    lib.dsa_topk_select.restype = ctypes.c_int
    lib.dsa_kv_insert.argtypes = [vp, ctypes.c_int64, vp, vp, ctypes.c_int32, vp, ctypes.c_float, ctypes.c_float, vp,
                                  ctypes.c_int64, ctypes.c_uint32, vp, vp]
    lib.dsa_kv_insert.restype = ctypes.c_int
    i32, i64 = ctypes.c_int32, ctypes.c_int64
    lib.dsa_page_map.argtypes = [vp, vp, i32, vp, i64, i32, vp, i32, i32, i32, vp, vp, vp, vp, vp, vp, vp]
    lib.dsa_page_map.restype = ctypes.c_int
    lib.dsa_kv8_insert.argtypes = [vp, i64, i64, vp, i64, i64, vp, i32, i32, vp, vp, vp, vp, i32, i32, i32, i32, vp, vp]
    lib.dsa_kv8_insert.restype = ctypes.c_int
    p8 = ctypes.POINTER(DsaKv8Params)
    lib.dsa_kv8_params_init.argtypes = [p8, i32, i32, i32, i32, i32, i32, i32, i32]
    lib.dsa_kv8_params_init.restype = ctypes.c_int
    lib.dsa_kv8_attn_workspace_size.argtypes = [p8, ctypes.c_int]
    lib.dsa_kv8_attn_workspace_size.restype = sz
    lib.dsa_kv8_attn_fwd.argtypes = [vp, i64, i64, vp, vp, vp, vp, vp, i64, vp, vp, vp, i64, i64, vp, p8, vp, sz, vp]
    lib.dsa_kv8_attn_fwd.restype = ctypes.c_int
    pq = ctypes.POINTER(DsaQkParams)
    lib.dsa_qk_params_init.argtypes = [pq, i32, i32, i32, i32]
    lib.dsa_qk_params_init.restype = ctypes.c_int
    lib.dsa_qk_norm_rope.argtypes = [vp, i64, i64, vp, i64, i64, vp, vp, vp, vp, i64, i64, vp, i64, i64, pq, vp]
    lib.dsa_qk_norm_rope.restype = ctypes.c_int
    lib.dsa_kv_gather.argtypes = [vp, i64, vp, i64, i32, i32, vp, vp, i32, vp, i64, i32, vp, vp]
    lib.dsa_kv_gather.restype = ctypes.c_int
    lib.dsa_kv8_prefix_workspace_size.argtypes = [p8, i32, ctypes.c_int]
    lib.dsa_kv8_prefix_workspace_size.restype = sz
    lib.dsa_kv8_prefix_attn_fwd.argtypes = [vp, i64, i64, vp, vp, vp, vp, vp, i64, vp, vp, vp, vp, i32, vp, i64, i64, vp, p8, vp, sz, vp]
    lib.dsa_kv8_prefix_attn_fwd.restype = ctypes.c_int
    pm = ctypes.POINTER(DsaMlaParams)
    lib.dsa_mla_params_init.argtypes = [pm, i32, i32, i32, i32]
    lib.dsa_mla_params_init.restype = ctypes.c_int
    lib.dsa_mla_prefill_workspace_size.argtypes = [pm, ctypes.c_int]
    lib.dsa_mla_prefill_workspace_size.restype = sz
    lib.dsa_mla_prefill_fwd.argtypes = [vp, i64, i64, vp, i64, i64, vp, i64, vp, i64, i64, vp, vp, vp, i64, i64, vp, pm, vp, sz, vp]
    lib.dsa_mla_prefill_fwd.restype = ctypes.c_int
    _lib = lib
    return lib


def sf_swizzled_bytes(s_q: int, h_q: int) -> int:
    """Size of out_sf with DSA_FLAG_SF_SWIZZLED (DSA_SF_SWIZZLED_BYTES in the header)."""
    return ((int(s_q) + 127) // 128) * 128 * 16 * int(h_q)


def dsa_error_string(code: int) -> str:
    return library().dsa_error_string(int(code)).decode()


def dsa_params_init(s_q, h_q, topk, n_swa_cols, n_swa_rows, n_cmp_rows, **overrides) -> DsaParams:
    p = DsaParams()
    rc = library().dsa_params_init(ctypes.byref(p), s_q, h_q, topk, n_swa_cols, n_swa_rows, n_cmp_rows)
    if rc != DSA_OK:
        raise DsaError(rc, "dsa_params_init")
    for k, v in overrides.items():
        setattr(p, k, v)
    return p


def dsa_sparse_attn_workspace_size(p: DsaParams, num_sms: int = 0) -> int:
    return int(library().dsa_sparse_attn_workspace_size(ctypes.byref(p), int(num_sms)))


def dsa_sparse_attn_num_splits(p: DsaParams, num_sms: int = 0) -> int:
    return int(library().dsa_sparse_attn_num_splits(ctypes.byref(p), int(num_sms)))


def _ptr(x):
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


# Bound by _bind_torch at the first call that needs them: a program that passes pointers and a
# stream of its own needs no torch.
torch = _raw_stream = _I32 = _I64 = _F32 = _U8 = None
_KV8_TYPES = {}


def _bind_torch() -> None:
    global torch, _raw_stream, _I32, _I64, _F32, _U8
    import torch as module
    # torch.cuda.current_stream() builds a Stream object, which takes longer than a launch
    _raw_stream = getattr(module._C, "_cuda_getCurrentRawStream", None)
    _I32, _I64, _F32, _U8 = module.int32, module.int64, module.float32, module.uint8
    _KV8_TYPES.update({module.bfloat16: DSA_KV8_BF16, module.float16: DSA_KV8_FP16})
    torch = module


def _stream(stream, dev=None):
    if stream is None:
        if dev is not None and _raw_stream is not None:   # the current device, as _device found it
            return _raw_stream(dev)
        if torch is None:
            _bind_torch()
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def dsa_sparse_attn_fwd(q, kv_swa, kv_cmp, indices, topk_length, positions, norm_w, out_fp8, out_sf,
                        p: DsaParams, workspace, workspace_bytes=None, stream=None) -> None:
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    rc = library().dsa_sparse_attn_fwd(_ptr(q), _ptr(kv_swa), _ptr(kv_cmp), _ptr(indices), _ptr(topk_length),
                                       _ptr(positions), _ptr(norm_w), _ptr(out_fp8), _ptr(out_sf), ctypes.byref(p),
                                       _ptr(workspace), int(workspace_bytes), _stream(stream))
    if rc != DSA_OK:
        raise DsaError(rc, "dsa_sparse_attn_fwd")


def dsa_sparse_attn_fwd_debug(q, kv_swa, kv_cmp, indices, topk_length, positions, norm_w, out_fp8, out_sf,
                              out_precast, lse, p: DsaParams, workspace, workspace_bytes=None, stream=None) -> None:
    if workspace_bytes is None:
        workspace_bytes = workspace.numel() * workspace.element_size()
    rc = library().dsa_sparse_attn_fwd_debug(_ptr(q), _ptr(kv_swa), _ptr(kv_cmp), _ptr(indices), _ptr(topk_length),
                                             _ptr(positions), _ptr(norm_w), _ptr(out_fp8), _ptr(out_sf),
                                             _ptr(out_precast), _ptr(lse), ctypes.byref(p), _ptr(workspace),
                                             int(workspace_bytes), _stream(stream))
    if rc != DSA_OK:
        raise DsaError(rc, "dsa_sparse_attn_fwd_debug")


def dsa_sparse_attn_fwd_noalloc(q, kv_swa, kv_cmp, indices, topk_length, positions, norm_w, out_fp8, out_sf,
                                p: DsaParams, status_out=None, stream=None) -> None:
    rc = library().dsa_sparse_attn_fwd_noalloc(_ptr(q), _ptr(kv_swa), _ptr(kv_cmp), _ptr(indices),
                                               _ptr(topk_length), _ptr(positions), _ptr(norm_w), _ptr(out_fp8),
                                               _ptr(out_sf), ctypes.byref(p), _ptr(status_out), _stream(stream))
    if rc != DSA_OK:
        raise DsaError(rc, "dsa_sparse_attn_fwd_noalloc")


def dsa_topk_select(logits, k: int, indices, topk_length, lengths=None, stream=None) -> None:
    """Top-k column selection (include/dsa_topk.h). logits: bf16 [s_q, ld] device tensor
    whose first n = logits.shape[1] columns are the candidates; indices: int32 [s_q, k];
    topk_length: int32 [s_q]; lengths: int32 [s_q] or None."""
    s_q, n = int(logits.shape[0]), int(logits.shape[1])
    if s_q > 0 and int(logits.stride(1)) != 1:
        raise DsaError(DSA_ERR_INVALID_ARG, "dsa_topk_select: logits rows must be contiguous")
    ld = int(logits.stride(0)) if s_q > 0 else n
    rc = library().dsa_topk_select(_ptr(logits), ld, _ptr(lengths), s_q, n, int(k), _ptr(indices),
                                   _ptr(topk_length), _stream(stream))
    if rc != DSA_OK:
        raise DsaError(rc, "dsa_topk_select")


def dsa_kv_insert(kv, positions, slots, kv_norm_w, pool, rms_eps: float = 1e-6, rope_base: float = 10000.0,
                  check_slots: bool = False, status=None, stream=None) -> None:
    """KV-cache insert (include/dsa_kv_insert.h). kv: bf16 [s_new, ld >= 576] device tensor
    (512 latent then 64 rotary values per row); positions: int32 [s_new]; slots: int64
    [s_new] (< 0 = skip); kv_norm_w: bf16 [512]; pool: uint8 [n_rows, 656]; status: uint32
    [1] device tensor or None."""
    s_new = int(kv.shape[0])
    if s_new > 0 and int(kv.stride(1)) != 1:
        raise DsaError(DSA_ERR_INVALID_ARG, "dsa_kv_insert: kv rows must be contiguous")
    ld = int(kv.stride(0)) if s_new > 0 else 576
    rc = library().dsa_kv_insert(_ptr(kv), ld, _ptr(positions), _ptr(slots), s_new, _ptr(kv_norm_w),
                                 float(rms_eps), float(rope_base), _ptr(pool), int(pool.shape[0]),
                                 DSA_KV_FLAG_CHECK_SLOTS if check_slots else 0, _ptr(status), _stream(stream))
    if rc != DSA_OK:
        raise DsaError(rc, "dsa_kv_insert")


def _refuse(where: str, what: str) -> None:
    raise DsaError(DSA_ERR_INVALID_ARG, f"{where}: {what}")


def _device(where: str, x) -> int:
    """The current CUDA device, where the library launches; x has to be on it."""
    if torch is None:
        _bind_torch()
    dev = x.get_device()
    if dev < 0 or dev != torch.cuda.current_device():
        _refuse(where, "every tensor must be on the current CUDA device")
    return dev


def _dense(where: str, dev: int, *specs) -> None:
    """Each (tensor, name, dtype, shape) is a contiguous tensor of that dtype and shape on device dev.  (The entry
    points look at their tensors in one expression first, which takes half the time, and come here for the reason.)"""
    for x, name, dtype, shape in specs:
        if x.dtype is not dtype or x.shape != shape or not x.is_contiguous() or x.get_device() != dev:
            _refuse(where, f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on the current CUDA "
                    f"device, got {x.dtype} {tuple(x.shape)} on {x.device}")


def _table_pitch(where: str, dev: int, x, n_req: int, cols: int) -> int:
    """Row pitch of a block table: int32 [n_req, cols] with dense rows."""
    ld, one = x.stride() if x.dim() == 2 else (0, 0)
    if (x.dtype is not _I32 or x.shape != (n_req, cols) or (cols > 1 and one != 1) or (n_req > 1 and ld < cols)
            or x.get_device() != dev):
        _refuse(where, "block_table must be an int32 [n_req, cols] tensor of dense rows that do not overlap, on the "
                "current CUDA device")
    return ld if n_req > 1 else cols


def _heads(where: str, dev: int, x, name: str, dtype, n: int, h: int, d: int):
    """(token pitch, head pitch) of a [n, h, d] tensor whose last dimension is dense."""
    if x.shape == (n, h, d) and x.dtype is dtype and x.get_device() == dev:
        ld, hd, one = x.stride()
        if one == 1 or n == 0:
            # a pitch that no second row uses may be anything: give the dense one
            return (ld if n > 1 else h * d), (hd if h > 1 else d)
    _refuse(where, f"{name} must be a {dtype} tensor of shape {(n, h, d)} with a dense last dimension on the "
            f"current CUDA device, got {x.dtype} {tuple(x.shape)} on {x.device}")


def dsa_page_map(ctx_lens, new_lens, block_table, free_pages, page_size: int, cu_new, kv_lens, positions, slots,
                 token_req, info, stream=None) -> None:
    """Page map of one serving step (include/dsa_page_map.h). ctx_lens, new_lens, kv_lens:
    int32 [n_req]; block_table: int32 [n_req, cols] (in and out; a row pitch is allowed);
    free_pages: int32 [n_free]; cu_new: int32 [n_req + 1]; positions, token_req (or None):
    int32 [n_tokens]; slots: int64 [n_tokens]; info: int32 [2] (pages taken, status bits)."""
    where = "dsa_page_map"
    n_req, n_tokens, cols = ctx_lens.shape[0], slots.shape[0], block_table.shape[-1]
    dev = _device(where, ctx_lens)
    t, r = (n_tokens,), (n_req,)
    if not (ctx_lens.dtype is new_lens.dtype is free_pages.dtype is cu_new.dtype is kv_lens.dtype is positions.dtype
            is info.dtype is _I32 and slots.dtype is _I64 and ctx_lens.shape == new_lens.shape == kv_lens.shape == r
            and positions.shape == slots.shape == t and cu_new.numel() == n_req + 1 and info.numel() == 2
            and ctx_lens.is_contiguous() and new_lens.is_contiguous() and free_pages.is_contiguous()
            and cu_new.is_contiguous() and kv_lens.is_contiguous() and positions.is_contiguous()
            and slots.is_contiguous() and info.is_contiguous()
            and new_lens.get_device() == free_pages.get_device() == cu_new.get_device() == kv_lens.get_device()
            == positions.get_device() == slots.get_device() == info.get_device() == dev):
        _dense(where, dev, (ctx_lens, "ctx_lens", _I32, r), (new_lens, "new_lens", _I32, r),
               (free_pages, "free_pages", _I32, (free_pages.numel(),)), (cu_new, "cu_new", _I32, (n_req + 1,)),
               (kv_lens, "kv_lens", _I32, r), (positions, "positions", _I32, t), (slots, "slots", _I64, t),
               (info, "info", _I32, (2,)))
    if token_req is not None:
        _dense(where, dev, (token_req, "token_req", _I32, t))
    ld = _table_pitch(where, dev, block_table, n_req, cols)
    rc = library().dsa_page_map(ctx_lens.data_ptr(), new_lens.data_ptr(), n_req, block_table.data_ptr(), ld, cols,
                                free_pages.data_ptr(), free_pages.numel(), page_size, n_tokens, cu_new.data_ptr(),
                                kv_lens.data_ptr(), positions.data_ptr(), slots.data_ptr(), _ptr(token_req),
                                info.data_ptr(), _stream(stream))
    if rc != DSA_OK:
        raise DsaError(rc, where)


def _kv8_pools(where, dev, k_pool, v_pool, k_scale, v_scale):
    shape = k_pool.shape
    if len(shape) != 4:
        _refuse(where, "k_pool must be [n_pages, h_kv, page_size, d]")
    if not (k_pool.dtype is v_pool.dtype is _U8 and k_scale.dtype is v_scale.dtype is _F32 and v_pool.shape == shape
            and k_scale.shape == v_scale.shape == shape[:2] and k_pool.is_contiguous() and v_pool.is_contiguous()
            and k_scale.is_contiguous() and v_scale.is_contiguous()
            and k_pool.get_device() == v_pool.get_device() == k_scale.get_device() == v_scale.get_device() == dev):
        _dense(where, dev, (k_pool, "k_pool", _U8, shape), (v_pool, "v_pool", _U8, shape),
               (k_scale, "k_scale", _F32, shape[:2]), (v_scale, "v_scale", _F32, shape[:2]))
    return shape


def dsa_kv8_insert(k, v, slots, k_pool, v_pool, k_scale, v_scale, status=None, stream=None) -> None:
    """Insert into the paged 8-bit cache (include/dsa_kv8.h). k, v: bf16 or fp16
    [n_tokens, h_kv, d] device tensors (token and head pitches allowed); slots: int64
    [n_tokens] (< 0 = skip); k_pool, v_pool: uint8 [n_pages, h_kv, page_size, d]; k_scale,
    v_scale: fp32 [n_pages, h_kv]; status: uint32 or int32 [1] device tensor or None."""
    where = "dsa_kv8_insert"
    dev = _device(where, k)
    n_pages, h_kv, page, d = _kv8_pools(where, dev, k_pool, v_pool, k_scale, v_scale)
    n, dtype = slots.shape[0], k.dtype
    if dtype not in _KV8_TYPES:
        _refuse(where, "k must be bfloat16 or float16")
    if not (slots.dtype is _I64 and slots.dim() == 1 and slots.is_contiguous() and slots.get_device() == dev):
        _dense(where, dev, (slots, "slots", _I64, (n,)))
    k_ld, k_hd = _heads(where, dev, k, "k", dtype, n, h_kv, d)
    v_ld, v_hd = _heads(where, dev, v, "v", dtype, n, h_kv, d)
    if status is not None and (status.element_size() != 4 or status.get_device() != dev):
        _refuse(where, "status must be a 32-bit word on the current CUDA device")
    rc = library().dsa_kv8_insert(k.data_ptr(), k_ld, k_hd, v.data_ptr(), v_ld, v_hd, slots.data_ptr(), n,
                                  _KV8_TYPES[dtype], k_pool.data_ptr(), v_pool.data_ptr(), k_scale.data_ptr(),
                                  v_scale.data_ptr(), n_pages, h_kv, page, d, _ptr(status), _stream(stream))
    if rc != DSA_OK:
        raise DsaError(rc, where)


def dsa_kv8_params_init(q, k_pool, block_table, max_q_len=None, **overrides) -> DsaKv8Params:
    """Parameters of dsa_kv8_attn_fwd for these tensors' shapes and type: q bf16 or fp16
    [n_tokens, h_q, d], k_pool uint8 [n_pages, h_kv, page_size, d], block_table
    [n_req, cols]. max_q_len: most query rows of a request (default: n_tokens);
    overrides: window, softmax_scale, flags."""
    where = "dsa_kv8_params_init"
    if torch is None:
        _bind_torch()
    if (q.dim() != 3 or k_pool.dim() != 4 or block_table.dim() != 2 or q.dtype not in _KV8_TYPES
            or q.shape[2] != k_pool.shape[3]):
        _refuse(where, "q, k_pool and block_table do not belong together")
    p = DsaKv8Params()
    n_pages, h_kv, page, d = (int(x) for x in k_pool.shape)
    rc = library().dsa_kv8_params_init(ctypes.byref(p), int(q.shape[0]), int(block_table.shape[0]), int(q.shape[1]),
                                       h_kv, d, page, n_pages, int(block_table.shape[1]))
    if rc != DSA_OK:
        raise DsaError(rc, where)
    p.type = _KV8_TYPES[q.dtype]
    if max_q_len is not None:
        p.max_q_len = int(max_q_len)
    for name, value in overrides.items():
        if name not in ("window", "softmax_scale", "flags"):
            _refuse(where, f"unknown parameter {name}")
        setattr(p, name, value)
    return p


def dsa_kv8_attn_workspace_size(p: DsaKv8Params, num_sms: int = 0) -> int:
    n = int(library().dsa_kv8_attn_workspace_size(ctypes.byref(p), int(num_sms)))
    if n == 0:
        raise DsaError(DSA_ERR_INVALID_ARG, "dsa_kv8_attn_workspace_size")
    return n


def _kv8_attn_args(where, q, k_pool, v_pool, k_scale, v_scale, block_table, cu_q, kv_lens, out, p, workspace, lse):
    """(device, arguments up to kv_lens, arguments from out to lse) of a call of the attention, checked."""
    dev = _device(where, q)
    if _kv8_pools(where, dev, k_pool, v_pool, k_scale, v_scale) != (p.n_pages, p.h_kv, p.page_size, p.d):
        _refuse(where, "the pools are not those of p")
    n, h_q, n_req, dtype = p.n_tokens, p.h_q, p.n_req, q.dtype
    if _KV8_TYPES.get(dtype) != p.type:
        _refuse(where, "q's type is not that of p")
    q_ld, q_hd = _heads(where, dev, q, "q", dtype, n, h_q, p.d)
    out_ld, out_hd = _heads(where, dev, out, "out", dtype, n, h_q, p.d)
    if not (cu_q.dtype is kv_lens.dtype is _I32 and cu_q.shape == (n_req + 1,) and kv_lens.shape == (n_req,)
            and cu_q.is_contiguous() and kv_lens.is_contiguous() and cu_q.get_device() == kv_lens.get_device() == dev):
        _dense(where, dev, (cu_q, "cu_q", _I32, (n_req + 1,)), (kv_lens, "kv_lens", _I32, (n_req,)))
    if lse is not None:
        _dense(where, dev, (lse, "lse", _F32, (n, h_q)))
    table_ld = _table_pitch(where, dev, block_table, n_req, p.table_cols)
    if workspace.get_device() != dev or not workspace.is_contiguous():
        _refuse(where, "the workspace must be contiguous and on the current CUDA device")
    return (dev, (q.data_ptr(), q_ld, q_hd, k_pool.data_ptr(), v_pool.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(),
                  block_table.data_ptr(), table_ld, cu_q.data_ptr(), kv_lens.data_ptr()),
            (out.data_ptr(), out_ld, out_hd, _ptr(lse)))


def dsa_kv8_attn_fwd(q, k_pool, v_pool, k_scale, v_scale, block_table, cu_q, kv_lens, out, p: DsaKv8Params, workspace,
                     lse=None, stream=None) -> None:
    """Attention over the paged 8-bit cache (include/dsa_kv8.h). q, out: bf16 or fp16
    [n_tokens, h_q, d] (token and head pitches allowed); pools and scales as
    dsa_kv8_insert; block_table: int32 [n_req, cols]; cu_q: int32 [n_req + 1]; kv_lens:
    int32 [n_req]; lse: fp32 [n_tokens, h_q] or None; workspace: uint8, 256-byte aligned
    (dsa_kv8_attn_workspace_size(p) bytes)."""
    where = "dsa_kv8_attn_fwd"
    _, front, back = _kv8_attn_args(where, q, k_pool, v_pool, k_scale, v_scale, block_table, cu_q, kv_lens, out, p, workspace, lse)
    rc = library().dsa_kv8_attn_fwd(*front, *back, ctypes.byref(p), workspace.data_ptr(), workspace.nbytes, _stream(stream))
    if rc != DSA_OK:
        raise DsaError(rc, where)


def dsa_kv8_prefix_workspace_size(p: DsaKv8Params, n_groups: int, num_sms: int = 0) -> int:
    n = int(library().dsa_kv8_prefix_workspace_size(ctypes.byref(p), int(n_groups), int(num_sms)))
    if n == 0:
        raise DsaError(DSA_ERR_INVALID_ARG, "dsa_kv8_prefix_workspace_size")
    return n


def dsa_kv8_prefix_attn_fwd(q, k_pool, v_pool, k_scale, v_scale, block_table, cu_q, kv_lens, cu_groups, prefix_lens, out,
                            p: DsaKv8Params, workspace, lse=None, stream=None) -> None:
    """dsa_kv8_attn_fwd for a batch whose requests share prefixes, whose pages are read once for all
    (include/dsa_kv8_prefix.h). cu_groups: int32 [n_groups + 1], the requests of each group; prefix_lens: int32
    [n_groups]; workspace: dsa_kv8_prefix_workspace_size(p, n_groups) bytes; the others as in dsa_kv8_attn_fwd."""
    where = "dsa_kv8_prefix_attn_fwd"
    dev, front, back = _kv8_attn_args(where, q, k_pool, v_pool, k_scale, v_scale, block_table, cu_q, kv_lens, out, p, workspace, lse)
    n = prefix_lens.shape[0] if prefix_lens.dim() == 1 else -1
    if not (cu_groups.dtype is prefix_lens.dtype is _I32 and n >= 0 and cu_groups.shape == (n + 1,) and cu_groups.is_contiguous()
            and prefix_lens.is_contiguous() and cu_groups.get_device() == prefix_lens.get_device() == dev):
        _dense(where, dev, (prefix_lens, "prefix_lens", _I32, (max(n, 0),)), (cu_groups, "cu_groups", _I32, (n + 1,)))
    rc = library().dsa_kv8_prefix_attn_fwd(*front, cu_groups.data_ptr(), prefix_lens.data_ptr(), n, *back, ctypes.byref(p),
                                           workspace.data_ptr(), workspace.nbytes, _stream(stream, dev))
    if rc != DSA_OK:
        raise DsaError(rc, where)


def dsa_qk_params_init(q, k=None, rotary_dim=None, rotary_start: int = 0, interleaved: bool = False,
                       rms_eps: float = 1e-6, rope_base: float = 10000.0) -> DsaQkParams:
    """Parameters of dsa_qk_norm_rope for these tensors' shapes and type: q bf16 or fp16 [n_tokens, h_q, d], k
    [n_tokens, h_k, d] or None. rotary_dim: how many of a head's values turn (default: d), from rotary_start on, in
    pairs of neighbours if `interleaved`, else with the value half of them further on."""
    where = "dsa_qk_params_init"
    if torch is None:
        _bind_torch()
    if q.dim() != 3 or q.dtype not in _KV8_TYPES:
        _refuse(where, "q must be a bfloat16 or float16 tensor [n_tokens, h_q, d]")
    n, h_q, d = (int(x) for x in q.shape)
    if k is not None and (k.dim() != 3 or k.dtype is not q.dtype or k.shape[0] != n or k.shape[2] != d):
        _refuse(where, f"k must be a {q.dtype} tensor [{n}, h_k, {d}]")
    p = DsaQkParams()
    rc = library().dsa_qk_params_init(ctypes.byref(p), n, h_q, 0 if k is None else int(k.shape[1]), d)
    if rc != DSA_OK:
        raise DsaError(rc, where)
    p.type = _KV8_TYPES[q.dtype]
    p.rotary_dim = d if rotary_dim is None else int(rotary_dim)
    p.rotary_start, p.flags = int(rotary_start), DSA_QK_FLAG_INTERLEAVED if interleaved else 0
    p.rms_eps, p.rope_base = float(rms_eps), float(rope_base)
    return p


def dsa_qk_norm_rope(q, k, positions, q_weight, k_weight, q_out, k_out, p: DsaQkParams, stream=None) -> None:
    """RMS norm and rotation of the heads of queries and keys (include/dsa_qk_norm_rope.h). q, q_out: bf16 or fp16
    [n_tokens, h_q, d]; k, k_out: [n_tokens, h_k, d], or None where p has no keys (token and head pitches allowed;
    an output may be its input itself); positions: int32 [n_tokens]; q_weight, k_weight: [d], or None for no norm."""
    where = "dsa_qk_norm_rope"
    dev = _device(where, q)
    n, h_q, h_k, d, dtype = p.n_tokens, p.h_q, p.h_k, p.d, q.dtype
    if _KV8_TYPES.get(dtype) != p.type:
        _refuse(where, "q's type is not that of p")
    q_ld, q_hd = _heads(where, dev, q, "q", dtype, n, h_q, d)
    qo_ld, qo_hd = (q_ld, q_hd) if q_out is q else _heads(where, dev, q_out, "q_out", dtype, n, h_q, d)
    k_at = ko_at = kw_at = qw_at = None
    k_ld = k_hd = ko_ld = ko_hd = 0
    if h_k:
        if k is None or k_out is None:
            _refuse(where, "k and k_out must be given where p has keys")
        k_ld, k_hd = _heads(where, dev, k, "k", dtype, n, h_k, d)
        ko_ld, ko_hd = (k_ld, k_hd) if k_out is k else _heads(where, dev, k_out, "k_out", dtype, n, h_k, d)
        k_at, ko_at = k.data_ptr(), k_out.data_ptr()
    elif k is not None or k_out is not None:
        _refuse(where, "k and k_out must be None where p has no keys")
    if not (positions.dtype is _I32 and positions.shape == (n,) and positions.is_contiguous() and positions.get_device() == dev):
        _dense(where, dev, (positions, "positions", _I32, (n,)))
    if q_weight is not None:
        if not (q_weight.dtype is dtype and q_weight.shape == (d,) and q_weight.is_contiguous() and q_weight.get_device() == dev):
            _dense(where, dev, (q_weight, "q_weight", dtype, (d,)))
        qw_at = q_weight.data_ptr()
    if k_weight is not None:
        if not (k_weight.dtype is dtype and k_weight.shape == (d,) and k_weight.is_contiguous() and k_weight.get_device() == dev):
            _dense(where, dev, (k_weight, "k_weight", dtype, (d,)))
        kw_at = k_weight.data_ptr()
    rc = library().dsa_qk_norm_rope(q.data_ptr(), q_ld, q_hd, k_at, k_ld, k_hd, positions.data_ptr(), qw_at, kw_at,
                                    q_out.data_ptr(), qo_ld, qo_hd, ko_at, ko_ld, ko_hd, ctypes.byref(p), _stream(stream, dev))
    if rc != DSA_OK:
        raise DsaError(rc, where)


def dsa_kv_gather(pool, block_table, cu_rows, out, page_size: int, lens=None, status=None, stream=None) -> None:
    """Latent rows read back from the cache (include/dsa_kv_gather.h). pool: uint8 [n_rows, 656]; block_table: int32
    [n_req, cols] (a row pitch is allowed); cu_rows: int32 [n_req + 1]; out: bf16 [n_out, ld >= 576]; lens: int32
    [n_req] or None; status: uint32 or int32 [1] device tensor or None."""
    where = "dsa_kv_gather"
    dev = _device(where, pool)
    rows = pool.shape[0] if pool.dim() == 2 else 0
    if not (pool.dtype is _U8 and pool.shape == (rows, DSA_ROW_BYTES) and pool.is_contiguous()):
        _dense(where, dev, (pool, "pool", _U8, (rows, DSA_ROW_BYTES)))
    n_req, cols = block_table.shape[0], block_table.shape[-1]
    table_ld = _table_pitch(where, dev, block_table, n_req, cols)
    if not (cu_rows.dtype is _I32 and cu_rows.shape == (n_req + 1,) and cu_rows.is_contiguous() and cu_rows.get_device() == dev):
        _dense(where, dev, (cu_rows, "cu_rows", _I32, (n_req + 1,)))
    if lens is not None:
        _dense(where, dev, (lens, "lens", _I32, (n_req,)))
    n_out, (ld, one) = out.shape[0], out.stride() if out.dim() == 2 else (0, 0)
    if out.dtype is not torch.bfloat16 or out.dim() != 2 or out.shape[1] < 576 or (n_out > 0 and one != 1) or out.get_device() != dev:
        _refuse(where, "out must be a bfloat16 tensor [n_out, >= 576] of dense rows on the current CUDA device")
    if n_out > 1 and ld < 576:
        _refuse(where, "the rows of out overlap")
    if status is not None and (status.element_size() != 4 or status.get_device() != dev):
        _refuse(where, "status must be a 32-bit word on the current CUDA device")
    rc = library().dsa_kv_gather(pool.data_ptr(), rows, block_table.data_ptr(), table_ld, cols, int(page_size),
                                 cu_rows.data_ptr(), _ptr(lens), n_req, out.data_ptr(), ld if n_out > 1 else 576, n_out,
                                 _ptr(status), _stream(stream, dev))
    if rc != DSA_OK:
        raise DsaError(rc, where)


def dsa_mla_params_init(q, k_nope, cu_q, max_q_len=None, max_kv_len=None, **overrides) -> DsaMlaParams:
    """Parameters of dsa_mla_prefill_fwd for these tensors' shapes and type: q bf16 or fp16 [n_tokens, h, 192], k_nope
    [n_keys, h, 128], cu_q int32 [n_req + 1]. Other fields (softmax_scale, flags) by keyword."""
    where = "dsa_mla_params_init"
    if torch is None:
        _bind_torch()
    if q.dim() != 3 or q.shape[2] != 192 or q.dtype not in _KV8_TYPES:
        _refuse(where, "q must be a bfloat16 or float16 tensor [n_tokens, h, 192]")
    if k_nope.dim() != 3 or k_nope.shape[1:] != (q.shape[1], 128) or k_nope.dtype is not q.dtype:
        _refuse(where, f"k_nope must be a {q.dtype} tensor [n_keys, {q.shape[1]}, 128]")
    if cu_q.dim() != 1 or cu_q.shape[0] < 1:
        _refuse(where, "cu_q must be [n_req + 1]")
    p = DsaMlaParams()
    rc = library().dsa_mla_params_init(ctypes.byref(p), q.shape[0], k_nope.shape[0], cu_q.shape[0] - 1, q.shape[1])
    if rc != DSA_OK:
        raise DsaError(rc, where)
    p.type = _KV8_TYPES[q.dtype]
    if max_q_len is not None:
        p.max_q_len = int(max_q_len)
    if max_kv_len is not None:
        p.max_kv_len = int(max_kv_len)
    for name, value in overrides.items():
        if name not in ("softmax_scale", "flags"):
            _refuse(where, f"unknown parameter {name}")
        setattr(p, name, value)
    return p


def dsa_mla_prefill_workspace_size(p: DsaMlaParams, num_sms: int = 0) -> int:
    n = int(library().dsa_mla_prefill_workspace_size(ctypes.byref(p), int(num_sms)))
    if n == 0:
        raise DsaError(DSA_ERR_INVALID_ARG, "dsa_mla_prefill_workspace_size")
    return n


def dsa_mla_prefill_fwd(q, k_nope, k_rope, v, cu_q, cu_kv, out, p: DsaMlaParams, workspace, lse=None, stream=None) -> None:
    """Latent attention with expanded keys and values (include/dsa_mla_prefill.h). q: bf16 or fp16 [n_tokens, h, 192];
    k_nope, v: [n_keys, h, 128]; k_rope: [n_keys, 64] (a row pitch is allowed); out: [n_tokens, h, 128] (token and head
    pitches allowed); cu_q, cu_kv: int32 [n_req + 1]; lse: fp32 [n_tokens, h] or None; workspace:
    dsa_mla_prefill_workspace_size(p) bytes on the device."""
    where = "dsa_mla_prefill_fwd"
    dev = _device(where, q)
    n, m, h, n_req, dtype = p.n_tokens, p.n_keys, p.h, p.n_req, q.dtype
    if _KV8_TYPES.get(dtype) != p.type:
        _refuse(where, "q's type is not that of p")
    q_ld, q_hd = _heads(where, dev, q, "q", dtype, n, h, 192)
    k_ld, k_hd = _heads(where, dev, k_nope, "k_nope", dtype, m, h, 128)
    v_ld, v_hd = _heads(where, dev, v, "v", dtype, m, h, 128)
    out_ld, out_hd = _heads(where, dev, out, "out", dtype, n, h, 128)
    r_ld, one = k_rope.stride() if k_rope.dim() == 2 else (0, 0)
    if k_rope.dtype is not dtype or k_rope.shape != (m, 64) or (m > 0 and one != 1) or k_rope.get_device() != dev:
        _refuse(where, f"k_rope must be a {dtype} tensor of shape {(m, 64)} of dense rows on the current CUDA device")
    if not (cu_q.dtype is cu_kv.dtype is _I32 and cu_q.shape == cu_kv.shape == (n_req + 1,) and cu_q.is_contiguous()
            and cu_kv.is_contiguous() and cu_q.get_device() == cu_kv.get_device() == dev):
        _dense(where, dev, (cu_q, "cu_q", _I32, (n_req + 1,)), (cu_kv, "cu_kv", _I32, (n_req + 1,)))
    if lse is not None:
        _dense(where, dev, (lse, "lse", _F32, (n, h)))
    if workspace.get_device() != dev or not workspace.is_contiguous():
        _refuse(where, "the workspace must be contiguous and on the current CUDA device")
    rc = library().dsa_mla_prefill_fwd(q.data_ptr(), q_ld, q_hd, k_nope.data_ptr(), k_ld, k_hd, k_rope.data_ptr(), r_ld if m > 1 else 64,
                                       v.data_ptr(), v_ld, v_hd, cu_q.data_ptr(), cu_kv.data_ptr(), out.data_ptr(), out_ld,
                                       out_hd, _ptr(lse), ctypes.byref(p), workspace.data_ptr(),
                                       workspace.nbytes, _stream(stream, dev))
    if rc != DSA_OK:
        raise DsaError(rc, where)


def dsa_sparse_attn_read_status(workspace, stream=None) -> int:
    st = ctypes.c_uint32(0)
    rc = library().dsa_sparse_attn_read_status(_ptr(workspace), ctypes.byref(st), _stream(stream))
    if rc != DSA_OK:
        raise DsaError(rc, "dsa_sparse_attn_read_status")
    return int(st.value)
