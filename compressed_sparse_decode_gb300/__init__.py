"""Python binding of libcsa, the GB300 (sm_103a) CSA decode library.

Argument marshalling only: every function below checks tensor devices,
dtypes and shapes, passes raw device pointers and the current CUDA stream to
the extern "C" entry point of the same name (include/csa.h), and raises
``CsaError`` on a non-zero status. All compute runs in the library's CUDA
kernels. There is no fallback: if libcsa.so is missing or cannot be loaded,
``load()`` raises.

PyTorch supplies device memory and streams only.
"""
from __future__ import annotations

import ctypes as C
import os
import threading

import torch

from ._build import LIB, build  # noqa: F401  (build() compiles libcsa.so in-tree)

HEADS, DIM, NOPE, ROPE, SCALE_BLOCK, RECORD_BYTES = 128, 512, 448, 64, 128, 592
IDX_HEADS, IDX_DIM = 64, 128
MAX_TOKENS_PER_SEQ, MAX_TOPK, MAX_SWA_WINDOW = 128, 2048, 512

OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_CUDA, ERR_TIMEOUT, ERR_BAD_INDEX = range(7)
FORMAT_FP8, FORMAT_FP4 = range(2)
FP4_RECORD_BYTES = 384
FORMAT_BYTES = (RECORD_BYTES, FP4_RECORD_BYTES)
OP_INDEXER, OP_TOPK, OP_ATTENTION, OP_HCA_ATTENTION, OP_DECODE_STEP = range(5)
OP_TREE_ATTENTION, OP_HCA_TREE_ATTENTION, OP_TREE_STEP, OP_VERIFY = range(5, 9)

EXPORTED = ["csa_workspace_bytes", "csa_indexer_logits", "csa_topk", "csa_gather_swa",
            "csa_sink_attention_decode", "hca_sink_attention_decode", "csa_decode_step",
            "csa_check_device_status", "csa_read_device_error", "csa_debug_set_wait_limit_ns",
            "csa_status_string", "csa_version", "csa_kernel_launches",
            "csa_sink_attention_decode_noalloc", "csa_pipeline_staging_bytes", "csa_pipeline_create",
            "csa_decode_step_host", "csa_pipeline_wait", "csa_pipeline_sync", "csa_pipeline_destroy",
            "csa_sink_attention_decode_ex", "hca_sink_attention_decode_ex", "csa_decode_step_ex",
            "csa_head_norm_rope", "csa_head_norm_rope_e4m3", "csa_cache_append", "csa_cache_read",
            "csa_sink_attention_decode_fp4", "hca_sink_attention_decode_fp4", "csa_decode_step_fp4",
            "csa_tree_attention_decode", "hca_tree_attention_decode", "csa_tree_decode_step", "csa_verify_drafts",
            "csa_cache_commit"]
PIPELINE_MAX_DEPTH = 4


class CsaError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: status {status} ({status_string(status)})")
        self.status = status


class csa_cache_desc(C.Structure):
    _fields_ = [("base", C.c_void_p), ("n_records", C.c_int64), ("seq_stride", C.c_int64),
                ("block_table", C.c_void_p), ("page_records", C.c_int32), ("max_pages", C.c_int32),
                ("seq_capacity", C.c_int32)]
    # what cache_desc knows of the tensors: format, device, block-table rows, and
    # whether the records had to be copied
    _fmt, _dev, _seqs, _copied = FORMAT_FP8, None, None, False


class csa_attention_epilogue(C.Structure):
    _fields_ = [("inverse_rope", C.c_int32), ("rope_theta", C.c_float), ("out_fp4", C.c_void_p),
                ("out_fp4_scale", C.c_void_p)]


class csa_norm_rope(C.Structure):
    _fields_ = [("norm", C.c_int32), ("eps", C.c_float), ("weight", C.c_void_p), ("rope_dim", C.c_int32),
                ("rope_theta", C.c_float)]


class csa_index_append(C.Structure):
    _fields_ = [("key", C.c_void_p), ("seq_stride", C.c_int64), ("token_stride", C.c_int64), ("k_idx", C.c_void_p),
                ("k_idx_scale", C.c_void_p), ("Ncap", C.c_int32)]


class csa_draft_tree(C.Structure):
    _fields_ = [("records", C.c_void_p), ("parent", C.c_void_p)]


_lib = None
_lock = threading.Lock()


def load(path: str | None = None):
    """Load libcsa.so (built in-tree by ``build()``); raises if it is absent."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = path or LIB
        if not os.path.exists(path):
            raise RuntimeError(f"libcsa.so not found at {path}: run compressed_sparse_decode_gb300.build()")
        lib = C.CDLL(path)
        P, i32, sz, f32 = C.c_void_p, C.c_int, C.c_size_t, C.c_float
        st = C.c_int
        lib.csa_version.restype = C.c_int
        lib.csa_kernel_launches.restype = C.c_uint64
        lib.csa_status_string.argtypes = [C.c_int]
        lib.csa_status_string.restype = C.c_char_p
        lib.csa_workspace_bytes.argtypes = [C.c_int, i32, i32, i32, i32]
        lib.csa_workspace_bytes.restype = sz
        lib.csa_indexer_logits.argtypes = [P] * 7 + [i32] * 4 + [P, P, P]
        lib.csa_indexer_logits.restype = st
        lib.csa_topk.argtypes = [P, P, P] + [i32] * 5 + [P, P, P, sz, P, P]
        lib.csa_topk.restype = st
        lib.csa_gather_swa.argtypes = [csa_cache_desc, P, i32, i32, P, P, P, i32, i32, i32, P, P, P, P]
        lib.csa_gather_swa.restype = st
        lib.csa_sink_attention_decode.argtypes = ([P, P, f32, csa_cache_desc, P, i32, i32, P, P, P, i32, i32, i32,
                                                   P, P, P, sz, P, P])
        lib.csa_sink_attention_decode.restype = st
        lib.hca_sink_attention_decode.argtypes = ([P, P, f32, csa_cache_desc, P, P, i32, i32, P, i32, i32, i32,
                                                   P, P, P, sz, P, P])
        lib.hca_sink_attention_decode.restype = st
        lib.csa_decode_step.argtypes = ([P] * 7 + [f32, csa_cache_desc, P, i32, i32, P, P] + [i32] * 5
                                        + [P, P, P, P, P, sz, P, P])
        lib.csa_decode_step.restype = st
        lib.csa_sink_attention_decode_noalloc.argtypes = ([P, P, f32, csa_cache_desc, P, i32, i32, P, P, P, i32, i32,
                                                           i32, P, P, P, P])
        lib.csa_sink_attention_decode_noalloc.restype = st
        EP = C.POINTER(csa_attention_epilogue)
        lib.csa_sink_attention_decode_ex.argtypes = ([P, P, f32, csa_cache_desc, P, i32, i32, P, P, P, i32, i32, i32,
                                                      P, P, EP, P, sz, P, P])
        lib.csa_sink_attention_decode_ex.restype = st
        lib.hca_sink_attention_decode_ex.argtypes = ([P, P, f32, csa_cache_desc, P, P, i32, i32, P, i32, i32, i32,
                                                      P, P, EP, P, sz, P, P])
        lib.hca_sink_attention_decode_ex.restype = st
        lib.csa_decode_step_ex.argtypes = ([P] * 7 + [f32, csa_cache_desc, P, i32, i32, P, P] + [i32] * 5
                                           + [P, P, P, P, EP, P, sz, P, P])
        lib.csa_decode_step_ex.restype = st
        lib.csa_pipeline_staging_bytes.argtypes = [i32, i32, i32]
        lib.csa_pipeline_staging_bytes.restype = sz
        lib.csa_pipeline_create.argtypes = [C.POINTER(C.c_void_p), i32, i32, i32, P, sz, P]
        lib.csa_pipeline_create.restype = st
        lib.csa_decode_step_host.argtypes = ([P] * 9 + [f32, csa_cache_desc, P, i32, i32, P] + [i32] * 3
                                             + [P, P, P, sz, P, C.POINTER(C.c_int64)])
        lib.csa_decode_step_host.restype = st
        lib.csa_pipeline_wait.argtypes = [P, C.c_int64]
        lib.csa_pipeline_wait.restype = st
        lib.csa_pipeline_sync.argtypes = [P]
        lib.csa_pipeline_sync.restype = st
        lib.csa_pipeline_destroy.argtypes = [P]
        lib.csa_pipeline_destroy.restype = st
        lib.csa_check_device_status.argtypes = [P, P, P]
        lib.csa_check_device_status.restype = st
        lib.csa_read_device_error.argtypes = [P, C.POINTER(C.c_int32), P]
        lib.csa_read_device_error.restype = st
        lib.csa_debug_set_wait_limit_ns.argtypes = [C.c_uint64]
        lib.csa_debug_set_wait_limit_ns.restype = None
        i64, NR = C.c_int64, C.POINTER(csa_norm_rope)
        lib.csa_head_norm_rope.argtypes = [P, i32, i64, i64, i64, P, i32, i32, i32, i32, NR, P, P, P]
        lib.csa_head_norm_rope.restype = st
        lib.csa_head_norm_rope_e4m3.argtypes = [P, i32, i64, i64, i64, P, i32, i32, i32, i32, NR, P, P, P, P]
        lib.csa_head_norm_rope_e4m3.restype = st
        lib.csa_cache_append.argtypes = [csa_cache_desc, i32, i32, P, i32, i64, i64, P, P, i32, i32, i32, NR,
                                         C.POINTER(csa_index_append), P, P]
        lib.csa_cache_append.restype = st
        lib.csa_cache_read.argtypes = [csa_cache_desc, i32, i32, P, P, i32, i32, P, P, P]
        lib.csa_cache_read.restype = st
        for name in ("csa_sink_attention_decode", "hca_sink_attention_decode", "csa_decode_step"):
            fp4, ex = getattr(lib, name + "_fp4"), getattr(lib, name + "_ex")
            fp4.argtypes, fp4.restype = ex.argtypes, st
        TR = C.POINTER(csa_draft_tree)
        lib.csa_tree_attention_decode.argtypes = ([P, P, f32, csa_cache_desc, i32, P, i32, i32, TR, P, P, P, i32, i32,
                                                   i32, P, P, EP, P, sz, P, P])
        lib.csa_tree_attention_decode.restype = st
        lib.hca_tree_attention_decode.argtypes = ([P, P, f32, csa_cache_desc, i32, P, P, i32, i32, TR, P, i32, i32,
                                                   i32, P, P, EP, P, sz, P, P])
        lib.hca_tree_attention_decode.restype = st
        lib.csa_tree_decode_step.argtypes = ([P] * 7 + [f32, csa_cache_desc, i32, P, i32, i32, TR, P, P] + [i32] * 5
                                             + [P, P, P, P, EP, P, sz, P, P])
        lib.csa_tree_decode_step.restype = st
        lib.csa_verify_drafts.argtypes = [P, i32, i64, i64, P, i32] + [P] * 5 + [i32] * 3 + [P] * 4 + [sz, P, P]
        lib.csa_verify_drafts.restype = st
        lib.csa_cache_commit.argtypes = [csa_cache_desc, i32, i32, P, i32, P, P, P, i32, i32, P, P]
        lib.csa_cache_commit.restype = st
        _lib = lib
        return lib


def status_string(status: int) -> str:
    return load().csa_status_string(int(status)).decode()


def csa_version() -> int:
    return int(load().csa_version())


def csa_kernel_launches() -> int:
    """Kernels launched so far by this process through the library."""
    return int(load().csa_kernel_launches())


def _check(status: int, where: str):
    if status != OK:
        raise CsaError(status, where)


def _stream(stream) -> int:
    if stream is None:  # the handle itself: a Stream object costs 3 us a call
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t: torch.Tensor | None, name: str, dtype=None, shape=None):
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t.data_ptr()


_status_words: dict[int, torch.Tensor] = {}
_status_ptrs: dict[int, int] = {}  # their addresses (the words live as long as the process)


def status_word(device=None) -> torch.Tensor:
    """The binding's default status word for a device: one int32 in device
    memory (created zeroed on first use), passed to the library by every call
    below that is not given its own ``status`` tensor. Make it, by this call or any
    other, before the first capture of a graph: made inside one, it is zeroed by every
    replay, not at once."""
    dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    if dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    with _lock:
        w = _status_words.get(dev.index)
        if w is None:
            w = torch.zeros(1, dtype=torch.int32, device=dev)
            _status_words[dev.index] = w
            _status_ptrs[dev.index] = w.data_ptr()
    return w


def _status(status, device) -> int:
    if status is None:
        status = status_word(device)
    return _ptr(status, "status", torch.int32, (1,))


def cache_desc(records: torch.Tensor, seq_capacity: int, seq_stride: int = 0,
               block_table: torch.Tensor | None = None, page_records: int = 0,
               fmt: int = FORMAT_FP8) -> csa_cache_desc:
    """Describe a cache of latent records: ``records`` is uint8 [n, 592], or of
    another number of dimensions and whole records in all (a flat buffer,
    [B, Ncap, 592]); contiguous mode uses ``seq_stride``, paged mode a
    ``block_table`` [B, max_pages] int32 and ``page_records``. With
    ``fmt=FORMAT_FP4`` the records are the 384-byte 4-bit ones; the calls below
    take the format from the description. Records that are not contiguous are
    described by a copy, as they are now: nothing can be appended to it, and what is
    written to the tensor later is not in it."""
    if fmt not in (FORMAT_FP8, FORMAT_FP4):
        raise ValueError(f"unknown record format {fmt}")
    size = FORMAT_BYTES[fmt]
    last = records.shape[-1] if records.dim() > 1 else size  # (a flat buffer says nothing about its records)
    if records.numel() % size or (last != size and (records.dim() == 2 or last in FORMAT_BYTES)):
        raise ValueError(f"records must be [n, {size}] uint8")
    rec = records.reshape(-1, size) if records.dim() != 2 else records
    _ptr(rec, "records", torch.uint8)
    d = csa_cache_desc()
    d.base = rec.data_ptr()
    d.n_records = rec.shape[0]
    d.seq_stride = int(seq_stride)
    d.seq_capacity = int(seq_capacity)
    if block_table is not None:
        _ptr(block_table, "block_table", torch.int32)
        if block_table.get_device() != rec.get_device():
            raise ValueError(f"block_table is on cuda:{block_table.get_device()}, the records on cuda:{rec.get_device()}")
        d.block_table = block_table.data_ptr()
        d.page_records = int(page_records)
        d.max_pages = int(block_table.shape[-1])
    d._keepalive = (rec, block_table)  # noqa: SLF001
    d._fmt = fmt  # noqa: SLF001
    d._dev = rec.get_device()  # noqa: SLF001
    d._seqs = None if block_table is None else block_table.numel() // max(1, block_table.shape[-1])  # noqa: SLF001
    d._copied = rec.data_ptr() != records.data_ptr()  # noqa: SLF001
    return d


def _format(comp: csa_cache_desc, fmt: int, where: str) -> csa_cache_desc:
    """The description itself, if it describes records of format ``fmt``."""
    if comp._fmt != fmt:
        raise ValueError(f"{where} reads {FORMAT_BYTES[fmt]}-byte records; the cache holds the other format")
    return comp


def csa_workspace_bytes(op: int, B: int, T: int, Ncap: int, k: int) -> int:
    return int(load().csa_workspace_bytes(int(op), B, T, Ncap, k))


def workspace(op: int, B: int, T: int, Ncap: int, k: int, device=None) -> torch.Tensor | None:
    """Allocate (through PyTorch) a workspace of the size the library asks for."""
    n = csa_workspace_bytes(op, B, T, Ncap, k)
    if n == 0:
        return None
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def csa_indexer_logits(q_idx, q_idx_scale, w_idx, k_idx, k_idx_scale, q_pos, n_comp, m: int,
                       logits: torch.Tensor | None = None, stream=None, status=None) -> torch.Tensor:
    B, T = q_pos.shape
    Ncap = k_idx.shape[1]
    if logits is None:
        logits = torch.empty((B, T, Ncap), dtype=torch.float32, device=q_idx.device)
    u8 = (torch.uint8, torch.float8_e4m3fn)
    args = [_ptr(q_idx, "q_idx", u8, (B, T, IDX_HEADS, IDX_DIM)),
            _ptr(q_idx_scale, "q_idx_scale", torch.float32, (B, T, IDX_HEADS)),
            _ptr(w_idx, "w_idx", torch.float32, (B, T, IDX_HEADS)),
            _ptr(k_idx, "k_idx", u8, (B, Ncap, IDX_DIM)),
            _ptr(k_idx_scale, "k_idx_scale", torch.float32, (B, Ncap)),
            _ptr(q_pos, "q_pos", torch.int32, (B, T)), _ptr(n_comp, "n_comp", torch.int32, (B,))]
    _check(load().csa_indexer_logits(*args, B, T, Ncap, int(m),
                                     _ptr(logits, "logits", torch.float32, (B, T, Ncap)),
                                     _status(status, q_idx.device), _stream(stream)),
           "csa_indexer_logits")
    return logits


def csa_topk(logits, q_pos, n_comp, m: int, k: int, topk_idx=None, topk_cnt=None, ws=None, stream=None,
             status=None):
    B, T, Ncap = logits.shape
    dev = logits.device
    if topk_idx is None:
        topk_idx = torch.empty((B, T, k), dtype=torch.int32, device=dev)
    if topk_cnt is None:
        topk_cnt = torch.empty((B, T), dtype=torch.int32, device=dev)
    if ws is None:
        ws = workspace(OP_TOPK, B, T, Ncap, k, dev)
    _check(load().csa_topk(_ptr(logits, "logits", torch.float32), _ptr(q_pos, "q_pos", torch.int32, (B, T)),
                           _ptr(n_comp, "n_comp", torch.int32, (B,)), B, T, Ncap, int(m), int(k),
                           _ptr(topk_idx, "topk_idx", torch.int32, (B, T, k)),
                           _ptr(topk_cnt, "topk_cnt", torch.int32, (B, T)),
                           _ptr(ws, "workspace", torch.uint8), 0 if ws is None else ws.numel(),
                           _status(status, dev), _stream(stream)),
           "csa_topk")
    return topk_idx, topk_cnt


def csa_gather_swa(comp: csa_cache_desc, swa_ring, W: int, topk_idx, topk_cnt, q_pos, kv_out=None, kv_cnt=None,
                   stream=None, status=None):
    B, T, k = topk_idx.shape
    R = swa_ring.shape[1]
    dev = swa_ring.device
    if kv_out is None:
        kv_out = torch.empty((B, T, k + W, RECORD_BYTES), dtype=torch.uint8, device=dev)
    if kv_cnt is None:
        kv_cnt = torch.empty((B, T), dtype=torch.int32, device=dev)
    _check(load().csa_gather_swa(_format(comp, FORMAT_FP8, "csa_gather_swa"), _ptr(swa_ring, "swa_ring", torch.uint8, (B, R, RECORD_BYTES)), R, int(W),
                                 _ptr(topk_idx, "topk_idx", torch.int32), _ptr(topk_cnt, "topk_cnt", torch.int32, (B, T)),
                                 _ptr(q_pos, "q_pos", torch.int32, (B, T)), B, T, k,
                                 _ptr(kv_out, "kv_out", torch.uint8, (B, T, k + W, RECORD_BYTES)),
                                 _ptr(kv_cnt, "kv_cnt", torch.int32, (B, T)), _status(status, dev), _stream(stream)),
           "csa_gather_swa")
    return kv_out, kv_cnt


def _epilogue(B: int, T: int, dev, inverse_rope: bool, rope_theta: float, fp4_out: bool, out_fp4, out_fp4_scale):
    """The output-epilogue struct (None when neither step is asked for) and
    the E2M1 output tensors."""
    if not inverse_rope and not fp4_out:
        return None, None, None
    if fp4_out:
        if out_fp4 is None:
            out_fp4 = torch.empty((B, T, HEADS, DIM // 2), dtype=torch.uint8, device=dev)
        if out_fp4_scale is None:
            out_fp4_scale = torch.empty((B, T, HEADS, DIM // SCALE_BLOCK), dtype=torch.float32, device=dev)
    epi = csa_attention_epilogue(1 if inverse_rope else 0, float(rope_theta),
                                 _ptr(out_fp4, "out_fp4", torch.uint8, (B, T, HEADS, DIM // 2)) if fp4_out else None,
                                 _ptr(out_fp4_scale, "out_fp4_scale", torch.float32,
                                      (B, T, HEADS, DIM // SCALE_BLOCK)) if fp4_out else None)
    return epi, out_fp4, out_fp4_scale


def csa_sink_attention_decode(q, sink, softmax_scale: float, comp: csa_cache_desc, swa_ring, W: int, topk_idx,
                              topk_cnt, q_pos, out=None, lse=None, ws=None, stream=None, status=None,
                              inverse_rope: bool = False, rope_theta: float = 10000.0, fp4_out: bool = False,
                              out_fp4=None, out_fp4_scale=None):
    """Returns (out, lse); with fp4_out, ((out_fp4, out_fp4_scale), lse).
    inverse_rope / fp4_out select the output epilogue (csa_attention_epilogue)."""
    B, T = q_pos.shape
    k = topk_idx.shape[2]
    R = swa_ring.shape[1]
    dev = q.device
    epi, out_fp4, out_fp4_scale = _epilogue(B, T, dev, inverse_rope, rope_theta, fp4_out, out_fp4, out_fp4_scale)
    if out is None and not fp4_out:
        out = torch.empty((B, T, HEADS, DIM), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((B, T, HEADS), dtype=torch.float32, device=dev)
    if ws is None:
        ws = workspace(OP_ATTENTION, B, T, comp.seq_capacity, k, dev)
    args = [_ptr(q, "q", torch.bfloat16, (B, T, HEADS, DIM)), _ptr(sink, "sink", torch.float32, (HEADS,)),
            float(softmax_scale), _format(comp, FORMAT_FP8, "csa_sink_attention_decode"),
            _ptr(swa_ring, "swa_ring", torch.uint8, (B, R, RECORD_BYTES)), R, int(W),
            _ptr(topk_idx, "topk_idx", torch.int32, (B, T, k)), _ptr(topk_cnt, "topk_cnt", torch.int32, (B, T)),
            _ptr(q_pos, "q_pos", torch.int32, (B, T)), B, T, k,
            _ptr(out, "out", torch.bfloat16, (B, T, HEADS, DIM)), _ptr(lse, "lse", torch.float32, (B, T, HEADS))]
    tail = [_ptr(ws, "workspace", torch.uint8), 0 if ws is None else ws.numel(), _status(status, dev), _stream(stream)]
    if epi is None:
        _check(load().csa_sink_attention_decode(*args, *tail), "csa_sink_attention_decode")
    else:
        _check(load().csa_sink_attention_decode_ex(*args, C.byref(epi), *tail), "csa_sink_attention_decode_ex")
    return ((out_fp4, out_fp4_scale) if fp4_out else out), lse


def csa_sink_attention_decode_noalloc(q, sink, softmax_scale: float, comp: csa_cache_desc, swa_ring, W: int, topk_idx,
                                      topk_cnt, q_pos, out=None, lse=None, stream=None, status=None):
    """csa_sink_attention_decode without a workspace: for callers that cannot
    allocate device memory on the decode path (see include/csa.h); the split
    partials use the library's static device scratch."""
    B, T = q_pos.shape
    k = topk_idx.shape[2]
    R = swa_ring.shape[1]
    dev = q.device
    if out is None:
        out = torch.empty((B, T, HEADS, DIM), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((B, T, HEADS), dtype=torch.float32, device=dev)
    _check(load().csa_sink_attention_decode_noalloc(
        _ptr(q, "q", torch.bfloat16, (B, T, HEADS, DIM)), _ptr(sink, "sink", torch.float32, (HEADS,)),
        float(softmax_scale), _format(comp, FORMAT_FP8, "csa_sink_attention_decode_noalloc"),
        _ptr(swa_ring, "swa_ring", torch.uint8, (B, R, RECORD_BYTES)), R, int(W),
        _ptr(topk_idx, "topk_idx", torch.int32, (B, T, k)), _ptr(topk_cnt, "topk_cnt", torch.int32, (B, T)),
        _ptr(q_pos, "q_pos", torch.int32, (B, T)), B, T, k,
        _ptr(out, "out", torch.bfloat16, (B, T, HEADS, DIM)), _ptr(lse, "lse", torch.float32, (B, T, HEADS)),
        _status(status, dev), _stream(stream)), "csa_sink_attention_decode_noalloc")
    return out, lse


def hca_sink_attention_decode(q, sink, softmax_scale: float, comp: csa_cache_desc, n_comp, swa_ring, W: int, q_pos,
                              m_hca: int = 128, out=None, lse=None, ws=None, stream=None, status=None,
                              inverse_rope: bool = False, rope_theta: float = 10000.0, fp4_out: bool = False,
                              out_fp4=None, out_fp4_scale=None):
    """Returns (out, lse); with fp4_out, ((out_fp4, out_fp4_scale), lse)."""
    B, T = q_pos.shape
    R = swa_ring.shape[1]
    dev = q.device
    epi, out_fp4, out_fp4_scale = _epilogue(B, T, dev, inverse_rope, rope_theta, fp4_out, out_fp4, out_fp4_scale)
    if out is None and not fp4_out:
        out = torch.empty((B, T, HEADS, DIM), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((B, T, HEADS), dtype=torch.float32, device=dev)
    if ws is None:
        ws = workspace(OP_HCA_ATTENTION, B, T, comp.seq_capacity, 0, dev)
    args = [_ptr(q, "q", torch.bfloat16, (B, T, HEADS, DIM)), _ptr(sink, "sink", torch.float32, (HEADS,)),
            float(softmax_scale), _format(comp, FORMAT_FP8, "hca_sink_attention_decode"), _ptr(n_comp, "n_comp", torch.int32, (B,)),
            _ptr(swa_ring, "swa_ring", torch.uint8, (B, R, RECORD_BYTES)), R, int(W),
            _ptr(q_pos, "q_pos", torch.int32, (B, T)), B, T, int(m_hca),
            _ptr(out, "out", torch.bfloat16, (B, T, HEADS, DIM)), _ptr(lse, "lse", torch.float32, (B, T, HEADS))]
    tail = [_ptr(ws, "workspace", torch.uint8), 0 if ws is None else ws.numel(), _status(status, dev), _stream(stream)]
    if epi is None:
        _check(load().hca_sink_attention_decode(*args, *tail), "hca_sink_attention_decode")
    else:
        _check(load().hca_sink_attention_decode_ex(*args, C.byref(epi), *tail), "hca_sink_attention_decode_ex")
    return ((out_fp4, out_fp4_scale) if fp4_out else out), lse


def csa_decode_step(q_idx, q_idx_scale, w_idx, k_idx, k_idx_scale, q, sink, softmax_scale: float,
                    comp: csa_cache_desc, swa_ring, W: int, q_pos, n_comp, m: int, k: int, out=None, lse=None,
                    topk_idx=None, topk_cnt=None, ws=None, stream=None, status=None, inverse_rope: bool = False,
                    rope_theta: float = 10000.0, fp4_out: bool = False, out_fp4=None, out_fp4_scale=None):
    """Returns (out, lse); with fp4_out, ((out_fp4, out_fp4_scale), lse)."""
    B, T = q_pos.shape
    Ncap = k_idx.shape[1]
    R = swa_ring.shape[1]
    dev = q.device
    epi, out_fp4, out_fp4_scale = _epilogue(B, T, dev, inverse_rope, rope_theta, fp4_out, out_fp4, out_fp4_scale)
    if out is None and not fp4_out:
        out = torch.empty((B, T, HEADS, DIM), dtype=torch.bfloat16, device=dev)
    if lse is None:
        lse = torch.empty((B, T, HEADS), dtype=torch.float32, device=dev)
    if ws is None:
        ws = workspace(OP_DECODE_STEP, B, T, Ncap, k, dev)
    u8 = (torch.uint8, torch.float8_e4m3fn)
    args = [_ptr(q_idx, "q_idx", u8, (B, T, IDX_HEADS, IDX_DIM)),
            _ptr(q_idx_scale, "q_idx_scale", torch.float32, (B, T, IDX_HEADS)),
            _ptr(w_idx, "w_idx", torch.float32, (B, T, IDX_HEADS)), _ptr(k_idx, "k_idx", u8, (B, Ncap, IDX_DIM)),
            _ptr(k_idx_scale, "k_idx_scale", torch.float32, (B, Ncap)),
            _ptr(q, "q", torch.bfloat16, (B, T, HEADS, DIM)), _ptr(sink, "sink", torch.float32, (HEADS,)),
            float(softmax_scale), _format(comp, FORMAT_FP8, "csa_decode_step"),
            _ptr(swa_ring, "swa_ring", torch.uint8, (B, R, RECORD_BYTES)), R, int(W),
            _ptr(q_pos, "q_pos", torch.int32, (B, T)), _ptr(n_comp, "n_comp", torch.int32, (B,)),
            B, T, Ncap, int(m), int(k),
            _ptr(out, "out", torch.bfloat16, (B, T, HEADS, DIM)), _ptr(lse, "lse", torch.float32, (B, T, HEADS)),
            _ptr(topk_idx, "topk_idx", torch.int32, (B, T, k)), _ptr(topk_cnt, "topk_cnt", torch.int32, (B, T))]
    tail = [_ptr(ws, "workspace", torch.uint8), 0 if ws is None else ws.numel(), _status(status, dev), _stream(stream)]
    if epi is None:
        _check(load().csa_decode_step(*args, *tail), "csa_decode_step")
    else:
        _check(load().csa_decode_step_ex(*args, C.byref(epi), *tail), "csa_decode_step_ex")
    return ((out_fp4, out_fp4_scale) if fp4_out else out), lse


_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}


def _own_status(status, dev: int) -> int:
    """Address of the status word: the caller's, or the device's default one."""
    if status is not None:
        return _arg(status, "status", torch.int32, (1,), dev)
    return _status_ptrs.get(dev) or _status(None, torch.device("cuda", dev))


def _dev(t: torch.Tensor, name: str) -> int:
    """Index of the CUDA device that ``t`` is on, which has to be the current one
    (the library launches there)."""
    i = t.get_device()
    if i < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if i != torch._C._cuda_getDevice():
        raise ValueError(f"{name} is on cuda:{i}, not on the current device: make that device current for the call")
    return i


def _on(stream, dev: int) -> int:
    """Handle of the stream, or of the current one of device ``dev``."""
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)


def _arg(t: torch.Tensor, name: str, dtype, shape, dev: int) -> int:
    """Data pointer of a dense tensor of this dtype and shape on device ``dev``."""
    if t.get_device() != dev or t.dtype != dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on cuda:{dev}: got "
                         f"{t.dtype} {tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _codes(t: torch.Tensor, name: str, shape, dev: int) -> int:
    """_arg for E4M3 codes, as bytes or as torch's type."""
    return _arg(t, name, torch.float8_e4m3fn if t.dtype == torch.float8_e4m3fn else torch.uint8, shape, dev)


def _rows(t: torch.Tensor, name: str, dev: int):
    """(data pointer, element type, strides of the leading dimensions) of a
    floating tensor whose last dimension is dense; 0 for a dimension of one
    element (PyTorch leaves any number there)."""
    dt = _DTYPES.get(t.dtype)
    *s, last = t.stride()
    if dt is None or last != 1 or t.get_device() != dev:
        raise ValueError(f"{name} must be a bf16, fp16 or fp32 tensor on cuda:{dev} with a dense last dimension: got "
                         f"{t.dtype} {tuple(t.shape)}, strides {t.stride()}, on {t.device}")
    shape = t.shape
    if 1 in shape:
        s = [0 if n == 1 else v for n, v in zip(shape, s)]
    return t.data_ptr(), dt, s


def _new(make, shape, dtype, device, stream) -> torch.Tensor:
    """make(shape) (torch.empty or torch.zeros) for a call on ``stream``: from
    that stream's memory and, where it writes, in its order."""
    if stream is None:
        return make(shape, dtype=dtype, device=device)
    s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(_stream(stream), device=device)
    with torch.cuda.stream(s):
        return make(shape, dtype=dtype, device=device)


def _attention_outputs(B: int, T: int, device, stream, out, lse, fp4_out: bool, out_fp4, out_fp4_scale):
    """The outputs of an attention call; those that the caller did not pass, made here."""
    if fp4_out:
        if out_fp4 is None:
            out_fp4 = _new(torch.empty, (B, T, HEADS, DIM // 2), torch.uint8, device, stream)
        if out_fp4_scale is None:
            out_fp4_scale = _new(torch.empty, (B, T, HEADS, DIM // SCALE_BLOCK), torch.float32, device, stream)
        if out_fp4.device != device or out_fp4_scale.device != device:
            raise ValueError(f"out_fp4 and out_fp4_scale must be on {device}")
    elif out is None:
        out = _new(torch.empty, (B, T, HEADS, DIM), torch.bfloat16, device, stream)
    if lse is None:
        lse = _new(torch.empty, (B, T, HEADS), torch.float32, device, stream)
    return out, lse, out_fp4, out_fp4_scale


def _own_workspace(op: int, B: int, T: int, Ncap: int, k: int, device, stream):
    n = csa_workspace_bytes(op, B, T, Ncap, k)
    return _new(torch.empty, (n,), torch.uint8, device, stream) if n else None


def _how(norm: bool, weight, eps: float, rope_dim: int, rope_theta: float, D: int, dev: int) -> csa_norm_rope:
    w = _arg(weight, "weight", torch.float32, (D,), dev) if weight is not None else None
    return csa_norm_rope(1 if norm else 0, eps, w, rope_dim, rope_theta)


def csa_head_norm_rope(x, pos, weight=None, norm: bool = True, eps: float = 1e-6, rope_dim: int = ROPE,
                       rope_theta: float = 10000.0, out=None, stream=None, status=None) -> torch.Tensor:
    """RMS norm of every head of ``x`` [B, T, H, D] (bf16, fp16 or fp32; any
    strides but a dense last dimension) and the rotation of its last
    ``rope_dim`` values at ``pos`` [B, T] int32, in one pass; BF16 [B, T, H, D].
    Rows of tokens with pos < 0 are left as they were: pass an ``out`` of your
    own with padded batches. ``rope_dim=0`` rotates nothing, ``norm=False``
    normalises nothing; ``out`` may be ``x``."""
    B, T, H, D = x.shape
    dev = _dev(x, "x")
    if out is None:
        out = _new(torch.empty, (B, T, H, D), torch.bfloat16, x.device, stream)
    ptr, dt, s = _rows(x, "x", dev)
    _check((_lib or load()).csa_head_norm_rope(ptr, dt, *s,
                                     _arg(pos, "pos", torch.int32, (B, T), dev), B, T, H, D,
                                     _how(norm, weight, eps, rope_dim, rope_theta, D, dev),
                                     _arg(out, "out", torch.bfloat16, (B, T, H, D), dev), _own_status(status, dev),
                                     _on(stream, dev)), "csa_head_norm_rope")
    return out


def csa_head_norm_rope_e4m3(x, pos, weight=None, norm: bool = True, eps: float = 1e-6, rope_dim: int = ROPE,
                            rope_theta: float = 10000.0, codes=None, scale=None, stream=None, status=None):
    """csa_head_norm_rope with E4M3 output: (codes [B, T, H, D] uint8, or
    float8_e4m3fn where ``codes`` is; scale [B, T, H] fp32), the form csa_indexer_logits reads its queries in."""
    B, T, H, D = x.shape
    dev = _dev(x, "x")
    if codes is None:
        codes = _new(torch.empty, (B, T, H, D), torch.uint8, x.device, stream)
    if scale is None:
        scale = _new(torch.empty, (B, T, H), torch.float32, x.device, stream)
    ptr, dt, s = _rows(x, "x", dev)
    _check((_lib or load()).csa_head_norm_rope_e4m3(ptr, dt, *s,
                                          _arg(pos, "pos", torch.int32, (B, T), dev), B, T, H, D,
                                          _how(norm, weight, eps, rope_dim, rope_theta, D, dev),
                                          _codes(codes, "codes", (B, T, H, D), dev),
                                          _arg(scale, "scale", torch.float32, (B, T, H), dev),
                                          _own_status(status, dev), _on(stream, dev)), "csa_head_norm_rope_e4m3")
    return codes, scale


def csa_cache_append(cache: csa_cache_desc, x, first, count=None, ring: bool = False, norm: bool = False, weight=None,
                     eps: float = 1e-6, rope_theta: float | None = 10000.0, pos_stride: int = 1, key=None,
                     k_idx=None, k_idx_scale=None, stream=None, status=None) -> None:
    """Append the latents ``x`` [B, T, 512] (bf16, fp16 or fp32) as entries
    first[b] .. first[b] + count[b] of their sequences, in the cache's own
    format, normalised (``norm``) and rotated at entry * pos_stride
    (``rope_theta=None``: not rotated) on the way. ``ring``: entry modulo the
    cache's capacity. ``key`` [B, T, 128] adds the entries' indexer keys to
    ``k_idx`` [B, Ncap, 128] and ``k_idx_scale`` [B, Ncap]. See include/csa.h."""
    B, T, D = x.shape
    dev = _dev(x, "x")
    if D != DIM:
        raise ValueError(f"x has shape {tuple(x.shape)}, expected [B, T, {DIM}]")
    if cache._copied:
        raise ValueError("the cache's records were not contiguous: the description holds a copy of them")
    ptr, dt, s = _rows(x, "x", dev)
    idx = None
    if (key is None) != (k_idx is None) or (key is None) != (k_idx_scale is None):
        raise ValueError("key, k_idx and k_idx_scale go together")
    if key is not None:
        ncap = k_idx.shape[1]
        if key.shape != (B, T, IDX_DIM) or key.dtype != x.dtype:
            raise ValueError(f"key must be a {x.dtype} tensor of shape {(B, T, IDX_DIM)}: got {key.dtype} "
                             f"{tuple(key.shape)}")
        key_ptr, _, key_s = _rows(key, "key", dev)
        idx = csa_index_append(key_ptr, *key_s, _codes(k_idx, "k_idx", (B, ncap, IDX_DIM), dev),
                               _arg(k_idx_scale, "k_idx_scale", torch.float32, (B, ncap), dev), ncap)
    rope_dim, theta = (0, 0.0) if rope_theta is None else (ROPE, rope_theta)
    _check((_lib or load()).csa_cache_append(_cache(cache, B, dev), cache._fmt, 1 if ring else 0, ptr, dt, *s,
                                             _arg(first, "first", torch.int32, (B,), dev),
                                             None if count is None else _arg(count, "count", torch.int32, (B,), dev),
                                             B, T, pos_stride, _how(norm, weight, eps, rope_dim, theta, DIM, dev), idx,
                                             _own_status(status, dev), _on(stream, dev)), "csa_cache_append")


def csa_cache_read(cache: csa_cache_desc, first, count, T: int, ring: bool = False, out=None, stream=None,
                   status=None) -> torch.Tensor:
    """The entries first[b] .. first[b] + count[b] (``count`` None: T of them) of
    each sequence as BF16 latents [B, T, 512]; rows behind a sequence's count
    are left as they were (zero in an ``out`` made here)."""
    dev = _dev(first, "first")
    B = first.shape[0]
    if out is None:
        out = _new(torch.zeros, (B, T, DIM), torch.bfloat16, first.device, stream)
    _check((_lib or load()).csa_cache_read(_cache(cache, B, dev), cache._fmt, 1 if ring else 0,
                                 _arg(first, "first", torch.int32, (B,), dev),
                                 None if count is None else _arg(count, "count", torch.int32, (B,), dev), B, T,
                                 _arg(out, "out", torch.bfloat16, (B, T, DIM), dev), _own_status(status, dev),
                                 _on(stream, dev)), "csa_cache_read")
    return out


def csa_sink_attention_decode_fp4(q, sink, softmax_scale: float, comp: csa_cache_desc, swa_ring, W: int, topk_idx,
                                  topk_cnt, q_pos, out=None, lse=None, ws=None, stream=None, status=None,
                                  inverse_rope: bool = False, rope_theta: float = 10000.0, fp4_out: bool = False,
                                  out_fp4=None, out_fp4_scale=None):
    """csa_sink_attention_decode over caches of 4-bit records (``comp`` made with
    ``fmt=FORMAT_FP4``, ``swa_ring`` [B, R, 384]). Returns (out, lse); with
    fp4_out, ((out_fp4, out_fp4_scale), lse)."""
    B, T, k = topk_idx.shape
    R = swa_ring.shape[1]
    dev = _dev(q, "q")
    out, lse, out_fp4, out_fp4_scale = _attention_outputs(B, T, q.device, stream, out, lse, fp4_out, out_fp4,
                                                          out_fp4_scale)
    epi, out_fp4, out_fp4_scale = _epilogue(B, T, q.device, inverse_rope, rope_theta, fp4_out, out_fp4, out_fp4_scale)
    if ws is None:
        ws = _own_workspace(OP_ATTENTION, B, T, comp.seq_capacity, k, q.device, stream)
    i32, f32 = torch.int32, torch.float32
    _check((_lib or load()).csa_sink_attention_decode_fp4(
        _arg(q, "q", torch.bfloat16, (B, T, HEADS, DIM), dev), _arg(sink, "sink", f32, (HEADS,), dev), softmax_scale,
        _format(_cache(comp, B, dev), FORMAT_FP4, "csa_sink_attention_decode_fp4"),
        _arg(swa_ring, "swa_ring", torch.uint8, (B, R, FP4_RECORD_BYTES), dev), R, W,
        _arg(topk_idx, "topk_idx", i32, (B, T, k), dev), _arg(topk_cnt, "topk_cnt", i32, (B, T), dev),
        _arg(q_pos, "q_pos", i32, (B, T), dev), B, T, k,
        None if out is None else _arg(out, "out", torch.bfloat16, (B, T, HEADS, DIM), dev),
        _arg(lse, "lse", f32, (B, T, HEADS), dev), epi, *_ws(ws, dev), _own_status(status, dev), _on(stream, dev)),
        "csa_sink_attention_decode_fp4")
    return ((out_fp4, out_fp4_scale) if fp4_out else out), lse


def hca_sink_attention_decode_fp4(q, sink, softmax_scale: float, comp: csa_cache_desc, n_comp, swa_ring, W: int,
                                  q_pos, m_hca: int = 128, out=None, lse=None, ws=None, stream=None, status=None,
                                  inverse_rope: bool = False, rope_theta: float = 10000.0, fp4_out: bool = False,
                                  out_fp4=None, out_fp4_scale=None):
    """hca_sink_attention_decode over caches of 4-bit records."""
    B, T = q_pos.shape
    R = swa_ring.shape[1]
    dev = _dev(q, "q")
    out, lse, out_fp4, out_fp4_scale = _attention_outputs(B, T, q.device, stream, out, lse, fp4_out, out_fp4,
                                                          out_fp4_scale)
    epi, out_fp4, out_fp4_scale = _epilogue(B, T, q.device, inverse_rope, rope_theta, fp4_out, out_fp4, out_fp4_scale)
    if ws is None:
        ws = _own_workspace(OP_HCA_ATTENTION, B, T, comp.seq_capacity, 0, q.device, stream)
    i32, f32 = torch.int32, torch.float32
    _check((_lib or load()).hca_sink_attention_decode_fp4(
        _arg(q, "q", torch.bfloat16, (B, T, HEADS, DIM), dev), _arg(sink, "sink", f32, (HEADS,), dev), softmax_scale,
        _format(_cache(comp, B, dev), FORMAT_FP4, "hca_sink_attention_decode_fp4"), _arg(n_comp, "n_comp", i32, (B,), dev),
        _arg(swa_ring, "swa_ring", torch.uint8, (B, R, FP4_RECORD_BYTES), dev), R, W,
        _arg(q_pos, "q_pos", i32, (B, T), dev), B, T, m_hca,
        None if out is None else _arg(out, "out", torch.bfloat16, (B, T, HEADS, DIM), dev),
        _arg(lse, "lse", f32, (B, T, HEADS), dev), epi, *_ws(ws, dev), _own_status(status, dev), _on(stream, dev)),
        "hca_sink_attention_decode_fp4")
    return ((out_fp4, out_fp4_scale) if fp4_out else out), lse


def csa_decode_step_fp4(q_idx, q_idx_scale, w_idx, k_idx, k_idx_scale, q, sink, softmax_scale: float,
                        comp: csa_cache_desc, swa_ring, W: int, q_pos, n_comp, m: int, k: int, out=None, lse=None,
                        topk_idx=None, topk_cnt=None, ws=None, stream=None, status=None, inverse_rope: bool = False,
                        rope_theta: float = 10000.0, fp4_out: bool = False, out_fp4=None, out_fp4_scale=None):
    """csa_decode_step over caches of 4-bit records (the indexer keys stay FP8)."""
    B, T = q_pos.shape
    Ncap = k_idx.shape[1]
    R = swa_ring.shape[1]
    dev = _dev(q, "q")
    out, lse, out_fp4, out_fp4_scale = _attention_outputs(B, T, q.device, stream, out, lse, fp4_out, out_fp4,
                                                          out_fp4_scale)
    epi, out_fp4, out_fp4_scale = _epilogue(B, T, q.device, inverse_rope, rope_theta, fp4_out, out_fp4, out_fp4_scale)
    if ws is None:
        ws = _own_workspace(OP_DECODE_STEP, B, T, Ncap, k, q.device, stream)
    i32, f32 = torch.int32, torch.float32
    _check((_lib or load()).csa_decode_step_fp4(
        _codes(q_idx, "q_idx", (B, T, IDX_HEADS, IDX_DIM), dev),
        _arg(q_idx_scale, "q_idx_scale", f32, (B, T, IDX_HEADS), dev), _arg(w_idx, "w_idx", f32, (B, T, IDX_HEADS), dev),
        _codes(k_idx, "k_idx", (B, Ncap, IDX_DIM), dev), _arg(k_idx_scale, "k_idx_scale", f32, (B, Ncap), dev),
        _arg(q, "q", torch.bfloat16, (B, T, HEADS, DIM), dev), _arg(sink, "sink", f32, (HEADS,), dev), softmax_scale,
        _format(_cache(comp, B, dev), FORMAT_FP4, "csa_decode_step_fp4"),
        _arg(swa_ring, "swa_ring", torch.uint8, (B, R, FP4_RECORD_BYTES), dev), R, W,
        _arg(q_pos, "q_pos", i32, (B, T), dev), _arg(n_comp, "n_comp", i32, (B,), dev), B, T, Ncap, m, k,
        None if out is None else _arg(out, "out", torch.bfloat16, (B, T, HEADS, DIM), dev),
        _arg(lse, "lse", f32, (B, T, HEADS), dev),
        None if topk_idx is None else _arg(topk_idx, "topk_idx", i32, (B, T, k), dev),
        None if topk_cnt is None else _arg(topk_cnt, "topk_cnt", i32, (B, T), dev),
        epi, *_ws(ws, dev), _own_status(status, dev), _on(stream, dev)), "csa_decode_step_fp4")
    return ((out_fp4, out_fp4_scale) if fp4_out else out), lse


def _tree(draft, parent, comp: csa_cache_desc, swa_ring, B: int, N: int, dev: int):
    """(the tree's struct, pointer of the ring, its length): records of the cache's format."""
    size = FORMAT_BYTES[comp._fmt]
    R = swa_ring.shape[1]
    ring = _arg(swa_ring, "swa_ring", torch.uint8, (B, R, size), dev)
    return csa_draft_tree(_arg(draft, "draft", torch.uint8, (B, N, size), dev),
                          _arg(parent, "parent", torch.int32, (B, N), dev)), ring, R


def csa_tree_attention_decode(q, sink, softmax_scale: float, comp: csa_cache_desc, swa_ring, W: int, draft, parent,
                              topk_idx, topk_cnt, q_pos, out=None, lse=None, ws=None, stream=None, status=None,
                              inverse_rope: bool = False, rope_theta: float = 10000.0, fp4_out: bool = False,
                              out_fp4=None, out_fp4_scale=None):
    """csa_sink_attention_decode for a tree of N drafted tokens a sequence (q [B, N, 128, 512]): token i follows
    token ``parent[b, i]`` < i (-1: the last committed token) and attends, beside its selected entries, to itself, to
    its ancestors among ``draft`` [B, N, record bytes] and to the committed tokens of its window in ``swa_ring``.
    ``comp``, ring and drafts hold records of the cache's format, FP8 or 4-bit. Entries that the tree's own tokens
    complete are not among the compressed ones (see include/csa.h). Tokens with q_pos < 0 are padding: what their rows
    of the selection hold does not matter, and their rows are left as they were (pass outputs of your own). Returns
    (out, lse); with fp4_out, ((out_fp4, out_fp4_scale), lse)."""
    B, N, k = topk_idx.shape
    dev = _dev(q, "q")
    out, lse, out_fp4, out_fp4_scale = _attention_outputs(B, N, q.device, stream, out, lse, fp4_out, out_fp4,
                                                          out_fp4_scale)
    epi, out_fp4, out_fp4_scale = _epilogue(B, N, q.device, inverse_rope, rope_theta, fp4_out, out_fp4, out_fp4_scale)
    if ws is None:
        ws = _own_workspace(OP_TREE_ATTENTION, B, N, comp.seq_capacity, k, q.device, stream)
    tree, ring, R = _tree(draft, parent, comp, swa_ring, B, N, dev)
    i32, f32 = torch.int32, torch.float32
    _check((_lib or load()).csa_tree_attention_decode(
        _arg(q, "q", torch.bfloat16, (B, N, HEADS, DIM), dev), _arg(sink, "sink", f32, (HEADS,), dev), softmax_scale,
        _cache(comp, B, dev), comp._fmt, ring, R, W, tree, _arg(topk_idx, "topk_idx", i32, (B, N, k), dev),
        _arg(topk_cnt, "topk_cnt", i32, (B, N), dev), _arg(q_pos, "q_pos", i32, (B, N), dev), B, N, k,
        None if out is None else _arg(out, "out", torch.bfloat16, (B, N, HEADS, DIM), dev),
        _arg(lse, "lse", f32, (B, N, HEADS), dev), epi, *_ws(ws, dev), _own_status(status, dev), _on(stream, dev)),
        "csa_tree_attention_decode")
    return ((out_fp4, out_fp4_scale) if fp4_out else out), lse


def hca_tree_attention_decode(q, sink, softmax_scale: float, comp: csa_cache_desc, n_comp, swa_ring, W: int, draft,
                              parent, q_pos, m_hca: int = 128, out=None, lse=None, ws=None, stream=None, status=None,
                              inverse_rope: bool = False, rope_theta: float = 10000.0, fp4_out: bool = False,
                              out_fp4=None, out_fp4_scale=None):
    """csa_tree_attention_decode over every visible entry instead of a selection (hca_sink_attention_decode for a
    tree)."""
    B, N = q_pos.shape
    dev = _dev(q, "q")
    out, lse, out_fp4, out_fp4_scale = _attention_outputs(B, N, q.device, stream, out, lse, fp4_out, out_fp4,
                                                          out_fp4_scale)
    epi, out_fp4, out_fp4_scale = _epilogue(B, N, q.device, inverse_rope, rope_theta, fp4_out, out_fp4, out_fp4_scale)
    if ws is None:
        ws = _own_workspace(OP_HCA_TREE_ATTENTION, B, N, comp.seq_capacity, 0, q.device, stream)
    tree, ring, R = _tree(draft, parent, comp, swa_ring, B, N, dev)
    i32, f32 = torch.int32, torch.float32
    _check((_lib or load()).hca_tree_attention_decode(
        _arg(q, "q", torch.bfloat16, (B, N, HEADS, DIM), dev), _arg(sink, "sink", f32, (HEADS,), dev), softmax_scale,
        _cache(comp, B, dev), comp._fmt, _arg(n_comp, "n_comp", i32, (B,), dev), ring, R, W, tree,
        _arg(q_pos, "q_pos", i32, (B, N), dev), B, N, m_hca,
        None if out is None else _arg(out, "out", torch.bfloat16, (B, N, HEADS, DIM), dev),
        _arg(lse, "lse", f32, (B, N, HEADS), dev), epi, *_ws(ws, dev), _own_status(status, dev), _on(stream, dev)),
        "hca_tree_attention_decode")
    return ((out_fp4, out_fp4_scale) if fp4_out else out), lse


def csa_tree_decode_step(q_idx, q_idx_scale, w_idx, k_idx, k_idx_scale, q, sink, softmax_scale: float,
                         comp: csa_cache_desc, swa_ring, W: int, draft, parent, q_pos, n_comp, m: int, k: int,
                         out=None, lse=None, topk_idx=None, topk_cnt=None, ws=None, stream=None, status=None,
                         inverse_rope: bool = False, rope_theta: float = 10000.0, fp4_out: bool = False, out_fp4=None,
                         out_fp4_scale=None):
    """csa_decode_step for a tree of drafted tokens: indexer and top-k for every token of the tree at its own
    position, then csa_tree_attention_decode."""
    B, N = q_pos.shape
    Ncap = k_idx.shape[1]
    dev = _dev(q, "q")
    out, lse, out_fp4, out_fp4_scale = _attention_outputs(B, N, q.device, stream, out, lse, fp4_out, out_fp4,
                                                          out_fp4_scale)
    epi, out_fp4, out_fp4_scale = _epilogue(B, N, q.device, inverse_rope, rope_theta, fp4_out, out_fp4, out_fp4_scale)
    if ws is None:
        ws = _own_workspace(OP_TREE_STEP, B, N, Ncap, k, q.device, stream)
    tree, ring, R = _tree(draft, parent, comp, swa_ring, B, N, dev)
    i32, f32 = torch.int32, torch.float32
    _check((_lib or load()).csa_tree_decode_step(
        _codes(q_idx, "q_idx", (B, N, IDX_HEADS, IDX_DIM), dev),
        _arg(q_idx_scale, "q_idx_scale", f32, (B, N, IDX_HEADS), dev), _arg(w_idx, "w_idx", f32, (B, N, IDX_HEADS), dev),
        _codes(k_idx, "k_idx", (B, Ncap, IDX_DIM), dev), _arg(k_idx_scale, "k_idx_scale", f32, (B, Ncap), dev),
        _arg(q, "q", torch.bfloat16, (B, N, HEADS, DIM), dev), _arg(sink, "sink", f32, (HEADS,), dev), softmax_scale,
        _cache(comp, B, dev), comp._fmt, ring, R, W, tree, _arg(q_pos, "q_pos", i32, (B, N), dev),
        _arg(n_comp, "n_comp", i32, (B,), dev), B, N, Ncap, m, k,
        None if out is None else _arg(out, "out", torch.bfloat16, (B, N, HEADS, DIM), dev),
        _arg(lse, "lse", f32, (B, N, HEADS), dev),
        None if topk_idx is None else _arg(topk_idx, "topk_idx", i32, (B, N, k), dev),
        None if topk_cnt is None else _arg(topk_cnt, "topk_cnt", i32, (B, N), dev),
        epi, *_ws(ws, dev), _own_status(status, dev), _on(stream, dev)), "csa_tree_decode_step")
    return ((out_fp4, out_fp4_scale) if fp4_out else out), lse


def csa_verify_drafts(logits, tokens, parent, uniform, noise, temperature=None, draft_probs=None, path=None,
                      accepted=None, next_token=None, ws=None, stream=None, status=None):
    """Accept a path of the drafted tokens ``tokens`` [B, N] int32 of a tree (token 0 is the newest known one, the
    others follow ``parent``) against the target's ``logits`` [B, N, V] (bf16, fp16 or fp32; any strides but a dense
    last dimension), and draw the token that follows it. ``draft_probs`` [B, N, V]: row i is the distribution that the
    children of token i were drawn from; without it drafts are accepted as fixed guesses. ``uniform`` [B, N] fp32 in
    [0, 1), ``noise`` [B, V] fp32 of exponential variates, ``temperature`` [B] fp32 (0: greedy). Returns (path [B, N]
    int32: the accepted tokens' numbers and -1 behind them, accepted [B], next_token [B]). ``ws`` may be None: none is
    needed at present."""
    B, N, V = logits.shape
    dev = _dev(logits, "logits")
    i32, f32 = torch.int32, torch.float32
    device, rows, one = logits.device, (B, N), (B,)
    if path is None:  # (what is made here needs no checks: 0.3 us each)
        path = _new(torch.empty, rows, i32, device, stream)
        path_ptr = path.data_ptr()
    else:
        path_ptr = _arg(path, "path", i32, rows, dev)
    if accepted is None:
        accepted = _new(torch.empty, one, i32, device, stream)
        accepted_ptr = accepted.data_ptr()
    else:
        accepted_ptr = _arg(accepted, "accepted", i32, one, dev)
    if next_token is None:
        next_token = _new(torch.empty, one, i32, device, stream)
        next_ptr = next_token.data_ptr()
    else:
        next_ptr = _arg(next_token, "next_token", i32, one, dev)
    ptr, dt, s = _rows(logits, "logits", dev)
    q, q_dt = None, 0
    if draft_probs is not None:
        q_dt = _DTYPES.get(draft_probs.dtype)
        if q_dt is None:
            raise ValueError(f"draft_probs must be a bf16, fp16 or fp32 tensor: got {draft_probs.dtype}")
        q = _arg(draft_probs, "draft_probs", draft_probs.dtype, (B, N, V), dev)
    _check((_lib or load()).csa_verify_drafts(
        ptr, dt, *s, q, q_dt, _arg(tokens, "tokens", i32, rows, dev), _arg(parent, "parent", i32, rows, dev),
        _arg(uniform, "uniform", f32, rows, dev), _arg(noise, "noise", f32, (B, V), dev),
        None if temperature is None else _arg(temperature, "temperature", f32, one, dev), B, N, V, path_ptr,
        accepted_ptr, next_ptr, *_ws(ws, dev), _own_status(status, dev), _on(stream, dev)), "csa_verify_drafts")
    return path, accepted, next_token


def csa_cache_commit(cache: csa_cache_desc, records, select, count, first, ring: bool = False, stream=None,
                     status=None) -> None:
    """Put record ``select[b, t]`` of ``records`` [B, N, record bytes] (of the cache's format) into the cache as entry
    ``first[b] + t`` of sequence b, for t < ``count[b]``, byte for byte: after csa_verify_drafts, ``select`` and
    ``count`` are its path and its accepted. ``select`` None: record t; ``count`` None: all of them. ``ring``: entry
    modulo the cache's capacity. ``records`` must not be part of the cache. ``select``, ``count`` and ``first`` begin on
    16 bytes (a path that is a slice of a larger tensor may not)."""
    B, N, size = records.shape
    dev = _dev(records, "records")
    if cache._copied:
        raise ValueError("the cache's records were not contiguous: the description holds a copy of them")
    T = N if select is None else select.shape[1]
    _check((_lib or load()).csa_cache_commit(
        _cache(cache, B, dev), cache._fmt, 1 if ring else 0,
        _arg(records, "records", torch.uint8, (B, N, FORMAT_BYTES[cache._fmt]), dev), N,
        None if select is None else _arg(select, "select", torch.int32, (B, T), dev),
        _arg(first, "first", torch.int32, (B,), dev),
        None if count is None else _arg(count, "count", torch.int32, (B,), dev), B, T, _own_status(status, dev),
        _on(stream, dev)), "csa_cache_commit")


def _ws(ws, dev: int):
    """(pointer, bytes) of a workspace; (None, 0) for none."""
    return (None, 0) if ws is None else (_arg(ws, "workspace", torch.uint8, ws.shape, dev), ws.numel())


def _cache(cache: csa_cache_desc, B: int, dev: int) -> csa_cache_desc:
    """The description itself, if its records lie on device ``dev`` and its block
    table has a row for each of the B sequences."""
    if cache._dev is not None and cache._dev != dev:
        raise ValueError(f"the cache is on cuda:{cache._dev}, not on cuda:{dev}")
    if cache._seqs is not None and cache._seqs < B:
        raise ValueError(f"the cache's block table has {cache._seqs} rows for {B} sequences")
    return cache


def _hptr(t: torch.Tensor, name: str, dtype, shape):
    """Host tensor check for the pipeline: CPU, contiguous, dtype, shape."""
    if t.is_cuda:
        raise ValueError(f"{name} must be a host (CPU) tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t.data_ptr()


def csa_pipeline_staging_bytes(B: int, T: int, depth: int) -> int:
    return int(load().csa_pipeline_staging_bytes(B, T, depth))


def csa_pipeline_create(B: int, T: int, depth: int, staging: torch.Tensor, stream=None) -> int:
    """Handle of a new host-I/O pipeline on the current device; ``staging`` is
    a uint8 device tensor of at least csa_pipeline_staging_bytes(B, T, depth)."""
    h = C.c_void_p()
    _check(load().csa_pipeline_create(C.byref(h), B, T, depth, _ptr(staging, "staging", torch.uint8),
                                      staging.numel(), _stream(stream)), "csa_pipeline_create")
    return h.value


def csa_decode_step_host(pipeline: int, B: int, T: int, h_q_idx, h_q_idx_scale, h_w_idx, h_q, h_q_pos, k_idx,
                         k_idx_scale, sink, softmax_scale: float, comp: csa_cache_desc, swa_ring, W: int, n_comp,
                         m: int, k: int, h_out, h_lse, ws, status=None) -> int:
    """Enqueue one step; h_* are host tensors (page-locked for overlap), the
    rest is the device-resident layer state. Returns the step's ordinal."""
    Ncap = k_idx.shape[1]
    R = swa_ring.shape[1]
    u8 = (torch.uint8, torch.float8_e4m3fn)
    step = C.c_int64(-1)
    _check(load().csa_decode_step_host(
        C.c_void_p(pipeline), _hptr(h_q_idx, "h_q_idx", u8, (B, T, IDX_HEADS, IDX_DIM)),
        _hptr(h_q_idx_scale, "h_q_idx_scale", torch.float32, (B, T, IDX_HEADS)),
        _hptr(h_w_idx, "h_w_idx", torch.float32, (B, T, IDX_HEADS)),
        _hptr(h_q, "h_q", torch.bfloat16, (B, T, HEADS, DIM)), _hptr(h_q_pos, "h_q_pos", torch.int32, (B, T)),
        _ptr(k_idx, "k_idx", u8, (B, Ncap, IDX_DIM)), _ptr(k_idx_scale, "k_idx_scale", torch.float32, (B, Ncap)),
        _ptr(sink, "sink", torch.float32, (HEADS,)), float(softmax_scale),
        _format(comp, FORMAT_FP8, "csa_decode_step_host"),
        _ptr(swa_ring, "swa_ring", torch.uint8, (B, R, RECORD_BYTES)), R, int(W),
        _ptr(n_comp, "n_comp", torch.int32, (B,)), Ncap, int(m), int(k),
        _hptr(h_out, "h_out", torch.bfloat16, (B, T, HEADS, DIM)), _hptr(h_lse, "h_lse", torch.float32, (B, T, HEADS)),
        _ptr(ws, "workspace", torch.uint8), 0 if ws is None else ws.numel(), _status(status, k_idx.device),
        C.byref(step)), "csa_decode_step_host")
    return int(step.value)


def csa_pipeline_wait(pipeline: int, step: int):
    _check(load().csa_pipeline_wait(C.c_void_p(pipeline), int(step)), "csa_pipeline_wait")


def csa_pipeline_sync(pipeline: int):
    _check(load().csa_pipeline_sync(C.c_void_p(pipeline)), "csa_pipeline_sync")


def csa_pipeline_destroy(pipeline: int):
    _check(load().csa_pipeline_destroy(C.c_void_p(pipeline)), "csa_pipeline_destroy")


class HostPipeline:
    """Owns a pipeline handle and its device staging area (torch memory).
    ``step(...)`` enqueues csa_decode_step_host and returns the ordinal;
    ``wait(i)`` / ``sync()`` block until results are in host memory."""

    def __init__(self, B: int, T: int, depth: int = 2, device=None, stream=None):
        n = csa_pipeline_staging_bytes(B, T, depth)
        if n == 0:
            raise ValueError(f"unsupported pipeline sizes B={B} T={T} depth={depth}")
        self.B, self.T, self.depth = B, T, depth
        self.staging = torch.empty(n, dtype=torch.uint8, device=device or torch.device("cuda"))
        self.handle = csa_pipeline_create(B, T, depth, self.staging, stream)

    def step(self, h_q_idx, h_q_idx_scale, h_w_idx, h_q, h_q_pos, k_idx, k_idx_scale, sink, softmax_scale, comp,
             swa_ring, W, n_comp, m, k, h_out, h_lse, ws, status=None) -> int:
        return csa_decode_step_host(self.handle, self.B, self.T, h_q_idx, h_q_idx_scale, h_w_idx, h_q, h_q_pos,
                                    k_idx, k_idx_scale, sink, softmax_scale, comp, swa_ring, W, n_comp, m, k,
                                    h_out, h_lse, ws, status)

    def wait(self, step: int):
        csa_pipeline_wait(self.handle, step)

    def sync(self):
        csa_pipeline_sync(self.handle)

    def close(self):
        if self.handle:
            h, self.handle = self.handle, None
            csa_pipeline_destroy(h)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def csa_check_device_status(host_status: torch.Tensor, status: torch.Tensor | None = None, stream=None,
                            device=None):
    """Enqueue (no synchronisation) a copy of the status word into
    ``host_status`` (an int32 CPU tensor of one element, page-locked for an
    asynchronous copy) and a reset of the word. Read ``host_status`` once the
    stream has passed this point."""
    if host_status.is_cuda or host_status.dtype != torch.int32 or host_status.numel() != 1:
        raise ValueError("host_status must be a one-element int32 CPU tensor")
    dev = status.device if status is not None else device
    _check(load().csa_check_device_status(_status(status, dev), host_status.data_ptr(), _stream(stream)),
           "csa_check_device_status")


def csa_read_device_error(stream=None, status: torch.Tensor | None = None, device=None) -> int:
    """Read and clear a status word (the device's default one unless given);
    blocking: synchronises the stream. For tests and diagnostics."""
    code = C.c_int32(0)
    dev = status.device if status is not None else device
    _check(load().csa_read_device_error(_status(status, dev), C.byref(code), _stream(stream)), "csa_read_device_error")
    return int(code.value)


def csa_debug_set_wait_limit_ns(ns: int):
    """Diagnostic: limit of the kernels' bounded waits for later launches (0 =
    the default of one second); see include/csa.h."""
    load().csa_debug_set_wait_limit_ns(int(ns))
