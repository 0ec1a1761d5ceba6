"""Python binding of the MI355X paged MQA indexer C ABI (include/paged_mqa_indexer.h).

Argument marshalling only: tensors are checked for dtype, device, shape and
layout, their device pointers and the current HIP stream are handed to the C
entry points of ``libpaged_mqa_indexer.so``, and a non-zero status raises
``IndexerError``.  Every step of the computation runs in the library's HIP
kernels; there is no fallback path.  PyTorch only supplies device memory and
streams.

Entry points (same names as the C ABI):
  indexer_logits(q, kv_pages, k_scales, weights, block_table, context_lens,
                 next_n, logits, hist=None, events=None)        float32 logits
  indexer_logits_f16(... same ..., logits, hist=None, events=None) float16 logits
  indexer_logits_mxfp4(q, kv_pages, weights, block_table, context_lens, next_n,
                       logits, hist=None, events=None)  packed MXFP4 K, float32 logits
  topk_workspace_bytes(rows, logits_stride, k)
  topk_rows(logits, hist, context_lens, k, key_dtype, indices, workspace=None,
            events=None)                                          float32 scores
  topk_rows_f16(logits, hist, context_lens, k, indices, workspace=None,
                events=None)                                      float16 scores
  topk_rows_noalloc(logits, hist, context_lens, k, key_dtype, indices,
                    events=None)          float32 scores, the library's fixed scratch
  score_histogram(scores, context_lens, hist)
  block_amax8(scores, context_lens, out)                       two-level candidate indexer:
  sort_candidate_blocks(blocks, context_lens, max_len, block_table, next_n,
                        table, slots, sparse_lens)
  indexer_sparse_logits(q, kv_pages, k_scales, weights, table, slots,
                        context_lens, logits)
  sparse_to_logical(indices, table, out)
  sparse_topk(scores, hist, sparse_lens, k, key_dtype, table, out)
  index_k_append(k, positions, slots, rope, kv_pages, k_scales, interleaved)  paged caches:
  index_k_append_mxfp4(k, positions, slots, rope, kv_pages, interleaved)
  latent_append(kv, positions, slots, rope, latent_pages, interleaved)
  latent_append_mxfp4(kv, positions, slots, rope, latent_pages, interleaved)   4-bit latent rows
  axis_rotations(positions, axis_map, rope, out)                    rotary positions, several axes:
  rotate_queries(x, positions, rope, out, axis_map, interleaved)
  rotate_index_queries(q, positions, rope, codes, axis_map, interleaved)
  axis_map(axis_of)
  release_pages(block_table, lens, ended, refs, new_lens, new_refs)        care of the pages:
  fork_pages(block_table, lens, parents, refs, new_lens, new_refs, src, dst, tokens, counts)
  compact_pages(block_table, lens, refs, new_table, new_refs, src, dst, counts)
  copy_pages(caches, src, dst, tokens=None, count=None), PageCaches(caches)
  pages_workspace_bytes(requests, num_pages)
  paged_attention(q, latent_pages, block_table, row_lens, next_n, scale, out, ...)
  shared_prefix_attention(..., next_n, prefix_pages, scale, out, ...)
  sparse_attention(q, latent_pages, block_table, indices, next_n, scale, out, ...)
  paged_attention_mxfp4, shared_prefix_attention_mxfp4, sparse_attention_mxfp4: the same over 4-bit rows
  attention_workspace_bytes(rows, heads, requests), shared_prefix_workspace_bytes(...)
  indexer_status_str(status)
  indexer_time_next_call(start, stop)
  hbm_read_probe(src, sink, events=None)
  hbm_read_probe_nt(src, sink, events=None)
  hbm_gather_probe(kv_pages, k_scales, page_list, sink, events=None)
  mfma_valu_probe(mode, waves_per_simd, iters, out, events=None)
With ``events=(start, stop)`` (torch.cuda.Event with timing enabled, either
may be None) the call is preceded by indexer_time_next_call, so its own
kernel dispatches record the events: start when its first kernel begins,
stop when its last kernel ends.
"""

from __future__ import annotations

import ctypes
import os

import torch

__all__ = [
    "IndexerError", "KEY_FP32", "KEY_FP16", "NUM_BINS", "CANDIDATE_CAPACITY",
    "EXPORTED_SYMBOLS", "load_library", "library_path", "indexer_logits", "indexer_logits_f16",
    "indexer_logits_mxfp4", "block_amax8", "sort_candidate_blocks", "indexer_sparse_logits",
    "indexer_sparse_logits_mxfp4", "indexer_prefill_logits", "indexer_prefill_logits_mxfp4",
    "sparse_to_logical", "sparse_topk",
    "topk_workspace_bytes", "topk_rows", "topk_rows_f16", "topk_rows_noalloc", "score_histogram",
    "indexer_status_str", "indexer_time_next_call", "hbm_read_probe", "hbm_read_probe_nt",
    "hbm_gather_probe", "mfma_valu_probe", "latent_append_mxfp4", "axis_map", "axis_rotations", "rotate_queries",
    "rotate_index_queries", "PageCaches", "pages_workspace_bytes", "release_pages", "fork_pages", "compact_pages",
    "copy_pages", "paged_attention_mxfp4", "shared_prefix_attention_mxfp4", "sparse_attention_mxfp4",
]

KEY_FP32 = 0
KEY_FP16 = 1
NUM_BINS = 1024
CANDIDATE_CAPACITY = 8192
HEADS = 32
HEAD_DIM = 128
PAGE_TOKENS = 64
MXFP4_TOKEN_BYTES = 68
LATENT_DIM = 512
ROPE_DIM = 64
LATENT_ROW = 576
LATENT_MXFP4_ROW = 400
MAX_AXES = 4
MAX_CACHES = 1024
VALUE_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}

EXPORTED_SYMBOLS = ("indexer_logits", "indexer_logits_f16", "indexer_logits_mxfp4", "block_amax8",
                    "sort_candidate_blocks", "indexer_sparse_logits", "indexer_sparse_logits_mxfp4",
                    "indexer_prefill_logits", "indexer_prefill_logits_mxfp4", "sparse_to_logical", "sparse_topk",
                    "topk_workspace_bytes", "topk_rows", "topk_rows_noalloc",
                    "topk_rows_f16", "score_histogram", "indexer_status_str",
                    "indexer_time_next_call", "hbm_read_probe", "hbm_read_probe_nt", "hbm_gather_probe",
                    "mfma_valu_probe", "index_k_append", "index_k_append_mxfp4", "latent_append",
                    "attention_workspace_bytes", "shared_prefix_workspace_bytes", "paged_attention",
                    "shared_prefix_attention", "sparse_attention", "latent_append_mxfp4", "axis_rotations",
                    "rotate_queries", "rotate_index_queries", "pages_workspace_bytes", "release_pages", "fork_pages",
                    "compact_pages", "copy_pages", "paged_attention_mxfp4", "shared_prefix_attention_mxfp4",
                    "sparse_attention_mxfp4")

_PKG_DIR = os.path.dirname(os.path.abspath(__file__))
_LIB_NAME = "libpaged_mqa_indexer.so"
_lib = None


class IndexerError(RuntimeError):
    """A C entry point returned a non-zero idx_status."""

    def __init__(self, func: str, status: int, msg: str):
        super().__init__(f"{func} failed: {msg} (status {status})")
        self.status = status


def library_path() -> str:
    return os.environ.get("PMQA_INDEXER_LIB", os.path.join(_PKG_DIR, _LIB_NAME))


def load_library() -> ctypes.CDLL:
    """Load the HIP library (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise RuntimeError(
            f"HIP library {path} is missing: build it with "
            "`python -m paged_mqa_logits_indexer_amd.build` (or __graft_entry__.build())")
    lib = ctypes.CDLL(path)
    vp, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    lib.indexer_logits.argtypes = [vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, vp, i64, vp, vp]
    lib.indexer_logits.restype = ctypes.c_int
    lib.topk_workspace_bytes.argtypes = [i32, i64, i32]
    lib.topk_workspace_bytes.restype = sz
    lib.topk_rows.argtypes = [vp, i64, vp, vp, i32, i32, i32, vp, vp, sz, vp]
    lib.topk_rows.restype = ctypes.c_int
    lib.score_histogram.argtypes = [vp, i64, vp, i32, vp, vp]
    lib.score_histogram.restype = ctypes.c_int
    lib.indexer_status_str.argtypes = [i32]
    lib.indexer_status_str.restype = ctypes.c_char_p
    lib.hbm_read_probe.argtypes = [vp, sz, vp, vp]
    lib.hbm_read_probe.restype = ctypes.c_int
    lib.hbm_read_probe_nt.argtypes = [vp, sz, vp, vp]
    lib.hbm_read_probe_nt.restype = ctypes.c_int
    lib.hbm_gather_probe.argtypes = [vp, vp, vp, i32, i32, vp, vp]
    lib.hbm_gather_probe.restype = ctypes.c_int
    lib.mfma_valu_probe.argtypes = [i32, i32, i32, vp, i64, vp]
    lib.mfma_valu_probe.restype = ctypes.c_int
    lib.indexer_logits_f16.argtypes = lib.indexer_logits.argtypes
    lib.indexer_logits_f16.restype = ctypes.c_int
    lib.indexer_logits_mxfp4.argtypes = [vp, vp, vp, vp, vp, i32, i32, i32, i32, vp, i64, vp, vp]
    lib.indexer_logits_mxfp4.restype = ctypes.c_int
    lib.block_amax8.argtypes = [vp, i64, vp, i32, vp, i64, vp, vp, vp]
    lib.block_amax8.restype = ctypes.c_int
    lib.sort_candidate_blocks.argtypes = [vp, i32, vp, i32, i64, vp, i32, i32, vp, vp, vp, vp]
    lib.sort_candidate_blocks.restype = ctypes.c_int
    lib.indexer_sparse_logits.argtypes = [vp, vp, vp, vp, vp, vp, i32, vp, i32, i32, vp, i64, vp]
    lib.indexer_sparse_logits.restype = ctypes.c_int
    lib.indexer_sparse_logits_mxfp4.argtypes = [vp, vp, vp, vp, vp, i32, vp, i32, i32, vp, i64, vp]
    lib.indexer_sparse_logits_mxfp4.restype = ctypes.c_int
    lib.indexer_prefill_logits.argtypes = [vp, vp, vp, vp, vp, i32, vp, i32, i32, vp, i32, vp, i64, vp]
    lib.indexer_prefill_logits.restype = ctypes.c_int
    lib.indexer_prefill_logits_mxfp4.argtypes = [vp, vp, vp, vp, i32, vp, i32, i32, vp, i32, vp, i64, vp]
    lib.indexer_prefill_logits_mxfp4.restype = ctypes.c_int
    lib.sparse_to_logical.argtypes = [vp, i32, vp, i32, i32, vp, vp]
    lib.sparse_topk.argtypes = [vp, i64, vp, vp, i32, i32, i32, vp, i32, vp, vp]
    lib.sparse_topk.restype = ctypes.c_int
    lib.sparse_to_logical.restype = ctypes.c_int
    lib.topk_rows_f16.argtypes = [vp, i64, vp, vp, i32, i32, vp, vp, sz, vp]
    lib.topk_rows_f16.restype = ctypes.c_int
    lib.topk_rows_noalloc.argtypes = [vp, i64, vp, vp, i32, i32, i32, vp, vp]
    lib.topk_rows_noalloc.restype = ctypes.c_int
    lib.indexer_time_next_call.argtypes = [vp, vp]
    lib.indexer_time_next_call.restype = ctypes.c_int
    f32 = ctypes.c_float
    lib.index_k_append.argtypes = [vp, i64, i32, vp, vp, vp, i32, i32, i32, i32, vp, vp, vp]
    lib.index_k_append.restype = ctypes.c_int
    lib.index_k_append_mxfp4.argtypes = [vp, i64, i32, vp, vp, vp, i32, i32, i32, i32, vp, vp]
    lib.index_k_append_mxfp4.restype = ctypes.c_int
    lib.latent_append.argtypes = lib.index_k_append_mxfp4.argtypes
    lib.latent_append.restype = ctypes.c_int
    for name in ("attention_workspace_bytes", "shared_prefix_workspace_bytes"):
        getattr(lib, name).argtypes = [i32, i32, i32]
        getattr(lib, name).restype = sz
    lib.paged_attention.argtypes = [vp, vp, i32, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, f32, f32, vp, vp,
                                    vp, vp, vp, sz, vp]
    lib.paged_attention.restype = ctypes.c_int
    lib.shared_prefix_attention.argtypes = [vp, vp, i32, vp, vp, vp, i32, i32, i32, i32, i32, i32, i32, f32, f32,
                                            vp, vp, vp, vp, vp, sz, vp]
    lib.shared_prefix_attention.restype = ctypes.c_int
    lib.sparse_attention.argtypes = [vp, vp, i32, vp, vp, i32, vp, i32, i32, i32, i32, i32, i32, f32, f32, vp, vp,
                                     vp, vp, vp, sz, vp]
    lib.sparse_attention.restype = ctypes.c_int
    for name in ("paged_attention", "shared_prefix_attention", "sparse_attention"):
        getattr(lib, name + "_mxfp4").argtypes = getattr(lib, name).argtypes
        getattr(lib, name + "_mxfp4").restype = ctypes.c_int
    lib.latent_append_mxfp4.argtypes = lib.latent_append.argtypes
    lib.latent_append_mxfp4.restype = ctypes.c_int
    u64 = ctypes.c_uint64
    lib.axis_rotations.argtypes = [vp, i32, u64, i32, vp, i32, vp, vp]
    lib.axis_rotations.restype = ctypes.c_int
    lib.rotate_queries.argtypes = [vp, i64, i64, i32, vp, i32, u64, vp, i32, i32, i32, i32, vp, i64, i64, vp]
    lib.rotate_queries.restype = ctypes.c_int
    lib.rotate_index_queries.argtypes = [vp, i64, i64, i32, vp, i32, u64, vp, i32, i32, i32, vp, vp]
    lib.rotate_index_queries.restype = ctypes.c_int
    lib.pages_workspace_bytes.argtypes = [i32, i32]
    lib.pages_workspace_bytes.restype = sz
    lib.release_pages.argtypes = [vp, vp, vp, i32, i32, vp, i32, vp, vp, vp]
    lib.release_pages.restype = ctypes.c_int
    lib.fork_pages.argtypes = [vp, vp, vp, i32, i32, vp, i32, vp, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.fork_pages.restype = ctypes.c_int
    lib.compact_pages.argtypes = [vp, vp, i32, i32, vp, i32, vp, vp, vp, vp, vp, vp, sz, vp]
    lib.compact_pages.restype = ctypes.c_int
    lib.copy_pages.argtypes = [vp, vp, i32, i32, vp, vp, vp, vp, i32, vp]
    lib.copy_pages.restype = ctypes.c_int
    _lib = lib
    return lib


def indexer_status_str(status: int) -> str:
    return load_library().indexer_status_str(int(status)).decode()


def _check(func: str, status: int) -> None:
    if status != 0:
        raise IndexerError(func, status, indexer_status_str(status))


# The current stream's handle without building a Stream object around it
# (0.1 us instead of 1.9 us a call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_ptr(device: torch.device) -> int:
    if _raw_stream is not None and device.index is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _need(t: torch.Tensor, name: str, dtype, device=None, ndim=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a GPU tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {tuple(t.shape)}")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _event_handles(events, device: torch.device):
    """hipEvent_t handles of (start, stop), either of which may be None; a
    torch event that was never recorded has no HIP event yet, so it is
    recorded once to create it."""
    start, stop = events
    handles = []
    for ev in (start, stop):
        if ev is None:
            handles.append(None)
            continue
        if not isinstance(ev, torch.cuda.Event):
            raise TypeError("events must be a pair of torch.cuda.Event (or None)")
        if not ev.cuda_event:
            ev.record(torch.cuda.current_stream(device))
        handles.append(ev.cuda_event)
    return handles


def indexer_time_next_call(start, stop, device=None) -> None:
    """Arm this host thread's next library call to record (start, stop)
    from its own kernel dispatches (torch.cuda.Event, or None)."""
    dev = device if device is not None else torch.device("cuda", torch.cuda.current_device())
    h = _event_handles((start, stop), dev)
    _check("indexer_time_next_call", load_library().indexer_time_next_call(*h))


def _arm(events, device) -> None:
    if events is not None:
        indexer_time_next_call(events[0], events[1], device)


def _logits_call(name, dtype, q, kv_pages, k_scales, weights, block_table, context_lens, next_n,
                 logits, hist, events):
    """k_scales None: MXFP4 pages [P, 64, 68] (indexer_logits_mxfp4)."""
    dev = q.device
    mx = k_scales is None
    _need(q, "q", torch.uint8, dev, 3)
    _need(kv_pages, "kv_pages", torch.uint8, dev, 3)
    if not mx:
        _need(k_scales, "k_scales", torch.float32, dev, 2)
    _need(weights, "weights", torch.float32, dev, 2)
    _need(block_table, "block_table", torch.int32, dev, 2)
    _need(context_lens, "context_lens", torch.int32, dev, 1)
    _need(logits, "logits", dtype, dev, 2)
    B, max_pages = block_table.shape
    rows = B * next_n
    if tuple(q.shape) != (rows, HEADS, HEAD_DIM) or not q.is_contiguous():
        raise ValueError(f"q must be contiguous [{rows}, 32, 128]")
    P = kv_pages.shape[0]
    tok = MXFP4_TOKEN_BYTES if mx else HEAD_DIM
    if tuple(kv_pages.shape) != (P, PAGE_TOKENS, tok) or not kv_pages.is_contiguous():
        raise ValueError(f"kv_pages must be contiguous [P, 64, {tok}]")
    if not mx and (tuple(k_scales.shape) != (P, PAGE_TOKENS) or not k_scales.is_contiguous()):
        raise ValueError("k_scales must be contiguous [P, 64]")
    if tuple(weights.shape) != (rows, HEADS) or not weights.is_contiguous():
        raise ValueError(f"weights must be contiguous [{rows}, 32]")
    if not block_table.is_contiguous():
        raise ValueError("block_table must be contiguous")
    if tuple(context_lens.shape) != (rows,) or not context_lens.is_contiguous():
        raise ValueError(f"context_lens must be contiguous [{rows}]")
    if logits.shape[0] != rows or logits.stride(1) != 1:
        raise ValueError(f"logits must be [{rows}, stride] with unit column stride")
    if hist is not None:
        _need(hist, "hist", torch.int32, dev, 2)
        if tuple(hist.shape) != (rows, NUM_BINS) or not hist.is_contiguous():
            raise ValueError(f"hist must be contiguous [{rows}, 1024]")
    lib = load_library()
    with torch.cuda.device(dev):
        _arm(events, dev)
        tail = (_ptr(weights), _ptr(block_table), _ptr(context_lens), int(B), int(next_n), int(P),
                int(max_pages), _ptr(logits), int(logits.stride(0)), _ptr(hist), _stream_ptr(dev))
        if mx:
            st = getattr(lib, name)(_ptr(q), _ptr(kv_pages), *tail)
        else:
            st = getattr(lib, name)(_ptr(q), _ptr(kv_pages), _ptr(k_scales), *tail)
    _check(name, st)


def indexer_logits(q, kv_pages, k_scales, weights, block_table, context_lens, next_n,
                   logits, hist=None, events=None):
    """Paged MQA logits (and histogram) on the current stream of q's device.

    q [B*next_n, 32, 128] uint8 (e4m3fn codes); kv_pages [P, 64, 128] uint8;
    k_scales [P, 64] float32; weights [B*next_n, 32] float32;
    block_table [B, max_pages] int32; context_lens [B*next_n] int32;
    logits [B*next_n, stride] float32 with unit column stride;
    hist [B*next_n, 1024] int32 or None (accumulated into).
    """
    _logits_call("indexer_logits", torch.float32, q, kv_pages, k_scales, weights, block_table,
                 context_lens, next_n, logits, hist, events)


def indexer_logits_f16(q, kv_pages, k_scales, weights, block_table, context_lens, next_n,
                       logits, hist=None, events=None):
    """indexer_logits writing float16 logits [B*next_n, stride] (stride % 8 == 0)."""
    _logits_call("indexer_logits_f16", torch.float16, q, kv_pages, k_scales, weights, block_table,
                 context_lens, next_n, logits, hist, events)


def indexer_logits_mxfp4(q, kv_pages, weights, block_table, context_lens, next_n, logits,
                         hist=None, events=None):
    """indexer_logits with packed MXFP4 keys: kv_pages [P, 64, 68] uint8 (64 bytes
    of E2M1 codes, then four E8M0 block scales per token); float32 logits."""
    _logits_call("indexer_logits_mxfp4", torch.float32, q, kv_pages, None, weights, block_table,
                 context_lens, next_n, logits, hist, events)


def _rows2(t, name, dtype, dev, rows=None):
    _need(t, name, dtype, dev, 2)
    if not t.is_contiguous() or (rows is not None and t.shape[0] != rows):
        raise ValueError(f"{name} must be contiguous [{rows if rows is not None else 'rows'}, n]")


def block_amax8(scores, context_lens, out, hist=None, block_lens=None, events=None):
    """Block maxima of 8 scores per row (newest block +inf) into out [rows, >= ceil(stride/8)];
    with ``hist`` [rows, 1024] int32 their coarse histogram is accumulated too, and
    ``block_lens`` [rows] int32 receives each row's block count ceil(len / 8) (the
    lengths the block top-k takes)."""
    dev = scores.device
    _need(scores, "scores", torch.float32, dev, 2)
    rows = scores.shape[0]
    _rows2(out, "out", torch.float32, dev, rows)
    _need(context_lens, "context_lens", torch.int32, dev, 1)
    if scores.stride(1) != 1 or tuple(context_lens.shape) != (rows,):
        raise ValueError("scores must have unit column stride; context_lens [rows]")
    lib = load_library()
    with torch.cuda.device(dev):
        _arm(events, dev)
        if hist is not None:
            _rows2(hist, "hist", torch.int32, dev, rows)
        if block_lens is not None:
            _need(block_lens, "block_lens", torch.int32, dev, 1)
            if tuple(block_lens.shape) != (rows,) or not block_lens.is_contiguous():
                raise ValueError("block_lens must be a contiguous int32 [rows]")
        st = lib.block_amax8(_ptr(scores), int(scores.stride(0)), _ptr(context_lens), int(rows), _ptr(out),
                             int(out.stride(0)), _ptr(hist), _ptr(block_lens), _stream_ptr(dev))
    _check("block_amax8", st)


def sort_candidate_blocks(blocks, context_lens, max_len, block_table, next_n, table, slots, sparse_lens,
                          events=None):
    """Ascending INT32_MAX-padded block tables, pool slots / 8 and sparse row lengths."""
    dev = blocks.device
    _rows2(blocks, "blocks", torch.int32, dev)
    rows, kb = blocks.shape
    _rows2(table, "table", torch.int32, dev, rows)
    _rows2(slots, "slots", torch.int32, dev, rows)
    _rows2(block_table, "block_table", torch.int32, dev)
    _need(context_lens, "context_lens", torch.int32, dev, 1)
    _need(sparse_lens, "sparse_lens", torch.int32, dev, 1)
    if table.shape[1] != kb or slots.shape[1] != kb:
        raise ValueError("table and slots must be [rows, kb] like blocks")
    lib = load_library()
    with torch.cuda.device(dev):
        _arm(events, dev)
        st = lib.sort_candidate_blocks(_ptr(blocks), int(kb), _ptr(context_lens), int(rows), int(max_len),
                                       _ptr(block_table), int(block_table.shape[1]), int(next_n),
                                       _ptr(table), _ptr(slots), _ptr(sparse_lens), _stream_ptr(dev))
    _check("sort_candidate_blocks", st)


def indexer_sparse_logits(q, kv_pages, k_scales, weights, table, slots, context_lens, logits,
                          events=None):
    """Logits of the listed 8-token blocks only: logits [rows, >= 8 kb].  With
    k_scales None, kv_pages are packed MXFP4 tokens [P, 64, 68]
    (indexer_sparse_logits_mxfp4)."""
    dev = q.device
    mx = k_scales is None
    _need(q, "q", torch.uint8, dev, 3)
    _need(kv_pages, "kv_pages", torch.uint8, dev, 3)
    if kv_pages.shape[1:] != ((PAGE_TOKENS, MXFP4_TOKEN_BYTES) if mx else (PAGE_TOKENS, HEAD_DIM)):
        raise ValueError("kv_pages must be [P, 64, 68] (MXFP4) or [P, 64, 128] with k_scales")
    if not mx:
        _need(k_scales, "k_scales", torch.float32, dev, 2)
    _need(weights, "weights", torch.float32, dev, 2)
    _rows2(table, "table", torch.int32, dev)
    rows, kb = table.shape
    _rows2(slots, "slots", torch.int32, dev, rows)
    _need(context_lens, "context_lens", torch.int32, dev, 1)
    _need(logits, "logits", torch.float32, dev, 2)
    if tuple(q.shape) != (rows, HEADS, HEAD_DIM) or tuple(weights.shape) != (rows, HEADS):
        raise ValueError(f"q [{rows}, 32, 128] and weights [{rows}, 32] (one per row)")
    if logits.shape[0] != rows or logits.stride(1) != 1:
        raise ValueError("logits must be [rows, stride] with unit column stride")
    lib = load_library()
    with torch.cuda.device(dev):
        _arm(events, dev)
        tail = (_ptr(weights), _ptr(table), _ptr(slots), int(kb), _ptr(context_lens), int(rows),
                int(kv_pages.shape[0]), _ptr(logits), int(logits.stride(0)), _stream_ptr(dev))
        if mx:
            st = lib.indexer_sparse_logits_mxfp4(_ptr(q), _ptr(kv_pages), *tail)
        else:
            st = lib.indexer_sparse_logits(_ptr(q), _ptr(kv_pages), _ptr(k_scales), *tail)
    _check("indexer_sparse_logits_mxfp4" if mx else "indexer_sparse_logits", st)


def indexer_prefill_logits(q, kv_pages, k_scales, weights, block_table, cu_q, row_lens, logits,
                           events=None):
    """Ragged prefill logits: request r owns rows cu_q[r] .. cu_q[r+1]-1; row t
    scores keys [0, row_lens[t]) of its request into logits [tokens, stride].
    With k_scales None, kv_pages are packed MXFP4 tokens
    (indexer_prefill_logits_mxfp4)."""
    dev = q.device
    mx = k_scales is None
    _need(q, "q", torch.uint8, dev, 3)
    _need(kv_pages, "kv_pages", torch.uint8, dev, 3)
    if kv_pages.shape[1:] != ((PAGE_TOKENS, MXFP4_TOKEN_BYTES) if mx else (PAGE_TOKENS, HEAD_DIM)):
        raise ValueError("kv_pages must be [P, 64, 68] (MXFP4) or [P, 64, 128] with k_scales")
    if not mx:
        _need(k_scales, "k_scales", torch.float32, dev, 2)
    _need(weights, "weights", torch.float32, dev, 2)
    _rows2(block_table, "block_table", torch.int32, dev)
    _need(cu_q, "cu_q", torch.int32, dev, 1)
    _need(row_lens, "row_lens", torch.int32, dev, 1)
    _need(logits, "logits", torch.float32, dev, 2)
    tokens = q.shape[0]
    requests = block_table.shape[0]
    if tuple(q.shape) != (tokens, HEADS, HEAD_DIM) or tuple(weights.shape) != (tokens, HEADS):
        raise ValueError(f"q [{tokens}, 32, 128] and weights [{tokens}, 32] (one per row)")
    if cu_q.shape[0] != requests + 1 or row_lens.shape[0] != tokens:
        raise ValueError("cu_q must be [requests + 1] and row_lens [tokens]")
    if logits.shape[0] != tokens or logits.stride(1) != 1:
        raise ValueError("logits must be [tokens, stride] with unit column stride")
    lib = load_library()
    with torch.cuda.device(dev):
        _arm(events, dev)
        tail = (_ptr(weights), _ptr(block_table), int(block_table.shape[1]), _ptr(cu_q), int(requests),
                int(tokens), _ptr(row_lens), int(kv_pages.shape[0]), _ptr(logits), int(logits.stride(0)),
                _stream_ptr(dev))
        if mx:
            st = lib.indexer_prefill_logits_mxfp4(_ptr(q), _ptr(kv_pages), *tail)
        else:
            st = lib.indexer_prefill_logits(_ptr(q), _ptr(kv_pages), _ptr(k_scales), *tail)
    _check("indexer_prefill_logits_mxfp4" if mx else "indexer_prefill_logits", st)


def sparse_to_logical(indices, table, out, events=None):
    """Sparse-row columns -> logical key positions (-1 stays -1)."""
    dev = indices.device
    _rows2(indices, "indices", torch.int32, dev)
    rows, k = indices.shape
    _rows2(table, "table", torch.int32, dev, rows)
    _rows2(out, "out", torch.int32, dev, rows)
    lib = load_library()
    with torch.cuda.device(dev):
        _arm(events, dev)
        st = lib.sparse_to_logical(_ptr(indices), int(k), _ptr(table), int(table.shape[1]), int(rows),
                                   _ptr(out), _stream_ptr(dev))
    _check("sparse_to_logical", st)


def sparse_topk(scores, hist, sparse_lens, k, key_dtype, table, out, events=None):
    """Top-k inside the sparse rows (float32 [rows, stride <= 16384]) written
    as logical key positions through ``table`` [rows, kb]: topk_rows followed
    by sparse_to_logical in one launch."""
    dev = scores.device
    _need(scores, "scores", torch.float32, dev, 2)
    rows = scores.shape[0]
    _need(sparse_lens, "sparse_lens", torch.int32, dev, 1)
    _rows2(table, "table", torch.int32, dev, rows)
    _rows2(out, "out", torch.int32, dev, rows)
    if scores.stride(1) != 1 or tuple(sparse_lens.shape) != (rows,) or out.shape[1] != k:
        raise ValueError("scores must have unit column stride; sparse_lens [rows]; out [rows, k]")
    if hist is not None:
        _rows2(hist, "hist", torch.int32, dev, rows)
    lib = load_library()
    with torch.cuda.device(dev):
        _arm(events, dev)
        st = lib.sparse_topk(_ptr(scores), int(scores.stride(0)), _ptr(hist), _ptr(sparse_lens), int(rows),
                             int(k), int(key_dtype), _ptr(table), int(table.shape[1]), _ptr(out),
                             _stream_ptr(dev))
    _check("sparse_topk", st)


def topk_workspace_bytes(rows: int, logits_stride: int, k: int) -> int:
    return int(load_library().topk_workspace_bytes(int(rows), int(logits_stride), int(k)))


def _topk_call(name, dtype, logits, hist, context_lens, k, key_dtype, indices, workspace, events):
    dev = logits.device
    _need(logits, "logits", dtype, dev, 2)
    _need(context_lens, "context_lens", torch.int32, dev, 1)
    _need(indices, "indices", torch.int32, dev, 2)
    rows = logits.shape[0]
    if logits.stride(1) != 1:
        raise ValueError("logits must have unit column stride")
    if tuple(context_lens.shape) != (rows,) or not context_lens.is_contiguous():
        raise ValueError(f"context_lens must be contiguous [{rows}]")
    if tuple(indices.shape) != (rows, k) or not indices.is_contiguous():
        raise ValueError(f"indices must be contiguous [{rows}, {k}]")
    if hist is not None:
        _need(hist, "hist", torch.int32, dev, 2)
        if tuple(hist.shape) != (rows, NUM_BINS) or not hist.is_contiguous():
            raise ValueError(f"hist must be contiguous [{rows}, 1024]")
    if name == "topk_rows_noalloc":
        workspace = None
    elif workspace is None:
        workspace = _device_workspace(dev, topk_workspace_bytes(rows, logits.stride(0), k))
    else:
        _need(workspace, "workspace", torch.uint8, dev)
    lib = load_library()
    with torch.cuda.device(dev):
        _arm(events, dev)
        head = (_ptr(logits), int(logits.stride(0)), _ptr(hist), _ptr(context_lens), int(rows), int(k))
        if workspace is None:
            tail = (_ptr(indices), _stream_ptr(dev))
        else:
            tail = (_ptr(indices), _ptr(workspace), int(workspace.numel()), _stream_ptr(dev))
        if key_dtype is None:
            st = getattr(lib, name)(*head, *tail)
        else:
            st = getattr(lib, name)(*head, int(key_dtype), *tail)
    _check(name, st)


# One workspace per device for calls that pass none, allocated the first time
# a call needs more than the current one holds and reused after that.
_workspaces: dict = {}


def _device_workspace(dev: torch.device, need: int) -> torch.Tensor:
    key = dev.index if dev.index is not None else torch.cuda.current_device()
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < need:
        ws = torch.zeros(max(need, 256), dtype=torch.uint8, device=dev)
        _workspaces[key] = ws
    return ws


def topk_rows(logits, hist, context_lens, k, key_dtype, indices, workspace=None, events=None):
    """Exact per-row top-k indices of float32 scores into ``indices`` [rows, k].

    ``workspace`` is a uint8 GPU tensor of at least topk_workspace_bytes()
    bytes (no initialisation needed).  When None, the device's shared
    workspace of this module is used (allocated, or grown, only when a call
    needs more than it holds); calls that use it must be ordered on one
    stream.
    """
    _topk_call("topk_rows", torch.float32, logits, hist, context_lens, k, key_dtype, indices,
               workspace, events)


def topk_rows_f16(logits, hist, context_lens, k, indices, workspace=None, events=None):
    """topk_rows over float16 scores [rows, stride] (stride % 8 == 0), FP16 keys."""
    _topk_call("topk_rows_f16", torch.float16, logits, hist, context_lens, k, None, indices,
               workspace, events)


def topk_rows_noalloc(logits, hist, context_lens, k, key_dtype, indices, events=None):
    """topk_rows with the library's fixed per-GPU scratch instead of a workspace
    (at most 128 rows when rows hold more than 16384 scores); allocates
    nothing.  Calls that overlap on one GPU race on that scratch."""
    _topk_call("topk_rows_noalloc", torch.float32, logits, hist, context_lens, k, key_dtype, indices,
               None, events)


def score_histogram(scores, context_lens, hist):
    """Add the coarse bins of every live non-NaN score of each row to ``hist``."""
    dev = scores.device
    _need(scores, "scores", torch.float32, dev, 2)
    _need(context_lens, "context_lens", torch.int32, dev, 1)
    _need(hist, "hist", torch.int32, dev, 2)
    rows = scores.shape[0]
    if scores.stride(1) != 1:
        raise ValueError("scores must have unit column stride")
    if tuple(context_lens.shape) != (rows,) or not context_lens.is_contiguous():
        raise ValueError(f"context_lens must be contiguous [{rows}]")
    if tuple(hist.shape) != (rows, NUM_BINS) or not hist.is_contiguous():
        raise ValueError(f"hist must be contiguous [{rows}, 1024]")
    lib = load_library()
    with torch.cuda.device(dev):
        st = lib.score_histogram(_ptr(scores), int(scores.stride(0)), _ptr(context_lens),
                                 int(rows), _ptr(hist), _stream_ptr(dev))
    _check("score_histogram", st)


_entry_points: dict = {}


def _launch(name, dev, events, *args):
    """One call of the C entry point on the current stream of ``dev``."""
    fn = _entry_points.get(name)
    if fn is None:
        fn = _entry_points[name] = getattr(load_library(), name)
    if dev.index == torch.cuda.current_device():
        if events is not None:
            _arm(events, dev)
        st = fn(*args, _stream_ptr(dev))
    else:
        with torch.cuda.device(dev):
            _arm(events, dev)
            st = fn(*args, _stream_ptr(dev))
    if st:
        _check(name, st)


def _need_shaped(t, name, dtype, dev, shape):
    """A contiguous tensor of ``dtype`` and ``shape`` on ``dev``.  The calls of a
    decode step take longer on the host than on the GPU, so what holds is seen
    in one condition and only what does not is looked into."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.is_cuda and t.shape == shape and
            t.is_contiguous() and t.device == dev):
        _need(t, name, dtype, dev, len(shape))
        raise ValueError(f"{name} must be contiguous {list(shape)}")


def _append_call(name, dim, dtypes, rows, positions, slots, rope, pages, tail, interleaved, events):
    dev, dtype = rows.device, rows.dtype
    if dtype not in dtypes:
        raise TypeError(f"rows must be one of {dtypes}, got {dtype}")
    _need(rows, "rows", dtype, dev, 2)
    tokens, width = rows.shape
    stride, unit = rows.stride()
    if width != dim or unit != 1:
        raise ValueError(f"rows must be [tokens, {dim}] with unit column stride")
    if tokens == 1:
        stride = dim  # the stride of a single row carries no meaning
    _need_shaped(positions, "positions", torch.int32, dev, (tokens,))
    _need_shaped(slots, "slots", torch.int32, dev, (tokens,))
    max_positions = rope.shape[0]
    _need_shaped(rope, "rope", torch.float32, dev, (max_positions, ROPE_DIM))
    _launch(name, dev, events, rows.data_ptr(), stride, VALUE_DTYPES[dtype], positions.data_ptr(), slots.data_ptr(),
            rope.data_ptr(), max_positions, 1 if interleaved else 0, tokens, pages.shape[0], pages.data_ptr(), *tail)


def index_k_append(k, positions, slots, rope, kv_pages, k_scales, interleaved=False, events=None):
    """Rotate index keys by their positions and append them to the FP8 cache.

    k [tokens, 128] bfloat16, float16 or float32 with unit column stride and
    16-byte rows (a slice of a wider tensor is fine); positions [tokens] int32;
    slots [tokens] int32 = page * 64 + place, negative to write nothing; rope
    [max_positions, 64] float32, 32 cosines then 32 sines; kv_pages [P, 64, 128]
    uint8 and k_scales [P, 64] float32 as indexer_logits reads them.  The first
    64 dimensions are rotated in pairs (i, i + 32), or (2i, 2i + 1) with
    ``interleaved``.
    """
    dev, pages = k.device, kv_pages.shape[0]
    _need_shaped(kv_pages, "kv_pages", torch.uint8, dev, (pages, PAGE_TOKENS, HEAD_DIM))
    _need_shaped(k_scales, "k_scales", torch.float32, dev, (pages, PAGE_TOKENS))
    _append_call("index_k_append", HEAD_DIM, (torch.bfloat16, torch.float16, torch.float32), k, positions, slots,
                 rope, kv_pages, (_ptr(k_scales),), interleaved, events)


def index_k_append_mxfp4(k, positions, slots, rope, kv_pages, interleaved=False, events=None):
    """index_k_append into packed MXFP4 tokens: kv_pages [P, 64, 68] uint8.  A key
    with a NaN or an infinity has logits of 0 here, which can be selected (an FP8
    key's are NaN, which cannot): keep such keys out."""
    _need_shaped(kv_pages, "kv_pages", torch.uint8, k.device, (kv_pages.shape[0], PAGE_TOKENS, MXFP4_TOKEN_BYTES))
    _append_call("index_k_append_mxfp4", HEAD_DIM, (torch.bfloat16, torch.float16, torch.float32), k, positions,
                 slots, rope, kv_pages, (), interleaved, events)


def latent_append(kv, positions, slots, rope, latent_pages, interleaved=False, events=None):
    """Append rows of 512 latent and 64 rotated dimensions to the latent cache.

    kv [tokens, 576] bfloat16 or float16 (unit column stride, 16-byte rows);
    latent_pages [P, 64, 576] of the same type; positions, slots, rope and
    ``interleaved`` as for index_k_append; dimensions 512..575 are rotated.
    """
    _need_shaped(latent_pages, "latent_pages", kv.dtype, kv.device, (latent_pages.shape[0], PAGE_TOKENS, LATENT_ROW))
    _append_call("latent_append", LATENT_ROW, (torch.bfloat16, torch.float16), kv, positions, slots, rope,
                 latent_pages, (), interleaved, events)


def latent_append_mxfp4(kv, positions, slots, rope, latent_pages, interleaved=False, events=None):
    """latent_append into 4-bit rows: latent_pages [P, 64, 400] uint8, per token 256
    bytes of E2M1 codes, 16 E8M0 bytes (one per 32 dimensions) and the 64 rotated
    dimensions in kv's type.  A block with a NaN or an infinity becomes NaN."""
    _need_shaped(latent_pages, "latent_pages", torch.uint8, kv.device,
                 (latent_pages.shape[0], PAGE_TOKENS, LATENT_MXFP4_ROW))
    _append_call("latent_append_mxfp4", LATENT_ROW, (torch.bfloat16, torch.float16), kv, positions, slots, rope,
                 latent_pages, (), interleaved, events)


def axis_map(axis_of) -> int:
    """The axis of each of the 32 angles (a sequence of 32 numbers below 4) as the
    integer that the rotations take: two bits per angle."""
    axis_of = [int(a) for a in axis_of]
    if len(axis_of) != ROPE_DIM // 2 or not all(0 <= a < MAX_AXES for a in axis_of):
        raise ValueError(f"axis_of must be {ROPE_DIM // 2} axes in 0 .. {MAX_AXES - 1}")
    return sum(a << (2 * i) for i, a in enumerate(axis_of))


def _rotary_positions(positions, rope, dev, tokens):
    """positions [tokens] or [axes, tokens] -> axes, rows of the table."""
    axes = 1 if positions.dim() == 1 else positions.shape[0]
    _need_shaped(positions, "positions", torch.int32, dev, (tokens,) if positions.dim() == 1 else (axes, tokens))
    max_positions = rope.shape[0]
    _need_shaped(rope, "rope", torch.float32, dev, (max_positions, ROPE_DIM))
    return axes, max_positions


def axis_rotations(positions, axis_map, rope, out, events=None):
    """Each token's cosines and sines of several axes in one row.

    positions [axes, tokens] int32; axis_map as axis_map() gives it; rope
    [max_positions, 64] float32 as for the appends; out [tokens, 64] float32.  The
    appends take ``out`` as their table, with positions 0 .. tokens - 1.
    """
    dev, tokens = out.device, out.shape[0]
    _need_shaped(out, "out", torch.float32, dev, (tokens, ROPE_DIM))
    axes, max_positions = _rotary_positions(positions, rope, dev, tokens)
    _launch("axis_rotations", dev, events, positions.data_ptr(), axes, axis_map, tokens, rope.data_ptr(),
            max_positions, out.data_ptr())


def _strided_rows(t, name, dtype, dev, shape):
    """Strides of [tokens, heads, dim] rows; those of a dimension of one element
    carry no meaning and become those of a packed tensor."""
    token, head, unit = t.stride() if isinstance(t, torch.Tensor) and t.dim() == 3 else (0, 0, 0)
    if not (unit == 1 and t.shape == shape and t.dtype is dtype and t.is_cuda and t.device == dev):
        _need(t, name, dtype, dev, 3)
        raise ValueError(f"{name} must be {list(shape)} with unit stride in the last dimension")
    tokens, heads, dim = shape
    if heads == 1:
        head = dim
    if tokens == 1:
        token = heads * max(head, dim)
    return token, head


def rotate_queries(x, positions, rope, out, axis_map=0, interleaved=False, events=None):
    """Turn the rotated part of every head of every query row by its position.

    x and out [tokens, heads, 64] bfloat16 or float16, any strides with 16-byte
    rows (such as slices of wider tensors); out may be x itself, otherwise they
    share no element.  positions [tokens] int32, or [axes, tokens] with
    ``axis_map``; rope [max_positions, 64] float32; pairs (i, i + 32), or
    (2i, 2i + 1) with ``interleaved``.
    """
    dev, dtype = x.device, x.dtype
    if dtype is not torch.bfloat16 and dtype is not torch.float16:
        raise TypeError(f"x must be bfloat16 or float16, got {dtype}")
    if x.dim() != 3:
        raise ValueError(f"x must have 3 dims, got {tuple(x.shape)}")
    tokens, heads = x.shape[:2]
    shape = (tokens, heads, ROPE_DIM)
    strides, out_strides = _strided_rows(x, "x", dtype, dev, shape), _strided_rows(out, "out", dtype, dev, shape)
    axes, max_positions = _rotary_positions(positions, rope, dev, tokens)
    _launch("rotate_queries", dev, events, x.data_ptr(), *strides, VALUE_DTYPES[dtype], positions.data_ptr(), axes,
            axis_map, rope.data_ptr(), max_positions, 1 if interleaved else 0, tokens, heads, out.data_ptr(),
            *out_strides)


def rotate_index_queries(q, positions, rope, codes, axis_map=0, interleaved=False, events=None):
    """Turn the first 64 of 128 dimensions of the indexer's queries and write all of
    them as the E4M3 codes that indexer_logits reads.

    q [tokens, 32, 128] bfloat16, float16 or float32 with 16-byte rows; codes
    [tokens, 32, 128] uint8; other arguments as for rotate_queries.  Values beyond
    +-448, infinities among them, become +-448; nothing is scaled: divide a head's
    row by a factor beforehand and multiply its weight by it where that matters.
    """
    dev, dtype = q.device, q.dtype
    if dtype not in VALUE_DTYPES:
        raise TypeError(f"q must be bfloat16, float16 or float32, got {dtype}")
    if q.dim() != 3:
        raise ValueError(f"q must have 3 dims, got {tuple(q.shape)}")
    tokens = q.shape[0]
    shape = (tokens, HEADS, HEAD_DIM)
    strides = _strided_rows(q, "q", dtype, dev, shape)
    _need_shaped(codes, "codes", torch.uint8, dev, shape)
    axes, max_positions = _rotary_positions(positions, rope, dev, tokens)
    _launch("rotate_index_queries", dev, events, q.data_ptr(), *strides, VALUE_DTYPES[dtype], positions.data_ptr(),
            axes, axis_map, rope.data_ptr(), max_positions, 1 if interleaved else 0, tokens, codes.data_ptr())


class PageCaches:
    """The caches that one pool of page ids serves, as copy_pages takes them: GPU
    tensors [num_pages, 64, ...], contiguous, of the same number of pages (index
    codes, scales and latent rows of all layers).  Holds on to the tensors."""

    def __init__(self, caches):
        caches = list(caches)
        if not 1 <= len(caches) <= MAX_CACHES:
            raise ValueError(f"1 .. {MAX_CACHES} caches, got {len(caches)}")
        dev, pages = caches[0].device, caches[0].shape[0]
        for i, t in enumerate(caches):
            _need(t, f"caches[{i}]", t.dtype, dev)
            if t.dim() < 2 or t.shape[0] != pages or t.shape[1] != PAGE_TOKENS or not t.is_contiguous():
                raise ValueError(f"caches[{i}] must be contiguous [{pages}, {PAGE_TOKENS}, ...], got {tuple(t.shape)}")
        self.tensors, self.device, self.num_pages = caches, dev, pages
        self.pointers = (ctypes.c_void_p * len(caches))(*[t.data_ptr() for t in caches])
        self.token_bytes = (ctypes.c_int32 * len(caches))(*[t[0, 0].numel() * t.element_size() for t in caches])


def copy_pages(caches, src, dst, tokens=None, count=None, events=None):
    """Page src[i] to page dst[i] in every cache (PageCaches, or a list of tensors
    that becomes one for the call).

    src, dst [n] int32, entries outside the pool (-1) copy nothing; tokens [n] int32:
    how many of a page's first tokens, or None for all; count int32 [1]: only the
    first so many entries.  No destination is also a source or given twice.
    """
    if not isinstance(caches, PageCaches):
        caches = PageCaches(caches)
    dev, n = caches.device, src.shape[0]
    _need_shaped(src, "src", torch.int32, dev, (n,))
    _need_shaped(dst, "dst", torch.int32, dev, (n,))
    if tokens is not None:
        _need_shaped(tokens, "tokens", torch.int32, dev, (n,))
    if count is not None:
        _need_shaped(count, "count", torch.int32, dev, (1,))
    _launch("copy_pages", dev, events, caches.pointers, caches.token_bytes, len(caches.tensors), caches.num_pages,
            src.data_ptr(), dst.data_ptr(), _ptr(tokens), _ptr(count), n)


def pages_workspace_bytes(requests: int, num_pages: int) -> int:
    """Workspace of fork_pages and compact_pages."""
    return int(load_library().pages_workspace_bytes(int(requests), int(num_pages)))


def _pool(block_table, lens, refs, of_requests, of_pages):
    """Shapes of a pool -- requests, max_pages, num_pages -- and the checks of the
    tensors, by name, that hold an int32 for each request and for each page."""
    dev = block_table.device
    if block_table.dim() != 2:
        raise ValueError(f"block_table must have 2 dims, got {tuple(block_table.shape)}")
    requests, max_pages = block_table.shape
    num_pages = refs.shape[0]
    _need_shaped(block_table, "block_table", torch.int32, dev, (requests, max_pages))
    _need_shaped(lens, "lens", torch.int32, dev, (requests,))
    _need_shaped(refs, "refs", torch.int32, dev, (num_pages,))
    for name, t in of_requests.items():
        _need_shaped(t, name, torch.int32, dev, (requests,))
    for name, t in of_pages.items():
        _need_shaped(t, name, torch.int32, dev, (num_pages,))
    return dev, requests, max_pages, num_pages


def _pool_workspace(workspace, requests, num_pages, dev):
    if workspace is None:
        return torch.empty(pages_workspace_bytes(requests, num_pages), dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", torch.uint8, dev)
    if not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return workspace


def release_pages(block_table, lens, ended, refs, new_lens, new_refs, events=None):
    """Requests with ended[b] != 0 give up their pages.

    block_table [requests, max_pages] int32, of which request b holds the first
    ceil(lens[b] / 64) entries; refs [num_pages] int32 holders of each page (0:
    free); ended [requests] int32.  new_lens and new_refs are written, and may be
    lens and refs.
    """
    dev, requests, max_pages, num_pages = _pool(block_table, lens, refs, dict(ended=ended, new_lens=new_lens),
                                                dict(new_refs=new_refs))
    _launch("release_pages", dev, events, block_table.data_ptr(), lens.data_ptr(), ended.data_ptr(), requests,
            max_pages, refs.data_ptr(), num_pages, new_lens.data_ptr(), new_refs.data_ptr())


def fork_pages(block_table, lens, parents, refs, new_lens, new_refs, src, dst, tokens, counts, workspace=None,
               events=None):
    """Request b without tokens becomes a copy of request parents[b] (negative: none).

    It shares the full pages; the page that the parent has begun is to be copied to
    the lowest free one: src, dst, tokens [requests] int32 name the copies as
    copy_pages takes them (-1, -1, 0: none).  Rows of block_table are written for
    the forked requests; new_lens and new_refs may be lens and refs.  counts [2]
    int32: pages taken, and requests not forked because none was left.
    ``workspace``: pages_workspace_bytes(requests, num_pages) bytes, allocated for
    the call when None.
    """
    dev, requests, max_pages, num_pages = _pool(
        block_table, lens, refs, dict(parents=parents, new_lens=new_lens, src=src, dst=dst, tokens=tokens),
        dict(new_refs=new_refs))
    _need_shaped(counts, "counts", torch.int32, dev, (2,))
    workspace = _pool_workspace(workspace, requests, num_pages, dev)
    _launch("fork_pages", dev, events, block_table.data_ptr(), lens.data_ptr(), parents.data_ptr(), requests,
            max_pages, refs.data_ptr(), num_pages, new_lens.data_ptr(), new_refs.data_ptr(), src.data_ptr(),
            dst.data_ptr(), tokens.data_ptr(), counts.data_ptr(), workspace.data_ptr(), workspace.numel())


def compact_pages(block_table, lens, refs, new_table, new_refs, src, dst, counts, workspace=None, events=None):
    """Plan the moves that make the pool dense: with L pages held, the held pages from
    L on go to the free ones below L.

    src and dst [num_pages] int32 name the moves (-1 behind the last), counts [2]
    int32 is L and their number: copy_pages(caches, src, dst, count=counts[1:]).
    new_table [requests, max_pages] and new_refs [num_pages] say where the pages
    then are, and may be block_table and refs.
    """
    dev, requests, max_pages, num_pages = _pool(block_table, lens, refs, {}, dict(new_refs=new_refs, src=src, dst=dst))
    _need_shaped(counts, "counts", torch.int32, dev, (2,))
    _need_shaped(new_table, "new_table", torch.int32, dev, (requests, max_pages))
    workspace = _pool_workspace(workspace, requests, num_pages, dev)
    _launch("compact_pages", dev, events, block_table.data_ptr(), lens.data_ptr(), requests, max_pages,
            refs.data_ptr(), num_pages, new_table.data_ptr(), new_refs.data_ptr(), src.data_ptr(), dst.data_ptr(),
            counts.data_ptr(), workspace.data_ptr(), workspace.numel())


def attention_workspace_bytes(rows: int, heads: int, requests: int) -> int:
    """Workspace of paged_attention and sparse_attention."""
    return int(load_library().attention_workspace_bytes(int(rows), int(heads), int(requests)))


def shared_prefix_workspace_bytes(rows: int, heads: int, requests: int) -> int:
    return int(load_library().shared_prefix_workspace_bytes(int(rows), int(heads), int(requests)))


def _attention_call(name, q, latent_pages, block_table, keys, next_n, cu_q, starts, prefix_pages, scale, out, lse,
                    softcap, slopes, row_positions, workspace, events):
    """keys: row_lens [rows], or the selected keys [rows, k] (sparse_attention).
    The _mxfp4 entry points take the cache in 4-bit rows."""
    dev, dtype = q.device, q.dtype
    if dtype is not torch.bfloat16 and dtype is not torch.float16:
        raise TypeError(f"q must be bfloat16 or float16, got {dtype}")
    if q.dim() != 3:
        raise ValueError(f"q must have 3 dims, got {tuple(q.shape)}")
    rows, heads = q.shape[:2]
    _need_shaped(q, "q", dtype, dev, (rows, heads, LATENT_ROW))
    pages = latent_pages.shape[0]
    if name.endswith("_mxfp4"):
        _need_shaped(latent_pages, "latent_pages", torch.uint8, dev, (pages, PAGE_TOKENS, LATENT_MXFP4_ROW))
    else:
        _need_shaped(latent_pages, "latent_pages", dtype, dev, (pages, PAGE_TOKENS, LATENT_ROW))
    if block_table.dim() != 2:
        raise ValueError(f"block_table must have 2 dims, got {tuple(block_table.shape)}")
    requests, max_pages = block_table.shape
    _need_shaped(block_table, "block_table", torch.int32, dev, (requests, max_pages))
    sparse = name.startswith("sparse_attention")
    if sparse:
        _need_shaped(keys, "indices", torch.int32, dev, (rows, keys.shape[-1]))
    else:
        _need_shaped(keys, "row_lens", torch.int32, dev, (rows,))
    if starts is not None:
        _need_shaped(starts, "row_starts", torch.int32, dev, (rows,))
    if cu_q is not None:
        _need_shaped(cu_q, "cu_q", torch.int32, dev, (requests + 1,))
    if row_positions is not None:
        _need_shaped(row_positions, "row_positions", torch.int32, dev, (rows,))
    if slopes is not None:
        _need_shaped(slopes, "slopes", torch.float32, dev, (heads,))
    _need_shaped(out, "out", dtype, dev, (rows, heads, LATENT_DIM))
    if lse is not None:
        _need_shaped(lse, "lse", torch.float32, dev, (rows, heads))
    if workspace is None:
        # the caching allocator orders it with the stream, and inside a graph
        # capture it belongs to that graph
        size = shared_prefix_workspace_bytes if prefix_pages is not None else attention_workspace_bytes
        workspace = torch.empty(size(rows, heads, requests), dtype=torch.uint8, device=dev)
    else:
        _need(workspace, "workspace", torch.uint8, dev)
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
    head = (q.data_ptr(), latent_pages.data_ptr(), VALUE_DTYPES[dtype], block_table.data_ptr(), keys.data_ptr())
    shape = (rows, heads, requests, next_n)
    tail = (pages, max_pages, scale, softcap, _ptr(slopes), _ptr(row_positions), out.data_ptr(),
            _ptr(lse), workspace.data_ptr(), workspace.numel())
    if sparse:
        _launch(name, dev, events, *head, keys.shape[1], _ptr(cu_q), *shape, *tail)
    elif prefix_pages is not None:
        _launch(name, dev, events, *head, _ptr(starts), *shape, prefix_pages, *tail)
    else:
        _launch(name, dev, events, *head, _ptr(starts), _ptr(cu_q), *shape, *tail)


def paged_attention(q, latent_pages, block_table, row_lens, next_n, scale, out, lse=None, cu_q=None, row_starts=None,
                    softcap=0.0, slopes=None, row_positions=None, workspace=None, events=None):
    """Attention of every row over its request's pages of the latent cache.

    q [rows, heads, 576] bfloat16 or float16; latent_pages [P, 64, 576] of the
    same type, whose first 512 dimensions are the values; block_table
    [requests, max_pages] int32; row_lens [rows] int32: row r sees keys
    row_starts[r] (default 0) up to row_lens[r].  next_n rows per request, or
    next_n = 0 with cu_q [requests + 1] int32 for a ragged batch.  Scores are
    scale q . k, then softcap * tanh(z / softcap) if softcap > 0, then minus
    slopes[h] * |row_positions[r] - s| (default position row_lens - 1).  The work
    is sized by the block table's width, so a table much wider than the rows'
    lengths costs time.
    out [rows, heads, 512] of q's type; lse [rows, heads] float32 or None.  A
    row that sees no key gets out 0 and lse -inf.

    ``workspace`` is a uint8 GPU tensor of attention_workspace_bytes(rows,
    heads, requests) bytes, allocated for the call when None; calls that share
    one must be ordered on one stream.
    """
    _attention_call("paged_attention", q, latent_pages, block_table, row_lens, next_n, cu_q, row_starts, None, scale,
                    out, lse, softcap, slopes, row_positions, workspace, events)


def shared_prefix_attention(q, latent_pages, block_table, row_lens, next_n, prefix_pages, scale, out, lse=None,
                            row_starts=None, softcap=0.0, slopes=None, row_positions=None, workspace=None,
                            events=None):
    """paged_attention for a batch whose requests' first ``prefix_pages`` pages
    are the same (the first entries of every block_table row): their keys are
    read once for all rows.  Workspace: shared_prefix_workspace_bytes(), which
    grows with the batch (about 4 KB for each row and head, with every request's
    rows times heads rounded up to 128) and is allocated for the call when None."""
    _attention_call("shared_prefix_attention", q, latent_pages, block_table, row_lens, next_n, None, row_starts,
                    prefix_pages, scale, out, lse, softcap, slopes, row_positions, workspace, events)


def sparse_attention(q, latent_pages, block_table, indices, next_n, scale, out, lse=None, cu_q=None, softcap=0.0,
                     slopes=None, row_positions=None, workspace=None, events=None):
    """Attention of every row over its selected keys: indices [rows, k] int32,
    logical key positions as topk_rows gives them (-1 padding is skipped).
    Other arguments as for paged_attention; slopes need row_positions."""
    _attention_call("sparse_attention", q, latent_pages, block_table, indices, next_n, cu_q, None, None, scale, out,
                    lse, softcap, slopes, row_positions, workspace, events)


def paged_attention_mxfp4(q, latent_pages, block_table, row_lens, next_n, scale, out, lse=None, cu_q=None,
                          row_starts=None, softcap=0.0, slopes=None, row_positions=None, workspace=None, events=None):
    """paged_attention over the 4-bit latent cache: latent_pages [P, 64, 400] uint8 as
    latent_append_mxfp4 writes it, from rows of q's type."""
    _attention_call("paged_attention_mxfp4", q, latent_pages, block_table, row_lens, next_n, cu_q, row_starts, None,
                    scale, out, lse, softcap, slopes, row_positions, workspace, events)


def shared_prefix_attention_mxfp4(q, latent_pages, block_table, row_lens, next_n, prefix_pages, scale, out, lse=None,
                                  row_starts=None, softcap=0.0, slopes=None, row_positions=None, workspace=None,
                                  events=None):
    """shared_prefix_attention over the 4-bit latent cache [P, 64, 400] uint8."""
    _attention_call("shared_prefix_attention_mxfp4", q, latent_pages, block_table, row_lens, next_n, None, row_starts,
                    prefix_pages, scale, out, lse, softcap, slopes, row_positions, workspace, events)


def sparse_attention_mxfp4(q, latent_pages, block_table, indices, next_n, scale, out, lse=None, cu_q=None,
                           softcap=0.0, slopes=None, row_positions=None, workspace=None, events=None):
    """sparse_attention over the 4-bit latent cache [P, 64, 400] uint8."""
    _attention_call("sparse_attention_mxfp4", q, latent_pages, block_table, indices, next_n, cu_q, None, None, scale,
                    out, lse, softcap, slopes, row_positions, workspace, events)


def _read_probe(name: str, src: torch.Tensor, sink: torch.Tensor, events) -> None:
    if src.device.type != "cuda" or not src.is_contiguous():
        raise ValueError("src must be a contiguous GPU tensor")
    _need(sink, "sink", torch.int32, src.device)
    lib = load_library()
    nbytes = src.numel() * src.element_size()
    with torch.cuda.device(src.device):
        _arm(events, src.device)
        st = getattr(lib, name)(_ptr(src), nbytes - nbytes % 16, _ptr(sink), _stream_ptr(src.device))
    _check(name, st)


def hbm_read_probe(src: torch.Tensor, sink: torch.Tensor, events=None) -> None:
    """Stream all bytes of ``src`` (contiguous GPU tensor) once with ordinary
    loads (a cache sweep for large buffers); checksum to sink."""
    _read_probe("hbm_read_probe", src, sink, events)


def hbm_read_probe_nt(src: torch.Tensor, sink: torch.Tensor, events=None) -> None:
    """hbm_read_probe with non-temporal loads: the contiguous read ceiling."""
    _read_probe("hbm_read_probe_nt", src, sink, events)


def hbm_gather_probe(kv_pages: torch.Tensor, k_scales: torch.Tensor, page_list: torch.Tensor,
                     sink: torch.Tensor, events=None) -> None:
    """Read the FP8 K pages (and their scales) listed in ``page_list`` once,
    the way the paged K stream is read; checksum to ``sink``."""
    dev = kv_pages.device
    _need(kv_pages, "kv_pages", torch.uint8, dev, 3)
    _need(k_scales, "k_scales", torch.float32, dev, 2)
    _need(page_list, "page_list", torch.int32, dev, 1)
    _need(sink, "sink", torch.int32, dev)
    if not (kv_pages.is_contiguous() and k_scales.is_contiguous() and page_list.is_contiguous()):
        raise ValueError("kv_pages, k_scales and page_list must be contiguous")
    if tuple(kv_pages.shape[1:]) != (PAGE_TOKENS, HEAD_DIM):
        raise ValueError("kv_pages must be [num_pages, 64, 128]")
    lib = load_library()
    with torch.cuda.device(dev):
        _arm(events, dev)
        st = lib.hbm_gather_probe(_ptr(kv_pages), _ptr(k_scales), _ptr(page_list), int(page_list.numel()),
                                  int(kv_pages.shape[0]), _ptr(sink), _stream_ptr(dev))
    _check("hbm_gather_probe", st)


def mfma_valu_probe(mode: int, waves_per_simd: int, iters: int, out: torch.Tensor, events=None) -> None:
    """MFMA / VALU co-issue probe: mode 0 fp8 MFMAs only, 1 fp32 FMAs only,
    2 both (independent, eight FMAs per MFMA); ``out`` float32 with at least
    CUs * waves_per_simd * 256 elements."""
    dev = out.device
    _need(out, "out", torch.float32, dev)
    if not out.is_contiguous():
        raise ValueError("out must be contiguous")
    lib = load_library()
    with torch.cuda.device(dev):
        _arm(events, dev)
        st = lib.mfma_valu_probe(int(mode), int(waves_per_simd), int(iters), _ptr(out), int(out.numel()),
                                 _stream_ptr(dev))
    _check("mfma_valu_probe", st)
