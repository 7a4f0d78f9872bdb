"""Python binding of libmla.so (the C ABI in include/mla.h): argument marshalling only.

Every step of the decode path runs in the library's CUDA kernels; PyTorch tensors are used
only as device buffers (their data pointers are passed through) and for the current stream.
There is no fallback: if the library is missing or fails to load, importing this package
raises.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmla.so")

N_HEADS, D_HEAD, D_LATENT, D_ROPE, D_ROW, PAGE_SIZE = 128, 128, 512, 64, 576, 64

STATUS = {0: "MLA_OK", 1: "MLA_ERR_INVALID_ARG", 2: "MLA_ERR_UNSUPPORTED", 3: "MLA_ERR_WORKSPACE",
          4: "MLA_ERR_CUDA", 5: "MLA_ERR_DEVICE"}
DEVERR_POS_RANGE, DEVERR_BLOCK_RANGE, DEVERR_SEQLEN_RANGE, DEVERR_WAIT_TIMEOUT = 1, 2, 4, 8


class MlaError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {STATUS.get(status, status)}")
        self.status = status


class CacheDesc(ctypes.Structure):
    _fields_ = [("page_size", ctypes.c_int32), ("max_seq_len", ctypes.c_int32),
                ("max_blocks_per_seq", ctypes.c_int32), ("num_seqs", ctypes.c_int32),
                ("num_rows", ctypes.c_int64)]


def contiguous_desc(num_seqs: int, max_seq_len: int) -> CacheDesc:
    return CacheDesc(0, max_seq_len, 0, num_seqs, num_seqs * max_seq_len)


def paged_desc(num_seqs: int, max_blocks_per_seq: int, num_blocks: int) -> CacheDesc:
    return CacheDesc(PAGE_SIZE, max_blocks_per_seq * PAGE_SIZE, max_blocks_per_seq, num_seqs,
                     num_blocks * PAGE_SIZE)


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python mla_latent_kv_20_b200/build.py` "
                          "(or __graft_entry__.build()); there is no non-CUDA fallback")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, I64, F32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    sigs = {
        "mla_status_string": (ctypes.c_char_p, [ctypes.c_int]),
        "mla_version": (I32, []),
        "mla_cache_append": (ctypes.c_int, [P, P, P, P, P, P, CacheDesc, I32, F32, P]),
        "mla_cache_append_fp8": (ctypes.c_int, [P, P, P, P, P, P, P, CacheDesc, I32, F32, P]),
        "mla_decode_attn_fp8": (ctypes.c_int, [P, P, P, P, P, CacheDesc, I32, F32, I32, P, SZ, P, P, P]),
        "mla_project_append": (ctypes.c_int, [P, P, P, P, P, P, P, CacheDesc, I32, F32, P]),
        "mla_output_proj": (ctypes.c_int, [P, P, P, I32, P]),
        "mla_append_absorb": (ctypes.c_int, [P, P, P, P, P, P, CacheDesc, I32, P, P, P, P, P, I32, F32, P]),
        "mla_selftest_wait_timeout": (ctypes.c_int, [ctypes.c_uint32, P, P]),
        "mla_absorb_q": (ctypes.c_int, [P, P, P, P, P, I32, F32, P]),
        "mla_decode_num_splits": (I32, [I32, I32, I32]),
        "mla_decode_workspace_size": (SZ, [I32, I32, I32]),
        "mla_decode_attn": (ctypes.c_int, [P, P, P, P, CacheDesc, I32, F32, I32, P, SZ, P, P, P]),
        "mla_prefill_attn": (ctypes.c_int, [P, P, P, P, P, CacheDesc, I32, F32, I32, P, SZ, P, P, P]),
        "mla_decode_attn_window": (ctypes.c_int, [P, P, P, P, CacheDesc, I32, I32, I32, F32, I32, P, SZ, P, P, P]),
        "mla_decode_attn_window_fp8": (ctypes.c_int,
                                       [P, P, P, P, P, CacheDesc, I32, I32, I32, F32, I32, P, SZ, P, P, P]),
        "mla_prefill_attn_window": (ctypes.c_int,
                                    [P, P, P, P, P, CacheDesc, I32, I32, I32, F32, I32, P, SZ, P, P, P]),
        "mla_window_span": (I32, [I32, I32, I32]),
        "mla_cache_append_at": (ctypes.c_int, [P, P, P, P, P, P, P, CacheDesc, I32, F32, P]),
        "mla_cache_append_at_fp8": (ctypes.c_int, [P, P, P, P, P, P, P, P, CacheDesc, I32, F32, P]),
        "mla_attn_weights": (ctypes.c_int, [P, P, P, P, CacheDesc, I32, F32, P, P, F32, P, P]),
        "mla_attn_weights_fp8": (ctypes.c_int, [P, P, P, P, P, CacheDesc, I32, F32, P, P, F32, P, P]),
        "mla_prefill_attn_weights_workspace_size": (SZ, [I32, I32, I32]),
        "mla_prefill_attn_weights": (ctypes.c_int, [P, P, P, P, P, P, CacheDesc, I32, I32, F32, P, P, F32, P, SZ, P,
                                                    P]),
        "mla_evict_workspace_size": (SZ, [I32, I32]),
        "mla_cache_evict": (ctypes.c_int, [P, P, P, P, CacheDesc, I32, I32, I32, I32, P, P, CacheDesc, P, P, P, P, SZ,
                                           P]),
        "mla_cache_evict_fp8": (ctypes.c_int, [P, P, P, P, P, CacheDesc, I32, I32, I32, I32, P, P, P, CacheDesc, P, P,
                                               P, P, SZ, P]),
        "mla_unabsorb_v": (ctypes.c_int, [P, P, P, I32, P]),
        "mla_decode_attn_noalloc": (ctypes.c_int, [P, P, P, P, CacheDesc, I32, F32, I32, P, P, P]),
        "mla_noalloc_scratch_bytes": (SZ, []),
        "mla_get_device_error": (ctypes.c_int, [ctypes.POINTER(I32)]),
    }
    for name, (res, args) in sigs.items():
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args
    return lib


lib = _load()


def _ptr(x):
    """Device pointer of a tensor (or an int address, or None -> NULL)."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(stream):
    if stream is None:
        import torch
        if torch.cuda.is_initialized():   # the handle alone: current_stream() makes an object, 2.5 us of a 9 us call
            return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(status: int, what: str):
    if status != 0:
        raise MlaError(status, what)


def status_string(s: int) -> str:
    return lib.mla_status_string(s).decode()


def cache_append(c_new, kr_new, pos, cache, desc: CacheDesc, *, seq_ids=None, block_table=None,
                 rope_base: float = 10000.0, stream=None, n_tokens: int | None = None):
    n = c_new.shape[0] if n_tokens is None else n_tokens
    _check(lib.mla_cache_append(_ptr(c_new), _ptr(kr_new), _ptr(seq_ids), _ptr(pos), _ptr(cache),
                                _ptr(block_table), desc, n, rope_base, _stream(stream)), "mla_cache_append")


def cache_append_fp8(c_new, kr_new, pos, cache, scales, desc: CacheDesc, *, seq_ids=None, block_table=None,
                     rope_base: float = 10000.0, stream=None, n_tokens: int | None = None):
    """mla_cache_append_fp8: rows as E4M3 codes (cache, uint8 [rows, 576]) with E8M0 row scales
    (scales, uint8 [rows])."""
    n = c_new.shape[0] if n_tokens is None else n_tokens
    _check(lib.mla_cache_append_fp8(_ptr(c_new), _ptr(kr_new), _ptr(seq_ids), _ptr(pos), _ptr(cache), _ptr(scales),
                                    _ptr(block_table), desc, n, rope_base, _stream(stream)), "mla_cache_append_fp8")


def cache_append_at(c_new, kr_new, pos, slots, cache, desc: CacheDesc, *, seq_ids=None, block_table=None,
                    rope_base: float = 10000.0, stream=None, n_tokens: int | None = None):
    """mla_cache_append_at: token i's row goes to slot slots[i], its key is rotated at pos[i] (a cache
    shortened by cache_evict)."""
    n = c_new.shape[0] if n_tokens is None else n_tokens
    _check(lib.mla_cache_append_at(_ptr(c_new), _ptr(kr_new), _ptr(seq_ids), _ptr(pos), _ptr(slots), _ptr(cache),
                                   _ptr(block_table), desc, n, rope_base, _stream(stream)), "mla_cache_append_at")


def cache_append_at_fp8(c_new, kr_new, pos, slots, cache, scales, desc: CacheDesc, *, seq_ids=None, block_table=None,
                        rope_base: float = 10000.0, stream=None, n_tokens: int | None = None):
    """mla_cache_append_at_fp8: cache_append_at into an FP8 cache."""
    n = c_new.shape[0] if n_tokens is None else n_tokens
    _check(lib.mla_cache_append_at_fp8(_ptr(c_new), _ptr(kr_new), _ptr(seq_ids), _ptr(pos), _ptr(slots), _ptr(cache),
                                       _ptr(scales), _ptr(block_table), desc, n, rope_base, _stream(stream)),
           "mla_cache_append_at_fp8")


def project_append(h, w_dkv, w_kr, pos, cache, desc: CacheDesc, *, seq_ids=None, block_table=None,
                   rope_base: float = 10000.0, stream=None, n_tokens: int | None = None):
    n = h.shape[0] if n_tokens is None else n_tokens
    _check(lib.mla_project_append(_ptr(h), _ptr(w_dkv), _ptr(w_kr), _ptr(seq_ids), _ptr(pos), _ptr(cache),
                                  _ptr(block_table), desc, n, rope_base, _stream(stream)), "mla_project_append")


def append_absorb(c_new, kr_new, pos, cache, desc: CacheDesc, q_nope, q_pe, w_uk, q_full, *, seq_ids=None,
                  block_table=None, q_pos=None, rope_base: float = 10000.0, stream=None):
    """mla_cache_append and mla_absorb_q in one launch."""
    _check(lib.mla_append_absorb(_ptr(c_new), _ptr(kr_new), _ptr(seq_ids), _ptr(pos), _ptr(cache), _ptr(block_table),
                                 desc, c_new.shape[0], _ptr(q_nope), _ptr(q_pe), _ptr(q_pos), _ptr(w_uk), _ptr(q_full),
                                 q_nope.shape[0], rope_base, _stream(stream)), "mla_append_absorb")


def selftest_wait_timeout(limit_us: int, result, *, stream=None):
    """Run the bounded-wait self-test; result is a device int32[2] tensor (see mla.h)."""
    _check(lib.mla_selftest_wait_timeout(limit_us, _ptr(result), _stream(stream)), "mla_selftest_wait_timeout")


def output_proj(out, w_o, y, *, stream=None, batch: int | None = None):
    b = out.shape[0] if batch is None else batch
    _check(lib.mla_output_proj(_ptr(out), _ptr(w_o), _ptr(y), b, _stream(stream)), "mla_output_proj")


def absorb_q(q_nope, q_pe, w_uk, q_full, *, q_pos=None, rope_base: float = 10000.0, stream=None,
             batch: int | None = None):
    b = q_nope.shape[0] if batch is None else batch
    _check(lib.mla_absorb_q(_ptr(q_nope), _ptr(q_pe), _ptr(q_pos), _ptr(w_uk), _ptr(q_full), b, rope_base,
                            _stream(stream)), "mla_absorb_q")


def decode_num_splits(batch: int, max_seq_len: int, num_splits: int = 0) -> int:
    return lib.mla_decode_num_splits(batch, max_seq_len, num_splits)


def decode_workspace_size(batch: int, max_seq_len: int, num_splits: int = 0) -> int:
    return lib.mla_decode_workspace_size(batch, max_seq_len, num_splits)


def decode_attn(q_full, cache, seq_lens, desc: CacheDesc, workspace, out_lat, *, lse=None, block_table=None,
                softmax_scale: float = 1.0 / 192 ** 0.5, num_splits: int = 0, stream=None,
                batch: int | None = None, workspace_bytes: int | None = None):
    b = q_full.shape[0] if batch is None else batch
    wb = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    _check(lib.mla_decode_attn(_ptr(q_full), _ptr(cache), _ptr(block_table), _ptr(seq_lens), desc, b,
                               softmax_scale, num_splits, _ptr(workspace), wb, _ptr(out_lat), _ptr(lse),
                               _stream(stream)), "mla_decode_attn")


def decode_attn_fp8(q_full, cache, scales, seq_lens, desc: CacheDesc, workspace, out_lat, *, lse=None,
                    block_table=None, softmax_scale: float = 1.0 / 192 ** 0.5, num_splits: int = 0, stream=None,
                    batch: int | None = None, workspace_bytes: int | None = None):
    """mla_decode_attn_fp8: decode over an FP8 cache (E4M3 codes + E8M0 row scales)."""
    b = q_full.shape[0] if batch is None else batch
    wb = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    _check(lib.mla_decode_attn_fp8(_ptr(q_full), _ptr(cache), _ptr(scales), _ptr(block_table), _ptr(seq_lens), desc,
                                   b, softmax_scale, num_splits, _ptr(workspace), wb, _ptr(out_lat), _ptr(lse),
                                   _stream(stream)), "mla_decode_attn_fp8")


def prefill_attn(q_full, cache, q_seq, q_len, desc: CacheDesc, workspace, out_lat, *, lse=None,
                 block_table=None, softmax_scale: float = 1.0 / 192 ** 0.5, num_splits: int = 0, stream=None,
                 n_queries: int | None = None, workspace_bytes: int | None = None):
    """mla_prefill_attn: query row i (a new token of sequence q_seq[i]) attends to the first
    q_len[i] cached tokens of that sequence."""
    n = q_full.shape[0] if n_queries is None else n_queries
    wb = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    _check(lib.mla_prefill_attn(_ptr(q_full), _ptr(cache), _ptr(block_table), _ptr(q_seq), _ptr(q_len), desc, n,
                                softmax_scale, num_splits, _ptr(workspace), wb, _ptr(out_lat), _ptr(lse),
                                _stream(stream)), "mla_prefill_attn")


def window_span(max_seq_len: int, window: int, sinks: int = 0) -> int:
    """Cached tokens a windowed row reads at most; sizes the workspace of the windowed calls
    (decode_workspace_size(rows, window_span(capacity, window, sinks), num_splits))."""
    return lib.mla_window_span(max_seq_len, window, sinks)


def decode_attn_window(q_full, cache, seq_lens, desc: CacheDesc, workspace, out_lat, *, window: int, sinks: int = 0,
                       lse=None, block_table=None, softmax_scale: float = 1.0 / 192 ** 0.5, num_splits: int = 0,
                       stream=None, batch: int | None = None, workspace_bytes: int | None = None):
    """mla_decode_attn_window: row b attends to the first `sinks` and the last `window` tokens of sequence b."""
    b = q_full.shape[0] if batch is None else batch
    wb = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    _check(lib.mla_decode_attn_window(_ptr(q_full), _ptr(cache), _ptr(block_table), _ptr(seq_lens), desc, b, window,
                                      sinks, softmax_scale, num_splits, _ptr(workspace), wb, _ptr(out_lat), _ptr(lse),
                                      _stream(stream)), "mla_decode_attn_window")


def decode_attn_window_fp8(q_full, cache, scales, seq_lens, desc: CacheDesc, workspace, out_lat, *, window: int,
                           sinks: int = 0, lse=None, block_table=None, softmax_scale: float = 1.0 / 192 ** 0.5,
                           num_splits: int = 0, stream=None, batch: int | None = None,
                           workspace_bytes: int | None = None):
    """mla_decode_attn_window_fp8: the windowed decode over an FP8 cache."""
    b = q_full.shape[0] if batch is None else batch
    wb = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    _check(lib.mla_decode_attn_window_fp8(_ptr(q_full), _ptr(cache), _ptr(scales), _ptr(block_table), _ptr(seq_lens),
                                          desc, b, window, sinks, softmax_scale, num_splits, _ptr(workspace), wb,
                                          _ptr(out_lat), _ptr(lse), _stream(stream)), "mla_decode_attn_window_fp8")


def prefill_attn_window(q_full, cache, q_seq, q_len, desc: CacheDesc, workspace, out_lat, *, window: int,
                        sinks: int = 0, lse=None, block_table=None, softmax_scale: float = 1.0 / 192 ** 0.5,
                        num_splits: int = 0, stream=None, n_queries: int | None = None,
                        workspace_bytes: int | None = None):
    """mla_prefill_attn_window: query row i attends to the first `sinks` and the last `window` of the
    first q_len[i] tokens of sequence q_seq[i]."""
    n = q_full.shape[0] if n_queries is None else n_queries
    wb = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    _check(lib.mla_prefill_attn_window(_ptr(q_full), _ptr(cache), _ptr(block_table), _ptr(q_seq), _ptr(q_len), desc, n,
                                       window, sinks, softmax_scale, num_splits, _ptr(workspace), wb, _ptr(out_lat),
                                       _ptr(lse), _stream(stream)), "mla_prefill_attn_window")


def attn_weights(q_full, cache, seq_lens, desc: CacheDesc, lse, weights, *, prev=None, decay: float = 1.0,
                 block_table=None, softmax_scale: float = 1.0 / 192 ** 0.5, stream=None, batch: int | None = None):
    """mla_attn_weights: weights[b, t] = decay * prev[b, t] + the attention weight of token t over the
    heads of query row b, whose log-sum-exps lse decode_attn wrote (prev None: 0; weights may be prev)."""
    b = q_full.shape[0] if batch is None else batch
    _check(lib.mla_attn_weights(_ptr(q_full), _ptr(cache), _ptr(block_table), _ptr(seq_lens), desc, b, softmax_scale,
                                _ptr(lse), _ptr(prev), decay, _ptr(weights), _stream(stream)), "mla_attn_weights")


def attn_weights_fp8(q_full, cache, scales, seq_lens, desc: CacheDesc, lse, weights, *, prev=None, decay: float = 1.0,
                     block_table=None, softmax_scale: float = 1.0 / 192 ** 0.5, stream=None,
                     batch: int | None = None):
    """mla_attn_weights_fp8: attn_weights over an FP8 cache."""
    b = q_full.shape[0] if batch is None else batch
    _check(lib.mla_attn_weights_fp8(_ptr(q_full), _ptr(cache), _ptr(scales), _ptr(block_table), _ptr(seq_lens), desc, b,
                                    softmax_scale, _ptr(lse), _ptr(prev), decay, _ptr(weights), _stream(stream)),
           "mla_attn_weights_fp8")


def prefill_attn_weights_workspace_size(batch: int, max_seq_len: int, n_queries: int) -> int:
    return lib.mla_prefill_attn_weights_workspace_size(batch, max_seq_len, n_queries)


def prefill_attn_weights(q_full, cache, seq_lens, q_start, q_len, desc: CacheDesc, lse, workspace, weights, *,
                         prev=None, decay: float = 1.0, block_table=None, softmax_scale: float = 1.0 / 192 ** 0.5,
                         stream=None, batch: int | None = None, n_queries: int | None = None,
                         workspace_bytes: int | None = None):
    """mla_prefill_attn_weights: attn_weights with the rows q_start[b] .. q_start[b + 1] - 1 of sequence b,
    row i counting for its first q_len[i] tokens."""
    b = seq_lens.shape[0] if batch is None else batch
    n = q_full.shape[0] if n_queries is None else n_queries
    wb = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    _check(lib.mla_prefill_attn_weights(_ptr(q_full), _ptr(cache), _ptr(block_table), _ptr(seq_lens), _ptr(q_start),
                                        _ptr(q_len), desc, b, n, softmax_scale, _ptr(lse), _ptr(prev), decay,
                                        _ptr(workspace), wb, _ptr(weights), _stream(stream)),
           "mla_prefill_attn_weights")


def evict_workspace_size(batch: int, keep: int) -> int:
    return lib.mla_evict_workspace_size(batch, keep)


def _in_place(desc, block_table, desc_out, block_table_out):
    """The output's descriptor and block table of an eviction within one buffer: the source's where none is
    given (its table only where the output's descriptor has rows of that width)."""
    if desc_out is None:
        desc_out = desc
    if block_table_out is None and desc_out.max_blocks_per_seq == desc.max_blocks_per_seq:
        block_table_out = block_table
    return desc_out, block_table_out


def cache_evict(cache, seq_lens, weights, desc: CacheDesc, kept, lens_out, weights_out, workspace, *, keep: int,
                sinks: int = 0, recent: int = 0, block_table=None, cache_out=None, desc_out: CacheDesc | None = None,
                block_table_out=None, stream=None, batch: int | None = None, workspace_bytes: int | None = None):
    """mla_cache_evict: each sequence longer than `keep` keeps its first `sinks`, its last `recent` and the
    heaviest tokens between, moved in order to the front of cache_out, or (cache_out None) of the same cache; there
    block_table_out, with desc_out unless it is as wide as block_table, may name fresh pages of the same pool."""
    b = seq_lens.shape[0] if batch is None else batch
    wb = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    if cache_out is None:
        cache_out, desc_out, block_table_out = cache, *_in_place(desc, block_table, desc_out, block_table_out)
    _check(lib.mla_cache_evict(_ptr(cache), _ptr(block_table), _ptr(seq_lens), _ptr(weights), desc, b, keep, sinks,
                               recent, _ptr(cache_out), _ptr(block_table_out), desc_out, _ptr(kept), _ptr(lens_out),
                               _ptr(weights_out), _ptr(workspace), wb, _stream(stream)), "mla_cache_evict")


def cache_evict_fp8(cache, scales, seq_lens, weights, desc: CacheDesc, kept, lens_out, weights_out, workspace, *,
                    keep: int, sinks: int = 0, recent: int = 0, block_table=None, cache_out=None, scales_out=None,
                    desc_out: CacheDesc | None = None, block_table_out=None, stream=None, batch: int | None = None,
                    workspace_bytes: int | None = None):
    """mla_cache_evict_fp8: cache_evict over an FP8 cache (codes and row scales)."""
    b = seq_lens.shape[0] if batch is None else batch
    wb = workspace.numel() * workspace.element_size() if workspace_bytes is None else workspace_bytes
    if cache_out is None:
        cache_out, scales_out = cache, scales if scales_out is None else scales_out
        desc_out, block_table_out = _in_place(desc, block_table, desc_out, block_table_out)
    _check(lib.mla_cache_evict_fp8(_ptr(cache), _ptr(scales), _ptr(block_table), _ptr(seq_lens), _ptr(weights), desc, b,
                                   keep, sinks, recent, _ptr(cache_out), _ptr(scales_out), _ptr(block_table_out),
                                   desc_out, _ptr(kept), _ptr(lens_out), _ptr(weights_out), _ptr(workspace), wb,
                                   _stream(stream)), "mla_cache_evict_fp8")


NOALLOC_SCRATCH_BYTES = int(lib.mla_noalloc_scratch_bytes())   # the library's own constant


def decode_attn_noalloc(q_full, cache, seq_lens, desc: CacheDesc, out_lat, *, lse=None, block_table=None,
                        softmax_scale: float = 1.0 / 192 ** 0.5, num_splits: int = 0, stream=None,
                        batch: int | None = None):
    """mla_decode_attn without a workspace: for callers that cannot allocate device memory at
    decode time; range partials go to the library's static 48 MiB device buffer."""
    b = q_full.shape[0] if batch is None else batch
    _check(lib.mla_decode_attn_noalloc(_ptr(q_full), _ptr(cache), _ptr(block_table), _ptr(seq_lens), desc, b,
                                       softmax_scale, num_splits, _ptr(out_lat), _ptr(lse), _stream(stream)),
           "mla_decode_attn_noalloc")


def unabsorb_v(out_lat, w_uv, out, *, stream=None, batch: int | None = None):
    b = out_lat.shape[0] if batch is None else batch
    _check(lib.mla_unabsorb_v(_ptr(out_lat), _ptr(w_uv), _ptr(out), b, _stream(stream)), "mla_unabsorb_v")


def get_device_error() -> int:
    code = ctypes.c_int32(0)
    _check(lib.mla_get_device_error(ctypes.byref(code)), "mla_get_device_error")
    return code.value
