"""Thin ctypes binding of libdsa (include/dsa.h).

Argument marshalling only: every step runs in the library's CUDA kernels.  The functions
keep the C names and take torch tensors (device memory) or raw integer pointers; streams
default to torch's current stream.  If the shared library is missing the first call raises
-- there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libdsa.so")

DSA_OK, DSA_ERR_INVALID_ARG, DSA_ERR_UNSUPPORTED, DSA_ERR_WORKSPACE, DSA_ERR_CUDA, DSA_ERR_DEVICE_CHECK, \
    DSA_ERR_TIMEOUT = range(7)
DSA_F32, DSA_BF16, DSA_FP8_E4M3 = 0, 1, 2
DSA_OP_INDEXER, DSA_OP_TOPK, DSA_OP_ATTN_PREFILL, DSA_OP_ATTN_DECODE, DSA_OP_CACHE_APPEND, DSA_OP_INDEXER_TOPK = \
    0, 1, 2, 3, 4, 5
DSA_OP_PAGED_DECODE, DSA_OP_BATCH_EXTEND, DSA_OP_BATCH_RELEASE, DSA_OP_QK_NORM_ROPE = 6, 7, 8, 9
DSA_ROPE_PAIRS, DSA_ROPE_HALVES = 0, 1

EXPORTS = ("dsa_workspace_size", "dsa_indexer_scores", "dsa_topk", "dsa_sparse_attn_prefill",
           "dsa_sparse_attn_decode", "dsa_read_device_status", "dsa_status_string", "dsa_last_error",
           "dsa_version", "dsa_launch_count", "dsa_topk_noalloc", "dsa_cache_append", "dsa_selftest_wait_timeout",
           "dsa_cp_candidates", "dsa_cp_rows", "dsa_cp_select_local", "dsa_cp_merge", "dsa_block_scores",
           "dsa_expand_blocks", "dsa_reuse_candidates", "dsa_indexer_scores_at", "dsa_gather_positions",
           "dsa_indexer_scores_append", "dsa_indexer_topk", "dsa_batch_workspace_size", "dsa_batch_extend",
           "dsa_batch_release", "dsa_qk_norm_rope", "dsa_paged_attn_decode")


class dsa_batch_t(ctypes.Structure):
    _fields_ = [
        ("num_seqs", ctypes.c_int32),
        ("page_size", ctypes.c_int32),
        ("num_blocks", ctypes.c_int32),
        ("max_blocks_per_seq", ctypes.c_int32),
        ("block_table", ctypes.c_void_p),
        ("seq_lens", ctypes.c_void_p),
        ("cu_q", ctypes.c_void_p),
        ("total_q", ctypes.c_int32),
        ("max_q_per_seq", ctypes.c_int32),
        ("max_seq_len", ctypes.c_int32),
    ]


class dsa_rope_part_t(ctypes.Structure):
    _fields_ = [
        ("x", ctypes.c_void_p),
        ("out", ctypes.c_void_p),
        ("weight", ctypes.c_void_p),
        ("out_scale", ctypes.c_void_p),
        ("slots", ctypes.c_void_p),
        ("x_row_stride", ctypes.c_int64),
        ("x_head_stride", ctypes.c_int64),
        ("out_row_stride", ctypes.c_int64),
        ("out_head_stride", ctypes.c_int64),
        ("out_rows", ctypes.c_int64),
        ("H", ctypes.c_int32),
        ("D", ctypes.c_int32),
        ("norm_off", ctypes.c_int32),
        ("norm_len", ctypes.c_int32),
        ("rope_off", ctypes.c_int32),
        ("rope_len", ctypes.c_int32),
        ("x_dt", ctypes.c_int),
        ("w_dt", ctypes.c_int),
        ("out_dt", ctypes.c_int),
        ("rope_style", ctypes.c_int),
        ("eps", ctypes.c_float),
    ]


class DSAError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        super().__init__(f"{where}: status {status} ({detail})")
        self.status = status


_lib = None


def load(path: str = LIB_PATH):
    """Load libdsa and declare its signatures (once)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(path):
        raise RuntimeError(f"libdsa.so not found at {path}; build it with "
                           f"`python -m sparse_attention_long_dsa_b200.build`")
    lib = ctypes.CDLL(path)
    P, I32, I64, SZ, F = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t, ctypes.c_float
    B = ctypes.POINTER(dsa_batch_t)
    sig = {
        "dsa_workspace_size": [I32, B, I32, I32, I32, ctypes.POINTER(SZ)],
        "dsa_indexer_scores": [P, I32, P, P, I32, P, I32, I32, B, P, I64, P, SZ, P],
        "dsa_topk": [P, I64, B, I32, P, P, SZ, P],
        "dsa_indexer_topk": [P, I32, P, P, I32, P, I32, I32, B, I32, P, I64, P, P, SZ, P],
        "dsa_topk_noalloc": [P, I64, B, I32, P, P],
        "dsa_sparse_attn_prefill": [P, I32, P, P, I32, I32, I32, F, P, I32, B, P, P, P, SZ, P],
        "dsa_sparse_attn_decode": [P, I32, P, P, I32, I32, I32, F, P, I32, B, P, P, P, SZ, P],
        "dsa_cache_append": [P, I32, P, I32, I32, I32, B, P, P, P, P, SZ, P],
        "dsa_selftest_wait_timeout": [ctypes.c_uint64, P, SZ, P],
        "dsa_block_scores": [P, I64, B, P, I64, P, P],
        "dsa_reuse_candidates": [P, I32, P, I32, B, P, P, SZ, P],
        "dsa_indexer_scores_append": [P, I32, P, I32, P, P, I32, P, P, I32, P, I32, I32, B, P, I64, P, SZ, P],
        "dsa_indexer_scores_at": [P, I32, P, P, I32, P, I32, I32, B, P, I32, P, P, SZ, P],
        "dsa_gather_positions": [P, I32, P, I32, I32, P, P],
        "dsa_expand_blocks": [P, I32, B, P, P],
        "dsa_cp_candidates": [P, I64, P, I32, I32, P, P, P, P],
        "dsa_cp_rows": [P, I32, I32, I32, P, I64, P],
        "dsa_cp_select_local": [P, P, I32, I32, I32, P, P, P, P],
        "dsa_cp_merge": [P, I32, P, I32, I32, I32, I32, P, P, P],
        "dsa_batch_workspace_size": [I32, I32, ctypes.POINTER(SZ)],
        "dsa_batch_extend": [P, P, I32, I32, I32, I32, I32, P, I32, P, P, P, P, P, P, P, P, SZ, P],
        "dsa_batch_release": [P, I32, I32, I32, I32, P, P, P, I32, P, P, SZ, P],
        "dsa_qk_norm_rope": [ctypes.POINTER(dsa_rope_part_t), I32, P, I32, P, P, SZ, P],
        "dsa_paged_attn_decode": [P, I32, P, P, I32, I32, I32, F, P, I32, B, P, P, P, SZ, P],
        "dsa_read_device_status": [P, P],
    }
    for name, args in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    for name in ("dsa_status_string",):
        getattr(lib, name).argtypes = [ctypes.c_int]
        getattr(lib, name).restype = ctypes.c_char_p
    lib.dsa_launch_count.argtypes = []
    lib.dsa_launch_count.restype = ctypes.c_uint64
    for name in ("dsa_last_error", "dsa_version"):
        getattr(lib, name).argtypes = []
        getattr(lib, name).restype = ctypes.c_char_p
    _lib = lib
    return lib


def _check(status: int, where: str):
    if status != DSA_OK:
        lib = load()
        raise DSAError(status, where, f"{lib.dsa_status_string(status).decode()}: {lib.dsa_last_error().decode()}")


def _ptr(t) -> Optional[int]:
    """Address of a tensor's data, or an integer address passed through.  A tensor must be a dense CUDA tensor:
    the kernels read and write its bytes in the layout include/dsa.h gives, so a host tensor would hand them a
    host address and a strided view would be read as if it were dense."""
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_cuda:
        raise DSAError(DSA_ERR_INVALID_ARG, "argument",
                       f"a {tuple(t.shape)} tensor on {t.device}; the library takes device memory")
    if not t.is_contiguous():
        raise DSAError(DSA_ERR_INVALID_ARG, "argument",
                       f"a strided {tuple(t.shape)} tensor (strides {tuple(t.stride())}); the library takes dense arrays")
    return t.data_ptr()


def _stream(stream, device: Optional[int] = None) -> Optional[int]:
    """A stream's handle; None: the current stream of the current device (device, where the caller knows it)."""
    if stream is None:
        import torch
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device() if device is None else device)
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def make_batch(block_table, seq_lens, cu_q, *, num_blocks: int, page_size: int, total_q: int,
               max_q_per_seq: int, max_seq_len: int) -> dsa_batch_t:
    """dsa_batch_t from device int32 tensors (block_table [B, max_blocks], seq_lens [B], cu_q [B+1])."""
    return dsa_batch_t(num_seqs=int(seq_lens.shape[0]), page_size=page_size, num_blocks=num_blocks,
                       max_blocks_per_seq=int(block_table.shape[1]), block_table=_ptr(block_table),
                       seq_lens=_ptr(seq_lens), cu_q=_ptr(cu_q), total_q=total_q, max_q_per_seq=max_q_per_seq,
                       max_seq_len=max_seq_len)


def dsa_workspace_size(op: int, batch: dsa_batch_t, k: int = 0, H: int = 0, Dv: int = 0) -> int:
    out = ctypes.c_size_t(0)
    _check(load().dsa_workspace_size(op, ctypes.byref(batch), k, H, Dv, ctypes.byref(out)), "dsa_workspace_size")
    return out.value


def dsa_indexer_scores(q_idx, q_dt: int, w, k_idx_pool, k_dt: int, k_scale_pool, Hi: int, Di: int,
                       batch: dsa_batch_t, scores, ld_scores: int, ws, ws_bytes: int, stream=None):
    _check(load().dsa_indexer_scores(_ptr(q_idx), q_dt, _ptr(w), _ptr(k_idx_pool), k_dt, _ptr(k_scale_pool), Hi, Di,
                                     ctypes.byref(batch), _ptr(scores), ld_scores, _ptr(ws), ws_bytes,
                                     _stream(stream)), "dsa_indexer_scores")


def dsa_topk(scores, ld_scores: int, batch: dsa_batch_t, k: int, idx, ws, ws_bytes: int, stream=None):
    _check(load().dsa_topk(_ptr(scores), ld_scores, ctypes.byref(batch), k, _ptr(idx), _ptr(ws), ws_bytes,
                           _stream(stream)), "dsa_topk")


def dsa_indexer_topk(q_idx, q_dt: int, w, k_idx_pool, k_dt: int, k_scale_pool, Hi: int, Di: int,
                     batch: dsa_batch_t, k: int, scores, ld_scores: int, idx, ws, ws_bytes: int, stream=None):
    """Indexer scores and the top-k selection in one call (the selection fused into the scoring)."""
    _check(load().dsa_indexer_topk(_ptr(q_idx), q_dt, _ptr(w), _ptr(k_idx_pool), k_dt, _ptr(k_scale_pool), Hi, Di,
                                   ctypes.byref(batch), k, _ptr(scores), ld_scores, _ptr(idx), _ptr(ws), ws_bytes,
                                   _stream(stream)), "dsa_indexer_topk")


def dsa_topk_noalloc(scores, ld_scores: int, batch: dsa_batch_t, k: int, idx, stream=None):
    """Top-k with the library's built-in scratch instead of a caller workspace (no device allocation)."""
    _check(load().dsa_topk_noalloc(_ptr(scores), ld_scores, ctypes.byref(batch), k, _ptr(idx), _stream(stream)),
           "dsa_topk_noalloc")


def dsa_sparse_attn_prefill(q, dt: int, kv_pool, v_pool, H: int, Dqk: int, Dv: int, softmax_scale: float, idx,
                            k: int, batch: dsa_batch_t, out, lse, ws, ws_bytes: int, stream=None):
    _check(load().dsa_sparse_attn_prefill(_ptr(q), dt, _ptr(kv_pool), _ptr(v_pool), H, Dqk, Dv, softmax_scale,
                                          _ptr(idx), k, ctypes.byref(batch), _ptr(out), _ptr(lse), _ptr(ws),
                                          ws_bytes, _stream(stream)), "dsa_sparse_attn_prefill")


def dsa_sparse_attn_decode(q, dt: int, kv_pool, v_pool, H: int, Dqk: int, Dv: int, softmax_scale: float, idx,
                           k: int, batch: dsa_batch_t, out, lse, ws, ws_bytes: int, stream=None):
    _check(load().dsa_sparse_attn_decode(_ptr(q), dt, _ptr(kv_pool), _ptr(v_pool), H, Dqk, Dv, softmax_scale,
                                         _ptr(idx), k, ctypes.byref(batch), _ptr(out), _ptr(lse), _ptr(ws),
                                         ws_bytes, _stream(stream)), "dsa_sparse_attn_decode")


def dsa_cache_append(kv_new, kv_dt: int, k_new, k_dt: int, Dqk: int, Di: int, batch: dsa_batch_t, kv_pool, k_idx_pool,
                     k_scale_pool, ws, ws_bytes: int, stream=None):
    _check(load().dsa_cache_append(_ptr(kv_new), kv_dt, _ptr(k_new), k_dt, Dqk, Di, ctypes.byref(batch), _ptr(kv_pool),
                                   _ptr(k_idx_pool), _ptr(k_scale_pool), _ptr(ws), ws_bytes, _stream(stream)),
           "dsa_cache_append")


def dsa_selftest_wait_timeout(budget_cycles: int, ws, ws_bytes: int, stream=None):
    _check(load().dsa_selftest_wait_timeout(budget_cycles, _ptr(ws), ws_bytes, _stream(stream)),
           "dsa_selftest_wait_timeout")


def dsa_indexer_scores_append(kv_new, kv_dt: int, k_new, k_new_dt: int, kv_pool, q_idx, q_dt: int, w, k_idx_pool,
                              k_dt: int, k_scale_pool, Hi: int, Di: int, batch: dsa_batch_t, scores, ld_scores: int,
                              ws, ws_bytes: int, stream=None):
    _check(load().dsa_indexer_scores_append(_ptr(kv_new), kv_dt, _ptr(k_new), k_new_dt, _ptr(kv_pool), _ptr(q_idx),
                                            q_dt, _ptr(w), _ptr(k_idx_pool), k_dt, _ptr(k_scale_pool), Hi, Di,
                                            ctypes.byref(batch), _ptr(scores), ld_scores, _ptr(ws), ws_bytes,
                                            _stream(stream)), "dsa_indexer_scores_append")


def dsa_reuse_candidates(prev_idx, k: int, prev_lens, max_new: int, batch: dsa_batch_t, cand, ws, ws_bytes: int,
                         stream=None):
    _check(load().dsa_reuse_candidates(_ptr(prev_idx), k, _ptr(prev_lens), max_new, ctypes.byref(batch), _ptr(cand),
                                       _ptr(ws), ws_bytes, _stream(stream)), "dsa_reuse_candidates")


def dsa_indexer_scores_at(q_idx, q_dt: int, w, k_idx_pool, k_dt: int, k_scale_pool, Hi: int, Di: int,
                          batch: dsa_batch_t, cand, m: int, cand_scores, ws, ws_bytes: int, stream=None):
    _check(load().dsa_indexer_scores_at(_ptr(q_idx), q_dt, _ptr(w), _ptr(k_idx_pool), k_dt, _ptr(k_scale_pool), Hi, Di,
                                        ctypes.byref(batch), _ptr(cand), m, _ptr(cand_scores), _ptr(ws), ws_bytes,
                                        _stream(stream)), "dsa_indexer_scores_at")


def dsa_gather_positions(sel, k: int, cand, m: int, T: int, idx, stream=None):
    _check(load().dsa_gather_positions(_ptr(sel), k, _ptr(cand), m, T, _ptr(idx), _stream(stream)),
           "dsa_gather_positions")


def dsa_block_scores(scores, ld_scores: int, batch: dsa_batch_t, blk_scores, ld_blk: int, blk_lens, stream=None):
    _check(load().dsa_block_scores(_ptr(scores), ld_scores, ctypes.byref(batch), _ptr(blk_scores), ld_blk,
                                   _ptr(blk_lens), _stream(stream)), "dsa_block_scores")


def dsa_expand_blocks(blk_idx, kb: int, batch: dsa_batch_t, idx, stream=None):
    _check(load().dsa_expand_blocks(_ptr(blk_idx), kb, ctypes.byref(batch), _ptr(idx), _stream(stream)),
           "dsa_expand_blocks")


def dsa_cp_candidates(scores, ld_scores: int, idx, T: int, k: int, offsets, cand_score, cand_gidx, stream=None):
    _check(load().dsa_cp_candidates(_ptr(scores), ld_scores, _ptr(idx), T, k, _ptr(offsets), _ptr(cand_score),
                                    _ptr(cand_gidx), _stream(stream)), "dsa_cp_candidates")


def dsa_cp_rows(g_score, G: int, T: int, k: int, rows, ld_rows: int, stream=None):
    _check(load().dsa_cp_rows(_ptr(g_score), G, T, k, _ptr(rows), ld_rows, _stream(stream)), "dsa_cp_rows")


def dsa_cp_select_local(sel, g_gidx, G: int, T: int, k: int, lo, hi, local_idx, stream=None):
    _check(load().dsa_cp_select_local(_ptr(sel), _ptr(g_gidx), G, T, k, _ptr(lo), _ptr(hi), _ptr(local_idx),
                                      _stream(stream)), "dsa_cp_select_local")


def dsa_cp_merge(part_out, dt: int, part_lse, G: int, T: int, H: int, Dv: int, out, lse, stream=None):
    _check(load().dsa_cp_merge(_ptr(part_out), dt, _ptr(part_lse), G, T, H, Dv, _ptr(out), _ptr(lse),
                               _stream(stream)), "dsa_cp_merge")


def _dense(what: str, dtype, *tensors):
    """Addresses of dense tensors of one dtype on the current device."""
    import torch
    dev = tensors[0].get_device()
    cur = torch._C._cuda_getDevice() if dev >= 0 else -2
    at = [t.data_ptr() for t in tensors if t.dtype is dtype and t.get_device() == cur and t.is_contiguous()]
    if len(at) == len(tensors):
        return at
    for t in tensors:
        if t.dtype is not dtype:
            raise DSAError(DSA_ERR_INVALID_ARG, what, f"a {t.dtype} tensor; expected {dtype}")
        _ptr(t)                                      # names a host or strided tensor
    raise DSAError(DSA_ERR_INVALID_ARG, what, f"a tensor on another device than the current one, cuda:{torch.cuda.current_device()}")


def _here(what: str, *tensors):
    """_ptr of tensors that have to be on the current device: its kernels could not reach them anywhere else."""
    at, cur = [], None
    for t in tensors:
        if t is not None and not isinstance(t, int):
            on = t.get_device()
            if on < 0 or not t.is_contiguous():
                _ptr(t)                              # names a host or strided tensor
            if cur is None:
                import torch
                cur = torch._C._cuda_getDevice()
            if on != cur:
                raise DSAError(DSA_ERR_INVALID_ARG, what, f"a tensor on cuda:{on}; the current device is cuda:{cur}")
            t = t.data_ptr()
        at.append(t)
    return at


def _shape(t, shape: tuple, what: str):
    if t.shape != shape:
        raise DSAError(DSA_ERR_INVALID_ARG, what, f"shape {tuple(t.shape)}; expected {shape}")


def dsa_batch_workspace_size(op: int, num_seqs: int) -> int:
    out = ctypes.c_size_t(0)
    _check(load().dsa_batch_workspace_size(op, num_seqs, ctypes.byref(out)), "dsa_batch_workspace_size")
    return out.value


def dsa_batch_extend(cached_lens, new_lens, page_size: int, num_blocks: int, total_q: int, free_blocks, free_count,
                     block_table, seq_lens, cu_q, slots, positions, free_left, ws, ws_bytes: int, stream=None):
    """Block tables, slots and positions of a step, from device lengths (cached_lens, new_lens [B]): block_table [B,
    max_blocks] and the stack free_blocks / free_count lose and gain pages on the device.  seq_lens may be cached_lens
    and free_left may be free_count.  cu_q None: a decode step of one row per sequence (total_q = B, new_lens of 0 or 1)."""
    import torch
    w = "dsa_batch_extend"
    n, table_shape = cached_lens.numel(), block_table.shape
    if new_lens.shape != (n,) or seq_lens.shape != (n,) or (cu_q is not None and cu_q.shape != (n + 1,)):
        raise DSAError(DSA_ERR_INVALID_ARG, w, f"new_lens {tuple(new_lens.shape)}, seq_lens {tuple(seq_lens.shape)}, cu_q "
                       f"{None if cu_q is None else tuple(cu_q.shape)}; expected ({n},), ({n},), ({n + 1},)")
    if len(table_shape) != 2 or table_shape[0] != n or slots.numel() < total_q or positions.numel() < total_q:
        raise DSAError(DSA_ERR_INVALID_ARG, w, f"block_table [{n}, max_blocks], slots and positions [total_q] expected")
    cached, new, free, count, table, seq, pos, left, *cu = _dense(w, torch.int32, cached_lens, new_lens, free_blocks, free_count,
                                                                  block_table, seq_lens, positions, free_left,
                                                                  *(() if cu_q is None else (cu_q,)))
    slot, = _dense(w, torch.int64, slots)
    _check((_lib or load()).dsa_batch_extend(cached, new, n, page_size, table_shape[1], num_blocks, total_q, free,
                                             free_blocks.numel(), count, table, seq, cu[0] if cu else None, slot, pos, left,
                                             *_here(w, ws), ws_bytes,
                                             _stream(stream, cached_lens.get_device())), w)


def dsa_batch_release(done, page_size: int, num_blocks: int, block_table, seq_lens, free_blocks, free_count, ws,
                      ws_bytes: int, stream=None):
    """Gives the blocks of the sequences with done[b] != 0 back to the stack; their seq_lens become 0."""
    import torch
    w = "dsa_batch_release"
    n = done.numel()
    _shape(seq_lens, (n,), w)
    if block_table.dim() != 2 or block_table.shape[0] != n:
        raise DSAError(DSA_ERR_INVALID_ARG, w, f"block_table [{n}, max_blocks] expected")
    d, table, seq, free, count = _dense(w, torch.int32, done, block_table, seq_lens, free_blocks, free_count)
    _check((_lib or load()).dsa_batch_release(d, n, page_size, block_table.shape[1], num_blocks, table, seq, free,
                                              free_blocks.numel(), count, *_here(w, ws), ws_bytes, _stream(stream)), w)


_PARTS = tuple(dsa_rope_part_t * n for n in range(5))


def rope_part(x, out, *, weight=None, norm=(0, 0), eps: float = 1e-6, rope=(0, 0), style: str = "pairs", slots=None,
              scale=None) -> dsa_rope_part_t:
    """One tensor of dsa_qk_norm_rope: x [T, H, D] or [T, D] (f32 or bf16, any strides with a dense last dimension; so a
    view of a fused projection), out [N, H, D] or [N, D] (f32, bf16, e4m3 or uint8 for e4m3 codes; a view too).  norm and
    rope are (offset, length) in entries of a row, style "pairs" or "halves", slots [T] int64 out rows, scale [N, H] or
    [N] f32.  The part holds the tensors' addresses and keeps the tensors alive."""
    w = "rope_part"
    floats, codes = {"float32": DSA_F32, "bfloat16": DSA_BF16}, {"uint8": DSA_FP8_E4M3, "float8_e4m3fn": DSA_FP8_E4M3}

    def fail(msg):
        raise DSAError(DSA_ERR_INVALID_ARG, w, msg)

    def view(t, name, kinds):
        if not t.is_cuda:
            fail(f"{name} on {t.device}; the library takes device memory")
        if t.device != x.device:
            fail(f"{name} on {t.device}, x on {x.device}")
        kind = kinds.get(str(t.dtype)[6:])
        if kind is None:
            fail(f"{name} is {t.dtype}; expected {' or '.join(kinds)}")
        if t.dim() not in (2, 3) or (t.shape[-1] > 1 and t.stride(-1) != 1):
            fail(f"{name} must be [rows, heads, D] or [rows, D] with a dense last dimension")
        if t.dim() == 2:
            return kind, t.shape[0], 1, t.shape[1], t.stride(0), t.shape[1]
        return kind, t.shape[0], t.shape[1], t.shape[2], t.stride(0), t.stride(1)

    x_dt, T, H, D, x_row, x_head = view(x, "x", floats)
    o_dt, rows, o_h, o_d, o_row, o_head = view(out, "out", {**floats, **codes})
    if (o_h, o_d) != (H, D):
        fail(f"out rows are [{o_h}, {o_d}], x rows [{H}, {D}]")
    if rows == 1:
        o_row = max(o_row, D)
    if style not in ("pairs", "halves"):
        fail(f"style {style!r}; expected 'pairs' or 'halves'")
    if slots is not None and (str(slots.dtype) != "torch.int64" or tuple(slots.shape) != (T,)):
        fail("slots must be [T] int64")
    if scale is not None and (str(scale.dtype) != "torch.float32" or scale.numel() != rows * H):
        fail("scale must be [rows, H] float32")
    for name, t in (("weight", weight), ("slots", slots), ("scale", scale)):
        if t is not None and t.device != x.device:
            fail(f"{name} on {t.device}, x on {x.device}")
    if norm[1] and (weight is None or weight.numel() != norm[1] or str(weight.dtype)[6:] not in floats):
        fail("a norm needs a weight of its length, f32 or bf16")
    part = dsa_rope_part_t(x=x.data_ptr(), out=out.data_ptr(), weight=_ptr(weight), out_scale=_ptr(scale),
                           slots=_ptr(slots), x_row_stride=x_row, x_head_stride=x_head, out_row_stride=o_row,
                           out_head_stride=o_head, out_rows=rows, H=H, D=D, norm_off=norm[0], norm_len=norm[1],
                           rope_off=rope[0], rope_len=rope[1], x_dt=x_dt,
                           w_dt=floats[str(weight.dtype)[6:]] if weight is not None else DSA_F32, out_dt=o_dt,
                           rope_style=DSA_ROPE_HALVES if style == "halves" else DSA_ROPE_PAIRS, eps=eps)
    part.rows = T
    part.device = x.get_device()
    part.rotated = rope[1]
    part.tensors = (x, out, weight, scale, slots)
    return part


def dsa_qk_norm_rope(parts, positions, inv_freq, ws, ws_bytes: int, stream=None):
    """RMS norm and position rotation of up to four tensors (rope_part) in one launch: positions [T] int32, inv_freq
    [rope_len / 2] float64."""
    import torch
    w = "dsa_qk_norm_rope"
    if not 1 <= len(parts) <= 4:
        raise DSAError(DSA_ERR_UNSUPPORTED, w, f"{len(parts)} parts; 1 to 4 are taken")
    T, cur = parts[0].rows, torch._C._cuda_getDevice()       # the parts hold CUDA tensors: CUDA is up
    half = None if inv_freq is None else inv_freq.numel()
    for p in parts:
        if p.rows != T:
            raise DSAError(DSA_ERR_INVALID_ARG, w, f"parts of {T} and {p.rows} rows")
        if p.device != cur:
            raise DSAError(DSA_ERR_INVALID_ARG, w, f"a part on cuda:{p.device}; the current device is cuda:{cur}")
        if half is not None and p.rotated and half != p.rotated // 2:
            raise DSAError(DSA_ERR_INVALID_ARG, w, f"{half} frequencies for rope_len {p.rotated}")
    if positions is not None:
        _shape(positions, (T,), w)
    pos = None if positions is None else _dense(w, torch.int32, positions)[0]
    freq = None if inv_freq is None else _dense(w, torch.float64, inv_freq)[0]
    arr = _PARTS[len(parts)](*parts)
    _check((_lib or load()).dsa_qk_norm_rope(arr, len(parts), pos, T, freq, *_here(w, ws), ws_bytes,
                                             _stream(stream, cur)), w)


def page_list_width(pages, rows: int) -> int:
    """kb of a page list [rows, kb] int32 on the current device; 0 for None (every page).  kb = 0 is refused: an empty tensor
    has no address, so the library would take it for None."""
    import torch
    if pages is None:
        return 0
    w = "dsa_paged_attn_decode"
    if pages.dim() != 2 or pages.shape[1] == 0:
        raise DSAError(DSA_ERR_INVALID_ARG, w, f"pages {tuple(pages.shape)}; expected [{rows}, kb], kb >= 1")
    _shape(pages, (rows, pages.shape[1]), w)
    _dense(w, torch.int32, pages)
    return pages.shape[1]


def dsa_paged_attn_decode(q, dt: int, kv_pool, v_pool, H: int, Dqk: int, Dv: int, softmax_scale: float, pages, kb: int,
                          batch: dsa_batch_t, out, lse, ws, ws_bytes: int, stream=None):
    """Attention of one new token per sequence over every cached page, or over its list of pages [B, kb]."""
    w = "dsa_paged_attn_decode"
    if pages is not None and not isinstance(pages, int) and page_list_width(pages, batch.total_q) != kb:
        raise DSAError(DSA_ERR_INVALID_ARG, w, f"pages {tuple(pages.shape)} with kb {kb}")
    q, kv_pool, v_pool, pages, out, lse, ws = _here(w, q, kv_pool, v_pool, pages, out, lse, ws)
    _check(load().dsa_paged_attn_decode(q, dt, kv_pool, v_pool, H, Dqk, Dv, softmax_scale, pages, kb, ctypes.byref(batch), out, lse,
                                        ws, ws_bytes, _stream(stream)), w)


def dsa_read_device_status(ws, stream=None):
    _check(load().dsa_read_device_status(_ptr(ws), _stream(stream)), "dsa_read_device_status")


def dsa_version() -> str:
    return load().dsa_version().decode()


def dsa_launch_count() -> int:
    return int(load().dsa_launch_count())
