"""A paged latent cache whose bookkeeping stays on the device: lengths, block tables and the stack of free blocks.

`PagedCache` holds the three pools of the MLA path (latent rows, FP8 indexer keys, key scales) with the state that
places tokens in them, and enqueues a serving step on one stream:

    cache.extend(new_lens)                     a decode step, one row per sequence slot: tables, slots, positions
    cache.extend(new_lens, total_q)            any step, rows packed by cu_q (dsa_batch_extend)
    cache.store(kv, k_idx, ...)                norms and rotation of the step's rows, written to their slots, and of
                                               its queries (dsa_qk_norm_rope)
    cache.attend(q, out, ...)                  one-token attention over every cached page or a list of pages
                                               (dsa_paged_attn_decode); or the sparse path on `cache.batch(...)`
    cache.release(done)                        finished sequences give their blocks back (dsa_batch_release)

In a decode step row b of every tensor is slot b, paused and empty slots included, which is what `attend` and the decode calls
take.  In a packed step rows follow one another by cu_q, so a slot without a new token shifts the rows behind it: its tensors
go with `batch`, and `attend` then wants a q of its own, one row per slot.

Nothing here computes any part of the method, and no call reads the device: a step that does not fit is refused on the
device and shows in `check_status`.  Every call may be captured into a graph after its first run outside one.
"""
from __future__ import annotations

import torch

from . import binding as B

PAGE = 64
LATENT, VALUE, ROPE = 576, 512, 64
IDX_H, IDX_D = 64, 128


class PagedCache:
    """num_seqs sequence slots of at most max_blocks pages each, over num_blocks blocks of 64 tokens.

    kv_pool [num_blocks, 64, 576] bf16, ki_pool [num_blocks, 64, 128] uint8 (e4m3), ks_pool [num_blocks, 64] f32;
    block_table [num_seqs, max_blocks], seq_lens [num_seqs], free_blocks / free_count: device int32.  heads: query heads
    of attend(), 1 to 128."""

    def __init__(self, num_seqs: int, num_blocks: int, max_blocks: int, heads: int = 128, device="cuda"):
        dv = self.device = torch.device(device)
        self.num_seqs, self.num_blocks, self.max_blocks, self.heads = num_seqs, num_blocks, max_blocks, heads
        self.kv_pool = torch.zeros((num_blocks, PAGE, LATENT), dtype=torch.bfloat16, device=dv)
        self.ki_pool = torch.zeros((num_blocks, PAGE, IDX_D), dtype=torch.uint8, device=dv)
        self.ks_pool = torch.ones((num_blocks, PAGE), dtype=torch.float32, device=dv)
        self.block_table = torch.zeros((num_seqs, max_blocks), dtype=torch.int32, device=dv)
        self.seq_lens = torch.zeros(num_seqs, dtype=torch.int32, device=dv)
        self.cu_q = torch.zeros(num_seqs + 1, dtype=torch.int32, device=dv)
        self.free_blocks = torch.arange(num_blocks - 1, -1, -1, dtype=torch.int32, device=dv)   # block 0 on top
        self.free_count = torch.full((1,), num_blocks, dtype=torch.int32, device=dv)
        self._rows = {}                              # rows -> (slots, positions): kept, so that captured steps stay valid
        self.slots = self.positions = None
        self.packed = True                           # how the last step's rows are laid out
        self._one_each = torch.arange(num_seqs + 1, dtype=torch.int32, device=dv)
        size = max(B.dsa_batch_workspace_size(B.DSA_OP_BATCH_EXTEND, num_seqs),
                   B.dsa_workspace_size(B.DSA_OP_PAGED_DECODE, self.decode_batch(), 0, heads, VALUE))
        self.ws = torch.zeros(size, dtype=torch.uint8, device=dv)

    def extend(self, new_lens, total_q=None, stream=None):
        """A step of new_lens [num_seqs] tokens (device int32): grows the tables and lengths and fills slots and positions.
        total_q None: a decode step, new_lens of 0 or 1, one row per slot (slot and position -1 where it is 0); cu_q stays as
        it was.  Otherwise rows are packed, total_q of them or fewer, and cu_q is filled; rows behind the last one have slot
        and position -1.  Steps of similar sizes write the same buffers."""
        rows = self.num_seqs if total_q is None else total_q
        cap = 1 << max(0, rows - 1).bit_length()
        if cap not in self._rows:
            self._rows[cap] = (torch.empty(cap, dtype=torch.int64, device=self.device),
                               torch.empty(cap, dtype=torch.int32, device=self.device))
        slots, positions = self._rows[cap]
        self.slots, self.positions, self.packed = slots[:rows], positions[:rows], total_q is not None
        B.dsa_batch_extend(self.seq_lens, new_lens, PAGE, self.num_blocks, rows, self.free_blocks, self.free_count,
                           self.block_table, self.seq_lens, self.cu_q if self.packed else None, self.slots, self.positions,
                           self.free_count, self.ws, self.ws.numel(), stream)

    def release(self, done, stream=None):
        """Sequences with done[b] != 0 give their blocks back and become empty."""
        B.dsa_batch_release(done, PAGE, self.num_blocks, self.block_table, self.seq_lens, self.free_blocks, self.free_count,
                            self.ws, self.ws.numel(), stream)

    def store(self, kv, kv_weight, inv_freq, k_idx=None, k_idx_weight=None, q_rot=None, q=None, q_idx=None, q_idx_out=None,
              eps: float = 1e-6, stream=None, packed: bool = False):
        """The step's rows, total_q of them (a decode step: num_seqs): kv [total_q, 576] (512 normed by kv_weight, 64 rotated in
        pairs) and k_idx [total_q, 128] (normed by k_idx_weight, its first 64 rotated in halves, e4m3 with a scale) go to their
        slots; q_rot [total_q, heads, 64] is rotated into q[:, :, 512:] and q_idx [total_q, 64, 128] (first 64 rotated in halves)
        into q_idx_out as e4m3 codes of the values themselves (no scale: +-448 at most), row by row; rows without a position stay as
        they were.  Up to three of them may be left out.  A packed step of num_seqs rows makes
        a q that attend would take with its rows shifted behind a slot without a new token: it is refused unless packed says
        that the packed rows are meant."""
        for name, x, dest, what in (("q_rot", q_rot, q, "q"), ("q_idx", q_idx, q_idx_out, "q_idx_out")):
            if x is not None and dest is None:
                raise B.DSAError(B.DSA_ERR_INVALID_ARG, "store", f"{name} goes with {what}")
        if self.slots is None:
            raise B.DSAError(B.DSA_ERR_INVALID_ARG, "store", "no step: extend first")
        if q_rot is not None and self.packed and not packed and self.num_seqs > 1 and q_rot.shape[0] == self.num_seqs:
            raise B.DSAError(B.DSA_ERR_INVALID_ARG, "store", "queries of a packed step of num_seqs rows: extend without total_q lays "
                             "a decode step out one row per slot, as attend takes it; packed=True keeps the packed rows")
        parts = [B.rope_part(kv, self.kv_pool.view(-1, LATENT), weight=kv_weight, norm=(0, VALUE), eps=eps, rope=(VALUE, ROPE),
                             slots=self.slots)]
        if k_idx is not None:
            parts.append(B.rope_part(k_idx, self.ki_pool.view(-1, IDX_D), weight=k_idx_weight, norm=(0, IDX_D), eps=eps,
                                     rope=(0, ROPE), style="halves", slots=self.slots, scale=self.ks_pool.view(-1)))
        if q_rot is not None:
            parts.append(B.rope_part(q_rot, q[:, :, VALUE:], rope=(0, ROPE)))
        if q_idx is not None:
            parts.append(B.rope_part(q_idx, q_idx_out, rope=(0, ROPE), style="halves"))
        B.dsa_qk_norm_rope(parts, self.positions, inv_freq, self.ws, self.ws.numel(), stream)

    def batch(self, total_q: int, max_q_per_seq: int, max_seq_len: int):
        """The last step's batch descriptor for the other calls: total_q as in extend (num_seqs for a decode step), upper bounds of
        rows per sequence and of lengths.  A packed step's is never a decode batch (its rows need not be the slots'), so the
        sparse attention on it is dsa_sparse_attn_prefill."""
        if not self.packed:
            if total_q != self.num_seqs:
                raise B.DSAError(B.DSA_ERR_INVALID_ARG, "batch", f"total_q {total_q}; a decode step has {self.num_seqs} rows")
            return self._batch(self._one_each, total_q, 1, max_seq_len)
        most = max(2, max_q_per_seq, -(-total_q // self.num_seqs))
        return self._batch(self.cu_q, total_q, most, max(max_seq_len, most))

    def _batch(self, cu_q, total_q, max_q_per_seq, max_seq_len):
        return B.make_batch(self.block_table, self.seq_lens, cu_q, num_blocks=self.num_blocks, page_size=PAGE, total_q=total_q,
                            max_q_per_seq=max_q_per_seq, max_seq_len=max_seq_len)

    def decode_batch(self):
        """One row per sequence slot, empty ones included."""
        return self._batch(self._one_each, self.num_seqs, 1, self.max_blocks * PAGE)

    def attend(self, q, out, softmax_scale: float, pages=None, lse=None, stream=None):
        """q [num_seqs, heads, 576], row b of slot b, over every cached token of its sequence, or over the tokens of the pages in
        pages [num_seqs, kb] (int32, -1: none); out [num_seqs, heads, 512].  Empty slots give zeros."""
        B._shape(q, (self.num_seqs, self.heads, LATENT), "attend")
        B._shape(out, (self.num_seqs, self.heads, VALUE), "attend")
        B._dense("attend", torch.bfloat16, q, out)
        if lse is not None:
            B._shape(lse, (self.num_seqs, self.heads), "attend")
            B._dense("attend", torch.float32, lse)
        kb = B.page_list_width(pages, self.num_seqs)
        B.dsa_paged_attn_decode(q, B.DSA_BF16, self.kv_pool, None, self.heads, LATENT, VALUE, softmax_scale, pages, kb,
                                self.decode_batch(), out, lse, self.ws, self.ws.numel(), stream)

    def check_status(self, stream=None):
        B.dsa_read_device_status(self.ws, stream)
