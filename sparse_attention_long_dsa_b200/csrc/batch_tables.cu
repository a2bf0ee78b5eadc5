// Block tables and slot maps from the requests' lengths, on the device.
//
// A step appends new_lens[b] tokens to sequence b, which holds cached_lens[b].  With held_b = ceil(cached_b / 64) pages
// owned and need_b = ceil((cached_b + new_b) / 64) - held_b to add, the j-th page of the step (sequences in order, then
// pages) is the j-th from the top of the stack of free blocks:
//   block_table[b, held_b + i] = free_blocks[free_count - 1 - (sum_{a<b} need_a + i)],   0 <= i < need_b
//   seq_lens[b] = cached_b + new_b,   cu_q[b] = sum_{a<b} new_a
//   slots[r] = 64 block_table[b, pos / 64] + pos % 64,   pos = positions[r] = cached_b + r - cu_q[b]
// or, without cu_q, for new_b of 0 or 1, one row per sequence: positions[b] = cached_b, and slot and position -1 where new_b = 0.
// ("Day-0 Adaptation: Running Trillion-Parameter Models on Domestic AI Accelerators", 3.2: paged cache, block table from
// logical to physical blocks.)  Release is the inverse: the blocks of finished sequences go back on the stack.
//
// A plan (one CTA: a scan over the sequences) decides everything before anything is written, so that a step that does
// not fit changes neither the tables nor the stack; the expansion is one thread per four query rows.  The first row of
// a page (pos % 64 == 0, always one of the step's rows when the page is new) also writes the table entry, so pages
// need no pass of their own.  Bound by latency (a few bytes per sequence and 12 per row).  On the device: 4.2 us for a decode
// step of 32 sequences, 5.9 us for two 8,192-row chunks beside 16 decodes, 8.4 us for 64 prompts of 1 to 16,384 rows (6.7 MB).
// Release, a CTA per sequence: 4.2 us for 32 sequences of 512 pages, 8.5 us for one of 16,384.
#include <algorithm>

#include "common.cuh"

namespace dsa {

constexpr int kBtPage = 64;
constexpr int kBtPlanThreads = 1024;
constexpr int kBtThreads = 256;
constexpr int kBtRows = 4;                 // query rows per thread

// what the plan leaves in the workspace for the expansion
struct BtHead {
  int32_t refused;                         // nothing may be written
  int32_t rows;                            // cu_q[num_seqs]
  int32_t top;                             // free blocks (extend), or where the first released block goes
};

struct ExtendArgs {
  const int32_t *cached, *add, *free_blocks, *free_count;
  int32_t *table, *seq_lens, *cu_q, *positions, *free_left;      // cu_q nullptr: one row per sequence
  int64_t *slots;
  int num_seqs, max_blocks, num_blocks, total_q, free_cap;
  BtHead *head;                            // workspace
  int32_t *ws_cached, *ws_first;           // workspace [num_seqs]: cached length; the step's first new page of the sequence
  uint32_t *status;
};

// block-wide exclusive scan of two 64-bit values (sums of lengths of a large batch pass 32 bits)
__device__ __forceinline__ void scan2(int64_t a, int64_t b, int64_t (*tmp)[2], int64_t *ea, int64_t *eb, int64_t *ta,
                                      int64_t *tb) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  int64_t x = a, y = b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, x, o), w = __shfl_up_sync(0xffffffffu, y, o);
    if (lane >= o) {
      x += u;
      y += w;
    }
  }
  if (lane == 31) {
    tmp[warp][0] = x;
    tmp[warp][1] = y;
  }
  __syncthreads();
  if (warp == 0) {
    int64_t u = lane < nw ? tmp[lane][0] : 0, w = lane < nw ? tmp[lane][1] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t p = __shfl_up_sync(0xffffffffu, u, o), q = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) {
        u += p;
        w += q;
      }
    }
    tmp[lane][0] = u;
    tmp[lane][1] = w;
  }
  __syncthreads();
  *ea = x - a + (warp ? tmp[warp - 1][0] : 0);
  *eb = y - b + (warp ? tmp[warp - 1][1] : 0);
  *ta = tmp[31][0];
  *tb = tmp[31][1];
  __syncthreads();
}

__device__ __forceinline__ int32_t clamp31(int64_t x, int64_t hi) { return (int32_t)(x < 0 ? 0 : (x > hi ? hi : x)); }

__device__ __forceinline__ void extend_plan(const ExtendArgs &a) {
  __shared__ int64_t tmp[32][2];
  const int64_t cap = (int64_t)a.max_blocks * kBtPage;
  const int32_t count = *a.free_count;            // may be the word free_left points to: written at the end
  int64_t rows = 0, need = 0;
  int bad = 0;
  for (int b0 = 0; b0 < a.num_seqs; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    int64_t add = 0, pages = 0;
    int32_t cached = 0;
    if (b < a.num_seqs) {
      const int64_t c = a.cached[b], n = a.add[b];
      bad |= c < 0 || n < 0 || c + n > cap || (!a.cu_q && n > 1);
      cached = clamp31(c, cap);
      add = n < 0 ? 0 : n;
      const int32_t seq = clamp31(cached + add, cap);
      pages = (seq + kBtPage - 1) / kBtPage - (cached + kBtPage - 1) / kBtPage;
    }
    int64_t er, en, tr, tn;
    scan2(add, pages, tmp, &er, &en, &tr, &tn);
    if (b < a.num_seqs) {
      a.ws_cached[b] = cached;
      a.ws_first[b] = clamp31(need + en, 0x7FFFFFFF);
      if (a.cu_q) a.cu_q[b + 1] = clamp31(rows + er + add, a.total_q);
    }
    rows += tr;
    need += tn;
  }
  bad = __syncthreads_or(bad);
  const bool refused = bad || rows > a.total_q || count < 0 || count > a.free_cap || need > count;
  // seq_lens may be the array `cached` itself: every entry of it has been read by now
  for (int b = threadIdx.x; b < a.num_seqs; b += blockDim.x) {
    a.seq_lens[b] = a.ws_cached[b] + (refused ? 0 : a.add[b]);
    // no rows: cached lengths with the refused rows would put rows at negative positions (b's thread wrote the entry above)
    if (refused && a.cu_q) a.cu_q[b + 1] = 0;
  }
  if (threadIdx.x == 0) {
    if (a.cu_q) a.cu_q[0] = 0;
    a.head->refused = refused;
    a.head->rows = clamp31(rows, a.total_q);
    a.head->top = count;
    *a.free_left = refused ? count : count - (int32_t)need;
    if (refused) set_status(a.status, kStatusBadIndex);
  }
}

// slot of token pos of sequence b (c tokens cached, the step's first new page `first` from the top of the stack), -1 for a bad
// block id; the first row of a new page writes its table entry
__device__ __forceinline__ int64_t place_token(const ExtendArgs &a, int b, int pos, int c, int first, int top) {
  const int page = pos / kBtPage, held = (c + kBtPage - 1) / kBtPage;
  int32_t *entry = a.table + (int64_t)b * a.max_blocks + page;
  int32_t blk = page < held ? *entry : __ldg(a.free_blocks + (top - 1 - (first + page - held)));
  int64_t slot = -1;
  if ((unsigned)blk >= (unsigned)a.num_blocks) {
    set_status(a.status, kStatusBadIndex);
    blk = -1;
  } else {
    slot = (int64_t)blk * kBtPage + pos % kBtPage;
  }
  if (page >= held && pos % kBtPage == 0) *entry = blk;
  return slot;
}

__device__ __forceinline__ void extend_rows(const ExtendArgs &a, int r0) {
  // the plan's results: written by this grid's own block or by the launch before, so not through the read-only path
  const int refused = a.head->refused, rows = a.head->rows, top = a.head->top;
  if (r0 >= a.total_q) return;
  if (!a.cu_q) {                           // row b is sequence b; total_q == num_seqs
    for (int b = r0; b < min(r0 + kBtRows, a.total_q); ++b) {
      const bool has = !refused && a.add[b] > 0;
      const int pos = has ? a.ws_cached[b] : -1;
      a.positions[b] = pos;
      a.slots[b] = has ? place_token(a, b, pos, pos, a.ws_first[b], top) : -1;
    }
    return;
  }
  int b = 0;
  if (!refused && r0 < rows) {             // largest b with cu_q[b] <= r0
    int hi = a.num_seqs - 1;
    while (b < hi) {
      const int mid = (b + hi + 1) >> 1;
      if (a.cu_q[mid] <= r0) b = mid; else hi = mid - 1;
    }
  }
  int seen = -1, c = 0, first = 0, q0 = 0, q1 = 0;
#pragma unroll
  for (int e = 0; e < kBtRows; ++e) {
    const int r = r0 + e;
    if (r >= a.total_q) return;
    int pos = -1;
    int64_t slot = -1;
    if (!refused && r < rows) {
      if (seen < 0) q1 = a.cu_q[b + 1];
      while (q1 <= r) q1 = a.cu_q[++b + 1];        // r < rows = cu_q[num_seqs]: ends at a sequence with rows
      if (seen != b) {
        seen = b;
        q0 = a.cu_q[b];
        c = a.ws_cached[b];
        first = a.ws_first[b];
      }
      pos = c + (r - q0);
      slot = place_token(a, b, pos, c, first, top);
    }
    a.positions[r] = pos;
    a.slots[r] = slot;
  }
}

// plan and expansion in one CTA (few rows)
__global__ void __launch_bounds__(kBtPlanThreads) extend_one_kernel(const ExtendArgs a) {
  pdl_wait();
  pdl_trigger();
  extend_plan(a);
  __syncthreads();
  for (int r = threadIdx.x * kBtRows; r < a.total_q; r += kBtPlanThreads * kBtRows) extend_rows(a, r);
}
__global__ void __launch_bounds__(kBtPlanThreads) extend_plan_kernel(const ExtendArgs a) {
  pdl_wait();
  pdl_trigger();
  extend_plan(a);
}
__global__ void __launch_bounds__(kBtThreads) extend_rows_kernel(const ExtendArgs a) {
  pdl_wait();
  pdl_trigger();
  extend_rows(a, (int)((blockIdx.x * (unsigned)kBtThreads + threadIdx.x) * kBtRows));
}

// ------------------------------------------------------------------------------------------------ release
struct ReleaseArgs {
  const int32_t *done, *table;
  int32_t *seq_lens, *free_blocks, *free_count;
  int num_seqs, max_blocks, num_blocks, free_cap;
  BtHead *head;
  int32_t *ws_pages, *ws_first;            // workspace [num_seqs]: pages given back, and where on the stack
  uint32_t *status;
};

__global__ void __launch_bounds__(kBtPlanThreads) release_plan_kernel(const ReleaseArgs a) {
  pdl_wait();
  pdl_trigger();
  __shared__ int64_t tmp[32][2];
  const int64_t cap = (int64_t)a.max_blocks * kBtPage;
  const int32_t count = *a.free_count;
  int64_t total = 0;
  int bad = 0;
  for (int b0 = 0; b0 < a.num_seqs; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    int64_t pages = 0;
    if (b < a.num_seqs && __ldg(a.done + b) != 0) {
      const int64_t n = a.seq_lens[b];
      bad |= n < 0 || n > cap;
      pages = (clamp31(n, cap) + kBtPage - 1) / kBtPage;
    }
    int64_t ep, e2, tp, t2;
    scan2(pages, 0, tmp, &ep, &e2, &tp, &t2);
    if (b < a.num_seqs) {
      a.ws_pages[b] = (int32_t)pages;
      a.ws_first[b] = clamp31(total + ep, 0x7FFFFFFF);
    }
    total += tp;
  }
  bad = __syncthreads_or(bad);
  const bool refused = bad || count < 0 || count > a.free_cap || total > a.free_cap - count;
  if (threadIdx.x == 0) {
    a.head->refused = refused;
    a.head->top = count;
    if (refused) set_status(a.status, kStatusBadIndex);
    else *a.free_count = count + (int32_t)total;
  }
  if (!refused)
    for (int b = threadIdx.x; b < a.num_seqs; b += blockDim.x)
      if (__ldg(a.done + b) != 0) a.seq_lens[b] = 0;
}

// one CTA per sequence
__global__ void __launch_bounds__(kBtThreads) release_pages_kernel(const ReleaseArgs a) {
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x;
  if (a.head->refused) return;
  const int pages = a.ws_pages[b];
  int32_t *to = a.free_blocks + a.head->top + a.ws_first[b];
  for (int i = threadIdx.x; i < pages; i += kBtThreads) {
    const int32_t blk = __ldg(a.table + (int64_t)b * a.max_blocks + i);
    if ((unsigned)blk >= (unsigned)a.num_blocks) set_status(a.status, kStatusBadIndex);
    to[i] = blk;                           // an id outside the pool stays one: extend refuses to place rows in it
  }
}

// ------------------------------------------------------------------------------------------------ host
size_t batch_tables_ws_bytes(int num_seqs) { return kWsHeader + 256 + 8 * (size_t)num_seqs; }

// Rows up to which one CTA does plan and expansion: 4.4 us against 6.3 for 32 rows, 5.4 against 6.2 for 2,056, 8.2 against
// 6.1 for 4,104.
constexpr int kBtOneCtaRows = 2560;

dsa_status_t batch_extend_launch(const int32_t *cached, const int32_t *add, int num_seqs, int max_blocks, int num_blocks,
                                 int total_q, const int32_t *free_blocks, int free_cap, const int32_t *free_count,
                                 int32_t *table, int32_t *seq_lens, int32_t *cu_q, int64_t *slots, int32_t *positions,
                                 int32_t *free_left, void *ws, cudaStream_t stream) {
  ExtendArgs a{cached, add, free_blocks, free_count, table, seq_lens, cu_q, positions, free_left, slots,
               num_seqs, max_blocks, num_blocks, total_q, free_cap, nullptr, nullptr, nullptr, nullptr};
  char *p = (char *)ws;
  a.status = (uint32_t *)p;
  a.head = (BtHead *)(p + kWsHeader);
  a.ws_cached = (int32_t *)(p + kWsHeader + 256);
  a.ws_first = a.ws_cached + num_seqs;
  if (total_q <= kBtOneCtaRows) {
    DSA_LAUNCH_PDL("extend_one_kernel", extend_one_kernel, dim3(1), dim3(kBtPlanThreads), 0, stream, a);
    return DSA_OK;
  }
  DSA_LAUNCH_PDL("extend_plan_kernel", extend_plan_kernel, dim3(1), dim3(kBtPlanThreads), 0, stream, a);
  const unsigned grid = (unsigned)(((int64_t)total_q + kBtThreads * kBtRows - 1) / (kBtThreads * kBtRows));
  DSA_LAUNCH_PDL("extend_rows_kernel", extend_rows_kernel, dim3(grid), dim3(kBtThreads), 0, stream, a);
  return DSA_OK;
}

dsa_status_t batch_release_launch(const int32_t *done, int num_seqs, int max_blocks, int num_blocks, const int32_t *table,
                                  int32_t *seq_lens, int32_t *free_blocks, int free_cap, int32_t *free_count, void *ws,
                                  cudaStream_t stream) {
  ReleaseArgs a{done, table, seq_lens, free_blocks, free_count, num_seqs, max_blocks, num_blocks, free_cap,
                nullptr, nullptr, nullptr, nullptr};
  char *p = (char *)ws;
  a.status = (uint32_t *)p;
  a.head = (BtHead *)(p + kWsHeader);
  a.ws_pages = (int32_t *)(p + kWsHeader + 256);
  a.ws_first = a.ws_pages + num_seqs;
  DSA_LAUNCH_PDL("release_plan_kernel", release_plan_kernel, dim3(1), dim3(kBtPlanThreads), 0, stream, a);
  DSA_LAUNCH_PDL("release_pages_kernel", release_pages_kernel, dim3(num_seqs), dim3(kBtThreads), 0, stream, a);
  return DSA_OK;
}

}  // namespace dsa
