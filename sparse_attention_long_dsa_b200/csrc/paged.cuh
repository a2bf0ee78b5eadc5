// One-token attention over the paged cache: how its kernels walk the pages of a batch.
//
// Every row of a decode batch has a number of page slots (all pages of its sequence, or the kb entries of its page
// list).  The slots of all rows, one row after another, form one flat range of P slots, and every worker takes a
// contiguous piece of it that it finds from the lengths alone (they stay on the device), in one of two ways:
//   * the flat split: worker w of np takes [floor(w P / np), floor((w + 1) P / np)), equal to within one page whatever
//     the lengths are, but for borders inside short rows, which move to the row's end;
//   * the split by rows: every row is cut into pieces of its own, so that no worker takes the end of one row and the
//     beginning of the next.
// The piece of a row inside a worker's range is a segment.  A segment that holds its whole row writes the row's
// result; the others write a partial result, normalised with its log-sum-exp, to a slot of the workspace: slot
// 2w + 1 when the row starts in worker w (and goes on), 2w when it started before.  Worker w notes in info[w] the
// row that ends in it after starting elsewhere, and the combine kernel joins that row's partials in the workers'
// order, so results do not depend on timing.
#pragma once

#include "common.cuh"

namespace dsa {

constexpr int kPage = 64;

struct PagedView {
  const int32_t *block_table;   // [T, max_blocks]
  const int32_t *seq_lens;      // [T]
  const int32_t *pages;         // [T, kb] or nullptr: every page
  int T, kb, max_blocks, num_blocks;
};

struct PagedOut {
  void *out;                    // [T, H, Dv]
  float *lse;                   // [T, H] or nullptr
  float *part_o;                // [2 workers, H, Dv]
  float *part_lse;              // [2 workers, H]
  int2 *info;                   // [workers] (row, first worker), row -1: none
  uint32_t *status;
};

// How finely rows may be cut, in page slots.
struct PagedRule {
  uint32_t min_slots;           // a worker for every so many
  uint32_t whole;               // rows up to this stay whole
  uint32_t uncut;               // with more rows than workers, rows up to this too, unless a worker's range would get longer
  uint32_t row_over;            //   than the average one by more than this through a single row
  float range_over;             //   or than this through the number of rows, which the workers share unevenly
};

struct PagedPlan {
  uint32_t total;               // P
  uint32_t start, end;          // this worker's slots
  int np;                       // the flat split: workers that have any
  int row, page;                // where `start` lies
  int first;                    // split by rows: the worker that `row` starts in; -1: the flat split
};

__device__ __forceinline__ int row_slots(const PagedView &v, int row) {
  const int n = __ldg(v.seq_lens + row);
  if (n <= 0) return 0;
  if (v.pages) return v.kb;
  const int p = (int)(((int64_t)n + kPage - 1) / kPage);
  return p < v.max_blocks ? p : v.max_blocks;
}

// cached tokens of a row, cut to what its block-table row can hold
__device__ __forceinline__ int row_tokens(const PagedView &v, int row, uint32_t *status) {
  const int n = __ldg(v.seq_lens + row);
  const int64_t cap = (int64_t)v.max_blocks * kPage;
  if (n > cap) {
    set_status(status, kStatusBadIndex);
    return (int)cap;
  }
  return n;
}

// tokens that slot i of a row holds, and its physical block; 0 tokens: the slot is skipped
__device__ __forceinline__ int slot_tokens(const PagedView &v, int row, int n, int i, int *block, uint32_t *status) {
  int pg = i;
  if (v.pages) pg = __ldg(v.pages + (int64_t)row * v.kb + i);
  if (pg < 0 || pg >= v.max_blocks || pg * (int64_t)kPage >= n) return 0;
  const int blk = __ldg(v.block_table + (int64_t)row * v.max_blocks + pg);
  if ((unsigned)blk >= (unsigned)v.num_blocks) {
    set_status(status, kStatusBadIndex);
    return 0;
  }
  *block = blk;
  const int left = n - pg * kPage;
  return left < kPage ? left : kPage;
}

__device__ __forceinline__ int worker_of_slot(uint32_t f, const PagedPlan &p) {
  return (int)((((uint64_t)f + 1) * (uint64_t)p.np - 1) / p.total);
}

// The threads that make a plan: one warp (up to 32 rows: no barriers, 0.5 us less), or the block.
template <bool kWarp>
struct PlanThreads {
  uint32_t *tmp;                // 33 words, for the block
  __device__ __forceinline__ int count() const { return kWarp ? 32 : (int)blockDim.x; }
  __device__ __forceinline__ uint32_t scan(uint32_t v, uint32_t *total) const {
    if (!kWarp) return block_exclusive_scan(v, tmp, total);
    uint32_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
      if ((int)threadIdx.x >= o) x += y;
    }
    *total = __shfl_sync(0xffffffffu, x, 31);
    return x - v;
  }
  __device__ __forceinline__ bool all(bool x) const { return kWarp ? __all_sync(0xffffffffu, x) : __syncthreads_and(x); }
  __device__ __forceinline__ bool any(bool x) const { return kWarp ? __any_sync(0xffffffffu, x) : __syncthreads_or(x); }
  __device__ __forceinline__ int sum(uint32_t x) const {       // (a scan is four times the code)
    if (threadIdx.x == 0) tmp[0] = 0;
    __syncthreads();
    x = __reduce_add_sync(0xffffffffu, x);
    if ((threadIdx.x & 31) == 0) atomicAdd(tmp, x);
    __syncthreads();
    return (int)tmp[0];
  }
  __device__ __forceinline__ int that(bool x) const { return kWarp ? __popc(__ballot_sync(0xffffffffu, x)) : __syncthreads_count(x); }
};

// The split by rows; thread r has row r, of `mine` slots behind `before` others.  c0, c1, c2: the longest pieces to try; c2 needs
// at most W workers, the others at most 2 W; rows of at most `whole` slots stay whole.  false: a piece would be longer than `limit`.
template <bool kWarp>
__device__ __forceinline__ bool split_rows(const PlanThreads<kWarp> &th, int worker, uint32_t mine, uint32_t before, uint32_t total,
                                           uint32_t limit, uint32_t W, uint32_t whole, uint32_t c0, uint32_t c1, uint32_t c2,
                                           PagedPlan *p) {
  // 10 bits for each count of workers: W <= 148
  uint32_t n0 = (mine + c0 - 1) / c0, n1 = (mine + c1 - 1) / c1, n2 = (mine + c2 - 1) / c2;
  if (mine <= whole) n0 = n1 = n2 = min(mine, 1u);
  uint32_t sums;
  uint32_t at = th.scan(n0 | n1 << 10 | n2 << 20, &sums);
  uint32_t n = n2, c = c2, shift = 20;
  if (((sums >> 10) & 1023u) <= W && c1 <= c) n = n1, c = c1, shift = 10;
  if ((sums & 1023u) <= W && c0 <= c) n = n0, shift = 0;
  at = (at >> shift) & 1023u;
  const uint32_t size = mine / max(n, 1u), longer = mine - size * n;       // the first `longer` pieces have size + 1 slots
  if (th.any(size + (longer > 0) > limit)) return false;
  const uint32_t w = (uint32_t)worker, piece = w - at;
  if (w >= at && piece < n) {                          // one thread: the worker's piece is of its row
    const uint32_t from = piece * size + min(piece, longer);
    p->start = before + from;
    p->end = before + from + size + (piece < longer);
    p->row = (int)threadIdx.x;
    p->page = (int)from;
    p->first = (int)at;
  }
  if (threadIdx.x == 0 && w >= ((sums >> shift) & 1023u)) p->start = p->end = total;
  return true;
}

template <bool kWarp>
__device__ __forceinline__ void make_plan(const PlanThreads<kWarp> &th, const PagedView &v, int worker, int workers,
                                          const PagedRule &rule, PagedPlan *p) {
  const uint32_t min_slots = rule.min_slots, whole = rule.whole;
  const int nt = th.count(), per = kWarp ? 1 : (v.T + nt - 1) / nt;
  const int r0 = min(v.T, (int)threadIdx.x * per), r1 = min(v.T, r0 + per);
  uint32_t mine = 0, some = 0;
  for (int r = r0; r < r1; ++r) {
    const uint32_t n = (uint32_t)row_slots(v, r);
    mine += n;
    some += n > 0;
  }
  uint32_t total;
  const uint32_t before = th.scan(mine, &total);
  // A worker for every min_slots page slots, and rows of at most `whole` slots in one piece: cutting a row costs partial results
  // and their join.  One row of 64 min_slots and more: twice the slots, because its join grows with its pieces (latent
  // cache, 8,192 tokens: 20.9 -> 19.4 us; f32: 10.5 -> 9.0 us).
  const uint32_t want = total / (v.T == 1 && total >= 64 * min_slots ? 2 * min_slots : min_slots);
  int np = want < 1u || (v.T == 1 && total <= whole) ? 1 : (want < (uint32_t)workers ? (int)want : workers);
  // A second segment costs a worker what kSegment pages do (q, the epilogue, a pipeline that runs empty).  So no worker takes
  // the end of one row and the beginning of the next where the longest piece is not longer than the flat split's by more than
  // that.  Rows of one length (a batch of page lists) only need a number of workers that is the same for each: 32 rows of 8
  // pages 18 us, 22 us with the flat split.  Others, of n slots each, are cut into ceil(n / c) pieces, c the smallest of three
  // lengths that needs no more workers than there are.  Latent cache: 8 rows of 2 - 3 pages 13.7 us, 18.2 with the flat split; 26
  // rows of one page or none 11.9, 15.3; 16 rows of 1 - 13 pages 18.0, 20.7.  f32: 16 rows of 4 - 128 pages, 4 heads of 64 13.2,
  // 13.9; 16 heads of 128 33.6, 38.4.  Where it turns out not to pay, looking for it costs 0.3 us.
  constexpr uint32_t kSegment = 4;
  uint32_t keep = whole;
  if (v.T > 1) {
    const uint32_t n0 = total / (uint32_t)v.T;
    const bool same = th.all(mine == n0 * (uint32_t)(r1 - r0));
    const int rows = same ? v.T : per == 1 ? th.that(mine > 0) : th.sum(some);       // that hold tokens
    // More rows than workers: a border that moves to a row's end saves a segment, partial results and their join, but the call waits
    // for the worker with the most rows, ceil(rows / np) of them where the average one has rows / np.
    const uint32_t mean = total / (uint32_t)np, limit = mean + kSegment;
    if (rows > workers) {
      // (approximate: divisions and branches here run cold, and cost a call up to 1 us)
      const float each = __fdividef((float)rows, (float)np), idle = ceilf(each - 1e-3f) - each;
      if (idle * (float)mean <= rule.range_over * each) keep = max(whole, min(rule.uncut, mean + rule.row_over));
    }
    if (same && rows <= workers) {
      const uint32_t each = rows < np && n0 > whole ? (uint32_t)np / (uint32_t)rows : 1u;
      if (n0 / each <= limit) np = (int)each * rows;
    }
    if (!same && per == 1 && rows > 1 && rows <= workers && total > (uint32_t)np) {
      const uint32_t R = (uint32_t)rows, W = max((uint32_t)np, R), avg = (total + R - 1) / R;
      const uint32_t c0 = (avg + W / R - 1) / (W / R), c1 = (total + W - R / 2 - 1) / (W - R / 2);
      const uint32_t c2 = W > R ? (total + W - R - 1) / (W - R) : total;
      if (min(min(c0, c1), c2) <= limit &&
          split_rows(th, worker, mine, before, total, limit, W, whole, max(c0, min_slots), max(c1, min_slots), max(c2, min_slots), p))
        return;
    }
  }
  const bool any = worker < np;
  const uint32_t start = any ? (uint32_t)((uint64_t)worker * total / np) : total;
  const uint32_t end = any ? (uint32_t)((uint64_t)(worker + 1) * total / np) : total;
  if (threadIdx.x == 0) {
    p->total = total;
    p->np = np;
    p->first = -1;
    if (start >= end) p->start = total;
    if (start >= end || end == total) p->end = total;
  }
  // The threads whose rows the two borders lie in.  A border inside a row of at most `keep` slots moves to the nearer end of it: a
  // cut costs a segment, partial results and their join.
  if (start < end) {
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const uint32_t x = side == 0 ? start : end;
      if (x >= before && x < before + mine) {
        uint32_t at = before, n = mine;
        int r = r0;
        if (per > 1)
          for (;; ++r) {
            n = (uint32_t)row_slots(v, r);
            if (x < at + n) break;
            at += n;
          }
        uint32_t page = x - at;
        if (page > 0 && n <= keep) {
          if (2 * page >= n) {
            at += n;
            ++r;
          }
          page = 0;
        }
        if (side == 0) {
          p->start = at + page;
          p->row = r;
          p->page = (int)page;
        } else {
          p->end = at + page;
        }
      }
    }
  }
}

// Every thread of the block calls this (blockDim.x a multiple of 32, at most 1024); `tmp` holds 33 words.
__device__ __forceinline__ void plan_pages(const PagedView &v, int worker, int workers, const PagedRule &rule, uint32_t *tmp,
                                           PagedPlan *p) {
  if (v.T > 32) make_plan(PlanThreads<false>{tmp}, v, worker, workers, rule, p);
  else if (threadIdx.x < 32) make_plan(PlanThreads<true>{tmp}, v, worker, workers, rule, p);
  __syncthreads();
}

// the segments of a worker's range, in order
struct SegmentWalk {
  uint32_t pos;
  int row, page;                // next slot
  __device__ __forceinline__ explicit SegmentWalk(const PagedPlan &p) : pos(p.start), row(p.row), page(p.page) {}
  // slots [a, b) of row r, of n; part: partial slot or -1 for a whole row
  __device__ __forceinline__ bool next(const PagedView &v, const PagedPlan &p, int worker, int *r, int *a, int *b,
                                       int *part) {
    while (pos < p.end) {
      const int n = row_slots(v, row);
      if (n == 0) {
        ++row;
        continue;
      }
      const int room = n - page, left = (int)(p.end - pos);
      *r = row;
      *a = page;
      *b = page + (room < left ? room : left);
      *part = (*a == 0 && *b == n) ? -1 : 2 * worker + (*a == 0 ? 1 : 0);
      pos += (uint32_t)(*b - *a);
      ++row;
      page = 0;
      return true;
    }
    return false;
  }
};

// what the combine kernel has to join at this worker (one thread calls it)
__device__ __forceinline__ int2 worker_info(const PagedView &v, const PagedPlan &p) {
  if (p.start >= p.end || p.page == 0) return make_int2(-1, 0);
  const int n = row_slots(v, p.row);
  if ((uint32_t)(n - p.page) > p.end - p.start) return make_int2(-1, 0);      // the row goes on in the next worker
  return make_int2(p.row, p.first >= 0 ? p.first : worker_of_slot(p.start - (uint32_t)p.page, p));
}

// Rows without a cached token: zeros, and -inf for the log-sum-exp.  Whole warps call it, `mine` of `warps`; row r belongs to warp
// r % warps, 32 rows looked at per load.
template <typename T>
__device__ __forceinline__ void zero_empty_rows(const PagedView &v, const PagedOut &o, int H, int Dv, int64_t mine, int64_t warps) {
  const int lane = threadIdx.x & 31;
  for (int64_t r0 = mine; r0 < v.T; r0 += 32 * warps) {
    const int64_t r = r0 + lane * warps;
    uint32_t empty = __ballot_sync(0xffffffffu, r < v.T && row_slots(v, (int)r) == 0);
    while (empty) {
      const int64_t row = r0 + (__ffs(empty) - 1) * warps;
      empty &= empty - 1;
      T *out = (T *)o.out + row * H * Dv;
      if (((int64_t)H * Dv * sizeof(T)) % 16 == 0) {
        for (int i = lane; i < (int)(H * Dv * sizeof(T) / 16); i += 32) reinterpret_cast<uint4 *>(out)[i] = make_uint4(0, 0, 0, 0);
      } else {
        for (int i = lane; i < H * Dv; i += 32) out[i] = T(0.f);
      }
      if (o.lse)
        for (int i = lane; i < H; i += 32) o.lse[row * H + i] = -INFINITY;
    }
  }
}

}  // namespace dsa
