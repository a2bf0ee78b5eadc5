// One-token attention over the paged latent cache on tcgen05 tensor cores, one CTA pair (cluster of 2) per worker.
//
//   z[h, s] = scale * q[h, :] . K[s],   out[h, :] = sum_s softmax_s(z[h, :]) V[s],   V[s] = first 512 of the 576 entries
// for up to 128 heads of the row, over the tokens of every page of the sequence or of a list of pages ("Engineering
// Practices for Day-0 Adaptation of Million-Token Context Models on Domestic AI Chips", Four Key Layers 3: decode
// prefetches the next KV block while the current one is computed, partial results are merged by a cross-block reduction).
//
// A token costs 1152 bytes of HBM and 2 x 128 x 1088 products whatever the number of heads (missing heads are zero rows of
// q): 0.176 ns of copy bandwidth against 0.169 ns of tensor peak.  So copies and matrix instructions both have to run without
// a pause.  Split of a pair's work (rank r = 0, 1), one page of 64 tokens at a time, over the flat range of page slots that
// paged.cuh gives it; 384 threads per CTA:
//   * keys   : one warp walks the slots (32 table entries per load, the next 32 ahead), publishes the pages that hold tokens
//              to the other roles through a ring (physical row, tokens, row, first / last of its segment) and copies this
//              CTA's 32 tokens of the page, all 576 entries, by one tiled TMA copy into one of four buffers [9 blocks]
//              [32 tokens][128 B] (a page is contiguous; pieces of a page gathered row by row cost 2 us on a last page);
//   * QK^T   : M = 128 heads (64 per CTA), N = 64 tokens (32 from each CTA), K = 576, up to four pages ahead of P V;
//   * values : each CTA needs 256 of the 512 value entries of all 64 tokens: the peer's 32 tokens' half (16 KB, an L2 hit)
//              is copied over the blocks that QK^T no longer needs, as soon as it has run.  In a sequence's last page the
//              rows past its end become zeros before P V reads them, and whole steps of 16 tokens past it are left out;
//   * softmax: two groups of four warps take alternate pages, one (head, 32-token half) per thread.  Both use one reference
//              per head, and O is rescaled in TMEM only when a score outgrows it by 2^8 (exact: the final division uses the
//              same reference);
//   * P V    : two N = 256 MMAs for each 16 tokens; O (64 heads x 512 fp32 per CTA) stays in TMEM.  P lies half in the
//              page's ninth block, half in one of two 4 KB buffers, so that two pages of it are in flight.
// P is rounded to bf16 for P V, as the tensor cores take it (2^-8 of a weight); the sum l keeps the unrounded weights in fp32.
//
// Measured on one B200, whole calls (the join included) back to back for seconds, where the 1000 W cap holds the SM clock: 1 row
// of 1,048,576 tokens 323 us at 1.33 GHz (3.7 TB/s of keys, 0.9 PFLOP/s; 278 us in bursts of four calls at full clock); 32 rows of
// 4K - 32K tokens 158 us at 1.42 GHz (140 in bursts, of which this kernel 129: DRAM 54 %, tensor pipe 53 % busy); 61 rows up
// to 8K, 16 heads, 81 us at 1.61 GHz; 1 row of 130 tokens 11 us.
// A page takes 1.2 us of a pair at full clock: 0.83 us is what DRAM gives, 1,425 cycles the matrix instructions (QK^T 36 steps of 25.3
// cycles, held by the operand reads at N = 64; P V 8 of 64.3), and what is left is the way of a buffer through copy, QK^T,
// softmax, P V.
// What lost: QK^T of two pages as one N = 128 instruction (32.3 cycles a step, but a page then waits for the next one: 1M row
// 280 -> 299 us), the latent entries split over the pair with partial scores exchanged (831 us: 32 KB through distributed
// shared memory take 1,950 cycles), pages brought into L2 ahead of their copies (no gain with four buffers).
#include <algorithm>
#include <atomic>

#include "paged.cuh"
#include "tc.cuh"

namespace dsa {

constexpr int kPtD = 576, kPtDv = 512;
constexpr int kPtHalf = kPage / 2;
constexpr int kPtNBuf = 4;                         // page buffers, and score tiles
constexpr int kPtRing = 8;                         // published pages in flight
// Fewest pages of a worker, and the longest row that stays whole: a page takes 1.2 us of a pair, cutting a row 3 us.  One row of 4
// pages 13.0 us whole, 14.3 in two pieces; 16 rows of 5 pages 14.6, 16.7; one row of 8 pages 14.5 us in pieces of two, 16.0 of
// four; of 128 pages 20.4 in pieces of two, 19.2 of four (one row of 64 times min_slots takes twice as many).
constexpr uint32_t kPtMinSlots = 2, kPtWhole = 5;
// More rows than workers, whole against cut anywhere.  128 heads: 128 rows of 8 pages 32.2 us, 40.5 cut, 100 of 8 - 13 37.8, 40.6; but
// 75 of 16 (the longest worker has 32 pages, 16 more than the average) 44.4, 41.4, and one of 16 beside 74 of one 26.9, 18.5.
// Up to 32 heads, where q and the results of a segment count less: 128 of 8 28.2, 30.8; 150 of 8 36.7, 33.4; 75 of 8 27.0, 24.0.
__device__ __forceinline__ PagedRule pt_rule(int H) {
  return H > 32 ? PagedRule{kPtMinSlots, kPtWhole, 16, 6, 12.f} : PagedRule{kPtMinSlots, kPtWhole, 10, 4, 5.f};
}
constexpr int kPtThreads = 384;                    // softmax x 8, keys, QK^T, P V, values
constexpr int kPtGroup = 128;                      // threads of a softmax group (4 warps)
constexpr int kPtWarpKeys = 8, kPtWarpQK = 9, kPtWarpPV = 10, kPtWarpValues = 11;
constexpr uint32_t kPtBlk = kPtHalf * 128;         // one 64-entry block of a CTA's 32 tokens: 4 KB
constexpr uint32_t kPtBuf = 9 * kPtBlk;
constexpr uint32_t kPtQSize = 9 * 8192;
constexpr uint32_t kPtP = 4096;                    // half of P: [64 heads][32 tokens] bf16, 64-byte swizzle
constexpr uint32_t kPtTmemO = 0, kPtTmemS = 256;
constexpr float kPtRescale = 8.0f;
constexpr long long kPtSettle = 2000000;           // SM cycles, about 1 ms
constexpr int kPtFirst = 1, kPtLast = 2, kPtEmpty = 4, kPtEnd = 8, kPtQ = 16;     // kPtQ: q of an empty segment was loaded

struct PtSmem {
  uint64_t buf_full[kPtNBuf];       // rank 0: bytes of both CTAs' tokens
  uint64_t buf_empty[kPtNBuf];      // MMA commit to both CTAs after P V
  uint64_t v_full[kPtNBuf];         // rank 0: both CTAs have the peer's values
  uint64_t tail_full;               // the peer's values of a sequence's last page
  uint64_t q_full, q_empty;
  uint64_t s_full[kPtNBuf];
  uint64_t p_full[2], pv_done[2];   // by page parity
  uint64_t o_empty, drain[2];
  uint64_t ent_full[kPtRing], ent_empty[kPtRing];
  uint32_t tmem_base;
  int abort;
  int4 ent[kPtRing];                // physical row, tokens, row, flags | (part + 1) << 8
  uint64_t dec[2];                  // the references of a page are decided, by its parity
  uint64_t l_ready[2];              // lp is written
  uint64_t st_free;                 // the staging tiles of a segment's epilogue have been read
  float ref[64];                    // reference of each head, log2 units
  float x[2][kPtGroup];             // maxima, then sums, of the threads of a head
  float lp[2][kPtGroup];            // the other group's sums of a segment, by its parity
  uint32_t tmp[33];
  PagedPlan plan;
};

struct PtArgs {
  PagedView view;
  PagedOut o;
  int H;
  float scale_log2;
};

// Waits of whole warps.  A phase that is already complete costs one test and a branch: with what stands between two waits 100 to
// 160 cycles, where the general form (its loop and a warp vote inline) took 150 to 250; ten of them lie on the way of a page.
__device__ __noinline__ bool pt_wait_slow(uint32_t bar, uint32_t parity, volatile int *abort, uint32_t *status) {
  return tc::mbar_wait(bar, parity, abort, status);
}
__device__ __noinline__ bool pt_wait_slow_cl(uint32_t bar, uint32_t parity, volatile int *abort, uint32_t *status) {
  return tc::mbar_wait_cl(bar, parity, abort, status);
}
__device__ __forceinline__ bool pt_wait(uint32_t bar, uint32_t parity, volatile int *abort, uint32_t *status) {
  bool ok = tc::mbar_try_wait(bar, parity);
  if (__builtin_expect(!ok, 0)) ok = pt_wait_slow(bar, parity, abort, status);
  __syncwarp();
  return ok;
}
// for barriers that receive the other CTA's arrivals
__device__ __forceinline__ bool pt_wait_cl(uint32_t bar, uint32_t parity, volatile int *abort, uint32_t *status) {
  bool ok = tc::mbar_try_wait_cl(bar, parity);
  if (__builtin_expect(!ok, 0)) ok = pt_wait_slow_cl(bar, parity, abort, status);
  __syncwarp();
  return ok;
}
// .cta_group::2: the completion bytes may be counted on the other CTA's barrier
__device__ __forceinline__ void pt_load_3d_pair(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
      "[%0], [%1, {%3, %4, %5}], [%2];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}
// true if any thread of softmax group g says so
__device__ __forceinline__ bool pt_any(int g, bool x) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %3, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"((uint32_t)x), "n"(kPtGroup), "r"(3 + g)
      : "memory");
  return r != 0;
}
// K-major operand in rows of 64 bytes, 8-row atoms of 512 bytes, 64-byte swizzle
__device__ __forceinline__ uint64_t pt_desc_sw64(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)1u << 16;
  d |= (uint64_t)(512u >> 4) << 32;
  d |= (uint64_t)1u << 46;                              // descriptor version (sm_100)
  d |= (uint64_t)4u << 61;                              // layout: 64-byte swizzle
  return d;
}
// arrive on a barrier of this or the other CTA with bytes to come
__device__ __forceinline__ void pt_expect_tx_cluster(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cluster.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool pt_elect() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(r));
  return r != 0;
}
__device__ __forceinline__ void pt_mma_pair(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d_tmem), "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)accumulate)
      : "memory");
}

struct PtMaps {
  CUtensorMap q;                    // [T][H][576] in boxes of 64 heads x 64 entries
  CUtensorMap keys, values;         // [9 blocks][tokens][64] in boxes of 32 tokens and 9 / 4 blocks
};

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPtThreads, 1)
    paged_mla_kernel(const __grid_constant__ PtMaps tm, const PtArgs a) {
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t *sQ = smem;                              // [9 blocks][64 heads][128 B]
  uint8_t *sBuf = sQ + kPtQSize;                       // 4 x [9 blocks][32 tokens][128 B]
  uint8_t *sP = sBuf + kPtNBuf * kPtBuf;           // second halves of two pages' P; epilogue staging
  PtSmem *S = (PtSmem *)(sP + 2 * kPtP);

  const uint32_t rank = tc::cluster_ctarank();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kPtNBuf; ++i) {
      tc::mbar_init(tc::smem_u32(&S->buf_full[i]), 1);
      tc::mbar_init(tc::smem_u32(&S->buf_empty[i]), 1);
      tc::mbar_init(tc::smem_u32(&S->v_full[i]), 2);
      tc::mbar_init(tc::smem_u32(&S->s_full[i]), 1);
    }
    tc::mbar_init(tc::smem_u32(&S->st_free), 4);
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(tc::smem_u32(&S->p_full[i]), 8);
      tc::mbar_init(tc::smem_u32(&S->pv_done[i]), 1);
      tc::mbar_init(tc::smem_u32(&S->dec[i]), 4);
      tc::mbar_init(tc::smem_u32(&S->l_ready[i]), 4);
    }
    tc::mbar_init(tc::smem_u32(&S->tail_full), 1);
    tc::mbar_init(tc::smem_u32(&S->q_full), 1);
    tc::mbar_init(tc::smem_u32(&S->q_empty), 1);
    tc::mbar_init(tc::smem_u32(&S->o_empty), 8);
    for (int i = 0; i < 2; ++i) tc::mbar_init(tc::smem_u32(&S->drain[i]), 1);
    for (int i = 0; i < kPtRing; ++i) {
      tc::mbar_init(tc::smem_u32(&S->ent_full[i]), 1);
      tc::mbar_init(tc::smem_u32(&S->ent_empty[i]), rank == 0 ? 11 : 9);   // softmax x 8, values, QK^T and P V (rank 0)
    }
    S->abort = 0;
    tc::fence_barrier_init();
    tc::prefetch_tmap(&tm.q);
    tc::prefetch_tmap(&tm.keys);
    tc::prefetch_tmap(&tm.values);
  }
  if (warp == kPtWarpPV) {
    tc::tmem_alloc2(tc::smem_u32(&S->tmem_base), 512);
    tc::tmem_relinquish2();
  }
  tc::fence_before_sync();
  __syncthreads();
  tc::cluster_sync();
  tc::fence_after_sync();
  const uint32_t tmem = S->tmem_base;
  volatile int *abort = &S->abort;
  uint32_t *status = a.o.status;
  // inputs come from earlier work on the stream
  pdl_wait();
  pdl_trigger();
  plan_pages(a.view, pair, npairs, pt_rule(a.H), S->tmp, &S->plan);

  // next entry of the ring, for a whole warp: false ends the role (the end of the work, or a wait that ran out)
  auto next_entry = [&](uint32_t &ec, int4 *e) -> bool {
    const uint32_t slot = ec % kPtRing;
    const bool ok = pt_wait(tc::smem_u32(&S->ent_full[slot]), (ec / kPtRing) & 1u, abort, status);
    if (!ok) return false;
    *e = S->ent[slot];
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(tc::smem_u32(&S->ent_empty[slot]));
    ++ec;
    return true;
  };

  if (warp == kPtWarpKeys) {
    // ====================================================================== pages, keys and q
    const uint32_t buf_full_r0 = tc::map_to_rank(tc::smem_u32(&S->buf_full[0]), 0);
    const uint32_t q_full_r0 = tc::map_to_rank(tc::smem_u32(&S->q_full), 0);
    uint32_t ec = 0, c = 0, v = 0;
    auto publish = [&](int phys, int ntok, int row, int info) -> bool {
      const uint32_t slot = ec % kPtRing;
      if (!pt_wait(tc::smem_u32(&S->ent_empty[slot]), ((ec / kPtRing) & 1u) ^ 1u, abort, status)) return false;
      if (lane == 0) {
        S->ent[slot] = make_int4(phys, ntok, row, info);
        tc::mbar_arrive(tc::smem_u32(&S->ent_full[slot]));
      }
      __syncwarp();
      ++ec;
      return true;
    };
    auto load_q = [&](int row) {
      if (lane == 0 && rank == 0) tc::mbar_expect_tx(tc::smem_u32(&S->q_full), 2u * kPtQSize);
      __syncwarp();
      if (lane < 9) pt_load_3d_pair(tc::smem_u32(sQ + lane * 8192), &tm.q, lane * 64, 64 * (int)rank, row, q_full_r0);
      ++v;
    };
    bool q_loaded = false;
    auto page = [&](int phys, int ntok, int row, int info) -> bool {
      if (!publish(phys, ntok, row, info)) return false;
      const uint32_t b = c % kPtNBuf;
      if (!pt_wait(tc::smem_u32(&S->buf_empty[b]), ((c / kPtNBuf) & 1u) ^ 1u, abort, status)) return false;
      if (lane == 0) {
        if (rank == 0) tc::mbar_expect_tx(tc::smem_u32(&S->buf_full[b]), 2u * kPtBuf);
        pt_load_3d_pair(tc::smem_u32(sBuf + b * kPtBuf), &tm.keys, 0, phys + kPtHalf * (int)rank, 0, buf_full_r0 + b * 8);
      }
      __syncwarp();
      if ((info & kPtFirst) && !q_loaded) {
        // q is overwritten once the previous segment's last QK^T has run
        if (!pt_wait(tc::smem_u32(&S->q_empty), (v - 1) & 1u, abort, status)) return false;
        load_q(row);
      }
      if (info & kPtFirst) q_loaded = false;
      ++c;
      return true;
    };
    SegmentWalk walk(S->plan);
    int row, sa, sb, part;
    bool ok = true;
    while (ok && walk.next(a.view, S->plan, pair, &row, &sa, &sb, &part)) {
      // the first segment's q is on its way while its pages are looked up (later ones' pages come first)
      if (v == 0) {
        load_q(row);
        q_loaded = true;
      }
      const int n = row_tokens(a.view, row, status);
      const int tag = (part + 1) << 8;
      // 32 slots per load, the next 32 loaded ahead; one page is held back until it is known whether another follows
      int flags = kPtFirst, h_phys = 0, h_ntok = 0, blk = 0, nt = 0;
      if (sa + lane < sb) nt = slot_tokens(a.view, row, n, sa + lane, &blk, status);
      for (int s0 = sa; s0 < sb && ok; s0 += 32) {
        int blk_n = 0, nt_n = 0;
        if (s0 + 32 + lane < sb) nt_n = slot_tokens(a.view, row, n, s0 + 32 + lane, &blk_n, status);
        uint32_t have = __ballot_sync(0xffffffffu, nt > 0);
        while (have && ok) {
          const int l = __ffs(have) - 1;
          have &= have - 1;
          if (h_ntok) {
            ok = page(h_phys, h_ntok, row, flags | tag);
            flags = 0;
          }
          h_phys = __shfl_sync(0xffffffffu, blk, l) * kPage;
          h_ntok = __shfl_sync(0xffffffffu, nt, l);
        }
        blk = blk_n;
        nt = nt_n;
      }
      if (ok) ok = h_ntok ? page(h_phys, h_ntok, row, flags | kPtLast | tag) : publish(0, 0, row, kPtEmpty | tag | (q_loaded ? kPtQ : 0));
      q_loaded = false;
    }
    if (ok) publish(0, 0, 0, kPtEnd);
    if (lane == 0 && rank == 0) a.o.info[pair] = worker_info(a.view, S->plan);
  } else if (warp == kPtWarpValues) {
    // ====================================================================== the peer's values
    // Token half t of a page lies in blocks 4t .. 4t + 3 of either CTA: its own tokens' values where the key copy put them,
    // the peer's copied here.
    const uint32_t v_full_r0 = tc::map_to_rank(tc::smem_u32(&S->v_full[0]), 0);
    const uint32_t tail = tc::smem_u32(&S->tail_full);
    const int other = (int)(rank ^ 1u);
    uint32_t ec = 0, c = 0, tails = 0;
    int4 e;
    while (next_entry(ec, &e)) {
      if (e.w & kPtEnd) break;
      if (e.w & kPtEmpty) continue;
      const uint32_t b = c % kPtNBuf, full = v_full_r0 + b * 8;
      uint8_t *buf = sBuf + b * kPtBuf;
      const uint32_t dst = tc::smem_u32(buf + 4 * other * kPtBlk);
      // QK^T of this page has read the buffers
      if (!pt_wait(tc::smem_u32(&S->s_full[b]), (c / kPtNBuf) & 1u, abort, status)) break;
      if (e.y == kPage) {
        if (lane == 0) {
          pt_expect_tx_cluster(full, 4u * kPtBlk);
          pt_load_3d_pair(dst, &tm.values, 0, e.x + kPtHalf * other, 4 * (int)rank, full);
        }
      } else {
        // A sequence's last page: P V takes its tokens in steps of 16 and leaves out the steps behind the last one; in that one
        // the rows past the sequence become zeros here, so that 0 x (whatever the cache holds there) never enters a sum.
        if (e.y > kPtHalf * other) {
          if (lane == 0) {
            tc::mbar_expect_tx(tail, 4u * kPtBlk);
            pt_load_3d_pair(dst, &tm.values, 0, e.x + kPtHalf * other, 4 * (int)rank, tail);
          }
          __syncwarp();
          if (!pt_wait(tail, tails++ & 1u, abort, status)) break;
        }
        const int last = (e.y - 1) / 16, t = last / 2;                       // the last step, and its token half
        const int r0 = e.y - kPtHalf * t, rows = 16 * (last + 1) - e.y;      // rows r0 .. r0 + rows - 1 of that half
        for (int i = lane; i < rows * 4 * 8; i += 32)
          *reinterpret_cast<uint4 *>(buf + (4 * t + (i >> 3) % 4) * kPtBlk + (r0 + (i >> 5)) * 128 + (i & 7) * 16) =
              make_uint4(0, 0, 0, 0);
        tc::fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          if (rank == 0) tc::mbar_arrive(full);
          else tc::mbar_arrive_remote(full);
        }
      }
      __syncwarp();
      ++c;
    }
  } else if (warp == kPtWarpQK || warp == kPtWarpPV) {
    // ====================================================================== MMA issuers (rank 0, whole warps); empty rows (rank 1)
    // Two warps, because issuing a page's MMAs and waiting for its operands takes one warp longer (about 1,900 cycles) than
    // the tensor core needs to run them (1,425).  A page's score tile is free when its buffer is.
    if (rank == 0) {
      const uint16_t both = 3;
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      uint32_t ec = 0, c = 0, segs = 0;
      int4 e;
      const int which = warp == kPtWarpPV;
      if (which == 0) {
        constexpr uint32_t idesc = tc::make_idesc(1, 1, 128, kPage, false, false);
        const uint64_t q_desc = tc::desc_sw128(tc::smem_u32(sQ), 1024);
        const uint64_t kv_desc = tc::desc_sw128(tc::smem_u32(sBuf), 1024);
        while (next_entry(ec, &e)) {
          const int info = __shfl_sync(0xffffffffu, e.w, 0);
          if (info & kPtEnd) break;
          if (info & kPtQ) {
            if (!pt_wait(tc::smem_u32(&S->q_full), segs++ & 1u, abort, status)) break;
            tc::mma_commit_pair_w(tc::smem_u32(&S->q_empty), both);
          }
          if (info & kPtEmpty) continue;
          const uint32_t b = c % kPtNBuf;
          if ((info & kPtFirst) && !pt_wait(tc::smem_u32(&S->q_full), segs++ & 1u, abort, status)) break;
          if (!pt_wait(tc::smem_u32(&S->buf_full[b]), (c / kPtNBuf) & 1u, abort, status)) break;
          tc::fence_after_sync();
          const uint64_t kb = kv_desc + ((b * kPtBuf) >> 4);
          const uint32_t d = tm + kPtTmemS + kPtHalf * b;
          if (pt_elect()) {
#pragma unroll
            for (int i = 0; i < 9; ++i)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                pt_mma_pair(d, q_desc + ((i * 8192) >> 4) + 2 * k, kb + ((i * kPtBlk) >> 4) + 2 * k, idesc, i + k > 0);
          }
          __syncwarp();
          tc::mma_commit_pair_w(tc::smem_u32(&S->s_full[b]), both);
          if (info & kPtLast) tc::mma_commit_pair_w(tc::smem_u32(&S->q_empty), both);
          ++c;
        }
      } else {
        constexpr uint32_t idesc = tc::make_idesc(1, 1, 128, 256, false, true);
        const uint64_t p0_desc = pt_desc_sw64(tc::smem_u32(sBuf + 8 * kPtBlk)), p1_desc = pt_desc_sw64(tc::smem_u32(sP));
        const uint64_t v_desc = tc::desc_sw128_lbo(tc::smem_u32(sBuf), kPtBlk, 1024);
        while (next_entry(ec, &e)) {
          const int info = __shfl_sync(0xffffffffu, e.w, 0);
          if (info & kPtEnd) break;
          if (info & kPtEmpty) continue;
          const uint32_t b = c % kPtNBuf;
          const bool first = info & kPtFirst;
          const int steps = (__shfl_sync(0xffffffffu, e.y, 0) + 15) / 16;
          if (first) {
            if (segs > 0 && !pt_wait_cl(tc::smem_u32(&S->o_empty), (segs - 1) & 1u, abort, status)) break;
            ++segs;
          }
          if (!pt_wait(tc::smem_u32(&S->v_full[b]), (c / kPtNBuf) & 1u, abort, status)) break;
          if (!pt_wait_cl(tc::smem_u32(&S->p_full[c & 1u]), (c >> 1) & 1u, abort, status)) break;
          tc::fence_after_sync();
          const uint64_t vb = v_desc + ((b * kPtBuf) >> 4);
          const uint64_t p0 = p0_desc + ((b * kPtBuf) >> 4), p1 = p1_desc + (((c & 1u) * kPtP) >> 4);
          if (pt_elect()) {
            // K steps of 16 tokens: token half (4 blocks apart) x two steps of 16 rows; both value halves share a step of P
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if (k >= steps) break;
#pragma unroll
              for (int p = 0; p < 2; ++p)
                pt_mma_pair(tm + kPtTmemO + 128 * p, (k < 2 ? p0 : p1) + 2 * (k & 1),
                            vb + ((2 * p * kPtBlk + (k >> 1) * 4 * kPtBlk + (k & 1) * 16 * 128) >> 4), idesc, k > 0 || !first);
            }
          }
          __syncwarp();
          tc::mma_commit_pair_w(tc::smem_u32(&S->buf_empty[b]), both);
          tc::mma_commit_pair_w(tc::smem_u32(&S->pv_done[c & 1u]), both);
          ++c;
        }
      }
      tc::mma_commit_pair_local_w(tc::smem_u32(&S->drain[which]));
      volatile int no_abort = 0;
      __all_sync(0xffffffffu, tc::mbar_wait(tc::smem_u32(&S->drain[which]), 0, &no_abort, status));
    } else {
      zero_empty_rows<__nv_bfloat16>(a.view, a.o, a.H, kPtDv, 2 * pair + (warp == kPtWarpPV), 2 * npairs);
    }
  } else {
    // ====================================================================== softmax + epilogue (two groups of 4 warps)
    // Group g takes the pages c with c % 2 == g.  Thread: TMEM lane L = (head h, token half), that half's 32 tokens.  P of a
    // page is 2^(z - ref) with one reference per head for both groups: the owner of page c decides it after the owner of
    // page c - 1 has (dec), changes it only where a score outgrows it by 2^8, and then rescales O (exact: the final division
    // uses the same reference).  The warps of a group leave the loop together (one vote per entry): they hold named barriers.
    const int g = warp >> 2, L = threadIdx.x & (kPtGroup - 1);
    const int h = L & 63, half = L >> 6;
    const int head = 64 * (int)rank + h;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t p_full_r0 = tc::map_to_rank(tc::smem_u32(&S->p_full[0]), 0) + 8 * g;
    const uint32_t o_empty_r0 = tc::map_to_rank(tc::smem_u32(&S->o_empty), 0);
    __nv_bfloat16 *out = (__nv_bfloat16 *)a.o.out;
    float m_run = -INFINITY, l_run = 0.f;          // this thread's tokens of the segment: reference, sum of weights
    uint32_t ec = 0, c = 0, seg = 0;
    int4 e = make_int4(0, 0, 0, 0);
    for (;;) {
      bool ok = next_entry(ec, &e);
      const bool page = ok && !(e.w & (kPtEnd | kPtEmpty));
      const bool first = e.w & kPtFirst, last = e.w & kPtLast;
      if (page && first) {
        m_run = -INFINITY;
        l_run = 0.f;
      }
      if (page && (int)(c & 1u) != g) {            // the other group's page
        if (last) {                                // hand over the sums, at the segment's final references
          pt_wait(tc::smem_u32(&S->dec[c & 1u]), (c >> 1) & 1u, abort, status);
          S->lp[seg & 1u][L] = l_run != 0.f ? l_run * tc::ex2(m_run - S->ref[h]) : 0.f;
          __syncwarp();
          if (lane == 0) tc::mbar_arrive(tc::smem_u32(&S->l_ready[seg & 1u]));
          ++seg;
        }
        ++c;
        continue;
      }
      float sv[kPtHalf];
      float mx = -INFINITY;
      if (page) {
        ok = pt_wait(tc::smem_u32(&S->s_full[c % kPtNBuf]), (c / kPtNBuf) & 1u, abort, status);
        tc::fence_after_sync();
        tc::tmem_ld32(tmem + lane_base + kPtTmemS + kPtHalf * (c % kPtNBuf), sv);
        tc::tmem_wait_ld();
        if (e.y < kPage) {
#pragma unroll
          for (int i = 0; i < kPtHalf; ++i) sv[i] = i < e.y - kPtHalf * half ? sv[i] : -INFINITY;
        }
        float m4[4] = {sv[0], sv[1], sv[2], sv[3]};
#pragma unroll
        for (int i = 4; i < kPtHalf; ++i) m4[i & 3] = fmaxf(m4[i & 3], sv[i]);
        mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * a.scale_log2;
        if (c > 0) ok = pt_wait(tc::smem_u32(&S->dec[(c - 1) & 1u]), ((c - 1) >> 1) & 1u, abort, status) && ok;
        if (!first) {
          const float r = S->ref[h];
          if (r != m_run) {                        // the other group has moved it
            l_run *= tc::ex2(m_run - r);
            m_run = r;
          }
        }
      }
      // One vote per entry: has a wait run out, or a score outgrown its reference?
      if (pt_any(g, !ok || (page && (first || mx > m_run + kPtRescale)))) {
        if (pt_any(g, !ok)) break;
        // the new reference of a head is the largest score so far
        S->x[g][L] = fmaxf(m_run, mx);
        tc::named_bar_sync(1 + g, kPtGroup);
        const float m_new = fmaxf(S->x[g][L], S->x[g][L ^ 64]);
        // TMEM accesses are warp-collective: every row of the warp is brought to its new reference.  P V of the previous
        // page must have finished before O is touched.
        if (!first && __any_sync(0xffffffffu, m_new > m_run)) {
          // (P V of page c - 2 first: it shows that page c - 3's has run too, so that the phase asked for is the next one)
          if (c >= 2) pt_wait(tc::smem_u32(&S->pv_done[g]), ((c - 2) >> 1) & 1u, abort, status);
          ok = pt_wait(tc::smem_u32(&S->pv_done[g ^ 1]), ((c - 1) >> 1) & 1u, abort, status);
          tc::fence_after_sync();
          const float alpha = m_new > m_run ? tc::ex2(m_run - m_new) : 1.f;
          if (ok) {
            for (int cc = 0; cc < 8; ++cc) {
              float ov[32];
              tc::tmem_ld32(tmem + lane_base + kPtTmemO + 32 * cc, ov);
              tc::tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) ov[i] *= alpha;
              tc::tmem_st32(tmem + lane_base + kPtTmemO + 32 * cc, ov);
            }
            tc::tmem_wait_st();
          }
          tc::fence_before_sync();
          l_run *= alpha;
        }
        m_run = m_new;
        if (half == 0) S->ref[h] = m_new;
      }
      if (e.w & kPtEnd) break;
      const int row = e.z, part = (e.w >> 8) - 1;
      if (e.w & kPtEmpty) {                        // no page of the segment holds a token
        if (head < a.H && g == 0) {
          if (part < 0) {
            __nv_bfloat16 *o = out + ((int64_t)row * a.H + head) * kPtDv + 256 * half;
            for (int i = 0; i < 256; i += 8) *reinterpret_cast<uint4 *>(o + i) = make_uint4(0, 0, 0, 0);
            if (a.o.lse && half == 0) a.o.lse[(int64_t)row * a.H + head] = -INFINITY;
          } else {
            float *o = a.o.part_o + ((int64_t)part * a.H + head) * kPtDv + 256 * half;
            for (int i = 0; i < 256; i += 4) *reinterpret_cast<float4 *>(o + i) = make_float4(0.f, 0.f, 0.f, 0.f);
            if (half == 0) a.o.part_lse[(int64_t)part * a.H + head] = -INFINITY;
          }
        }
        continue;
      }
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(tc::smem_u32(&S->dec[g]));
      // P = exp2(z - ref) in bf16 into the 128-byte-swizzled A operand; masked tokens hold -inf and give 0
      const float m_use = m_run == -INFINITY ? 0.f : m_run;
      uint32_t pw[16];
      float ls[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float p0 = tc::ex2(fmaf(sv[2 * i], a.scale_log2, -m_use)), p1 = tc::ex2(fmaf(sv[2 * i + 1], a.scale_log2, -m_use));
        ls[i & 3] += p0 + p1;
        const __nv_bfloat162 pb = __floats2bfloat162_rn(p0, p1);
        pw[i] = *reinterpret_cast<const uint32_t *>(&pb);
      }
      l_run += (ls[0] + ls[1]) + (ls[2] + ls[3]);
      // Tokens 0-31 go where the page's last key block was (QK^T has read it), tokens 32-63 to one of two buffers, last read by
      // P V of page c - 2 or by the epilogue of the segment before
      if (c >= 2) ok = pt_wait(tc::smem_u32(&S->pv_done[g]), ((c - 2) >> 1) & 1u, abort, status) && ok;
      if (first && seg > 0) ok = pt_wait(tc::smem_u32(&S->st_free), (seg - 1) & 1u, abort, status) && ok;
      if (ok) {
        uint8_t *pbuf = (half == 0 ? sBuf + (c % kPtNBuf) * kPtBuf + 8 * kPtBlk : sP + g * kPtP) + h * 64;
#pragma unroll
        for (int q8 = 0; q8 < 4; ++q8)
          *reinterpret_cast<uint4 *>(pbuf + ((q8 ^ ((h >> 1) & 3)) << 4)) =
              make_uint4(pw[4 * q8], pw[4 * q8 + 1], pw[4 * q8 + 2], pw[4 * q8 + 3]);
      }
      tc::fence_proxy_async();
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        if (rank == 0) tc::mbar_arrive(tc::smem_u32(&S->p_full[g]));
        else tc::mbar_arrive_remote(p_full_r0);
      }
      ++c;
      if (!last) continue;

      // ---- epilogue: wait for the last P V, add up the sums, normalise and store
      ok = pt_wait(tc::smem_u32(&S->pv_done[g]), ((c - 1) >> 1) & 1u, abort, status) && ok;
      ok = pt_wait(tc::smem_u32(&S->l_ready[seg & 1u]), (seg >> 1) & 1u, abort, status) && ok;
      tc::fence_after_sync();
      S->x[g][L] = l_run + S->lp[seg & 1u][L];
      tc::named_bar_sync(1 + g, kPtGroup);
      const float l_tot = S->x[g][h] + S->x[g][h + 64];
      const float inv = l_tot != 0.f ? 1.f / l_tot : 0.f;
      if (ok) {
        // Through a per-warp tile of 32 rows x 64 bytes in the P buffer (16-byte group j of a row at j ^ (row / 2 & 3)), in
        // 64-byte pieces of rows: 32 entries of a result, 16 of a partial one
        float *stg = reinterpret_cast<float *>(sP) + (warp & 3) * 512;
        const int head0 = 64 * (int)rank + 32 * (warp & 1), col0 = 256 * half;
        if (head0 < a.H) {
          auto store = [&](const float (&ov)[32], int col) {
            if (part < 0) {
              uint8_t *tile = reinterpret_cast<uint8_t *>(stg);
#pragma unroll
              for (int q8 = 0; q8 < 4; ++q8) {
                uint32_t w[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const __nv_bfloat162 b = __floats2bfloat162_rn(ov[8 * q8 + 2 * i] * inv, ov[8 * q8 + 2 * i + 1] * inv);
                  w[i] = *reinterpret_cast<const uint32_t *>(&b);
                }
                *reinterpret_cast<uint4 *>(tile + lane * 64 + ((q8 ^ ((lane >> 1) & 3)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
              }
              __syncwarp();
#pragma unroll
              for (int it = 0; it < 4; ++it) {
                const int r = 8 * it + (lane >> 2), j = lane & 3;
                if (head0 + r < a.H)
                  *reinterpret_cast<uint4 *>(out + ((int64_t)row * a.H + head0 + r) * kPtDv + col + 8 * j) =
                      *reinterpret_cast<const uint4 *>(tile + r * 64 + ((j ^ ((r >> 1) & 3)) << 4));
              }
              __syncwarp();
            } else {
#pragma unroll
              for (int hh = 0; hh < 2; ++hh) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  const float *f = ov + 16 * hh + 4 * j;
                  *reinterpret_cast<float4 *>(stg + lane * 16 + 4 * (j ^ ((lane >> 1) & 3))) =
                      make_float4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
                }
                __syncwarp();
#pragma unroll
                for (int it = 0; it < 4; ++it) {
                  const int r = 8 * it + (lane >> 2), j = lane & 3;
                  if (head0 + r < a.H)
                    *reinterpret_cast<float4 *>(a.o.part_o + ((int64_t)part * a.H + head0 + r) * kPtDv + col + 16 * hh + 4 * j) =
                        *reinterpret_cast<const float4 *>(stg + r * 16 + 4 * (j ^ ((r >> 1) & 3)));
                }
                __syncwarp();
              }
            }
          };
          for (int cc = 0; cc < 8; cc += 2) {
            float o0[32], o1[32];
            tc::tmem_ld32(tmem + lane_base + kPtTmemO + 32 * cc, o0);
            tc::tmem_ld32(tmem + lane_base + kPtTmemO + 32 * cc + 32, o1);
            tc::tmem_wait_ld();
            store(o0, col0 + 32 * cc);
            store(o1, col0 + 32 * cc + 32);
          }
        }
        if (half == 0 && head < a.H) {
          const float lse = l_tot != 0.f ? (m_run + __log2f(l_tot)) * 0.69314718055994531f : -INFINITY;
          if (part >= 0) a.o.part_lse[(int64_t)part * a.H + head] = lse;
          else if (a.o.lse) a.o.lse[(int64_t)row * a.H + head] = lse;
        }
      }
      tc::fence_before_sync();
      __syncwarp();
      if (lane == 0) {
        tc::mbar_arrive(tc::smem_u32(&S->st_free));
        if (rank == 0) tc::mbar_arrive(tc::smem_u32(&S->o_empty));
        else tc::mbar_arrive_remote(o_empty_r0);
      }
      ++seg;
    }
  }

  // ---- teardown: every role is done; MMAs drained; the peer done with our barriers, buffers and TMEM
  tc::fence_before_sync();
  __syncthreads();
  if (*abort) {
    // A wait ran out, so that copies of keys, values or q may be on their way that no role will wait for, some counted on the other
    // CTA's barrier.  They land long before this ends; their shared memory stays this pair's until then.
    for (const long long t0 = clock64(); clock64() - t0 < kPtSettle;) {
    }
  }
  tc::cluster_sync();
  if (warp == kPtWarpPV) {
    tc::fence_after_sync();
    tc::tmem_dealloc2(tmem, 512);
  }
}

// ------------------------------------------------------------------------------------------------ host
typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn encode_tiled_fn();

// bf16, [d2][d1][d0] with strides s1, s2 (entries), in boxes of b2 x b1 x 64 entries, 128-byte swizzle
static bool pt_map(CUtensorMap *m, const void *base, uint64_t d0, uint64_t d1, uint64_t d2, uint64_t s1,
                   uint64_t s2, uint32_t b1, uint32_t b2) {
  EncodeTiledFn enc = encode_tiled_fn();
  if (!enc) return false;
  cuuint64_t dims[3] = {d0, d1, d2}, strides[2] = {s1 * 2, s2 * 2};
  cuuint32_t box[3] = {64, b1, b2}, es[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The main kernel of the latent cache; returns the workers (CTA pairs) through *workers for the join.
dsa_status_t paged_mla_launch(const void *q, const void *kv, int H, float softmax_scale, const PagedView &view,
                              const PagedOut &o, int max_workers, cudaStream_t stream, int num_sms, int *workers) {
  PtArgs a{view, o, H, softmax_scale * 1.4426950408889634f};
  PtMaps tm;
  const uint64_t rows = (uint64_t)view.num_blocks * kPage, D = kPtD;
  if (!pt_map(&tm.q, q, D, (uint64_t)H, (uint64_t)view.T, D, D * H, 64, 1) ||
      !pt_map(&tm.keys, kv, 64, rows, 9, D, 64, kPtHalf, 9) || !pt_map(&tm.values, kv, 64, rows, 9, D, 64, kPtHalf, 4)) {
    set_error("paged attention: cuTensorMapEncodeTiled failed");
    return DSA_ERR_CUDA;
  }
  constexpr size_t smem = kPtQSize + kPtNBuf * kPtBuf + 2 * kPtP + sizeof(PtSmem);
  static_assert(smem <= 227 * 1024, "shared memory of a CTA");
  // as many CTA pairs as can be resident at once, found once per device (threads that race on the first call
  // compute the same number)
  static std::atomic<int> resident[kMaxDevices];
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
    set_error("no current CUDA device");
    return DSA_ERR_CUDA;
  }
  if (cudaFuncSetAttribute(paged_mla_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) {
    set_error("paged attention: %s", cudaGetErrorString(cudaGetLastError()));
    return DSA_ERR_CUDA;
  }
  int pairs = resident[dev].load(std::memory_order_relaxed);
  if (pairs == 0) {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.gridDim = dim3(num_sms & ~1);
    cfg.blockDim = dim3(kPtThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, paged_mla_kernel, &cfg) != cudaSuccess || n < 1) {
      cudaGetLastError();
      n = num_sms / 2;
    }
    pairs = std::max(1, std::min(n, num_sms / 2));
    resident[dev].store(pairs, std::memory_order_relaxed);
  }
  *workers = std::min(pairs, max_workers);
  DSA_LAUNCH_PDL("paged_mla_kernel", paged_mla_kernel, dim3(2 * *workers), dim3(kPtThreads), smem, stream, tm, a);
  return DSA_OK;
}

}  // namespace dsa
