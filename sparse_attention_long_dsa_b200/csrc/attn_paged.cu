// One-token attention over the paged cache: the f32 path on CUDA cores, the join of split rows, and the choice of path.
//
//   z[h, s] = scale * q[h, :] . K[s],   out[h, :] = sum_s softmax_s(z[h, :]) V[s],   lse[h] = log sum_s exp(z[h, s])
// over every cached token s of the row's sequence, or over the tokens of the pages in the row's list ("Engineering
// Practices for Day-0 Adaptation of Million-Token Context Models on Domestic AI Chips", Four Key Layers 3: the decode
// unit walks the KV blocks and the partial results are merged by a cross-block reduction).
//
// The f32 path: a CTA takes a range of page slots (paged.cuh) for up to 16 heads.  Per tile: keys and values to shared memory as
// f32, one dot product per (token, head) thread slot, a running maximum and sum per head, then P V with the outputs
// of a thread in registers.  Tokens past the sequence are never multiplied: what the cache holds there may be anything.
#include <algorithm>

#include "paged.cuh"

namespace dsa {

dsa_status_t paged_mla_launch(const void *q, const void *kv, int H, float softmax_scale, const PagedView &view,
                              const PagedOut &o, int max_workers, cudaStream_t stream, int num_sms, int *workers);

constexpr int kPsThreads = 256;
constexpr int kPsHeads = 16;                       // most heads
constexpr int kPsTok = kPage;
constexpr int kPsOut = kPsHeads * 128 / kPsThreads;  // most outputs of a thread

struct PsArgs {
  const float *q, *kv, *v;
  PagedView view;
  PagedOut o;
  int H, Dqk, Dv;
  float scale;
};

__device__ __forceinline__ void ps_store(float *p, float v) { *p = v; }
__device__ __forceinline__ void ps_store(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void ps_store4(float *p, const float *v) {
  *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void ps_store4(__nv_bfloat16 *p, const float *v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v[0], v[1]), b = __floats2bfloat162_rn(v[2], v[3]);
  *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
}

__host__ __device__ constexpr int ps_stride(int Dqk) { return (Dqk + 3) / 4 * 4 + 4; }

__global__ void __launch_bounds__(kPsThreads) paged_simt_kernel(const PsArgs a, int min_slots) {
  extern __shared__ float4 sm4[];
  __shared__ uint32_t s_tmp[33];
  __shared__ PagedPlan s_plan;
  __shared__ float s_m[kPsHeads], s_l[kPsHeads], s_alpha[kPsHeads];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int worker = blockIdx.x, nh = a.H;
  const int Dqk = a.Dqk, Dv = a.Dv, D4 = (Dqk + 3) / 4, KS = ps_stride(Dqk);
  float *sq = reinterpret_cast<float *>(sm4);      // [16][4 * D4]
  float *sk = sq + kPsHeads * 4 * D4;              // [kPsTok][KS]
  float *sp = sk + kPsTok * KS;                       // [16][kPsTok]
  float *sv = sp + kPsHeads * kPsTok;              // [64][Dv]
  pdl_wait();
  pdl_trigger();
  plan_pages(a.view, worker, gridDim.x, min_slots, s_tmp, &s_plan);
  if (tid == 0) a.o.info[worker] = worker_info(a.view, s_plan);

  SegmentWalk walk(s_plan);
  int row, sa, sb, part;
  while (walk.next(a.view, s_plan, worker, &row, &sa, &sb, &part)) {
    const int n = row_tokens(a.view, row, a.o.status);
    __syncthreads();
    for (int i = tid; i < kPsHeads * 4 * D4; i += kPsThreads) {
      const int h = i / (4 * D4), d = i % (4 * D4);
      sq[i] = h < nh && d < Dqk ? __ldg(a.q + ((int64_t)row * nh + h) * Dqk + d) : 0.f;
    }
    if (tid < kPsHeads) {
      s_m[tid] = -INFINITY;
      s_l[tid] = 0.f;
    }
    float o[kPsOut];
#pragma unroll
    for (int j = 0; j < kPsOut; ++j) o[j] = 0.f;
    for (int sl = sa; sl < sb; ++sl) {
      int blk;
      const int ntok = slot_tokens(a.view, row, n, sl, &blk, a.o.status);
      if (ntok > 0) {
        const int nt = ntok;
        const int64_t base = (int64_t)blk * kPage;
        __syncthreads();
        for (int i = tid; i < nt * 4 * D4; i += kPsThreads) {
          const int t = i / (4 * D4), d = i % (4 * D4);
          sk[t * KS + d] = d < Dqk ? __ldg(a.kv + (base + t) * Dqk + d) : 0.f;
        }
        for (int i = tid; i < nt * Dv; i += kPsThreads) sv[i] = __ldg(a.v + base * Dv + i);
        __syncthreads();
        for (int i = tid; i < kPsHeads * kPsTok; i += kPsThreads) {
          const int t = i % kPsTok, h = i / kPsTok;
          float z = -INFINITY;
          if (t < nt && h < nh) {
            const float4 *kr = reinterpret_cast<const float4 *>(sk + t * KS);
            const float4 *qr = reinterpret_cast<const float4 *>(sq + h * 4 * D4);
            float acc = 0.f;
            for (int d = 0; d < D4; ++d) {
              const float4 k4 = kr[d], q4 = qr[d];
              acc = fmaf(q4.x, k4.x, acc);
              acc = fmaf(q4.y, k4.y, acc);
              acc = fmaf(q4.z, k4.z, acc);
              acc = fmaf(q4.w, k4.w, acc);
            }
            z = acc * a.scale;
          }
          sp[h * kPsTok + t] = z;
        }
        __syncthreads();
        for (int h = warp; h < nh; h += kPsThreads / 32) {
          float mx = -INFINITY;
          for (int t = lane; t < kPsTok; t += 32) mx = fmaxf(mx, sp[h * kPsTok + t]);
#pragma unroll
          for (int off = 16; off; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
          const float m_old = s_m[h], m_new = fmaxf(m_old, mx), m_use = m_new == -INFINITY ? 0.f : m_new;
          float ls = 0.f;
          for (int t = lane; t < kPsTok; t += 32) {
            const float e = expf(sp[h * kPsTok + t] - m_use);
            sp[h * kPsTok + t] = e;
            ls += e;
          }
#pragma unroll
          for (int off = 16; off; off >>= 1) ls += __shfl_xor_sync(0xffffffffu, ls, off);
          if (lane == 0) {
            const float al = expf(m_old - m_use);
            s_alpha[h] = al;
            s_l[h] = s_l[h] * al + ls;
            s_m[h] = m_new;
          }
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kPsOut; ++j) {
          const int i = tid + kPsThreads * j;
          if (i < nh * Dv) {
            const int h = i / Dv, d = i % Dv;
            float acc = o[j] * s_alpha[h];
            for (int t = 0; t < nt; ++t) acc = fmaf(sp[h * kPsTok + t], sv[t * Dv + d], acc);
            o[j] = acc;
          }
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < kPsOut; ++j) {
      const int i = tid + kPsThreads * j;
      if (i < nh * Dv) {
        const int h = i / Dv, d = i % Dv;
        const float l = s_l[h], val = l != 0.f ? o[j] / l : 0.f;
        if (part < 0) ps_store((float *)a.o.out + ((int64_t)row * nh + h) * Dv + d, val);
        else a.o.part_o[((int64_t)part * nh + h) * Dv + d] = val;
      }
    }
    if (tid < nh) {
      const float lse = s_l[tid] != 0.f ? s_m[tid] + logf(s_l[tid]) : -INFINITY;
      if (part >= 0) a.o.part_lse[(int64_t)part * nh + tid] = lse;
      else if (a.o.lse) a.o.lse[(int64_t)row * nh + tid] = lse;
    }
  }
  // rows without a cached token: zeros, and -inf for the log-sum-exp
  for (int r = worker; r < a.view.T; r += gridDim.x) {
    if (row_slots(a.view, r) > 0) continue;
    for (int i = tid; i < nh * Dv; i += kPsThreads) ps_store((float *)a.o.out + (int64_t)r * nh * Dv + i, 0.f);
    if (a.o.lse && tid < nh) a.o.lse[(int64_t)r * nh + tid] = -INFINITY;
  }
}

// ------------------------------------------------------------------------------------------------ join
// out[row, h, :] = sum_w exp(lse_w - lse) o_w,  lse = log sum_w exp(lse_w)  over the workers w that hold a part of the row.
// At most min(T, workers) rows are split; CTA x finds the x-th of them in info, a warp takes a head (kGroup = 1) or every
// kGroup-th part of one (the sums of the kGroup warps are added in a fixed order).  A lane holds kN pieces of the row (four
// values each where Dv % 4 == 0, else single ones).  Bound by latency: three dependent loads, so it is the number of warps in
// flight that counts.  Few rows have many parts each: kGroup = 8 up to 1,184 (row, head) pairs, one CTA of 8 warps per head
// (a 1M-token row, 74 parts of 128 heads: 8 us, 90 us with one warp per head and part after part); more rows have few parts:
// a warp per head (the 32-row decode batch, 3.3 parts each: 6 us, 28 us with 16 warps per head).
constexpr int kPcThreads = 256, kPcWarps = kPcThreads / 32, kPcMaxWorkers = 160;

template <typename T, int kGroup, int kN, bool kVec>
__global__ void __launch_bounds__(kPcThreads) paged_combine_kernel(const PagedOut o, int workers, int H, int Dv) {
  constexpr int kLane = kVec ? 4 : 1, kBlocks = kPcMaxWorkers / 32;
  __shared__ float s_acc[kGroup > 1 ? kPcWarps : 1][kN * kLane * 32];
  pdl_wait();
  pdl_trigger();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.y * (kPcWarps / kGroup) + warp / kGroup, sub = warp % kGroup;
  int2 info[kBlocks];
#pragma unroll
  for (int i = 0; i < kBlocks; ++i)
    info[i] = 32 * i + lane < workers ? __ldg(o.info + 32 * i + lane) : make_int2(-1, 0);
  int last = -1, row = -1, first = 0, seen = 0;
#pragma unroll
  for (int i = 0; i < kBlocks; ++i) {
    const uint32_t m = __ballot_sync(0xffffffffu, info[i].x >= 0);
    const uint32_t me = __ballot_sync(0xffffffffu, info[i].x >= 0 && seen + __popc(m & ((1u << lane) - 1u)) == (int)blockIdx.x);
    if (me) {
      const int l = __ffs(me) - 1;
      last = 32 * i + l;
      row = __shfl_sync(0xffffffffu, info[i].x, l);
      first = __shfl_sync(0xffffffffu, info[i].y, l);
    }
    seen += __popc(m);
  }
  if (row < 0) return;                             // the same for every warp of the CTA
  const int n = last - first + 1;
  const bool live = h < H;
  float acc[kN * kLane];
#pragma unroll
  for (int i = 0; i < kN * kLane; ++i) acc[i] = 0.f;
  float lse = -INFINITY;
  if (live) {
    // part s: the first worker's odd slot, then the even slots of the workers after it
    auto slot = [&](int s) { return (int64_t)(2 * (first + s) + (s == 0 ? 1 : 0)) * H + h; };
    float w[kBlocks], mx = -INFINITY, tot = 0.f;
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
      w[i] = 32 * i + lane < n ? __ldg(o.part_lse + slot(32 * i + lane)) : -INFINITY;
      mx = fmaxf(mx, w[i]);
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
      w[i] = mx == -INFINITY ? 0.f : expf(w[i] - mx);
      tot += w[i];
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, off);
    const float inv = tot != 0.f ? 1.f / tot : 0.f;
    lse = tot != 0.f ? mx + logf(tot) : -INFINITY;
#pragma unroll
    for (int i = 0; i < kBlocks; ++i) {
      if (32 * i >= n) break;
      const int top = min(32, n - 32 * i);
#pragma unroll 2
      for (int l = sub; l < top; l += kGroup) {    // 32 is a multiple of kGroup
        const float ws = __shfl_sync(0xffffffffu, w[i], l) * inv;
        const float *p = o.part_o + slot(32 * i + l) * Dv;
#pragma unroll
        for (int k = 0; k < kN; ++k) {
          const int d = (32 * k + lane) * kLane;
          if (d < Dv) {
            if (kVec) {
              const float4 v = __ldg(reinterpret_cast<const float4 *>(p + d));
              acc[kLane * k] = fmaf(ws, v.x, acc[kLane * k]);
              acc[kLane * k + kLane / 4] = fmaf(ws, v.y, acc[kLane * k + kLane / 4]);
              acc[kLane * k + kLane / 2] = fmaf(ws, v.z, acc[kLane * k + kLane / 2]);
              acc[kLane * k + kLane - 1] = fmaf(ws, v.w, acc[kLane * k + kLane - 1]);
            } else {
              acc[k] = fmaf(ws, __ldg(p + d), acc[k]);
            }
          }
        }
      }
    }
  }
  if (kGroup > 1) {
#pragma unroll
    for (int i = 0; i < kN * kLane; ++i) s_acc[warp][32 * i + lane] = acc[i];
    __syncthreads();
    if (sub > 0) return;
#pragma unroll
    for (int i = 0; i < kN * kLane; ++i)
      for (int g = 1; g < kGroup; ++g) acc[i] += s_acc[warp + g][32 * i + lane];
  }
  if (!live) return;
  T *out = (T *)o.out + ((int64_t)row * H + h) * Dv;
#pragma unroll
  for (int k = 0; k < kN; ++k) {
    const int d = (32 * k + lane) * kLane;
    if (d >= Dv) continue;
    if (kVec) ps_store4(out + d, acc + kLane * k);
    else ps_store(out + d, acc[k]);
  }
  if (o.lse && lane == 0) o.lse[(int64_t)row * H + h] = lse;
}

template <typename T, int kN, bool kVec>
static dsa_status_t combine_launch(const PagedOut &o, int workers, int T_rows, int H, int Dv, cudaStream_t stream) {
  const int rows = std::min(workers, T_rows);
  if ((int64_t)T_rows * H <= 8 * 148) {
    DSA_LAUNCH_PDL("paged_combine_kernel", (paged_combine_kernel<T, 8, kN, kVec>), dim3(rows, H), dim3(kPcThreads), 0, stream, o,
                   workers, H, Dv);
  } else {
    DSA_LAUNCH_PDL("paged_combine_kernel", (paged_combine_kernel<T, 1, kN, kVec>), dim3(rows, (H + kPcWarps - 1) / kPcWarps),
                   dim3(kPcThreads), 0, stream, o, workers, H, Dv);
  }
  return DSA_OK;
}

// ------------------------------------------------------------------------------------------------ host
static size_t pg_al(size_t x) { return (x + 255) / 256 * 256; }

// The most workers a launch uses; they size the workspace.  Value width tells the two paths apart: 512 is the latent
// cache's (CTA pairs of a B200's 148 SMs), up to 128 the f32 path's.
static int paged_max_workers(int Dv) { return Dv > 128 ? 74 : 148; }

size_t paged_workspace_bytes(int H, int Dv) {
  const size_t w = (size_t)paged_max_workers(Dv);
  return kWsHeader + pg_al(w * sizeof(int2)) + pg_al(2 * w * H * 4) + pg_al(2 * w * H * Dv * 4);
}

static PagedOut paged_out(void *ws, int H, int Dv, void *out, float *lse) {
  const size_t w = (size_t)paged_max_workers(Dv);
  PagedOut o{};
  char *p = (char *)ws;
  o.status = (uint32_t *)p;
  p += kWsHeader;
  o.info = (int2 *)p;
  p += pg_al(w * sizeof(int2));
  o.part_lse = (float *)p;
  p += pg_al(2 * w * H * 4);
  o.part_o = (float *)p;
  o.out = out;
  o.lse = lse;
  return o;
}

dsa_status_t paged_attn_launch(const void *q, bool bf16, const void *kv, const void *v, int H, int Dqk, int Dv,
                               float scale, const int32_t *pages, int kb, const dsa_batch_t *b, void *out, float *lse,
                               void *ws, cudaStream_t stream, int num_sms) {
  PsArgs a{};
  a.q = (const float *)q;
  a.kv = (const float *)kv;
  a.v = (const float *)v;
  a.view = PagedView{b->block_table, b->seq_lens, pages, b->total_q, kb, b->max_blocks_per_seq, b->num_blocks};
  a.o = paged_out(ws, H, Dv, out, lse);
  a.H = H;
  a.Dqk = Dqk;
  a.Dv = Dv;
  a.scale = scale;
  if (bf16) {
    int workers = 0;
    const dsa_status_t st = paged_mla_launch(q, kv, H, scale, a.view, a.o, paged_max_workers(Dv), stream, num_sms, &workers);
    if (st != DSA_OK) return st;
    return combine_launch<__nv_bfloat16, 4, true>(a.o, workers, b->total_q, H, Dv, stream);
  }
  const int workers = std::min(num_sms, paged_max_workers(Dv));
  const int D4 = (Dqk + 3) / 4;
  const size_t smem = 4 * ((size_t)kPsHeads * 4 * D4 + (size_t)kPsTok * ps_stride(Dqk) + kPsHeads * kPsTok + (size_t)kPsTok * Dv);
  cudaFuncSetAttribute(paged_simt_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  DSA_LAUNCH_PDL("paged_simt_kernel", paged_simt_kernel, dim3(workers), dim3(kPsThreads), smem, stream, a, 2);
  if (Dv % 4 == 0) return combine_launch<float, 1, true>(a.o, workers, b->total_q, H, Dv, stream);
  return combine_launch<float, 4, false>(a.o, workers, b->total_q, H, Dv, stream);
}

}  // namespace dsa
