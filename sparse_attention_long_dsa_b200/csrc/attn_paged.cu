// One-token attention over the paged cache on CUDA cores, and the join of split rows.
//
//   z[h, s] = scale * q[h, :] . K[s],   out[h, :] = sum_s softmax_s(z[h, :]) V[s],   lse[h] = log sum_s exp(z[h, s])
// over every cached token s of the row's sequence, or over the tokens of the pages in the row's list ("Engineering
// Practices for Day-0 Adaptation of Million-Token Context Models on Domestic AI Chips", Four Key Layers 3: the decode
// unit walks the KV blocks and the partial results are merged by a cross-block reduction).
//
// A CTA takes a range of page slots (paged.cuh) for up to 16 heads.  Per tile: keys and values to shared memory as
// f32, one dot product per (token, head) thread slot, a running maximum and sum per head, then P V with the outputs
// of a thread in registers.  Tokens past the sequence are never multiplied: what the cache holds there may be anything.
#include <algorithm>

#include "paged.cuh"

namespace dsa {

constexpr int kPsThreads = 256;
constexpr int kPsHeads = 16;                       // heads per CTA

struct PsArgs {
  const void *q, *kv, *v;
  PagedView view;
  PagedOut o;
  int H, Dqk, Dv;
  float scale;
};

__device__ __forceinline__ float ps_load(const float *p) { return __ldg(p); }
__device__ __forceinline__ float ps_load(const __nv_bfloat16 *p) { return __bfloat162float(*p); }
__device__ __forceinline__ void ps_store(float *p, float v) { *p = v; }
__device__ __forceinline__ void ps_store(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }

__host__ __device__ constexpr int ps_stride(int Dqk) { return (Dqk + 3) / 4 * 4 + 4; }

template <typename T, int TOK, int NO, bool kShared>
__global__ void __launch_bounds__(kPsThreads) paged_simt_kernel(const PsArgs a, int min_slots) {
  extern __shared__ float4 sm4[];
  __shared__ uint32_t s_tmp[33];
  __shared__ PagedPlan s_plan;
  __shared__ float s_m[kPsHeads], s_l[kPsHeads], s_alpha[kPsHeads];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int worker = blockIdx.x, h0 = blockIdx.y * kPsHeads, nh = min(kPsHeads, a.H - h0);
  const int Dqk = a.Dqk, Dv = a.Dv, D4 = (Dqk + 3) / 4, KS = ps_stride(Dqk);
  float *sq = reinterpret_cast<float *>(sm4);      // [16][4 * D4]
  float *sk = sq + kPsHeads * 4 * D4;              // [TOK][KS]
  float *sp = sk + TOK * KS;                       // [16][TOK]
  float *sv = kShared ? sk : sp + kPsHeads * TOK;  // [TOK][Dv]
  const int VS = kShared ? KS : Dv;
  pdl_wait();
  pdl_trigger();
  plan_pages(a.view, worker, gridDim.x, min_slots, s_tmp, &s_plan);
  if (tid == 0 && blockIdx.y == 0) a.o.info[worker] = worker_info(a.view, s_plan);

  SegmentWalk walk(s_plan);
  int row, sa, sb, part;
  while (walk.next(a.view, s_plan, worker, &row, &sa, &sb, &part)) {
    const int n = row_tokens(a.view, row, a.o.status);
    __syncthreads();
    for (int i = tid; i < kPsHeads * 4 * D4; i += kPsThreads) {
      const int h = i / (4 * D4), d = i % (4 * D4);
      sq[i] = h < nh && d < Dqk ? ps_load((const T *)a.q + ((int64_t)row * a.H + h0 + h) * Dqk + d) : 0.f;
    }
    if (tid < kPsHeads) {
      s_m[tid] = -INFINITY;
      s_l[tid] = 0.f;
    }
    float o[NO];
#pragma unroll
    for (int j = 0; j < NO; ++j) o[j] = 0.f;
    for (int sl = sa; sl < sb; ++sl) {
      int blk;
      const int ntok = slot_tokens(a.view, row, n, sl, &blk, a.o.status);
      for (int t0 = 0; t0 < ntok; t0 += TOK) {
        const int nt = min(TOK, ntok - t0);
        const int64_t base = (int64_t)blk * kPage + t0;
        __syncthreads();
        for (int i = tid; i < nt * 4 * D4; i += kPsThreads) {
          const int t = i / (4 * D4), d = i % (4 * D4);
          sk[t * KS + d] = d < Dqk ? ps_load((const T *)a.kv + (base + t) * Dqk + d) : 0.f;
        }
        if (!kShared)
          for (int i = tid; i < nt * Dv; i += kPsThreads) sv[i] = ps_load((const T *)a.v + base * Dv + i);
        __syncthreads();
        for (int i = tid; i < kPsHeads * TOK; i += kPsThreads) {
          const int t = i % TOK, h = i / TOK;
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
          sp[h * TOK + t] = z;
        }
        __syncthreads();
        for (int h = warp; h < nh; h += kPsThreads / 32) {
          float mx = -INFINITY;
          for (int t = lane; t < TOK; t += 32) mx = fmaxf(mx, sp[h * TOK + t]);
#pragma unroll
          for (int off = 16; off; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
          const float m_old = s_m[h], m_new = fmaxf(m_old, mx), m_use = m_new == -INFINITY ? 0.f : m_new;
          float ls = 0.f;
          for (int t = lane; t < TOK; t += 32) {
            const float e = expf(sp[h * TOK + t] - m_use);
            sp[h * TOK + t] = e;
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
        for (int j = 0; j < NO; ++j) {
          const int i = tid + kPsThreads * j;
          if (i < nh * Dv) {
            const int h = i / Dv, d = i % Dv;
            float acc = o[j] * s_alpha[h];
            for (int t = 0; t < nt; ++t) acc = fmaf(sp[h * TOK + t], sv[t * VS + d], acc);
            o[j] = acc;
          }
        }
      }
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NO; ++j) {
      const int i = tid + kPsThreads * j;
      if (i < nh * Dv) {
        const int h = i / Dv, d = i % Dv;
        const float l = s_l[h], val = l != 0.f ? o[j] / l : 0.f;
        if (part < 0) ps_store((T *)a.o.out + ((int64_t)row * a.H + h0 + h) * Dv + d, val);
        else a.o.part_o[((int64_t)part * a.H + h0 + h) * Dv + d] = val;
      }
    }
    if (tid < nh) {
      const float lse = s_l[tid] != 0.f ? s_m[tid] + logf(s_l[tid]) : -INFINITY;
      if (part >= 0) a.o.part_lse[(int64_t)part * a.H + h0 + tid] = lse;
      else if (a.o.lse) a.o.lse[(int64_t)row * a.H + h0 + tid] = lse;
    }
  }
  // rows without a cached token: zeros, and -inf for the log-sum-exp
  for (int r = worker; r < a.view.T; r += gridDim.x) {
    if (row_slots(a.view, r) > 0) continue;
    for (int i = tid; i < nh * Dv; i += kPsThreads) ps_store((T *)a.o.out + ((int64_t)r * a.H + h0) * Dv + i, 0.f);
    if (a.o.lse && tid < nh) a.o.lse[(int64_t)r * a.H + h0 + tid] = -INFINITY;
  }
}

// ------------------------------------------------------------------------------------------------ join
// out[row, h, :] = sum_w exp(lse_w - lse) o_w,  lse = log sum_w exp(lse_w)  over the workers w that hold a part of the row.
// One CTA per (worker in which a split row ends, head).
template <typename T>
__global__ void __launch_bounds__(128) paged_combine_kernel(const PagedOut o, int H, int Dv) {
  pdl_wait();
  pdl_trigger();
  const int last = blockIdx.x, h = blockIdx.y;
  const int2 who = __ldg(o.info + last);
  if (who.x < 0) return;
  const int n = last - who.y + 1;
  // part s: the first worker's odd slot, then the even slots of the workers after it
  auto slot = [&](int s) { return (int64_t)(2 * (who.y + s) + (s == 0 ? 1 : 0)) * H + h; };
  float mx = -INFINITY;
  for (int s = 0; s < n; ++s) mx = fmaxf(mx, __ldg(o.part_lse + slot(s)));
  float tot = 0.f;
  if (mx != -INFINITY)
    for (int s = 0; s < n; ++s) tot += expf(__ldg(o.part_lse + slot(s)) - mx);
  for (int d = threadIdx.x; d < Dv; d += 128) {
    float acc = 0.f;
    if (tot > 0.f)
      for (int s = 0; s < n; ++s) acc = fmaf(expf(__ldg(o.part_lse + slot(s)) - mx) / tot, __ldg(o.part_o + slot(s) * Dv + d), acc);
    ps_store((T *)o.out + ((int64_t)who.x * H + h) * Dv + d, acc);
  }
  if (o.lse && threadIdx.x == 0) o.lse[(int64_t)who.x * H + h] = tot > 0.f ? mx + logf(tot) : -INFINITY;
}

// ------------------------------------------------------------------------------------------------ host
static size_t pg_al(size_t x) { return (x + 255) / 256 * 256; }

constexpr int kPagedWorkers = 148;                 // sizes the workspace; launches use at most this many

size_t paged_workspace_bytes(int H, int Dv) {
  return kWsHeader + pg_al(kPagedWorkers * sizeof(int2)) + pg_al((size_t)2 * kPagedWorkers * H * 4) +
         pg_al((size_t)2 * kPagedWorkers * H * Dv * 4);
}

static PagedOut paged_out(void *ws, int H, void *out, float *lse) {
  PagedOut o{};
  char *p = (char *)ws;
  o.status = (uint32_t *)p;
  p += kWsHeader;
  o.info = (int2 *)p;
  p += pg_al(kPagedWorkers * sizeof(int2));
  o.part_lse = (float *)p;
  p += pg_al((size_t)2 * kPagedWorkers * H * 4);
  o.part_o = (float *)p;
  o.out = out;
  o.lse = lse;
  return o;
}

template <typename T, int TOK, int NO, bool kShared>
static dsa_status_t simt_launch(const PsArgs &a, int workers, cudaStream_t stream) {
  const int D4 = (a.Dqk + 3) / 4;
  const size_t smem = 4 * ((size_t)kPsHeads * 4 * D4 + (size_t)TOK * ps_stride(a.Dqk) + kPsHeads * TOK +
                           (kShared ? 0 : (size_t)TOK * a.Dv));
  auto *k = paged_simt_kernel<T, TOK, NO, kShared>;
  cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  DSA_LAUNCH_PDL("paged_simt_kernel", k, dim3(workers, (a.H + kPsHeads - 1) / kPsHeads), dim3(kPsThreads), smem, stream, a, 2);
  DSA_LAUNCH_PDL("paged_combine_kernel", paged_combine_kernel<T>, dim3(workers, a.H), dim3(128), 0, stream, a.o, a.H, a.Dv);
  return DSA_OK;
}

dsa_status_t paged_attn_launch(const void *q, bool bf16, const void *kv, const void *v, int H, int Dqk, int Dv,
                               float scale, const int32_t *pages, int kb, const dsa_batch_t *b, void *out, float *lse,
                               void *ws, cudaStream_t stream, int num_sms) {
  PsArgs a{};
  a.q = q;
  a.kv = kv;
  a.v = v;
  a.view = PagedView{b->block_table, b->seq_lens, pages, b->total_q, kb, b->max_blocks_per_seq, b->num_blocks};
  a.o = paged_out(ws, H, out, lse);
  a.H = H;
  a.Dqk = Dqk;
  a.Dv = Dv;
  a.scale = scale;
  const int workers = std::min(num_sms, kPagedWorkers);
  if (bf16) return simt_launch<__nv_bfloat16, 32, 32, true>(a, workers, stream);
  return simt_launch<float, 64, 8, false>(a, workers, stream);
}

}  // namespace dsa
