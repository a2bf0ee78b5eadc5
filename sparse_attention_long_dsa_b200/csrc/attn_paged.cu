// One-token attention over the paged cache: the f32 path on CUDA cores, the join of split rows, and the choice of path.
//
//   z[h, s] = scale * q[h, :] . K[s],   out[h, :] = sum_s softmax_s(z[h, :]) V[s],   lse[h] = log sum_s exp(z[h, s])
// over every cached token s of the row's sequence, or over the tokens of the pages in the row's list ("Engineering
// Practices for Day-0 Adaptation of Million-Token Context Models on Domestic AI Chips", Four Key Layers 3: the decode
// unit walks the KV blocks and the partial results are merged by a cross-block reduction).
//
// The f32 path: a CTA takes a range of page slots (paged.cuh) and its 8 or 12 warps take batches of 8 to 32 tokens of it in turn.
// LT lanes stand over a token's entries, four each, so keys and values go from HBM to registers in whole rows, eight keys and
// eight values per lane in flight; a lane holds its four entries of every head's q and output.  The partial dot products of
// HP heads are summed over the LT lanes by halving exchanges (each step halves the values a lane carries: HP - 1 shuffles
// instead of HP log2(LT)), which leaves each (token, head) in one lane for the softmax; the weights come back through a
// warp's own shared memory.  Warps are joined at the end of a segment, in their order.  Tokens past the sequence are not
// loaded: what the cache holds there may be anything.
// Bound by the issue of loads, FMAs and shuffles from two or three warps per scheduler (q, output, keys and values of a batch take most
// of the registers).  16 rows of 256 - 8,192 tokens (61,000 in all, 31 MB at 4 heads of 64): 12 us, the bytes alone 4.8 us;
// 16 heads of 64: 23 us, 16 heads of 128 (64 MB): 34 us; lists of 32 pages, 16 rows, 4 heads of 64 (17 MB): 10 us; one row of 131,072 tokens, 4 heads of 64: 20 us (67 MB, 3.3 TB/s).
// Two CTAs per SM with half the registers, and the next batch's keys loaded a batch ahead, were both slower.
#include <algorithm>

#include "paged.cuh"

namespace dsa {

dsa_status_t paged_mla_launch(const void *q, const void *kv, int H, float softmax_scale, const PagedView &view,
                              const PagedOut &o, int max_workers, cudaStream_t stream, int num_sms, int *workers);

constexpr int kPsSteps = 8;                        // keys (and values) of a lane in flight

struct PsArgs {
  const float *q, *kv, *v;
  PagedView view;
  PagedOut o;
  int H, Dqk, Dv;
  float scale_log2;
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

// entries d .. d + 3 of a row of D
__device__ __forceinline__ float4 ps_load4(const float *row, int d, int D, bool vec) {
  if (vec) return d < D ? __ldg(reinterpret_cast<const float4 *>(row + d)) : make_float4(0.f, 0.f, 0.f, 0.f);
  return make_float4(d < D ? __ldg(row + d) : 0.f, d + 1 < D ? __ldg(row + d + 1) : 0.f, d + 2 < D ? __ldg(row + d + 2) : 0.f,
                     d + 3 < D ? __ldg(row + d + 3) : 0.f);
}

// z[0..HP) summed over the LT lanes of a token: z[0..HV) of a lane are heads first .. first + HV - 1 afterwards
template <int LT, int HP>
__device__ __forceinline__ void ps_reduce(float (&z)[HP], int lane) {
  int n = HP;
#pragma unroll
  for (int bit = LT / 2; bit; bit >>= 1) {
    if (n > 1) {
      n /= 2;
      const bool up = lane & bit;
#pragma unroll
      for (int i = 0; i < HP / 2; ++i)
        if (i < n) {
          const float send = up ? z[i] : z[i + n], keep = up ? z[i + n] : z[i];
          z[i] = keep + __shfl_xor_sync(0xffffffffu, send, bit);
        }
    } else {
      z[0] += __shfl_xor_sync(0xffffffffu, z[0], bit);
    }
  }
}

template <int LT, int HP, int NW>
struct PsSmem {
  static constexpr int kTok = 32 / LT * kPsSteps;  // tokens of a batch
  float p[NW][kTok][HP];
  float alpha[NW][HP], m[NW][HP], l[NW][HP];
  float o[NW][HP][4 * LT];
  uint32_t tmp[33];
  PagedPlan plan;
};

template <int LT, int HP, int NW>
__global__ void __launch_bounds__(32 * NW) paged_simt_kernel(const PsArgs a) {
  using Smem = PsSmem<LT, HP, NW>;
  constexpr int TW = 32 / LT, kTok = Smem::kTok, HV = HP > LT ? HP / LT : 1;
  extern __shared__ float4 sm4[];
  Smem &S = *reinterpret_cast<Smem *>(sm4);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int worker = blockIdx.x, H = a.H, Dqk = a.Dqk, Dv = a.Dv;
  const bool vk = (Dqk & 3) == 0, vv = (Dv & 3) == 0, whole = Dqk == 4 * LT && Dv == 4 * LT;
  const int tg = lane / LT, d0 = 4 * (lane % LT);
  int first = 0;                                   // this lane's first head after ps_reduce
  {
    int n = HP;
#pragma unroll
    for (int bit = LT / 2; bit; bit >>= 1)
      if (n > 1) {
        n /= 2;
        if (lane & bit) first += n;
      }
  }
  pdl_wait();
  pdl_trigger();
  // One row of 8 pages: 7.3 us with a page per worker, 9.0 with two.  More rows than workers, whole against cut anywhere; the wider the
  // rows, the more pages of waiting a cut is worth less than.  16 heads of 128: 220 rows of 3 pages 36.9 us, 40.6 cut, but 149 of 8 66.4,
  // 47.6, and one of 8 beside 150 of one 34.3, 24.7; of 64: 26.7, 32.5; 39.1, 31.8; 20.9, 21.4; 13 of 32: 18.6, 26.4; 25.1, 24.3; 17.6, 19.7.
  plan_pages(a.view, worker, gridDim.x, PagedRule{1, 1, 8, LT <= 16 ? 7 : 4, LT == 8 ? 7.f : LT == 16 ? 5.f : 2.f}, S.tmp, &S.plan);
  if (tid == 0) a.o.info[worker] = worker_info(a.view, S.plan);

  SegmentWalk walk(S.plan);
  int row, sa, sb, part;
  while (walk.next(a.view, S.plan, worker, &row, &sa, &sb, &part)) {
    const int n = row_tokens(a.view, row, a.o.status);
    float4 q[HP], o[HP];
#pragma unroll
    for (int h = 0; h < HP; ++h) {
      q[h] = h < H ? ps_load4(a.q + ((int64_t)row * H + h) * Dqk, d0, Dqk, vk) : make_float4(0.f, 0.f, 0.f, 0.f);
      q[h].x *= a.scale_log2;
      q[h].y *= a.scale_log2;
      q[h].z *= a.scale_log2;
      q[h].w *= a.scale_log2;
      o[h] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float m[HV], l[HV];
#pragma unroll
    for (int i = 0; i < HV; ++i) {
      m[i] = -INFINITY;
      l[i] = 0.f;
    }
    constexpr int kPer = kPage / kTok;             // batches of a page
    for (int u = sa * kPer + warp; u < sb * kPer; u += NW) {
      int blk = 0;
      const int t0 = (u % kPer) * kTok, ntok = slot_tokens(a.view, row, n, u / kPer, &blk, a.o.status) - t0;
      if (ntok <= 0) continue;                     // the same for the whole warp
      const float *kr = a.kv + ((int64_t)blk * kPage + t0) * Dqk, *vr = a.v + ((int64_t)blk * kPage + t0) * Dv;
      float4 k[kPsSteps], v[kPsSteps];
      if (ntok >= kTok && whole) {                 // every lane has four entries of every token
        const float *kp = kr + tg * Dqk + d0, *vp = vr + tg * Dv + d0;
#pragma unroll
        for (int s = 0; s < kPsSteps; ++s) {
          k[s] = __ldg(reinterpret_cast<const float4 *>(kp + s * TW * Dqk));
          v[s] = __ldg(reinterpret_cast<const float4 *>(vp + s * TW * Dv));
        }
      } else {
#pragma unroll
        for (int s = 0; s < kPsSteps; ++s) {
          const int t = s * TW + tg;
          k[s] = v[s] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (t < ntok) {
            k[s] = ps_load4(kr + t * Dqk, d0, Dqk, vk);
            v[s] = ps_load4(vr + t * Dv, d0, Dv, vv);
          }
        }
      }
      float z[kPsSteps][HV], mx[HV];
#pragma unroll
      for (int i = 0; i < HV; ++i) mx[i] = -INFINITY;
#pragma unroll
      for (int s = 0; s < kPsSteps; ++s) {
        float d[HP];
#pragma unroll
        for (int h = 0; h < HP; ++h)
          d[h] = fmaf(q[h].x, k[s].x, fmaf(q[h].y, k[s].y, fmaf(q[h].z, k[s].z, q[h].w * k[s].w)));
        ps_reduce<LT, HP>(d, lane);
#pragma unroll
        for (int i = 0; i < HV; ++i) {
          z[s][i] = d[i];
          if (s * TW + tg >= ntok) z[s][i] = -INFINITY;
          mx[i] = fmaxf(mx[i], z[s][i]);
        }
      }
      bool moved = false;
      float alpha[HV];
#pragma unroll
      for (int i = 0; i < HV; ++i) {
#pragma unroll
        for (int bit = LT; bit < 32; bit <<= 1) mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], bit));
        const float mn = fmaxf(m[i], mx[i]), use = mn == -INFINITY ? 0.f : mn;
        alpha[i] = exp2f(m[i] - use);
        moved |= mn != m[i];
        m[i] = mn;
        float ls = 0.f;
#pragma unroll
        for (int s = 0; s < kPsSteps; ++s) {
          const float p = exp2f(z[s][i] - use);
          S.p[warp][s * TW + tg][first + i] = p;
          ls += p;
        }
#pragma unroll
        for (int bit = LT; bit < 32; bit <<= 1) ls += __shfl_xor_sync(0xffffffffu, ls, bit);
        l[i] = l[i] * alpha[i] + ls;
        S.alpha[warp][first + i] = alpha[i];
      }
      moved = __any_sync(0xffffffffu, moved);
      __syncwarp();
      if (moved) {
#pragma unroll
        for (int h = 0; h < HP; ++h) {
          const float al = S.alpha[warp][h];
          o[h].x *= al;
          o[h].y *= al;
          o[h].z *= al;
          o[h].w *= al;
        }
      }
#pragma unroll
      for (int s = 0; s < kPsSteps; ++s) {
        const float4 *pr = reinterpret_cast<const float4 *>(S.p[warp][s * TW + tg]);
#pragma unroll
        for (int h4 = 0; h4 < HP / 4; ++h4) {
          const float4 p4 = pr[h4];
          const float ph[4] = {p4.x, p4.y, p4.z, p4.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float4 &oh = o[4 * h4 + e];
            oh.x = fmaf(ph[e], v[s].x, oh.x);
            oh.y = fmaf(ph[e], v[s].y, oh.y);
            oh.z = fmaf(ph[e], v[s].z, oh.z);
            oh.w = fmaf(ph[e], v[s].w, oh.w);
          }
        }
      }
      __syncwarp();
    }
    // join the warps, in their order
#pragma unroll
    for (int h = 0; h < HP; ++h) {
#pragma unroll
      for (int bit = LT; bit < 32; bit <<= 1) {
        o[h].x += __shfl_xor_sync(0xffffffffu, o[h].x, bit);
        o[h].y += __shfl_xor_sync(0xffffffffu, o[h].y, bit);
        o[h].z += __shfl_xor_sync(0xffffffffu, o[h].z, bit);
        o[h].w += __shfl_xor_sync(0xffffffffu, o[h].w, bit);
      }
      if (tg == 0) *reinterpret_cast<float4 *>(&S.o[warp][h][d0]) = o[h];
    }
#pragma unroll
    for (int i = 0; i < HV; ++i) {
      S.m[warp][first + i] = m[i];
      S.l[warp][first + i] = l[i];
    }
    __syncthreads();
    for (int i = tid; i < H * Dv; i += 32 * NW) {
      const int h = i / Dv, d = i - h * Dv;
      float M = -INFINITY, L = 0.f, acc = 0.f;
#pragma unroll
      for (int w = 0; w < NW; ++w) M = fmaxf(M, S.m[w][h]);
      const float use = M == -INFINITY ? 0.f : M;
#pragma unroll
      for (int w = 0; w < NW; ++w) {
        const float e = exp2f(S.m[w][h] - use);
        L = fmaf(e, S.l[w][h], L);
        acc = fmaf(e, S.o[w][h][d], acc);
      }
      const float val = L != 0.f ? acc / L : 0.f;
      if (part < 0) ((float *)a.o.out)[((int64_t)row * H + h) * Dv + d] = val;
      else a.o.part_o[((int64_t)part * H + h) * Dv + d] = val;
      if (d == 0) {
        const float lse = L != 0.f ? (M + log2f(L)) * 0.69314718055994531f : -INFINITY;
        if (part >= 0) a.o.part_lse[(int64_t)part * H + h] = lse;
        else if (a.o.lse) a.o.lse[(int64_t)row * H + h] = lse;
      }
    }
    __syncthreads();
  }
  zero_empty_rows<float>(a.view, a.o, H, Dv, (int64_t)blockIdx.x * NW + warp, (int64_t)gridDim.x * NW);
}

// ------------------------------------------------------------------------------------------------ join
// out[row, h, :] = sum_w exp(lse_w - lse) o_w,  lse = log sum_w exp(lse_w)  over the workers w that hold a part of the row.
// At most min(T, workers) rows are split, and CTA x finds the x-th of them in info; a warp takes a head (kGroup = 1) or every
// kGroup-th part of one (the sums of the kGroup warps are added in a fixed order).  A lane holds kN pieces of the row (four
// values each where Dv % 4 == 0, else single ones).  Bound by latency, so it is the number of warps in flight that counts.
// Few rows have many parts each: with eight warps per head a 1M-token row (74 parts of 128 heads) takes 8 us, part after part
// 90 us.  Many rows have few: the 32-row decode batch (3.3 parts each) takes 5 us with a warp per head, 28 us with sixteen.
// The bf16 forms of several warps per head spill 28 bytes at four CTAs per SM.
constexpr int kPcThreads = 256, kPcWarps = kPcThreads / 32;

// kBlocks: workers / 32, rounded up.  Four CTAs per SM, so that the decode batch's 4,096 warps run in one wave.
template <typename T, int kGroup, int kN, bool kVec, int kBlocks>
__global__ void __launch_bounds__(kPcThreads, 4) paged_combine_kernel(const PagedOut o, int workers, int H, int Dv) {
  constexpr int kLane = kVec ? 4 : 1;
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
    auto load = [&](int s, float (&v)[kN * kLane]) {
      const float *p = o.part_o + slot(s) * Dv;
#pragma unroll
      for (int k = 0; k < kN; ++k) {
        const int d = (32 * k + lane) * kLane;
        if (kVec) {
          const float4 f = d < Dv ? __ldg(reinterpret_cast<const float4 *>(p + d)) : make_float4(0.f, 0.f, 0.f, 0.f);
          v[kLane * k] = f.x;
          v[kLane * k + kLane / 4] = f.y;
          v[kLane * k + kLane / 2] = f.z;
          v[kLane * k + kLane - 1] = f.w;
        } else {
          v[k] = d < Dv ? __ldg(p + d) : 0.f;
        }
      }
    };
    // the first parts' values are on their way while the weights are worked out
    constexpr int kAhead = kN * kLane <= 4 ? 8 : 2;
    float v[kAhead][kN * kLane];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (sub + j * kGroup < n) load(sub + j * kGroup, v[j]);
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
      w[i] = w[i] == -INFINITY ? 0.f : expf(w[i] - mx);        // a part that is NaN makes its row NaN
      tot += w[i];
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) tot += __shfl_xor_sync(0xffffffffu, tot, off);
    const float inv = tot != 0.f ? 1.f / tot : 0.f;
    lse = tot != 0.f ? mx + logf(tot) : -INFINITY;
    for (int s0 = sub; s0 < n; s0 += kAhead * kGroup) {
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int s = s0 + j * kGroup;             // the same for the whole warp
        if (s >= n) break;
        float ws = 0.f;
#pragma unroll
        for (int i = 0; i < kBlocks; ++i)
          if (s / 32 == i) ws = w[i];
        ws = __shfl_sync(0xffffffffu, ws, s & 31) * inv;
#pragma unroll
        for (int k = 0; k < kN * kLane; ++k) acc[k] = fmaf(ws, v[j][k], acc[k]);
        if (s + kAhead * kGroup < n) load(s + kAhead * kGroup, v[j]);
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

template <typename T, int kN, bool kVec, int kBlocks>
static dsa_status_t combine_launch(const PagedOut &o, int workers, int T_rows, int H, int Dv, cudaStream_t stream) {
  const int rows = std::min(workers, T_rows);
  auto go = [&](auto *kernel, int group) -> dsa_status_t {
    const int heads = kPcWarps / group;
    DSA_LAUNCH_PDL("paged_combine_kernel", kernel, dim3(rows, (H + heads - 1) / heads), dim3(kPcThreads), 0, stream, o, workers, H,
                   Dv);
    return DSA_OK;
  };
  // as many warps per (row, head) as run in one wave, 32 per SM (8 rows of 2,048 tokens, 128 heads: the whole call 18.9 us with
  // four warps, 20.6 with one)
  const int64_t pairs = (int64_t)rows * H, wave = 148 * 32;
  if (8 * pairs <= wave) return go(paged_combine_kernel<T, 8, kN, kVec, kBlocks>, 8);
  if (4 * pairs <= wave) return go(paged_combine_kernel<T, 4, kN, kVec, kBlocks>, 4);
  if (2 * pairs <= wave) return go(paged_combine_kernel<T, 2, kN, kVec, kBlocks>, 2);
  return go(paged_combine_kernel<T, 1, kN, kVec, kBlocks>, 1);
}

// ------------------------------------------------------------------------------------------------ host
static size_t pg_al(size_t x) { return (x + 255) / 256 * 256; }

// The most workers a launch uses; they size the workspace.  Value width tells the two paths apart: 512 is the latent
// cache's (CTA pairs of a B200's 148 SMs), up to 128 the f32 path's.
constexpr int kPagedPairs = 74, kPagedCtas = 148;
static int paged_max_workers(int Dv) { return Dv > 128 ? kPagedPairs : kPagedCtas; }

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

template <int LT, int HP, int NW>
static dsa_status_t simt_launch(const PsArgs &a, int workers, cudaStream_t stream) {
  auto *k = paged_simt_kernel<LT, HP, NW>;
  constexpr size_t smem = sizeof(PsSmem<LT, HP, NW>);
  if (smem > 48 * 1024 && cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) {
    set_error("paged_simt_kernel: %s", cudaGetErrorString(cudaGetLastError()));
    return DSA_ERR_CUDA;
  }
  DSA_LAUNCH_PDL("paged_simt_kernel", k, dim3(workers), dim3(32 * NW), smem, stream, a);
  return DSA_OK;
}
// 8 warps of up to 255 registers.  Up to 4 heads 128 are enough, so 12 warps run where every CTA has rows of its own: 256 rows of 8 -
// 13 pages 24.7 us, 32.2 with 8 warps, 180 of 11 - 24 pages, 128 entries wide 46.7, 60.8; but one row of 2 pages 7.3, 6.8, one of
// 131,072 tokens 22.5, 19.6.
template <int LT>
static dsa_status_t simt_heads(const PsArgs &a, int workers, cudaStream_t stream) {
  if (a.H <= 4 && a.view.T > workers) return simt_launch<LT, 4, 12>(a, workers, stream);
  if (a.H <= 4) return simt_launch<LT, 4, 8>(a, workers, stream);
  if (a.H <= 8) return simt_launch<LT, 8, 8>(a, workers, stream);
  return simt_launch<LT, 16, 8>(a, workers, stream);
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
  a.scale_log2 = scale * 1.4426950408889634f;
  if (bf16) {
    int workers = 0;
    const dsa_status_t st = paged_mla_launch(q, kv, H, scale, a.view, a.o, paged_max_workers(Dv), stream, num_sms, &workers);
    if (st != DSA_OK) return st;
    return combine_launch<__nv_bfloat16, 4, true, (kPagedPairs + 31) / 32>(a.o, workers, b->total_q, H, Dv, stream);
  }
  const int workers = std::min(num_sms, paged_max_workers(Dv));
  // the fewest lanes that cover a row with four entries each, the fewest heads in steps of 4, 8, 16
  const int D = std::max(Dqk, Dv);
  dsa_status_t st;
  if (D <= 32) st = simt_heads<8>(a, workers, stream);
  else if (D <= 64) st = simt_heads<16>(a, workers, stream);
  else st = simt_heads<32>(a, workers, stream);
  if (st != DSA_OK) return st;
  if (Dv % 4 == 0) return combine_launch<float, 1, true, (kPagedCtas + 31) / 32>(a.o, workers, b->total_q, H, Dv, stream);
  return combine_launch<float, 4, false, (kPagedCtas + 31) / 32>(a.o, workers, b->total_q, H, Dv, stream);
}

}  // namespace dsa
