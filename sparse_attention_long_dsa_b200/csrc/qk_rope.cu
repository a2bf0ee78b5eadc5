// RMS norm and position rotation of query and key rows in one pass.
//
// A part is a tensor of rows x[t, h, 0..D) (queries, latent rows, indexer queries, indexer keys).  For every row t with a
// position p = positions[t] >= 0 and every head h:
//   y = x in fp32;  over [norm_off, norm_off + norm_len):  y_i *= weight_i / sqrt(mean(y^2) + eps)
//   over the rot_len entries from rot_off, with theta_i = p * inv_freq[i], pairs (a, b) = (2i, 2i + 1) or (i, i + rot_len / 2):
//     (y_a, y_b) <- (y_a cos theta_i - y_b sin theta_i,  y_b cos theta_i + y_a sin theta_i)
//   out[slots[t] or t, h, :] = y rounded once to bf16 / f32 / e4m3; e4m3 with a scale: scale = max|y| / 448 (1 when that is
//   0), codes of y / scale, the form dsa_cache_append stores indexer keys in.
// ("Day-0 Adaptation for LLMs: Implementing Sparse Attention and Low-Precision Weights", III.1: FP8 index scoring;
// "Engineering Practices for Day-0 Adaptation of Million-Token Context Models on Domestic AI Chips", Four Key Layers 3: the
// decode step writes the new token into the KV cache.)
//
// Angles: theta in turns, reduced to [-1/2, 1/2] in 64 bits, because at position 10^6 a 32-bit product is off by 0.06
// radians; the sine and cosine of the reduced angle are 32-bit and computed once per (row, i) for all heads of a CTA.
//
// One read and one write of every row: bound by HBM, and for few rows by latency.  A 16,384-row prompt (128 query heads' 64
// rotated entries, latent rows, 64 indexer heads, indexer key; 984 MB) takes 193 us, 5.1 TB/s: the query part moves pieces of
// 128 bytes at strides of 384 and 1,152 (torch's strided copy of them reaches 1.8 TB/s); dense rows of 128 take 6.1 TB/s.  The
// 32 rows of a decode step take 7.9 us.  Four CTAs of 256 threads per SM: 217 us with three.
#include <algorithm>

#include "common.cuh"

namespace dsa {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxParts = 4;
constexpr int kRopeAngles = 1024;          // (row, i) pairs whose sine and cosine a CTA keeps
constexpr int kRopeRows = 64;              // most rows of a CTA
constexpr int kRopeChunks = 4;             // 8-element pieces a lane works on at a time

struct RopePartDev {
  const void *x, *weight;
  void *out;
  float *scale;
  const int64_t *slots;
  int64_t x_row, x_head, o_row, o_head;    // strides in elements
  int64_t out_rows;
  int H, D, norm_off, norm_len, rot_off, rot_len;
  float eps;
  uint8_t x_dt, w_dt, o_dt, halves, x_vec, w_vec, o_vec, lanes;   // *_vec: 16-byte accesses allowed; lanes: per row
  int rows_per_cta, heads_per_cta, head_blocks, cta0, log_gh;
};

struct RopeArgs {
  RopePartDev part[kRopeMaxParts];
  int nparts, T;
  const int32_t *positions;
  const double *inv_freq;
  uint32_t *status;
};

// 8 entries; constant dt and vec leave one branch of these
__device__ __forceinline__ void rope_load8(const void *base, int64_t i, int dt, bool vec, float (&v)[8]) {
  if (dt == DSA_BF16) {
    const uint16_t *p = reinterpret_cast<const uint16_t *>(base) + i;
    uint32_t w[4];
    if (vec) {
      const uint4 u = *reinterpret_cast<const uint4 *>(p);
      w[0] = u.x; w[1] = u.y; w[2] = u.z; w[3] = u.w;
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) w[e] = (uint32_t)p[2 * e] | ((uint32_t)p[2 * e + 1] << 16);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      v[2 * e] = __uint_as_float(w[e] << 16);
      v[2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
    }
  } else {
    const float *p = reinterpret_cast<const float *>(base) + i;
    if (vec) {
      const float4 f = *reinterpret_cast<const float4 *>(p), g = *reinterpret_cast<const float4 *>(p + 4);
      v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
      v[4] = g.x; v[5] = g.y; v[6] = g.z; v[7] = g.w;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = p[e];
    }
  }
}

__device__ __forceinline__ void rope_store8(void *base, int64_t i, int dt, bool vec, const float (&v)[8]) {
  if (dt == DSA_BF16) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
      w[e] = *reinterpret_cast<const uint32_t *>(&b);
    }
    uint16_t *p = reinterpret_cast<uint16_t *>(base) + i;
    if (vec) {
      *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        p[2 * e] = (uint16_t)w[e];
        p[2 * e + 1] = (uint16_t)(w[e] >> 16);
      }
    }
  } else if (dt == DSA_F32) {
    float *p = reinterpret_cast<float *>(base) + i;
    if (vec) {
      *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4 *>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) p[e] = v[e];
    }
  } else {
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < 4; ++e)
      w[e >> 1] |= (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(v[2 * e], v[2 * e + 1]), __NV_SATFINITE, __NV_E4M3)
                   << (16 * (e & 1));
    uint8_t *p = reinterpret_cast<uint8_t *>(base) + i;
    if (vec) {
      *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) p[e] = (uint8_t)(w[e >> 2] >> (8 * (e & 3)));
    }
  }
}

// G lanes work on a row of a head, NI rows at a time.  A lane holds NR pieces of 8 entries, two and two: the pieces that
// rotate with one another in the "halves" order, rot_len / 2 entries apart, fall to the same lane, and the pieces outside the
// rotated range fill up.  So no order of pairs needs another lane, and a warp's loads still cover whole rows.
// Groups of G lanes stand in a grid of gr rows x gh heads (gh a power of two).
struct RopeTables {
  float2 turn[kRopeAngles];                // cosine, sine of (row, i)
  int64_t dst[kRopeRows];                  // output row, -1: skipped
};

// what the heads of a CTA's rows share; every thread calls it, after its first loads are under way
__device__ __forceinline__ void rope_tables(const RopeArgs &a, const RopePartDev &p, int row0, int rows, RopeTables &tab) {
  for (int r = threadIdx.x; r < rows; r += kRopeThreads) {
    const int t = row0 + r;
    int64_t d = -1;
    if (!a.positions || __ldg(a.positions + t) >= 0) {
      d = p.slots ? __ldg(p.slots + t) : t;
      if (d >= p.out_rows) {
        set_status(a.status, kStatusBadIndex);
        d = -1;
      }
    }
    tab.dst[r] = d;
  }
  const int half = p.rot_len / 2;
  for (int i = threadIdx.x; i < rows * half; i += kRopeThreads) {
    const int r = i / half;
    double turns = (double)__ldg(a.positions + row0 + r) * (__ldg(a.inv_freq + (i - r * half)) * 0.15915494309189535);
    turns -= rint(turns);
    float s, c;
    sincospif(2.f * (float)turns, &s, &c);
    tab.turn[i] = make_float2(c, s);
  }
  __syncthreads();
}

// XT, OT: types of x and out, all accesses 16 bytes wide; -1: whatever the part says.
template <int G, int NR, int XT, int OT>
__device__ __forceinline__ void rope_rows(const RopeArgs &a, const RopePartDev &p, int row0, int rows, int head0, int heads,
                                          RopeTables &tab) {
  constexpr int NI = kRopeChunks / NR, kGroups = kRopeThreads / G;
  const int lane = threadIdx.x % G, group = threadIdx.x / G;
  const int gh = 1 << p.log_gh, gr = kGroups >> p.log_gh, h_first = group & (gh - 1), r_first = group >> p.log_gh;
  const int half = p.rot_len / 2;
  const int n0 = p.norm_off / 8, n1 = n0 + p.norm_len / 8, r0 = p.rot_off / 8, np = half / 8;
  const int singles = p.D / 8 - 2 * np, sh = (singles + 1) / 2;
  int piece[NR];                           // -1: none
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    const int d = (r / 2) * G + lane;      // the lane's pair of pieces
    if (d < np) {
      piece[r] = r0 + d + (r & 1) * np;
    } else {
      const int s = d - np + (r & 1) * sh;
      const bool ok = d - np < sh && s < singles;
      piece[r] = ok ? (s < r0 ? s : s + 2 * np) : -1;
    }
  }
  // a lane's heads are the same in every row (heads <= gh * NI)
  int64_t x_off[NI], o_off[NI];
  bool has[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int h = i * gh + h_first;
    has[i] = h < heads;
    x_off[i] = (int64_t)(head0 + h) * p.x_head;
    o_off[i] = (int64_t)(head0 + h) * p.o_head;
  }
  for (int rb = 0; rb < rows; rb += gr) {
    const int row = rb + r_first;
    const int64_t x_row = (int64_t)(row0 + row) * p.x_row;
    float v[NI][NR][8];
#pragma unroll
    for (int i = 0; i < NI; ++i)
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        if (row < rows && has[i] && piece[r] >= 0) {
          rope_load8(p.x, x_row + x_off[i] + 8 * piece[r], XT < 0 ? p.x_dt : XT, XT >= 0 || p.x_vec, v[i][r]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[i][r][e] = 0.f;
        }
      }
    if (rb == 0) rope_tables(a, p, row0, rows, tab);
    const int64_t dst = row < rows ? tab.dst[row] : -1;
    const float2 *tr = tab.turn + row * half;
    if (p.norm_len) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        float ss = 0.f;
#pragma unroll
        for (int r = 0; r < NR; ++r)
          if (piece[r] >= n0 && piece[r] < n1)
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(v[i][r][e], v[i][r][e], ss);
#pragma unroll
        for (int o = G / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float inv = 1.f / sqrtf(ss / (float)p.norm_len + p.eps);
#pragma unroll
        for (int r = 0; r < NR; ++r)
          if (piece[r] >= n0 && piece[r] < n1) {
            float w[8];
            rope_load8(p.weight, 8 * (piece[r] - n0), p.w_dt, p.w_vec, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[i][r][e] *= inv * w[e];
          }
      }
    }
#pragma unroll
    for (int r = 0; r < NR; r += 2) {
      const int d = (r / 2) * G + lane;
      if (d >= np || row >= rows) continue;
      if (p.halves) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 c = tr[8 * d + e];
#pragma unroll
          for (int i = 0; i < NI; ++i) {
            const float x0 = v[i][r][e], x1 = v[i][r + 1][e];
            v[i][r][e] = fmaf(x0, c.x, -x1 * c.y);
            v[i][r + 1][e] = fmaf(x1, c.x, x0 * c.y);
          }
        }
      } else {
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 c = tr[4 * d + q * (half / 2) + e];
#pragma unroll
            for (int i = 0; i < NI; ++i) {
              const float x0 = v[i][r + q][2 * e], x1 = v[i][r + q][2 * e + 1];
              v[i][r + q][2 * e] = fmaf(x0, c.x, -x1 * c.y);
              v[i][r + q][2 * e + 1] = fmaf(x1, c.x, x0 * c.y);
            }
          }
      }
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const bool live = dst >= 0 && has[i];
      if (p.scale) {
        float am = 0.f;
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
          for (int e = 0; e < 8; ++e) am = fmaxf(am, fabsf(v[i][r][e]));
#pragma unroll
        for (int o = G / 2; o; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
        float sc = am / 448.0f;
        if (sc == 0.f) sc = 1.f;
        if (live && lane == 0) p.scale[dst * p.H + head0 + i * gh + h_first] = sc;
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
          for (int e = 0; e < 8; ++e) v[i][r][e] /= sc;
      }
      if (!live) continue;
      const int64_t at = dst * p.o_row + o_off[i];
#pragma unroll
      for (int r = 0; r < NR; ++r)
        if (piece[r] >= 0)
          rope_store8(p.out, at + 8 * piece[r], OT < 0 ? p.o_dt : OT, OT >= 0 || p.o_vec, v[i][r]);
    }
  }
}

template <int XT, int OT>
__device__ __forceinline__ void rope_part_rows(const RopeArgs &a, const RopePartDev &p, int row0, int rows, int head0, int heads,
                                               RopeTables &tab) {
  if (p.lanes == 4) rope_rows<4, 2, XT, OT>(a, p, row0, rows, head0, heads, tab);
  else if (p.lanes == 32) rope_rows<32, 4, XT, OT>(a, p, row0, rows, head0, heads, tab);
  else if (p.D <= 128) rope_rows<8, 2, XT, OT>(a, p, row0, rows, head0, heads, tab);
  else rope_rows<8, 4, XT, OT>(a, p, row0, rows, head0, heads, tab);
}

__global__ void __launch_bounds__(kRopeThreads, 4) qk_rope_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ RopeTables tab;
  int ip = 0;
  while (ip + 1 < a.nparts && (int)blockIdx.x >= a.part[ip + 1].cta0) ++ip;
  const RopePartDev &p = a.part[ip];
  const int blk = (int)blockIdx.x - p.cta0;
  const int row0 = blk / p.head_blocks * p.rows_per_cta, head0 = blk % p.head_blocks * p.heads_per_cta;
  const int rows = min(p.rows_per_cta, a.T - row0), heads = min(p.heads_per_cta, p.H - head0);
  pdl_wait();
  pdl_trigger();
  // Types and alignment resolved once per CTA for the common ones: tested at every access they cost 169 instructions per 8
  // entries and a 16k-row prompt 303 us.  4,096 rows of 32 heads of 128, normed and half rotated: bf16 to bf16 23 us, to e4m3 22, f32 to
  // f32 30; tested at every access f32 to bf16 26, to e4m3 25, bf16 to f32 33, and views off their 16 bytes 77 - 81.
  const bool wide = p.x_vec && p.o_vec;
  if (wide && p.x_dt == DSA_BF16 && p.o_dt == DSA_BF16) rope_part_rows<DSA_BF16, DSA_BF16>(a, p, row0, rows, head0, heads, tab);
  else if (wide && p.x_dt == DSA_BF16 && p.o_dt == DSA_FP8_E4M3)
    rope_part_rows<DSA_BF16, DSA_FP8_E4M3>(a, p, row0, rows, head0, heads, tab);
  else if (wide && p.x_dt == DSA_F32 && p.o_dt == DSA_F32) rope_part_rows<DSA_F32, DSA_F32>(a, p, row0, rows, head0, heads, tab);
  else rope_part_rows<-1, -1>(a, p, row0, rows, head0, heads, tab);
}

// ------------------------------------------------------------------------------------------------ host
static bool vec_ok(const void *base, int64_t s0, int64_t s1, size_t esz, size_t align) {
  return (uintptr_t)base % align == 0 && s0 * (int64_t)esz % (int64_t)align == 0 && s1 * (int64_t)esz % (int64_t)align == 0;
}
static size_t dt_size(int dt) { return dt == DSA_F32 ? 4 : dt == DSA_BF16 ? 2 : 1; }

dsa_status_t qk_rope_launch(const dsa_rope_part_t *parts, int nparts, const int32_t *positions, int T, const double *inv_freq,
                            void *ws, cudaStream_t stream) {
  RopeArgs a{};
  a.nparts = nparts;
  a.T = T;
  a.positions = positions;
  a.inv_freq = inv_freq;
  a.status = (uint32_t *)ws;
  int64_t ctas = 0;
  for (int i = 0; i < nparts; ++i) {
    const dsa_rope_part_t &s = parts[i];
    RopePartDev &p = a.part[i];
    p.x = s.x;
    p.weight = s.weight;
    p.out = s.out;
    p.scale = s.out_scale;
    p.slots = s.slots;
    p.x_row = s.x_row_stride;
    p.x_head = s.x_head_stride;
    p.o_row = s.out_row_stride;
    p.o_head = s.out_head_stride;
    p.out_rows = s.out_rows;
    p.H = s.H;
    p.D = s.D;
    p.norm_off = s.norm_off;
    p.norm_len = s.norm_len;
    p.rot_off = s.rope_off;
    p.rot_len = s.rope_len;
    p.eps = s.eps;
    p.x_dt = (uint8_t)s.x_dt;
    p.w_dt = (uint8_t)s.w_dt;
    p.o_dt = (uint8_t)s.out_dt;
    p.halves = s.rope_style == DSA_ROPE_HALVES;
    p.x_vec = vec_ok(s.x, p.x_row, s.H > 1 ? p.x_head : 0, dt_size(s.x_dt), 16);
    p.w_vec = (uintptr_t)s.weight % 16 == 0;
    p.o_vec = vec_ok(s.out, p.o_row, s.H > 1 ? p.o_head : 0, dt_size(s.out_dt), s.out_dt == DSA_FP8_E4M3 ? 8 : 16);
    p.lanes = s.D <= 64 ? 4 : s.D <= 256 ? 8 : 32;
    const int groups = kRopeThreads / p.lanes, ni = p.D <= 128 ? 2 : 1;      // a CTA holds groups * ni (row, head) pairs at a time
    p.heads_per_cta = std::min(p.H, groups * ni);
    p.head_blocks = (p.H + p.heads_per_cta - 1) / p.heads_per_cta;
    p.log_gh = 0;
    while ((ni << p.log_gh) < p.heads_per_cta) ++p.log_gh;                   // <= log2(groups)
    // Many rows: several passes per CTA, so that sines and cosines are computed by whole CTAs and not by one warp each.
    const int gr = groups >> p.log_gh;
    const int64_t passes = std::min<int64_t>(8, (int64_t)T * p.head_blocks / ((int64_t)148 * 8 * gr));
    p.rows_per_cta = std::min<int>(kRopeRows, gr * (int)std::max<int64_t>(1, passes));
    if (p.rot_len) p.rows_per_cta = std::min(p.rows_per_cta, kRopeAngles / (p.rot_len / 2));
    p.cta0 = (int)ctas;
    ctas += (int64_t)((T + p.rows_per_cta - 1) / p.rows_per_cta) * p.head_blocks;
    if (ctas > 0x7FFFFFFF) {
      set_error("too many rows and heads for one launch");
      return DSA_ERR_UNSUPPORTED;
    }
  }
  DSA_LAUNCH_PDL("qk_rope_kernel", qk_rope_kernel, dim3((unsigned)ctas), dim3(kRopeThreads), 0, stream, a);
  return DSA_OK;
}

}  // namespace dsa
