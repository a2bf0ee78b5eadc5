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
#include <algorithm>

#include "common.cuh"

namespace dsa {

constexpr int kRopeThreads = 256;
constexpr int kRopeMaxParts = 4;
constexpr int kRopeAngles = 1024;          // (row, i) pairs whose sine and cosine a CTA keeps
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
  uint8_t x_dt, w_dt, o_dt, halves, x_vec, w_vec, o_vec, wide;   // *_vec: 16-byte accesses allowed; wide: 32 lanes per row
  int rows_per_cta, heads_per_cta, head_blocks, cta0;
};

struct RopeArgs {
  RopePartDev part[kRopeMaxParts];
  int nparts, T;
  const int32_t *positions;
  const double *inv_freq;
  uint32_t *status;
};

__device__ __forceinline__ void rope_load8(const void *base, int64_t i, uint8_t dt, bool vec, float (&v)[8]) {
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

__device__ __forceinline__ void rope_store8(void *base, int64_t i, uint8_t dt, bool vec, const float (&v)[8]) {
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

// G lanes work on a row of a head; a lane holds NR pieces of NI rows at a time (NR * NI = kRopeChunks).
template <int G, int NR>
__device__ __forceinline__ void rope_rows(const RopeArgs &a, const RopePartDev &p, int row0, int rows, int head0, int heads,
                                          const float2 *turn, float4 *scratch) {
  constexpr int NI = kRopeChunks / NR, kGroups = kRopeThreads / G;
  const int lane = threadIdx.x % G, group = threadIdx.x / G;
  const int items = rows * heads, D8 = p.D / 8, half = p.rot_len / 2;
  const int n0 = p.norm_off / 8, n1 = n0 + p.norm_len / 8, r0 = p.rot_off / 8, r1 = r0 + p.rot_len / 8;
  float4 *mine = scratch + group * (NI * NR * G * 2);      // [item][low, high half of a piece][piece]
  for (int i0 = 0; i0 < items; i0 += kGroups * NI) {
    float v[NI][NR][8];
    int row[NI], head[NI];
    int64_t dst[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      const int it = i0 + i * kGroups + group;
      dst[i] = -1;
      row[i] = it < items ? it / heads : 0;
      head[i] = head0 + (it < items ? it % heads : 0);
      if (it < items) {
        const int t = row0 + row[i];
        if (!a.positions || __ldg(a.positions + t) >= 0) {
          dst[i] = p.slots ? __ldg(p.slots + t) : t;
          if (dst[i] >= p.out_rows) {
            set_status(a.status, kStatusBadIndex);
            dst[i] = -1;
          }
        }
      }
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const int c = r * G + lane;
        if (dst[i] >= 0 && c < D8) {
          rope_load8(p.x, (int64_t)(row0 + row[i]) * p.x_row + (int64_t)head[i] * p.x_head + 8 * c, p.x_dt, p.x_vec, v[i][r]);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[i][r][e] = 0.f;
        }
      }
    }
    if (p.norm_len) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        float ss = 0.f;
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const int c = r * G + lane;
          if (c >= n0 && c < n1)
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(v[i][r][e], v[i][r][e], ss);
        }
#pragma unroll
        for (int o = G / 2; o; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        const float inv = 1.f / sqrtf(ss / (float)p.norm_len + p.eps);
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const int c = r * G + lane;
          if (c >= n0 && c < n1) {
            float w[8];
            rope_load8(p.weight, 8 * (c - n0), p.w_dt, p.w_vec, w);
#pragma unroll
            for (int e = 0; e < 8; ++e) v[i][r][e] *= inv * w[e];
          }
        }
      }
    }
    if (p.rot_len) {
      if (p.halves) {                      // partners lie rot_len / 2 entries apart, in another lane's piece
        __syncwarp();
#pragma unroll
        for (int i = 0; i < NI; ++i)
#pragma unroll
          for (int r = 0; r < NR; ++r) {
            const int c = r * G + lane;
            if (c >= r0 && c < r1) {
              mine[(2 * i) * (NR * G) + c] = make_float4(v[i][r][0], v[i][r][1], v[i][r][2], v[i][r][3]);
              mine[(2 * i + 1) * (NR * G) + c] = make_float4(v[i][r][4], v[i][r][5], v[i][r][6], v[i][r][7]);
            }
          }
        __syncwarp();
      }
#pragma unroll
      for (int i = 0; i < NI; ++i)
#pragma unroll
        for (int r = 0; r < NR; ++r) {
          const int c = r * G + lane;
          if (c < r0 || c >= r1) continue;
          const int at = 8 * (c - r0);
          const float2 *tr = turn + row[i] * half;
          if (p.halves) {
            const bool low = at < half;
            const int pc = low ? c + half / 8 : c - half / 8;
            const float4 f = mine[(2 * i) * (NR * G) + pc], g = mine[(2 * i + 1) * (NR * G) + pc];
            const float u[8] = {f.x, f.y, f.z, f.w, g.x, g.y, g.z, g.w};
            const float2 *t2 = tr + (low ? at : at - half);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float2 cs = t2[e];
              v[i][r][e] = fmaf(v[i][r][e], cs.x, low ? -u[e] * cs.y : u[e] * cs.y);
            }
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 cs = tr[at / 2 + e];
              const float x0 = v[i][r][2 * e], x1 = v[i][r][2 * e + 1];
              v[i][r][2 * e] = fmaf(x0, cs.x, -x1 * cs.y);
              v[i][r][2 * e + 1] = fmaf(x1, cs.x, x0 * cs.y);
            }
          }
        }
    }
    if (p.scale) {
#pragma unroll
      for (int i = 0; i < NI; ++i) {
        float am = 0.f;
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
          for (int e = 0; e < 8; ++e) am = fmaxf(am, fabsf(v[i][r][e]));
#pragma unroll
        for (int o = G / 2; o; o >>= 1) am = fmaxf(am, __shfl_xor_sync(0xffffffffu, am, o));
        float sc = am / 448.0f;
        if (sc == 0.f) sc = 1.f;
        if (dst[i] >= 0 && lane == 0) p.scale[dst[i] * p.H + head[i]] = sc;
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
          for (int e = 0; e < 8; ++e) v[i][r][e] /= sc;
      }
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) {
      if (dst[i] < 0) continue;
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        const int c = r * G + lane;
        if (c < D8) rope_store8(p.out, dst[i] * p.o_row + (int64_t)head[i] * p.o_head + 8 * c, p.o_dt, p.o_vec, v[i][r]);
      }
    }
  }
}

__global__ void __launch_bounds__(kRopeThreads) qk_rope_kernel(const __grid_constant__ RopeArgs a) {
  __shared__ float2 turn[kRopeAngles];
  __shared__ float4 scratch[kRopeThreads * kRopeChunks * 2];
  int ip = 0;
  while (ip + 1 < a.nparts && (int)blockIdx.x >= a.part[ip + 1].cta0) ++ip;
  const RopePartDev &p = a.part[ip];
  const int blk = (int)blockIdx.x - p.cta0;
  const int row0 = blk / p.head_blocks * p.rows_per_cta, head0 = blk % p.head_blocks * p.heads_per_cta;
  const int rows = min(p.rows_per_cta, a.T - row0), heads = min(p.heads_per_cta, p.H - head0);
  pdl_wait();
  pdl_trigger();
  if (p.rot_len) {
    const int half = p.rot_len / 2;
    for (int i = threadIdx.x; i < rows * half; i += kRopeThreads) {
      const int t = __ldg(a.positions + row0 + i / half);
      double turns = (double)t * (__ldg(a.inv_freq + i % half) * 0.15915494309189535);
      turns -= rint(turns);
      float s, c;
      sincospif(2.f * (float)turns, &s, &c);
      turn[i] = make_float2(c, s);
    }
    __syncthreads();
  }
  if (p.wide) rope_rows<32, 4>(a, p, row0, rows, head0, heads, turn, scratch);
  else if (p.D <= 64) rope_rows<8, 1>(a, p, row0, rows, head0, heads, turn, scratch);
  else if (p.D <= 128) rope_rows<8, 2>(a, p, row0, rows, head0, heads, turn, scratch);
  else rope_rows<8, 4>(a, p, row0, rows, head0, heads, turn, scratch);
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
    p.wide = s.D > 256;
    const int groups = kRopeThreads / (p.wide ? 32 : 8);
    const int at_once = groups * (p.D <= 64 ? 4 : p.D <= 128 ? 2 : 1);
    p.heads_per_cta = std::min(p.H, at_once);
    p.head_blocks = (p.H + p.heads_per_cta - 1) / p.heads_per_cta;
    p.rows_per_cta = std::max(1, at_once / p.heads_per_cta);
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
