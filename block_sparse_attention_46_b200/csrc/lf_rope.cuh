// lf_rope.cuh — rotary positions with three axes (time, height, width) on the frames of a
// chunk or of the key cache, with the RMS norm that precedes them, and their gradient.
//
// Per token: xn = x * r, r = 1 / sqrt(mean(x^2) + eps) over each head's d channels or over
// the token's H * d; y = R(theta) (w * xn), R turning channel pair p by
// theta_p = (position on p's axis) * base^(-i / n_axis), i the pair's index on its axis.
// Gradient: g = R(-theta) dy; dw = sum over tokens of g * xn (and over heads for the
// per-head weight); dx = r * (w g - xn * mean(w g xn)), the mean over the norm's channels.
//
// Everything is bound by HBM: 4 bytes per element forward, 6 backward with a norm.  A token
// is held in the registers of `tpt` threads (4 to 32 lanes of a warp, or several warps for
// wide tokens), 16 channels (two 16-byte loads) per unit and up to kRopeUnits units per
// thread, so x is read once although the norm needs a sum over it first.  A unit holds whole
// pairs: 16 adjacent channels, or 8 from each half of the head.  Each token's d / 2 angles
// are computed once by its threads and shared: position * frequency in turns in 64 bits,
// reduced to [-1/2, 1/2] there, then sine and cosine in 32 bits, so the angle's error does
// not grow with the position (a 32-bit product would be off by 2^-24 of it).
#pragma once
#include "lf_common.cuh"

namespace lf {

constexpr int kRopeMaxPairs = 64;            // d / 2
constexpr int kRopeUnits = 3;                // 16-channel units per thread, at most
constexpr int kRopeThreads = 256;            // per CTA, at most; a token's threads are in one CTA
static_assert(kRopeUnits * 16 * kRopeThreads == LF_MAX_ROPE_CHANNELS, "the widest token");
constexpr int kRopeBwdCtas = 296;            // backward with a norm: CTAs (partial sums of dw), at most

struct RopeHead {
  const __nv_bfloat16* x;      // rows of H * d channels, x_stride elements apart
  const __nv_bfloat16* dout;   // backward
  const float* weight;         // [d] (norm per head), [H * d] (per token) or null
  __nv_bfloat16* out;          // forward: y; backward: dx
  float* part;                 // backward: [CTAs, d or H * d] partial sums of dw
  int64_t x_stride, dout_stride, out_stride;
  int64_t n_tokens;
  int H, d, T, width;
  int units;                   // H * d / 16
  int tpt, groups;             // threads per token, tokens per CTA at a time
  int upd;                     // units per head, d / 16
  int norm, halves;
  int p_t, p_h, p_w;           // ends of the three axes' pairs; pairs from p_w on are not turned
  float eps, inv_n, sign;      // sign: +1 turns by theta, -1 by -theta
  double turns[kRopeMaxPairs];             // frequency / 2 pi
};

// Frames by value: up to kRopeFewFrames in 1.2 KB of kernel arguments, up to LF_MAX_FRAMES in
// 4.7 KB, which cost a launch about 2 us more.
constexpr int kRopeFewFrames = 32;

template <int NF>
struct RopeArgs : RopeHead {
  int32_t pos[NF], x_slot[NF], dout_slot[NF], out_slot[NF];
};

// A unit's 16 channels as 32-bit values: pairs (v[2j], v[2j + 1]) when adjacent,
// (v[j], v[8 + j]) when split in halves.
__device__ __forceinline__ void rope_unpack(const uint4& a, const uint4& b, float* v) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 rope_pack(const float* v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<uint32_t*>(&t);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Turns a unit's eight pairs; cs holds (cos, sin) of the head's pairs, o is the unit's
// index in its head.
__device__ __forceinline__ void rope_turn(float* v, const float2* cs, int o, int halves) {
  const float4* c4 = reinterpret_cast<const float4*>(cs + o * 8);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float4 c = c4[j];
    if (halves) {
      const float a0 = v[2 * j], b0 = v[8 + 2 * j], a1 = v[2 * j + 1], b1 = v[8 + 2 * j + 1];
      v[2 * j] = a0 * c.x - b0 * c.y;
      v[8 + 2 * j] = a0 * c.y + b0 * c.x;
      v[2 * j + 1] = a1 * c.z - b1 * c.w;
      v[8 + 2 * j + 1] = a1 * c.w + b1 * c.z;
    } else {
      const float a0 = v[4 * j], b0 = v[4 * j + 1], a1 = v[4 * j + 2], b1 = v[4 * j + 3];
      v[4 * j] = a0 * c.x - b0 * c.y;
      v[4 * j + 1] = a0 * c.y + b0 * c.x;
      v[4 * j + 2] = a1 * c.z - b1 * c.w;
      v[4 * j + 3] = a1 * c.w + b1 * c.z;
    }
  }
}

// (cos, sin) of every pair of the token at frame f, offset t, by the token's threads.
template <typename Args>
__device__ __forceinline__ void rope_angles(const Args& A, int f, int t, int lane_t, float2* cs) {
  const int row = t / A.width, col = t - row * A.width;
  for (int p = lane_t; p < A.d / 2; p += A.tpt) {
    float2 v = make_float2(1.f, 0.f);
    if (p < A.p_w) {
      const int at = p < A.p_t ? A.pos[f] : p < A.p_h ? row : col;
      double u = (double)at * A.turns[p];
      u -= rint(u);
      float s, c;
      sincospif(2.f * (float)u, &s, &c);
      v = make_float2(c, A.sign * s);
    }
    cs[p] = v;
  }
}

// Sum of v over the lanes of a warp whose index differs in the bits of [lo, hi).
__device__ __forceinline__ float rope_lane_sum(float v, int lo, int hi) {
  for (int o = lo; o < hi; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Sum over a token's threads: lanes, then (wide tokens) its warps in order.  Every thread of
// the CTA calls it.
__device__ __forceinline__ float rope_token_sum(const RopeHead& A, float v, float* s_warp) {
  v = rope_lane_sum(v, 1, A.tpt < 32 ? A.tpt : 32);
  if (A.tpt <= 32) return v;
  const int warp = threadIdx.x >> 5, wpt = A.tpt / 32, first = warp / wpt * wpt;
  __syncthreads();                       // the previous sum has been read
  if ((threadIdx.x & 31) == 0) s_warp[warp] = v;
  __syncthreads();
  float s = 0.f;
  for (int i = 0; i < wpt; ++i) s += s_warp[first + i];
  return s;
}

template <int U, int NF>
__global__ void __launch_bounds__(kRopeThreads)
rope_kernel(const __grid_constant__ RopeArgs<NF> A) {
  extern __shared__ float2 s_cs[];                       // [groups][d / 2], then the warp sums
  float* s_warp = reinterpret_cast<float*>(s_cs + A.groups * (A.d / 2));
  const int grp = threadIdx.x / A.tpt, lane_t = threadIdx.x - grp * A.tpt;
  const int64_t tok = (int64_t)blockIdx.x * A.groups + grp;
  const bool live = tok < A.n_tokens;
  const int f = live ? (int)(tok / A.T) : 0, t = live ? (int)(tok - (int64_t)f * A.T) : 0;
  const int o = lane_t % A.upd;
  const int ca = A.halves ? o * 8 : o * 16, cb = A.halves ? A.d / 2 + o * 8 : o * 16 + 8;
  const __nv_bfloat16* xr = A.x + ((int64_t)A.x_slot[f] * A.T + t) * A.x_stride;
  uint4 a[U], b[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int id = lane_t + u * A.tpt, base = id / A.upd * A.d;
    a[u] = b[u] = make_uint4(0, 0, 0, 0);
    if (live && id < A.units) {
      a[u] = *reinterpret_cast<const uint4*>(xr + base + ca);
      b[u] = *reinterpret_cast<const uint4*>(xr + base + cb);
    }
  }
  float2* cs = s_cs + grp * (A.d / 2);
  if (live) rope_angles(A, f, t, lane_t, cs);
  __syncthreads();
  float v[U][16], r[U];
  float ss = 0.f;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    rope_unpack(a[u], b[u], v[u]);
    r[u] = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) r[u] = fmaf(v[u][i], v[u][i], r[u]);
    ss += r[u];
  }
  if (A.norm == LF_NORM_TOKEN) {
    ss = rsqrtf(rope_token_sum(A, ss, s_warp) * A.inv_n + A.eps);
#pragma unroll
    for (int u = 0; u < U; ++u) r[u] = ss;
  } else if (A.norm == LF_NORM_HEAD) {
#pragma unroll
    for (int u = 0; u < U; ++u) r[u] = rsqrtf(rope_lane_sum(r[u], 1, A.upd) * A.inv_n + A.eps);
  }
  if (!live) return;
  __nv_bfloat16* yr = A.out + ((int64_t)A.out_slot[f] * A.T + t) * A.out_stride;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int id = lane_t + u * A.tpt, base = id / A.upd * A.d;
    if (id >= A.units) break;
    if (A.norm != LF_NORM_NONE) {
      const float* w = A.weight + (A.norm == LF_NORM_TOKEN ? base : 0);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float4 w4 = *reinterpret_cast<const float4*>(w + (q < 2 ? ca : cb) + (q & 1) * 4);
        v[u][4 * q] *= r[u] * w4.x;
        v[u][4 * q + 1] *= r[u] * w4.y;
        v[u][4 * q + 2] *= r[u] * w4.z;
        v[u][4 * q + 3] *= r[u] * w4.w;
      }
    }
    rope_turn(v[u], cs, o, A.halves);
    *reinterpret_cast<uint4*>(yr + base + ca) = rope_pack(v[u]);
    *reinterpret_cast<uint4*>(yr + base + cb) = rope_pack(v[u] + 8);
  }
}

// Gradient with a norm.  Each CTA walks tokens blockIdx.x, + gridDim.x, ... (groups of them)
// in order and keeps its part of dw in registers; the parts of its warps are added in warp
// order, those of the CTAs in CTA order by rope_dweight_kernel, so dw does not depend on
// timing.
template <int U, int NF>
__global__ void __launch_bounds__(kRopeThreads)
rope_bwd_kernel(const __grid_constant__ RopeArgs<NF> A) {
  extern __shared__ float2 s_cs[];
  float* s_warp = reinterpret_cast<float*>(s_cs + A.groups * (A.d / 2));
  float* s_dw = s_warp + 32;                             // [d or H * d]
  const int grp = threadIdx.x / A.tpt, lane_t = threadIdx.x - grp * A.tpt;
  const int o = lane_t % A.upd;
  const int ca = A.halves ? o * 8 : o * 16, cb = A.halves ? A.d / 2 + o * 8 : o * 16 + 8;
  float2* cs = s_cs + grp * (A.d / 2);
  const bool per_token = A.norm == LF_NORM_TOKEN;
  float dw[U][16];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < 16; ++i) dw[u][i] = 0.f;

  const int64_t n_steps = (A.n_tokens + A.groups - 1) / A.groups;
  for (int64_t step = blockIdx.x; step < n_steps; step += gridDim.x) {
    const int64_t tok = step * A.groups + grp;
    const bool live = tok < A.n_tokens;
    const int f = live ? (int)(tok / A.T) : 0, t = live ? (int)(tok - (int64_t)f * A.T) : 0;
    const __nv_bfloat16* xr = A.x + ((int64_t)A.x_slot[f] * A.T + t) * A.x_stride;
    const __nv_bfloat16* gr = A.dout + ((int64_t)A.dout_slot[f] * A.T + t) * A.dout_stride;
    uint4 xa[U], xb[U], ga[U], gb[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int id = lane_t + u * A.tpt, base = id / A.upd * A.d;
      xa[u] = xb[u] = ga[u] = gb[u] = make_uint4(0, 0, 0, 0);
      if (live && id < A.units) {
        xa[u] = *reinterpret_cast<const uint4*>(xr + base + ca);
        xb[u] = *reinterpret_cast<const uint4*>(xr + base + cb);
        ga[u] = *reinterpret_cast<const uint4*>(gr + base + ca);
        gb[u] = *reinterpret_cast<const uint4*>(gr + base + cb);
      }
    }
    __syncthreads();                                     // the previous token's angles were read
    if (live) rope_angles(A, f, t, lane_t, cs);
    __syncthreads();
    float r[U], c[U];
    {
      float ss = 0.f;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float x[16];
        rope_unpack(xa[u], xb[u], x);
        r[u] = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) r[u] = fmaf(x[i], x[i], r[u]);
        ss += r[u];
      }
      if (per_token) {
        ss = rsqrtf(rope_token_sum(A, ss, s_warp) * A.inv_n + A.eps);
#pragma unroll
        for (int u = 0; u < U; ++u) r[u] = ss;
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u)
          r[u] = rsqrtf(rope_lane_sum(r[u], 1, A.upd) * A.inv_n + A.eps);
      }
    }
    // c = mean(w g xn); dw += g xn
    float g[U][16];
    float cc = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int id = lane_t + u * A.tpt, base = id / A.upd * A.d;
      float x[16];
      rope_unpack(xa[u], xb[u], x);
      rope_unpack(ga[u], gb[u], g[u]);
      c[u] = 0.f;
      if (live && id < A.units) {
        rope_turn(g[u], cs, o, A.halves);
        const float* w = A.weight + (per_token ? base : 0);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float4 w4 = *reinterpret_cast<const float4*>(w + (q < 2 ? ca : cb) + (q & 1) * 4);
          const float wv[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int i = 4 * q + k;
            const float gx = g[u][i] * (x[i] * r[u]);
            dw[u][i] += gx;
            c[u] = fmaf(wv[k], gx, c[u]);
            g[u][i] *= wv[k];
          }
        }
      }
      cc += c[u];
    }
    if (per_token) {
      cc = rope_token_sum(A, cc, s_warp) * A.inv_n;
#pragma unroll
      for (int u = 0; u < U; ++u) c[u] = cc;
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) c[u] = rope_lane_sum(c[u], 1, A.upd) * A.inv_n;
    }
    if (live) {
      __nv_bfloat16* dr = A.out + ((int64_t)A.out_slot[f] * A.T + t) * A.out_stride;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int id = lane_t + u * A.tpt, base = id / A.upd * A.d;
        if (id >= A.units) break;
        float x[16];
        rope_unpack(xa[u], xb[u], x);
        const float rc = r[u] * r[u] * c[u];
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = fmaf(r[u], g[u][i], -rc * x[i]);
        *reinterpret_cast<uint4*>(dr + base + ca) = rope_pack(x);
        *reinterpret_cast<uint4*>(dr + base + cb) = rope_pack(x + 8);
      }
    }
  }

  // dw of the CTA: lanes with the same channels, then the warps in order
  const int n_dw = per_token ? A.H * A.d : A.d;
  for (int i = threadIdx.x; i < n_dw; i += blockDim.x) s_dw[i] = 0.f;
  if (!per_token) {
#pragma unroll
    for (int u = 1; u < U; ++u)
#pragma unroll
      for (int i = 0; i < 16; ++i) dw[0][i] += dw[u][i];
  }
  const int same = per_token ? (A.tpt < 32 ? A.tpt : 32) : A.upd;
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < 16; ++i) dw[u][i] = rope_lane_sum(dw[u][i], same, 32);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int w = 0; w < (int)blockDim.x / 32; ++w) {
    __syncthreads();
    if (warp != w || lane >= same) continue;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int id = lane_t + u * A.tpt, base = per_token ? id / A.upd * A.d : 0;
      if (per_token ? id >= A.units : u > 0) break;
#pragma unroll
      for (int i = 0; i < 16; ++i) s_dw[base + (i < 8 ? ca + i : cb + i - 8)] += dw[u][i];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n_dw; i += blockDim.x) A.part[(size_t)blockIdx.x * n_dw + i] = s_dw[i];
}

// dweight[c] = sum of the CTAs' parts, in a fixed order: 32 channels per CTA, 16 threads a
// channel.
__global__ void __launch_bounds__(512)
rope_dweight_kernel(const float* __restrict__ part, int n_part, int n_dw, float* __restrict__ dweight) {
  __shared__ float s[16][33];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), k = threadIdx.x >> 5;
  float v = 0.f;
  if (c < n_dw)
    for (int i = k; i < n_part; i += 16) v += part[(size_t)i * n_dw + c];
  s[k][threadIdx.x & 31] = v;
  __syncthreads();
  if (k == 0 && c < n_dw) {
    for (int i = 1; i < 16; ++i) v += s[i][threadIdx.x];
    dweight[c] = v;
  }
}

}  // namespace lf
