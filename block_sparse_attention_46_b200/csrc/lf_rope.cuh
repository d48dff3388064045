// lf_rope.cuh — rotary positions with three axes (time, height, width) on the frames of a
// chunk or of the key cache, with the RMS norm that precedes them, and their gradient.
//
// Per token: xn = x * r, r = 1 / sqrt(mean(x^2) + eps) over each head's d channels or over
// the token's H * d; y = R(theta) (w * xn), R turning channel pair p by
// theta_p = (position on p's axis) * base^(-i / n_axis), i the pair's index on its axis.
// Gradient: g = R(-theta) dy; dw = sum over tokens of g * xn (and over heads for the
// per-head weight); dx = r * (w g - xn * mean(w g xn)), the mean over the norm's channels.
//
// 4 bytes per element forward, 6 backward with a norm.  Large calls without a norm are bound by
// memory (24 frames of 1560 x 12 x 128: 43-45 us, 0.78-0.82 of the copy rate, gradient 42 us); with
// one, warps wait for sums and weights (into cache slots 60 us, 0.58 of the copy rate, norm per
// head 54; gradient 133 us, 0.40, per head 111).  Small calls: the host's side of the call.  A token
// is held in the registers of `tpt` threads (4 to 32 lanes of a warp, or several warps for
// wide tokens), 16 channels (two 16-byte loads) per unit and up to kRopeUnits units per
// thread, so x is read once although the norm needs a sum over it first.  A unit is 8 channels
// of each half of its head: whole pairs in either pairing, and every load and store of a warp
// covers whole 128-byte lines (as 16 adjacent channels per thread, in two pieces, 24 cached
// frames of 12 x 128 channels took 54 us instead of 43).  Each token's d / 2 angles
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
// Forward, tokens of one unit per thread: with four tokens per thread a long call has more loads
// in flight, a shorter one fewer CTAs than it needs.  By the CTAs of one token per thread, four
// tokens against one: from 2000 to 9000 up to 40 % slower (at best 8 % faster, where a wave just
// fills), 0.95 to 1.03 of the time between 9000 and 16000, from there 0.88 to 1.01, 0.97 for 24
// cached frames.  CTAs of 160 threads (20 heads of 128, 40 of 64) do not gain at any size; one
// head alone has too many tokens per CTA for four times their angles (64 KB).
constexpr int kRopeTokens = 4, kRopeManyCtas = 16000, kRopeManyThreads = 192;
// Backward with a norm: CTAs, each with a partial sum of dw, at most: the two that an SM's
// registers hold, on 148 SMs.  A constant, so that dw's order of additions, and with it its bits,
// and the workspace do not depend on the device.
constexpr int kRopeBwdCtas = 296;

struct RopeHead {
  const __nv_bfloat16* x;      // rows of H * d channels, x_stride elements apart
  const __nv_bfloat16* dout;   // backward
  const float* weight;         // [d] (norm per head), [H * d] (per token) or null
  __nv_bfloat16* out;          // forward: y; backward: dx
  float* part;                 // backward: [CTAs, d or H * d] partial sums of dw
  int64_t x_stride, dout_stride, out_stride;
  int H, d, T, width, n_frames;
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
__device__ __forceinline__ void rope_turn(float* v, const float2* cs, int o, int quarter, int halves) {
  const float4* c4 = reinterpret_cast<const float4*>(cs + o * (halves ? 8 : 4));
  const float4* c4b = reinterpret_cast<const float4*>(cs + (halves ? o * 8 + 4 : quarter + o * 4));
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float4 c = j < 2 ? c4[j] : c4b[j - 2];
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

// A CTA is tpt x groups threads: x within the token, y the group of NT successive tokens, all
// loaded before the first is worked on.  grid.y: frames.
template <int U, int NT, int NF>
__global__ void __launch_bounds__(kRopeThreads)
rope_kernel(const __grid_constant__ RopeArgs<NF> A) {
  extern __shared__ float2 s_cs[];                       // [groups][NT][d / 2], then the warp sums
  float* s_warp = reinterpret_cast<float*>(s_cs + A.groups * NT * (A.d / 2));   // [NT][warps]
  const int grp = threadIdx.y, lane_t = threadIdx.x;
  const int f = blockIdx.y, t0 = (blockIdx.x * A.groups + grp) * NT;
  const int o = lane_t & (A.upd - 1);                    // unit in its head (upd: 4 or 8)
  const int ca = o * 8, cb = A.d / 2 + o * 8;            // the unit's two pieces of its head
  const __nv_bfloat16* xr = A.x + ((int64_t)A.x_slot[f] * A.T + t0) * A.x_stride;
  uint4 a[NT][U], b[NT][U];
#pragma unroll
  for (int k = 0; k < NT; ++k)
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int id = lane_t + u * A.tpt, base = (id - o) * 16;   // 16 * upd = d channels a head
      a[k][u] = b[k][u] = make_uint4(0, 0, 0, 0);
      if (t0 + k < A.T && id < A.units) {
        a[k][u] = *reinterpret_cast<const uint4*>(xr + k * A.x_stride + base + ca);
        b[k][u] = *reinterpret_cast<const uint4*>(xr + k * A.x_stride + base + cb);
      }
    }
  float2* cs = s_cs + grp * NT * (A.d / 2);
  if (A.p_w > 0) {
#pragma unroll
    for (int k = 0; k < NT; ++k)
      if (t0 + k < A.T) rope_angles(A, f, t0 + k, lane_t, cs + k * (A.d / 2));
  }
  float r[NT][U];
  if (A.norm != LF_NORM_NONE) {
#pragma unroll
    for (int k = 0; k < NT; ++k) {
      float ss = 0.f;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float v[16];
        rope_unpack(a[k][u], b[k][u], v);
        r[k][u] = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) r[k][u] = fmaf(v[i], v[i], r[k][u]);
        if (A.norm == LF_NORM_HEAD)
          r[k][u] = rsqrtf(rope_lane_sum(r[k][u], 1, A.upd) * A.inv_n + A.eps);
        ss += r[k][u];
      }
      if (A.norm == LF_NORM_TOKEN) {
        ss = rope_lane_sum(ss, 1, A.tpt < 32 ? A.tpt : 32);
        if (A.tpt > 32 && (lane_t & 31) == 0)
          s_warp[k * (kRopeThreads / 32) + ((grp * A.tpt + lane_t) >> 5)] = ss;
        r[k][0] = ss;
      }
    }
  }
  __syncthreads();                                       // angles and warp sums
  __nv_bfloat16* yr = A.out + ((int64_t)A.out_slot[f] * A.T + t0) * A.out_stride;
#pragma unroll
  for (int k = 0; k < NT; ++k) {
    if (t0 + k >= A.T) return;
    if (A.norm == LF_NORM_TOKEN) {
      float ss = r[k][0];
      if (A.tpt > 32) {
        ss = 0.f;
        for (int i = 0; i < A.tpt >> 5; ++i) ss += s_warp[k * (kRopeThreads / 32) + grp * (A.tpt >> 5) + i];
      }
      ss = rsqrtf(ss * A.inv_n + A.eps);
#pragma unroll
      for (int u = 0; u < U; ++u) r[k][u] = ss;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int id = lane_t + u * A.tpt, base = (id - o) * 16;
      if (id >= A.units) break;
      float v[16];
      rope_unpack(a[k][u], b[k][u], v);
      if (A.norm != LF_NORM_NONE) {
        const float* w = A.weight + (A.norm == LF_NORM_TOKEN ? base : 0);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float4 w4 = *reinterpret_cast<const float4*>(w + (q < 2 ? ca : cb) + (q & 1) * 4);
          v[4 * q] *= r[k][u] * w4.x;
          v[4 * q + 1] *= r[k][u] * w4.y;
          v[4 * q + 2] *= r[k][u] * w4.z;
          v[4 * q + 3] *= r[k][u] * w4.w;
        }
      }
      if (A.p_w > 0) rope_turn(v, cs + k * (A.d / 2), o, A.d / 4, A.halves);
      *reinterpret_cast<uint4*>(yr + k * A.out_stride + base + ca) = rope_pack(v);
      *reinterpret_cast<uint4*>(yr + k * A.out_stride + base + cb) = rope_pack(v + 8);
    }
  }
}

// Gradient with a norm, both of its sums over channels in one pass: with xn = r x and
// mu = r mean(w g x) = mean(w g xn),
//   dx = r (w g - mu xn),  dw += g xn.
// xn and mu have the size of 1 and of w g whatever the rows' size; r^3, which a form with one
// multiplication fewer has, leaves fp32 at rows of 2^42 (or 2^-42 with eps = 0).
// Each CTA walks steps blockIdx.x, + gridDim.x, ... (`groups` tokens of a frame each) in order,
// loading the next step's channels while it works on this one's, and keeps its part of dw in
// registers; the parts of its warps are added in warp order, those of the CTAs in a fixed
// order by rope_dweight_kernel, so dw does not depend on timing.  Angles and warp sums have
// two buffers, which leaves two barriers per step.
template <int U, int NF>
__global__ void __launch_bounds__(kRopeThreads)
rope_bwd_kernel(const __grid_constant__ RopeArgs<NF> A) {
  extern __shared__ float2 s_cs[];                       // [2][groups][d / 2]
  const int cs_len = A.groups * (A.d / 2);
  float2* s_warp = s_cs + 2 * cs_len;                    // [2][warps] sums of x^2 and of w g x
  float* s_dw = reinterpret_cast<float*>(s_warp + 2 * (kRopeThreads / 32));   // [d or H * d]
  const int grp = threadIdx.y, lane_t = threadIdx.x, tid = grp * A.tpt + lane_t;
  const int o = lane_t & (A.upd - 1);
  const int ca = o * 8, cb = A.d / 2 + o * 8;            // the unit's two pieces of its head
  const bool per_token = A.norm == LF_NORM_TOKEN;
  const int wpt = A.tpt >> 5;                            // warps per token, 0: lanes of one
  float dw[U][16];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int i = 0; i < 16; ++i) dw[u][i] = 0.f;

  const int per_frame = (A.T + A.groups - 1) / A.groups;
  struct Place { int f, i; };                            // frame and step in it
  auto advance = [&](Place p, int n) {
    p.i += n;
    while (p.f < A.n_frames && p.i >= per_frame) p.i -= per_frame, ++p.f;
    return p;
  };
  uint4 nxa[U], nxb[U], nga[U], ngb[U];
  auto load = [&](Place p) {
    const int t = p.i * A.groups + grp;
    const bool live = p.f < A.n_frames && t < A.T;
    const int f = p.f < A.n_frames ? p.f : 0;
    const __nv_bfloat16* xr = A.x + ((int64_t)A.x_slot[f] * A.T + t) * A.x_stride;
    const __nv_bfloat16* gr = A.dout + ((int64_t)A.dout_slot[f] * A.T + t) * A.dout_stride;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int id = lane_t + u * A.tpt, base = (id - o) * 16;
      nxa[u] = nxb[u] = nga[u] = ngb[u] = make_uint4(0, 0, 0, 0);
      if (live && id < A.units) {
        nxa[u] = *reinterpret_cast<const uint4*>(xr + base + ca);
        nxb[u] = *reinterpret_cast<const uint4*>(xr + base + cb);
        nga[u] = *reinterpret_cast<const uint4*>(gr + base + ca);
        ngb[u] = *reinterpret_cast<const uint4*>(gr + base + cb);
      }
    }
  };
  Place at = advance(Place{0, 0}, blockIdx.x);
  load(at);
  for (int buf = 0; at.f < A.n_frames; buf ^= 1) {
    const int f = at.f, t = at.i * A.groups + grp;
    const bool live = t < A.T;
    float2* cs = s_cs + buf * cs_len + grp * (A.d / 2);
    if (live && A.p_w > 0) rope_angles(A, f, t, lane_t, cs);
    uint4 xa[U], xb[U];
    float g[U][16];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      xa[u] = nxa[u], xb[u] = nxb[u];
      rope_unpack(nga[u], ngb[u], g[u]);
    }
    at = advance(at, gridDim.x);
    load(at);
    __syncthreads();                                     // angles
    float ss[U], m[U], ss_all = 0.f, m_all = 0.f;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int id = lane_t + u * A.tpt, base = (id - o) * 16;
      float x[16];
      rope_unpack(xa[u], xb[u], x);
      ss[u] = m[u] = 0.f;
      if (live && id < A.units) {
        if (A.p_w > 0) rope_turn(g[u], cs, o, A.d / 4, A.halves);
        const float* w = A.weight + (per_token ? base : 0);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float4 w4 = *reinterpret_cast<const float4*>(w + (q < 2 ? ca : cb) + (q & 1) * 4);
          const float wv[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int i = 4 * q + k;
            ss[u] = fmaf(x[i], x[i], ss[u]);
            m[u] = fmaf(wv[k], g[u][i] * x[i], m[u]);
          }
        }
      }
      ss_all += ss[u];
      m_all += m[u];
    }
    if (per_token) {
      ss_all = rope_lane_sum(ss_all, 1, A.tpt < 32 ? A.tpt : 32);
      m_all = rope_lane_sum(m_all, 1, A.tpt < 32 ? A.tpt : 32);
      if (wpt > 1) {
        float2* sw = s_warp + buf * (kRopeThreads / 32);
        if ((lane_t & 31) == 0) sw[tid >> 5] = make_float2(ss_all, m_all);
        __syncthreads();
        ss_all = m_all = 0.f;
        for (int i = 0; i < wpt; ++i) {
          const float2 v = sw[grp * wpt + i];
          ss_all += v.x;
          m_all += v.y;
        }
      }
    } else {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        ss[u] = rope_lane_sum(ss[u], 1, A.upd);
        m[u] = rope_lane_sum(m[u], 1, A.upd);
      }
    }
    if (!live) continue;                                 // (the same for a token's threads)
    __nv_bfloat16* dr = A.out + ((int64_t)A.out_slot[f] * A.T + t) * A.out_stride;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int id = lane_t + u * A.tpt, base = (id - o) * 16;
      if (id >= A.units) break;
      if (!per_token) ss_all = ss[u], m_all = m[u];
      const float r = rsqrtf(ss_all * A.inv_n + A.eps), mu = r * (m_all * A.inv_n);
      const float* w = A.weight + (per_token ? base : 0);
      float x[16];
      rope_unpack(xa[u], xb[u], x);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float4 w4 = *reinterpret_cast<const float4*>(w + (q < 2 ? ca : cb) + (q & 1) * 4);
        const float wv[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int i = 4 * q + k;
          const float xn = r * x[i];
          dw[u][i] = fmaf(g[u][i], xn, dw[u][i]);
          x[i] = r * fmaf(wv[k], g[u][i], -mu * xn);
        }
      }
      *reinterpret_cast<uint4*>(dr + base + ca) = rope_pack(x);
      *reinterpret_cast<uint4*>(dr + base + cb) = rope_pack(x + 8);
    }
  }

  // dw of the CTA: lanes with the same channels, then the warps in order
  const int n_dw = per_token ? A.H * A.d : A.d, n_thr = A.tpt * A.groups;
  for (int i = tid; i < n_dw; i += n_thr) s_dw[i] = 0.f;
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
  const int lane = tid & 31, warp = tid >> 5;
  for (int w = 0; w < n_thr / 32; ++w) {
    __syncthreads();
    if (warp != w || lane >= same) continue;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int id = lane_t + u * A.tpt, base = per_token ? (id - o) * 16 : 0;
      if (per_token ? id >= A.units : u > 0) break;
#pragma unroll
      for (int i = 0; i < 16; ++i) s_dw[base + (i < 8 ? ca + i : cb + i - 8)] += dw[u][i];
    }
  }
  __syncthreads();
  for (int i = tid; i < n_dw; i += n_thr) A.part[(size_t)blockIdx.x * n_dw + i] = s_dw[i];
}

// dweight[c] = sum of the CTAs' parts, in a fixed order: 32 channels per CTA, 16 threads a
// channel.
__global__ void __launch_bounds__(512)
rope_dweight_kernel(const float* __restrict__ part, int n_part, int n_dw, float* __restrict__ dweight) {
  __shared__ float s[16][33];
  const int c = blockIdx.x * 32 + (threadIdx.x & 31), k = threadIdx.x >> 5;
  float v = 0.f;
  if (c < n_dw) {
#pragma unroll 8
    for (int i = k; i < n_part; i += 16) v += part[(size_t)i * n_dw + c];
  }
  s[k][threadIdx.x & 31] = v;
  __syncthreads();
  if (k == 0 && c < n_dw) {
    for (int i = 1; i < 16; ++i) v += s[i][threadIdx.x];
    dweight[c] = v;
  }
}

}  // namespace lf
