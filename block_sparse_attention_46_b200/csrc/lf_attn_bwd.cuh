// lf_attn_bwd.cuh — gradient of stage (d), block-sparse attention.
//
// With c = scale * log2(e), P = 2^(c q.k - lse * log2(e)) recomputed from the forward call's
// lse, dP = dout . v and D = sum_d dout * out per row:
//   dS = P (dP - D),  dq = scale sum_k dS k,  dk = scale sum_q dS q,  dv = sum_q P dout.
// Two passes, so that every output is summed by one owner in a fixed order (no float
// atomics): dq over query tiles, through the forward pass's key plans; dk and dv over tiles
// of 128 keys, through the transposed plans (which query blocks attend to which key tile).
// Scores and dP are computed twice for it: seven products of 2 d FLOPs per pair instead of
// the five that one pass with atomics would need.
#pragma once
#include "lf_attn.cuh"

namespace lf {

// ---------------------------------------------------------------------------------
// Rows: what the gradient needs of every query row, -lse * log2(e) and -D, padded so that
// whole tiles can be read: `dense` rows in token order, [H, pad128(ncur)], and `blk` rows by
// query block, [H, nqb * B] (only where some key tile has a list of query blocks).  Padding rows and rows that attend to nothing hold -inf, which
// makes their P zero.
// ---------------------------------------------------------------------------------
struct BwdRows {
  float *dense_nlse, *dense_nd;    // [H, pad128(ncur)]
  float *blk_nlse, *blk_nd;        // [H, nqb * B]
};

__host__ __device__ inline int bwd_dense_rows(const Dims& D) { return cdiv(D.ncur, 128) * 128; }
__host__ __device__ inline int bwd_blk_rows(const Dims& D) { return D.nqb * D.B; }

// d / 8 threads per (row, head), 16-byte loads, heads fastest (a token's row is contiguous).
// Also zeroes the entry counter of the transposed plans.
__global__ void __launch_bounds__(256)
bwd_rows_kernel(const __nv_bfloat16* __restrict__ out, const __nv_bfloat16* __restrict__ dout,
                const float* __restrict__ lse, BwdRows R, int32_t* inv_total, bool blk,
                const Dims D) {
  if (blockIdx.x == 0 && threadIdx.x == 0) *inv_total = 0;
  const int per = D.d / 8;
  const long long idx = (long long)blockIdx.x * blockDim.x + threadIdx.x;
  const long long item = idx / per;
  const int part = (int)(idx % per);
  const int blk_rows = bwd_blk_rows(D), dense_rows = bwd_dense_rows(D);
  const long long p = item / D.H;                        // padded row; then the dense padding
  const int h = (int)(item % D.H);
  int tok = -1;
  if (p < blk_rows) {
    const int qb = (int)p / D.B, i = (int)p % D.B;
    if (i < block_len(D, qb % D.nbpf)) tok = (qb / D.nbpf) * D.T + (qb % D.nbpf) * D.B + i;
  }
  float s = 0.f;
  if (tok >= 0) {
    const size_t off = ((size_t)tok * D.H + h) * D.d + part * 8;
    const uint4 a = *reinterpret_cast<const uint4*>(out + off);
    const uint4 b = *reinterpret_cast<const uint4*>(dout + off);
    const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s = fmaf(__uint_as_float(wa[i] << 16), __uint_as_float(wb[i] << 16), s);
      s = fmaf(__uint_as_float(wa[i] & 0xffff0000u), __uint_as_float(wb[i] & 0xffff0000u), s);
    }
  }
  for (int o = 1; o < per; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  if (part != 0) return;
  float nl = -INFINITY;
  if (tok >= 0) {
    const float l = lse[(size_t)h * D.ncur + tok];
    if (l != -INFINITY) nl = -l * 1.4426950408889634f;
  }
  if (p < blk_rows) {
    if (blk) {
      R.blk_nlse[(size_t)h * blk_rows + p] = nl;
      R.blk_nd[(size_t)h * blk_rows + p] = -s;
    }
    if (tok >= 0) {
      R.dense_nlse[(size_t)h * dense_rows + tok] = nl;
      R.dense_nd[(size_t)h * dense_rows + tok] = -s;
    }
  } else if (p - blk_rows < dense_rows - D.ncur) {
    const size_t at = (size_t)h * dense_rows + D.ncur + (size_t)(p - blk_rows);
    R.dense_nlse[at] = -INFINITY;
    R.dense_nd[at] = 0.f;
  }
}

// ---------------------------------------------------------------------------------
// Key tiles of the dk, dv pass: 128 key rows of one frame (two 64-token blocks, or one of
// 128), or of the dense current chunk as a whole.  In launch order, heads outermost in each
// kind: the dense current chunk, the sink frames (both attended to by every query), then the
// tiles with lists: the sparse current chunk's frames and the history frames.
// ---------------------------------------------------------------------------------
struct KeyTiles {
  int per_frame;        // ceil(T / 128)
  int n_dense;          // current-chunk tiles (0 when the current chunk is sparse)
  int n_sink;           // sink tiles (0 without gradients into the cache)
  int fl_cur, fl_hist;  // frames with lists: current (sparse current chunk), history
  __host__ __device__ int n_list() const { return (fl_cur + fl_hist) * per_frame; }
  __host__ __device__ int total() const { return n_dense + n_sink + n_list(); }
};

__host__ __device__ inline KeyTiles key_tiles(const Dims& D, bool cache_grad) {
  KeyTiles k;
  k.per_frame = cdiv(D.T, 128);
  k.n_dense = D.kc > 0 ? 0 : cdiv(D.ncur, 128);
  k.n_sink = cache_grad ? D.S * k.per_frame : 0;
  k.fl_cur = D.kc > 0 ? D.Fc : 0;
  k.fl_hist = cache_grad ? D.F : 0;
  return k;
}

// One key tile of the launch.
struct KeyTile {
  int h;
  int kind;          // 0: dense current chunk, 1: sink, 2: current with a list, 3: history
  int frame;         // kind 1: sink, 2: current frame, 3: history position
  int row;           // first row, in the current chunk (kind 0) or in the frame
  int list;          // kinds 2, 3: index of the list, else -1
};

__device__ __forceinline__ KeyTile key_tile_of(int u, const KeyTiles& K, const Dims& D) {
  KeyTile k;
  k.list = -1;
  k.frame = 0;
  if (u < K.n_dense * D.H) {
    k.kind = 0;
    k.h = u / K.n_dense;
    k.row = (u % K.n_dense) * 128;
    return k;
  }
  u -= K.n_dense * D.H;
  if (u < K.n_sink * D.H) {
    k.kind = 1;
    k.h = u / K.n_sink;
    u %= K.n_sink;
    k.frame = u / K.per_frame;
    k.row = (u % K.per_frame) * 128;
    return k;
  }
  u -= K.n_sink * D.H;
  k.list = u;
  k.h = u / K.n_list();
  u %= K.n_list();
  k.frame = u / K.per_frame;
  k.row = (u % K.per_frame) * 128;
  k.kind = k.frame < K.fl_cur ? 2 : 3;
  if (k.kind == 3) k.frame -= K.fl_cur;
  return k;
}

// Transposed plans.  One warp per (head, key tile with a list): each lane looks the tile's
// blocks up in one query tile's plan (ascending within its current-chunk and history parts),
// and the query blocks that hold them are written in ascending order as qb << 2 | mask, bit 0:
// the tile's first 64 rows, bit 1: its last 64.  A query block enters a tile's list at most
// once, so all lists fit in H * nqb * (kc + nsel) entries; where a list lies depends on the
// order of the allocations, its contents do not.
constexpr int kInvWarps = 4;

__device__ __forceinline__ int plan_key(uint32_t pe, const Dims& D) {
  const int p = (int)(pe >> 16), b = (int)((pe >> 4) & 0xFFFu);
  const int f = p >= D.S + D.F ? p - (D.S + D.F) : p - D.S + (D.kc > 0 ? D.Fc : 0);
  return f * D.nbpf + b;
}

__global__ void __launch_bounds__(kInvWarps * 32)
bwd_transpose_kernel(const uint32_t* __restrict__ plan, const int32_t* __restrict__ plan_cnt,
                     const KeyTiles K, uint32_t* __restrict__ inv, int32_t* inv_total,
                     int32_t* __restrict__ inv_off, int32_t* __restrict__ inv_cnt, const Dims D) {
  const int u = blockIdx.x * kInvWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (u >= K.n_list() * D.H) return;
  const KeyTile k = key_tile_of(u + (K.n_dense + K.n_sink) * D.H, K, D);
  const int ntiles = tile_count(D), stride = plan_stride(D), nsink = D.S * D.nbpf;
  const int b0 = k.row / D.B;
  const int fkey = k.kind == 2 ? k.frame : k.frame + (D.kc > 0 ? D.Fc : 0);
  const int key0 = fkey * D.nbpf + b0;
  const bool two = D.B == 64 && b0 + 1 < D.nbpf;
  int base = 0;
  for (int pass = 0; pass < 2; ++pass) {
    int n = 0;
    for (int t0 = 0; t0 < ntiles; t0 += 32) {
      const int t = t0 + lane;
      uint32_t m0 = 0, m1 = 0;           // masks of the tile's query blocks 2t and 2t + 1 (or t)
      if (t < ntiles) {
        const uint32_t* pl = plan + ((size_t)k.h * ntiles + t) * stride;
        const int cnt = plan_cnt[(size_t)k.h * ntiles + t];
        int lo = nsink, hi = cnt;
        while (lo < hi) {
          const int mid = (lo + hi) >> 1;
          if (plan_key(pl[mid], D) < key0) lo = mid + 1; else hi = mid;
        }
        uint32_t ma = 0, mb = 0;
        if (lo < cnt && plan_key(pl[lo], D) == key0) ma = pl[lo++] & 3u;
        if (two && lo < cnt && plan_key(pl[lo], D) == key0 + 1) mb = pl[lo] & 3u;
        if (D.B == 64) {
          m0 = (ma & 1u) | ((mb & 1u) << 1);
          m1 = (ma >> 1) | (mb & 2u);
        } else {
          m0 = ma ? 3u : 0u;
        }
      }
      const int mine = (m0 != 0) + (m1 != 0);
      int pre = mine;
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, pre, o);
        if (lane >= o) pre += v;
      }
      if (pass == 1) {
        uint32_t* w = inv + base + n + pre - mine;
        const uint32_t qb = D.B == 64 ? 2u * t : (uint32_t)t;
        if (m0) *w++ = qb << 2 | m0;
        if (m1) *w = (qb + 1) << 2 | m1;
      }
      n += __shfl_sync(0xffffffffu, pre, 31);
    }
    if (pass == 0) {
      if (lane == 0) {
        base = atomicAdd(inv_total, n);
        inv_off[u] = base;
        inv_cnt[u] = n;
      }
      base = __shfl_sync(0xffffffffu, base, 0);
    }
  }
}

// ---------------------------------------------------------------------------------
// The two passes, one warp per output row; each lane holds d / 32 channels.
// ---------------------------------------------------------------------------------
struct BwdArgs {
  const __nv_bfloat16 *q, *k_cur, *v_cur, *k_cache, *v_cache, *dout;
  __nv_bfloat16 *dq, *dk_cur, *dv_cur, *dk_cache, *dv_cache;
  const uint32_t* plan;
  const int32_t* plan_cnt;
  BwdRows rows;
  KeyTiles kt;
  const uint32_t* inv;
  const int32_t *inv_off, *inv_cnt;
  int slots[LF_MAX_FRAMES];
};

template <int NC>
__device__ __forceinline__ void row_load(const __nv_bfloat16* p, int lane, float* v) {
#pragma unroll
  for (int i = 0; i < NC / 2; ++i) {
    const uint32_t w = reinterpret_cast<const uint32_t*>(p)[lane + 32 * i];
    v[2 * i] = __uint_as_float(w << 16);
    v[2 * i + 1] = __uint_as_float(w & 0xffff0000u);
  }
}

template <int NC>
__device__ __forceinline__ void row_store(__nv_bfloat16* p, int lane, const float* v) {
#pragma unroll
  for (int i = 0; i < NC / 2; ++i) {
    __nv_bfloat162 t = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    reinterpret_cast<uint32_t*>(p)[lane + 32 * i] = *reinterpret_cast<uint32_t*>(&t);
  }
}

template <int NC>
__device__ __forceinline__ float row_dot(const float* a, const float* b) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < NC; ++i) s = fmaf(a[i], b[i], s);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

template <int HD>
__global__ void __launch_bounds__(256) bwd_dq_simple_kernel(const __grid_constant__ BwdArgs A, const Dims D) {
  constexpr int NC = HD / 32;
  const int lane = threadIdx.x & 31;
  const int tok = blockIdx.x * 8 + (threadIdx.x >> 5), h = blockIdx.y;
  if (tok >= D.ncur) return;
  const float c = D.scale * 1.4426950408889634f;
  const size_t row = ((size_t)tok * D.H + h) * HD;
  float q[NC], g[NC], acc[NC] = {};
  row_load<NC>(A.q + row, lane, q);
  row_load<NC>(A.dout + row, lane, g);
  const float nl = A.rows.dense_nlse[(size_t)h * bwd_dense_rows(D) + tok];
  const float nd = A.rows.dense_nd[(size_t)h * bwd_dense_rows(D) + tok];
  auto keys = [&](const __nv_bfloat16* kp, const __nv_bfloat16* vp, size_t first, int n) {
    for (int i = 0; i < n; ++i) {
      float k[NC], v[NC];
      const size_t at = ((first + i) * D.H + h) * HD;
      row_load<NC>(kp + at, lane, k);
      row_load<NC>(vp + at, lane, v);
      const float s = row_dot<NC>(q, k), dp = row_dot<NC>(g, v);
      const float ds = exp2f(fmaf(s, c, nl)) * (dp + nd);
      for (int j = 0; j < NC; ++j) acc[j] = fmaf(ds, k[j], acc[j]);
    }
  };
  if (D.kc == 0) keys(A.k_cur, A.v_cur, 0, D.ncur);
  const int qb = tok / D.T * D.nbpf + tok % D.T / D.B;
  const int t = D.B == 64 ? qb / 2 : qb;
  const uint32_t bit = D.B == 64 && (qb & 1) ? 2u : 1u;
  const size_t tile = (size_t)h * tile_count(D) + t;
  const int cnt = A.plan_cnt[tile];
  for (int e = 0; e < cnt; ++e) {
    const uint32_t pe = A.plan[tile * plan_stride(D) + e];
    if (!(pe & bit)) continue;
    const int p = (int)(pe >> 16), b = (int)((pe >> 4) & 0xFFFu);
    if (p >= D.S + D.F)
      keys(A.k_cur, A.v_cur, (size_t)(p - D.S - D.F) * D.T + b * D.B, block_len(D, b));
    else
      keys(A.k_cache, A.v_cache, (size_t)A.slots[p] * D.T + b * D.B, block_len(D, b));
  }
  for (int j = 0; j < NC; ++j) acc[j] *= D.scale;
  row_store<NC>(A.dq + row, lane, acc);
}

template <int HD>
__global__ void __launch_bounds__(256) bwd_dkv_simple_kernel(const __grid_constant__ BwdArgs A, const Dims D) {
  constexpr int NC = HD / 32;
  const int lane = threadIdx.x & 31;
  const KeyTile kt = key_tile_of(blockIdx.x, A.kt, D);
  const int r = blockIdx.y * 8 + (threadIdx.x >> 5);     // row of the tile
  const int h = kt.h;
  const int n_rows = kt.kind == 0 ? D.ncur : D.T;
  if (kt.row + r >= n_rows) return;
  const bool cur = kt.kind == 0 || kt.kind == 2;
  const size_t tok = kt.kind == 0 ? (size_t)(kt.row + r)
                     : (size_t)(kt.kind == 2   ? kt.frame
                                : kt.kind == 1 ? A.slots[kt.frame]
                                               : A.slots[D.S + kt.frame]) * D.T + kt.row + r;
  const size_t row = (tok * D.H + h) * HD;
  float k[NC], v[NC], dk[NC] = {}, dv[NC] = {};
  row_load<NC>((cur ? A.k_cur : A.k_cache) + row, lane, k);
  row_load<NC>((cur ? A.v_cur : A.v_cache) + row, lane, v);
  const float c = D.scale * 1.4426950408889634f;
  auto queries = [&](int first, int n, const float* nl, const float* nd) {
    for (int i = 0; i < n; ++i) {
      float q[NC], g[NC];
      const size_t at = ((size_t)(first + i) * D.H + h) * HD;
      row_load<NC>(A.q + at, lane, q);
      row_load<NC>(A.dout + at, lane, g);
      const float p = exp2f(fmaf(row_dot<NC>(q, k), c, nl[i]));
      const float ds = p * (row_dot<NC>(g, v) + nd[i]);
      for (int j = 0; j < NC; ++j) {
        dv[j] = fmaf(p, g[j], dv[j]);
        dk[j] = fmaf(ds, q[j], dk[j]);
      }
    }
  };
  if (kt.list < 0) {
    const size_t at = (size_t)h * bwd_dense_rows(D);
    queries(0, D.ncur, A.rows.dense_nlse + at, A.rows.dense_nd + at);
  } else {
    const uint32_t* list = A.inv + A.inv_off[kt.list];
    for (int e = 0; e < A.inv_cnt[kt.list]; ++e) {
      if (!(list[e] & (r < 64 ? 1u : 2u))) continue;
      const int qb = (int)(list[e] >> 2);
      const size_t at = (size_t)h * bwd_blk_rows(D) + (size_t)qb * D.B;
      queries(qb / D.nbpf * D.T + qb % D.nbpf * D.B, block_len(D, qb % D.nbpf),
              A.rows.blk_nlse + at, A.rows.blk_nd + at);
    }
  }
  for (int j = 0; j < NC; ++j) dk[j] *= D.scale;
  row_store<NC>((cur ? A.dk_cur : A.dk_cache) + row, lane, dk);
  row_store<NC>((cur ? A.dv_cur : A.dv_cache) + row, lane, dv);
}

}  // namespace lf
