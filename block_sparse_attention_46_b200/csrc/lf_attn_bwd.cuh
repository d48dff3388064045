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
// Rows: what the gradient needs of every query row, -lse * log2(e) and -D, in boxes of 64
// rows (64 floats of the one, then 64 of the other; one 512-byte bulk copy): `dense` boxes
// in token order, [H, 2 * ceil(ncur / 128)], and, only where some key tile has a list of
// query blocks, `blk` boxes by query block, [H, nqb * B / 64] and one box of padding.
// Padding rows and rows that attend to nothing hold -inf, which makes their P zero.
// ---------------------------------------------------------------------------------
constexpr int kBoxFloats = 128;

static_assert(kPlanWarps * 32 == kBoxFloats, "one thread per value of the padding box");

struct BwdRows {
  float *dense, *blk;
};

__host__ __device__ inline int bwd_dense_boxes(const Dims& D) { return cdiv(D.ncur, 128) * 2; }
__host__ __device__ inline int bwd_blk_boxes(const Dims& D) { return D.nqb * (D.B / 64); }

// What the two passes start from, in one launch (apart, the plans' 10 us of latency on the 480p
// chunk came on top of the rows' 13): per head (grid.y) the first plan_ctas CTAs make key plans,
// a warp each, the others the row values with d / 8 threads per row and 16-byte loads.  Also
// zeroes the entry counter of the transposed plans.
constexpr int kPrepThreads = kPlanWarps * 32, kPrepRows = 4;   // rows per thread, loaded at once

__global__ void __launch_bounds__(kPrepThreads)
bwd_prep_kernel(const __nv_bfloat16* __restrict__ out, const __nv_bfloat16* __restrict__ dout,
                const float* __restrict__ lse, BwdRows R, bool blk,
                const int32_t* __restrict__ block_idx, const int32_t* __restrict__ cur_idx,
                uint32_t* __restrict__ plan, int32_t* __restrict__ plan_cnt, int32_t* inv_total,
                int plan_ctas, int longest, const Dims D) {
  extern __shared__ int32_t s_lists[];                 // two lists per warp
  if ((int)blockIdx.x < plan_ctas) {
    const int w = threadIdx.x >> 5, t = blockIdx.x * kPlanWarps + w;
    if (blockIdx.x == 0 && blockIdx.y == 0) {
      if (threadIdx.x == 0) *inv_total = 0;
      if (blk)                                         // the box of padding
        R.blk[(size_t)D.H * bwd_blk_boxes(D) * kBoxFloats + threadIdx.x] =
            threadIdx.x < 64 ? -INFINITY : 0.f;
    }
    if (t < tile_count(D))
      plan_tile(block_idx, cur_idx, plan, plan_cnt, t, blockIdx.y, s_lists + 2 * w * longest,
                s_lists + (2 * w + 1) * longest, D);
    return;
  }
  const int lg = D.d == 128 ? 4 : 3, per = 1 << lg;      // threads per row
  const int part = threadIdx.x & (per - 1), h = blockIdx.y, step = kPrepThreads >> lg;
  const int blk_rows = D.nqb * D.B, dense_rows = bwd_dense_boxes(D) * 64;
  // p0 + k step: padded rows; then the dense padding
  const int p0 = (blockIdx.x - plan_ctas) * (kPrepRows * step) + (threadIdx.x >> lg);
  int tok[kPrepRows];
  uint4 a[kPrepRows], b[kPrepRows];
#pragma unroll
  for (int k = 0; k < kPrepRows; ++k) {
    const int p = p0 + k * step;
    tok[k] = -1;
    a[k] = b[k] = make_uint4(0, 0, 0, 0);
    if (p < blk_rows) {
      const int qb = D.B == 128 ? p >> 7 : p >> 6, f = qb / D.nbpf;
      const int t = p - f * D.nbpf * D.B;              // in the padded frame
      if (t < D.T) tok[k] = f * D.T + t;
    }
    if (tok[k] >= 0) {
      const size_t off = ((size_t)tok[k] * D.H + h) * D.d + part * 8;
      a[k] = *reinterpret_cast<const uint4*>(out + off);
      b[k] = *reinterpret_cast<const uint4*>(dout + off);
    }
  }
#pragma unroll
  for (int k = 0; k < kPrepRows; ++k) {
    const int p = p0 + k * step;
    const uint32_t wa[4] = {a[k].x, a[k].y, a[k].z, a[k].w}, wb[4] = {b[k].x, b[k].y, b[k].z, b[k].w};
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      s = fmaf(__uint_as_float(wa[i] << 16), __uint_as_float(wb[i] << 16), s);
      s = fmaf(__uint_as_float(wa[i] & 0xffff0000u), __uint_as_float(wb[i] & 0xffff0000u), s);
    }
    for (int o = 1; o < per; o <<= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (part != 0) continue;
    float nl = -INFINITY;
    if (tok[k] >= 0) {
      const float l = lse[(size_t)h * D.ncur + tok[k]];
      if (l != -INFINITY) nl = -l * 1.4426950408889634f;
    }
    auto put = [&](float* base, size_t box0, int row) {
      float* x = base + (box0 + row / 64) * kBoxFloats + row % 64;
      x[0] = nl;
      x[64] = -s;
    };
    if (p < blk_rows) {
      if (blk) put(R.blk, (size_t)h * bwd_blk_boxes(D), p);
      if (tok[k] >= 0) put(R.dense, (size_t)h * bwd_dense_boxes(D), tok[k]);
    } else if (p - blk_rows < dense_rows - D.ncur) {
      put(R.dense, (size_t)h * bwd_dense_boxes(D), D.ncur + p - blk_rows);
    }
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
// The two passes, in one launch: CTAs [0, tiles * H) take a (head, 128-row query tile) each
// and give dq, the others a key tile each and give dk and dv.  A CTA keeps its own two
// operand tiles in shared memory (Q and dout; K and V) and streams the other side's through
// two rings; its accumulators stay in tensor memory until the end.
//
//   dq:      S = Q K^T, dP = dout V^T, dS = P (dP - D) as bf16 over S, dq += dS K
//   dk, dv:  S^T = K Q^T, P^T as bf16 over S^T, dv += P^T dout,
//            dP^T = V dout^T, dS^T as bf16 beside P^T, dk += dS^T Q
//
// Four warps issue (two TMA, two tcgen05.mma: scores and dP by one, the accumulating products
// by the other, so that neither waits behind the other's operands), two warpgroups make P and
// dS, a thread one row of columns [64 w, 64 w + 64) of every tile.  Tensor memory has 512
// columns; the accumulators take 128 (dq) or 256 (dk and dv):
//   dq: buffers S0, S1 and one of dP.  S of tile j + 1 and, once this tile's is read, dP of
//   tile j + 1 run under the exponentials of tile j.
//   dk, dv: buffers X0, X1.  Tile j has S in X[j & 1] and dP in the other one, P and dS both
//   go over S, so dP's buffer is free for the next tile's S once it has been read, and the
//   exponentials of tile j + 1 overlap dk of tile j and dP of tile j + 1.
//
// What bounds it: the tensor pipe is active 62 % of the cycles (480p chunk with cache
// gradients: 1.00 ms at 1.69 GHz, 467 MB read, 177 MB written).  A 128 x 128 tile takes 2160-2200
// clk for dq (1536 of products) and 2890-2940 for dk and dv (2048).  The rest is taken to be
// the chain through one tile: S, exponentials (1024 clk of the special-function units), dP,
// dS, the product that frees the buffer for the next S, with 130-150 clk per mbarrier hop.
// A CTA's start and end add 7300-9500 clk, which the short key tiles feel most.  Measured
// instead, on the 480p chunk: dq's warpgroups on alternate tiles 8 % slower; left operands in
// tensor memory and units of 64 columns 7-15 %, with two teams of eight row warps 10 %; part
// of the exponentials on the multiply-add units 1 %; own tiles loaded before the allocation
// of tensor memory 2-3 %; no register split 3 %.
//
// P and dS enter their products rounded to bf16, the type of the tensor-core operands beside
// them (K, Q and dout): each term of a sum is off by at most 2^-8 of it, half a step.  Nothing
// else is lost: fp32 with these two roundings and the final one gives the kernel's outputs to
// within 3e-4, in one of 24 cases 1e-3.  Against 64 bits the outputs' relative error is 0.0022 to
// 0.0025 where sums have dozens of terms or more and 0.0019 to 0.0033 where they have a few (one
// to ten keys per row); with fp32 operands it is 0.0016 to 0.0018.  dq loses most, since
// sum_k dS = 0 cancels what a row's keys have in common but not its rounding errors.
//
// A barrier that is waited for every other tile, or whose next completion does not depend on
// the waiting thread, exists twice, one for even and one for odd tiles: a wait on a parity
// sees at most one completion ahead.  An MMA that overwrites an operand of an earlier one
// waits for that one's completion.
// ---------------------------------------------------------------------------------
constexpr int kBwdThreads = 384;
// Register split: 128 x 136 + 256 x 184 = 384 x 168.  Issuers at 120, 136 and 152: single calls
// of the large chunk 3231, 3161 and 3184 us, the other sizes alike within 2 %.
constexpr int kBwdLaunchRegs = 168, kBwdLowRegs = 136, kBwdHighRegs = 184;
static_assert(128 * kBwdLowRegs + 256 * kBwdHighRegs <= kBwdThreads * kBwdLaunchRegs, "register split");

struct BwdParams {
  // rows of H * d channels: 2-D over the chunk's tokens, boxes of 64 channels x 128 rows, and
  // 3-D per frame, boxes of 64 x 64
  CUtensorMap q2, q3, g2, g3, kc2, kc3, vc2, vc3, kh, vh;
  CUtensorMap dq3, dk2, dk3, dkh, dv2, dv3, dvh;   // outputs, boxes of 64 x 64
  __nv_bfloat16 *dq, *dk_cur, *dv_cur, *dk_cache, *dv_cache;
  const uint32_t* plan;
  const int32_t* plan_cnt;
  BwdRows rows;
  KeyTiles kt;
  const uint32_t* inv;
  const int32_t *inv_off, *inv_cnt;
  int n_dq;                   // query tiles of all heads
  long long wait_limit_clk;   // limit of a CTA's waits, from its start
  int debug_stall;            // test hook: the CTA whose own tiles never come, + 1; 0: none
  int slots[LF_MAX_FRAMES];
};

enum BwdBar {
  kBbIn = 0,                   // the CTA's own tiles
  kBbS = 1,                    // [2] S of a tile
  kBbDP = 3,                   // [2] dP of a tile
  kBbP = 5,                    // [2] P written (dk, dv)
  kBbRd = 7,                   // dP read
  kBbDS = 8,                   // [2] dS written
  kBbAcc = 10,                 // [2] accumulating products of a tile complete
  kBbDone = 12,                // everything issued is complete (two issuers)
  kBbRing0 = 13,               // full[3], empty[3]
  kBbRing1 = 19,               // full[2], empty[2]
  kBbCount = 23
};
constexpr int kRing0 = 3, kRing1 = 2;
constexpr int kNbStore = 1;            // named barriers of a warpgroup's epilogue, + warpgroup

template <int HD>
struct BwdLayout {
  static constexpr int NH = HD / 64;
  static constexpr int kRegion = 128 * 128;            // 128 rows x 64 channels
  static constexpr int kTile = NH * kRegion;
  static constexpr int kMisc = kBbCount * 8;           // tensor-memory address
  static constexpr int kCols = 1024;                   // two tiles' boxes of row values
  static constexpr int kIn0 = kCols + 2 * 2 * kBoxFloats * 4;
  static constexpr int kIn1 = kIn0 + kTile;
  static constexpr int kR0 = kIn1 + kTile;
  static constexpr int kR1 = kR0 + kRing0 * kTile;
  static constexpr int kBytes = kR1 + kRing1 * kTile;  // 227 KB at d = 128
  static constexpr uint32_t kAcc0 = 0, kAcc1 = 128;    // dq or dk; dv
  static constexpr uint32_t kX0 = 256, kX1 = 384;      // dk, dv
  static constexpr uint32_t kS0 = 128, kS1 = 256, kDP = 384;   // dq
};
static_assert(BwdLayout<128>::kIn0 % 1024 == 0 && BwdLayout<128>::kBytes <= 227 * 1024, "shared memory");

// Tensor-core and copy instructions of one elected lane, issued from code that the whole warp
// runs: their operands (descriptors, addresses) then stay in uniform registers.  Issued from
// a lane-0 branch, 8 MMAs took the issuer 850-1100 clk instead of the 560 that they run.
__device__ __forceinline__ uint32_t elect_lane() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(r));
  return r;
}

// One product's MMAs (16 columns of A each), d (+)= A B with the first one's accumulation
// given: A and B in shared memory, descriptors `step` apart, four to a 64-channel region.
template <int N>
__device__ __forceinline__ void mma_ss_if(uint32_t lead, uint32_t d, uint64_t a, uint64_t b,
                                          uint32_t idesc, uint32_t region) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const uint64_t off = ((i >> 2) * region + (i & 3) * 32) >> 4;
    if (i == 0)
      asm volatile(
          "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, 0, 0;\n\tsetp.ne.b32 q, %4, 0;\n\t"
          "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
          ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(lead) : "memory");
    else
      asm volatile(
          "{\n\t.reg .pred p, q;\n\tsetp.eq.b32 p, 0, 0;\n\tsetp.ne.b32 q, %4, 0;\n\t"
          "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
          ::"r"(d), "l"(a + off), "l"(b + off), "r"(idesc), "r"(lead) : "memory");
  }
}

__device__ __forceinline__ void mma_ts_if(uint32_t lead, uint32_t d, uint32_t a, uint64_t b,
                                          uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc), "r"(lead) : "memory");
}

__device__ __forceinline__ void commit_if(uint32_t lead, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
      ::"r"(smem_u32(bar)), "r"(lead) : "memory");
}

__device__ __forceinline__ void expect_if(uint32_t lead, uint64_t* bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t.reg .b64 st;\n\tsetp.ne.b32 q, %2, 0;\n\t"
      "@q mbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n\t}"
      ::"r"(smem_u32(bar)), "r"(bytes), "r"(lead) : "memory");
}

__device__ __forceinline__ void bulk_load_if(uint32_t lead, void* dst, const void* src,
                                             uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %4, 0;\n\t"
      "@q cp.async.bulk.shared::cta.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];\n\t}"
      ::"r"(smem_u32(dst)), "l"(src), "r"(bytes), "r"(smem_u32(bar)), "r"(lead) : "memory");
}

// 128 rows x HD channels of one head from a 2-D map at `row`.
template <int HD>
__device__ __forceinline__ void load_tile_if(uint32_t lead, uint8_t* tile, const CUtensorMap* m,
                                             uint64_t* bar, int h, int row) {
#pragma unroll
  for (int c = 0; c < HD / 64; ++c)
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %5, 0;\n\t"
        "@q cp.async.bulk.tensor.2d.shared::cta.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];\n\t}"
        ::"r"(smem_u32(tile + c * BwdLayout<HD>::kRegion)), "l"(m), "r"(smem_u32(bar)),
          "r"(h * HD + c * 64), "r"(row), "r"(lead) : "memory");
}

// 64 rows x HD channels of one head into rows [64 box, 64 box + 64) of a tile, from a 3-D map
// at frame and row; rows past the frame's end, and frames past the last, read as zeros.
template <int HD>
__device__ __forceinline__ void load_box_if(uint32_t lead, uint8_t* tile, int box,
                                            const CUtensorMap* m, uint64_t* bar, int h, int row,
                                            int frame) {
#pragma unroll
  for (int c = 0; c < HD / 64; ++c)
    asm volatile(
        "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %6, 0;\n\t"
        "@q cp.async.bulk.tensor.3d.shared::cta.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];\n\t}"
        ::"r"(smem_u32(tile + c * BwdLayout<HD>::kRegion + box * 64 * 128)), "l"(m),
          "r"(smem_u32(bar)), "r"(h * HD + c * 64), "r"(row), "r"(frame), "r"(lead) : "memory");
}

// D = A B^T over HD channels, both tiles K-major in shared memory.
template <int HD>
__device__ __forceinline__ void mma_scores(uint32_t lead, uint32_t d, uint32_t a, uint32_t b) {
  constexpr uint32_t idesc = idesc_bf16_f32(128, 128, 0, 0);
  mma_ss_if<HD / 16>(lead, d, smem_desc_sw128(a, 16, 1024), smem_desc_sw128(b, 16, 1024), idesc,
                     BwdLayout<HD>::kRegion);
}

// D (+)= A B over 128 columns of A: bf16 pairs in tensor memory, `half` columns between the
// pairs of A's first and last 64 columns; B: 128 rows x HD in shared memory.
template <int HD>
__device__ __forceinline__ void mma_accumulate(uint32_t lead, uint32_t d, uint32_t a_tmem, int half,
                                               uint32_t b, bool acc) {
  constexpr uint32_t idesc = idesc_bf16_f32(128, HD, 0, 1);
  const uint64_t db = smem_desc_sw128(b, BwdLayout<HD>::kRegion, 1024);
#pragma unroll
  for (int ks = 0; ks < 8; ++ks)
    mma_ts_if(lead, d, a_tmem + (ks >> 2) * half + (ks & 3) * 8, db + (ks * 16 * 128 >> 4), idesc,
              acc || ks > 0 ? 1u : 0u);
}

// Two values rounded to bf16 and packed.
__device__ __forceinline__ float pack_bf16(float a, float b) {
  __nv_bfloat162 t = __floats2bfloat162_rn(a, b);
  return __uint_as_float(*reinterpret_cast<uint32_t*>(&t));
}

// A row warp hands its tensor-memory reads or writes to the MMA issuers.
__device__ __forceinline__ void warp_arrive(uint64_t* bar) {
  tc_fence_before();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// N (64 or 128) accumulators of a row, times f, as bf16 into the row of a tile in shared memory,
// in the 128-byte swizzle of the tensor maps.
template <int N>
__device__ __forceinline__ void stage_row(uint8_t* tile, int r, uint32_t taddr, float f) {
#pragma unroll 1
  for (int ch = 0; ch < N / 32; ++ch) {
    float v[32];
    tmem_ld32(taddr + ch * 32, v);
    tmem_ld_wait();
    reg_fence32(v);
    uint8_t* row = tile + (ch >> 1) * (128 * 128) + r * 128;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint4 w;
      w.x = __float_as_uint(pack_bf16(v[8 * e] * f, v[8 * e + 1] * f));
      w.y = __float_as_uint(pack_bf16(v[8 * e + 2] * f, v[8 * e + 3] * f));
      w.z = __float_as_uint(pack_bf16(v[8 * e + 4] * f, v[8 * e + 5] * f));
      w.w = __float_as_uint(pack_bf16(v[8 * e + 6] * f, v[8 * e + 7] * f));
      *reinterpret_cast<uint4*>(row + ((((ch & 1) * 4 + e) ^ (r & 7)) << 4)) = w;
    }
  }
}

// 64 rows x 64 channels of a staged tile to memory; what lies past the tensor's (or frame's)
// end is not written.
__device__ __forceinline__ void store_box(const void* src, const CUtensorMap* m, int x, int row, int frame) {
  if (frame < 0)
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%2, %3}], [%1];"
                 ::"l"(m), "r"(smem_u32(src)), "r"(x), "r"(row) : "memory");
  else
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];"
                 ::"l"(m), "r"(smem_u32(src)), "r"(x), "r"(row), "r"(frame) : "memory");
}

// The stores issued by this thread have read shared memory (their writes end with the kernel).
__device__ __forceinline__ void stores_read() {
  asm volatile("cp.async.bulk.commit_group;\n\tcp.async.bulk.wait_group.read 0;" ::: "memory");
}

// Whole-warp wait for an mbarrier's phase, until the deadline (in clocks) at the latest.  It
// branches on votes alone, so the warp leaves it together (what follows runs in uniform
// registers).  Small, because the loops of all roles together have to stay within the 32 KB of
// the instruction cache.
__device__ __forceinline__ bool wait_until(uint64_t* bar, uint32_t parity, long long deadline) {
#pragma unroll 1
  for (;;) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if (__any_sync(0xffffffffu, clock64() >= deadline)) return false;
  }
}

template <int HD, int BLK, bool is_dq>
__device__ __forceinline__ void bwd_tile(const BwdParams& P, const Dims& D, const int tile) {
  using L = BwdLayout<HD>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem);
  uint32_t* s_tmem = reinterpret_cast<uint32_t*>(smem + L::kMisc);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long deadline = clock64() + P.wait_limit_clk;

  // ---- the CTA's tile and the number of tiles that it streams
  const int ntiles = tile_count(D);
  const int n_dense = D.kc > 0 ? 0 : cdiv(D.ncur, 128);
  int h, n_iter, cnt, qbA = 0, qbB = -1;
  const uint32_t* entries;                          // key plan, or list of query blocks
  KeyTile kt{};
  int d0;                                           // tiles before this one are dense
  if (is_dq) {
    const int t = tile % ntiles;
    h = tile / ntiles;
    qbA = BLK == 64 ? 2 * t : t;
    if (BLK == 64 && 2 * t + 1 < D.nqb) qbB = 2 * t + 1;
    cnt = P.plan_cnt[tile];
    entries = P.plan + (size_t)tile * plan_stride(D);
    d0 = n_dense;
    n_iter = d0 + (BLK == 64 ? cdiv(cnt, 2) : cnt);
  } else {
    kt = key_tile_of(tile, P.kt, D);
    h = kt.h;
    if (kt.list < 0) {
      cnt = 0;
      entries = nullptr;
      n_iter = d0 = cdiv(D.ncur, 128);
    } else {
      cnt = P.inv_cnt[kt.list];
      entries = P.inv + P.inv_off[kt.list];
      d0 = 0;
      n_iter = BLK == 64 ? cdiv(cnt, 2) : cnt;
    }
  }

  // nothing to stream (a key tile that no query attends to): zeros, without the machinery
  if (n_iter == 0) {
    for (int i = threadIdx.x; i < 128 * (HD / 8); i += kBwdThreads) {
      const int r = i / (HD / 8), col = h * HD + i % (HD / 8) * 8;
      const uint4 zero = make_uint4(0, 0, 0, 0);
      if (is_dq) {
        const int qb = BLK == 64 && r >= 64 ? qbB : qbA, i0 = BLK == 64 ? r & 63 : r;
        if (qb < 0 || i0 >= block_len(D, qb % D.nbpf)) continue;
        const size_t tok = (size_t)(qb / D.nbpf) * D.T + (qb % D.nbpf) * BLK + i0;
        *reinterpret_cast<uint4*>(P.dq + tok * D.H * HD + col) = zero;
      } else if (kt.row + r < D.T) {                // only tiles with lists can be empty
        const bool cur = kt.kind == 2;
        const size_t at = ((size_t)(cur ? kt.frame : P.slots[D.S + kt.frame]) * D.T + kt.row + r) * D.H * HD + col;
        *reinterpret_cast<uint4*>((cur ? P.dk_cur : P.dk_cache) + at) = zero;
        *reinterpret_cast<uint4*>((cur ? P.dv_cur : P.dv_cache) + at) = zero;
      }
    }
    return;
  }

  if (threadIdx.x == 0) {
    for (int i = 0; i < kBbCount; ++i) {
      const bool rows = i == kBbP || i == kBbP + 1 || i == kBbRd || i == kBbDS || i == kBbDS + 1;
      mbar_init(&bars[i], rows ? 8 : i == kBbDone ? 2 : 1);
    }
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(s_tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  constexpr uint32_t tmem = 0;        // all 512 columns are this CTA's: they start at 0
  uint8_t* in0 = smem + L::kIn0;
  uint8_t* in1 = smem + L::kIn1;
  // the window of dynamic shared memory starts on 1024 bytes (swizzled tiles need it)
  const bool run = (smem_u32(smem) & 1023u) == 0;
  if (!run && threadIdx.x == 0) record_status(LF_ERR_CUDA);
  auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_until(bar, parity, deadline); };
  // for what has been issued and has to end before the CTA may exit: a limit of its own
  auto drain = [&](uint64_t* bar, uint32_t parity) {
    if (!wait_until(bar, parity, clock64() + P.wait_limit_clk) && lane == 0) record_status(LF_ERR_TIMEOUT);
  };

  bool ok = run;                      // false for a warp once one of its waits has run out
  if (warp < 4) {
    regs_dec<kBwdLowRegs>();
    const uint32_t lead = elect_lane();
    if (warp == 0 || warp == 2) {
      // ---------------------------------------------------------- TMA issuers
      const bool side0 = warp == 0;                 // Q / K ring and both inputs; else V / dout
      const int n_slot = side0 ? kRing0 : kRing1;
      uint64_t* full = &bars[side0 ? kBbRing0 : kBbRing1];
      uint64_t* empty = full + n_slot;
      uint8_t* ring = smem + (side0 ? L::kR0 : L::kR1);
      const bool stall = P.debug_stall == (int)blockIdx.x + 1;
      if (side0 && run && !stall) {
        expect_if(lead, &bars[kBbIn], 2 * L::kTile);
        if (!is_dq && kt.kind == 0) {
          load_tile_if<HD>(lead, in0, &P.kc2, &bars[kBbIn], h, kt.row);
          load_tile_if<HD>(lead, in1, &P.vc2, &bars[kBbIn], h, kt.row);
        } else {
          for (int box = 0; box < 2; ++box) {
            int f, row;
            if (is_dq) {
              const int qb = BLK == 64 && box ? qbB : qbA;
              f = qb >= 0 ? qb / D.nbpf : D.Fc;                // frame Fc reads as zeros
              row = qb >= 0 ? (qb % D.nbpf) * BLK + (BLK == 128 ? box * 64 : 0) : 0;
            } else {
              f = kt.kind == 2 ? kt.frame : P.slots[kt.kind == 1 ? kt.frame : D.S + kt.frame];
              row = kt.row + box * 64;
            }
            load_box_if<HD>(lead, in0, box, is_dq ? &P.q3 : kt.kind == 2 ? &P.kc3 : &P.kh,
                            &bars[kBbIn], h, row, f);
            load_box_if<HD>(lead, in1, box, is_dq ? &P.g3 : kt.kind == 2 ? &P.vc3 : &P.vh,
                            &bars[kBbIn], h, row, f);
          }
        }
      }
      int j = 0, slot = 0, rnd = 0;
#pragma unroll 1
      for (; run && j < n_iter; ++j) {
        if (rnd > 0 && !(ok = wait(&empty[slot], (rnd & 1) ^ 1))) break;
        // the row values' buffer of tile j - 2 has been read
        const bool cols = !is_dq && side0;
        if (cols && j >= 2 && !(ok = wait(&bars[kBbDS + (j & 1)], ((j >> 1) & 1) ^ 1))) break;
        expect_if(lead, &full[slot], L::kTile + (cols ? 2 * kBoxFloats * 4 : 0));
        uint8_t* dst = ring + slot * L::kTile;
        float* col = reinterpret_cast<float*>(smem + L::kCols) + (j & 1) * 2 * kBoxFloats;
        if (j < d0) {
          if (is_dq) {
            load_tile_if<HD>(lead, dst, side0 ? &P.kc2 : &P.vc2, &full[slot], h, j * 128);
          } else {
            load_tile_if<HD>(lead, dst, side0 ? &P.q2 : &P.g2, &full[slot], h, j * 128);
            if (cols)
              bulk_load_if(lead, col,
                           P.rows.dense + ((size_t)h * bwd_dense_boxes(D) + 2 * j) * kBoxFloats,
                           2 * kBoxFloats * 4, &full[slot]);
          }
        } else {
          for (int box = 0; box < 2; ++box) {
            const int e = BLK == 64 ? 2 * (j - d0) + box : j - d0;
            const uint32_t pe = e < cnt ? entries[e] : 0u;
            int f = D.Fc, row = 0;                             // past the end: zeros
            if (is_dq) {
              bool cached = false;
              if (e < cnt) {
                const int p = (int)(pe >> 16);
                row = (int)((pe >> 4) & 0xFFFu) * BLK + (BLK == 128 ? box * 64 : 0);
                cached = p < D.S + D.F;
                f = cached ? P.slots[p] : p - (D.S + D.F);
              }
              load_box_if<HD>(lead, dst, box,
                              cached ? (side0 ? &P.kh : &P.vh) : (side0 ? &P.kc3 : &P.vc3),
                              &full[slot], h, row, f);
            } else {
              size_t at = (size_t)D.H * bwd_blk_boxes(D);      // the box of padding
              if (e < cnt) {
                const int qb = (int)(pe >> 2);
                f = qb / D.nbpf;
                row = (qb % D.nbpf) * BLK + (BLK == 128 ? box * 64 : 0);
                at = (size_t)h * bwd_blk_boxes(D) + (BLK == 128 ? 2 * qb + box : qb);
              }
              load_box_if<HD>(lead, dst, box, side0 ? &P.q3 : &P.g3, &full[slot], h, row, f);
              if (cols)
                bulk_load_if(lead, col + box * kBoxFloats, P.rows.blk + at * kBoxFloats,
                             kBoxFloats * 4, &full[slot]);
            }
          }
        }
        if (++slot == n_slot) { slot = 0; ++rnd; }
      }
      // every copy issued lands before the CTA may exit
      if (run && side0 && !stall) drain(&bars[kBbIn], 0);
      for (int x = max(0, j - n_slot); x < j; ++x)
        drain(&full[x % n_slot], (x / n_slot) & 1);
    } else {
      // ---------------------------------------------------------- MMA issuers
      const uint32_t a0 = smem_u32(in0), a1 = smem_u32(in1);
      const uint32_t r0 = smem_u32(smem + L::kR0), r1 = smem_u32(smem + L::kR1);
      uint64_t* f0 = &bars[kBbRing0];
      uint64_t* e0 = f0 + kRing0;
      uint64_t* f1 = &bars[kBbRing1];
      uint64_t* e1 = f1 + kRing1;
      auto ring0 = [&](int j) { return wait(&f0[j % kRing0], (j / kRing0) & 1); };
      auto ring1 = [&](int j) { return wait(&f1[j % kRing1], (j / kRing1) & 1); };
      auto slot0 = [&](int j) { return r0 + (j % kRing0) * L::kTile; };
      auto slot1 = [&](int j) { return r1 + (j % kRing1) * L::kTile; };
      ok = run && wait(&bars[kBbIn], 0);
      if (warp == 1) {
        // dq: S of tile j - 1 ahead; dP over dP of tile j - 1, once that is read; S over dS of
        // tile j - 1, once that is consumed.  dk, dv: dP over P and dS of tile j - 1, once they
        // are consumed; S over dP of tile j, once that is read.
#pragma unroll 1
        for (int j = is_dq ? -2 : -1; ok && j < n_iter; ++j) {
          const int jp = is_dq ? j + 1 : j, js = is_dq ? j + 2 : j + 1;
          if (jp >= 0 && jp < n_iter) {
            ok = ring1(jp) && (is_dq ? j < 0 || wait(&bars[kBbRd], j & 1)
                                     : j == 0 || wait(&bars[kBbAcc + ((j - 1) & 1)], ((j - 1) >> 1) & 1));
            if (!ok) break;
            tc_fence_after();
            mma_scores<HD>(lead, tmem + (is_dq ? L::kDP : j & 1 ? L::kX0 : L::kX1), a1, slot1(jp));
            commit_if(lead, &bars[kBbDP + (jp & 1)]);
            if (is_dq) commit_if(lead, &e1[jp % kRing1]);
          }
          if (js < n_iter) {
            ok = ring0(js) && (is_dq ? j < 0 || wait(&bars[kBbAcc + (j & 1)], (j >> 1) & 1)
                                     : j < 0 || wait(&bars[kBbRd], j & 1));
            if (!ok) break;
            tc_fence_after();
            mma_scores<HD>(lead, tmem + (is_dq ? (js & 1 ? L::kS1 : L::kS0) : js & 1 ? L::kX1 : L::kX0), a0,
                           slot0(js));
            commit_if(lead, &bars[kBbS + (js & 1)]);
          }
        }
      } else if (is_dq) {
#pragma unroll 1
        for (int j = 0; ok && j < n_iter; ++j) {
          ok = ring0(j) && wait(&bars[kBbDS + (j & 1)], (j >> 1) & 1);
          if (!ok) break;
          tc_fence_after();
          mma_accumulate<HD>(lead, tmem + L::kAcc0, tmem + (j & 1 ? L::kS1 : L::kS0), 64, slot0(j), j > 0);
          commit_if(lead, &bars[kBbAcc + (j & 1)]);
          commit_if(lead, &e0[j % kRing0]);
        }
      } else {
#pragma unroll 1
        for (int j = 0; ok && j < n_iter; ++j) {
          const uint32_t x = tmem + (j & 1 ? L::kX1 : L::kX0);
          ok = ring1(j) && wait(&bars[kBbP + (j & 1)], (j >> 1) & 1);
          if (!ok) break;
          tc_fence_after();
          mma_accumulate<HD>(lead, tmem + L::kAcc1, x, 64, slot1(j), j > 0);
          ok = ring0(j) && wait(&bars[kBbDS + (j & 1)], (j >> 1) & 1);
          if (!ok) break;
          tc_fence_after();
          mma_accumulate<HD>(lead, tmem + L::kAcc0, x + 32, 64, slot0(j), j > 0);
          commit_if(lead, &bars[kBbAcc + (j & 1)]);
          commit_if(lead, &e0[j % kRing0]);
          // dout's slot only now: dP, the other issuer's, may end after dv, but dS follows it
          commit_if(lead, &e1[j % kRing1]);
        }
      }
      commit_if(lead, &bars[kBbDone]);
    }
  } else {
    regs_inc<kBwdHighRegs>();
    // ------------------------------------------------------------ P and dS
    const int wg = (warp - 4) >> 2;
    const int r = (warp & 3) * 32 + lane;           // row = tensor-memory lane
    const uint32_t t_row = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const float c = D.scale * 1.4426950408889634f;
    if (is_dq) {
      const uint32_t bit = (BLK == 64 && r >= 64) ? 2u : 1u;
      const int qb = BLK == 64 ? (r < 64 ? qbA : qbB) : qbA, i0 = BLK == 64 ? (r & 63) : r;
      const bool valid = qb >= 0 && i0 < block_len(D, qb % D.nbpf);
      const int tok = valid ? (qb / D.nbpf) * D.T + (qb % D.nbpf) * BLK + i0 : 0;
      float nl = -INFINITY, nd = 0.f;
      if (valid) {
        const float* b = P.rows.dense + ((size_t)h * bwd_dense_boxes(D) + tok / 64) * kBoxFloats + tok % 64;
        nl = b[0];
        nd = b[64];
      }
      // valid key columns of this half of tile j for this row (the same for a warp's rows),
      // read one tile ahead
      auto columns = [&](int j) {
        if (j >= n_iter) return 0;
        if (j < d0) return max(0, min(64, D.ncur - j * 128 - wg * 64));
        const int e = BLK == 64 ? 2 * (j - d0) + wg : j - d0;
        const uint32_t pe = e < cnt ? entries[e] : 0u;
        const int len = (pe & bit) ? block_len(D, (pe >> 4) & 0xFFF) : 0;
        return BLK == 64 ? len : max(0, min(64, len - wg * 64));
      };
      int v_next = columns(0);
#pragma unroll 1
      for (int j = 0; ok && j < n_iter; ++j) {
        const int v = v_next;
        v_next = columns(j + 1);
        const uint32_t s_col = t_row + (j & 1 ? L::kS1 : L::kS0) + wg * 64;
        if (!(ok = wait(&bars[kBbS + (j & 1)], (j >> 1) & 1))) break;
        tc_fence_after();
        float s[64], g[64];
        if (v > 0) {
          tmem_ld32(s_col, s);
          tmem_ld32(s_col + 32, s + 32);
          tmem_ld_wait();
          reg_fence32(s);
          reg_fence32(s + 32);
#pragma unroll
          for (int i = 0; i < 64; ++i) s[i] = ex2_approx(fmaf(s[i], c, nl));
          if (v < 64) {                             // keys past the block's end
#pragma unroll
            for (int i = 0; i < 64; ++i)
              if (i >= v) s[i] = 0.f;
          }
        }
        if (!(ok = wait(&bars[kBbDP + (j & 1)], (j >> 1) & 1))) break;
        tc_fence_after();
        if (v > 0) {
          tmem_ld32(t_row + L::kDP + wg * 64, g);
          tmem_ld32(t_row + L::kDP + wg * 64 + 32, g + 32);
          tmem_ld_wait();
          reg_fence32(g);
          reg_fence32(g + 32);
        }
        warp_arrive(&bars[kBbRd]);
#pragma unroll
        for (int ch = 0; ch < 2; ++ch) {
          float pk[16];
          const float *p = s + ch * 32, *x = g + ch * 32;
#pragma unroll
          for (int i = 0; i < 16; ++i)
            pk[i] = v > 0 ? pack_bf16(p[2 * i] * (x[2 * i] + nd), p[2 * i + 1] * (x[2 * i + 1] + nd)) : 0.f;
          tmem_st16(s_col + ch * 16, pk);
        }
        tmem_st_wait();
        warp_arrive(&bars[kBbDS + (j & 1)]);
      }
      if (run) ok = wait(&bars[kBbDone], 0) && ok;
      tc_fence_after();
      // 64 channels each (d = 64: the first warpgroup alone), over Q, which no MMA reads any more
      const bool mine = HD == 128 || wg == 0;
      if (mine && ok) {
        stage_row<64>(in0 + wg * L::kRegion, r, t_row + L::kAcc0 + wg * 64, D.scale);
        fence_proxy_async_smem();
      }
      named_bar_sync(kNbStore + wg, 128);
      if (mine && ok && r < 2) {   // a box each
        const int q2 = BLK == 64 && r ? qbB : qbA, row = (q2 % D.nbpf) * BLK + (BLK == 128 ? r * 64 : 0);
        if (q2 >= 0 && row < D.T)
          store_box(in0 + wg * L::kRegion + r * 64 * 128, &P.dq3, h * HD + wg * 64, row, q2 / D.nbpf);
        stores_read();
      }
    } else {
      const uint32_t bit = r < 64 ? 1u : 2u;
      auto entry = [&](int j) {                     // dense: every row attends
        const int e = BLK == 64 ? 2 * j + wg : j;
        return j < d0 ? 3u : j < n_iter && e < cnt ? entries[e] : 0u;
      };
      uint32_t pe = entry(0);
#pragma unroll 1
      for (int j = 0; ok && j < n_iter; ++j) {
        const bool on = (pe & bit) != 0;
        pe = entry(j + 1);
        const uint32_t s_col = t_row + (j & 1 ? L::kX1 : L::kX0) + wg * 64;
        const uint32_t p_col = t_row + (j & 1 ? L::kX0 : L::kX1) + wg * 64;
        const float4* nl4 = reinterpret_cast<const float4*>(
            smem + L::kCols + ((j & 1) * 2 + wg) * kBoxFloats * 4);
        // the row values came with the ring slot that S is computed from; the issuer of S
        // has waited for it, their readers have to as well (asynchronous copies)
        ok = wait(&bars[kBbRing0 + j % kRing0], (j / kRing0) & 1) &&
             wait(&bars[kBbS + (j & 1)], (j >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        float s[64];
        if (on) {
          tmem_ld32(s_col, s);
          tmem_ld32(s_col + 32, s + 32);
          tmem_ld_wait();
          reg_fence32(s);
          reg_fence32(s + 32);
#pragma unroll
          for (int i = 0; i < 64; i += 4) {
            const float4 n = nl4[i / 4];
            s[i] = ex2_approx(fmaf(s[i], c, n.x));
            s[i + 1] = ex2_approx(fmaf(s[i + 1], c, n.y));
            s[i + 2] = ex2_approx(fmaf(s[i + 2], c, n.z));
            s[i + 3] = ex2_approx(fmaf(s[i + 3], c, n.w));
          }
        }
#pragma unroll
        for (int ch = 0; ch < 2; ++ch) {
          float pk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e)
            pk[e] = on ? pack_bf16(s[ch * 32 + 2 * e], s[ch * 32 + 2 * e + 1]) : 0.f;
          tmem_st16(s_col + ch * 16, pk);
        }
        tmem_st_wait();
        warp_arrive(&bars[kBbP + (j & 1)]);
        if (!(ok = wait(&bars[kBbDP + (j & 1)], (j >> 1) & 1))) break;
        tc_fence_after();
        float g[64];
        if (on) {
          tmem_ld32(p_col, g);
          tmem_ld32(p_col + 32, g + 32);
          tmem_ld_wait();
          reg_fence32(g);
          reg_fence32(g + 32);
        }
        warp_arrive(&bars[kBbRd]);
#pragma unroll
        for (int ch = 0; ch < 2; ++ch) {
          float pk[16];
          if (on) {
#pragma unroll
            for (int i = ch * 32; i < ch * 32 + 32; i += 4) {
              const float4 n = nl4[16 + i / 4];
              pk[(i & 31) / 2] = pack_bf16(s[i] * (g[i] + n.x), s[i + 1] * (g[i + 1] + n.y));
              pk[(i & 31) / 2 + 1] = pack_bf16(s[i + 2] * (g[i + 2] + n.z), s[i + 3] * (g[i + 3] + n.w));
            }
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) pk[e] = 0.f;
          }
          tmem_st16(s_col + 32 + ch * 16, pk);
        }
        tmem_st_wait();
        warp_arrive(&bars[kBbDS + (j & 1)]);
      }
      if (run) ok = wait(&bars[kBbDone], 0) && ok;
      tc_fence_after();
      // dk over K and dv over V, which no MMA reads any more
      uint8_t* out = wg == 0 ? in0 : in1;
      if (ok) {
        stage_row<HD>(out, r, t_row + (wg == 0 ? L::kAcc0 : L::kAcc1), wg == 0 ? D.scale : 1.f);
        fence_proxy_async_smem();
      }
      named_bar_sync(kNbStore + wg, 128);
      if (ok && r < 2) {                            // a box each
        const int row = kt.row + r * 64;
        const int f = kt.kind == 0 ? -1 : kt.kind == 2 ? kt.frame
                                        : P.slots[kt.kind == 1 ? kt.frame : D.S + kt.frame];
        const CUtensorMap* m = wg == 0 ? (kt.kind == 0 ? &P.dk2 : kt.kind == 2 ? &P.dk3 : &P.dkh)
                                       : (kt.kind == 0 ? &P.dv2 : kt.kind == 2 ? &P.dv3 : &P.dvh);
        if (row < (kt.kind == 0 ? D.ncur : D.T))
          for (int c = 0; c < L::NH; ++c)
            store_box(out + c * L::kRegion + r * 64 * 128, m, h * HD + c * 64, row, f);
        stores_read();
      }
    }
    tc_fence_before();
  }
  if (run && !ok && lane == 0) record_status(LF_ERR_TIMEOUT);
  __syncthreads();
  if (warp == 1) {
    drain(&bars[kBbDone], 0);
    tc_fence_after();
    tmem_dealloc(*s_tmem, 512);
  }
}

template <int HD, int BLK>
__global__ void __launch_bounds__(kBwdThreads, 1)
attn_bwd_kernel(const __grid_constant__ BwdParams P, const Dims D) {
  if ((int)blockIdx.x < P.n_dq) bwd_tile<HD, BLK, true>(P, D, blockIdx.x);
  else bwd_tile<HD, BLK, false>(P, D, blockIdx.x - P.n_dq);
}

}  // namespace lf
