// cache_attn_rows.cu -- attention over the 8-bit K/V cache for few query rows per KV head (single
// tokens, a few tokens, heads that share a KV head), and for fp32 queries of any number.
//
// For each request b, KV head and the R = (H / Hk) * Nq query rows that share it:
//   lse_i = ln sum_{j < lens[b]} exp(scale q_i . k_j),  o_i = sum_j exp(s_ij - lse_i) v_j,
// k_j = code * scale of its 64-token block.  Consecutive query heads share a KV head, so the R rows
// are contiguous in q and o.
//
// Bound by reading the codes once: 2 D bytes per (token, KV head).  Up to 8 query rows cost the
// same as one, so a shared KV head is read once for all its query heads.
//
// Work is shared out by the lengths that the requests have: the cache blocks (64 tokens) of all
// units (request, KV head, 16-row tile) in a row are cut into equal shares, one per resident
// block of threads, so one launch is one full wave whatever the lengths.  A share may begin and
// end inside a unit; each piece writes its state in fp32 to a slot of its own and the join adds a
// unit's pieces in order, so results do not depend on the order in which blocks run.  (Equal
// numbers of splits per request instead: a batch with lengths from 0 to 4096 took 26 us for 55 MB,
// nearly half of it on the longest request's blocks.)  Short caches are not cut: blocks take whole
// units, and there is no join.
//
// Each warp takes 16 tokens of every block and runs two tiles ahead with TMA loads into a ring of
// its own: no barrier between warps in the loop, 128 KB in flight per SM.  (Plain and asynchronous
// 16-byte loads by the lanes moved the same bytes but filled the load-store queue: 56 us for the
// 236 MB of one 115200-token cache.)
//
// Tokens (and then channels) are the products' 16 rows and queries their 8 columns, so up to 8
// queries cost the same; 16-query tiles take two columns' worth.  Codes become product operands
// without shared-memory transposes because the inner index of a product may be permuted if both
// operands agree, and the outer one if the result is read accordingly:
//   S^T = K Q^T: lane (g, t) takes 16 bytes of tokens x(g) and 8 + x(g) per 64 channels, four per
//     k-step, and q is laid out the same way; x = token_of permutes 0..7 so that these reads and
//     those of V fall in different banks of the swizzled tile.  Codes go to f16, which holds every e4m3 value exactly; q is
//     scaled per row by a power of two so that its largest element is in [1, 2), exact in f16 but
//     for elements below 2^-14 of the largest (off by at most 2^-25 of it).  The block's scale
//     multiplies the fp32 score.
//   O^T += V^T P^T: lane (g, t) takes channels g D/8 .. of tokens x(2t), x(2t + 1) and 8 more; P^T
//     is the scores' fragment transposed.  Weights are held as 2^7 p vs / vmax (vmax: the piece's
//     largest scale; p <= 2^8) and rounded to f16: 2^-11 relative, or 2^-32 of the row's largest
//     weight where that is more.  A block whose scale is below 2^-16 of vmax would lose small
//     weights that way: it takes bf16 (2^-8, any magnitude) instead.
// fp32 queries take two f16 terms for each element of q and each weight (three bf16 ones in small
// blocks): 22 bits, for twice the products and the same conversions.  O errs by 1e-7 to 1e-6 of its
// norm (512 to 131072 tokens; plain fp32 sums: the same), up to 3e-6 where scores reach 20.
// The conversions (about 0.9 instructions per code) are most of the work: the 236 MB of one
// 115200-token cache take 49 us (53 with the join), with the issue slots and the ALU half busy and
// DRAM at 60%; what is left is the chain of a tile's steps in the 16 warps that registers allow.  With
// queries as the 16 rows and V in bf16 throughout they were 1.6 per code: 64 us, 46% of DRAM.
#include <cuda_fp16.h>

#include "pa_device.cuh"
#include "pa_launch.h"

namespace pa {
namespace {

constexpr int kWarps = 4;
constexpr int kTok = 16;               // tokens per tile
constexpr int kStages = 3;             // tiles in shared memory per warp
// What a piece costs besides its blocks, in blocks.  us with 0 / 2 / 4 / 8: 8 x 24 heads of up to 4096
// tokens 45 / 29.5 / 28.6 / 28.5, 64 x 8 heads of up to 2048 53.5 / 39.7 / 37.1 / 38.1.
constexpr int kPieceCost = 4;
// Places per share, at least.  us with 5 / 6 / 9 / 16: 8 heads x 1024 tokens 9.3 / 10.0 / 11.7 / 15.6,
// 2 x 4 heads x 3000 tokens 9.4 / 9.4 / 10.7 / 13.8.
constexpr int kMinPlaces = 6;
static_assert(kWarps * kTok == PA_CACHE_BLOCK, "the warps share one cache block");
constexpr float kUnit = 128.0f;        // weights are held as this times p vs / vmax
constexpr float kSmallScale = 1.0f / 65536.0f;

// Query rows in all up to which the join takes a block of threads per row instead of a warp.  us, block
// against warp: 40 rows x 115200 tokens 60 / 78, 256 rows x 8192 19.5 / 23.9, 1280 x 8192 47.3 / 45.4,
// 2048 x 8192 70.5 / 65.0.
constexpr int kWideRows = 1024;
constexpr int kMaxRows = 16;           // queries per tile: NT columns of 8, NT = 1 or 2 (fp32: 1)
template <typename T>
__host__ __device__ constexpr int row_columns(int R) { return R <= 8 || sizeof(T) == 4 ? 1 : 2; }
// Blocks of threads per SM, by registers.
template <typename T>
__host__ __device__ constexpr int resident(int nt) { return nt == 1 && sizeof(T) == 2 ? 4 : 3; }
constexpr float kLow = 4096.0f;        // the second f16 term of q is held times this
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleLog2 = 8.0f;   // move the running max only when it grows by more

__device__ __forceinline__ uint32_t f16x2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float2 f16_values(uint32_t f16) { return __half22float2(*reinterpret_cast<const __half2*>(&f16)); }

__device__ __forceinline__ uint32_t to_bf16(uint32_t f16) {
  const float2 f = f16_values(f16);
  return pack_bf16x2(f.x, f.y);
}

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

// Transpose of an 8 x 8 matrix of 16-bit elements held as a product fragment.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Token (of 8) in row g of the scores' fragment.  Rows 2t and 2t + 1 differ in bits 0 and 2, and
// over t either keeps bits 1 and 2 distinct.
__device__ __forceinline__ int token_of(int g) { return g & 1 ? ((g - 1) ^ 4) + 1 : g; }

// Tiles of 16 tokens as TMA writes them: K's codes, then V's; rows of D bytes, 16-byte chunks
// swizzled over 128 bytes (D = 128: chunk ^ row % 8) or 64 (D = 64: chunk ^ row / 2 % 4).
template <int D>
struct Ring {
  static constexpr int kVBytes = D / 8;              // a lane's bytes of a V row
  static constexpr int kPart = kTok * D;
  static constexpr int kTile = 2 * kPart;
  static constexpr int kSums = kMaxRows * (D + 4) * 4;         // the warp's sums reuse its ring
  static constexpr int kWarpBytes = ((kStages * kTile > kSums ? kStages * kTile : kSums) + 1023) / 1024 * 1024;
  static constexpr int kBytes = kWarps * kWarpBytes + 1024;

  static __device__ __forceinline__ int offset(int row, int byte) {
    const int sw = D == 128 ? row & 7 : (row >> 1) & 3;
    return row * D + (byte ^ (sw << 4));
  }
};

// ------------------------------------------------------------------ shares of the work
// Unit u = (b * Hk + h) * row_tiles + r has the cache blocks of request b.  In the row of all units
// it takes kPieceCost more places before its first block: what a piece costs besides its blocks
// (its queries, its join), so that a share of many short units is not longer than others.  All
// whole-warp functions.
struct Share {
  long long total;      // places of all units
  long long size;       // places per share
};

__device__ __forceinline__ int request_blocks(const CacheAttnParams& prm, int b) {
  return (cache_len(prm, b) + PA_CACHE_BLOCK - 1) / PA_CACHE_BLOCK;
}
__device__ __forceinline__ int unit_places(int blocks) { return blocks > 0 ? blocks + kPieceCost : 0; }

// The lengths of 32 requests at a time, one per lane: up to 32 requests are read once.
struct Requests {
  const CacheAttnParams& prm;
  int lane, base, nb;                    // request base + lane has nb blocks
  long long upto, sum;                   // places (of one KV head and row tile) up to and with it; of all 32
  __device__ __forceinline__ Requests(const CacheAttnParams& p, int l) : prm(p), lane(l) { read(0); }
  __device__ __forceinline__ void read(int b0) {
    base = b0;
    nb = b0 + lane < prm.B ? request_blocks(prm, b0 + lane) : 0;
    upto = unit_places(nb);
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, upto, off);
      if (lane >= off) upto += y;
    }
    sum = __shfl_sync(0xffffffffu, upto, 31);
  }
  __device__ __forceinline__ int blocks(int b) {
    if ((b & ~31) != base) read(b & ~31);
    return __shfl_sync(0xffffffffu, nb, b & 31);
  }
  __device__ __forceinline__ long long before(int b) {           // places of requests [0, b)
    long long acc = 0;
    for (int b0 = 0; b0 < b; b0 += 32) {
      if (base != b0) read(b0);
      acc += b0 + 32 <= b ? sum : __shfl_sync(0xffffffffu, upto, (b - 1) & 31);
    }
    return acc;
  }
  // Request that holds place x of all requests (x in units of one KV head and row tile), and its first.
  __device__ __forceinline__ int find(long long x, long long& first) {
    long long acc = 0;
    for (int b0 = 0;; b0 += 32) {
      if (base != b0) read(b0);
      const uint32_t hit = __ballot_sync(0xffffffffu, acc + upto > x);
      if (hit) {
        const int l = __ffs(hit) - 1;
        first = acc + __shfl_sync(0xffffffffu, upto - unit_places(nb), l);
        return b0 + l;
      }
      acc += sum;
    }
  }
};

__device__ __forceinline__ Share work_share(const CacheAttnParams& prm, Requests& req) {
  Share s;
  s.total = req.before(prm.B) * prm.Hk * prm.row_tiles;
  s.size = max((s.total + prm.shares - 1) / prm.shares, static_cast<long long>(kMinPlaces));
  return s;
}

// ------------------------------------------------------------------ one piece of a unit
// A place in a ring and the parity of the tile there.
struct Slot {
  int i = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++i == kStages) {
      i = 0;
      phase ^= 1;
    }
  }
};

struct Shared {
  uint64_t full[kWarps][kStages];
  int abort_flag;
  float m[kWarps][kMaxRows], l[kWarps][kMaxRows];
};

// Blocks [blk0, blk1) of unit `unit`.  `slot` < 0: the piece is the whole unit and its state is
// the result; else it goes to that slot of the scratch.
template <typename T, int D, int NT>
__device__ __forceinline__ bool attend_piece(const CacheAttnRowsParams& par, uint8_t* smem, Shared& sh, Slot& into, Slot& from,
                                             long long unit, int len, int blk0, int blk1, long long slot) {
  const CacheAttnParams& prm = par.c;
  constexpr bool kF32 = sizeof(T) == 4;
  constexpr int kTerms = kF32 ? 2 : 1;   // f16 terms of q and of the weights
  static_assert(!kF32 || NT == 1, "fp32 sums by the tile hold one column block");
  constexpr int kRows = 8 * NT;
  constexpr int kSteps = D / 16;         // k-steps of S^T; 16-channel blocks of O^T
  using R = Ring<D>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const long long bh = unit / prm.row_tiles;
  const int row0 = static_cast<int>(unit - bh * prm.row_tiles) * kRows;
  const int end = min(blk1 * PA_CACHE_BLOCK, len);
  const float* k_scale = prm.k_scale + static_cast<size_t>(bh) * prm.blocks;
  const float* v_scale = prm.v_scale + static_cast<size_t>(bh) * prm.blocks;
  uint8_t* ring = smem + warp * R::kWarpBytes;
  const uint32_t ring_u = smem_u32(ring);

  // Tile i of this warp: 16 tokens of block blk0 + i.
  const int tok0 = blk0 * PA_CACHE_BLOCK + warp * kTok;
  const int n = blk1 - blk0;
  const uint32_t full = smem_u32(&sh.full[warp][0]);
  auto fetch = [&](int tok) {              // lane 0; the slot is free
    const uint32_t bar = full + 8u * into.i, dst = ring_u + into.i * R::kTile;
    mbar_expect_tx(bar, R::kTile);
    tma_load_3d(dst, &par.tm_k, 0, tok, static_cast<int>(bh), bar);
    tma_load_3d(dst + R::kPart, &par.tm_v, 0, tok, static_cast<int>(bh), bar);
  };
#pragma unroll
  for (int i = 0; i < kStages - 1; ++i)
    if (i < n) {
      if (lane == 0) fetch(tok0 + i * PA_CACHE_BLOCK);
      into.next();
    }
  // Scales: 32 blocks' in the lanes, the next 32 blocks' on their way.
  float ks_next = 0.0f, vs_next = 0.0f;
  auto load_scales = [&](int blk) {
    const bool in = blk + lane < blk1;
    ks_next = in ? __ldg(k_scale + blk + lane) : 0.0f;
    vs_next = in ? __ldg(v_scale + blk + lane) : 0.0f;
  };
  load_scales(blk0);
  float ks = ks_next, vs = vs_next;
  load_scales(blk0 + 32);
  float vmax = fmaxf(vs, vs_next);
  for (int i = blk0 + 64 + lane; i < blk1; i += 32) vmax = fmaxf(vmax, __ldg(v_scale + i));

  // q in f16, laid out as the codes are: column g of column block c; fq = softmax scale * log2(e) /
  // the row's power of two, moved to the lanes that hold the row's scores (rows 2t, 2t + 1).
  uint32_t qb[kTerms][NT][kSteps][2];
  float fq[NT][2];
#pragma unroll
  for (int c = 0; c < NT; ++c) {
    const int r = row0 + 8 * c + g;
    float x[D / 4];
    float mx = 0.0f;
    const T* src = static_cast<const T*>(prm.q) + (static_cast<size_t>(bh) * prm.R + min(r, prm.R - 1)) * D + t * 16;
#pragma unroll
    for (int i = 0; i < D / 4; i += 4) {
      const float4 u = load4(src + i / 16 * 64 + i % 16);
      const bool in = r < prm.R;
      x[i] = in ? u.x : 0.0f;
      x[i + 1] = in ? u.y : 0.0f;
      x[i + 2] = in ? u.z : 0.0f;
      x[i + 3] = in ? u.w : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < D / 4; ++i) mx = fmaxf(mx, fabsf(x[i]));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    // 2^e, e = exponent of the largest element, kept where 2^-e and 2^e are normal
    const int e = min(max(static_cast<int>(__float_as_uint(mx) >> 23), 2), 252) - 127;
    const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    const float f = prm.scale * kLog2e * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
    fq[c][0] = __shfl_sync(0xffffffffu, f, 8 * t);              // lane (2t, 0)
    fq[c][1] = __shfl_sync(0xffffffffu, f, 8 * t + 4);          // lane (2t + 1, 0)
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float a = x[4 * s + 2 * i] * down, b = x[4 * s + 2 * i + 1] * down;
        qb[0][c][s][i] = f16x2(a, b);
        if (kF32) {
          const float2 h = f16_values(qb[0][c][s][i]);
          qb[kTerms - 1][c][s][i] = f16x2((a - h.x) * kLow, (b - h.y) * kLow);
        }
      }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, off));
  if (vmax == 0.0f) vmax = 1.0f;
  const float vinv = 1.0f / vmax;

  // o[c][b][2 h + e]: row 8 c + 2 t + e, channel g D/8 + 2 b + h; m, l: rows 8 c + 2 t + e.
  float o[NT][kSteps][4];
  float m[NT][2], l[NT][2];
#pragma unroll
  for (int c = 0; c < NT; ++c) {
    m[c][0] = m[c][1] = -INFINITY;
    l[c][0] = l[c][1] = 0.0f;
#pragma unroll
    for (int b = 0; b < kSteps; ++b) o[c][b][0] = o[c][b][1] = o[c][b][2] = o[c][b][3] = 0.0f;
  }
  const int xg = token_of(g);
  bool ok = true;
  for (int i = 0; i < n; ++i) {
    const int tok = tok0 + i * PA_CACHE_BLOCK;
    if (i + kStages - 1 < n) {
      __syncwarp();                        // every lane has read the slot's last tile
      if (lane == 0) fetch(tok + (kStages - 1) * PA_CACHE_BLOCK);
      into.next();
    }
    if (i % 32 == 0 && i > 0) {
      ks = ks_next;
      vs = vs_next;
      load_scales(blk0 + i + 32);
    }
    const float ks_now = __shfl_sync(0xffffffffu, ks, i % 32), ratio = __shfl_sync(0xffffffffu, vs, i % 32) * vinv;
    if (!(ok = mbar_wait_warp(full + 8u * from.i, from.phase, &sh.abort_flag, prm.status))) break;
    const uint8_t* tile = ring + from.i * R::kTile;
    from.next();
    if (tok >= end) continue;              // a warp without tokens in the last block

    float s[NT][4] = {}, s2[NT][4] = {};       // two chains of products; fp32: of q's two terms
#pragma unroll
    for (int a = 0; a < D / 64; ++a) {
      const uint4 u0 = *reinterpret_cast<const uint4*>(tile + R::offset(xg, a * 64 + t * 16));
      const uint4 u1 = *reinterpret_cast<const uint4*>(tile + R::offset(8 + xg, a * 64 + t * 16));
      const uint32_t w0[4] = {u0.x, u0.y, u0.z, u0.w}, w1[4] = {u1.x, u1.y, u1.z, u1.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t k[4];
        e4m3_to_f16(w0[e], k[0], k[2]);
        e4m3_to_f16(w1[e], k[1], k[3]);
#pragma unroll
        for (int c = 0; c < NT; ++c) {
          mma_f16(!kF32 && (e & 1) ? s2[c] : s[c], k, qb[0][c][4 * a + e]);
          if (kF32) mma_f16(s2[c], k, qb[kTerms - 1][c][4 * a + e]);
        }
      }
    }
#pragma unroll
    for (int c = 0; c < NT; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[c][e] = kF32 ? fmaf(s2[c][e], 1.0f / kLow, s[c][e]) : s[c][e] + s2[c][e];
    const bool partial = tok + kTok > end;
    uint32_t v[4][D / 32];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int x = token_of(2 * t + (b & 1)) + 8 * (b >> 1);
      const uint8_t* src = tile + R::kPart + R::offset(x, g * R::kVBytes);
      if (D == 128) {
        const uint4 u = *reinterpret_cast<const uint4*>(src);
        v[b][0] = u.x; v[b][1] = u.y; v[b][D / 32 - 2] = u.z; v[b][D / 32 - 1] = u.w;
      } else {
        const uint2 u = *reinterpret_cast<const uint2*>(src);
        v[b][0] = u.x; v[b][1] = u.y;
      }
      if (partial && tok + x >= end) {     // weight 0, but 0 times a NaN code is NaN
#pragma unroll
        for (int w = 0; w < D / 32; ++w) v[b][w] = 0u;
      }
    }
    // s[c][2 h + e]: token x(g) + 8 h, row 8 c + 2 t + e
    if (partial) {
#pragma unroll
      for (int c = 0; c < NT; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (tok + xg + 8 * (e >> 1) >= end) s[c][e] = -INFINITY;
    }
    // The running max only has to keep p <= 2^8: a vote on the lanes' own scores decides whether
    // it moves at all, and only then is it reduced over the lanes.
    float p[NT][4];
    bool grow = false;
    float f[NT][2], mt[NT][2];
#pragma unroll
    for (int c = 0; c < NT; ++c)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        f[c][e] = fq[c][e] * ks_now;
        mt[c][e] = fmaxf(s[c][e], s[c][2 + e]) * f[c][e];
        grow |= mt[c][e] > m[c][e] + kRescaleLog2;
      }
    if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
      for (int c = 0; c < NT; ++c) {
        float a[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {      // only rows whose own max grew: a row never depends on its neighbours
          float to = mt[c][e];
          to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, 4));
          to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, 8));
          to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, 16));
          to = to > m[c][e] + kRescaleLog2 ? to : m[c][e];
          a[e] = to > m[c][e] ? fast_exp2(m[c][e] - to) : 1.0f;
          m[c][e] = to;
          l[c][e] *= a[e];
        }
#pragma unroll
        for (int b = 0; b < kSteps; ++b) {
          o[c][b][0] *= a[0];
          o[c][b][1] *= a[1];
          o[c][b][2] *= a[0];
          o[c][b][3] *= a[1];
        }
      }
    }
#pragma unroll
    for (int c = 0; c < NT; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        p[c][e] = fast_exp2(fmaf(s[c][e], f[c][e & 1], -m[c][e & 1]));
        if (partial && tok + xg + 8 * (e >> 1) >= end) p[c][e] = 0.0f;     // also where -inf meets a scale of 0
        l[c][e & 1] += p[c][e];
      }
    // fp32: a tile's products start from zero and are added to O in fp32.  The tensor cores cut their
    // sums, an error of one sign that grows with the tokens (4 heads x 512 queries x 131072 tokens: 7e-5 of
    // O; added 2e-7, as plain fp32 sums, for 1% of the time).
    float part[2][4];
    auto sum = [&](int c, int b) -> float (&)[4] { return kF32 ? part[b & 1] : o[c][b]; };
    auto clear_sums = [&]() {
#pragma unroll
      for (int e = 0; e < 4; ++e) part[0][e] = part[1][e] = 0.0f;
    };
    auto add_sums = [&](int w) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        o[0][2 * w][e] += part[0][e];
        o[0][2 * w + 1][e] += part[1][e];
      }
    };
    const float unit = kUnit * ratio;
    if (ratio >= kSmallScale || !(ratio > 0.0f)) {
      uint32_t pb[kTerms][NT][2];
#pragma unroll
      for (int c = 0; c < NT; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float a = p[c][2 * h] * unit, b = p[c][2 * h + 1] * unit;
          const uint32_t w = f16x2(a, b);
          pb[0][c][h] = transpose8(w);
          if (kF32) {
            const float2 v = f16_values(w);
            pb[kTerms - 1][c][h] = transpose8(f16x2(a - v.x, b - v.y));
          }
        }
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {
        // bytes of two tokens side by side: channels 4 w + {0, 1} and + {2, 3}
        const uint32_t lo01 = __byte_perm(v[0][w], v[1][w], 0x5140), lo23 = __byte_perm(v[0][w], v[1][w], 0x7362);
        const uint32_t hi01 = __byte_perm(v[2][w], v[3][w], 0x5140), hi23 = __byte_perm(v[2][w], v[3][w], 0x7362);
        uint32_t a[4], b[4];
        e4m3_to_f16(lo01, a[0], a[1]);
        e4m3_to_f16(hi01, a[2], a[3]);
        e4m3_to_f16(lo23, b[0], b[1]);
        e4m3_to_f16(hi23, b[2], b[3]);
        if (kF32) clear_sums();
#pragma unroll
        for (int c = 0; c < NT; ++c)
#pragma unroll
          for (int e = 0; e < kTerms; ++e) {
            mma_f16(sum(c, 2 * w), a, pb[e][c]);
            mma_f16(sum(c, 2 * w + 1), b, pb[e][c]);
          }
        if (kF32) add_sums(w);
      }
    } else {
      constexpr int kWide = kF32 ? 3 : 1;
      uint32_t pb[kWide][NT][2];
#pragma unroll
      for (int c = 0; c < NT; ++c)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float a = p[c][2 * h] * unit, b = p[c][2 * h + 1] * unit;
#pragma unroll
          for (int e = 0; e < kWide; ++e) {
            const uint32_t w = pack_bf16x2(a, b);
            pb[e][c][h] = transpose8(w);
            a -= __uint_as_float(w << 16);
            b -= __uint_as_float(w & 0xFFFF0000u);
          }
        }
#pragma unroll
      for (int w = 0; w < D / 32; ++w) {
        const uint32_t lo01 = __byte_perm(v[0][w], v[1][w], 0x5140), lo23 = __byte_perm(v[0][w], v[1][w], 0x7362);
        const uint32_t hi01 = __byte_perm(v[2][w], v[3][w], 0x5140), hi23 = __byte_perm(v[2][w], v[3][w], 0x7362);
        uint32_t a[4], b[4];
        e4m3_to_f16(lo01, a[0], a[1]);
        e4m3_to_f16(hi01, a[2], a[3]);
        e4m3_to_f16(lo23, b[0], b[1]);
        e4m3_to_f16(hi23, b[2], b[3]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          a[i] = to_bf16(a[i]);
          b[i] = to_bf16(b[i]);
        }
        if (kF32) clear_sums();
#pragma unroll
        for (int c = 0; c < NT; ++c)
#pragma unroll
          for (int e = 0; e < kWide; ++e) {
            mma_bf16(sum(c, 2 * w), a, pb[e][c]);
            mma_bf16(sum(c, 2 * w + 1), b, pb[e][c]);
          }
        if (kF32) add_sums(w);
      }
    }
  }

  // Join the warps.  Each warp's sums go over its own ring, which has no load in flight.
  if (!ok && lane == 0)
    for (; from.i != into.i || from.phase != into.phase; from.next()) mbar_drain(full + 8u * from.i, from.phase);
  if (!__syncthreads_and(ok)) return false;
  float* own = reinterpret_cast<float*>(ring);
#pragma unroll
  for (int c = 0; c < NT; ++c)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float x = l[c][e];
      x += __shfl_xor_sync(0xffffffffu, x, 4);
      x += __shfl_xor_sync(0xffffffffu, x, 8);
      x += __shfl_xor_sync(0xffffffffu, x, 16);
      const int r = 8 * c + 2 * t + e;
      if (g == 0) {
        sh.m[warp][r] = m[c][e];
        sh.l[warp][r] = x;
      }
#pragma unroll
      for (int b = 0; b < kSteps; b += 2)
        *reinterpret_cast<float4*>(own + r * (D + 4) + g * (D / 8) + 2 * b) =
            make_float4(o[c][b][e], o[c][b][2 + e], o[c][b + 1][e], o[c][b + 1][2 + e]);
    }
  __syncthreads();
  const int rows = min(kRows, prm.R - row0);
  for (int i = threadIdx.x; i < rows * D / 4; i += kWarps * 32) {
    const int r = i / (D / 4), c = (i % (D / 4)) * 4;
    float mx = sh.m[0][r];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) mx = fmaxf(mx, sh.m[w][r]);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float a = mx > -INFINITY ? fast_exp2(sh.m[w][r] - mx) : 0.0f;    // 0 for a warp without tokens
      const float4 x = *reinterpret_cast<const float4*>(smem + w * R::kWarpBytes + (r * (D + 4) + c) * 4);
      sum = fmaf(a, sh.l[w][r], sum);
      acc.x = fmaf(a, x.x, acc.x);
      acc.y = fmaf(a, x.y, acc.y);
      acc.z = fmaf(a, x.z, acc.z);
      acc.w = fmaf(a, x.w, acc.w);
    }
    const float inv = 1.0f / (kUnit * sum);
    acc = make_float4(acc.x * inv * vmax, acc.y * inv * vmax, acc.z * inv * vmax, acc.w * inv * vmax);
    const float lse = (mx + fast_log2(sum)) * kLn2;
    if (slot >= 0) {
      const size_t at = static_cast<size_t>(slot) * prm.slot_rows + r;
      store4(prm.ws_o + at * D + c, acc);
      if (c == 0) prm.ws_lse[at] = lse;
    } else {
      const size_t at = static_cast<size_t>(bh) * prm.R + row0 + r;
      store4(static_cast<T*>(prm.o) + at * D + c, acc);
      if (c == 0) prm.lse[at] = lse;
    }
  }
  fence_async_smem();                      // the sums in the rings come before the next piece's loads
  __syncthreads();
  return true;
}

template <typename T, int D, int NT>
__global__ void __launch_bounds__(kWarps * 32, resident<T>(NT)) cache_attn_rows_kernel(const __grid_constant__ CacheAttnRowsParams par) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared sh;
  const CacheAttnParams& prm = par.c;
  uint8_t* smem = smem_raw + (1024u - smem_u32(smem_raw) % 1024u) % 1024u;
  asm volatile("griddepcontrol.launch_dependents;");
  if (threadIdx.x < kWarps * kStages) mbar_init(smem_u32(&sh.full[0][0]) + 8u * threadIdx.x, 1);
  if (threadIdx.x == 0) sh.abort_flag = 0;
  fence_mbar_init();
  __syncthreads();
  Slot into, from;                         // this warp's next tile to load, to use
  const int lane = threadIdx.x & 31;
  Requests req(prm, lane);
  const Share share = work_share(prm, req);
  long long x = blockIdx.x * share.size;
  const long long stop = min(x + share.size, share.total);
  if (x >= stop) return;
  const long long units = static_cast<long long>(prm.Hk) * prm.row_tiles;         // of a request
  long long first;
  int b = req.find(x / units, first);
  first *= units;
  int nb = req.blocks(b);
  while (x < stop) {
    const long long places = unit_places(nb);
    if (x >= first + places * units) {                           // on to the next request
      first += places * units;
      nb = req.blocks(++b);
      continue;
    }
    const long long in = (x - first) / places;                   // unit within the request
    const int p0 = static_cast<int>(x - first - in * places);
    const int p1 = static_cast<int>(min(places, p0 + (stop - x)));
    const int blk0 = max(p0 - kPieceCost, 0), blk1 = p1 - kPieceCost;
    if (blk1 > blk0) {
      const long long unit = b * units + in;
      // a share has at most one piece that goes on with a unit, and one that a later share goes on with
      const long long slot = blk0 == 0 && blk1 == nb ? -1 : 2LL * blockIdx.x + (blk0 == 0);
      if (!attend_piece<T, D, NT>(par, smem, sh, into, from, unit, cache_len(prm, b), blk0, blk1, slot)) return;
    }
    x += p1 - p0;
  }
}

// Short caches: a block takes whole units, and there is nothing to join.
template <typename T, int D, int NT>
__global__ void __launch_bounds__(kWarps * 32, resident<T>(NT)) cache_attn_short_kernel(const __grid_constant__ CacheAttnRowsParams par) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Shared sh;
  const CacheAttnParams& prm = par.c;
  uint8_t* smem = smem_raw + (1024u - smem_u32(smem_raw) % 1024u) % 1024u;
  if (threadIdx.x < kWarps * kStages) mbar_init(smem_u32(&sh.full[0][0]) + 8u * threadIdx.x, 1);
  if (threadIdx.x == 0) sh.abort_flag = 0;
  fence_mbar_init();
  __syncthreads();
  Slot into, from;
  const long long of_request = static_cast<long long>(prm.Hk) * prm.row_tiles;
  for (long long unit = blockIdx.x; unit < of_request * prm.B; unit += gridDim.x) {
    const int b = static_cast<int>(unit / of_request);
    const int len = cache_len(prm, b);
    if (len > 0) {
      if (!attend_piece<T, D, NT>(par, smem, sh, into, from, unit, len, 0, (len + PA_CACHE_BLOCK - 1) / PA_CACHE_BLOCK, -1)) return;
      continue;
    }
    const long long bh = unit / prm.row_tiles;
    const int row0 = static_cast<int>(unit - bh * prm.row_tiles) * 8 * NT;
    const size_t at = static_cast<size_t>(bh) * prm.R + row0;
    const int rows = min(8 * NT, prm.R - row0);
    for (int i = threadIdx.x; i < rows * D / 4; i += kWarps * 32) {
      store4(static_cast<T*>(prm.o) + at * D + 4 * i, make_float4(0.f, 0.f, 0.f, 0.f));
      if (i < rows) prm.lse[at + i] = -INFINITY;
    }
  }
}

// ------------------------------------------------------------------ join
// kWide: one block of 8 warps per query row, which take turns at the pieces, for few rows with many
// pieces; else one warp per row.  A lane holds D / 32 channels.  The weighted sums are taken in
// piece order within a warp and then in warp order.  Rows of a unit that one piece covered are
// done; rows without a token get the empty state.
constexpr int kJoinWarps = 8;

template <typename T, int D, bool kWide>
__global__ void __launch_bounds__(kJoinWarps * 32) cache_attn_rows_join_kernel(const __grid_constant__ CacheAttnParams prm) {
  constexpr int kC = D / 32;
  __shared__ float s_sum[kJoinWarps], s_acc[kJoinWarps][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long row = kWide ? blockIdx.x : static_cast<long long>(blockIdx.x) * kJoinWarps + warp;
  const long long of = min(row, prm.rows - 1);                  // rows behind the last set up for it, and wait
  const long long bh = of / prm.R;
  const int r = static_cast<int>(of - bh * prm.R);
  const int b = static_cast<int>(bh / prm.Hk);
  Requests req(prm, lane);
  const Share share = work_share(prm, req);
  const int nb = req.blocks(b);
  const int tile_rows = 8 * row_columns<T>(prm.R);
  const long long unit = bh * prm.row_tiles + r / tile_rows;
  const long long first = req.before(b) * prm.Hk * prm.row_tiles +
                          (unit - static_cast<long long>(b) * prm.Hk * prm.row_tiles) * unit_places(nb) + kPieceCost;
  // shares that hold a piece of the unit
  const long long p0 = first / share.size, p1 = (first + nb - 1) / share.size;
  // The pieces are written.  Every thread waits, also one without a piece to join: what comes next in
  // the stream is ordered behind this kernel only, so it must not end before the first has.
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (row >= prm.rows || (nb > 0 && p0 == p1)) return;
  const int pieces = nb > 0 ? static_cast<int>(p1 - p0 + 1) : 0;
  // piece i's row in the scratch: the first piece starts the unit, the others go on with it
  auto at = [&](int i) { return static_cast<size_t>(2 * (p0 + i) + (i == 0)) * prm.slot_rows + r % tile_rows; };

  constexpr int kStep = kWide ? kJoinWarps : 1;
  const int start = kWide ? warp : 0;
  float m = -INFINITY, sum = 0.0f;
  float acc[kC];
#pragma unroll
  for (int c = 0; c < kC; ++c) acc[c] = 0.0f;
  for (int i = lane; i < pieces; i += 32) m = fmaxf(m, prm.ws_lse[at(i)]);
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
  for (int i0 = start; i0 < pieces; i0 += 32 * kStep) {
    const int n = min(32, (pieces - i0 + kStep - 1) / kStep);
    const float own = lane < n ? expf(prm.ws_lse[at(i0 + lane * kStep)] - m) : 0.0f;
#pragma unroll 8
    for (int i = 0; i < n; ++i) {
      const float w = __shfl_sync(0xffffffffu, own, i);
      const float* src = prm.ws_o + at(i0 + i * kStep) * D + lane * kC;
      sum += w;
#pragma unroll
      for (int c = 0; c < kC; ++c) acc[c] = fmaf(w, src[c], acc[c]);
    }
  }
  if (kWide) {
    if (lane == 0) s_sum[warp] = sum;
#pragma unroll
    for (int c = 0; c < kC; ++c) s_acc[warp][lane * kC + c] = acc[c];
    __syncthreads();
    if (warp > 0) return;
    sum = 0.0f;
#pragma unroll
    for (int c = 0; c < kC; ++c) acc[c] = 0.0f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) {
      sum += s_sum[w];
#pragma unroll
      for (int c = 0; c < kC; ++c) acc[c] += s_acc[w][lane * kC + c];
    }
  }
  const float inv = nb > 0 ? 1.0f / sum : 0.0f;
  T* dst = static_cast<T*>(prm.o) + row * D + lane * kC;
#pragma unroll
  for (int c = 0; c < kC; c += 2) {
    if (sizeof(T) == 4)
      *reinterpret_cast<float2*>(dst + c) = make_float2(acc[c] * inv, acc[c + 1] * inv);
    else
      *reinterpret_cast<uint32_t*>(dst + c) = pack_bf16x2(acc[c] * inv, acc[c + 1] * inv);
  }
  if (lane == 0) prm.lse[row] = nb > 0 ? m + logf(sum) : -INFINITY;
}

// The join may be set up while the first kernel runs; it waits for all of it before it reads.
template <typename T, int D, int NT>
int rows_impl(const CacheAttnRowsParams& par, cudaStream_t st) {
  constexpr int smem = Ring<D>::kBytes;
  const CacheAttnParams& prm = par.c;
  cudaError_t e;
  if (prm.slot_rows == 0) {
    e = cudaFuncSetAttribute(cache_attn_short_kernel<T, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return static_cast<int>(e);
    cache_attn_short_kernel<T, D, NT><<<prm.shares, kWarps * 32, smem, st>>>(par);
    return static_cast<int>(cudaGetLastError());
  }
  e = cudaFuncSetAttribute(cache_attn_rows_kernel<T, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return static_cast<int>(e);
  cache_attn_rows_kernel<T, D, NT><<<prm.shares, kWarps * 32, smem, st>>>(par);
  if ((e = cudaGetLastError()) != cudaSuccess) return static_cast<int>(e);
  const bool wide = prm.rows <= kWideRows;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(wide ? prm.rows : (prm.rows + kJoinWarps - 1) / kJoinWarps));
  cfg.blockDim = dim3(kJoinWarps * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = wide ? cudaLaunchKernelEx(&cfg, cache_attn_rows_join_kernel<T, D, true>, prm)
           : cudaLaunchKernelEx(&cfg, cache_attn_rows_join_kernel<T, D, false>, prm);
  return static_cast<int>(e);
}

}  // namespace

int cache_attn_rows_tile_rows(int R, int dtype) {
  return 8 * (dtype == PA_F32 ? row_columns<float>(R) : row_columns<__nv_bfloat16>(R));
}
int cache_attn_rows_resident(int R, int dtype) {
  return dtype == PA_F32 ? resident<float>(1) : resident<__nv_bfloat16>(row_columns<__nv_bfloat16>(R));
}

int launch_cache_attn_rows(const CacheAttnRowsParams& par, int dtype, cudaStream_t st) {
  const bool d64 = par.c.D == 64;
  if (dtype == PA_F32) return d64 ? rows_impl<float, 64, 1>(par, st) : rows_impl<float, 128, 1>(par, st);
  if (row_columns<__nv_bfloat16>(par.c.R) == 1)
    return d64 ? rows_impl<__nv_bfloat16, 64, 1>(par, st) : rows_impl<__nv_bfloat16, 128, 1>(par, st);
  return d64 ? rows_impl<__nv_bfloat16, 64, 2>(par, st) : rows_impl<__nv_bfloat16, 128, 2>(par, st);
}

}  // namespace pa
