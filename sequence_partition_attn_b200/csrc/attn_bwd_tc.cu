// attn_bwd_tc.cu -- bf16 backward pass of attention with reuse on sm_100a tensor cores
// (tcgen05 + TMEM + TMA).  The mathematics is at the top of attn_bwd.cu.
//
// Two kinds of CTA, each owning a 128-row tile and streaming 128-row tiles of the other side over the
// fresh ranges of its group (neighbouring partitions join: the gradient needs no partition
// states).  No atomics: a tile's sums belong to one CTA, in a fixed order.
//
//   dK, dV  owns K, V; streams Q, dO.   S^T = K Q^T, dP^T = V dO^T (TMEM lanes are keys),
//           dV += P^T dO, dK += dS^T Q.  4 products of 128 x 128 x D.
//   dQ      owns Q, dO; streams K, V.   S = Q K^T, dP = dO V^T (lanes are queries),
//           dQ += dS K.  3 products.
// P and dS are rounded to bf16 for the second products, as the forward pass rounds P; they are
// written to TMEM over the scores they come from and read from there (A operand in TMEM), so
// neither goes through shared memory.
//
// Roles (384 threads, one CTA per SM).  warp 0: TMA producer.  warp 1: TMEM owner and MMA issuer
// (one thread).  warp 2, where a group streams a range shorter than a tile: zeroes the rows behind
// it, which may hold anything, and passes every tile on to the issuer (22 x 10 tokens in 32
// partitions: 20 us; 360 us with the issuing thread zeroing).  warp 3 (dK, dV): -LSE and -delta of
// the streamed queries into shared memory.  warps
// 4-7 and 8-11: two warpgroups, one TMEM lane per thread, columns 0-63 and 64-127 of the scores.
// Launched at 168 registers: warpgroup 0 drops to 88, the others rise to 208.
//
// Ordering.  tcgen05 products of one thread run in issue order and a commit tracks all earlier
// ones, so a product may overwrite columns that an earlier issued one reads.
#include "mma_tiles.cuh"
#include "pa_launch.h"

namespace pa {
namespace {

using namespace tiles;

constexpr int kThreads = 384;
constexpr int kRegsLow = 88, kRegsHigh = 208;
static_assert(kRegsLow + 2 * kRegsHigh == 3 * 168, "register split must equal the launch allocation");
constexpr float kLog2e = 1.4426950408889634f;

// 64 packed weights -> 32 TMEM columns.
__device__ __forceinline__ void store_weights(uint32_t tmem, const uint32_t (&w)[32]) {
  tmem_st32(tmem, w);
  tmem_wait_st();
  tc_fence_before();
}

__device__ __forceinline__ void read_scores(uint32_t tmem, float (&s)[64]) {
  uint32_t r[64];
  tmem_ld64(tmem, r);
  tmem_wait_ld();
#pragma unroll
  for (int i = 0; i < 64; ++i) s[i] = __uint_as_float(r[i]);
}

// The group, head and first row of a unit: groups in launch order, heads and then tiles in each.
template <int MP>
__device__ __forceinline__ int owner_tile(const BwdSide<MP>& side, int unit, int& bh, int& own0) {
  int i = 0;      // the last place that starts at or before the unit (those without rows end there)
  for (int n = side.QG; n > 1;) {
    const int half = n / 2;
    if (side.unit_start[i + half] <= unit) {
      i += half;
      n -= half;
    } else {
      n = half;
    }
  }
  const int g = side.order[i];
  const int rows = side.qg_row0[g + 1] - side.qg_row0[g];
  const int tiles = (rows + kRows - 1) / kRows;
  const int local = unit - side.unit_start[i];
  bh = local / tiles;
  own0 = side.qg_row0[g] + (local - bh * tiles) * kRows;
  return g;
}

// Dynamic shared memory starts on a 1024-byte boundary, as the swizzled tiles need (there is no
// room to move the base).  Checked, and recorded if it ever does not.
__device__ __forceinline__ bool smem_aligned(uint32_t base, int* status) {
  if ((base & 1023u) == 0) return true;
  if (threadIdx.x == 0) record_status(status, PA_ECUDA);
  return false;
}

// ------------------------------------------------------------------ dK, dV
// Q(j) is held until dK(j), dO(j) only until dV(j).  (With two stages of each the issuer waited
// 980 of 3190 cycles per tile for Q.)
constexpr int kQStages = 3, kOStages = 2;

template <int D>
struct KvLayout {
  static constexpr int kTile = tile_bytes<D>();
  static constexpr int kK = 0, kV = kTile;
  static constexpr int kQ = 2 * kTile;                        // [stage]
  static constexpr int kO = kQ + kQStages * kTile;            // dO [stage]
  static constexpr int kStat = kO + kOStages * kTile;         // [slot]{-LSE log2e [128], -delta [128]}
  static constexpr int kBar = kStat + 2 * 2 * kRows * 4;
  enum { KV_FULL = 0, Q_FULL = 1, O_FULL = Q_FULL + kQStages, Q_EMPTY = O_FULL + kOStages,
         O_EMPTY = Q_EMPTY + kQStages, STAT_FULL = O_EMPTY + kOStages, STAT_EMPTY = STAT_FULL + 2,
         S_FULL = STAT_EMPTY + 2, DP_FULL, P_LO, P_HI, DS_FULL, FINAL,
         Q_FIXED, O_FIXED = Q_FIXED + kQStages, NBAR = O_FIXED + kOStages };
  static constexpr int kSlot = kBar + NBAR * 8;
  static constexpr int kAbort = kSlot + 8;
  static constexpr int kBytes = kAbort + 8;
  static_assert(kBytes <= 227 * 1024, "shared memory budget");
};

template <int D, int MP>
__device__ __forceinline__ void dkdv_unit(const BwdTcParams<MP>& prm, int unit, uint8_t* gbase, const uint32_t base) {
  using L = KvLayout<D>;
  auto bar = [&](int i) { return base + L::kBar + 8u * i; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + L::kAbort);
  int* status = prm.status;
  const BwdSide<MP>& t = prm.kv;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int bh, own0;
  const int g = owner_tile(prm.kv, unit, bh, own0);
  const int own1 = t.qg_row0[g + 1];

  if (threadIdx.x == 0) {
    for (int i = 0; i < L::NBAR; ++i) {
      uint32_t n = 1;
      if (i == L::STAT_FULL || i == L::STAT_FULL + 1 || i >= L::Q_FIXED) n = 32;
      if (i == L::STAT_EMPTY || i == L::STAT_EMPTY + 1 || i == L::P_LO || i == L::P_HI || i == L::DS_FULL) n = 256;
      mbar_init(bar(i), n);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(base + L::kSlot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  constexpr uint32_t tmem = 0;             // an allocation of all 512 columns starts at column 0
  const uint32_t tX = tmem, tY = tmem + 128, tDV = tmem + 256, tDK = tmem + 384;
  auto sQ = [&](int s) { return base + L::kQ + s * L::kTile; };
  auto sO = [&](int u) { return base + L::kO + u * L::kTile; };
  const int n_tiles = t.tiles[g];
  const bool shorts = t.shorts[g];

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLow));
    if (warp == 0) {
      // ---------------------------------------------------------------- producer
      if (lane == 0 && n_tiles > 0) {
        mbar_expect_tx(bar(L::KV_FULL), 2 * L::kTile);
        load_tile<D>(base + L::kK, &prm.tm_k, own0, bh, bar(L::KV_FULL));
        load_tile<D>(base + L::kV, &prm.tm_v, own0, bh, bar(L::KV_FULL));
        int j = 0, nq = 0, no = 0;
        for (TileWalk w(t, g); w.valid(); w.next(), ++j) {
          const int s = j % kQStages, u = j % kOStages;
          if (j >= kQStages && !mbar_wait(bar(L::Q_EMPTY + s), (j / kQStages - 1) & 1, abort_flag, status)) break;
          mbar_expect_tx(bar(L::Q_FULL + s), L::kTile);
          load_tile<D>(sQ(s), &prm.tm_q, w.row(), bh, bar(L::Q_FULL + s));
          ++nq;
          if (j >= kOStages && !mbar_wait(bar(L::O_EMPTY + u), (j / kOStages - 1) & 1, abort_flag, status)) break;
          mbar_expect_tx(bar(L::O_FULL + u), L::kTile);
          load_tile<D>(sO(u), &prm.tm_do, w.row(), bh, bar(L::O_FULL + u));
          ++no;
        }
        // every load issued lands before the CTA exits
        mbar_drain(bar(L::KV_FULL), 0);
        for (int i = max(0, nq - kQStages); i < nq; ++i) mbar_drain(bar(L::Q_FULL + i % kQStages), (i / kQStages) & 1);
        for (int i = max(0, no - kOStages); i < no; ++i) mbar_drain(bar(L::O_FULL + i % kOStages), (i / kOStages) & 1);
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------------- MMA issuer
      if (n_tiles > 0 && elect_one()) {
        const uint64_t aK = kmajor(base + L::kK), aV = kmajor(base + L::kV);
        auto wait = [&](int b, uint32_t parity) { return mbar_wait(bar(b), parity & 1, abort_flag, status); };
        auto commit = [&](int b) { mma_commit(bar(b)); };
        const int q_full = shorts ? L::Q_FIXED : L::Q_FULL, o_full = shorts ? L::O_FIXED : L::O_FULL;
        bool ok = wait(L::KV_FULL, 0) && wait(q_full, 0) && wait(o_full, 0);
        int done = 0, freed = 0;         // Q_EMPTY, O_EMPTY commits issued
        if (ok) {
          tc_fence_after();
          product_nt<D>(tX, aK, kmajor(sQ(0)));
          commit(L::S_FULL);
          product_nt<D>(tY, aV, kmajor(sO(0)));
          commit(L::DP_FULL);
        }
        int s = 0, u = 0;                // stages of Q(j), dO(j)
        uint32_t phq = 0;                // parity of Q(j + 1)
        for (int j = 0; ok && j < n_tiles; ++j) {
          const int s1 = s + 1 == kQStages ? 0 : s + 1, u1 = u ^ 1;
          const bool more = j + 1 < n_tiles;
          if (s1 == 0) phq ^= 1;
          if (more) {
            ok = wait(q_full + s1, phq) && wait(o_full + u1, (j + 1) / kOStages) && wait(L::P_LO, j);
          } else {
            ok = wait(L::P_LO, j);
          }
          if (!ok) break;
          tc_fence_after();
          product_w<D, 64, 0x33>(tDV, tX, mnmajor(sO(u)), j == 0);      // columns 0-31 and 64-95 of P
          if (!(ok = wait(L::P_HI, j))) break;
          tc_fence_after();
          product_w<D, 64, 0xCC>(tDV, tX, mnmajor(sO(u)), false);
          commit(L::O_EMPTY + u);
          ++freed;
          if (more) {
            product_nt<D>(tX, aK, kmajor(sQ(s1)));
            commit(L::S_FULL);
          }
          if (!(ok = wait(L::DS_FULL, j & 1))) break;
          tc_fence_after();
          product_w<D, 64>(tDK, tY, mnmajor(sQ(s)), j == 0);
          commit(L::Q_EMPTY + s);
          ++done;
          if (more) {
            product_nt<D>(tY, aV, kmajor(sO(u1)));
            commit(L::DP_FULL);
          } else {
            commit(L::FINAL);
          }
          s = s1;
          u = u1;
        }
        {                                // the last commits arrive before the CTA exits
          for (int i = max(0, freed - kOStages); i < freed; ++i) mbar_drain(bar(L::O_EMPTY + i % kOStages), (i / kOStages) & 1);
          for (int i = max(0, done - kQStages); i < done; ++i) mbar_drain(bar(L::Q_EMPTY + i % kQStages), (i / kQStages) & 1);
        }
      }
    } else if (warp == 2 && shorts) {
      // ---------------------------------------------------------------- rows behind short ranges
      int j = 0;
      for (TileWalk w(t, g); w.valid(); w.next(), ++j) {
        const int s = j % kQStages, u = j % kOStages;
        if (!mbar_wait_warp(bar(L::Q_FULL + s), (j / kQStages) & 1, abort_flag, status)) break;
        if (w.is_short()) zero_rows<D>(gbase + L::kQ + s * L::kTile, w.last(), lane);
        mbar_arrive(bar(L::Q_FIXED + s));
        if (!mbar_wait_warp(bar(L::O_FULL + u), (j / kOStages) & 1, abort_flag, status)) break;
        if (w.is_short()) zero_rows<D>(gbase + L::kO + u * L::kTile, w.last(), lane);
        mbar_arrive(bar(L::O_FIXED + u));
      }
    } else if (warp == 3) {
      // ---------------------------------------------------------------- LSE and delta
      const size_t head = static_cast<size_t>(bh) * prm.N;
      asm volatile("griddepcontrol.wait;" ::: "memory");       // delta is written
      int j = 0;
      for (TileWalk w(t, g); w.valid(); w.next(), ++j) {
        const int s = j & 1;
        float nl[4], nd[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int c = lane * 4 + i;
          const bool in = c >= w.first() && c < w.last();
          const float l = in ? prm.lse[head + w.row() + c] : -INFINITY;
          // exp2(s + -inf) = 0: columns outside the tile's rows, and rows without any key
          nl[i] = l == -INFINITY ? -INFINITY : -l * kLog2e;
          nd[i] = in ? -prm.delta[head + w.row() + c] : 0.0f;
        }
        if (j >= 2 && !mbar_wait_warp(bar(L::STAT_EMPTY + s), (j / 2 - 1) & 1, abort_flag, status)) break;
        float* stat = reinterpret_cast<float*>(gbase + L::kStat) + s * 2 * kRows;
        *reinterpret_cast<float4*>(stat + lane * 4) = make_float4(nl[0], nl[1], nl[2], nl[3]);
        *reinterpret_cast<float4*>(stat + kRows + lane * 4) = make_float4(nd[0], nd[1], nd[2], nd[3]);
        mbar_arrive(bar(L::STAT_FULL + s));
      }
    }
  } else {
    // ---------------------------------------------------------------- P and dS, then the stores
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsHigh));
    const int x = (warp - 4) >> 2;                    // columns 64 x .. 64 x + 63
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t sX = tX + lane_off + x * 64, sY = tY + lane_off + x * 64;
    const float2 scale2 = make_float2(prm.scale_log2, prm.scale_log2);
    bool ok = true;
    for (int j = 0; j < n_tiles; ++j) {
      const int slot = j & 1;
      const float4* nl = reinterpret_cast<const float4*>(gbase + L::kStat + (slot * 2 * kRows + x * 64) * 4);
      const float4* nd = nl + kRows / 4;
      if (!mbar_wait(bar(L::STAT_FULL + slot), (j / 2) & 1, abort_flag, status) ||
          !mbar_wait(bar(L::S_FULL), j & 1, abort_flag, status)) {
        ok = false;
        break;
      }
      tc_fence_after();
      float p[64];
      read_scores(sX, p);
      uint32_t w[32];
#pragma unroll
      for (int h = 0; h < 2; ++h) {          // handed over in halves: dV starts on the first
#pragma unroll
        for (int i = 8 * h; i < 8 * h + 8; ++i) {
          const float4 l = nl[i];
          const float2 a = __ffma2_rn(make_float2(p[4 * i], p[4 * i + 1]), scale2, make_float2(l.x, l.y));
          const float2 b = __ffma2_rn(make_float2(p[4 * i + 2], p[4 * i + 3]), scale2, make_float2(l.z, l.w));
          p[4 * i] = fast_exp2(a.x);
          p[4 * i + 1] = fast_exp2(a.y);
          p[4 * i + 2] = fast_exp2(b.x);
          p[4 * i + 3] = fast_exp2(b.y);
          w[2 * i] = pack_bf16x2(p[4 * i], p[4 * i + 1]);
          w[2 * i + 1] = pack_bf16x2(p[4 * i + 2], p[4 * i + 3]);
        }
        uint32_t half[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) half[i] = w[16 * h + i];
        tmem_st16(sX + 16 * h, half);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(h ? L::P_HI : L::P_LO));
      }
      if (!mbar_wait(bar(L::DP_FULL), j & 1, abort_flag, status)) {
        ok = false;
        break;
      }
      tc_fence_after();
      float dp[64];
      read_scores(sY, dp);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float4 d = nd[i];
        const float2 a = __fmul2_rn(make_float2(p[4 * i], p[4 * i + 1]),
                                    __fadd2_rn(make_float2(dp[4 * i], dp[4 * i + 1]), make_float2(d.x, d.y)));
        const float2 b = __fmul2_rn(make_float2(p[4 * i + 2], p[4 * i + 3]),
                                    __fadd2_rn(make_float2(dp[4 * i + 2], dp[4 * i + 3]), make_float2(d.z, d.w)));
        w[2 * i] = pack_bf16x2(a.x, a.y);
        w[2 * i + 1] = pack_bf16x2(b.x, b.y);
      }
      store_weights(sY, w);
      mbar_arrive(bar(L::DS_FULL));
      mbar_arrive(bar(L::STAT_EMPTY + slot));
    }
    // warpgroup 0 stores dV, warpgroup 1 dK; over K and V, whose last products are done
    const int row0 = (warp & 3) * 32;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(x ? prm.dk : prm.dv) +
                         (static_cast<size_t>(bh) * prm.N + own0 + row0) * D;
    const int rows = own1 - own0 - row0;               // of this warp's 32
    if (n_tiles == 0) {
      if (lane < rows)
        for (int c = 0; c < D / 8; ++c) reinterpret_cast<uint4*>(out + lane * D)[c] = make_uint4(0, 0, 0, 0);
    } else if (__all_sync(0xffffffffu, ok) && mbar_wait_warp(bar(L::FINAL), 0, abort_flag, status)) {
      tc_fence_after();
      store_rows<D, D>((x ? tDK : tDV) + lane_off, gbase + L::kK + x * L::kTile + row0 * 2 * D, out,
                       x ? prm.scale : 1.0f, rows, lane);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ dQ
// Scores rotate through three TMEM regions so that S of the next tile is there when the threads
// turn to it: S(j) in R[2j % 3], dP(j) in R[(2j + 1) % 3] (dS(j) over it), S(j + 1) in the third.
// dP(j + 1) goes where S(j) was, once it has been read; S(j + 2) where dS(j) was, after dQ(j).
// S(j + 1) and dP(j + 1) are issued before the threads are done with tile j, so every barrier
// between the issuer and the threads comes in two, by the tile's parity: a waiter can be at most
// one phase behind on each.
constexpr int kKStages = 3, kVStages = 2;     // K(j) is held until dQ(j), V(j) only until dP(j)

template <int D>
struct QLayout {
  static constexpr int kTile = tile_bytes<D>();
  static constexpr int kQ = 0, kO = kTile;
  static constexpr int kK = 2 * kTile;                        // [stage]
  static constexpr int kV = kK + kKStages * kTile;            // [stage]
  static constexpr int kBar = kV + kVStages * kTile;
  enum { OWN_FULL = 0, K_FULL = 1, V_FULL = K_FULL + kKStages, K_EMPTY = V_FULL + kVStages,
         V_EMPTY = K_EMPTY + kKStages, S_FULL = V_EMPTY + kVStages,
         DP_FULL = S_FULL + 2, S_READ = DP_FULL + 2, DS_FULL = S_READ + 2, FINAL = DS_FULL + 2,
         K_FIXED, V_FIXED = K_FIXED + kKStages, NBAR = V_FIXED + kVStages };
  static constexpr int kSlot = kBar + NBAR * 8;
  static constexpr int kAbort = kSlot + 8;
  static constexpr int kBytes = kAbort + 8;
  static_assert(kBytes <= 227 * 1024, "shared memory budget");
};

template <int D, int MP>
__device__ __forceinline__ void dq_unit(const BwdTcParams<MP>& prm, int unit, uint8_t* gbase, const uint32_t base) {
  using L = QLayout<D>;
  auto bar = [&](int i) { return base + L::kBar + 8u * i; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + L::kAbort);
  int* status = prm.status;
  const BwdSide<MP>& t = prm.q;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int bh, own0;
  const int g = owner_tile(prm.q, unit, bh, own0);
  const int own1 = t.qg_row0[g + 1];

  if (threadIdx.x == 0) {
    for (int i = 0; i < L::NBAR; ++i)
      mbar_init(bar(i), i >= L::S_READ && i < L::FINAL ? 256u : i >= L::K_FIXED ? 32u : 1u);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(base + L::kSlot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  constexpr uint32_t tmem = 0;             // an allocation of all 512 columns starts at column 0
  const uint32_t tDQ = tmem + 384;
  auto region = [&](int i) { return tmem + 128u * (i % 3); };
  auto sK = [&](int j) { return base + L::kK + (j % kKStages) * L::kTile; };
  auto sV = [&](int j) { return base + L::kV + (j % kVStages) * L::kTile; };
  const int n_tiles = t.tiles[g];
  const bool shorts = t.shorts[g];

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLow));
    if (warp == 0) {
      // ---------------------------------------------------------------- producer
      if (lane == 0 && n_tiles > 0) {
        mbar_expect_tx(bar(L::OWN_FULL), 2 * L::kTile);
        load_tile<D>(base + L::kQ, &prm.tm_q, own0, bh, bar(L::OWN_FULL));
        load_tile<D>(base + L::kO, &prm.tm_do, own0, bh, bar(L::OWN_FULL));
        int j = 0, nk = 0, nv = 0;
        for (TileWalk w(t, g); w.valid(); w.next(), ++j) {
          const int s = j % kKStages, u = j % kVStages;
          if (j >= kKStages && !mbar_wait(bar(L::K_EMPTY + s), (j / kKStages - 1) & 1, abort_flag, status)) break;
          mbar_expect_tx(bar(L::K_FULL + s), L::kTile);
          load_tile<D>(sK(j), &prm.tm_k, w.row(), bh, bar(L::K_FULL + s));
          ++nk;
          if (j >= kVStages && !mbar_wait(bar(L::V_EMPTY + u), (j / kVStages - 1) & 1, abort_flag, status)) break;
          mbar_expect_tx(bar(L::V_FULL + u), L::kTile);
          load_tile<D>(sV(j), &prm.tm_v, w.row(), bh, bar(L::V_FULL + u));
          ++nv;
        }
        mbar_drain(bar(L::OWN_FULL), 0);
        for (int i = max(0, nk - kKStages); i < nk; ++i) mbar_drain(bar(L::K_FULL + i % kKStages), (i / kKStages) & 1);
        for (int i = max(0, nv - kVStages); i < nv; ++i) mbar_drain(bar(L::V_FULL + i % kVStages), (i / kVStages) & 1);
      }
    } else if (warp == 1) {
      // ---------------------------------------------------------------- MMA issuer
      if (n_tiles > 0 && elect_one()) {
        const uint64_t aQ = kmajor(base + L::kQ), aO = kmajor(base + L::kO);
        auto wait = [&](int b, uint32_t parity) { return mbar_wait(bar(b), parity & 1, abort_flag, status); };
        auto commit = [&](int b) { mma_commit(bar(b)); };
        const int k_full = shorts ? L::K_FIXED : L::K_FULL, v_full = shorts ? L::V_FIXED : L::V_FULL;
        bool ok = wait(L::OWN_FULL, 0) && wait(k_full, 0) && wait(v_full, 0) && (n_tiles < 2 || wait(k_full + 1, 0));
        int done = 0, freed = 0;         // K_EMPTY, V_EMPTY commits issued
        if (ok) {
          tc_fence_after();
          product_nt<D>(region(0), aQ, kmajor(sK(0)));
          commit(L::S_FULL);
          product_nt<D>(region(1), aO, kmajor(sV(0)));
          commit(L::V_EMPTY);
          ++freed;
          commit(L::DP_FULL);
          if (n_tiles > 1) {
            product_nt<D>(region(2), aQ, kmajor(sK(1)));
            commit(L::S_FULL + 1);
          }
        }
        int s = 0, r = 0;                // stage of K(j); region of S(j)
        uint32_t phk = 0;                // parity of K(j + 2)
        for (int j = 0; ok && j < n_tiles; ++j) {
          const int b = j & 1;
          const uint32_t ph = j / 2;
          const int s2 = s == 0 ? 2 : s - 1;                  // stage of K(j + 2)
          if (s2 == 0) phk ^= 1;
          const uint32_t tS = tmem + 128 * r, tP = tmem + 128 * (r == 2 ? 0 : r + 1);
          if (j + 1 < n_tiles) {
            ok = wait(v_full + (b ^ 1), (j + 1) / kVStages) && wait(L::S_READ + b, ph);
            if (!ok) break;
            tc_fence_after();
            product_nt<D>(tS, aO, kmajor(base + L::kV + (b ^ 1) * L::kTile));       // dP(j + 1) over S(j)
            commit(L::V_EMPTY + (b ^ 1));
            ++freed;
            commit(L::DP_FULL + (b ^ 1));
          }
          if (!(ok = wait(L::DS_FULL + b, ph))) break;
          tc_fence_after();
          product_w<D, 64>(tDQ, tP, mnmajor(base + L::kK + s * L::kTile), j == 0);
          commit(L::K_EMPTY + s);
          ++done;
          if (j + 2 < n_tiles) {
            // K(j + 2) takes the stage of K(j - 1), which dQ(j - 1) has just released: dQ(j) covers the load
            if (!(ok = wait(k_full + s2, phk))) break;
            tc_fence_after();
            product_nt<D>(tP, aQ, kmajor(base + L::kK + s2 * L::kTile));            // S(j + 2) over dS(j)
            commit(L::S_FULL + b);
          }
          if (j + 1 == n_tiles) commit(L::FINAL);
          s = s == kKStages - 1 ? 0 : s + 1;
          r = r == 0 ? 2 : r - 1;                             // 2 (j + 1) % 3
        }
        for (int i = max(0, done - kKStages); i < done; ++i) mbar_drain(bar(L::K_EMPTY + i % kKStages), (i / kKStages) & 1);
        for (int i = max(0, freed - kVStages); i < freed; ++i) mbar_drain(bar(L::V_EMPTY + i % kVStages), (i / kVStages) & 1);
      }
    } else if (warp == 2 && shorts) {
      // ---------------------------------------------------------------- rows behind short ranges
      int j = 0;
      for (TileWalk w(t, g); w.valid(); w.next(), ++j) {
        const int s = j % kKStages, u = j % kVStages;
        if (!mbar_wait_warp(bar(L::K_FULL + s), (j / kKStages) & 1, abort_flag, status)) break;
        if (w.is_short()) zero_rows<D>(gbase + L::kK + s * L::kTile, w.last(), lane);
        mbar_arrive(bar(L::K_FIXED + s));
        if (!mbar_wait_warp(bar(L::V_FULL + u), (j / kVStages) & 1, abort_flag, status)) break;
        if (w.is_short()) zero_rows<D>(gbase + L::kV + u * L::kTile, w.last(), lane);
        mbar_arrive(bar(L::V_FIXED + u));
      }
    }
  } else {
    // ---------------------------------------------------------------- dS, then the store
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsHigh));
    const int x = (warp - 4) >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_off = (static_cast<uint32_t>((warp & 3) * 32) << 16) + x * 64;
    const bool row_ok = own0 + row < own1;
    const size_t at = static_cast<size_t>(bh) * prm.N + own0 + row;
    asm volatile("griddepcontrol.wait;" ::: "memory");         // delta is written
    const float l = row_ok ? prm.lse[at] : -INFINITY;
    const float nl = l == -INFINITY ? -INFINITY : -l * kLog2e;    // no key: every P is 0
    const float nd = row_ok ? -prm.delta[at] : 0.0f;
    const float2 scale2 = make_float2(prm.scale_log2, prm.scale_log2);
    const float2 nl2 = make_float2(nl, nl), nd2 = make_float2(nd, nd);
    bool ok = true;
    TileWalk w(t, g);
    for (int j = 0; j < n_tiles; ++j, w.next()) {
      if (!mbar_wait(bar(L::S_FULL + (j & 1)), (j / 2) & 1, abort_flag, status)) {
        ok = false;
        break;
      }
      tc_fence_after();
      float p[64];
      read_scores(region(2 * j) + lane_off, p);
      tc_fence_before();
      mbar_arrive(bar(L::S_READ + (j & 1)));
      if (w.first() > 0 || w.last() < kRows) {
#pragma unroll
        for (int c = 0; c < 64; ++c)
          if (x * 64 + c < w.first() || x * 64 + c >= w.last()) p[c] = -INFINITY;
      }
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float2 a = __ffma2_rn(make_float2(p[2 * i], p[2 * i + 1]), scale2, nl2);
        p[2 * i] = fast_exp2(a.x);
        p[2 * i + 1] = fast_exp2(a.y);
      }
      if (!mbar_wait(bar(L::DP_FULL + (j & 1)), (j / 2) & 1, abort_flag, status)) {
        ok = false;
        break;
      }
      tc_fence_after();
      float dp[64];
      read_scores(region(2 * j + 1) + lane_off, dp);
      uint32_t ds[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float2 a = __fmul2_rn(make_float2(p[2 * i], p[2 * i + 1]),
                                    __fadd2_rn(make_float2(dp[2 * i], dp[2 * i + 1]), nd2));
        ds[i] = pack_bf16x2(a.x, a.y);
      }
      store_weights(region(2 * j + 1) + lane_off, ds);
      mbar_arrive(bar(L::DS_FULL + (j & 1)));
    }
    // each warpgroup stores half of dQ's columns, over Q, whose last product is done
    const int row0 = (warp & 3) * 32;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(prm.dq) +
                         (static_cast<size_t>(bh) * prm.N + own0 + row0) * D + x * (D / 2);
    const int rows = own1 - own0 - row0;
    if (n_tiles == 0) {
      if (lane < rows)
        for (int c = 0; c < D / 16; ++c) reinterpret_cast<uint4*>(out + lane * D)[c] = make_uint4(0, 0, 0, 0);
    } else if (__all_sync(0xffffffffu, ok) && mbar_wait_warp(bar(L::FINAL), 0, abort_flag, status)) {
      tc_fence_after();
      store_rows<D / 2, D>(tDQ + (lane_off & 0xFFFF0000u) + x * (D / 2), gbase + L::kQ + x * (L::kTile / 2) + row0 * D, out,
                           prm.scale, rows, lane);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// One launch: the CTAs of the dK, dV kernel first, those of dQ behind them, each longest first (the
// hardware hands them out in order), so that there is one tail instead of two.
template <int D, int MP>
__global__ void __launch_bounds__(kThreads, 1) attn_bwd_tc_kernel(const __grid_constant__ BwdTcParams<MP> prm) {
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_u32(smem);
  if (!smem_aligned(base, prm.status)) return;
  if (static_cast<int>(blockIdx.x) < prm.kv.units)
    dkdv_unit<D>(prm, blockIdx.x, smem, base);
  else
    dq_unit<D>(prm, blockIdx.x - prm.kv.units, smem, base);
}

// Launched ahead of the end of the delta kernel, whose results alone are waited for.
template <int D, int MP>
int tc_impl(const BwdTcParams<MP>& prm, cudaStream_t st) {
  constexpr int smem = KvLayout<D>::kBytes > QLayout<D>::kBytes ? KvLayout<D>::kBytes : QLayout<D>::kBytes;
  cudaError_t e = cudaFuncSetAttribute(attn_bwd_tc_kernel<D, MP>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return static_cast<int>(e);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(prm.kv.units + prm.q.units);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr = {};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return static_cast<int>(cudaLaunchKernelEx(&cfg, attn_bwd_tc_kernel<D, MP>, prm));
}

}  // namespace

int attn_bwd_tc_tile_rows() { return kRows; }

int launch_attn_bwd_tc(const BwdTcParams<32>& prm, int D, cudaStream_t st) {
  return D == 64 ? tc_impl<64, 32>(prm, st) : tc_impl<128, 32>(prm, st);
}

int launch_attn_bwd_tc(const BwdTcParams<PA_MAX_P>& prm, int D, cudaStream_t st) {
  return D == 64 ? tc_impl<64, PA_MAX_P>(prm, st) : tc_impl<128, PA_MAX_P>(prm, st);
}

}  // namespace pa
