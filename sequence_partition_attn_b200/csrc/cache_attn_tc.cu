// cache_attn_tc.cu -- attention over the 8-bit K/V cache for many query rows per KV head (bf16
// queries: prompts, a ring step's block) on sm_100a tensor cores.  Definition: cache_attn_rows.cu.
//
// Bound by the tensor cores and the exponentials, as the bf16 partition attention (attn_tc.cu),
// whose scheme of two 128-row query tiles per CTA it follows: S = Q K^T and O += P V on tcgen05,
// P written to TMEM over S.  What differs is where K and V come from: a warpgroup reads the codes
// of each 128-token tile, two cache blocks, with asynchronous copies a whole tile of K and V ahead,
// multiplies them by the block's scale in fp32 and writes bf16 to the swizzled tile that the
// products read.  The scale is a power of two, so code * scale is exact in bf16: nothing is
// rounded that the cache did not round already, and the scores need no scale of their own.
// The codes cross HBM and L2 in 8 bits; a pass that widened the cache to bf16 first would write
// and read it again at twice the size.  40 heads x 9450 queries x 9450 tokens, D = 128: 1.77 ms
// at the power cap, 1.56 ms before it is reached, a tile of 128 tokens every 3800 cycles, of which the softmax warps work 2200 and wait for the
// products between.  (Loads into registers one block ahead: 1.93 ms, as L2 answers in about a
// thousand cycles and a tile has four of them in a row.  f16 tiles with the scales in the softmax
// instead: fewer instructions to widen, but 500 more per tile in the softmax, which sets the pace.)
//
// Roles (512 threads, one CTA per SM; 128 registers at launch, then 80 / 176 / 176 / 80):
//   warp 0      loads Q_a, Q_b by TMA.     warp 1  TMEM owner and MMA issuer.
//   warps 4..7  softmax of query tile a; warps 8..11 of tile b (one row per thread), and at the end
//               the stores of its O and LSE.
//   warps 12..15 widen K and V.
// Rows are the (H / Hk) * Nq queries of one KV head.  A block of at most 128 rows runs tile a only.
#include <cuda_fp16.h>

#include "mma_tiles.cuh"
#include "pa_launch.h"

namespace pa {
namespace {

using tiles::kAtomBytes;

constexpr int kBM = 128, kBN = 128;
constexpr int kStages = 2;
constexpr int kThreads = 512;
constexpr int kRegsLow = 80, kRegsWiden = 80, kRegsHigh = 176;
static_assert(kRegsLow + kRegsWiden + 2 * kRegsHigh == kThreads / 128 * (65536 / kThreads),
              "register split must equal the launch allocation");
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleLog2 = 8.0f;    // move the running max only when it grows by > 8

template <int D>
struct Layout {
  static constexpr int kTile = tiles::tile_bytes<D>();
  static constexpr int kQ = 0;                                 // Q_a, Q_b
  static constexpr int kK = kQ + 2 * kTile;
  static constexpr int kV = kK + kStages * kTile;
  static constexpr int kItem = 64 * D;                         // codes of a cache block
  static constexpr int kCodes = kV + kStages * kTile;          // the next four items
  static constexpr int kBar = kCodes + 4 * kItem;
  enum { Q_FULL = 0, K_FULL = 1, V_FULL = K_FULL + kStages, K_EMPTY = V_FULL + kStages,
         V_EMPTY = K_EMPTY + kStages, S_FULL = V_EMPTY + kStages, P_LO = S_FULL + 2, P_HI = P_LO + 2,
         O_FINAL = P_HI + 2, O_READY = O_FINAL + 2, NBAR = O_READY + 2 };
  static constexpr int kSlot = kBar + NBAR * 8;
  static constexpr int kAbort = kSlot + 8;
  static constexpr int kBytes = kAbort + 8 + 1024;
  static_assert(kBytes <= 227 * 1024, "shared memory budget");
};

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

__device__ __forceinline__ float row_max(const float (&s)[kBN]) {
  float mx[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) mx[i] = max3(s[i], s[i + 8], s[i + 16]);
#pragma unroll
  for (int c = 24; c < 120; c += 16)
#pragma unroll
    for (int i = 0; i < 8; ++i) mx[i] = max3(mx[i], s[c + i], s[c + 8 + i]);
#pragma unroll
  for (int i = 0; i < 8; ++i) mx[i] = fmaxf(mx[i], s[120 + i]);
  return max3(max3(mx[0], mx[1], mx[2]), max3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7]));
}

// Weights of 64 columns: exponentials, row-sum chains, bf16 pairs (32 TMEM columns).
template <int H>
__device__ __forceinline__ void weights_half(const float (&s)[kBN], float m, float sl2, float2 (&acc)[4], uint32_t (&w)[32]) {
  const float2 scale2 = make_float2(sl2, sl2), neg_m2 = make_float2(-m, -m);
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const int c = H * 64 + 2 * i;
    const float2 a = __ffma2_rn(make_float2(s[c], s[c + 1]), scale2, neg_m2);
    const float e0 = fast_exp2(a.x), e1 = fast_exp2(a.y);
    acc[i & 3] = __fadd2_rn(acc[i & 3], make_float2(e0, e1));
    w[i] = pack_bf16x2(e0, e1);
  }
}

// Four codes times a power of two, as bf16 pairs.
__device__ __forceinline__ void widen(uint32_t codes, float2 scale, uint32_t& lo, uint32_t& hi) {
  uint32_t h[2];
  e4m3_to_f16(codes, h[0], h[1]);
  const float2 x = __fmul2_rn(__half22float2(*reinterpret_cast<const __half2*>(&h[0])), scale);
  const float2 y = __fmul2_rn(__half22float2(*reinterpret_cast<const __half2*>(&h[1])), scale);
  lo = pack_bf16x2(x.x, x.y);
  hi = pack_bf16x2(y.x, y.y);
}

// One item of the widening warpgroup: a cache block (64 tokens) of K or of V in 16-byte pieces.
// A thread copies the pieces that it widens itself, so its own wait is all that a copy needs.
template <int D>
struct Item {
  static constexpr int kSegs = D / 16;                 // 16-code pieces per token
  static constexpr int kPieces = 64 * kSegs / 128;     // per thread

  // Starts the copies; tokens at or behind `end` are not read and become 0.
  static __device__ __forceinline__ void fetch(uint32_t slot, const uint8_t* codes, int tok, int end, int thread) {
#pragma unroll
    for (int n = 0; n < kPieces; ++n) {
      const int i = n * 128 + thread;
      const int j = tok + i / kSegs;
      const bool in = j < end;
      const uint8_t* src = codes + (in ? static_cast<size_t>(j) * D + (i % kSegs) * 16 : 0);
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(slot + i * 16), "l"(src), "r"(in ? 16 : 0) : "memory");
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }

  // Into rows `row0` .. of a swizzled tile: 16-byte chunk c of row r lies at chunk c ^ (r & 7).
  static __device__ __forceinline__ void store(const uint8_t* slot, float scale, uint8_t* tile, int row0, int thread) {
    uint4 c[kPieces];
#pragma unroll
    for (int n = 0; n < kPieces; ++n) c[n] = *reinterpret_cast<const uint4*>(slot + (n * 128 + thread) * 16);
#pragma unroll
    for (int n = 0; n < kPieces; ++n) {
      const int i = n * 128 + thread;
      const int r = row0 + i / kSegs, seg = i % kSegs;
      const uint32_t w[4] = {c[n].x, c[n].y, c[n].z, c[n].w};
      uint32_t x[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) widen(w[k], make_float2(scale, scale), x[2 * k], x[2 * k + 1]);
      uint8_t* row = tile + (seg >> 2) * kAtomBytes + r * 128;
      const int ch = (seg & 3) * 2;
      // the two atoms share banks: the second one's lanes store their chunks in the other order
      const int sw = seg >> 2;
      const uint4 a = make_uint4(x[0], x[1], x[2], x[3]), b = make_uint4(x[4], x[5], x[6], x[7]);
      *reinterpret_cast<uint4*>(row + (((ch + sw) ^ (r & 7)) << 4)) = sw ? b : a;
      *reinterpret_cast<uint4*>(row + (((ch + 1 - sw) ^ (r & 7)) << 4)) = sw ? a : b;
    }
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 1) cache_attn_tc_kernel(const __grid_constant__ CacheAttnTcParams p) {
  using L = Layout<D>;
  const CacheAttnParams& prm = p.c;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* gbase = smem_raw + (base - raw);
  auto bar = [&](int i) { return base + L::kBar + 8u * i; };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(gbase + L::kAbort);
  int* status = prm.status;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // Unit: (KV head, 256-row block, split).
  const int split = blockIdx.x % prm.splits;
  const int unit = blockIdx.x / prm.splits;
  const int bh = unit / p.row_blocks;
  const int row0 = (unit - bh * p.row_blocks) * (2 * kBM);
  const int nx = prm.R - row0 > kBM ? 2 : 1;
  const int len = cache_len(prm, bh / prm.Hk);
  const int chunk = split_chunk(len, prm.splits);
  const int begin = min(split * chunk, len), end = min(begin + chunk, len);
  const int T = (end - begin + kBN - 1) / kBN;

  if (threadIdx.x == 0) {
    for (int i = 0; i < L::NBAR; ++i) {
      const bool threads = (i >= L::K_FULL && i < L::K_EMPTY) || (i >= L::P_LO && i < L::O_FINAL) || i >= L::O_READY;
      mbar_init(bar(i), threads ? 128u : 1u);
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
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(gbase + L::kSlot);
  auto sK = [&](int s) { return base + L::kK + s * L::kTile; };
  auto sV = [&](int s) { return base + L::kV + s * L::kTile; };

  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLow));
    if (warp == 0) {
      if (lane == 0 && T > 0) {
        mbar_expect_tx(bar(L::Q_FULL), nx * L::kTile);
        for (int x = 0; x < nx; ++x)
          tiles::load_tile<D>(base + L::kQ + x * L::kTile, &p.tm_q, row0 + x * kBM, bh, bar(L::Q_FULL));
        mbar_drain(bar(L::Q_FULL), 0);
      }
    } else if (warp == 1 && T > 0 && elect_one()) {
      // ---------------------------------------------------------------- MMA issuer
      // Per tile j: PV_a(j), S_a(j+1), PV_b(j), S_b(j+1); S_x(j+1) overwrites the P_x(j) that the
      // product issued before it reads.
      auto wait = [&](int b, uint32_t parity) { return mbar_wait(bar(b), parity, abort_flag, status); };
      auto commit = [&](int b) { mma_commit(bar(b)); };
      const uint64_t dq[2] = {tiles::kmajor(base + L::kQ), tiles::kmajor(base + L::kQ + L::kTile)};
      bool ok = wait(L::Q_FULL, 0) && wait(L::K_FULL, 0);
      if (ok) {
        tc_fence_after();
        for (int x = 0; x < nx; ++x) {
          tiles::product_nt<D>(tmem + x * 128, dq[x], tiles::kmajor(sK(0)));
          commit(L::S_FULL + x);
        }
        commit(L::K_EMPTY);
        ok = wait(L::V_FULL, 0);
      }
      int done = 0;
      for (int j = 0; ok && j < T; ++j) {
        const int s = j % kStages, s1 = (j + 1) % kStages;
        const uint32_t ph1 = ((j + 1) / kStages) & 1;
        const bool more = j + 1 < T;
        const uint64_t dv = tiles::mnmajor(sV(s)), dk = tiles::kmajor(sK(s1));
        for (int x = 0; ok && x < nx; ++x) {
          const uint32_t tP = tmem + x * 128, tO = tmem + 256 + x * 128;
          if (!(ok = wait(L::P_LO + x, j & 1))) break;
          tc_fence_after();
          tiles::product_w<D, 32, 0x0F>(tO, tP, dv, j == 0);
          // the next operands are checked while P's second half is still being produced
          if (more && !(ok = x == 0 ? wait(L::K_FULL + s1, ph1) : true)) break;
          if (more && x == nx - 1 && !(ok = wait(L::V_FULL + s1, ph1))) break;
          if (!(ok = wait(L::P_HI + x, j & 1))) break;
          tc_fence_after();
          tiles::product_w<D, 32, 0xF0>(tO, tP, dv, false);
          if (!more) commit(L::O_FINAL + x);
          if (x == nx - 1) commit(L::V_EMPTY + s);
          if (more) {
            tiles::product_nt<D>(tP, dq[x], dk);
            commit(L::S_FULL + x);
            if (x == nx - 1) commit(L::K_EMPTY + s1);
          }
        }
        if (ok) ++done;
      }
      for (int i = max(0, done - kStages); i < done; ++i) {   // the last commits arrive before the CTA exits
        mbar_drain(bar(L::K_EMPTY + i % kStages), (i / kStages) & 1);
        mbar_drain(bar(L::V_EMPTY + i % kStages), (i / kStages) & 1);
      }
    }
  } else if (warp < 12) {
    // ---------------------------------------------------------------- softmax
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsHigh));
    const int x = (warp - 4) >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_off + x * 128, tO = tS + 256;
    float m = -INFINITY, l = 0.0f;       // running max (log2 units, scaled) and sum
    const float sl2 = p.scale_log2;
    for (int j = 0; x < nx && j < T; ++j) {
      if (!mbar_wait(bar(L::S_FULL + x), j & 1, abort_flag, status)) break;
      tc_fence_after();
      float s[kBN];
      {
        uint32_t r[2][64];
        tmem_ld64(tS, r[0]);
        tmem_ld64(tS + 64, r[1]);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < kBN; ++i) s[i] = __uint_as_float(r[i >> 6][i & 63]);
      }
      const int nvalid = end - begin - j * kBN;
      if (nvalid < kBN) {
#pragma unroll
        for (int c = 0; c < kBN; ++c) s[c] = c < nvalid ? s[c] : -INFINITY;
      }
      const float mt = row_max(s) * sl2;
      if (j == 0) {
        m = mt;
      } else if (__any_sync(0xffffffffu, mt - m > kRescaleLog2)) {
        // only rows whose own max grew move it: a row never depends on its neighbours
        const float m_new = mt - m > kRescaleLog2 ? mt : m;
        const float alpha = fast_exp2(m - m_new);
#pragma unroll 1
        for (int c = 0; c < D / 16; ++c) {
          uint32_t v[16];
          tmem_ld16(tO + c * 16, v);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) * alpha);
          tmem_st16(tO + c * 16, v);
        }
        l *= alpha;
        m = m_new;
      }
      float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
      {
        uint32_t w[32];
        weights_half<0>(s, m, sl2, acc, w);
        tmem_st32(tS, w);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(L::P_LO + x));
      }
      {
        uint32_t w[32];
        weights_half<1>(s, m, sl2, acc, w);
        tmem_st32(tS + 32, w);
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(L::P_HI + x));
      }
      const float2 a = __fadd2_rn(__fadd2_rn(acc[0], acc[1]), __fadd2_rn(acc[2], acc[3]));
      l += a.x + a.y;
    }
    const int r = row0 + x * kBM + row;
    if (x < nx && (T == 0 || mbar_wait(bar(L::O_FINAL + x), 0, abort_flag, status))) {
      tc_fence_after();
      const bool row_ok = r < prm.R;
      const size_t at = (prm.splits > 1 ? static_cast<size_t>(split) * prm.rows : 0) + static_cast<size_t>(bh) * prm.R + r;
      const float inv = 1.0f / l;
#pragma unroll 2
      for (int c = 0; c < D / 16; ++c) {
        float v[16];
        if (T > 0) {
          uint32_t u[16];
          tmem_ld16(tO + c * 16, u);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(u[i]) * inv;
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) v[i] = 0.0f;
        }
        if (prm.splits > 1) {
          if (!row_ok) continue;
#pragma unroll
          for (int i = 0; i < 16; i += 4) store4(prm.ws_o + at * D + c * 16 + i, make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]));
        } else {                         // over Q_x, whose last product is done
          uint8_t* o = gbase + L::kQ + x * L::kTile + (c >> 2) * kAtomBytes + row * 128;
          const int ch = (c & 3) * 2, sw = row & 7;
          *reinterpret_cast<uint4*>(o + ((ch ^ sw) << 4)) =
              make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
          *reinterpret_cast<uint4*>(o + (((ch + 1) ^ sw) << 4)) =
              make_uint4(pack_bf16x2(v[8], v[9]), pack_bf16x2(v[10], v[11]), pack_bf16x2(v[12], v[13]), pack_bf16x2(v[14], v[15]));
        }
      }
      if (row_ok) (prm.splits > 1 ? prm.ws_lse : prm.lse)[at] = T > 0 ? (m + fast_log2(l)) * kLn2 : -INFINITY;
      if (prm.splits == 1) {
        fence_async_smem();
        mbar_arrive(bar(L::O_READY + x));
        // rows behind the head's last are not written
        if (row == 0 && mbar_wait(bar(L::O_READY + x), 0, abort_flag, status)) {
          for (int a = 0; a < D / 64; ++a)
            tma_store_3d(&p.tm_o, base + L::kQ + x * L::kTile + a * kAtomBytes, a * 64, row0 + x * kBM, bh);
          tma_store_wait();
        }
      }
    }
  } else {
    // ---------------------------------------------------------------- widening
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsWiden));
    const int thread = threadIdx.x - 384;
    const size_t head = static_cast<size_t>(bh) * prm.M * D;
    const uint8_t* codes[2] = {prm.k_codes + head, prm.v_codes + head};
    const float* scales[2] = {prm.k_scale + static_cast<size_t>(bh) * prm.blocks,
                              prm.v_scale + static_cast<size_t>(bh) * prm.blocks};
    bool ok = true;
    // item i of a tile: block i & 1 of K (i < 2) or V
    auto fetch = [&](int i, int tok) {
      Item<D>::fetch(base + L::kCodes + i * L::kItem, codes[i >> 1], tok + (i & 1) * 64, end, thread);
    };
    auto scale_of = [&](int i, int tok) {
      return tok + (i & 1) * 64 < end ? __ldg(scales[i >> 1] + tok / PA_CACHE_BLOCK + (i & 1)) : 0.0f;
    };
    float scale[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      fetch(i, begin);
      scale[i] = scale_of(i, begin);
    }
    for (int j = 0; ok && j < T; ++j) {
      const int s = j % kStages;
      const int tok = begin + j * kBN;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int kv = i >> 1;
        if ((i & 1) == 0 && j >= kStages &&
            !mbar_wait(bar((kv ? L::V_EMPTY : L::K_EMPTY) + s), (j / kStages - 1) & 1, abort_flag, status)) {
          ok = false;
          break;
        }
        asm volatile("cp.async.wait_group 3;" ::: "memory");
        Item<D>::store(gbase + L::kCodes + i * L::kItem, scale[i], gbase + (kv ? L::kV : L::kK) + s * L::kTile,
                       (i & 1) * 64, thread);
        fetch(i, tok + kBN);
        scale[i] = scale_of(i, tok + kBN);
        if (i & 1) {
          fence_async_smem();
          mbar_arrive(bar((kv ? L::V_FULL : L::K_FULL) + s));
        }
      }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Join of the splits' states: D / 4 threads per row, four channels each.
template <int D>
__global__ void __launch_bounds__(128) cache_join_kernel(const __grid_constant__ CacheAttnParams prm) {
  constexpr int TPR = D / 4;
  const long long row = static_cast<long long>(blockIdx.x) * (128 / TPR) + threadIdx.x / TPR;
  const int c = threadIdx.x % TPR;
  if (row >= prm.rows) return;
  float m = -INFINITY;
  for (int s = 0; s < prm.splits; ++s) m = fmaxf(m, prm.ws_lse[s * static_cast<size_t>(prm.rows) + row]);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float sum = 0.0f;
  for (int s = 0; s < prm.splits; ++s) {
    const size_t at = s * static_cast<size_t>(prm.rows) + row;
    const float lse = prm.ws_lse[at];
    const float w = lse == -INFINITY ? 0.0f : expf(lse - m);      // a split without tokens
    const float4 x = *reinterpret_cast<const float4*>(prm.ws_o + at * D + 4 * c);
    sum += w;
    acc.x = fmaf(w, x.x, acc.x);
    acc.y = fmaf(w, x.y, acc.y);
    acc.z = fmaf(w, x.z, acc.z);
    acc.w = fmaf(w, x.w, acc.w);
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
  store4(static_cast<__nv_bfloat16*>(prm.o) + static_cast<size_t>(row) * D + 4 * c, acc);
  if (c == 0) prm.lse[row] = sum == 0.0f ? -INFINITY : m + logf(sum);
}

template <int D>
int tc_impl(const CacheAttnTcParams& p, unsigned units, cudaStream_t st) {
  cudaError_t e = cudaFuncSetAttribute(cache_attn_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<D>::kBytes);
  if (e != cudaSuccess) return static_cast<int>(e);
  cache_attn_tc_kernel<D><<<units, kThreads, Layout<D>::kBytes, st>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess || p.c.splits == 1) return static_cast<int>(e);
  constexpr int kPerBlock = 128 / (D / 4);
  cache_join_kernel<D><<<static_cast<unsigned>((p.c.rows + kPerBlock - 1) / kPerBlock), 128, 0, st>>>(p.c);
  return static_cast<int>(cudaGetLastError());
}

}  // namespace

int cache_attn_tc_block_rows() { return 2 * kBM; }

int launch_cache_attn_tc(const CacheAttnTcParams& p, unsigned units, cudaStream_t st) {
  return p.c.D == 64 ? tc_impl<64>(p, units, st) : tc_impl<128>(p, units, st);
}

}  // namespace pa
