// attn_bwd.cu -- backward pass of attention with reuse: the per-row terms and the kernels on
// the FMA units (fp32 inputs).
//
// With the merged outputs (O, LSE) of pa_partition_attn + pa_merge_states, the fresh pairs'
// share of the output is P_ij v_j with P_ij = exp(s_ij - LSE_i), s = scale * q.k: the
// partition weights exp(LSE_p - LSE) and the partition probabilities exp(s - LSE_p) multiply
// to it, so the per-partition states are not needed.  Reused states are constants.  Hence
//   delta_i = dO_i . O_i - dLSE_i,   dS_ij = P_ij (dO_i . v_j - delta_i),
//   dQ_i = scale sum_j dS_ij k_j,    dK_j = scale sum_i dS_ij q_i,    dV_j = sum_i P_ij dO_i
// over the fresh pairs.  P is recomputed from q, k and LSE, never stored.
//
// Two kernels, each owning the rows of what it sums and streaming the other side: one for
// dQ (owns queries, streams keys), one for dK and dV (owns keys, streams queries).  Every sum
// is taken by one block in a fixed order, so results do not change from run to run; the price
// is that s and dO.v are computed twice (7 products instead of 5).
#include "pa_device.cuh"
#include "pa_launch.h"

namespace pa {
namespace {

// ------------------------------------------------------------------ delta
// One group of lanes per row, 16 bytes of O and dO per lane.  Bound by HBM: both read once.
template <typename T, int D>
__global__ void __launch_bounds__(256) delta_kernel(const T* __restrict__ o, const T* __restrict__ dout,
                                                    const float* __restrict__ dlse, float* __restrict__ delta,
                                                    long long rows) {
  constexpr int kLanes = D * sizeof(T) / 16;
  asm volatile("griddepcontrol.launch_dependents;");
  const long long row = (static_cast<long long>(blockIdx.x) * 256 + threadIdx.x) / kLanes;
  const int c = threadIdx.x % kLanes;
  float sum = 0.0f;
  if (row < rows) {
    const uint4 a = __ldg(reinterpret_cast<const uint4*>(o) + row * kLanes + c);
    const uint4 b = __ldg(reinterpret_cast<const uint4*>(dout) + row * kLanes + c);
    const uint32_t au[4] = {a.x, a.y, a.z, a.w}, bu[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (sizeof(T) == 4) {
        sum = fmaf(__uint_as_float(au[i]), __uint_as_float(bu[i]), sum);
      } else {
        sum = fmaf(__uint_as_float(au[i] << 16), __uint_as_float(bu[i] << 16), sum);
        sum = fmaf(__uint_as_float(au[i] & 0xFFFF0000u), __uint_as_float(bu[i] & 0xFFFF0000u), sum);
      }
    }
  }
#pragma unroll
  for (int off = kLanes / 2; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  if (row < rows && c == 0) delta[row] = sum - (dlse ? dlse[row] : 0.0f);
}

// ------------------------------------------------------------------ FMA kernels
// A block owns kOwn rows (queries for dQ, keys for dK and dV) and streams tiles of 64 rows of the
// other side through shared memory.  Products run on packed pairs of fp32 (two multiply-adds per
// instruction: the multiply-add pipe, not the issue slots, is then what bounds them); pairs run
// along the summed index in the first products and along the channels in the second.
constexpr int kT = 64;               // streamed rows per tile
constexpr int kThreads = 256;        // 16 x 16

template <int D, int kOwn>
struct Smem {
  static constexpr int kRow = D + 4;       // 16-byte reads of 8 rows then fall in different banks
  static constexpr int kOwnTile = kOwn * kRow;
  static constexpr int kTile = kT * kRow;
  static constexpr int kPRow = kOwn + 4;   // weights [streamed row][own row]
  static constexpr int kP = kT * kPRow;
  static constexpr int kBytes = (2 * kOwnTile + 2 * kTile + 2 * kP + 2 * kT) * 4;
};

// Rows [r0, r0 + kRows) of a [.., D] tensor into shared memory; rows at or past `end` read as 0,
// so that nothing outside the range (which may be non-finite) reaches a product.
template <int D, int kRows>
__device__ __forceinline__ void load_tile(float* dst, const float* src, int r0, int end) {
#pragma unroll 4
  for (int i = threadIdx.x; i < kRows * D / 4; i += kThreads) {
    const int r = i / (D / 4), c = (i % (D / 4)) * 4;
    const float4 v = r0 + r < end ? load4(src + static_cast<size_t>(r0 + r) * D + c) : make_float4(0.f, 0.f, 0.f, 0.f);
    *reinterpret_cast<float4*>(dst + r * (D + 4) + c) = v;
  }
}

// The same tile in two steps: into registers, while the one before is used, and on to shared memory.
template <int D>
struct Ahead {
  static constexpr int kN = kT * D / 4 / kThreads;
  float4 v[kN];
  __device__ __forceinline__ void load(const float* src, int r0, int end) {
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      const int i = n * kThreads + threadIdx.x;
      const int r = r0 + i / (D / 4);
      v[n] = r < end ? load4(src + static_cast<size_t>(r) * D + (i % (D / 4)) * 4) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  __device__ __forceinline__ void store(float* dst) const {
#pragma unroll
    for (int n = 0; n < kN; ++n) {
      const int i = n * kThreads + threadIdx.x;
      *reinterpret_cast<float4*>(dst + i / (D / 4) * (D + 4) + (i % (D / 4)) * 4) = v[n];
    }
  }
};

// acc[i][j] = a[RA ty + i] . b[tx + 16 j]
template <int D, int RA, int RB>
__device__ __forceinline__ void dot_tile(float (&acc)[RA][RB], const float* a, const float* b, int ty, int tx) {
  float2 sum[RA][RB];
#pragma unroll
  for (int i = 0; i < RA; ++i)
#pragma unroll
    for (int j = 0; j < RB; ++j) sum[i][j] = make_float2(0.0f, 0.0f);
#pragma unroll 4
  for (int d = 0; d < D; d += 4) {
    float4 x[RA], y[RB];
#pragma unroll
    for (int i = 0; i < RA; ++i) x[i] = *reinterpret_cast<const float4*>(a + (RA * ty + i) * (D + 4) + d);
#pragma unroll
    for (int j = 0; j < RB; ++j) y[j] = *reinterpret_cast<const float4*>(b + (tx + 16 * j) * (D + 4) + d);
#pragma unroll
    for (int i = 0; i < RA; ++i)
#pragma unroll
      for (int j = 0; j < RB; ++j) {
        sum[i][j] = __ffma2_rn(make_float2(x[i].x, x[i].y), make_float2(y[j].x, y[j].y), sum[i][j]);
        sum[i][j] = __ffma2_rn(make_float2(x[i].z, x[i].w), make_float2(y[j].z, y[j].w), sum[i][j]);
      }
  }
#pragma unroll
  for (int i = 0; i < RA; ++i)
#pragma unroll
    for (int j = 0; j < RB; ++j) acc[i][j] = sum[i][j].x + sum[i][j].y;
}

// acc[i][2 c + e] += sum_t w[t][RO ty + i] * x[t][4 tx + 64 c + 2 e ..] (pairs of channels)
template <int D, int RO>
__device__ __forceinline__ void add_product(float2 (&acc)[RO][D / 32], const float* w, const float* x, int ty, int tx) {
#pragma unroll 4
  for (int t = 0; t < kT; ++t) {
    float a[RO];
#pragma unroll
    for (int i = 0; i < RO; i += 2) {
      const float2 p = *reinterpret_cast<const float2*>(w + t * (16 * RO + 4) + RO * ty + i);
      a[i] = p.x;
      a[i + 1] = p.y;
    }
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      const float4 b = *reinterpret_cast<const float4*>(x + t * (D + 4) + 4 * tx + 64 * c);
#pragma unroll
      for (int i = 0; i < RO; ++i) {
        acc[i][2 * c] = __ffma2_rn(make_float2(a[i], a[i]), make_float2(b.x, b.y), acc[i][2 * c]);
        acc[i][2 * c + 1] = __ffma2_rn(make_float2(a[i], a[i]), make_float2(b.z, b.w), acc[i][2 * c + 1]);
      }
    }
  }
}

template <int D, int RO>
__device__ __forceinline__ void store_tile(float* dst, const float2 (&acc)[RO][D / 32], float f, int own0, int own1, int ty, int tx) {
#pragma unroll
  for (int i = 0; i < RO; ++i) {
    const int r = own0 + RO * ty + i;
    if (r >= own1) continue;
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
      store4(dst + static_cast<size_t>(r) * D + 4 * tx + 64 * c,
             make_float4(acc[i][2 * c].x * f, acc[i][2 * c].y * f, acc[i][2 * c + 1].x * f, acc[i][2 * c + 1].y * f));
  }
}

// kDq: the block owns queries and streams keys; else it owns keys and streams queries.
template <int D, int kOwn, bool kDq>
__device__ __forceinline__ void fma_unit(const BwdParams& prm, int tile, float* smem) {
  using S = Smem<D, kOwn>;
  constexpr int RO = kOwn / 16;                      // own rows per thread
  constexpr int RA = kDq ? RO : kT / 16, RB = kDq ? kT / 16 : RO;
  float* sOwn0 = smem;                               // Q | K
  float* sOwn1 = sOwn0 + S::kOwnTile;                // dO | V
  float* sStr0 = sOwn1 + S::kOwnTile;                // K | Q
  float* sStr1 = sStr0 + S::kTile;                   // V | dO
  float* sP = sStr1 + S::kTile;                      // dS | P, by streamed row
  float* sdS = sP + S::kP;                           //      dS
  float* sLse = sdS + S::kP;
  float* sDelta = sLse + kT;
  const AttnTables& t = kDq ? prm.tq : prm.tk;
  const int bh = blockIdx.y;
  // A warp covers 4 x 8 of the 16 x 16 threads.
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int ty = (warp >> 1) * 4 + (lane >> 3), tx = (warp & 1) * 8 + (lane & 7);
  int g = 0;
  while (g + 1 < t.QG && t.tile_start[g + 1] <= tile) ++g;
  const int own0 = t.qg_row0[g] + (tile - t.tile_start[g]) * kOwn;
  const int own1 = min(own0 + kOwn, t.qg_row0[g + 1]);
  const size_t head = static_cast<size_t>(bh) * prm.N;
  const float* q = static_cast<const float*>(prm.q) + head * D;
  const float* k = static_cast<const float*>(prm.k) + head * D;
  const float* v = static_cast<const float*>(prm.v) + head * D;
  const float* dout = static_cast<const float*>(prm.dout) + head * D;
  // +inf makes every P of the row 0: rows outside the range, and rows without any key
  auto load_stats = [&](int r0, int r1, int n) {
    if (static_cast<int>(threadIdx.x) < n) {
      const int r = r0 + threadIdx.x;
      const float l = r < r1 ? prm.lse[head + r] : INFINITY;
      sLse[threadIdx.x] = l == -INFINITY ? INFINITY : l;
      sDelta[threadIdx.x] = r < r1 ? prm.delta[head + r] : 0.0f;
    }
  };
  load_tile<D, kOwn>(sOwn0, kDq ? q : k, own0, own1);
  load_tile<D, kOwn>(sOwn1, kDq ? dout : v, own0, own1);
  if (kDq) load_stats(own0, own1, kOwn);

  float2 acc0[RO][D / 32], acc1[RO][D / 32];         // dQ | dK, dV
#pragma unroll
  for (int i = 0; i < RO; ++i)
#pragma unroll
    for (int c = 0; c < D / 32; ++c) acc0[i][c] = acc1[i][c] = make_float2(0.0f, 0.0f);
  const float* str0 = kDq ? k : q;
  const float* str1 = kDq ? v : dout;
  int s0, s1;
  int p = next_range(t, g, 0, s0, s1);
  int st0 = s0;
  Ahead<D> ahead0, ahead1;
  if (st0 < s1) {
    ahead0.load(str0, st0, s1);
    ahead1.load(str1, st0, s1);
  }
  while (st0 < s1) {
    const int end = min(st0 + kT, s1);               // of this tile's rows
    __syncthreads();
    ahead0.store(sStr0);
    ahead1.store(sStr1);
    if (!kDq) load_stats(st0, end, kT);
    __syncthreads();
    const int n = end - st0;
    st0 += kT;
    if (st0 >= s1) {
      p = next_range(t, g, p, s0, s1);
      st0 = s0;
    }
    if (st0 < s1) {
      ahead0.load(str0, st0, s1);
      ahead1.load(str1, st0, s1);
    }
    // rows of s are queries, columns keys
    float s[RA][RB], dp[RA][RB];
    dot_tile<D, RA, RB>(s, kDq ? sOwn0 : sStr0, kDq ? sStr0 : sOwn0, ty, tx);
    dot_tile<D, RA, RB>(dp, kDq ? sOwn1 : sStr1, kDq ? sStr1 : sOwn1, ty, tx);
    const int q1 = kDq ? own1 - own0 : n, k1 = kDq ? n : own1 - own0;
#pragma unroll
    for (int i = 0; i < RA; ++i)
#pragma unroll
      for (int j = 0; j < RB; ++j) {
        const int r = RA * ty + i, c = tx + 16 * j;
        const bool in = r < q1 && c < k1;
        const float pij = in ? expf(fmaf(s[i][j], prm.scale, -sLse[r])) : 0.0f;
        const float ds = in ? pij * (dp[i][j] - sDelta[r]) : 0.0f;
        if (kDq) {
          sP[c * S::kPRow + r] = ds;
        } else {
          sP[r * S::kPRow + c] = pij;
          sdS[r * S::kPRow + c] = ds;
        }
      }
    __syncthreads();
    add_product<D, RO>(acc0, kDq ? sP : sdS, sStr0, ty, tx);
    if (!kDq) add_product<D, RO>(acc1, sP, sStr1, ty, tx);
  }
  store_tile<D, RO>(static_cast<float*>(kDq ? prm.dq : prm.dk) + head * D, acc0, prm.scale, own0, own1, ty, tx);
  if (!kDq) store_tile<D, RO>(static_cast<float*>(prm.dv) + head * D, acc1, 1.0f, own0, own1, ty, tx);
}

// One launch for both: the heavier blocks (dK, dV: four products) first.
template <int D, int kOwn>
__global__ void __launch_bounds__(kThreads, D == 64 ? 2 : 1) attn_bwd_fma_kernel(const __grid_constant__ BwdParams prm) {
  extern __shared__ __align__(16) float smem[];
  if (static_cast<int>(blockIdx.x) < prm.tiles_k)
    fma_unit<D, kOwn, false>(prm, blockIdx.x, smem);
  else
    fma_unit<D, kOwn, true>(prm, blockIdx.x - prm.tiles_k, smem);
}

template <int D, int kOwn>
int fma_impl(const BwdParams& prm, cudaStream_t st) {
  constexpr int smem = Smem<D, kOwn>::kBytes;
  cudaError_t e = cudaFuncSetAttribute(attn_bwd_fma_kernel<D, kOwn>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return static_cast<int>(e);
  attn_bwd_fma_kernel<D, kOwn><<<dim3(prm.tiles_k + prm.tiles_q, prm.BH), kThreads, smem, st>>>(prm);
  return static_cast<int>(cudaGetLastError());
}

template <typename T, int D>
int delta_impl(const void* o, const void* dout, const float* dlse, float* delta, long long rows, cudaStream_t st) {
  constexpr int kPerBlock = 256 * 16 / (D * static_cast<int>(sizeof(T)));
  delta_kernel<T, D><<<static_cast<unsigned>((rows + kPerBlock - 1) / kPerBlock), 256, 0, st>>>(
      static_cast<const T*>(o), static_cast<const T*>(dout), dlse, delta, rows);
  return static_cast<int>(cudaGetLastError());
}

}  // namespace

int launch_delta(const void* o, const void* dout, const float* dlse, float* delta, long long rows, int D, int dtype,
                 cudaStream_t st) {
  if (dtype == PA_BF16)
    return D == 64 ? delta_impl<__nv_bfloat16, 64>(o, dout, dlse, delta, rows, st)
                   : delta_impl<__nv_bfloat16, 128>(o, dout, dlse, delta, rows, st);
  return D == 64 ? delta_impl<float, 64>(o, dout, dlse, delta, rows, st)
                 : delta_impl<float, 128>(o, dout, dlse, delta, rows, st);
}

int launch_attn_bwd_fma(const BwdParams& prm, int own_rows, cudaStream_t st) {
  if (own_rows == 64) return prm.D == 64 ? fma_impl<64, 64>(prm, st) : fma_impl<128, 64>(prm, st);
  return prm.D == 64 ? fma_impl<64, 32>(prm, st) : fma_impl<128, 32>(prm, st);
}

}  // namespace pa
