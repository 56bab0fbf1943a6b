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
constexpr int kT = 64;               // rows and keys per tile
constexpr int kThreads = 256;        // 16 x 16: four rows by four keys each

template <int D>
struct Smem {
  static constexpr int kRow = D + 4;     // 16-byte reads of 8 rows then fall in different banks
  static constexpr int kPRow = kT + 4;
  static constexpr int kTile = kT * kRow;
  static constexpr int kP = kT * kPRow;
  static constexpr int kBytes = (4 * kTile + 2 * kP + 2 * kT) * 4;
};

// Rows [r0, r0 + 64) of a [.., D] tensor into shared memory; rows at or past `end` read as 0,
// so that nothing outside the range (which may be non-finite) reaches a product.
template <int D>
__device__ __forceinline__ void load_tile(float* dst, const float* src, int r0, int end) {
  for (int i = threadIdx.x; i < kT * D / 4; i += kThreads) {
    const int r = i / (D / 4), c = (i % (D / 4)) * 4;
    const float4 v = r0 + r < end ? load4(src + static_cast<size_t>(r0 + r) * D + c) : make_float4(0.f, 0.f, 0.f, 0.f);
    *reinterpret_cast<float4*>(dst + r * Smem<D>::kRow + c) = v;
  }
}

// acc[i][j] = a[4 ty + i] . b[tx + 16 j]
template <int D>
__device__ __forceinline__ void dot_tile(float (&acc)[4][4], const float* a, const float* b, int ty, int tx) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.0f;
#pragma unroll 4
  for (int d = 0; d < D; d += 4) {
    float4 x[4], y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const float4*>(a + (4 * ty + i) * Smem<D>::kRow + d);
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = *reinterpret_cast<const float4*>(b + (tx + 16 * j) * Smem<D>::kRow + d);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[i][j] = fmaf(x[i].x, y[j].x, acc[i][j]);
        acc[i][j] = fmaf(x[i].y, y[j].y, acc[i][j]);
        acc[i][j] = fmaf(x[i].z, y[j].z, acc[i][j]);
        acc[i][j] = fmaf(x[i].w, y[j].w, acc[i][j]);
      }
  }
}

// acc[i][c] += sum_t w[t][4 ty + i] * x[t][4 tx + 64 (c / 4) + c % 4]
template <int D>
__device__ __forceinline__ void add_product(float (&acc)[4][D / 16], const float* w, const float* x, int ty, int tx) {
#pragma unroll 4
  for (int t = 0; t < kT; ++t) {
    const float4 a = *reinterpret_cast<const float4*>(w + t * Smem<D>::kPRow + 4 * ty);
    const float av[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      const float4 b = *reinterpret_cast<const float4*>(x + t * Smem<D>::kRow + 4 * tx + 64 * c);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        acc[i][4 * c] = fmaf(av[i], b.x, acc[i][4 * c]);
        acc[i][4 * c + 1] = fmaf(av[i], b.y, acc[i][4 * c + 1]);
        acc[i][4 * c + 2] = fmaf(av[i], b.z, acc[i][4 * c + 2]);
        acc[i][4 * c + 3] = fmaf(av[i], b.w, acc[i][4 * c + 3]);
      }
    }
  }
}

// kDq: the block owns 64 query rows and streams keys; else it owns 64 keys and streams queries.
// Four rows by four keys per thread: 8 shared 16-byte reads per 64 multiply-adds, which is what
// bounds it (shared memory reads at twice the rate the FMA pipe would need).
template <int D, bool kDq>
__global__ void __launch_bounds__(kThreads) attn_bwd_fma_kernel(const __grid_constant__ BwdParams prm) {
  extern __shared__ __align__(16) float smem[];
  float* sQ = smem;
  float* sdO = sQ + Smem<D>::kTile;
  float* sK = sdO + Smem<D>::kTile;
  float* sV = sK + Smem<D>::kTile;
  float* sP = sV + Smem<D>::kTile;         // dS^T [key][row] for dQ; P [row][key] for dV
  float* sdS = sP + Smem<D>::kP;           // dS [row][key] for dK
  float* sLse = sdS + Smem<D>::kP;
  float* sDelta = sLse + kT;
  const AttnTables& t = kDq ? prm.tq : prm.tk;
  const int bh = blockIdx.y;
  const int ty = threadIdx.x / 16, tx = threadIdx.x % 16;
  int g = 0;
  while (g + 1 < t.QG && t.tile_start[g + 1] <= static_cast<int>(blockIdx.x)) ++g;
  const int own0 = t.qg_row0[g] + (blockIdx.x - t.tile_start[g]) * kT;
  const int own1 = min(own0 + kT, t.qg_row0[g + 1]);
  const size_t head = static_cast<size_t>(bh) * prm.N;
  const float* q = static_cast<const float*>(prm.q) + head * D;
  const float* k = static_cast<const float*>(prm.k) + head * D;
  const float* v = static_cast<const float*>(prm.v) + head * D;
  const float* dout = static_cast<const float*>(prm.dout) + head * D;

  float acc0[4][D / 16] = {}, acc1[4][D / 16] = {};      // dQ | dK, dV
  for (int p = 0; p < t.P;) {
    int s0, s1;
    p = next_range(t, g, p, s0, s1);
    for (int st0 = s0; st0 < s1; st0 += kT) {
      const int q0 = kDq ? own0 : st0, q1 = kDq ? own1 : s1;
      const int k0 = kDq ? st0 : own0, k1 = kDq ? s1 : own1;
      __syncthreads();
      load_tile<D>(sQ, q, q0, q1);
      load_tile<D>(sdO, dout, q0, q1);
      load_tile<D>(sK, k, k0, k1);
      load_tile<D>(sV, v, k0, k1);
      if (threadIdx.x < kT) {
        const int r = q0 + threadIdx.x;
        // +inf makes every P of the row 0: rows outside the range, and rows without any key
        const float l = r < q1 ? prm.lse[head + r] : INFINITY;
        sLse[threadIdx.x] = l == -INFINITY ? INFINITY : l;
        sDelta[threadIdx.x] = r < q1 ? prm.delta[head + r] : 0.0f;
      }
      __syncthreads();
      float s[4][4], dp[4][4];
      dot_tile<D>(s, sQ, sK, ty, tx);
      dot_tile<D>(dp, sdO, sV, ty, tx);
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = 4 * ty + i, c = tx + 16 * j;
          const bool in = q0 + r < q1 && k0 + c < k1;
          const float pij = in ? expf(fmaf(s[i][j], prm.scale, -sLse[r])) : 0.0f;
          const float ds = in ? pij * (dp[i][j] - sDelta[r]) : 0.0f;
          if (kDq) {
            sP[c * Smem<D>::kPRow + r] = ds;
          } else {
            sP[r * Smem<D>::kPRow + c] = pij;
            sdS[r * Smem<D>::kPRow + c] = ds;
          }
        }
      __syncthreads();
      if (kDq) {
        add_product<D>(acc0, sP, sK, ty, tx);
      } else {
        add_product<D>(acc0, sdS, sQ, ty, tx);
        add_product<D>(acc1, sP, sdO, ty, tx);
      }
    }
  }
  float* out0 = static_cast<float*>(kDq ? prm.dq : prm.dk) + head * D;
  float* out1 = static_cast<float*>(prm.dv) + head * D;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = own0 + 4 * ty + i;
    if (r >= own1) continue;
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      const size_t at = static_cast<size_t>(r) * D + 4 * tx + 64 * c;
      store4(out0 + at, make_float4(acc0[i][4 * c] * prm.scale, acc0[i][4 * c + 1] * prm.scale,
                                    acc0[i][4 * c + 2] * prm.scale, acc0[i][4 * c + 3] * prm.scale));
      if (!kDq)
        store4(out1 + at, make_float4(acc1[i][4 * c], acc1[i][4 * c + 1], acc1[i][4 * c + 2], acc1[i][4 * c + 3]));
    }
  }
}

template <int D>
int fma_impl(const BwdParams& prm, cudaStream_t st) {
  constexpr int smem = Smem<D>::kBytes;
  cudaError_t e = cudaFuncSetAttribute(attn_bwd_fma_kernel<D, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(attn_bwd_fma_kernel<D, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return static_cast<int>(e);
  attn_bwd_fma_kernel<D, false><<<dim3(prm.tiles_k, prm.BH), kThreads, smem, st>>>(prm);
  attn_bwd_fma_kernel<D, true><<<dim3(prm.tiles_q, prm.BH), kThreads, smem, st>>>(prm);
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

int attn_bwd_fma_tile_rows() { return kT; }

int launch_delta(const void* o, const void* dout, const float* dlse, float* delta, long long rows, int D, int dtype,
                 cudaStream_t st) {
  if (dtype == PA_BF16)
    return D == 64 ? delta_impl<__nv_bfloat16, 64>(o, dout, dlse, delta, rows, st)
                   : delta_impl<__nv_bfloat16, 128>(o, dout, dlse, delta, rows, st);
  return D == 64 ? delta_impl<float, 64>(o, dout, dlse, delta, rows, st)
                 : delta_impl<float, 128>(o, dout, dlse, delta, rows, st);
}

int launch_attn_bwd_fma(const BwdParams& prm, cudaStream_t st) {
  return prm.D == 64 ? fma_impl<64>(prm, st) : fma_impl<128>(prm, st);
}

}  // namespace pa
