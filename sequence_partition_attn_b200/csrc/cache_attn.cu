// cache_attn.cu -- attention over the 8-bit K/V cache: the kernel on the FMA units (fp32
// queries) and the join of splits.
//
// For each request b, KV head and the R = (H / Hk) * Nq query rows that share it:
//   lse_i = ln sum_{j < lens[b]} exp(scale q_i . k_j),  o_i = sum_j exp(s_ij - lse_i) v_j,
// k_j = code * scale of its 64-token block.  Consecutive query heads share a KV head, so the
// R rows are contiguous in q and o.  The token axis may be split over blocks ("splits"); each
// writes its own state in fp32 and the join adds them in split order, so results do not depend
// on the order in which blocks run.
#include <cuda_fp8.h>

#include "pa_device.cuh"
#include "pa_launch.h"

namespace pa {
namespace {

constexpr int kRows = 64;
constexpr int kKeys = 32;             // divides a cache block: one scale per tile

// 4 codes times the block's scale.
__device__ __forceinline__ float4 decode4(uint32_t c, float scale) {
  const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c & 0xFFFFu), __NV_E4M3);
  const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(c >> 16), __NV_E4M3);
  const float2 a = __half22float2(*reinterpret_cast<const __half2*>(&lo));
  const float2 b = __half22float2(*reinterpret_cast<const __half2*>(&hi));
  return make_float4(a.x * scale, a.y * scale, b.x * scale, b.y * scale);
}

// 64 query rows per block, D / 64 threads per row (64 channels each); keys stream through
// shared memory with an online softmax, as in the fp32 partition attention.
template <int D>
__global__ void __launch_bounds__(kRows * (D / 64)) cache_attn_f32_kernel(const __grid_constant__ CacheAttnParams prm) {
  constexpr int TPR = D / 64;
  __shared__ __align__(16) float sK[kKeys][D];
  __shared__ __align__(16) float sV[kKeys][D];
  const int bh = blockIdx.y;
  const int split = blockIdx.z;
  const int len = cache_len(prm, bh / prm.Hk);
  const int chunk = split_chunk(len, prm.splits);
  const int k0 = min(split * chunk, len), k1 = min(k0 + chunk, len);
  const int row = blockIdx.x * kRows + threadIdx.x / TPR;
  const int half = threadIdx.x % TPR;
  const bool row_ok = row < prm.R;
  const size_t out_row = static_cast<size_t>(bh) * prm.R + row;
  const uint8_t* kc = prm.k_codes + static_cast<size_t>(bh) * prm.M * D;
  const uint8_t* vc = prm.v_codes + static_cast<size_t>(bh) * prm.M * D;
  const float* ks = prm.k_scale + static_cast<size_t>(bh) * prm.blocks;
  const float* vs = prm.v_scale + static_cast<size_t>(bh) * prm.blocks;

  float q[64], o[64];
  const float* qp = static_cast<const float*>(prm.q) + (row_ok ? out_row : static_cast<size_t>(bh) * prm.R) * D + half * 64;
#pragma unroll
  for (int d = 0; d < 64; d += 4) {
    const float4 v = load4(qp + d);
    q[d] = v.x; q[d + 1] = v.y; q[d + 2] = v.z; q[d + 3] = v.w;
  }
#pragma unroll
  for (int d = 0; d < 64; ++d) o[d] = 0.0f;
  float m = -INFINITY, l = 0.0f;
  for (int key0 = k0; key0 < k1; key0 += kKeys) {
    __syncthreads();
    const float sk = ks[key0 / PA_CACHE_BLOCK], sv = vs[key0 / PA_CACHE_BLOCK];
    for (int idx = threadIdx.x; idx < kKeys * D / 4; idx += blockDim.x) {
      const int j = idx / (D / 4), c = (idx % (D / 4)) * 4;
      float4 kv = make_float4(0.f, 0.f, 0.f, 0.f), vv = kv;
      if (key0 + j < k1) {
        kv = decode4(*reinterpret_cast<const uint32_t*>(kc + static_cast<size_t>(key0 + j) * D + c), sk);
        vv = decode4(*reinterpret_cast<const uint32_t*>(vc + static_cast<size_t>(key0 + j) * D + c), sv);
      }
      *reinterpret_cast<float4*>(&sK[j][c]) = kv;
      *reinterpret_cast<float4*>(&sV[j][c]) = vv;
    }
    __syncthreads();
    float s[kKeys];
    float mt = -INFINITY;
#pragma unroll
    for (int j = 0; j < kKeys; ++j) {
      float acc = 0.0f;
#pragma unroll
      for (int d = 0; d < 64; d += 4) {
        const float4 kv = *reinterpret_cast<const float4*>(&sK[j][half * 64 + d]);
        acc = fmaf(q[d], kv.x, acc);
        acc = fmaf(q[d + 1], kv.y, acc);
        acc = fmaf(q[d + 2], kv.z, acc);
        acc = fmaf(q[d + 3], kv.w, acc);
      }
      if (TPR == 2) acc += __shfl_xor_sync(0xffffffffu, acc, 1);
      s[j] = key0 + j < k1 ? acc * prm.scale : -INFINITY;
      mt = fmaxf(mt, s[j]);
    }
    const float m_new = fmaxf(m, mt);
    const float alpha = expf(m - m_new);     // 0 on the first tile (m = -inf)
    l *= alpha;
#pragma unroll
    for (int d = 0; d < 64; ++d) o[d] *= alpha;
#pragma unroll
    for (int j = 0; j < kKeys; ++j) {
      const float pj = expf(s[j] - m_new);
      l += pj;
#pragma unroll
      for (int d = 0; d < 64; d += 4) {
        const float4 vv = *reinterpret_cast<const float4*>(&sV[j][half * 64 + d]);
        o[d] = fmaf(pj, vv.x, o[d]);
        o[d + 1] = fmaf(pj, vv.y, o[d + 1]);
        o[d + 2] = fmaf(pj, vv.z, o[d + 2]);
        o[d + 3] = fmaf(pj, vv.w, o[d + 3]);
      }
    }
    m = m_new;
  }
  if (!row_ok) return;
  const float inv = k1 > k0 ? 1.0f / l : 0.0f;       // no key: o = 0, lse = -inf
  const size_t at = prm.splits > 1 ? static_cast<size_t>(split) * prm.rows + out_row : out_row;
#pragma unroll
  for (int d = 0; d < 64; d += 4) {
    const float4 x = make_float4(o[d] * inv, o[d + 1] * inv, o[d + 2] * inv, o[d + 3] * inv);
    if (prm.splits > 1)
      store4(prm.ws_o + at * D + half * 64 + d, x);
    else
      store4(static_cast<float*>(prm.o) + at * D + half * 64 + d, x);
  }
  if (half == 0) (prm.splits > 1 ? prm.ws_lse : prm.lse)[at] = k1 > k0 ? m + logf(l) : -INFINITY;
}

// Join of the splits' states: D / 4 threads per row, four channels each.
template <typename T, int D>
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
  store4(static_cast<T*>(prm.o) + static_cast<size_t>(row) * D + 4 * c, acc);
  if (c == 0) prm.lse[row] = sum == 0.0f ? -INFINITY : m + logf(sum);
}

template <typename T, int D>
int join_impl(const CacheAttnParams& prm, cudaStream_t st) {
  constexpr int kPerBlock = 128 / (D / 4);
  cache_join_kernel<T, D><<<static_cast<unsigned>((prm.rows + kPerBlock - 1) / kPerBlock), 128, 0, st>>>(prm);
  return static_cast<int>(cudaGetLastError());
}

}  // namespace

int cache_attn_f32_tile_rows() { return kRows; }

int launch_cache_attn_f32(const CacheAttnParams& prm, cudaStream_t st) {
  const dim3 grid((prm.R + kRows - 1) / kRows, prm.B * prm.Hk, prm.splits);
  if (prm.D == 64)
    cache_attn_f32_kernel<64><<<grid, kRows, 0, st>>>(prm);
  else
    cache_attn_f32_kernel<128><<<grid, kRows * 2, 0, st>>>(prm);
  return static_cast<int>(cudaGetLastError());
}

int launch_cache_join(const CacheAttnParams& prm, int dtype, cudaStream_t st) {
  if (dtype == PA_BF16) return prm.D == 64 ? join_impl<__nv_bfloat16, 64>(prm, st) : join_impl<__nv_bfloat16, 128>(prm, st);
  return prm.D == 64 ? join_impl<float, 64>(prm, st) : join_impl<float, 128>(prm, st);
}

}  // namespace pa
