// cache.cu -- the 8-bit K/V cache: e4m3 codes [B][Hk][M][D] with one scale per block of 64
// tokens and head, [B][Hk][ceil(M / 64)].
//
// A block's scale is the smallest power of two 2^e with amax <= 448 * 2^e (448 is the largest
// e4m3 value), e >= -126, and 0 for a block of zeros.  A power of two makes x / scale exact, so
// each code is one rounding (at most 2^-4 relative, half an e4m3 step), independent of how the
// division is done; and since e4m3 keeps its 3 mantissa bits at every exponent, a scale
// that is not amax / 448 itself costs no precision, only the unused top of the range.
//
// Storing rows behind a block's earlier tokens keeps the larger of the two scales.  If the
// scale grows, the older codes are rounded once more to the new one, which is exact unless they
// fall below e4m3's normal range.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "pa_device.cuh"
#include "pa_launch.h"

namespace pa {
namespace {

constexpr int kTok = PA_CACHE_BLOCK;
constexpr int kThreads = 256;
constexpr int kSeg = 8;               // channels per item: 16 (or 32) bytes in, 8 out

// An item's values as loaded; they are widened for the codes only, rather than held in fp32: twice
// the blocks fit an SM.
template <typename T>
struct Raw {
  static constexpr int kN = kSeg * sizeof(T) / 16;
  uint4 v[kN];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  }
  // The largest finite magnitude so far: one fp32, or one of the even and one of the odd bf16.
  // x 0 + x is NaN for infinities, and the maximum leaves NaN out: neither sets the scale
  // (infinities saturate, NaN stays NaN).
  __device__ __forceinline__ void largest(uint32_t& m) const {
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (sizeof(T) == 4) {
          const float x = fabsf(__uint_as_float(w[j]));
          m = __float_as_uint(fmaxf(__uint_as_float(m), fmaf(x, 0.0f, x)));
        } else {
          uint32_t x = w[j] & 0x7FFF7FFFu;
          asm("fma.rn.bf16x2 %0, %0, %1, %0;" : "+r"(x) : "r"(0u));
          asm("max.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(x));
        }
      }
    }
  }
  __device__ __forceinline__ void values(float2 (&x)[kSeg / 2]) const {
    if (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < kN; ++i) {
        x[2 * i] = make_float2(__uint_as_float(v[i].x), __uint_as_float(v[i].y));
        x[2 * i + 1] = make_float2(__uint_as_float(v[i].z), __uint_as_float(v[i].w));
      }
    } else {
      const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = make_float2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
    }
  }
};

// The larger of `m`'s magnitudes (one fp32 or two bf16) as an fp32 one.
template <typename T>
__device__ __forceinline__ float magnitude(uint32_t m) {
  return sizeof(T) == 4 ? __uint_as_float(m) : fmaxf(__uint_as_float(m & 0xFFFF0000u), __uint_as_float(m << 16));
}

// Smallest 2^e >= amax / 448 with e >= -126 (amax > 0, finite): 448 = 1.75 * 2^8.
__device__ __forceinline__ float block_scale(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = max(e, -126);                   // subnormal amax: u >> 23 is 0, below the limit anyway
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

__device__ __forceinline__ uint2 encode(const float2 (&x)[kSeg / 2], float inv) {
  const float2 inv2 = make_float2(inv, inv);
  uint32_t w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __nv_fp8x2_storage_t lo = __nv_cvt_float2_to_fp8x2(__fmul2_rn(x[2 * i], inv2), __NV_SATFINITE, __NV_E4M3);
    const __nv_fp8x2_storage_t hi = __nv_cvt_float2_to_fp8x2(__fmul2_rn(x[2 * i + 1], inv2), __NV_SATFINITE, __NV_E4M3);
    w[i] = static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
  }
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void decode(uint2 c, float2 (&x)[kSeg / 2]) {
  const uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t h[2];
    e4m3_to_f16(w[i], h[0], h[1]);
#pragma unroll
    for (int j = 0; j < 2; ++j) x[2 * i + j] = __half22float2(*reinterpret_cast<const __half2*>(&h[j]));
  }
}

// One block of threads per cache block that the new rows touch, for K or V of one head.  Bound
// by HBM: the rows are read once into registers, reduced, and written as codes.  5 heads x 75600
// bf16 rows, D = 128: 46 us, 6.3 TB/s; 24 x 4096: 12.8 us.  (A branch for infinities kept 32 registers
// from holding what it needs: 56 us.  Widening to fp32 before the maximum: 50 us.)
template <typename T, int D>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 8 : 5) cache_store_kernel(const __grid_constant__ CacheStoreParams prm) {
  constexpr int kSegs = D / kSeg;
  constexpr int kItems = kTok * kSegs / kThreads;      // (token, 8 channels) items per thread
  __shared__ float s_max[kThreads / 32];
  const int i = blockIdx.x % prm.touched;
  const int kv = (blockIdx.x / prm.touched) & 1;
  const int bh = blockIdx.x / prm.touched / 2;
  const int b = bh / prm.Hk;
  const int t0 = prm.start ? prm.start[b] : 0;
  if (t0 < 0 || t0 > prm.M - prm.T) {                  // the rows do not fit: leave the request's cache alone
    if (threadIdx.x == 0) record_status(prm.status, PA_EINVAL);
    return;
  }
  const int blk = t0 / kTok + i;
  const int tok0 = blk * kTok;
  if (tok0 >= t0 + prm.T) return;
  const T* src = static_cast<const T*>(kv ? prm.v : prm.k) + static_cast<size_t>(bh) * prm.T * D;
  uint8_t* codes = static_cast<uint8_t*>(kv ? prm.v_codes : prm.k_codes) + (static_cast<size_t>(bh) * prm.M + tok0) * D;
  float* scale = (kv ? prm.v_scale : prm.k_scale) + static_cast<size_t>(bh) * prm.blocks + blk;
  const float had = tok0 < t0 ? *scale : 0.0f;

  Raw<T> raw[kItems];
  uint32_t most = 0;
#pragma unroll
  for (int n = 0; n < kItems; ++n) {
    const int idx = n * kThreads + threadIdx.x;
    const int row = tok0 + idx / kSegs - t0;
    if (row >= 0 && row < prm.T) raw[n].load(src + static_cast<size_t>(row) * D + (idx % kSegs) * kSeg);
  }
#pragma unroll
  for (int n = 0; n < kItems; ++n) {
    const int row = tok0 + (n * kThreads + threadIdx.x) / kSegs - t0;
    if (row >= 0 && row < prm.T) raw[n].largest(most);
  }
  float amax = magnitude<T>(most);
  // non-negative floats compare as their bits do
  amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = amax;
  __syncthreads();                                     // also: every thread has read *scale
  amax = s_max[0];
#pragma unroll
  for (int w = 1; w < kThreads / 32; ++w) amax = fmaxf(amax, s_max[w]);
  const float need = amax > 0.0f ? block_scale(amax) : 0.0f;
  const float now = fmaxf(had, need);
  // 1 / now is a power of two too: exact, in range for every e in [-126, 120]
  const float inv = now > 0.0f ? 1.0f / now : 1.0f;
#pragma unroll
  for (int n = 0; n < kItems; ++n) {
    const int idx = n * kThreads + threadIdx.x;
    const int tok = idx / kSegs;
    const int row = tok0 + tok - t0;
    uint2* dst = reinterpret_cast<uint2*>(codes + static_cast<size_t>(tok) * D + (idx % kSegs) * kSeg);
    float2 x[kSeg / 2];
    if (row >= 0 && row < prm.T) {
      raw[n].values(x);
      *dst = encode(x, inv);
    } else if (row < 0 && now > had) {
      decode(*dst, x);
      *dst = encode(x, had * inv);
    }
  }
  if (threadIdx.x == 0) *scale = now;
}

template <typename T, int D>
int store_impl(const CacheStoreParams& prm, unsigned blocks, cudaStream_t st) {
  cache_store_kernel<T, D><<<blocks, kThreads, 0, st>>>(prm);
  return static_cast<int>(cudaGetLastError());
}

}  // namespace

int launch_cache_store(const CacheStoreParams& prm, unsigned blocks, int dtype, int D, cudaStream_t st) {
  if (dtype == PA_BF16)
    return D == 64 ? store_impl<__nv_bfloat16, 64>(prm, blocks, st) : store_impl<__nv_bfloat16, 128>(prm, blocks, st);
  return D == 64 ? store_impl<float, 64>(prm, blocks, st) : store_impl<float, 128>(prm, blocks, st);
}

}  // namespace pa
