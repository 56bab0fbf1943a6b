// cache_attn_rows.cu -- attention over the 8-bit K/V cache for few query rows per KV head (bf16
// queries: single tokens, a few tokens, heads that share a KV head).  Definition: cache_attn.cu.
//
// Bound by reading the codes once: 2 D bytes per (token, KV head).  Each warp streams tiles of 16
// tokens from global memory straight into registers, the next tile's loads in flight while the
// current one is multiplied, with its own running softmax; the block's four warps and then the
// splits are joined at the end, in a fixed order.  16 query rows (the m16n8k16 product's rows)
// cost the same as one, so a shared KV head is read once for all its query heads.
//
// Codes become product operands without shared memory because the inner index of a product may
// be permuted if both operands agree, and the outer one if the result is read accordingly:
//   S = Q K^T: lane (g, t) takes token g's bytes 16 t .. 16 t + 15 of each 64, four per k-step;
//     q is laid out the same way.  Codes go to f16, which holds every e4m3 value exactly; q is
//     scaled per row by a power of two so that its largest element is in [1, 2) and is exact in
//     f16 too, but for elements below 2^-14 of the largest (off by at most 2^-25 of it).  The
//     block's scale multiplies the fp32 score.
//   O += P V: lane (g, t) takes tokens 2t, 2t + 1, 2t + 8, 2t + 9 and channels g D/8 .. + D/8 - 1
//     of each.  Codes go to bf16 (exact); the weight times the block's scale is rounded to bf16
//     (2^-8), whose range holds any such product, so blocks of very different scales lose nothing.
#include <cuda_fp8.h>

#include "pa_device.cuh"
#include "pa_launch.h"

namespace pa {
namespace {

constexpr int kWarps = 4;
constexpr int kRowTile = 16;
constexpr int kTok = 16;               // tokens per tile; divides a cache block: one scale each
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleLog2 = 8.0f;   // move the running max only when it grows by more

__device__ __forceinline__ uint32_t f16_pair(uint32_t codes) {      // the two low bytes
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes & 0xFFFFu), __NV_E4M3);
  return static_cast<uint32_t>(h.x) | (static_cast<uint32_t>(h.y) << 16);
}

__device__ __forceinline__ uint32_t bf16_pair(uint32_t codes) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(codes & 0xFFFFu), __NV_E4M3);
  const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h));
  return pack_bf16x2(f.x, f.y);
}

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Streamed once: not kept in L1.
__device__ __forceinline__ uint4 load_codes16(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
__device__ __forceinline__ uint2 load_codes8(const uint8_t* p) {
  uint2 v;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
  return v;
}

// The codes of one tile of 16 tokens as one lane holds them.
template <int D>
struct Tile {
  uint32_t k[2][D / 16];          // tokens g and 8 + g: D / 4 bytes of each
  uint32_t v[4][D / 32];          // tokens 2t, 2t + 1, 2t + 8, 2t + 9: D / 8 bytes of each
  float ks, vs;

  // Tokens at or behind `end` are not read and become code 0.
  __device__ __forceinline__ void load(const uint8_t* kc, const uint8_t* vc, const float* k_scale, const float* v_scale,
                                       int tok, int end, int g, int t) {
    ks = __ldg(k_scale + tok / PA_CACHE_BLOCK);
    vs = __ldg(v_scale + tok / PA_CACHE_BLOCK);
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const int j = tok + 8 * n + g;
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        uint4 u = make_uint4(0u, 0u, 0u, 0u);
        if (j < end) u = load_codes16(kc + static_cast<size_t>(j) * D + c * 64 + t * 16);
        k[n][4 * c] = u.x; k[n][4 * c + 1] = u.y; k[n][4 * c + 2] = u.z; k[n][4 * c + 3] = u.w;
      }
    }
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      const int j = tok + 2 * t + (n & 1) + 8 * (n >> 1);
      if (D == 128) {
        uint4 u = make_uint4(0u, 0u, 0u, 0u);
        if (j < end) u = load_codes16(vc + static_cast<size_t>(j) * D + g * 16);
        v[n][0] = u.x; v[n][1] = u.y; v[n][D / 32 - 2] = u.z; v[n][D / 32 - 1] = u.w;
      } else {
        uint2 u = make_uint2(0u, 0u);
        if (j < end) u = load_codes8(vc + static_cast<size_t>(j) * D + g * 8);
        v[n][0] = u.x; v[n][1] = u.y;
      }
    }
  }
};

template <int D>
__global__ void __launch_bounds__(kWarps * 32, 2) cache_attn_rows_kernel(const __grid_constant__ CacheAttnParams prm) {
  constexpr int kSteps = D / 16;         // k-steps of S
  constexpr int kBlocks = D / 8;         // 8-channel blocks of O
  __shared__ float s_m[kWarps][kRowTile], s_l[kWarps][kRowTile];
  __shared__ __align__(16) float s_o[kWarps][kRowTile][D + 4];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int bh = blockIdx.y;
  const int split = blockIdx.x % prm.splits;
  const int row0 = blockIdx.x / prm.splits * kRowTile;
  // The request's own length is split evenly (whole cache blocks), so a short one costs little.
  const int len = cache_len(prm, bh / prm.Hk);
  const int chunk = split_chunk(len, prm.splits);
  const int begin = min(split * chunk, len), end = min(begin + chunk, len);
  const uint8_t* kc = prm.k_codes + static_cast<size_t>(bh) * prm.M * D;
  const uint8_t* vc = prm.v_codes + static_cast<size_t>(bh) * prm.M * D;
  const float* k_scale = prm.k_scale + static_cast<size_t>(bh) * prm.blocks;
  const float* v_scale = prm.v_scale + static_cast<size_t>(bh) * prm.blocks;

  int tok = begin + warp * kTok;
  Tile<D> cur, nxt;
  if (tok < end) cur.load(kc, vc, k_scale, v_scale, tok, end, g, t);

  // q in f16, laid out as the codes are; f = softmax scale * log2(e) / the row's power of two.
  uint32_t qa[kSteps][4];
  float f[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = row0 + g + 8 * h;
    float x[D / 4];
    float mx = 0.0f;
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint4 u = make_uint4(0u, 0u, 0u, 0u);
        if (r < prm.R)
          u = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(prm.q) +
                                                   (static_cast<size_t>(bh) * prm.R + r) * D + c * 64 + t * 16) + i);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[c * 16 + i * 8 + 2 * e] = __uint_as_float(w[e] << 16);
          x[c * 16 + i * 8 + 2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
        }
      }
#pragma unroll
    for (int i = 0; i < D / 4; ++i) mx = fmaxf(mx, fabsf(x[i]));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    // 2^e, e = exponent of the largest element, kept where 2^-e and 2^e are normal
    const int e = min(max(static_cast<int>(__float_as_uint(mx) >> 23), 2), 252) - 127;
    const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    f[h] = prm.scale * kLog2e * __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const __half2 p = __floats2half2_rn(x[4 * s + 2 * i] * down, x[4 * s + 2 * i + 1] * down);
        qa[s][2 * i + h] = *reinterpret_cast<const uint32_t*>(&p);
      }
  }

  float o[kBlocks][4];
#pragma unroll
  for (int i = 0; i < kBlocks; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.0f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
  while (tok < end) {
    const int next = tok + kWarps * kTok;
    if (next < end) nxt.load(kc, vc, k_scale, v_scale, next, end, g, t);
    float s[2][4] = {};
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int i = 0; i < kSteps; ++i) mma_f16(s[n], qa[i], f16_pair(cur.k[n][i]), f16_pair(cur.k[n][i] >> 16));
    // scores in log2 units: s[n][2 h + i] is row g + 8 h, token 8 n + 2 t + i
    const float fk[2] = {f[0] * cur.ks, f[1] * cur.ks};
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        s[n][i] = tok + 8 * n + 2 * t + (i & 1) < end ? s[n][i] * fk[i >> 1] : -INFINITY;
    float mt[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      mt[h] = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1]));
      mt[h] = fmaxf(mt[h], __shfl_xor_sync(0xffffffffu, mt[h], 1));
      mt[h] = fmaxf(mt[h], __shfl_xor_sync(0xffffffffu, mt[h], 2));
    }
    if (__any_sync(0xffffffffu, mt[0] > m[0] + kRescaleLog2 || mt[1] > m[1] + kRescaleLog2)) {
      float a[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {        // only rows whose own max grew: a row never depends on its neighbours
        const float to = mt[h] > m[h] + kRescaleLog2 ? mt[h] : m[h];
        a[h] = to > m[h] ? fast_exp2(m[h] - to) : 1.0f;
        m[h] = to;
        l[h] *= a[h];
      }
#pragma unroll
      for (int i = 0; i < kBlocks; ++i) {
        o[i][0] *= a[0];
        o[i][1] *= a[0];
        o[i][2] *= a[1];
        o[i][3] *= a[1];
      }
    }
    uint32_t pa[4];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float p0 = fast_exp2(s[n][2 * h] - m[h]), p1 = fast_exp2(s[n][2 * h + 1] - m[h]);
        l[h] += p0 + p1;
        pa[2 * n + h] = pack_bf16x2(p0 * cur.vs, p1 * cur.vs);
      }
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
      // bytes b of two tokens side by side: channels 4 w + {0, 1} and + {2, 3}
      const uint32_t lo01 = __byte_perm(cur.v[0][w], cur.v[1][w], 0x5140), lo23 = __byte_perm(cur.v[0][w], cur.v[1][w], 0x7362);
      const uint32_t hi01 = __byte_perm(cur.v[2][w], cur.v[3][w], 0x5140), hi23 = __byte_perm(cur.v[2][w], cur.v[3][w], 0x7362);
      mma_bf16(o[4 * w], pa, bf16_pair(lo01), bf16_pair(hi01));
      mma_bf16(o[4 * w + 1], pa, bf16_pair(lo01 >> 16), bf16_pair(hi01 >> 16));
      mma_bf16(o[4 * w + 2], pa, bf16_pair(lo23), bf16_pair(hi23));
      mma_bf16(o[4 * w + 3], pa, bf16_pair(lo23 >> 16), bf16_pair(hi23 >> 16));
    }
    cur = nxt;
    tok = next;
  }

  // Join the warps.  o[i][2 h + e] is row g + 8 h, channel (2 t + e) * D/8 + i.
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    if (t == 0) {
      s_m[warp][g + 8 * h] = m[h];
      s_l[warp][g + 8 * h] = l[h];
    }
#pragma unroll
    for (int e = 0; e < 2; ++e)
#pragma unroll
      for (int i = 0; i < kBlocks; i += 4)
        *reinterpret_cast<float4*>(&s_o[warp][g + 8 * h][(2 * t + e) * kBlocks + i]) =
            make_float4(o[i][2 * h + e], o[i + 1][2 * h + e], o[i + 2][2 * h + e], o[i + 3][2 * h + e]);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kRowTile * D / 4; i += kWarps * 32) {
    const int r = i / (D / 4), c = (i % (D / 4)) * 4;
    if (row0 + r >= prm.R) continue;
    float mx = s_m[0][r];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) mx = fmaxf(mx, s_m[w][r]);
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float a = mx > -INFINITY ? fast_exp2(s_m[w][r] - mx) : 0.0f;    // 0 for a warp without tokens
      const float4 x = *reinterpret_cast<const float4*>(&s_o[w][r][c]);
      sum = fmaf(a, s_l[w][r], sum);
      acc.x = fmaf(a, x.x, acc.x);
      acc.y = fmaf(a, x.y, acc.y);
      acc.z = fmaf(a, x.z, acc.z);
      acc.w = fmaf(a, x.w, acc.w);
    }
    const float inv = end > begin ? 1.0f / sum : 0.0f;
    acc = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    const size_t at = (prm.splits > 1 ? static_cast<size_t>(split) * prm.rows : 0) + static_cast<size_t>(bh) * prm.R + row0 + r;
    if (prm.splits > 1)
      store4(prm.ws_o + at * D + c, acc);
    else
      store4(static_cast<__nv_bfloat16*>(prm.o) + at * D + c, acc);
    if (c == 0) (prm.splits > 1 ? prm.ws_lse : prm.lse)[at] = end > begin ? (mx + fast_log2(sum)) * kLn2 : -INFINITY;
  }
}

}  // namespace

int cache_attn_rows_tile_rows() { return kRowTile; }

int launch_cache_attn_rows(const CacheAttnParams& prm, cudaStream_t st) {
  const dim3 grid((prm.R + kRowTile - 1) / kRowTile * prm.splits, prm.B * prm.Hk);
  if (prm.D == 64)
    cache_attn_rows_kernel<64><<<grid, kWarps * 32, 0, st>>>(prm);
  else
    cache_attn_rows_kernel<128><<<grid, kWarps * 32, 0, st>>>(prm);
  return static_cast<int>(cudaGetLastError());
}

}  // namespace pa
